"""include/moe_ckpt8.h on the host: every declared symbol is exported, bad arguments
are refused before any HIP call (no call here reaches a launch), the stage refuses
what the kernels would read wrongly, and the backward's definition is the
derivative of the forward's."""
import ctypes
import os
import re

import pytest
import torch

from oracle import i8 as Q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced
ODD = ctypes.c_void_p(0x1008)   # not 16-byte aligned
OK, EINVAL, EUNSUPPORTED, EWORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def B():
    from mixture_experts_expert_amd import binding
    return binding


def test_every_declared_symbol_is_exported(B):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_ckpt8.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))
    assert len(names) >= 6, names
    for n in names:
        assert hasattr(B.lib, n) and n in B._SIGS, n


def _with(args, at, value):
    args = list(args)
    args[at] = value
    return args


@pytest.mark.parametrize("name", ["moe_quantize_ckpt8", "moe_dequantize_ckpt8"])
def test_rows(B, name):
    fn = getattr(B.lib, name)
    for rows, K, code in ((-1, 64, EINVAL), (4, 0, EINVAL), (4, 12, EINVAL), ((1 << 29) - 32, 64, EUNSUPPORTED),
                          (1 << 28, 128, EUNSUPPORTED), (1 << 30, 1 << 30, EUNSUPPORTED)):
        assert fn(rows, K, FAKE, FAKE, FAKE, None) == code
    assert fn(0, 64, None, None, None, None) == OK
    for i in range(3):
        assert fn(4, 64, *_with([FAKE] * 3, i, None), None) == EINVAL
    for i in ((0, 1) if name == "moe_quantize_ckpt8" else (0, 2)):
        assert fn(4, 64, *_with([FAKE] * 3, i, ODD), None) == EINVAL


SHAPES = [((0, 64, 4, 2, 64, "bf16"), EINVAL), ((8, 64, 4, 5, 64, "bf16"), EINVAL), ((8, 64, 2000, 2, 64, "bf16"), EINVAL),
          ((8, 96, 4, 2, 64, "bf16"), EUNSUPPORTED), ((8, 64, 4, 2, 48, "bf16"), EUNSUPPORTED),
          ((8, 64, 4, 2, 64, "f32"), EUNSUPPORTED), ((1 << 24, 64, 4, 2, 64, "bf16"), EUNSUPPORTED)]


@pytest.mark.parametrize("name,n,tail", [("moe_gemm_gate_up_ckpt8", 10, [None]),
                                         ("moe_gemm_down_dgrad_ckpt8", 14, [1 << 40, None])])
def test_a_weight_and_a_tiles_rows_have_less_than_2_gib(B, name, n, tail):
    for H, I, code in ((1 << 15, 1 << 15, EUNSUPPORTED), (64, 1 << 24, EUNSUPPORTED), (64, 1 << 22, EUNSUPPORTED),
                       (1 << 22, 64, EUNSUPPORTED)):
        assert getattr(B.lib, name)(B.shape(1, H, 1, 1, I, "bf16"), *[FAKE] * n, *tail) == code


@pytest.mark.parametrize("name,n,optional,aligned", [
    ("moe_gemm_gate_up_ckpt8", 10, 1, (0, 3, 4, 5, 7, 9)), ("moe_gemm_down_dgrad_ckpt8", 14, None, (0, 5, 6, 8, 10, 11, 13)),
    ("moe_gemm_down_wgrad_dy", 5, None, (0, 2, 4))])
def test_products(B, name, n, optional, aligned):
    tail = {"moe_gemm_gate_up_ckpt8": [None], "moe_gemm_down_dgrad_ckpt8": [1 << 40, None],
            "moe_gemm_down_wgrad_dy": [0, FAKE, 1 << 40, None]}[name]
    call = lambda dims, args, tail=tail: getattr(B.lib, name)(B.shape(*dims), *args, *tail)
    for dims, code in SHAPES:
        assert call(dims, [FAKE] * n) == code, dims
    good = (8, 64, 4, 2, 64, "bf16")
    for i in range(n):
        if i != optional:
            assert call(good, _with([FAKE] * n, i, None)) == EINVAL, i
    for i in aligned:
        assert call(good, _with([FAKE] * n, i, ODD)) == EINVAL, i
    if name == "moe_gemm_down_dgrad_ckpt8":
        need = B.moe_ckpt8_workspace_bytes(B.shape(*good))
        assert 0 < need <= B.moe_workspace_bytes(B.shape(*good))
        assert call(good, [FAKE] * n, [need - 1, None]) == EWORKSPACE
    if name == "moe_gemm_down_wgrad_dy":
        assert call(good, [FAKE] * n, [2, FAKE, 1 << 40, None]) == EINVAL
        assert call(good, [FAKE] * n, [0, None, 1 << 40, None]) == EINVAL
        assert call(good, [FAKE] * n, [0, FAKE, 16, None]) == EWORKSPACE


def test_stage_refusals(B):
    st = B.Ckpt8Stage(8, 128, 4, 2, 64, device="cpu")  # buffers only
    z = lambda *d, dt=torch.bfloat16: torch.zeros(*d, dtype=dt)
    w = (z(4, 128), z(4, 64, 128), z(4, 64, 128), z(4, 128, 64))
    for x in (z(8, 128), z(7, 128), z(8, 128, dt=torch.float32), z(8, 256)[:, ::2], z(128, 8).T):
        with pytest.raises(ValueError):
            st.forward(x, *w)
        with pytest.raises(ValueError):
            st.backward(x)
    with pytest.raises(B.MoEError):
        B.Ckpt8Stage(8, 100, 4, 2, 64, device="cpu")
    scratch = {}
    B.Ckpt8Stage(8, 128, 4, 2, 64, device="cpu", scratch=scratch)
    B.Ckpt8Stage(8, 128, 4, 2, 64, device="cpu", scratch=scratch, x8=True)
    with pytest.raises(ValueError):
        B.Ckpt8Stage(8, 128, 4, 2, 128, device="cpu", scratch=scratch)
    # 2 I (1 + 4/64) bytes a row for g and u, and the sort's four words, where bf16 keeps 6 I + 2 H
    big = B.Ckpt8Stage(256, 2048, 8, 8, 768, device="cpu")
    M = 256 * 8
    assert big.kept_bytes() == M * (2 * 768 * 17 // 16 + 4 * 4 + 8) + 4 * 9
    assert big.kept_bytes() < M * (6 * 768 + 2 * 2048) / 5


def test_stage_refuses_weights_of_other_sizes_and_types(B):
    st = B.Ckpt8Stage(8, 128, 4, 2, 64, device="cpu")
    z = lambda *d, dt=torch.bfloat16: torch.zeros(*d, dtype=dt)
    good = {"x": z(8, 128), "w_router": z(4, 128), "w_gate": z(4, 64, 128), "w_up": z(4, 64, 128), "w_down": z(4, 128, 64),
            "logit_bias": z(4, dt=torch.float32)}
    for name, t in good.items():
        other = torch.bfloat16 if name == "logit_bias" else torch.float32
        for bad in (t.to(other), t[:-1], t.unsqueeze(0), torch.stack((t, t), -1)[..., 0]):
            with pytest.raises(ValueError, match=name + " has to be"):
                st.forward(**{**good, name: bad})
    with pytest.raises(ValueError, match="on one GPU"):
        st.forward(**good)


def test_backward_is_the_derivative():
    """Central differences of f = sum over rows of w <dy[t], a W_down^T> in g, u and w."""
    g = torch.Generator().manual_seed(1)
    r = lambda *d: torch.randn(*d, generator=g, dtype=torch.float64)
    dy, wd, gv, uv, w = r(3, 4), r(2, 4, 6), r(5, 6), r(5, 6), r(5)
    tok, off = torch.tensor([0, 2, 1, 1, 0]), [0, 2, 5]

    def f(gv, uv, w):
        a = gv * torch.sigmoid(gv) * uv
        o = torch.cat([a[:2] @ wd[0].T, a[2:] @ wd[1].T])
        return (w[:, None] * dy[tok] * o).sum()

    dgu, a_w, dot = Q.down_backward(dy, tok, w, off, wd, gv, uv)
    h = 1e-5
    for p in range(5):
        e = torch.zeros(5, dtype=torch.float64)
        e[p] = h
        assert abs((f(gv, uv, w + e) - f(gv, uv, w - e)) / (2 * h) - dot[p]) < 1e-8
        for i in range(6):
            d = torch.zeros(5, 6, dtype=torch.float64)
            d[p, i] = h
            assert abs((f(gv + d, uv, w) - f(gv - d, uv, w)) / (2 * h) - dgu[p, i]) < 1e-8
            assert abs((f(gv, uv + d, w) - f(gv, uv - d, w)) / (2 * h) - dgu[p, 6 + i]) < 1e-8
    assert torch.allclose(a_w, w[:, None] * gv * torch.sigmoid(gv) * uv)
