"""include/moe_i8.h on the host: every declared symbol is exported, and bad
arguments are refused before any HIP call (no call here reaches a launch)."""
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
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_i8.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))
    assert len(names) >= 7, names
    for n in names:
        assert hasattr(B.lib, n) and n in B._SIGS, n


def _with(args, at, value):
    args = list(args)
    args[at] = value
    return args


@pytest.mark.parametrize("rows,K,code", [
    (-1, 64, EINVAL), (4, 0, EINVAL), (4, 12, EINVAL), (0, 64, OK), (1 << 28, 64, EUNSUPPORTED),
    ((1 << 28) - 16, 512, EUNSUPPORTED), (1 << 26, 520, EUNSUPPORTED), (1 << 24, 2056, EUNSUPPORTED)])
def test_quantize_rows(B, rows, K, code):
    assert B.lib.moe_quantize_i8_rows(rows, K, FAKE, FAKE, FAKE, None) == code


def test_quantize_rows_pointers(B):
    for i in range(3):
        assert B.lib.moe_quantize_i8_rows(4, 64, *_with([FAKE] * 3, i, None), None) == EINVAL
    for i in range(2):
        assert B.lib.moe_quantize_i8_rows(4, 64, *_with([FAKE] * 3, i, ODD), None) == EINVAL
    assert B.lib.moe_quantize_i8_rows(0, 64, None, None, None, None) == OK


GEMM = [FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE]  # aq, a_scale, offsets, wq, w_scale, row_weight, out


@pytest.mark.parametrize("M,E,N,K,code", [
    (-1, 2, 64, 64, EINVAL), (8, 0, 64, 64, EINVAL), (8, 2, 0, 64, EINVAL), (8, 2, 64, 0, EINVAL),
    (8, 2, 60, 64, EUNSUPPORTED), (8, 2, 64, 72, EUNSUPPORTED), (8, 1025, 64, 64, EUNSUPPORTED),
    (8, 2, 1 << 16, 1 << 15, EUNSUPPORTED),  # N K
    (8, 2, 8, 1 << 17, EUNSUPPORTED),        # the sums' range
    (8, 2, 1 << 22, 16, EUNSUPPORTED),       # 512 N
    (1 << 30, 2, 64, 64, EUNSUPPORTED)])
def test_gemm_shapes(B, M, E, N, K, code):
    assert B.lib.moe_gemm_i8(M, E, N, K, *GEMM, None) == code


def test_gemm_pointers(B):
    call = lambda args, E=2, M=8: B.lib.moe_gemm_i8(M, E, 64, 64, *args, None)
    for i in (0, 1, 2, 3, 4, 6):
        assert call(_with(GEMM, i, None)) == EINVAL
    for i in (0, 3, 6):
        assert call(_with(GEMM, i, ODD)) == EINVAL
    assert call(_with(GEMM, 2, None), E=1, M=0) == OK


SHAPES = [((0, 64, 4, 2, 64, "bf16"), EINVAL), ((8, 64, 4, 5, 64, "bf16"), EINVAL), ((8, 64, 2000, 2, 64, "bf16"), EINVAL),
          ((8, 96, 4, 2, 64, "bf16"), EUNSUPPORTED), ((8, 64, 4, 2, 48, "bf16"), EUNSUPPORTED),
          ((8, 64, 4, 2, 64, "f32"), EUNSUPPORTED)]


@pytest.mark.parametrize("name,n,optional", [("moe_gemm_gate_up_i8", 11, None), ("moe_experts_i8", 22, None),
                                             ("moe_forward_fused_i8", 25, 2), ("moe_forward_few_i8", 14, 2)])
def test_layer_refusals(B, name, n, optional):
    fn = getattr(B.lib, name)
    for dims, code in SHAPES:
        assert fn(B.shape(*dims), *[FAKE] * n, 1 << 40, None) == code, dims
        assert B.moe_i8_workspace_bytes(B.shape(*dims)) == 0
    s = B.shape(8, 64, 4, 2, 64, "bf16")
    for i in range(n):
        if i != optional:
            assert fn(s, *_with([FAKE] * n, i, None), 1 << 40, None) == EINVAL, i
    for i in (0, n - 1):  # the activations, the workspace
        assert fn(s, *_with([FAKE] * n, i, ODD), 1 << 40, None) == EINVAL
    need = (B.moe_few_workspace_bytes if "few" in name else B.moe_i8_workspace_bytes)(s)
    assert need > 0 and fn(s, *[FAKE] * n, need - 1, None) == EWORKSPACE


def test_sums_stay_in_range(B):
    """H and I are reductions of at most 2^17 products of 2^14."""
    for dims in ((8, 1 << 17, 4, 2, 64, "bf16"), (8, 64, 4, 2, 1 << 17, "bf16")):
        assert B.lib.moe_experts_i8(B.shape(*dims), *[FAKE] * 22, 1 << 40, None) == EUNSUPPORTED


def test_definition():
    q, s = Q.codes(torch.tensor([[254.0, 1.0, 3.0, -254.0], [0.0, 0.0, 0.0, 0.0]]))
    assert q.tolist() == [[127, 0, 2, -127], [0, 0, 0, 0]] and s.tolist() == [[2.0], [0.0]]  # halves to even
    q, s = Q.codes(torch.tensor([[1.0] * 64 + [0.5, float("inf")]]), 64)
    assert q[0, :64].eq(127).all() and q[0, 64:].eq(0).all() and s[0, 1].isnan()


# ---- ServingStage on I8Weights ---------------------------------------------------

E, I, H, K = 4, 64, 128, 2


def _z(*d, dt=torch.bfloat16, dev="cpu"):
    return torch.zeros(*d, dtype=dt, device=dev)


def _stored(dt=torch.int8, dev="cpu", scale=torch.float32):
    f = lambda *d: _z(*d, dt=scale, dev=dev)
    return [(_z(E, I, H, dt=dt, dev=dev), f(E, I)), (_z(E, I, H, dt=dt, dev=dev), f(E, I)), (_z(E, H, I, dt=dt, dev=dev), f(E, H))]


def test_stage_refusals(B):
    good = _stored()
    for max_T in (8, 200):
        B.ServingStage(max_T, K, _z(E, H), B.I8Weights(stored=good))
    bad = [_stored(torch.uint8), _stored(torch.float8_e4m3fn), _stored(scale=torch.float64), _stored()[:2] + _stored(dev="meta")[2:],
           good[:2] + [(good[2][0], _z(E, I, dt=torch.float32))],                         # one scale per row of [E,H,I]
           good[:2] + [(good[2][0], _z(E, 1, 1, dt=torch.float32))],                      # block scales
           good[:2] + [(_z(E, I, H, dt=torch.int8).transpose(1, 2), good[2][1])]]
    for stored in bad:
        with pytest.raises(ValueError):
            B.ServingStage(200, K, _z(E, H), B.I8Weights(stored=stored))
    with pytest.raises(ValueError):
        B.I8Weights(_z(E, I, H), _z(E, I, H), _z(E, H, I))  # host tensors
    with pytest.raises(ValueError):
        B.ServingStage(8, K, _z(E, H), B.I8Weights(stored=good)).forward(_z(3, H))
