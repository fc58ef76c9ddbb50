"""GPU tests of the serving operators (include/moe_serve.h) at the ends of the
number range, with outlying values and with a wait that gives up."""
import ctypes

import pytest
import torch

from mixture_experts_expert_amd import binding as B
from oracle import serve as S

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
U = 2.0**-8  # one rounding to bf16


def _few_logits(x, wr, bias=None):
    """The logits of the few-token layer, on weights of zeros."""
    (T, H), E, I = x.shape, wr.shape[0], 64
    s = B.shape(T, H, E, 1, I, BF)
    z = lambda *d, dt=BF: torch.zeros(*d, dtype=dt, device="cuda")
    logits = torch.full((T, E), 7.0, device="cuda")
    B.moe_forward_few(s, x.cuda(), wr.cuda(), bias, z(E, I, H), z(E, I, H), z(E, H, I), logits, z(T, 1, dt=torch.int32),
                      z(T, 1, dt=torch.float32), z(T, H), z(B.moe_few_workspace_bytes(s), dt=torch.uint8))
    return logits.cpu()


@pytest.mark.parametrize("T", [1, 20])
def test_few_logits_of_products_beyond_fp32(T):
    """Products of 2^130 that cancel, and what is left beside them: exact in float64."""
    g = torch.Generator().manual_seed(1)
    H, E = 64, 6
    x = torch.randint(1, 8, (T, H), generator=g).double() * 2.0**70
    w = torch.randint(1, 8, (E, H), generator=g).double() * 2.0**60
    x[:, 1::2] = x[:, ::2]
    w[:, 1::2] = -w[:, ::2]
    x[:, -1] += torch.randint(1, 4, (T,), generator=g) * 2.0**66  # what is left: -1 to -3 times 2^126
    w[:, -1] = w[:, -1].sign() * 2.0**60
    w[:, -2] = 2.0**60
    want = x @ w.T
    assert want.abs().max() < 2.0**128 and want.abs().min() > 0
    assert torch.equal(x.to(BF).double(), x) and torch.equal(w.to(BF).double(), w)
    assert torch.equal(_few_logits(x.to(BF), w.to(BF)).double(), want)


@pytest.mark.parametrize("T", [1, 20])
def test_few_logits_of_products_below_fp32(T):
    """64 products of 2^-150, each half of fp32's smallest number."""
    x = torch.full((T, 64), 2.0**-75).to(BF)
    w = torch.full((3, 64), 2.0**-75).to(BF)
    assert torch.equal(_few_logits(x, w), torch.full((T, 3), 2.0**-144))


@pytest.mark.parametrize("ratio", [64, 4096])
@pytest.mark.parametrize("T", [5, 150, 500])  # each of the product's kernels
def test_experts_beside_outlying_columns(T, ratio):
    """One column in eight is `ratio` times the others, as some channels of a residual
    stream are: the others come out as exactly as from bf16 rows. Bounds: 2^-8 of
    each expert's result for its row, 2^-8 of y, and the product's own (oracle/serve.py)."""
    H, E, k, I = 192, 4, 2, 128
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, H, generator=g).to(BF)
    gate, up = ((torch.randn(E, I, H, generator=g) / H**0.5).to(BF) for _ in range(2))
    down = torch.randint(-7, 8, (E, H, I), generator=g) * 2.0**-6
    down[:, 3::8] *= ratio
    codes = [S.quantize_weights(gate), S.quantize_weights(up), (down.to(F8).view(torch.uint8), torch.ones(E, 2, 1).double())]
    w8 = B.FP8BlockWeights(stored=[(q.cuda(), s.float().cuda()) for q, s in codes])
    idx, w = S.route(torch.randn(T, E, generator=g), k)
    M, e = T * k, lambda *n, dt=torch.float32: torch.empty(*n, dtype=dt, device="cuda")
    i32, u8 = torch.int32, torch.uint8
    off, f2s, rw, aq, sa, op, y = e(E + 1, dt=i32), e(M, dt=i32), e(M), e(M, I, dt=u8), e(M, 1), e(M, H, dt=BF), e(T, H, dt=BF)
    s = B.shape(T, H, E, k, I, BF)
    B.moe_experts_fp8_block(s, x.cuda(), idx.to(i32).cuda(), w.float().cuda(), *w8.gate, *w8.up, *w8.down, e(E, dt=i32), off,
                            e(M, dt=i32), f2s, e(M, dt=i32), rw, e(T, H, dt=u8), e(T, 2), aq, sa, op, y,
                            e(B.moe_workspace_bytes(s), dt=u8))
    off, f2s, rw, y = off.cpu(), f2s.cpu().long(), rw.cpu().double(), y.cpu().double()
    a = S.dequantize_rows(aq.cpu(), sa.cpu())
    want, tol = torch.zeros(M, H).double(), torch.zeros(M, H).double()
    for n in range(E):
        lo, hi = off[n], off[n + 1]
        v, lost = S.product(a[lo:hi], down[n].double())
        f = rw[lo:hi, None]
        want[lo:hi] = v * f
        tol[lo:hi] = (lost + a[lo:hi].abs() @ down[n].double().abs().T * 2.0**-20) * f
    parts, slack = want[f2s].view(T, k, H), tol[f2s].view(T, k, H).sum(1)
    sums, mag = parts.sum(1), parts.abs().sum(1)
    assert ((y - sums).abs() <= sums.abs() * U + (mag * (U + 2.0**-20) + slack) * (1 + 2 * U)).all()
    held = S.shared8_values(op.cpu())
    assert ((held - want).abs() <= want.abs() * U + tol * (1 + U)).all()


class _FewArgs(ctypes.Structure):  # moe::FewArgs (csrc/moe_internal.h)
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "w_router", "bias", "w_gate", "w_up", "w_down", "gate_scale", "up_scale",
                                               "down_scale", "logits", "topk_idx", "topk_w", "y")] + [("polls", ctypes.c_uint32)]


@pytest.mark.parametrize("dims", [(1, 64, 4, 2, 64), (40, 320, 60, 6, 192)], ids=str)  # one group of experts, and several
def test_few_wait_that_gives_up_shows(dims):
    """A wait for the activations that ends early leaves NaN, never numbers made without them."""
    T, H, E, k, I = dims
    launch = B.lib["_ZN3moe10launch_fewERK9moe_shapeRKNS_7FewArgsEPvP12ihipStream_t"]
    launch.argtypes = [ctypes.c_void_p] * 4
    g = torch.Generator().manual_seed(3)
    ins = [torch.randn(T, H, generator=g), torch.randn(E, H, generator=g) / 8, torch.randn(E, I, H, generator=g) / 8,
           torch.randn(E, I, H, generator=g) / 8, torch.randn(E, H, I, generator=g) / 8]
    x, wr, gate, up, down = (t.to(BF).cuda() for t in ins)
    s = B.shape(*dims, BF)
    ws = torch.zeros(B.moe_few_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    new = lambda: (torch.empty(T, E, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda"),
                   torch.empty(T, k, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda"))
    right = new()
    B.moe_forward_few(s, x, wr, None, gate, up, down, *right, ws)
    for polls in (0, 1, 1 << 23):
        out = new()
        ws.zero_()  # activations of zeros, were they read too early
        a = _FewArgs(x.data_ptr(), wr.data_ptr(), None, gate.data_ptr(), up.data_ptr(), down.data_ptr(), None, None, None,
                     *(t.data_ptr() for t in out), polls)
        assert launch(ctypes.addressof(s), ctypes.addressof(a), ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out[:3], right[:3]))
        lost = out[3].isnan()
        assert torch.equal(out[3][~lost], right[3][~lost])
        assert {0: lost.all(), 1: True}.get(polls, not lost.any())


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_stage_enqueues_on_its_own_device(fmt, monkeypatch):
    """Whatever the current device is: the calls run with the tensors' device made current."""
    made_current = []

    class device(torch.cuda.device):
        def __init__(self, d):
            made_current.append(torch.device(d))
            super().__init__(d)

    E, I, H, k = 4, 64, 128, 2
    g = torch.Generator().manual_seed(4)
    w = [(torch.randn(E, *d, generator=g) / 8).to(BF).cuda() for d in ((I, H), (I, H), (H, I))]
    wr, x = torch.randn(E, H, generator=g).to(BF).cuda(), torch.randn(70, H, generator=g).to(BF).cuda()
    monkeypatch.setattr(torch.cuda, "device", device)
    weights = B.FP8BlockWeights(*w) if fmt == "fp8" else w
    assert made_current == [x.device] * (3 if fmt == "fp8" else 0)
    stage = B.ServingStage(70, k, wr, weights)
    made_current.clear()
    for T in (3, 70):
        assert stage.forward(x[:T]).isfinite().all()
    assert made_current == [x.device] * 2


def test_no_rows():
    """Empty tensors, as they are, through the calls and the stage."""
    E, I, H, k = 4, 64, 128, 2
    e = lambda *d, dt=BF: torch.empty(*d, dtype=dt, device="cuda")
    u8, f32 = torch.uint8, torch.float32
    B.moe_quantize_fp8_block_rows(0, H, e(0, H), e(0, H, dt=u8), e(0, 1, dt=f32))
    w, sw = torch.zeros(E, I, H, dtype=u8, device="cuda"), torch.zeros(E, 1, 1, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    B.moe_gemm_fp8_block(0, E, I, H, e(0, H, dt=u8), e(0, 1, dt=f32), off, w, sw, e(0, dt=f32), e(0, I))
    stage = B.ServingStage(70, k, torch.zeros(E, H, dtype=BF, device="cuda"), [t.to(BF) for t in (w, w, w.transpose(1, 2).contiguous())])
    y = stage.forward(e(0, H))
    assert y.shape == (0, H) and y.dtype == BF


def _definition(x, wr, k, idx, w, pairs, t):
    """Token t of the layer on block-scaled weights, float64: y and the sum of magnitudes."""
    H = x.shape[1]
    y, mag = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
    for j in range(k):
        e = int(idx[t, j])
        gate, up, down = (_weights64(q[e], s[e]) for q, s in pairs)
        a = float(w[t, j]) * S.silu_mul(gate @ x[t].double(), up @ x[t].double())
        y += down @ a
        mag += down.abs() @ a.abs()
    return y, mag


def _weights64(q, s):
    N, K = q.shape
    return q.view(F8).double() * s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def test_layer_past_2_to_31_weights():
    """520 experts of 2048 x 2048: expert bases past 2^31 bytes, in both forms, through the
    stage, whose workspace holds the sort's counts and nothing else."""
    E, I, H, k, T = 520, 2048, 2048, 3, 70
    g = torch.Generator("cuda").manual_seed(5)
    codes = torch.randint(0, 256, (1 << 22,), generator=g, device="cuda", dtype=torch.uint8)
    codes = (codes & 0xBF) | 0x10  # magnitudes of 1/32 to 2, and the sign
    pairs = []
    for N, K in ((I, H), (I, H), (H, I)):
        q = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
        for e in range(E):
            q[e] = codes.roll(1009 * e + len(pairs)).view(N, K)
        pairs.append((q, torch.rand(E, N // 128, K // 128, generator=g, device="cuda") * 0.02))
    x = torch.randn(T, H, generator=g, device="cuda").to(BF)
    wr = (torch.randn(E, H, generator=g, device="cuda") / 64).to(BF)
    bias = torch.zeros(E, device="cuda")
    bias[-6:] = 3.0  # the last experts, whose bases lie furthest out
    stage = B.ServingStage(T, k, wr, B.FP8BlockWeights(stored=pairs), bias)
    whole = torch.full((stage.ws.numel() + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    stage.ws = whole[: stage.ws.numel()]
    for n in (5, T):
        y = stage.forward(x[:n]).double()
        idx = stage.buf["topk_idx"].view(-1)[: n * k].view(n, k)
        w = stage.buf["topk_w"].view(-1)[: n * k].view(n, k)
        assert idx.max() == E - 1
        for t in (0, 3, n - 1):
            want, mag = _definition(x, wr, k, idx, w, pairs, t)
            # rounded a and y, in the norm; 70 tokens also quantise x and a: 2^-4 at most each
            tol = 2**0.5 * U if n <= 64 else 2**0.5 * 2.0**-4 + 2 * U
            assert (y[t] - want).norm() <= tol * want.norm()
    assert whole[stage.ws.numel():].eq(0xA5).all()


def _busy(stream):
    """About 50 ms of waiting on the stream, so that what follows there runs late."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)


def test_quantising_on_another_stream_keeps_off_freed_memory():
    """The codes made on a side stream lie in no block that the current stream still reads."""
    E, N, K = 16, 1024, 1024  # codes of 16 MiB: blocks of their own in torch's allocator
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    w = [torch.randn(E, N, K, device="cuda").to(BF) for _ in range(3)]
    side.wait_stream(here)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = [torch.full((E, N, K), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    _busy(here)
    kept = [f + 1 for f in freed]
    del freed
    w8 = B.FP8BlockWeights(*w, stream=side)
    torch.cuda.synchronize()
    assert all(t.eq(8).all() for t in kept)
    assert all(torch.equal(q, p) and torch.equal(s, r) for (q, s), (p, r) in
               zip((w8.gate, w8.up, w8.down), ((lambda v: (v.gate, v.up, v.down))(B.FP8BlockWeights(*w)))))


def test_inputs_of_another_stream_outlive_the_call():
    """Weights and x handed to a call on a side stream and dropped by the caller: their memory
    is not given out again before that stream has read them."""
    E, I, H, k, T = 4, 1024, 1024, 2, 70
    g = torch.Generator("cuda").manual_seed(6)
    w = [torch.randn(E, I, H, generator=g, device="cuda").to(BF) for _ in range(3)]
    x, wr = torch.randn(T, H, generator=g, device="cuda").to(BF), torch.randn(E, H, generator=g, device="cuda").to(BF)
    want8 = B.FP8BlockWeights(*w)
    stage = B.ServingStage(T, k, wr, want8)
    want = stage.forward(x).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ws, xs = [t.clone() for t in w], x.clone()
    torch.cuda.synchronize()
    _busy(side)
    got8 = B.FP8BlockWeights(*ws, stream=side)
    y = stage.forward(xs, stream=side)
    del ws, xs
    again = [torch.zeros(E, I, H, dtype=BF, device="cuda") for _ in range(3)] + [torch.zeros(T, H, dtype=BF, device="cuda")]
    torch.cuda.synchronize()
    assert torch.equal(y, want) and len(again) == 4
    for a, b in ((got8.gate, want8.gate), (got8.up, want8.up), (got8.down, want8.down)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
