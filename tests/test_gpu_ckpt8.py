"""GPU tests of activations kept in 8 bits (include/moe_ckpt8.h) against their
64-bit definitions (oracle/i8.py).

Tolerances. The codes of bf16 inputs are exact; a value read back is code * scale,
two fp32 roundings (2^-24 each) and one to bf16 (2^-8). In the fused product the
fp32 sums of K exact bf16 products are off by at most (K + 2) 2^-24 of their
magnitudes, and the scale by 2^-22: where that moves a value over a border
between codes, it is a whole step off, else half a step. In the backward dA is
such a sum too; the sigmoid and its products add less than 16 roundings of 2^-24,
and the results are rounded to bf16 once."""
import pytest
import torch

from mixture_experts_expert_amd import binding as B
from oracle import i8 as Q

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0**-8


def gen(seed):
    return torch.Generator().manual_seed(seed)


def dev(*ts):
    out = [t.cuda() if t is not None else None for t in ts]
    return out if len(out) > 1 else out[0]


@pytest.mark.parametrize("R,K", [(0, 64), (1, 8), (5, 56), (37, 64), (6, 72), (300, 1000), (9, 2048)])
def test_rows_and_back(R, K):
    x = torch.randn(R, K, generator=gen(1)) * torch.exp2(torch.randint(-20, 20, (R, 1), generator=gen(2)).float())
    if R > 4:
        x[0] = 0.0
        x[1], x[1, K // 2] = 0.0, -2.0**-130  # subnormal
        x[2] = 3.0e38
        x[3, K - 1] = float("nan")
        x[4, 0] = float("-inf")
    x = x.to(BF)
    q = torch.full((R + 1, K), 7, dtype=torch.int8, device="cuda")
    s = torch.full((R + 1, -(-K // 64)), -1.0, device="cuda")
    out = torch.full((R + 1, K), -3.0, dtype=BF, device="cuda")
    B.moe_quantize_ckpt8(R, K, dev(x) if R else None, q, s)
    B.moe_dequantize_ckpt8(R, K, q, s, out)
    assert (q[R] == 7).all() and (s[R] == -1).all() and (out[R] == -3).all()
    if R:
        want, scale = Q.codes(x, 64)
        got = s[:R].cpu().double()
        assert torch.equal(q[:R].cpu(), want) and torch.equal(got.isnan(), scale.isnan())
        fine = ~scale.isnan()
        assert (got - scale)[fine].abs().le(scale[fine] * 2.0**-24 + 2.0**-150).all()
        v, back = Q.values(want, scale), out[:R].cpu().double()
        assert torch.equal(back.isnan(), v.isnan())
        fine = ~v.isnan()
        assert (back - v)[fine].abs().le(v[fine].abs() * (U + 2.0**-23) + 2.0**-134 + 127 * 2.0**-150).all()


def routing(T, E, k, seed, skew=0.0, empty=()):
    g = gen(seed)
    score = torch.randn(T, E, generator=g) - skew * torch.arange(E)
    score[:, list(empty)] = -1e9
    p, idx = torch.softmax(score, 1).topk(k, dim=1)
    flat = idx.reshape(-1)
    order = torch.argsort(flat, stable=True)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    tw = (p / p.sum(1, keepdim=True)).float()
    return off, (order // k).to(torch.int32), tw.reshape(-1)[order].contiguous(), order.to(torch.int32), tw


CASES = [(1, 64, 1, 1, 64, 0.0, ()), (5, 128, 4, 2, 192, 0.0, (1,)), (70, 192, 4, 2, 320, 0.0, ()),
         (300, 256, 8, 3, 128, 0.5, (0, 7)), (700, 128, 3, 2, 576, 1.0, ()), (257, 320, 16, 16, 64, 0.0, ())]


@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("T,H,E,k,I,skew,empty", CASES)
def test_gate_up(T, H, E, k, I, skew, empty, gathered):
    off, tok, _, _, _ = routing(T, E, k, 3, skew, empty)
    g = gen(4)
    x = torch.randn(T, H, generator=g).to(BF)
    wg, wu = [(torch.randn(E, I, H, generator=g) * H**-0.5).to(BF) for _ in range(2)]
    M, s = T * k, B.shape(T, H, E, k, I, BF)
    rows = x if gathered else x[tok.long()]
    buf = lambda n, dt: torch.full((M + 1, n), 7, dtype=dt, device="cuda")
    gq, gs, uq, us, a = buf(I, torch.int8), buf(I // 64, torch.float32), buf(I, torch.int8), buf(I // 64, torch.float32), buf(I, BF)
    B.moe_gemm_gate_up_ckpt8(s, dev(rows), dev(tok) if gathered else None, *dev(off, wg, wu), gq, gs, uq, us, a)
    for t in (gq, gs, uq, us, a):
        assert (t[M] == 7).all()
    exact, size = [], []
    for w in (wg, wu):
        v, m = torch.zeros(M, I, dtype=torch.float64), torch.zeros(M, I, dtype=torch.float64)
        for e in range(E):
            r = slice(int(off[e]), int(off[e + 1]))
            xe = x[tok[r].long()].double()
            v[r], m[r] = xe @ w[e].double().T, xe.abs() @ w[e].double().abs().T
        exact.append(v)
        size.append(m * (H + 2) * 2.0**-24)
    for q, sc, v, err in ((gq, gs, exact[0], size[0]), (uq, us, exact[1], size[1])):
        got = Q.values(q[:M].cpu(), sc[:M].cpu()) if I > 64 else q[:M].cpu().double() * sc[:M].cpu().double()
        step = (v.abs().view(M, -1, 64).amax(2) / 127).repeat_interleave(64, 1)
        assert q.abs().max() <= 127
        assert (got - v).abs().le(step * 0.5 * (1 + 2.0**-14) + 2 * err + v.abs() * 2.0**-21).all()
        top = v.abs().view(M, -1, 64).amax(2)
        emax = err.view(M, -1, 64).amax(2)
        assert (sc[:M].cpu().double() * 127 - top).abs().le(emax + top * 2.0**-21).all()
    gv, uv = exact
    want = gv * torch.sigmoid(gv) * uv
    slack = (size[0] * (1.2 * uv.abs()) + size[1] * gv.abs()) * 1.01 + size[0] * size[1]  # |silu'| < 1.1
    assert (a[:M].cpu().double() - want).abs().le(want.abs() * (U + 2.0**-20) + slack + 1e-30).all()


@pytest.mark.parametrize("T,H,E,k,I,skew,empty", CASES)
def test_down_dgrad(T, H, E, k, I, skew, empty):
    off, tok, rw, order, tw = routing(T, E, k, 5, skew, empty)
    g = gen(6)
    dy = torch.randn(T, H, generator=g).to(BF)
    wd = (torch.randn(E, H, I, generator=g) * I**-0.5).to(BF)
    M, s = T * k, B.shape(T, H, E, k, I, BF)
    gq, gs = Q.codes(torch.randn(M, I, generator=g) * 2.0, 64)
    uq, us = Q.codes(torch.randn(M, I, generator=g), 64)
    gs, us = gs.float(), us.float()
    need = B.moe_ckpt8_workspace_bytes(s)
    ws = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
    dgu = torch.full((M + 1, 2 * I), -3.0, dtype=BF, device="cuda")
    aw = torch.full((M + 1, I), -3.0, dtype=BF, device="cuda")
    dt = torch.full((T + 1, k), -3.0, device="cuda")
    B.moe_gemm_down_dgrad_ckpt8(s, *dev(dy, tok, rw, order, off, wd, gq, gs, uq, us), dgu, aw, dt, ws, ws_bytes=need)
    assert (ws[need:] == 0xFF).all() and (dgu[M] == -3).all() and (aw[M] == -3).all() and (dt[T] == -3).all()
    val = lambda q, sc: q.double() * sc.double().repeat_interleave(64, 1)
    want_dgu, want_aw, want_dot = Q.down_backward(dy, tok, rw, off, wd, val(gq, gs), val(uq, us))
    size, _, _ = Q.down_backward(dy.abs(), tok, rw, off, wd.abs(), val(gq, gs), val(uq, us))  # dA's magnitudes
    f = 2.0**-24
    assert (aw[:M].cpu().double() - want_aw).abs().le(want_aw.abs() * (U + 16 * f) + 1e-30).all()
    # s (1 + g (1 - s)) cancels near its zero: its terms' size instead of its own
    gv, uv, w = val(gq, gs), val(uq, us), rw.double()[:, None]
    sg = torch.sigmoid(gv)
    terms = torch.cat([(w * uv * sg * (1 + gv.abs() * (1 - sg))).abs(), (w * gv * sg).abs()], 1)
    dA = (size[:, I:].abs() / (w * gv * sg).abs().clamp(min=1e-300)).nan_to_num(0.0)
    dA = torch.where((gv == 0), (dy.double().abs().max() * wd.double().abs().amax() * H).expand_as(dA), dA)
    assert (dgu[:M].cpu().double() - want_dgu).abs().le(
        want_dgu.abs() * U + terms * torch.cat([dA, dA], 1) * (H + 20) * f + 1e-30).all()
    mag = (dA * (gv * sg * uv).abs()).sum(1)
    got = dt[:T].cpu().double().reshape(-1)[order.long()]
    assert (got - want_dot).abs().le(mag * (H + I + 20) * f + 1e-30).all()


# More tiles than workgroups, of all the numbers of steps that end a tile differently.
SEVERAL = [(300, 64, 128, 4, 1088, 0.0, ()), (300, 128, 128, 4, 1088, 0.02, (3, 127)), (260, 192, 160, 3, 832, 0.0, (0,))]


@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("T,H,E,k,I,skew,empty", SEVERAL)
def test_gate_up_several_tiles_a_workgroup(T, H, E, k, I, skew, empty, gathered):
    test_gate_up(T, H, E, k, I, skew, empty, gathered)


@pytest.mark.parametrize("T,H,E,k,I,skew,empty", SEVERAL)
def test_down_dgrad_several_tiles_a_workgroup(T, H, E, k, I, skew, empty):
    test_down_dgrad(T, H, E, k, I, skew, empty)


# ---- the training step -------------------------------------------------------------


def layer(T, H, E, k, I, seed, zipf=0.0):
    g = gen(seed)
    x, dy = torch.randn(T, H, generator=g).to(BF), torch.randn(T, H, generator=g).to(BF)
    wr = (0.1 * torch.randn(E, H, generator=g)).to(BF)
    w = [(torch.randn(E, N, K, generator=g) * K**-0.5).to(BF) for N, K in ((I, H), (I, H), (H, I))]
    bias = (-zipf * torch.log(torch.arange(1, E + 1).float()))
    return x, dy, wr, w, bias


def reference(b, x, dy, w, gv, uv):
    """Gradients in 64 bits at the kept values gv, uv (and x), for the stage's own routing."""
    T, H = x.shape
    tok, off, rw = b["row_token"].cpu().long(), b["offsets"].cpu(), b["row_weight"].cpu()
    order, idx, tw = b["sorted_to_flat"].cpu().long(), b["topk_idx"].cpu().long(), b["topk_w"].cpu().double()
    E, I, _ = w[0].shape
    dgu, a_w, dot = Q.down_backward(dy, tok, rw, off, w[2], gv, uv)
    out = {"dx": torch.zeros(T, H, dtype=torch.float64)}
    dw = [torch.zeros(m.shape, dtype=torch.float64) for m in w]
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        xe, dye, dg, du = x[tok[r]].double(), dy[tok[r]].double(), dgu[r, :I], dgu[r, I:]
        out["dx"].index_add_(0, tok[r], dg @ w[0][e].double() + du @ w[1][e].double())
        dw[0][e], dw[1][e], dw[2][e] = dg.T @ xe, du.T @ xe, dye.T @ a_w[r]
    out.update(dw_gate=dw[0], dw_up=dw[1], dw_down=dw[2])
    d = torch.zeros(T * idx.shape[1], dtype=torch.float64)
    d[order] = dot
    d = d.view_as(tw)
    out["d_logits"] = torch.zeros(T, E, dtype=torch.float64).scatter_(1, idx, tw * (d - (tw * d).sum(1, keepdim=True)))
    return out


def off_by(got, want):
    return ((got.cpu().double() - want).norm() / want.norm().clamp(min=1e-30)).item()


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("T,H,E,k,I,zipf", [(1, 64, 2, 1, 64, 0.0), (70, 192, 4, 2, 320, 0.0), (300, 256, 16, 3, 128, 1.2),
                                            (600, 128, 4, 2, 192, 0.0)])
def test_training_step(T, H, E, k, I, zipf, x8):
    x, dy, wr, w, bias = layer(T, H, E, k, I, 21, zipf)
    xd, dyd, wrd, biasd, *wd = dev(x, dy, wr, bias, *w)
    st = B.Ckpt8Stage(T, H, E, k, I, x8=x8)
    plain = B.MoEStage(T, H, E, k, I, BF, gather_fused=True, dy_fused=True)
    y = st.forward(xd, wrd, *wd, biasd)
    assert torch.equal(y, plain.forward(xd, wrd, *wd, biasd))
    given = xd.clone()
    if x8:
        xd.zero_()  # the stage has its own
    dx = st.backward(dyd)
    b = st.buf
    kept = Q.values(b["xq"].cpu(), b["x_scale"].cpu()) if x8 and H > 64 else (
        b["xq"].cpu().double() * b["x_scale"].cpu().double() if x8 else x)
    kept = kept.to(BF) if x8 else x
    val = lambda q, s: q.cpu().double() * s.cpu().double().repeat_interleave(64, 1)
    want = reference(b, kept, dy, w, val(b["gq"], b["g_scale"]), val(b["uq"], b["u_scale"]))
    got = {"dx": dx, **{n: b[n] for n in ("dw_gate", "dw_up", "dw_down", "d_logits")}}
    # Rounded to bf16 on the way: dgu, dx_perm and dx (dx); dgu (dw_gate, dw_up); a_w (dw_down). 2^-8 each at most.
    for n, lim in (("dx", 3 * U), ("dw_gate", U), ("dw_up", U), ("dw_down", U), ("d_logits", 2.0**-14)):
        assert off_by(got[n], want[n]) <= lim, n
    # Beside the step without codes: a value of g or u is off by at most half a step, 1/254 of its block's
    # largest, which for 64 normal values is at most 5 of their deviations: 2% of one deviation, and each
    # gradient is linear in those errors with factors of at most 1.1 (silu') and 0.5 (silu'') beside values of
    # about one deviation: within 5%.
    plain.forward(given, wrd, *wd, biasd)
    plain.backward(dyd)
    for n in ("dx", "dw_gate", "dw_up", "dw_down"):
        assert off_by(got[n], plain.buf[n].cpu().double()) < 0.05, n
    # Added to, and again the same bits.
    first = {n: t.clone() for n, t in got.items()}
    if x8:
        xd.copy_(given)
    st.forward(xd, wrd, *wd, biasd)
    st.backward(dyd, accumulate_dw=True)
    assert torch.equal(b["dx"], first["dx"]) and torch.equal(b["d_logits"], first["d_logits"])
    for n in ("dw_gate", "dw_up", "dw_down"):
        assert off_by(b[n], 2 * first[n].cpu().double()) < 2.0**-20, n


def test_stages_that_share_scratch():
    """Two layers: forward, forward, backward, backward; the first's codes are still its own."""
    dims = (130, 128, 4, 2, 192)
    ls = [layer(*dims, seed) for seed in (1, 2)]
    scratch = {}
    pair = [B.Ckpt8Stage(*dims, x8=True, scratch=scratch) for _ in ls]
    alone = [B.Ckpt8Stage(*dims, x8=True) for _ in ls]
    for st, (x, dy, wr, w, bias) in list(zip(alone, ls)):
        st.forward(*dev(x, wr, *w, bias))
        st.backward(dev(dy))
    for st, (x, dy, wr, w, bias) in zip(pair, ls):
        st.forward(*dev(x, wr, *w, bias))
    for st, (x, dy, wr, w, bias) in reversed(list(zip(pair, ls))):
        st.backward(dev(dy))
    for a, b in zip(pair, alone):
        for n in ("y", "dx", "dw_gate", "dw_up", "dw_down", "d_logits"):
            assert torch.equal(a.buf[n], b.buf[n]), n
    with pytest.raises(ValueError):
        B.Ckpt8Stage(131, *dims[1:], scratch=scratch)


def test_step_in_a_graph_and_on_another_stream():
    dims = (200, 128, 4, 2, 192)
    x, dy, wr, w, bias = layer(*dims, 3)
    xd, dyd, wrd, biasd, *wd = dev(x, dy, wr, bias, *w)
    st = B.Ckpt8Stage(*dims, x8=True)
    names = ("y", "dx", "dw_gate", "dw_up", "dw_down", "d_logits")
    xs = [xd.clone(), (xd * 0.5).contiguous(), -xd]
    want = []
    for v in xs:
        st.forward(v, wrd, *wd, biasd)
        st.backward(dyd)
        want.append({n: st.buf[n].clone() for n in names})
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st.forward(xs[1], wrd, *wd, biasd, stream=side)
    st.backward(dyd, stream=side)
    side.synchronize()
    assert all(torch.equal(st.buf[n], want[1][n]) for n in names)
    buf = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        st.forward(buf, wrd, *wd, biasd)
        st.backward(dyd)
    for i in (2, 0, 1, 2):
        buf.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(st.buf[n], want[i][n]) for n in names), i
        st.forward(xs[(i + 1) % 3], wrd, *wd, biasd)  # eager work in between
        torch.cuda.synchronize()
