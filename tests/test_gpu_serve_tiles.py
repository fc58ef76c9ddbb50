"""The block-scaled products (include/moe_serve.h) where a workgroup takes several
tiles: more tiles than the device has compute units, experts longer than a band
of row tiles, more experts than one wavefront scans, tiles of both heights in
turn, and reductions of one to four steps.

Operands are small whole numbers with powers of two as scales: every product and
sum is exact in fp32, so the plain product is compared exactly (its one rounding
included) and every index is pinned. In the gate/up form g and u are exact, a is
off by 2^-18 (the exponential and the reciprocal), a code by 2^-4 of the value or
half the smallest code."""
import pytest
import torch

from mixture_experts_expert_amd import binding as B
from oracle import serve as S

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn

# name -> rows per expert. Up to 96 rows per expert on average run in tiles of
# 128 rows, more in tiles of 256.
ROWS = {
    "short tiles": [20 + i % 7 for i in range(20)] + [0, 1100, 0, 64, 65, 128, 129] + [19] * 14,
    "300 experts": [(i * 7) % 13 for i in range(300)],
    "long tiles": [2200, 130, 0, 1, 128, 129, 256, 257, 1000],
}


def _counts(rows, tile_columns):
    """The tiles of a launch: enough for a second and a third one per workgroup."""
    E, M = len(rows), sum(rows)
    bm = 128 if -(-M // E) <= 96 else 256
    tiles = sum(-(-r // bm) for r in rows) * tile_columns
    assert tiles > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    return E, M, torch.tensor([0] + rows).cumsum(0)


def _whole(g, *dims, top=1, keep=1.0):
    v = torch.randint(-top, top + 1, dims, generator=g, device="cuda").float()
    return v * (torch.rand(dims, generator=g, device="cuda") < keep)


def _two(g, lo, hi, *dims):
    return torch.exp2(torch.randint(lo, hi, dims, generator=g, device="cuda").float())


def _codes(v):
    return v.to(F8).view(torch.uint8)


@pytest.mark.parametrize("K", [16, 240, 272, 400])  # one to four steps, the last one short
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("rows", list(ROWS))
def test_gemm_many_tiles(rows, weighted, K):
    N = 8000 if rows == "long tiles" else 4000
    E, M, off = _counts(ROWS[rows], -(-N // 256))
    g = torch.Generator("cuda").manual_seed(31)
    a, w = _whole(g, M, K, top=2), _whole(g, E, N, K, keep=0.2)
    KB, NB = -(-K // 128), -(-N // 128)
    sa, sw = _two(g, -1, 2, M, KB), _two(g, -1, 1, E, NB, KB)
    rw = _two(g, -1, 2, M) if weighted else None
    out = torch.full((M + 1, N), -3.0, dtype=BF, device="cuda")
    for _ in range(2):
        B.moe_gemm_fp8_block(M, E, N, K, _codes(a), sa, off.to(torch.int32).cuda(), _codes(w), sw, rw, out)
    ad = a * S._spread(sa, 1, K).float()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        wd = w[e] * S._spread(S._spread(sw[e], 0, N), 1, K).float()
        want = ad[lo:hi].double() @ wd.double().T
        if weighted:
            want = want * rw[lo:hi, None]
        assert torch.equal(out[lo:hi], want.float().to(BF)), e
    assert out[M].eq(-3).all()


@pytest.mark.parametrize("H", [64, 192, 320, 448])  # one to four steps
@pytest.mark.parametrize("rows", list(ROWS))
def test_gate_up_many_tiles(rows, H):
    I, k = 4032, 2
    E, M, off = _counts(ROWS[rows], -(-I // 128))
    T = -(-M // k)
    g = torch.Generator("cuda").manual_seed(32)
    x, wg, wu = _whole(g, T, H, top=2), _whole(g, E, I, H, keep=0.1), _whole(g, E, I, H, keep=0.1)
    HB, IB = -(-H // 128), -(-I // 128)
    xs, sg, su = _two(g, -2, 1, T, HB), _two(g, -2, 1, E, IB, HB), _two(g, -2, 1, E, IB, HB)
    token = torch.randint(0, T, (T * k,), generator=g, device="cuda", dtype=torch.int32)
    aq = torch.full((T * k + 1, I), 7, dtype=torch.uint8, device="cuda")
    sa = torch.full((T * k + 1, IB), -1.0, device="cuda")
    s = B.shape(T, H, E, k, I, BF)
    for _ in range(2):
        B.moe_gemm_gate_up_fp8_block(s, _codes(x), xs, token, off.to(torch.int32).cuda(), _codes(wg), sg, _codes(wu), su,
                                     aq, sa)
    xd = x * S._spread(xs, 1, H).float()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        rowsx = xd[token[lo:hi].long()].double()
        gv, uv = (rowsx @ (w[e] * S._spread(S._spread(sc[e], 0, I), 1, H).float()).double().T for w, sc in ((wg, sg), (wu, su)))
        a = S.silu_mul(gv, uv)
        da = (gv * uv).abs() * 2.0**-18
        block = S._padded(a, 1).view(hi - lo, -1, 128).abs().amax(2)
        slack = S._padded(da, 1).view(hi - lo, -1, 128).amax(2)
        assert ((sa[lo:hi].double() - block / 448).abs() <= slack / 448 + block * 2.0**-20).all(), e
        got = aq[lo:hi].view(F8).double() * S._spread(sa[lo:hi], 1, I)
        step = a.abs() * 2.0**-4 + S._spread(block + slack, 1, I) / 448 * 2.0**-10
        assert ((got - a).abs() <= step * (1 + 2.0**-4) + 2 * da).all(), e
    assert aq[M:].eq(7).all() and sa[M:].eq(-1).all()  # rows of no expert are left
