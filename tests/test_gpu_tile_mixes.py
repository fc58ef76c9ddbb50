"""Grouped products whose workgroups meet row tiles of every height in turn: up to
32, 64 and 128 rows (and 256, where a kernel has such tiles), several tiles each, so
that every kind of tile follows every other and a tile's stores run on under a
shorter or a longer one's first steps.

Operands are small whole numbers with powers of two as scales: sums and scaled sums
are exact in fp32 and the one rounding to bf16 is compared exactly. The kept codes
and gradients go by the tolerances of test_gpu_ckpt8.py, the E4M3 codes by those of
test_gpu_serve_tiles.py."""
import pytest
import torch

import test_gpu_ckpt8 as C
import test_gpu_serve_tiles as V
from mixture_experts_expert_amd import binding as B

pytestmark = pytest.mark.gpu

BF, I8 = torch.bfloat16, torch.int8

# Rows per expert. A workgroup's next tile is some experts on: periods that no number of column tiles divides.
SHORT = [(20, 50, 100, 1, 64, 33, 128)[e % 7] for e in range(98)]
MIXED = [(20, 300, 33, 128, 64, 500, 129)[e % 7] for e in range(42)]  # longer experts among them, short on average
TALL = [100, 900, 20, 300, 128, 700, 1, 520, 129, 640, 60, 800]       # 256 rows each on average, and more


def offsets(counts):
    return torch.tensor([0] + counts).cumsum(0)


def whole(g, *dims, top=2):
    return torch.randint(-top, top + 1, dims, generator=g, device="cuda").to(I8)


def two(g, lo, hi, *dims):
    return torch.exp2(torch.randint(lo, hi, dims, generator=g, device="cuda").float())


@pytest.mark.parametrize("K", [16, 144, 208, 592])  # steps that end a tile differently, the last one short
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("counts", [SHORT, MIXED, TALL], ids=["short", "mixed", "tall"])
def test_gemm_i8(counts, weighted, K):
    E, M, off = len(counts), sum(counts), offsets(counts)
    N = 8000 if counts is TALL else 5000
    g = torch.Generator("cuda").manual_seed(41)
    aq, wq = whole(g, M, K), whole(g, E, N, K)
    sa, sw = two(g, -1, 2, M), two(g, -1, 2, E, N)
    rw = two(g, -1, 2, M) if weighted else None
    out = torch.full((M + 1, N), -3.0, dtype=BF, device="cuda")
    for _ in range(2):  # again over its own results
        B.moe_gemm_i8(M, E, N, K, aq, sa, off.to(torch.int32).cuda(), wq, sw, rw, out)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        want = (aq[r].double() @ wq[e].double().T) * sa[r, None] * sw[e]
        if weighted:
            want = want * rw[r, None]
        assert torch.equal(out[r], want.float().to(BF)), e
    assert out[M].eq(-3).all()


@pytest.mark.parametrize("H", [64, 128, 192, 320])
@pytest.mark.parametrize("counts", [SHORT, MIXED, [1, 3, 0, 2] * 9], ids=["short", "mixed", "few rows"])
def test_gate_up_i8(counts, H):
    """The codes of silu(g) u: every one within half a step of the value, but for fp32's roundings (less than 16,
    of 2^-24 each), the 24-bit form (2^-24 of the row's largest, and four roundings to it and back) and the scale's:
    127 (2^-20 + 2^-24 + 2 2^-22) < 127 2^-19 steps in all. (In 16 bits it would be 127 2^-17.)"""
    E, M, off = len(counts), sum(counts), offsets(counts)
    I = 2176
    g = torch.Generator("cuda").manual_seed(42)
    x, wg, wu = whole(g, M, H), whole(g, E, I, H, top=1), whole(g, E, I, H, top=1)
    xs, sg, su = two(g, -3, -1, M), two(g, -3, 0, E, I), two(g, -3, 0, E, I)
    s = B.shape(M, H, E, 1, I, BF)
    token = torch.randint(0, M, (M,), generator=g, device="cuda", dtype=torch.int32)
    aq = torch.full((M + 1, I), 7, dtype=I8, device="cuda")
    sa = torch.full((M + 1,), -1.0, device="cuda")
    nb = B.moe_i8_workspace_bytes(s)
    ws = torch.full((nb + 16,), 0x5a, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        B.moe_gemm_gate_up_i8(s, x, xs, token, off.to(torch.int32).cuda(), wg, sg, wu, su, aq, sa, ws, ws_bytes=nb)
    assert (aq[M] == 7).all() and sa[M] == -1 and (ws[nb:] == 0x5a).all()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e] == 0:
            continue
        rows = x[token[r].long()].double() * xs[token[r].long(), None]
        gv, uv = rows @ (wg[e] * sg[e][:, None].double()).T, rows @ (wu[e] * su[e][:, None].double()).T
        v = gv * torch.sigmoid(gv) * uv
        top, q, sc = v.abs().amax(1, keepdim=True), aq[r].double(), sa[r, None].double()
        assert ((sc - top / 127).abs() <= top * 2.0**-19 / 127).all(), e
        assert ((q * sc - v).abs() <= top / 127 * (0.5 + 127 * 2.0**-19) + 1e-30).all(), e


def experts_of(counts):
    """In place of test_gpu_ckpt8's routing: the given rows per expert, tokens in any order."""
    def routing(T, E, k, seed, skew=0.0, empty=()):
        assert k == 1 and T == sum(counts) and E == len(counts)
        g = torch.Generator().manual_seed(seed)
        token = torch.randperm(T, generator=g).to(torch.int32)
        w = torch.rand(T, generator=g) + 0.1
        tw = torch.empty(T)
        tw[token.long()] = w
        return offsets(counts).to(torch.int32), token, w, token.clone(), tw.view(T, 1)
    return routing


@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("H", [64, 128, 192])
@pytest.mark.parametrize("counts", [SHORT[:49], TALL + [0] * 2], ids=["short", "tall"])
def test_gate_up_ckpt8(counts, H, gathered, monkeypatch):
    """short: 128-row tiles, two workgroups per CU; tall: 256-row tiles (256 rows per expert on average)."""
    monkeypatch.setattr(C, "routing", experts_of(counts))
    C.test_gate_up(sum(counts), H, len(counts), 1, 4160 if counts[0] == 20 else 2240, 0.0, (), gathered)


@pytest.mark.parametrize("H", [64, 128, 192])
@pytest.mark.parametrize("counts", [SHORT, MIXED], ids=["short", "mixed"])
def test_down_dgrad_ckpt8(counts, H, monkeypatch):
    monkeypatch.setattr(C, "routing", experts_of(counts))
    C.test_down_dgrad(sum(counts), H, len(counts), 1, 3008 if counts is SHORT else 4160, 0.0, ())


@pytest.mark.parametrize("K", [16, 240, 272, 400])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("counts", [SHORT, MIXED], ids=["short", "mixed"])
def test_gemm_fp8_block(counts, weighted, K, monkeypatch):
    """short: 128-row tiles; mixed: 256-row tiles (more than 96 rows per expert on average)."""
    monkeypatch.setitem(V.ROWS, "mix", counts)
    V.test_gemm_many_tiles("mix", weighted, K)


@pytest.mark.parametrize("H", [64, 192, 320, 448])
@pytest.mark.parametrize("counts", [SHORT, MIXED], ids=["short", "mixed"])
def test_gate_up_fp8_block(counts, H, monkeypatch):
    monkeypatch.setitem(V.ROWS, "mix", counts)
    V.test_gate_up_many_tiles("mix", H)
