"""Rows that no expert has: where offsets begin past row 0 and end before the last, a
call on sorted rows computes the experts' rows and leaves the others' results as they
were, whatever the workspace holds (include/moe_i8.h, include/moe_ckpt8.h)."""
import pytest
import torch

from mixture_experts_expert_amd import binding as B

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
CASES = [([1, 0, 2], 3, 5), ([40, 0, 100], 1, 9), ([300, 270, 0], 70, 2), ([0, 0, 0], 4, 3)]


def rows(counts, before, behind):
    M, off = before + sum(counts) + behind, torch.tensor([before] + counts).cumsum(0)
    inside = torch.zeros(M, dtype=torch.bool, device="cuda")
    inside[before:before + sum(counts)] = True
    return M, off.to(torch.int32).cuda(), inside


def full(v, dt, *d):
    return torch.full(d, v, dtype=dt, device="cuda")


@pytest.mark.parametrize("counts,before,behind", CASES)
def test_gate_up_i8(counts, before, behind):
    M, off, inside = rows(counts, before, behind)
    E, H, I = len(counts), 128, 192
    g = torch.Generator("cuda").manual_seed(1)
    codes = lambda *d: torch.randint(-127, 128, d, generator=g, device="cuda").to(torch.int8)
    x, w = codes(M, H), [codes(E, I, H) for _ in range(2)]
    xs, sc = torch.rand(M, generator=g, device="cuda") + 0.1, [torch.rand(E, I, generator=g, device="cuda") * 1e-4 for _ in range(2)]
    token = torch.randperm(M, generator=g, device="cuda").to(torch.int32)
    s = B.shape(M, H, E, 1, I, BF)
    got = []
    for fill in (0x00, 0x5a, 0xff):
        aq, sa = full(7, torch.int8, M, I), full(-1.0, torch.float32, M)
        ws = full(fill, torch.uint8, B.moe_i8_workspace_bytes(s))
        B.moe_gemm_gate_up_i8(s, x, xs, token, off, w[0], sc[0], w[1], sc[1], aq, sa, ws)
        assert aq[~inside].eq(7).all() and sa[~inside].eq(-1).all()
        assert sa[inside].gt(0).all() and aq[inside].abs().amax(1).eq(127).all()
        got.append((aq, sa))
    assert all(torch.equal(a, got[0][0]) and torch.equal(b, got[0][1]) for a, b in got)


@pytest.mark.parametrize("counts,before,behind", CASES)
def test_down_dgrad_ckpt8(counts, before, behind):
    M, off, inside = rows(counts, before, behind)
    E, H, I = len(counts), 128, 192
    g = torch.Generator("cuda").manual_seed(2)
    r = lambda *d: torch.randn(*d, generator=g, device="cuda")
    codes = lambda *d: torch.randint(-127, 128, d, generator=g, device="cuda").to(torch.int8)
    dy, wd, rw = r(M, H).to(BF), r(E, H, I).to(BF), torch.rand(M, generator=g, device="cuda") + 0.1
    kept = [codes(M, I), torch.rand(M, I // 64, generator=g, device="cuda") * 0.01 + 0.01]
    kept += [codes(M, I), torch.rand(M, I // 64, generator=g, device="cuda") * 0.01 + 0.01]
    order = torch.randperm(M, generator=g, device="cuda").to(torch.int32)
    s = B.shape(M, H, E, 1, I, BF)
    got = []
    for fill in (0x00, 0x5a, 0xff):
        dgu, aw, dt = full(-3.0, BF, M, 2 * I), full(-3.0, BF, M, I), full(-3.0, torch.float32, M, 1)
        ws = full(fill, torch.uint8, B.moe_ckpt8_workspace_bytes(s))
        B.moe_gemm_down_dgrad_ckpt8(s, dy, order, rw, order, off, wd, *kept, dgu, aw, dt, ws)
        by_row = dt.view(-1)[order.long()]
        assert dgu[~inside].eq(-3).all() and aw[~inside].eq(-3).all() and by_row[~inside].eq(-3).all()
        assert not by_row[inside].eq(-3).any() and by_row.isfinite().all()
        got.append((dgu, aw, dt))
    assert all(torch.equal(a, b) for t in got for a, b in zip(t, got[0]))


@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("counts,before,behind", CASES + [([700, 600, 400], 3, 2)])  # the last: 256 rows per expert and more
def test_gate_up_ckpt8(counts, before, behind, gathered):
    M, off, inside = rows(counts, before, behind)
    E, H, I = len(counts), 128, 192
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda *d: torch.randn(*d, generator=g, device="cuda").to(BF)
    x, w, token = r(M, H), [r(E, I, H) for _ in range(2)], torch.randperm(M, generator=g, device="cuda").to(torch.int32)
    out = [full(7, torch.int8, M, I), full(-1.0, torch.float32, M, I // 64), full(7, torch.int8, M, I),
           full(-1.0, torch.float32, M, I // 64), full(-3.0, BF, M, I)]
    B.moe_gemm_gate_up_ckpt8(B.shape(M, H, E, 1, I, BF), x, token if gathered else None, off, *w, *out)
    for t, v in zip(out, (7, -1, 7, -1, -3)):
        assert t[~inside].eq(v).all()
    assert out[1][inside].gt(0).all() and out[3][inside].gt(0).all()
    assert out[0][inside].view(-1, 64).abs().amax(1).eq(127).all()
