"""Rows that no expert has: where offsets begin past row 0 and end before the last, a
call on sorted rows computes the experts' rows and leaves the others' results as they
were, whatever the workspace holds (include/moe_i8.h)."""
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
