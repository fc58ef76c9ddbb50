"""The integer expert stage (include/moe_i8.h) as a whole: the routed call against its
two halves, and the down product in the per-token sum's form (shared8.h) where a
workgroup takes several tiles, short and long ones in turn. The tolerance of the
latter is test_gpu_i8.py's."""
import pytest
import torch

import test_gpu_i8 as I8
from mixture_experts_expert_amd import binding as B

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("skew", [0.0, 0.03])
def test_down_product_of_several_tiles_a_workgroup(skew):
    """64 experts by 18 column tiles: more than two tiles for each of 512 workgroups, of up to 32 rows and more."""
    I8.test_experts(300, 4608, 64, 4, 64, skew, (5,))


@pytest.mark.parametrize("T,H,E,k,I", [(1, 64, 1, 1, 64), (65, 192, 8, 2, 320), (300, 256, 16, 16, 128), (1100, 512, 300, 4, 64)])
@pytest.mark.parametrize("bias", [False, True])
def test_routed_call_is_route_and_experts(T, H, E, k, I, bias):
    """Bit for bit, below and above the sort's 4096 pairs, every output included."""
    g = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").to(BF)
    wr = (0.1 * torch.randn(E, H, generator=g, device="cuda")).to(BF)
    lb = torch.randn(E, generator=g, device="cuda") if bias else None
    w8 = B.I8Weights(*[(torch.randn(E, n, m, generator=g, device="cuda") * m**-0.5).to(BF)
                       for n, m in ((I, H), (I, H), (H, I))])
    w = [*w8.gate, *w8.up, *w8.down]
    s, M = B.shape(T, H, E, k, I, BF), T * k
    nb = B.moe_i8_workspace_bytes(s)

    def buffers():
        i32 = lambda *d: torch.full(d, -9, dtype=torch.int32, device="cuda")
        f32 = lambda *d: torch.full(d, -9.0, device="cuda")
        i8 = lambda *d: torch.full(d, -9, dtype=torch.int8, device="cuda")
        bf = lambda *d: torch.full(d, -9.0, dtype=BF, device="cuda")
        return ([f32(T, E), i32(T, k), f32(T, k)], [i32(E), i32(E + 1), i32(M), i32(M), i32(M), f32(M), i8(T, H), f32(T),
                                                    i8(M, I), f32(M), bf(M, H), bf(T, H)],
                torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda"))

    (r0, e0, ws0), (r1, e1, ws1) = buffers(), buffers()
    B.moe_forward_fused_i8(s, x, wr, lb, *w, *r0, *e0, ws0)
    B.moe_route(s, x, wr, lb, *r1)
    B.moe_experts_i8(s, x, r1[1], r1[2], *w, *e1, ws1)
    for i, (a, b) in enumerate(zip(r0 + e0, r1 + e1)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i  # o_perm's form (shared8.h) looks like any bf16, NaN too
    assert not r0[0].eq(-9).any() and not e0[-1].eq(-9).all()
