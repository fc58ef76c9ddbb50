"""The codes of g and u over the range of fp32 (include/moe_ckpt8.h), in both forms of
the gate/up product: few rows per expert and 256 and more.

One product per sum, of a power of two and a bf16 number: the sums are exact. A code is
off by less than 0.5 + 2^-15 of a step, the scale by 2^-22 (the product with 1 / 127
and its constant), which 127 codes take to 2^-15 of a step."""
import pytest
import torch

from mixture_experts_expert_amd import binding as B

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("exponent", [-118, -80, -64, 0, 64, 100, 120, 125, 126, 127])
@pytest.mark.parametrize("T", [40, 600])  # 128-row tiles, 256-row tiles
def test_blocks_of_every_magnitude(T, exponent):
    H, I, half = 64, 192, exponent // 2
    g = torch.Generator().manual_seed(exponent + 200)
    x = torch.zeros(T, H)
    x[:, 5] = 2.0**half
    mantissa = torch.rand(2, 1, I, generator=g) * 1.98 - 0.99
    mantissa[:, :, ::64] = 0.99  # a block's largest: just below 2^exponent
    w = torch.zeros(2, 1, I, H)
    w[..., 5] = mantissa * 2.0**(exponent - half)
    x, w = x.to(BF), w.to(BF)
    s = B.shape(T, H, 1, 1, I, BF)
    i8 = lambda *d: torch.full(d, 7, dtype=torch.int8, device="cuda")
    f32 = lambda *d: torch.full(d, -1.0, device="cuda")
    q, sc, a = (i8(T, I), i8(T, I)), (f32(T, I // 64), f32(T, I // 64)), torch.empty(T, I, dtype=BF, device="cuda")
    token = torch.randperm(T, generator=g).to(torch.int32).cuda()
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    B.moe_gemm_gate_up_ckpt8(s, x.cuda(), token, off, w[0].cuda(), w[1].cuda(), q[0], sc[0], q[1], sc[1], a)
    for i in range(2):
        v = x[:, 5:6].double() @ w[i, 0, :, 5:6].double().T
        top = v.abs().view(T, -1, 64).amax(2)
        got, scale = q[i].cpu().double(), sc[i].cpu().double()
        assert (scale - top / 127).abs().le(top / 127 * 2.0**-22).all()
        back = got * scale.repeat_interleave(64, 1)
        step = (top / 127).repeat_interleave(64, 1)
        assert (back - v).abs().le(step * (0.5 + 2.0**-15 + 2.0**-15)).all()
        assert got.abs().view(T, -1, 64).amax(2).eq(127).all()
