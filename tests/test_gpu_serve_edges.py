"""GPU tests of the serving operators (include/moe_serve.h) at the ends of the
number range."""
import pytest
import torch

from mixture_experts_expert_amd import binding as B

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


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
