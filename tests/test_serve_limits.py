"""Limits of include/moe_serve.h on the host: empty calls, the largest launches,
and the shapes of large models. No call here reaches a launch."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced
OK, EINVAL, EUNSUPPORTED, EWORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def B():
    from mixture_experts_expert_amd import binding
    return binding


def test_no_rows_need_no_pointers(B):
    """An empty tensor has none."""
    assert B.lib.moe_quantize_fp8_block_rows(0, 64, None, None, None, None) == OK
    assert B.lib.moe_quantize_fp8_block_rows(0, 12, None, None, None, None) == EINVAL
    gemm = lambda E, off, wq: B.lib.moe_gemm_fp8_block(0, E, 64, 64, None, None, off, wq, FAKE, None, None, None)
    assert gemm(1, None, FAKE) == OK and gemm(2, FAKE, FAKE) == OK
    assert gemm(2, None, FAKE) == EINVAL and gemm(2, FAKE, None) == EINVAL


@pytest.mark.parametrize("rows", [(1 << 28) - 1, (1 << 28) - 15])
def test_quantize_rows_whole_workgroups(B, rows):
    """The limit counts the launch's threads, rounded up to workgroups of 16 blocks."""
    assert B.lib.moe_quantize_fp8_block_rows(rows, 8, FAKE, FAKE, FAKE, None) == EUNSUPPORTED


def test_quantize_weights_largest_product(B):
    top = (1 << 31) - 1
    for E, N, K in ((255, top, top - 7), (129, top, top - 7), (top, 128, top - 7), (256, top, top - 7)):
        assert B.lib.moe_quantize_fp8_block_weights(E, N, K, FAKE, FAKE, FAKE, None) == EUNSUPPORTED, (E, N, K)


LARGE = (256, 7168, 2048, 8), (160, 6144, 2560, 8), (1024, 4096, 4096, 4)  # E, H, I, k: all experts pass 2^31 weights


@pytest.mark.parametrize("E,H,I,k", LARGE)
def test_layers_of_large_models(B, E, H, I, k):
    """Only one expert's weights have to stay below 2^31: nothing about the training calls' limits."""
    for T in (1, 64):
        assert B.moe_few_workspace_bytes(B.shape(T, H, E, k, I, "bf16")) > 0
    s, too_wide = B.shape(4096, H, E, k, I, "bf16"), B.shape(4096, 1 << 16, E, k, 1 << 15, "bf16")
    ws = 1 << 40
    calls = [(B.lib.moe_experts_fp8_block, 22), (B.lib.moe_forward_fused_fp8_block, 25)]
    for fn, n in calls:  # the shape is accepted: only the workspace is short, and only a wider expert is refused
        assert fn(s, *[FAKE] * n, 16, None) == EWORKSPACE
        assert fn(too_wide, *[FAKE] * n, ws, None) == EUNSUPPORTED
    assert B.lib.moe_gemm_gate_up_fp8_block(s, *[None] * 11) == EINVAL
    assert B.lib.moe_gemm_gate_up_fp8_block(too_wide, *[FAKE] * 10, None) == EUNSUPPORTED
    assert B.moe_few_workspace_bytes(B.shape(8, 1 << 16, E, k, 1 << 15, "bf16")) == 0


@pytest.mark.parametrize("T,E,k,need", [(1, 4, 1, 256), (128, 64, 8, 256), (129, 64, 8, 512), (129, 65, 8, 768),
                                        (8192, 128, 8, 32768)])
def test_workspace_of_the_expert_stage(B, T, E, k, need):
    """E counts per 1024 (token, slot) pairs, in units of 256 bytes: no training buffers."""
    s = B.shape(T, 2048, E, k, 768, "bf16")
    assert B.fp8_block_workspace_bytes(s) == need <= B.moe_workspace_bytes(s)
    for fn, n in ((B.lib.moe_experts_fp8_block, 22), (B.lib.moe_forward_fused_fp8_block, 25)):
        assert fn(s, *[FAKE] * n, need - 1, None) == EWORKSPACE


def test_stage_of_a_large_layer(B):
    E, H, I, k = LARGE[0]
    m = lambda *d, dt: torch.empty(*d, dtype=dt, device="meta")
    pairs = [(m(E, a, b, dt=torch.uint8), m(E, a // 128, b // 128, dt=torch.float32)) for a, b in ((I, H), (I, H), (H, I))]
    stage = B.ServingStage(4096, k, m(E, H, dt=torch.bfloat16), B.FP8BlockWeights(stored=pairs))
    assert stage.few_T == 64 and stage.ws.numel() == 4 * E * 4096 * k // 1024
    with pytest.raises(B.MoEError):
        B.ServingStage(100, 0, m(E, H, dt=torch.bfloat16), B.FP8BlockWeights(stored=pairs))
