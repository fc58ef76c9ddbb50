"""ServingStage and FP8BlockWeights refuse tensors that the kernels would read
wrongly, before any call of the library (no GPU needed)."""
import pytest
import torch

BF = torch.bfloat16
E, I, H, K = 4, 64, 128, 2


@pytest.fixture(scope="module")
def B():
    from mixture_experts_expert_amd import binding
    return binding


def _z(*d, dt=BF, dev="cpu"):
    return torch.zeros(*d, dtype=dt, device=dev)


def _bf16(dev="cpu"):
    return [_z(E, I, H, dev=dev), _z(E, I, H, dev=dev), _z(E, H, I, dev=dev)]


def _stored(dt=torch.uint8, dev="cpu", scale_dev=None):
    f = lambda *d: _z(*d, dt=torch.float32, dev=scale_dev or dev)
    return [(_z(E, I, H, dt=dt, dev=dev), f(E, 1, 1)), (_z(E, I, H, dt=dt, dev=dev), f(E, 1, 1)),
            (_z(E, H, I, dt=dt, dev=dev), f(E, 1, 1))]


def test_bias_has_to_be_contiguous(B):
    wide = _z(E, 2, dt=torch.float32)
    B.ServingStage(8, K, _z(E, H), _bf16(), wide[:, 0].contiguous())
    for bias in (wide[:, 0], _z(1, dt=torch.float32).expand(E)):
        with pytest.raises(ValueError):
            B.ServingStage(8, K, _z(E, H), _bf16(), bias)


def test_one_device(B):
    """`meta` stands for any device but the weights' own."""
    bias = _z(E, dt=torch.float32)
    for weights, router, b in ((_bf16(), _z(E, H, dev="meta"), bias), (_bf16(), _z(E, H), bias.to("meta")),
                               (_bf16()[:2] + _bf16("meta")[2:], _z(E, H), bias), (_bf16("meta"), _z(E, H), bias),
                               (B.FP8BlockWeights(stored=_stored(scale_dev="meta")), _z(E, H), bias),
                               (B.FP8BlockWeights(stored=_stored()[:2] + _stored(dev="meta")[2:]), _z(E, H), bias)):
        with pytest.raises(ValueError):
            B.ServingStage(8, K, router, weights, b)


@pytest.mark.parametrize("dt", [torch.int8, torch.bool, torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz])
def test_codes_of_another_format(B, dt):
    for good in (torch.uint8, torch.float8_e4m3fn):
        B.ServingStage(8, K, _z(E, H), B.FP8BlockWeights(stored=_stored(good)))
    with pytest.raises(ValueError):
        B.ServingStage(8, K, _z(E, H), B.FP8BlockWeights(stored=_stored(dt)))
    with pytest.raises(ValueError):
        B.ServingStage(8, K, _z(E, H), B.FP8BlockWeights(stored=_stored()[:2] + _stored(dt)[2:]))


def test_nothing_runs_on_host_tensors(B):
    for weights in (_bf16(), B.FP8BlockWeights(stored=_stored())):
        stage = B.ServingStage(8, K, _z(E, H), weights)
        with pytest.raises(ValueError):
            stage.forward(_z(3, H))
    with pytest.raises(ValueError):
        B.FP8BlockWeights(*_bf16())


def test_shape_of_x(B):
    stage = B.ServingStage(8, K, _z(E, H), _bf16())
    for x in (torch.tensor(1.0, dtype=BF), _z(H), _z(1, 2, H)):
        with pytest.raises(ValueError):
            stage.forward(x)
