"""Ckpt8Stage on a stream of the caller's: what goes in may be dropped after the call,
and what it makes lies in no memory that the current stream still reads."""
import pytest
import torch

from mixture_experts_expert_amd import binding as B

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
DIMS = (4096, 1024, 4, 2, 1024)  # x and dy of 8 MiB, gradients of 16: blocks of their own in torch's allocator
GRADS = ("dx", "dw_gate", "dw_up", "dw_down", "d_logits")


def _busy(stream):
    """About 50 ms of waiting on the stream, so that what follows there runs late."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)


def _layer(seed):
    T, H, E, k, I = DIMS
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *d: torch.randn(*d, generator=g, device="cuda")
    return (r(T, H).to(BF), [(0.1 * r(E, H)).to(BF), *[(r(E, n, m) * m**-0.5).to(BF) for n, m in ((I, H), (I, H), (H, I))]],
            r(T, H).to(BF))


@pytest.mark.parametrize("x8", [False, True])
def test_inputs_of_another_stream_outlive_the_call(x8):
    x, w, dy = _layer(1)
    st = B.Ckpt8Stage(*DIMS, x8=x8)
    st.forward(x, *w)
    st.backward(dy)
    want = {n: st.buf[n].clone() for n in GRADS}
    other, w2, _ = _layer(2)
    side = torch.cuda.Stream()
    given = [t.clone() for t in (x, *w, dy)]
    for n in GRADS:
        st.buf[n].zero_()
    torch.cuda.synchronize()
    _busy(side)
    st.forward(given[0], *given[1:5], stream=side)
    st.backward(given[5], stream=side)
    del given
    st.forward(other, *w2, stream=side)  # the stage lets go of the first x and weights, too
    again = [torch.zeros_like(t) for t in (x, *w, dy)]
    torch.cuda.synchronize()
    assert len(again) == 6
    for n in GRADS:
        assert torch.equal(st.buf[n], want[n]), n


def test_first_gradients_keep_off_freed_memory():
    T, H, E, k, I = DIMS
    x, w, dy = _layer(3)
    ref = B.Ckpt8Stage(*DIMS)
    ref.forward(x, *w)
    ref.backward(dy)
    st = B.Ckpt8Stage(*DIMS)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = [torch.full((E, I, H), 7.0, device="cuda") for _ in range(3)] + [torch.full((T, H), 7.0, dtype=BF, device="cuda")]
    torch.cuda.synchronize()
    _busy(here)
    kept = [f + 1 for f in freed]
    del freed
    st.forward(x, *w, stream=side)
    st.backward(dy, stream=side)
    torch.cuda.synchronize()
    assert all(t.eq(8).all() for t in kept)
    for n in GRADS:
        assert torch.equal(st.buf[n], ref.buf[n]), n


@pytest.mark.parametrize("T, E, I", [(500, 16, 320), (700, 4, 320), (4096, 16, 768)])
def test_activations_are_the_plain_steps_at_full_depth(T, E, I):
    """a, before anything rounds it away further, beside MoEStage's at H = 2048: by 128-row tiles (62 rows per expert on
    average) and by 256-row ones."""
    H, k = 2048, 2
    g = torch.Generator("cuda").manual_seed(T)
    r = lambda *d: torch.randn(*d, generator=g, device="cuda")
    x, wr = r(T, H).to(BF), (0.1 * r(E, H)).to(BF)
    w = [(r(E, n, m) * m**-0.5).to(BF) for n, m in ((I, H), (I, H), (H, I))]
    st = B.Ckpt8Stage(T, H, E, k, I)
    plain = B.MoEStage(T, H, E, k, I, BF, gather_fused=True, dy_fused=True)
    y, want = st.forward(x, wr, *w), plain.forward(x, wr, *w)
    assert torch.equal(st.scratch["a"], plain.buf["a"])
    assert torch.equal(y, want)
