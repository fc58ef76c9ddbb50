"""Ckpt8Stage's care for memory on a stream of the caller's, on the CPU: the kernels
are left out, and what the stage tells torch's allocator is looked at."""
import contextlib

import pytest
import torch

BF = torch.bfloat16


class Stream:
    cuda_stream = 0


@pytest.fixture
def calls(monkeypatch):
    """The binding with no kernels behind it; (recorded, entered): the tensors recorded on a stream, and the streams
    that allocations were made under."""
    from mixture_experts_expert_amd import binding as B
    for name in [n for n in vars(B) if n.startswith("moe_") and callable(getattr(B, n))
                 and n not in ("moe_shape", "moe_workspace_bytes", "moe_ckpt8_workspace_bytes")]:
        monkeypatch.setattr(B, name, lambda *a, **k: None)
    monkeypatch.setattr(B.Ckpt8Stage, "_check_tensors", lambda self, *named: None)
    recorded, entered = [], []

    @contextlib.contextmanager
    def under(stream):
        entered.append(stream)
        yield

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    return B, recorded, entered


def _inputs():
    z = lambda *d, dt=BF: torch.zeros(*d, dtype=dt)
    return z(8, 128), (z(4, 128), z(4, 64, 128), z(4, 64, 128), z(4, 128, 64), z(4, dt=torch.float32)), z(8, 128)


@pytest.mark.parametrize("x8", [False, True])
def test_inputs_are_recorded_on_the_stream(calls, x8):
    B, recorded, entered = calls
    st = B.Ckpt8Stage(8, 128, 4, 2, 64, device="cpu", x8=x8)
    x, w, dy = _inputs()
    first, second = Stream(), Stream()
    st.forward(x, *w, stream=first)
    assert {(t.data_ptr(), first) for t in (x, *w)} <= set(recorded)
    del recorded[:]
    st.backward(dy, stream=second)  # reads the weights again, and x if that is kept as it is
    assert {(t.data_ptr(), second) for t in (dy, *w[1:4], *(() if x8 else (x,)))} <= set(recorded)
    assert entered == [second]  # the gradients, made at the first backward
    st.backward(dy, stream=first)
    assert entered == [second]


def test_nothing_is_recorded_on_the_current_stream(calls):
    B, recorded, _ = calls
    st = B.Ckpt8Stage(8, 128, 4, 2, 64, device="cpu")
    x, w, dy = _inputs()
    st.forward(x, *w)
    st.backward(dy)
    assert recorded == []


def test_scratch_of_other_types_is_refused():
    """A shared buffer of fewer bytes would be written past its end."""
    from mixture_experts_expert_amd import binding as B
    dims, scratch = (8, 128, 4, 2, 64), {}
    B.Ckpt8Stage(*dims, device="cpu", x8=True, scratch=scratch)
    B.Ckpt8Stage(*dims, device="cpu", x8=True, scratch=scratch)
    for n, t in scratch.items():
        for bad in (t.to(torch.int8 if t.dtype == BF else BF), torch.stack((t, t), -1)[..., 0]):
            with pytest.raises(ValueError, match=f"scratch {n}"):
                B.Ckpt8Stage(*dims, device="cpu", x8=True, scratch={**scratch, n: bad})


def test_tensors_off_a_16_byte_boundary_are_refused_before_any_launch():
    from mixture_experts_expert_amd import binding as B
    st = B.Ckpt8Stage(8, 128, 4, 2, 64, device="cpu")
    x, w, dy = _inputs()
    good = dict(zip(("x", "w_router", "w_gate", "w_up", "w_down", "logit_bias"), (x, *w)))
    for name, t in good.items():
        off = torch.cat((t.flatten()[:1], t.flatten()))[1:].view(t.shape)
        with pytest.raises(ValueError, match=f"{name} has to start"):
            st.forward(**{**good, name: off})
    with pytest.raises(ValueError, match="dy has to start"):
        st.backward(torch.cat((dy.flatten()[:1], dy.flatten()))[1:].view(dy.shape))


@pytest.mark.parametrize("H, I", [(1 << 15, 1 << 15), (64, 1 << 22), (1 << 22, 64)])
def test_no_workspace_for_a_shape_that_the_call_rejects(H, I):
    """One expert's weight, or 256 rows of g, past 2 GiB."""
    from mixture_experts_expert_amd import binding as B
    s = B.shape(1, H, 1, 1, I, BF)
    assert B.moe_workspace_bytes(s) > 0 and B.moe_ckpt8_workspace_bytes(s) == 0
    with pytest.raises(B.MoEError):
        B.Ckpt8Stage(1, H, 1, 1, I, device="meta")
