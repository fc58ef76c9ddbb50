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
