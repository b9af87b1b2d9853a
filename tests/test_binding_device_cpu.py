"""The losses' binding refuses inputs and workspaces of another GPU than the current one (CPU: tensors that say
where they are, and a library that is not called)."""
import types

import pytest
import torch

from output_projection_cross_gb300 import lossk


class Reached(Exception):
    """The call got as far as the library."""


class OnGpu:
    def __init__(self, t, index=0):
        self.t, self.index, self.is_cuda = t, index, index >= 0

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture(autouse=True)
def gpu0(monkeypatch):
    def reached(*_):
        raise Reached
    monkeypatch.setattr(lossk, "lib", types.SimpleNamespace(lossk_ce_fwd=reached, lossk_ce_from_logits=reached,
                                                            lossk_distill_from_logits=reached))
    monkeypatch.setattr(lossk, "_stream", lambda stream: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def arguments(name):
    y = torch.zeros(3, dtype=torch.int64)
    mask, ws = torch.ones(3, dtype=torch.uint8), torch.zeros(1 << 12, dtype=torch.uint8)
    out = dict(lse_out=torch.zeros(3), scalars_out=torch.zeros(3, dtype=torch.float64))
    if name == "lossk_ce_fwd":
        return dict(hidden=torch.zeros(3, 4), weight=torch.zeros(5, 4), targets=y, loss_mask=mask, ws=ws), \
            dict(out, ce_out=torch.zeros(3))
    if name == "lossk_ce_from_logits":
        return dict(logits=torch.zeros(3, 5), targets=y, loss_mask=mask, ws=ws), dict(out, ce_out=torch.zeros(3))
    return dict(logits=torch.zeros(3, 5), teacher_logits=torch.zeros(3, 5), loss_mask=mask, ws=ws), \
        dict(out, per_token_out=torch.zeros(3), want_grad=False)


@pytest.mark.parametrize("name", ["lossk_ce_fwd", "lossk_ce_from_logits", "lossk_distill_from_logits"])
def test_inputs_of_another_gpu(name):
    f = getattr(lossk, name)
    tensors, out = arguments(name)
    out = {k: OnGpu(t) if isinstance(t, torch.Tensor) else t for k, t in out.items()}
    with pytest.raises(Reached):
        f(**{k: OnGpu(t) for k, t in tensors.items()}, **out)
    for other in (1, -1):
        for k in tensors:
            with pytest.raises(ValueError):
                f(**{i: OnGpu(t, other if i == k else 0) for i, t in tensors.items()}, **out)


@pytest.mark.parametrize("name", ["lossk_ce_fwd", "lossk_ce_from_logits", "lossk_distill_from_logits"])
def test_what_a_call_makes_is_made_on_its_stream(name, monkeypatch):
    """Made on the current stream, a workspace would be zeroed there while the call runs on its own, and its
    memory given to the current stream's next allocation while the call still uses it."""
    current, made = [None], []

    class Stream:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *_):
            current.pop()

    def maker(make):
        def f(*args, device=None, **kw):
            made.append(current[-1])
            return OnGpu(make(*args, **kw))
        return f
    tensors, out = arguments(name)
    stub = {k: OnGpu(t) for k, t in tensors.items() if k != "ws"}
    monkeypatch.setattr(lossk, "lossk_workspace_bytes", lambda *_: 1 << 12)
    monkeypatch.setattr(torch.cuda, "stream", Stream)
    for n in ("empty", "zeros"):
        monkeypatch.setattr(torch, n, maker(getattr(torch, n)))
    rest = {"want_grad": False} if "want_grad" in out else {}
    for stream in ("side", None):
        made.clear()
        with pytest.raises(Reached):
            getattr(lossk, name)(**stub, **rest, stream=stream)
        assert len(made) >= 3 and all(s is stream for s in made)
