"""The decoding calls' binding, on the CPU: tensors that say they are on a GPU, and a library that is not called."""
import types

import pytest
import torch

from output_projection_cross_gb300 import decode

I32, BF16 = torch.int32, torch.bfloat16


class Reached(Exception):
    """The call got as far as the library."""


class OnGpu:
    """A CPU tensor that says it is on GPU `index`."""

    def __init__(self, t, index=0):
        self.t, self.index, self.is_cuda = t, index, index >= 0

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture(autouse=True)
def gpu0(monkeypatch):
    """GPU 0 is the current one; every call of the library raises Reached."""
    def reached(*_):
        raise Reached
    calls = {n: reached for n in dir(decode._calls) if n.startswith("lossk_")}
    for n in ("spans", "device"):
        if hasattr(decode._calls, n):
            calls[n] = getattr(decode._calls, n)
    monkeypatch.setattr(decode, "_calls", types.SimpleNamespace(**calls))
    monkeypatch.setattr(decode, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(decode, "_current_device", lambda: 0, raising=False)


def ws():
    return torch.zeros(1 << 16, dtype=torch.uint8)


def cache():
    return dict(table=torch.zeros(4, 3, dtype=I32), lens=torch.zeros(4, dtype=I32), ref=torch.zeros(9, dtype=I32))


def arguments(name):
    """The call's tensors and the rest of its arguments."""
    pool, pages = torch.zeros(2, 9, 4, 2, 8, dtype=BF16), torch.zeros(9, 4, 2, 8, dtype=BF16)
    if name == "lossk_beam_select":
        return dict(logits=torch.zeros(4, 10), scores=torch.zeros(2, 2), allow=torch.zeros(1, dtype=I32),
                    finished=torch.zeros(2, 2, dtype=torch.uint8), lengths=torch.zeros(2, 2, dtype=I32),
                    lse_out=torch.zeros(4), ws=ws(), out_parent=torch.zeros(2, 3, dtype=I32),
                    out_token=torch.zeros(2, 3, dtype=torch.int64), out_score=torch.zeros(2, 3),
                    out_finished=torch.zeros(2, 3, dtype=torch.uint8), out_length=torch.zeros(2, 3, dtype=I32)), dict(n_out=3)
    if name == "lossk_beam_gather":
        return dict(src=torch.zeros(2, 3, 4), parent=torch.zeros(2, 5, dtype=I32), dst=torch.zeros(2, 5, 4), ws=ws()), {}
    if name == "lossk_cache_fork":
        return dict(cache(), parent=torch.zeros(2, 3, dtype=I32), table_out=torch.zeros(6, 3, dtype=I32),
                    lens_out=torch.zeros(6, dtype=I32), ws=ws()), dict(page_size=4)
    if name == "lossk_cache_reserve":
        return dict(cache(), pool=pool, ws=ws()), dict(page_size=4)
    if name == "lossk_cache_free":
        return dict(cache(), drop=torch.zeros(4, dtype=torch.uint8), ws=ws()), dict(page_size=4)
    if name == "lossk_cache_compact":
        return dict(cache(), pool=pool, table_out=torch.zeros(4, 3, dtype=I32), ref_out=torch.zeros(9, dtype=I32),
                    n_live_out=torch.zeros(1, dtype=I32), ws=ws()), dict(page_size=4)
    if name == "lossk_cache_copy":
        return dict(src=torch.zeros(2, dtype=I32), dst=torch.zeros(2, dtype=I32), pool=pool, ws=ws()), {}
    c = cache()
    if name == "lossk_cache_write":
        return dict(k_new=torch.zeros(4, 2, 8, dtype=BF16), v_new=torch.zeros(4, 2, 8, dtype=BF16), k_pages=pages,
                    v_pages=pages.clone(), table=c["table"], lens=c["lens"], first=torch.zeros(5, dtype=I32), ws=ws()), {}
    assert name == "lossk_paged_attn"
    return dict(q=torch.zeros(4, 4, 8, dtype=BF16), k_pages=pages, v_pages=pages.clone(), table=c["table"],
                lens=c["lens"], out=torch.zeros(4, 4, 8, dtype=BF16), lse_out=torch.zeros(4, 4), ws=ws()), {}


NAMES = ["lossk_beam_select", "lossk_beam_gather", "lossk_cache_fork", "lossk_cache_reserve", "lossk_cache_free",
         "lossk_cache_compact", "lossk_cache_copy", "lossk_cache_write", "lossk_paged_attn"]


def call(name, tensors, rest):
    tensors = dict(tensors)
    out = {k[4:]: tensors.pop(k) for k in list(tensors) if k.startswith("out_")}
    return getattr(decode, name)(**tensors, **rest, **({"out": out} if out else {}))


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_is_on_the_current_gpu(name, monkeypatch):
    """The launches go to the current device, and addresses of another mean nothing there."""
    tensors, rest = arguments(name)
    with pytest.raises(Reached):
        call(name, {k: OnGpu(t) for k, t in tensors.items()}, rest)
    for other in (1, -1):                              # another GPU, the host
        for k in tensors:
            with pytest.raises(ValueError):
                call(name, {i: OnGpu(t, other if i == k else 0) for i, t in tensors.items()}, rest)
        with pytest.raises(ValueError):
            call(name, {i: OnGpu(t, other) for i, t in tensors.items()}, rest)
    monkeypatch.setattr(decode, "_current_device", lambda: 1, raising=False)
    with pytest.raises(ValueError):
        call(name, {k: OnGpu(t) for k, t in tensors.items()}, rest)


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_gpu(name):
    tensors, rest = arguments(name)
    stub = {k: OnGpu(t) for k, t in tensors.items()}
    with pytest.raises(Reached):
        call(name, stub, dict(rest, stream=types.SimpleNamespace(cuda_stream=0, device_index=0)))
    with pytest.raises(ValueError):
        call(name, stub, dict(rest, stream=types.SimpleNamespace(cuda_stream=0, device_index=1)))


# what each call makes where it is left out
MADE = {"lossk_beam_select": ["ws", "out_"], "lossk_beam_gather": ["ws", "dst"],
        "lossk_cache_fork": ["ws", "table_out", "lens_out"], "lossk_cache_reserve": ["ws"], "lossk_cache_free": ["ws"],
        "lossk_cache_compact": ["ws", "table_out", "ref_out", "n_live_out"], "lossk_cache_copy": ["ws"],
        "lossk_cache_write": ["ws"], "lossk_paged_attn": ["ws", "out"]}


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_makes_is_made_on_its_stream(name, monkeypatch):
    """Made on the current stream, a workspace would be zeroed there while the call runs on its own, and its
    memory given to the current stream's next allocation while the call still uses it."""
    side = types.SimpleNamespace(cuda_stream=0, device_index=0)
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
    monkeypatch.setattr(torch.cuda, "stream", Stream)
    for n in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, n, maker(getattr(torch, n)))
    tensors, rest = arguments(name)
    stub = {k: OnGpu(t) if not isinstance(t, OnGpu) else t for k, t in tensors.items()
            if not any(k == m or m.endswith("_") and k.startswith(m) for m in MADE[name])}
    made.clear()
    with pytest.raises(Reached):
        call(name, stub, dict(rest, stream=side))
    assert len(made) >= len(MADE[name]) and all(s is side for s in made)
    made.clear()
    with pytest.raises(Reached):
        call(name, stub, rest)
    assert all(s is None for s in made)
