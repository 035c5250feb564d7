"""The calls of beam search and of the pages run on the stream that they are given and on their
tensors' device, whatever the order of the arguments and however they are passed."""
import contextlib
import inspect
import types

import pytest
import torch

import speculative_decoding_verification_logits_gb300 as sd
from speculative_decoding_verification_logits_gb300 import beam, kv

CALLS = ("beam_select", "beam_reorder", "kv_fork", "kv_extend", "kv_free", "kv_compact", "kv_copy")


class OnDevice(torch.Tensor):
    """A host tensor that says it is on the second GPU."""
    is_cuda = True
    device = torch.device("cuda:1")

    def get_device(self):
        return 1


@pytest.fixture
def entered(monkeypatch):
    """The streams and devices that are made current, in order; the first GPU is current before."""
    seen = []

    def enter(kind):
        @contextlib.contextmanager
        def current(what):
            seen.append((kind, what))
            yield
        return current

    monkeypatch.setattr(torch.cuda, "stream", enter("stream"))
    monkeypatch.setattr(torch.cuda, "device", enter("device"))
    monkeypatch.setattr(kv, "_device", lambda: 0)
    return seen


@pytest.mark.parametrize("name", CALLS)
def test_stream_and_device_do_not_depend_on_the_order_of_arguments(entered, name):
    wrapped = getattr(sd, name).__wrapped__
    names = list(inspect.signature(wrapped).parameters)
    body = types.SimpleNamespace(args=None)

    def plain(*args, **kwargs):
        body.args = inspect.signature(wrapped).bind(*args, **kwargs).arguments

    plain.__signature__ = inspect.signature(wrapped)
    call = kv._on_device(plain)
    x = torch.zeros(3).as_subclass(OnDevice)
    side = types.SimpleNamespace(device=x.device)
    first = [x] if name == "kv_copy" else x
    given = {n: 4 for n in names[1:]}
    for kwargs in ({names[0]: first, **given}, {**given, names[0]: first}, None):
        for stream in (side, None):
            entered.clear()
            more = {} if stream is None else {"stream": stream}
            if kwargs is None:
                call(first, **given, **more)
            else:
                call(**more, **kwargs)
            assert entered == [("stream", side) if stream else ("device", x.device)]
            assert list(body.args) == names and body.args[names[0]] is first
    for other in (torch.device("cuda:0"), torch.device("cuda:2")):
        with pytest.raises(ValueError, match="stream is on"):
            call(stream=types.SimpleNamespace(device=other), **given, **{names[0]: first})


@pytest.mark.parametrize("pick", [iter, lambda v: {i: t for i, t in enumerate(v)}.values()])
def test_states_and_caches_from_an_iterator(entered, pick):
    got = []
    call = kv._on_device(lambda states, k: got.append(tuple(states)))
    x, y = (torch.zeros(2).as_subclass(OnDevice) for _ in range(2))
    side = types.SimpleNamespace(device=x.device)
    call(pick([x, y]), 3, stream=side)
    call(k=3, states=pick([x, y]), stream=side)
    call(k=3, states=pick([x, y]))
    assert entered == [("stream", side)] * 2 + [("device", x.device)]
    assert all(len(g) == 2 and g[0] is x and g[1] is y for g in got) and len(got) == 3


@pytest.mark.gpu
def test_keyword_calls_launch_on_their_stream(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev, used = torch.device("cuda:0"), []
    for module in (beam, kv):
        real = module._stream_of
        monkeypatch.setattr(module, "_stream_of", lambda d, real=real: used.append(real(d)) or used[-1])
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
    table = lambda: i(0, 1, -1, 2, -1, -1).view(2, 3)
    refs = lambda: i(1, 1, 1, 0, 0, 0)
    x = torch.randn((2, 3, 50), device=dev)
    zero, state = torch.zeros((2, 3), device=dev), torch.arange(12, device=dev).view(2, 3, 2)
    parents = i(0, 2, 1, 1, 1, 0).view(2, 3)
    cache = torch.zeros((1, 6, 4, 2), device=dev)
    first = {
        "beam_select": dict(logits=x, scores=zero, k=4),
        "beam_reorder": dict(states=state, parents=parents),
        "kv_fork": dict(block_table=table(), kv_len=i(6, 3), parents=i(1, 0, 0), refs=refs(), page_size=4),
        "kv_extend": dict(block_table=table(), kv_len=i(6, 3), refs=refs(), page_size=4, append=2),
        "kv_free": dict(pages=i(2, -1), refs=refs(), which=None),
        "kv_compact": dict(refs=refs(), status=None),
        "kv_copy": dict(caches=cache, src=i(2), dst=i(4), heads_first=False),
    }
    side = torch.cuda.Stream(dev)
    for name, kwargs in first.items():
        kwargs = dict(reversed(kwargs.items()))
        side.wait_stream(torch.cuda.current_stream(dev))
        used.clear()
        getattr(sd, name)(stream=side, **kwargs)
        assert used == [side.cuda_stream], name
        torch.cuda.current_stream(dev).wait_stream(side)
        used.clear()
        getattr(sd, name)(**kwargs)
        assert used == [torch.cuda.current_stream(dev).cuda_stream], name
    # a list that is made on the way
    used.clear()
    got = sd.beam_reorder((s for s in (state, state + 1)), parents, stream=side)
    side.synchronize()
    assert used == [side.cuda_stream]
    want = state.gather(1, parents.long()[..., None].expand(2, 3, 2))
    assert torch.equal(got[0], want) and torch.equal(got[1], want + 1)
