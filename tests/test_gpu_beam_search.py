"""Beam search with all of its operators, as the example runs it, against the texts alone."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_logits_gb300")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "beam_search.py")
    spec = importlib.util.spec_from_file_location("beam_search", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _entries(s):
    """What every row should hold, from its text."""
    e = s.emb[s.texts.view(s.B * s.W, -1)[:, :s.length].long()]
    return torch.stack([e, torch.tanh(e.roll(1, -1))])


def _held(s):
    pos = torch.arange(s.length, device=s.device)
    ids = s.table[:, pos // s.page].long()
    assert int(ids.min()) >= 0
    return s.cache[:, ids, pos % s.page]


def _refs(s):
    live = s.table[s.table >= 0].long()
    return torch.bincount(live, minlength=s.N).to(torch.int32)


def _step_from_texts(s):
    """The next beams from the texts, in 64 bits: scores, parents, tokens, flags [B][W]."""
    B, W, V = s.B, s.W, s.V
    e = _entries(s).double()
    k, v = e[0], e[1]
    w = torch.softmax((k * k[:, -1:]).sum(-1) / math.sqrt(s.dim), 1)
    x = torch.tanh((w[:, :, None] * v).sum(1) + k[:, -1]) @ s.head.double().T
    text = s.texts.view(B * W, -1)[:, :s.length].long()
    seen = torch.zeros((B * W, V), dtype=torch.bool, device=s.device).scatter_(1, text, True)
    th = s.repetition.double()[:, None]
    x = torch.where(seen, torch.where(x > 0, x / th, x * th), x)
    c = (s.scores.double().view(-1, 1) + torch.log_softmax(x, 1)).view(B, W, V)
    ended = s.finished > 0
    c = c.masked_fill(ended[:, :, None], -math.inf)
    c[:, :, s.eos] = torch.where(ended, s.scores.double(), c[:, :, s.eos])
    score, at = c.view(B, W * V).sort(dim=1, descending=True, stable=True)
    return score[:, :W + 1], at[:, :W + 1] // V, at[:, :W + 1] % V, ended


@pytest.mark.parametrize("B,W,V,prompt,page", [(3, 4, 211, 13, 4), (2, 7, 997, 16, 8), (1, 1, 50, 1, 16)])
def test_steps_follow_the_texts(example, B, W, V, prompt, page):
    s = example.Search(B=B, W=W, V=V, prompt=prompt, page=page, room=24, seed=B + W)
    for _ in range(20):
        score, parents, tokens, ended = _step_from_texts(s)
        b = s.step()
        # the logits are fp32 sums over dim and length: about 1e-5 of a nat
        gap = (score[:, :-1] - score[:, 1:]).abs()
        sure = (gap > 1e-3).all(1)
        assert bool(((b.scores.double() - score[:, :W]).abs() < 1e-3)[score[:, :W] > -math.inf].all())
        assert torch.equal(b.parents[sure].long(), parents[:, :W][sure])
        assert torch.equal(b.tokens[sure].long(), tokens[:, :W][sure])
        assert torch.equal(b.finished > 0, ended.gather(1, b.parents.long()) | (b.tokens == s.eos))
        # the cache, the counts of pages and of tokens are those of the texts
        assert torch.equal(_held(s), _entries(s)) and torch.equal(s.refs, _refs(s))
        out = torch.nn.functional.one_hot(s.texts[:, :, s.start:s.length].long(), V).sum(2)
        assert torch.equal((s.counts.long() & 0x7FFF), out)
        assert int(s.status) == 0


def test_ended_requests_leave_the_others_alone(example):
    s = example.Search(B=4, W=3, V=101, prompt=9, page=4, room=30, seed=5)
    for _ in range(10):
        s.step()
    before = _held(s)
    gone = torch.tensor([1, 0, 0, 1], device=s.device)
    c = s.end(gone)
    left = gone[:, None].expand(4, 3).reshape(-1) == 0
    assert int(s.table[~left].max()) == -1
    assert torch.equal(s.refs, _refs(s)) and int(c.live) == int((s.refs > 0).sum())
    assert int(s.table.max()) < int(c.live)
    table = s.table
    s.table = table.clamp(min=0)
    assert torch.equal(_held(s)[:, left], before[:, left])
    s.table = table
    assert int(s.status) == 0


def test_example_runs(example):
    s = example.main(30)
    assert s.length == s.start + 30 and int(s.status) == 0
