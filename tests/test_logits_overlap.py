"""Which outputs the logit operators take: memory of their own, the input itself, or rows that
lie between the input's (no GPU: the rule works on addresses and strides)."""
import itertools
import random

import pytest
import torch

from speculative_decoding_verification_logits_gb300 import logits as L


def _elements(t):
    """The addresses of a tensor's elements, one by one."""
    return {t.data_ptr() + t.element_size() * sum(i * s for i, s in zip(at, t.stride()))
            for at in itertools.product(*map(range, t.shape))}


def test_overlap_by_hand():
    V = 5
    buf = torch.zeros(4, 2 * V)
    assert not L._overlap(buf[:, :V], buf[:, V:])           # side by side
    assert not L._overlap(buf[:, V:], buf[:, :V])
    assert L._overlap(buf[:, :V], buf[:, V - 1:2 * V - 1])  # one element of a row in common
    assert L._overlap(buf[:, :V], buf[:, :V])
    assert not L._overlap(buf[::2], buf[1::2])              # every other row
    assert L._overlap(buf[:3], buf[1:])
    wide = torch.zeros(3, 4, 2 * V)
    assert not L._overlap(wide[..., :V], wide[..., V:])
    assert not L._overlap(wide[:, ::2], wide[:, 1::2])
    assert not L._overlap(wide.transpose(0, 1)[..., :V], wide.transpose(0, 1)[..., V:])
    assert not L._overlap(torch.zeros(0, V), torch.zeros(0, V))
    one = torch.zeros(1, V)
    assert L._overlap(one.expand(4, V), one.expand(4, V))
    assert not L._overlap(one.expand(4, V), buf[:, :V])


@pytest.mark.parametrize("seed", range(4))
def test_overlap_against_every_element(seed):
    rng = random.Random(seed)
    base = torch.zeros(400)
    found = set()
    for _ in range(300):
        A, B, V = rng.randint(1, 4), rng.randint(1, 4), rng.randint(1, 6)
        view = lambda: torch.as_strided(base, (A, B, V),
                                        (rng.choice([0, V, 2 * V, 13, 30]),
                                         rng.choice([0, V, 2 * V + 1, 7, 40]), 1),
                                        rng.randint(0, 60))
        x, y = view(), view()
        if rng.random() < 0.3:
            x, y = x[:, 0], y[:, 0]
        want = bool(_elements(x) & _elements(y))
        assert L._overlap(x, y) == want, (x.shape, x.stride(), y.stride())
        found.add((want, L._apart(x, y)))
    # both answers, and both ways to a no
    assert found == {(True, False), (False, False), (False, True)}


def test_the_input_itself_is_known_whatever_its_idle_strides():
    x = torch.zeros(3, 1, 7)
    y = torch.as_strided(x, (3, 1, 7), (7, 1, 1))
    assert x.stride() != y.stride() and L._same(x, y) and L._same(y, x)
    assert not L._same(x, x[:, :, 1:]) and not L._same(torch.zeros(4, 6)[::2], torch.zeros(2, 6))
    b = torch.zeros(4, 6)
    assert not L._same(b[:2], torch.as_strided(b, (2, 6), (12, 1)))
