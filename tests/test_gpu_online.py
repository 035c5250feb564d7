"""The logit operators together, as the example of a drafter trained on its rounds runs them."""
import pytest
import torch

from tests import logits_ref as ref

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_logits_gb300")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "online_drafter.py")
    spec = importlib.util.spec_from_file_location("online_drafter", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_drafter_learns_from_its_rounds(example):
    # an untrained drafter keeps about one token a round; a trained one several
    s = example.Round()
    taus, losses = [], []
    for _ in range(150):
        r, loss = s.step()
        assert int(r.status.item()) == 0
        taus.append(float(r.tau.float().mean()))
        losses.append(float(loss))
    first, last = sum(taus[:10]) / 10, sum(taus[-30:]) / 30
    assert first < 1.6 and last > first + 0.5, (first, last)
    assert losses[-1] < 0.5 * losses[0]


def test_counts_follow_the_emitted_tokens(example):
    s = example.Round(B=5, K=3, V=307, dim=16, seed=3)
    start, emitted = s.counts.clone().cpu(), []
    for _ in range(12):
        r, _ = s.step()
        emitted.append((r.out_tokens.cpu(), r.tau.cpu()))
    want = start
    for tokens, tau in emitted:
        want = ref.token_counts_add(want, tokens, tau)
    assert torch.equal(s.counts.cpu(), want)


def test_masked_tokens_are_never_emitted(example):
    s = example.Round(B=8, K=4, V=307, dim=16, seed=4)
    words = s.mask.cpu().long()
    for _ in range(12):
        r, _ = s.step()
        for b in range(8):
            for t in r.out_tokens[b, :int(r.tau[b])].tolist():
                assert (int(words[b, t // 32]) >> (t % 32)) & 1


def test_drafted_rows_and_target_rows_are_processed_alike(example):
    # a draft's row drawn on its own (base = j) is what the round's rows give it (base = 0)
    s = example.Round(B=4, K=5, V=509, dim=16, seed=5)
    tokens, drawn = s.draft()
    context = torch.cat([s.last[:, None], tokens[:, :-1]], 1)
    rows = s.rows(s.drafter.detach(), context)
    again = sd.process_logits(rows, counts=s.counts, prev=tokens, **s.rules)
    assert torch.equal(again, drawn)
