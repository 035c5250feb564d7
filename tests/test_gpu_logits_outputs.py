"""The logit operators with outputs that lie between their input's rows, and in place with
strides that say the same in another way."""
import pytest
import torch

from tests import test_gpu_logits as base

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_logits_gb300")

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _rows(shape, dtype, dev):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(6)) * 3).to(dtype).to(dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1001, 4096])
@pytest.mark.parametrize("N", [5, 90])
def test_outputs_between_the_rows(dev, dtype, V, N):
    x = _rows((N, V), dtype, dev)
    pen = dict(counts=torch.ones((N, V), dtype=torch.int16, device=dev),
               presence=torch.full((N,), 0.5, device=dev))
    t = sd.top_logits(_rows((N, V), F32, dev) + 1, 9)
    want = sd.process_logits(x, **pen)
    learn = base._want_distill(x.cpu(), t.ids.cpu(), t.vals.cpu(), t.rest.cpu(), 1.0, None)
    buf = torch.empty((N, 2 * V), dtype=dtype, device=dev)
    for at, to in ((slice(0, V), slice(V, None)), (slice(V, None), slice(0, V))):
        buf[:, at] = x
        assert torch.equal(sd.process_logits(buf[:, at], out=buf[:, to], **pen), want)
        assert torch.equal(buf[:, at], x)
        loss, g = sd.distill_grad(buf[:, at], t.ids, t.vals, t.rest, grad=buf[:, to])
        assert g.data_ptr() == buf[:, to].data_ptr() and torch.equal(buf[:, at], x)
        base._near_distill(loss, g, learn)
    for out in (buf[:, 1:V + 1], buf[:, V - 1:2 * V - 1]):
        with pytest.raises(ValueError, match="overlaps"):
            sd.process_logits(buf[:, :V], out=out, **pen)
        with pytest.raises(ValueError, match="overlaps"):
            sd.distill_grad(buf[:, :V], t.ids, t.vals, t.rest, grad=out)


def test_in_place_with_idle_strides(dev):
    B, V = 3, 700
    x = _rows((B, 1, V), BF, dev)
    pres, prev = torch.full((B,), 0.5, device=dev), torch.zeros((B, 1), dtype=torch.int32, device=dev)
    want = sd.process_logits(x, prev=prev, base=1, presence=pres)
    same = torch.as_strided(x, (B, 1, V), (V, 1, 1))
    assert torch.equal(sd.process_logits(x, prev=prev, base=1, presence=pres, out=same), want)
    assert torch.equal(x, want)


def test_rows_without_the_drafts_that_they_count_are_refused(dev):
    # no drafts at all (a tensor of no elements has no address) as well as too few
    x = _rows((2, 3, 50), F32, dev)
    prev = lambda n: torch.zeros((2, n), dtype=torch.int32, device=dev)
    for n, rows, start in ((0, 3, 0), (0, 1, 1), (0, 2, 5), (1, 3, 0), (2, 1, 3)):
        with pytest.raises((ValueError, sd.SDError)):
            sd.process_logits(x[:, :rows], prev=prev(n), base=start)
    for n, rows, start in ((0, 1, 0), (2, 3, 0), (2, 1, 2)):
        y = sd.process_logits(x[:, :rows], prev=prev(n), base=start)
        assert torch.equal(y, x[:, :rows])
    assert sd.process_logits(x[:0], prev=prev(0)[:0], base=1).shape == (0, 3, 50)
