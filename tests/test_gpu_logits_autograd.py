"""The logit operators beside autograd: what they write into memory that the caller owns counts
as an in-place change, so that a backward pass which still needs the old values says so."""
import pytest
import torch

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_logits_gb300")

F32 = torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _teacher(dev, N, V, k):
    t = torch.randn((N, V), generator=torch.Generator().manual_seed(1)).to(dev)
    return sd.top_logits(t, k)


def test_writing_over_what_autograd_saved_is_an_error(dev):
    N, V = 4, 300
    t = _teacher(dev, N, V, 5)
    w = torch.randn((N, V), generator=torch.Generator().manual_seed(2)).to(dev).requires_grad_(True)
    for write in (lambda s: sd.distill_grad(s, *_order(t), grad=s), lambda s: sd.process_logits(
            s, bias_ids=torch.zeros((N, 1), dtype=torch.int32, device=dev),
            bias_vals=torch.ones((N, 1), device=dev), out=s)):
        student = torch.tanh(w)          # saves its output
        z = torch.logsumexp(student, 1).sum()
        write(student)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            z.backward()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            student.backward(torch.ones_like(student))


def test_every_given_output_counts_as_changed(dev):
    N, V, k = 3, 200, 4
    x = torch.randn((N, V), device=dev)
    t = _teacher(dev, N, V, k)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    n = torch.full((N,), 2, dtype=torch.int32, device=dev)
    counts = torch.zeros((N, V), dtype=torch.int16, device=dev)
    y, loss, grad = torch.empty_like(x), torch.empty(N, device=dev), torch.empty_like(x)
    for outs, call in (((counts,), lambda: sd.token_counts(i32(N, 6), n, V, out=counts)),
                       ((counts,), lambda: sd.token_counts_add(counts, i32(N, 2), n)),
                       ((y,), lambda: sd.process_logits(x, out=y)),
                       (tuple(t), lambda: sd.top_logits(x, k, out=t)),
                       ((loss,), lambda: sd.distill_loss(x, t.ids, t.vals, t.rest, out=loss)),
                       ((grad,), lambda: sd.distill_grad(x, *_order(t), grad=grad))):
        before = [o._version for o in outs]
        call()
        assert [o._version for o in outs] == [b + 1 for b in before]
    # a call that is refused has written nothing
    before = y._version
    with pytest.raises(sd.SDError):
        sd.process_logits(x, prev=i32(N, 2), base=9, out=y)
    assert y._version == before


def _order(t):
    return t.ids, t.vals, t.rest


def test_in_place_gradient_reaches_the_leaves(dev):
    # a head that saves none of its outputs: in place gives what a buffer of its own gives
    N, V, k, D = 6, 500, 8, 16
    g = torch.Generator().manual_seed(3)
    t = _teacher(dev, N, V, k)
    h, w0 = torch.randn((N, D), generator=g).to(dev), torch.randn((D, V), generator=g).to(dev)
    got = []
    for in_place in (False, True):
        w = w0.clone().requires_grad_(True)
        student = h @ w
        _, grad = sd.distill_grad(student, *_order(t), grad=student if in_place else None)
        student.backward(grad)
        got.append(w.grad)
    assert torch.equal(*got) and float(got[0].abs().max()) > 0


def test_inference_tensors_are_written(dev):
    N, V = 3, 100
    with torch.inference_mode():
        x = torch.randn((N, V), device=dev)
        bias = dict(bias_ids=torch.ones((N, 1), dtype=torch.int32, device=dev),
                    bias_vals=torch.ones((N, 1), device=dev))
        want = sd.process_logits(x, **bias)
        y = x.clone()
        sd.process_logits(y, out=y, **bias)
        assert torch.equal(y, want)
    z = x.clone()   # outside the mode: an ordinary tensor
    sd.process_logits(z, out=z, **bias)
    assert torch.equal(z, want)
    sd.process_logits(x, out=x, **bias)   # and one of the mode's own
    assert torch.equal(x, want)
