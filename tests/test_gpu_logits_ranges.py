"""The logit operators on rows far from zero: finite stand-ins for -inf among ordinary logits,
rows moved by a large constant, teachers of nothing but a stand-in.  Against the definitions in
64 bits, for few rows (held on chip) and many (streamed)."""
import math

import pytest
import torch

from tests import logits_ref as ref

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_logits_gb300")

BF, F32 = torch.bfloat16, torch.float32
STREAMED = 61     # times a handful of rows: more than are held on chip


def f32(t):
    """A temperature as the library gets it."""
    return float(torch.tensor(t, dtype=F32))


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _g(seed):
    return torch.Generator().manual_seed(seed)


def _fills(dtype):
    return (-1e4, -1e9, -1e10, -1e30, float(torch.finfo(dtype).min))


# ---------------------------------------------------------------------- top --
def _masked_rows(V, dtype, fill, seed):
    """Ordinary logits in some places and the fill in all others."""
    g = _g(seed)
    x = torch.randn((5, V), generator=g) * 3
    i = torch.arange(V)
    keep = torch.stack([
        torch.rand(V, generator=g) < 0.1,        # spread over the row
        i >= V - 300,                            # at its end only
        i < 300,                                 # and at its start only
        torch.rand(V, generator=g) < 12 / V,     # a few: fewer than the larger k
        i == V // 2,                             # a single one
    ])
    return torch.where(keep, x, torch.full_like(x, fill)).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0.3, 1.0, 2.0, 100.0])
@pytest.mark.parametrize("times", [1, STREAMED])
def test_top_logits_among_finite_fills(dev, dtype, T, times):
    V, T = 9001, f32(T)
    for n, fill in enumerate(_fills(dtype)):
        x = _masked_rows(V, dtype, fill, n)
        for k in (4, 60):
            vals, ids, rest = ref.top(x, k, T)
            r = sd.top_logits(x.to(dev).repeat(times, 1), k, temperature=T)
            assert torch.equal(r.ids.cpu(), ids.repeat(times, 1))
            assert torch.equal(r.vals.cpu(), vals.repeat(times, 1))
            got = r.rest.cpu().to(ref.D).view(times, -1)
            tol = torch.tensor([ref.rest_tolerance(float(e), float(v), T, V)
                                for e, v in zip(rest, vals[:, 0])], dtype=ref.D)
            # the others all at a fill whose quotient by T is below fp32's range
            none = rest < -float(torch.finfo(F32).max)
            assert bool((got[:, none] == -math.inf).all())
            assert bool(((got - rest).abs() <= tol)[:, ~none].all()), (fill, k, got[0], rest)


# ------------------------------------------------------------------ distill --
def _want(x, ids, vals, rest, T, w):
    """(loss, gradient, their tolerances): ref.distill and ref.distill_tolerance for rows whose
    others may hold a share of the softmax below 64 bits' smallest.  The gradient is the
    formula's, w/T (q - p) and w/T (q_j - p_r s_j), with s the softmax among the others by
    itself.  Student and teacher are moved to a largest logit of zero first, which changes
    nothing but that 64 bits hold the logarithms of sums over logits of -1e9 and less."""
    N, V = x.shape
    x = x.to(ref.D)
    x = x - x.max(1, keepdim=True).values
    at = vals.to(ref.D).max(1).values
    at = torch.where(at > -math.inf, at, rest.to(ref.D) * T)
    at = torch.where(at > -math.inf, at, 0.0)      # nothing taught
    vals, rest = vals.to(ref.D) - at[:, None], rest.to(ref.D) - at / T
    loss, grad, shares = ref.distill(x, ids, vals, rest, T, w)
    lt, gt = ref.distill_tolerance(x, shares, T, w, V)
    E = 2 * ref.lse_error(V) + 2.0 ** -21
    for n in range(N):
        if shares[n] is None:
            continue
        p, q, d, named, ls = shares[n]
        others = torch.ones(V, dtype=torch.bool)
        others[named] = False
        f = (float(w[n]) if w is not None else 1.0) / T
        so = x[n, others]
        log_s = (so - so.max()) / T
        log_s = log_s - torch.logsumexp(log_s, 0)
        far = lambda l: E + (-l.clamp(min=-200) / math.log(2)) * 4 * ref.U
        lo = ls[others]
        grad[n, named] = f * (q - p)[:-1]
        grad[n, others] = f * (lo.exp() - p[-1] * log_s.exp())
        gt[n, others] = f * (far(lo) * lo.exp() + far(log_s) * p[-1] * log_s.exp()) + 2.0 ** -126
    return loss, grad, lt, gt


def _check(dev, x, ids, vals, rest, T, w, times):
    """Loss alone and loss with gradient of every copy of the rows."""
    loss, grad, lt, gt = _want(x, ids, vals, rest, T, w)
    up = lambda t: None if t is None else t.to(dev).repeat(*((times,) + (1,) * (t.dim() - 1)))
    a = [up(t) for t in (x, ids, vals, rest)]
    only = sd.distill_loss(*a, temperature=T, weight=up(w))
    both, g = sd.distill_grad(*a, temperature=T, weight=up(w))
    lt, gt = lt + ref.U * loss.abs(), gt + ref.half_step(x.dtype) * (grad.abs() + gt)
    for l in (only, both):
        off = (l.cpu().to(ref.D).view(times, -1) - loss).abs()
        assert bool((off <= lt).all()), (l[:len(loss)], loss, lt)
    off = (g.cpu().to(ref.D).view(times, *grad.shape) - grad).abs()
    assert bool((off <= gt).all()), (float((off / gt).max()), torch.isnan(g).sum())


def _teacher(N, V, k, T, seed, shift=0.0):
    g = _g(seed)
    t = torch.randn((N, V), generator=g) * 3 + shift
    vals, ids = t.topk(k, 1)
    rest = torch.logsumexp(t.scatter(1, ids, -math.inf).double() / T, 1).float()
    return t, vals, ids.to(torch.int32), rest


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0.3, 1.0, 2.0, 100.0])
@pytest.mark.parametrize("times", [1, STREAMED])
def test_distill_among_finite_fills(dev, dtype, T, times):
    V, k, T = 5003, 9, f32(T)
    for n, fill in enumerate(_fills(dtype)):
        t, vals, ids, rest = _teacher(6, V, k, T, 10 + n)
        g = _g(40 + n)
        x = t + torch.randn(t.shape, generator=g)
        named = torch.zeros((6, V), dtype=torch.bool).scatter_(1, ids.long(), True)
        i = torch.arange(V)
        keep = torch.ones((6, V), dtype=torch.bool)
        keep[0] = named[0] | (torch.rand(V, generator=g) < 0.05)   # others spread over the row
        keep[1] = named[1] | (i >= V - 200)                        # at its end only
        keep[2] = named[2]                  # the others all at the fill, no mass of the teacher's
        rest[2] = -math.inf
        keep[3] = False                     # the whole row at the fill
        # the teacher has mass where the student has the fill: its losses are the fill's size
        # (left as ordinary rows where that passes fp32's range, in powers of two)
        if fill / T * math.log2(math.e) > -3e38:
            keep[4] = named[4]
            keep[5] = ~named[5]
        x = torch.where(keep, x, torch.full_like(x, fill)).to(dtype)
        w = torch.rand(6, generator=g) + 0.5
        _check(dev, x, ids, vals, rest, T, w, times)


@pytest.mark.parametrize("T", [0.3, 1.0, 4.0])
@pytest.mark.parametrize("times", [1, STREAMED])
@pytest.mark.parametrize("dtype,of_student,of_teacher", [
    (F32, 1000.0, 1000.0), (F32, -1000.0, -1000.0), (F32, 3e4, 3e4), (F32, -3e4, -3e4),
    (F32, 100.0, 100.0), (BF, 1000.0, 1000.0), (F32, 1000.0, 0.0), (F32, -1000.0, 0.0),
    (F32, 0.0, 1000.0), (F32, 60.0, -60.0), (F32, 5000.0, 0.0), (F32, 3e4, -3e4)])
def test_distill_rows_moved_by_a_constant(dev, dtype, of_student, of_teacher, T, times):
    # the softmax does not know of the constant, and no tolerance here does
    V, k, T = 6007, 24, f32(T)
    t, vals, ids, rest = _teacher(6, V, k, T, 77, of_teacher)
    x = (t + torch.randn(t.shape, generator=_g(78)) + (of_student - of_teacher)).to(dtype)
    _check(dev, x, ids, vals, rest, T, None, times)


@pytest.mark.parametrize("T", [0.3, 0.7, 1.0, 3.0, 7.0])
@pytest.mark.parametrize("times", [1, STREAMED])
def test_distill_teacher_rows_of_nothing_but_a_fill(dev, T, times):
    # the mass of the others, given as its logarithm, and the named tokens' lie on either side
    # of one another by the roundings of `rest`: hundreds and more of powers of two
    V, k, T = 700, 5, f32(T)
    g = _g(5)
    for base in (1e9, 1e10, 1e12, 1e30, 1.5e38):
        t = (-base * (1 + torch.rand(8, 1, generator=g))).expand(8, V).contiguous()
        vals, ids = t[:, :k].contiguous(), torch.arange(k, dtype=torch.int32).repeat(8, 1)
        rest = (t[:, 0].double() / T + math.log(V - k)).float()
        ids[3, 2] = -1                               # an empty slot
        vals[4] = -math.inf                          # all of the mass with the others
        vals[5, 1:] = -math.inf
        rest[6] = 3.0                                # named tokens far below the others
        vals[7, 0] = 2.0                             # and far above
        x = torch.randn((8, V), generator=g) * 3
        _check(dev, x, ids, vals, rest, T, None, times)


@pytest.mark.parametrize("times", [1, STREAMED])
def test_distill_teacher_without_a_softmax(dev, times):
    # a NaN or +inf on the teacher's side (as top_logits hands them on) is not taken for mass
    V, k = 900, 4
    t, vals, ids, rest = _teacher(5, V, k, 1.0, 3)
    vals[0, 1] = math.inf
    rest[1] = math.nan
    vals[2], rest[2] = -math.inf, math.nan
    rest[3] = math.inf
    x = t + torch.randn(t.shape, generator=_g(4))
    a = [v.to(dev).repeat(*((times,) + (1,) * (v.dim() - 1))) for v in (x, ids, vals, rest)]
    loss = sd.distill_loss(*a).view(times, -1)
    assert bool(torch.isnan(loss[:, :4]).all()) and bool(torch.isfinite(loss[:, 4]).all())
