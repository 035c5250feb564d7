"""Rows of unlike kinds next to one another: in the streamed distillation kernels, where a CTA
takes good, bad and idle rows in turn, and in the logit processing, where the rows of a
sequence are shared out over several CTAs."""
import math

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


@pytest.mark.parametrize("V,dtype,k", [(5003, BF, 6), (5003, F32, 6), (1501, BF, 128),
                                       (40001, F32, 33)])
@pytest.mark.parametrize("in_place", [False, True])
def test_distill_rows_of_every_kind_in_turn(dev, V, dtype, k, in_place):
    # nine kinds of rows, 1017 rows: whatever the number of CTAs (two per SM) is, short of a
    # multiple of nine, each takes rows of several kinds one after the other
    kinds, times = 9, 113
    x, ids, vals, rest, w = base._distill_case(kinds, V, dtype, k, V + k, 1.5)
    teacher = base._logits((kinds, V), F32, V + k)
    ids[1, 2] = V                                                 # bad ids
    ids[2, 0] = -2
    ids[3, k - 1] = ids[3, 1]                                     # one named twice
    ids[4], vals[4], rest[4] = -1, -math.inf, -math.inf           # nothing taught
    w[5] = 0.0                                                    # not read
    x[5, 3] = math.nan
    ids[6, 1] = -1                                                # an empty slot
    vals[6, 3] = -math.inf
    x[7] = teacher[7].to(dtype)                                   # the teacher's own row
    x[8, ids[8, 2].long()] = -math.inf                            # an infinite loss
    more = lambda t: t.repeat(*((times,) + (1,) * (t.dim() - 1)))
    want = [more(t) for t in base._want_distill(x, ids, vals, rest, 1.5, w)]
    assert float(want[0][8]) == math.inf and float(want[0][1:6].abs().max()) == 0
    a = [more(t).to(dev) for t in (x, ids, vals, rest, w)]
    st = base._zero(dev)
    only = sd.distill_loss(*a[:4], temperature=1.5, weight=a[4], status=st)
    assert int(st) == sd.SD_STATUS_BAD_TOKEN
    base._near_distill(only, None, want)
    st = base._zero(dev)
    loss, grad = sd.distill_grad(*a[:4], temperature=1.5, weight=a[4], status=st,
                                 grad=a[0] if in_place else None)
    assert int(st) == sd.SD_STATUS_BAD_TOKEN
    base._near_distill(loss, grad, want)
    assert not bool(torch.isnan(grad).any())
    rows = grad.view(times, kinds, V)
    assert float(rows[:, 1:6].abs().max()) == 0
    # a row's copies at the same place of the 16-byte grid are equal bit for bit
    step = next(n for n in (1, 2, 4, 8) if n * kinds * V * x.element_size() % 16 == 0)
    assert torch.equal(rows[step:], rows[:-step])
    st = base._zero(dev)   # and nothing of the bad rows is left for a call without them
    good = [t.view(times, kinds, *t.shape[1:])[:, 4:].flatten(0, 1).contiguous() for t in a[1:]]
    student = more(x).view(times, kinds, V)[:, 4:].flatten(0, 1).contiguous().to(dev)
    sd.distill_grad(student, *good[:3], temperature=1.5, weight=good[3], status=st)
    assert int(st) == 0


# On 152 SMs a sequence's rows stay with one CTA per window in the first case; in the others
# they are shared out, in equal parts in the second, with a shorter last one from there on (the
# parts' number follows from the windows that there are).
@pytest.mark.parametrize("B,R,V,dtype", [(42, 4, 128256, BF), (8, 12, 128256, BF),
                                         (8, 16, 128256, BF), (8, 7, 128256, BF), (1, 32, 4099, BF),
                                         (1, 31, 32000, F32), (20, 11, 50021, BF)])
@pytest.mark.parametrize("start", [0, 1])
def test_process_rows_in_parts(dev, B, R, V, dtype, start):
    # the drafts are few tokens, so that rows on both sides of a boundary count the same ones
    x, k = base._process_case(B, R, V, dtype, 11 * R + V, base=start)
    k["prev"] = k["prev"] % 3 * (V // 4)
    k["bias_ids"][:, 0] = k["prev"][:, 0]
    y = sd.process_logits(x.to(dev), **base._to(k, dev))
    base._check_process(y, x, k)
    # row by row, as a drafter asks for them
    for r in (0, R // 2, R - 1):
        one = base._to({**k, "base": start + r, "mask": k["mask"][:, r].contiguous()}, dev)
        z = sd.process_logits(x[:, r].contiguous().to(dev), **one)
        assert torch.equal(torch.nan_to_num(z), torch.nan_to_num(y[:, r]))
