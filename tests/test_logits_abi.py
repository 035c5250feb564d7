"""Refusals of the logit operators, at the C ABI and in the binding, and their 64-bit
definitions against hand-worked values (no GPU: every call is refused before any launch)."""
import ctypes
import math

import pytest
import torch

import speculative_decoding_verification_logits_gb300 as sd
from speculative_decoding_verification_logits_gb300.logits import DistillArgs, ProcessArgs
from tests import logits_ref as ref

BAD = sd.SD_ERR_INVALID_ARG
FAKE = 1 << 20   # a non-null address that is never dereferenced: the checks fail first


def test_struct_layouts():
    L = sd.lib()
    assert L.sd_process_args_size() == ctypes.sizeof(ProcessArgs)
    assert L.sd_distill_args_size() == ctypes.sizeof(DistillArgs)


def test_count_entry_points_refuse_bad_requests():
    L = sd.lib()
    ok = dict(B=2, L=8, V=100, h=FAKE, n=FAKE, p=None, c=FAKE)
    for bad in (dict(B=-1), dict(L=-1), dict(V=0), dict(V=sd.SD_MAX_V + 1), dict(h=None),
                dict(n=None), dict(c=None), dict(c=FAKE + 1)):
        a = {**ok, **bad}
        assert L.sd_token_counts(a["B"], a["L"], a["V"], a["h"], a["n"], a["p"], a["c"], None,
                                 None) == BAD, bad
        if "h" in bad or "L" in bad:
            continue
        assert L.sd_token_counts_add(a["B"], 3, a["V"], FAKE, a["n"], a["c"], None, None) == BAD
    assert L.sd_token_counts_add(2, -1, 100, FAKE, FAKE, FAKE, None, None) == BAD
    assert L.sd_token_counts_add(2, 3, 100, None, FAKE, FAKE, None, None) == BAD
    assert L.sd_token_counts(0, 8, 100, None, None, None, None, None, None) == sd.SD_OK
    assert L.sd_token_counts_add(2, 0, 100, None, None, None, None, None) == sd.SD_OK


def test_process_refuses_bad_requests():
    L = sd.lib()
    ok = dict(B=2, R=3, V=100, dtype=sd.SD_BF16, logits=FAKE, logits_sb=300, logits_sr=100,
              out=2 * FAKE, out_sb=300, out_sr=100)
    assert L.sd_process_logits(None, None) == BAD
    for bad in (dict(B=-1), dict(R=-1), dict(V=0), dict(V=sd.SD_MAX_V + 1), dict(dtype=2),
                dict(logits=None), dict(out=None), dict(logits=FAKE + 1), dict(out=FAKE + 1),
                dict(counts=FAKE + 1), dict(mask=FAKE + 2), dict(n_bias=-1),
                dict(n_bias=sd.SD_MAX_BIAS + 1, bias_ids=FAKE, bias_vals=FAKE),
                dict(n_bias=3, bias_ids=FAKE), dict(n_bias=3, bias_vals=FAKE), dict(base=-1),
                dict(prev=FAKE, P=1), dict(prev=FAKE, P=2, base=1),
                dict(prev=FAKE, P=sd.SD_MAX_K + 1), dict(prev=FAKE, P=32, base=2 ** 31 - 1),
                dict(out_sr=99), dict(out_sb=299), dict(out_sb=50, out_sr=100)):
        assert L.sd_process_logits(ProcessArgs(**{**ok, **bad}), None) == BAD, bad
    for empty in (dict(B=0), dict(R=0)):
        assert L.sd_process_logits(ProcessArgs(**{**ok, **empty, "logits": None}), None) == sd.SD_OK


def test_top_and_distill_refuse_bad_requests():
    L = sd.lib()
    top = dict(N=2, V=100, dtype=sd.SD_F32, x=FAKE, s=100, k=5, T=1.0, vals=FAKE, ids=FAKE)
    for bad in (dict(N=-1), dict(V=0), dict(V=sd.SD_MAX_V + 1), dict(dtype=5), dict(k=0),
                dict(k=sd.SD_MAX_TOP + 1), dict(T=0.0), dict(T=-1.0), dict(T=math.inf),
                dict(T=math.nan), dict(x=None), dict(vals=None), dict(ids=None), dict(x=FAKE + 2)):
        a = {**top, **bad}
        assert L.sd_top_logits(a["N"], a["V"], a["dtype"], a["x"], a["s"], a["k"], a["T"],
                               a["vals"], a["ids"], None, None) == BAD, bad
    ok = dict(N=2, V=100, k=5, dtype=sd.SD_F32, student=FAKE, student_s=100, ids=FAKE, vals=FAKE,
              T=1.0, loss=FAKE, grad=2 * FAKE, grad_s=100)
    assert L.sd_distill(None, None) == BAD
    for bad in (dict(N=-1), dict(V=0), dict(V=sd.SD_MAX_V + 1), dict(k=-1),
                dict(k=sd.SD_MAX_TOP + 1), dict(dtype=2), dict(T=0.0), dict(T=math.nan),
                dict(student=None), dict(ids=None), dict(vals=None), dict(loss=None, grad=None),
                dict(student=FAKE + 2), dict(grad=FAKE + 2), dict(grad_s=99)):
        assert L.sd_distill(DistillArgs(**{**ok, **bad}), None) == BAD, bad
    assert L.sd_distill(DistillArgs(**{**ok, "N": 0, "student": None}), None) == sd.SD_OK


def test_binding_refuses_host_tensors():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    x = torch.zeros(2, 3, 40)
    for call in (lambda: sd.token_counts(i(2, 9), i(2), 40),
                 lambda: sd.token_counts_add(torch.zeros(2, 40, dtype=torch.int16), i(2, 3), i(2)),
                 lambda: sd.process_logits(x), lambda: sd.top_logits(x, 3),
                 lambda: sd.distill_loss(x, i(2, 3, 4), torch.zeros(2, 3, 4)),
                 lambda: sd.distill_grad(x, i(2, 3, 4), torch.zeros(2, 3, 4))):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------- the definitions --
def test_reference_counts_by_hand():
    h = torch.tensor([[1, 2, 2, 3, 9, 3]], dtype=torch.int32)
    c = ref.token_counts(h, torch.tensor([6]), 5, torch.tensor([2]))
    assert (c[0].long() & 0x7FFF).tolist() == [0, 0, 1, 2, 0]
    assert (c[0] < 0).tolist() == [False, True, True, False, False]
    c = ref.token_counts_add(c, torch.tensor([[1, 3, 7]]), torch.tensor([2]))
    assert (c[0].long() & 0x7FFF).tolist() == [0, 1, 1, 3, 0]


def test_reference_process_by_hand():
    x = torch.tensor([[[2.0, -2.0, 1.0, 0.5]]])
    y, _, touched = ref.process(x, counts=torch.tensor([[2, -32768, 0, 0]], dtype=torch.int16),
                                repetition=[2.0], presence=[0.5], frequency=[0.25],
                                bias_ids=torch.tensor([[2, 2]]), bias_vals=torch.tensor([[1.0, 2.0]]),
                                mask=torch.tensor([[[0b0111]]], dtype=torch.int32))
    assert y[0, 0].tolist() == [2 / 2 - 0.5 - 0.5, -4.0, 4.0, -math.inf]
    assert touched[0, 0].tolist() == [True, True, True, False]


def test_reference_gradient_is_the_formula_and_the_differences():
    g = torch.Generator().manual_seed(2)
    N, V, k, T = 3, 30, 4, 1.7
    t = torch.randn((N, V), generator=g) * 2
    x = t.double() + torch.randn((N, V), generator=g)
    vals, ids = t.topk(k, 1)
    rest = torch.logsumexp(t.scatter(1, ids, -math.inf).double() / T, 1)
    w = torch.rand(N, generator=g)
    loss, grad, _ = ref.distill(x, ids, vals, rest, T, w)
    lt = torch.cat([vals.double() / T, rest[:, None]], 1)
    p = torch.softmax(lt, 1)
    q = torch.softmax(x / T, 1)
    qr = 1 - q.gather(1, ids).sum(1, keepdim=True)
    f = q * (1 - p[:, k:] / qr)
    f = f.scatter(1, ids, q.gather(1, ids) - p[:, :k]) * w.double()[:, None] / T
    assert float((f - grad).abs().max()) < 1e-13
    h = 1e-5
    for v in range(V):
        e = torch.zeros(V, dtype=torch.float64)
        e[v] = h
        d = (ref.distill(x + e, ids, vals, rest, T, w)[0]
             - ref.distill(x - e, ids, vals, rest, T, w)[0]) / (2 * h)
        assert float((d - grad[:, v]).abs().max()) < 1e-9
    # the same over the whole vocabulary named is the plain divergence
    every = torch.arange(V).expand(N, V)
    full = ref.distill(x, every, t, None, T, w)[0]
    lp, lq = torch.log_softmax(t.double() / T, 1), torch.log_softmax(x / T, 1)
    assert float((full - w * (lp.exp() * (lp - lq)).sum(1)).abs().max()) < 1e-13
