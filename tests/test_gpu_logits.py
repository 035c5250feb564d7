"""The logit operators (token counts, penalties with biases and masks, a teacher's top
logits, the distillation loss and its gradient) against their definitions in 64 bits."""
import math

import pytest
import torch

from tests import logits_ref as ref

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_logits_gb300")

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _g(seed):
    return torch.Generator().manual_seed(seed)


def _logits(shape, dtype, seed, peaks=True):
    g = _g(seed)
    x = torch.randn(shape, generator=g) * 3
    if peaks:
        x[torch.rand(shape, generator=g) < 0.002] += 8
    return x.to(dtype)


def _zero(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


# ------------------------------------------------------------------- counts --
@pytest.mark.parametrize("B,L,V", [(1, 0, 5), (3, 1, 1), (4, 700, 33), (3, 5000, 50021),
                                   (2, 40000, 151936), (5, 333, 32768), (2, 64, 262144)])
def test_token_counts(dev, B, L, V):
    g = _g(B * L + V)
    h = (torch.rand((B, L), generator=g) ** 4 * V).to(torch.int32).clamp_(0, V - 1)
    n = torch.tensor([L, L // 2, 0, L + 9, -3][:B], dtype=torch.int32)
    p = torch.tensor([L // 3, L, 5, -1, 2][:B], dtype=torch.int32)
    for prompt in (None, p):
        st = _zero(dev)
        c = sd.token_counts(h.to(dev), n.to(dev), V, status=st,
                            prompt_lengths=None if prompt is None else prompt.to(dev))
        assert torch.equal(c.cpu(), ref.token_counts(h, n, V, prompt))
        assert int(st) == 0


def test_token_counts_saturate_and_skip_foreign_ids(dev):
    V, L = 11, 100003
    h = torch.full((2, L), 4, dtype=torch.int32)
    h[0, ::3] = 5
    h[1, 70000] = V
    h[1, 70001] = -7
    n = torch.full((2,), L, dtype=torch.int32)
    p = torch.tensor([0, 10], dtype=torch.int32)
    st = _zero(dev)
    c = sd.token_counts(h.to(dev), n.to(dev), V, prompt_lengths=p.to(dev), status=st)
    assert torch.equal(c.cpu(), ref.token_counts(h, n, V, p))
    assert int(c[0, 4]) == 32767 and int(c[0, 5]) == 32767 and int(c[1, 4]) == -1
    assert int(st) == sd.SD_STATUS_BAD_TOKEN


@pytest.mark.parametrize("V", [7, 4099, 128256])
def test_token_counts_add(dev, V):
    g = _g(V)
    B, M = 6, 9
    c = torch.randint(0, 5, (B, V), generator=g).to(torch.int16)
    c[0, 1] = 32767
    c[1, 2] = 32766
    c[2, 3] = -1            # saturated, in the prompt
    c[3, 0] = -32768        # in the prompt only
    t = torch.randint(0, min(V, 5), (B, M), generator=g, dtype=torch.int32)
    t[4, 2], t[4, 3] = -1, V
    n = torch.tensor([9, 9, 9, 30, 5, -2], dtype=torch.int32)
    d, st = c.to(dev), _zero(dev)
    r = sd.token_counts_add(d, t.to(dev), n.to(dev), status=st)
    assert r is d and torch.equal(d.cpu(), ref.token_counts_add(c, t, n))
    assert int(st) == sd.SD_STATUS_BAD_TOKEN
    # a round's tokens: history counted at once or round by round
    full = sd.token_counts(t.clamp(0, V - 1).to(dev), n.clamp(0, M).to(dev), V)
    step = torch.zeros_like(full)
    for i in range(M):
        sd.token_counts_add(step, t.clamp(0, V - 1)[:, i:i + 1].contiguous().to(dev),
                            (n > i).to(torch.int32).to(dev))
    assert torch.equal(full, step)


# ------------------------------------------------------------------ process --
def _process_case(B, R, V, dtype, seed, base=0, bias=9, mask="rows"):
    g = _g(seed)
    P = min(32, base + R - 1)
    k = dict(
        counts=torch.where(torch.rand((B, V), generator=g) < 0.2,
                           torch.randint(-32768, 32768, (B, V), generator=g),
                           torch.zeros(1, dtype=torch.long)).to(torch.int16),
        prev=torch.randint(0, V, (B, P), generator=g, dtype=torch.int32),
        base=base,
        repetition=0.5 + torch.rand(B, generator=g) * 1.5,
        presence=torch.rand(B, generator=g) * 2 - 0.5,
        frequency=torch.rand(B, generator=g) * 0.01,
        bias_ids=torch.randint(-1, V, (B, bias), generator=g, dtype=torch.int32),
        bias_vals=torch.randn((B, bias), generator=g) * 4)
    W = (V + 31) // 32
    if mask:
        shape = (B, R, W) if mask == "rows" else (B, W)
        k["mask"] = torch.randint(-2 ** 31, 2 ** 31, shape, generator=g).to(torch.int32)
        if mask == "rows":
            k["mask"][0, 0] = 0      # a row with nothing allowed
            k["mask"][-1, -1] = -1   # and one with everything
    return _logits((B, R, V), dtype, seed + 1), k


def _to(k, dev):
    return {n: v.to(dev) if torch.is_tensor(v) else v for n, v in k.items()}


def _check_process(y, x, k):
    want, size, touched = ref.process(x, **k)
    got = y.cpu()
    assert got.dtype == x.dtype and got.shape == x.shape
    same = ~touched
    out = torch.where(want == -math.inf, torch.full_like(x, -math.inf), x)
    # what nothing touches comes out as it was, bit for bit
    bits = torch.int16 if x.dtype == BF else torch.int32
    assert torch.equal(got.view(bits)[same], out.view(bits)[same])
    w, t = want[touched], ref.process_tolerance(want, size, x.dtype)[touched]
    gt = got[touched].to(ref.D)
    nan = torch.isnan(w)
    assert torch.equal(nan, torch.isnan(gt))
    fin = torch.isfinite(w)
    assert torch.equal(gt[~fin & ~nan], w[~fin & ~nan])
    assert bool(((gt - w)[fin].abs() <= t[fin]).all())


PROCESS = [(1, 1, 1, BF), (2, 3, 17, F32), (3, 2, 33, BF), (2, 5, 2049, BF), (4, 7, 4099, BF),
           (3, 4, 4099, F32), (1, 1, 32000, F32), (2, 33, 1000, BF), (5, 9, 8192, BF),
           (2, 3, 128256, BF), (1, 2, 262144, F32)]


@pytest.mark.parametrize("B,R,V,dtype", PROCESS)
def test_process_logits(dev, B, R, V, dtype):
    x, k = _process_case(B, R, V, dtype, B * R + V)
    st = _zero(dev)
    _check_process(sd.process_logits(x.to(dev), status=st, **_to(k, dev)), x, k)
    assert int(st) == 0


@pytest.mark.parametrize("parts", [("counts", "prev", "base", "frequency"), ("mask",),
                                   ("bias_ids", "bias_vals", "counts", "repetition")])
@pytest.mark.parametrize("B,R,V,dtype", [(40, 2, 128256, BF), (80, 1, 32000, F32),
                                         (101, 3, 50021, BF)])
def test_process_logits_many_sequences(dev, B, R, V, dtype, parts):
    # more CTAs than the device holds at once: a window's rows stay with one CTA
    x, k = _process_case(B, R, V, dtype, 6)
    k = {n: k[n] for n in parts}
    _check_process(sd.process_logits(x.to(dev), **_to(k, dev)), x, k)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("parts", [(), ("counts",), ("counts", "repetition"), ("prev", "base"),
                                   ("prev", "base", "frequency", "presence"), ("mask",),
                                   ("bias_ids", "bias_vals"), ("presence", "repetition")])
def test_process_logits_parts(dev, dtype, parts):
    x, k = _process_case(3, 4, 1003, dtype, 5, base=3, mask="shared" if dtype == F32 else "rows")
    k = {n: k[n] for n in parts}
    _check_process(sd.process_logits(x.to(dev), **_to(k, dev)), x, k)


def test_process_logits_rows_count_their_drafts(dev):
    # drafts 7, 7, 3: row r sees the first r of them, two of the same count twice
    x = torch.ones((1, 4, 50))
    prev = torch.tensor([[7, 7, 3]], dtype=torch.int32)
    y = sd.process_logits(x.to(dev), prev=prev.to(dev),
                          frequency=torch.tensor([0.25]).to(dev)).cpu()
    assert y[0, :, 7].tolist() == [1.0, 0.75, 0.5, 0.5]
    assert y[0, :, 3].tolist() == [1.0, 1.0, 1.0, 0.75]
    # one row at a time, as the drafter draws them
    for j in range(4):
        z = sd.process_logits(x[:, 0].to(dev), prev=prev.to(dev), base=j,
                              frequency=torch.tensor([0.25]).to(dev)).cpu()
        assert torch.equal(z[0], y[0, j])


def test_process_logits_repeated_biases_add_in_order(dev):
    V = 5000
    n = 1024
    ids = torch.full((2, n), -1, dtype=torch.int32)
    vals = torch.zeros((2, n))
    ids[0, :900] = 77                     # all in one place: summed in list order, in fp32
    vals[0, :900] = torch.randn(900, generator=_g(3))
    ids[1] = torch.arange(n, dtype=torch.int32) * 4 + 1
    vals[1] = torch.arange(n, dtype=torch.float32)
    x = torch.zeros((2, 1, V))
    y = sd.process_logits(x.to(dev), bias_ids=ids.to(dev), bias_vals=vals.to(dev)).cpu()
    s = torch.zeros(1)
    for z in vals[0, :900]:
        s = s + z
    assert float(y[0, 0, 77]) == float(s)
    assert torch.equal(y[1, 0, 1:4097:4], vals[1]) and int((y[1] != 0).sum()) == n - 1


def test_process_logits_values_at_masked_and_odd_places(dev):
    inf, nan = math.inf, math.nan
    for dtype in (F32, BF):
        x = torch.tensor([[[1.0, -inf, nan, inf, -2.0, torch.finfo(dtype).min, nan, inf]]],
                         dtype=dtype)
        c = torch.tensor([[3, 3, 0, 0, 1, 0, 0, 0]], dtype=torch.int16)
        k = dict(counts=c, repetition=torch.tensor([2.0]), presence=torch.tensor([1.0]),
                 bias_ids=torch.tensor([[1, 4, 5]], dtype=torch.int32),
                 bias_vals=torch.tensor([[inf, -inf, -1.0]]),
                 mask=torch.tensor([[[0b00111111]]], dtype=torch.int32))
        y = sd.process_logits(x.to(dev), **_to(k, dev)).cpu()[0, 0].float()
        assert float(y[0]) == 1.0 / 2 - 1 and float(y[1]) == -inf and math.isnan(y[2])
        assert float(y[3]) == inf and float(y[4]) == -inf
        assert float(y[5]) == torch.finfo(dtype).min   # -1 is far below its half step
        assert float(y[6]) == -inf and float(y[7]) == -inf


def test_process_logits_bad_penalties_and_ids(dev):
    B, R, V = 6, 2, 600
    x = _logits((B, R, V), BF, 8)
    rep = torch.tensor([1.0, 0.0, -1.0, math.nan, math.inf, 1.5])
    pres = torch.tensor([math.inf, 0.0, 0.0, 0.0, 0.0, 0.5])
    st = _zero(dev)
    y = sd.process_logits(x.to(dev), repetition=rep.to(dev), presence=pres.to(dev), status=st).cpu()
    assert torch.isnan(y[:5]).all() and torch.equal(y[5], x[5])
    assert int(st) == sd.SD_STATUS_BAD_PENALTY
    for name, t in (("prev", [[5, V], [1, 2]]), ("prev", [[-1, 5], [1, 2]]),
                    ("bias_ids", [[5, V], [1, 2]]), ("bias_ids", [[-2, 5], [1, 2]])):
        st = _zero(dev)
        k = {name: torch.tensor(t, dtype=torch.int32)}
        if name == "prev":
            k.update(frequency=torch.tensor([0.5, 0.25]), base=1)
        else:
            k["bias_vals"] = torch.ones((2, 2))
        _check_process(sd.process_logits(x[:2].to(dev), status=st, **_to(k, dev)), x[:2], k)
        assert int(st) == sd.SD_STATUS_BAD_TOKEN
    st = _zero(dev)   # drafts that no row counts are not read
    sd.process_logits(x[:1].to(dev), status=st,
                      prev=torch.tensor([[3, V, V]], dtype=torch.int32).to(dev))
    assert int(st) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1000, 1003])
def test_process_logits_strides_and_outputs(dev, dtype, V):
    x, k = _process_case(3, 4, V, dtype, 21)
    kd = _to(k, dev)
    want = sd.process_logits(x.to(dev), **kd)
    _check_process(want, x, k)
    bits = torch.int16 if dtype == BF else torch.int32
    same = lambda a, b: torch.equal(a.contiguous().view(bits), b.contiguous().view(bits))
    # rows of a padded vocabulary, an output of another alignment, rows before sequences
    pad = torch.zeros((3, 4, V + 29), dtype=dtype, device=dev)
    pad[..., 5:5 + V] = x.to(dev)
    view = pad[..., 5:5 + V]
    assert same(sd.process_logits(view, **kd), want)
    buf = torch.full((3, 4, V + 29), 99.0, dtype=dtype, device=dev)
    for off in (0, 1, 5, 8):
        buf.fill_(99.0)
        o = buf[..., off:off + V]
        assert sd.process_logits(view, out=o, **kd) is o
        assert same(o, want)
        assert bool((buf[..., :off] == 99).all()) and bool((buf[..., off + V:] == 99).all())
    t = x.to(dev).transpose(0, 1).contiguous().transpose(0, 1)
    assert same(sd.process_logits(t, **kd), want)
    # in place, contiguous and padded; what lies around the rows is left alone
    for z in (x.to(dev), view):
        assert sd.process_logits(z, out=z, **kd) is z and same(z, want)
    assert float(pad[..., :5].abs().max()) == 0 and float(pad[..., 5 + V:].abs().max()) == 0


def test_process_logits_long_offsets(dev):
    # sequences that start beyond 2^31 elements into the tensor
    V, step = 1000, 2 ** 30 + 12345
    base = torch.empty(2 * step + 4 * V, dtype=BF, device=dev)
    x = torch.as_strided(base, (3, 2, V), (step, 2 * V, 1))
    x.copy_(_logits((3, 2, V), BF, 4).to(dev))
    pres = torch.tensor([0.5, 1.0, 1.5], device=dev)
    prev = torch.tensor([[3], [4], [5]], dtype=torch.int32, device=dev)
    y = sd.process_logits(x, prev=prev, presence=pres)
    _check_process(y, x.cpu(), dict(prev=prev.cpu(), presence=pres.cpu()))
    m = base[2 * step:2 * step + 4 * V].view(2, 2, V)[:, 0]
    assert torch.equal(sd.top_logits(x[2], 5).ids, sd.top_logits(m.contiguous(), 5).ids)
    del base


def test_empty_batches(dev):
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device=dev)
    i = lambda *s: e(*s, dt=torch.int32)
    assert sd.process_logits(e(0, 3, 10)).shape == (0, 3, 10)
    assert sd.process_logits(e(2, 0, 10)).shape == (2, 0, 10)
    assert sd.token_counts(i(0, 4), i(0), 10).shape == (0, 10)
    assert sd.top_logits(e(0, 10), 3).ids.shape == (0, 3)
    assert sd.distill_loss(e(0, 10), i(0, 3), e(0, 3, dt=F32)).shape == (0,)
    assert sd.distill_grad(e(0, 10), i(0, 3), e(0, 3, dt=F32))[1].shape == (0, 10)


# ---------------------------------------------------------------------- top --
def _check_top(x, k, T, dev, xd=None):
    r = sd.top_logits(x.to(dev) if xd is None else xd, k, temperature=T)
    vals, ids, rest = ref.top(x.reshape(-1, x.shape[-1]), k, T)
    assert torch.equal(r.ids.cpu().reshape(ids.shape), ids)
    assert torch.equal(r.vals.cpu().reshape(vals.shape), vals)
    got = r.rest.cpu().to(ref.D).reshape(-1)
    for n in range(len(rest)):
        if math.isnan(rest[n]):
            assert math.isnan(got[n])
        elif math.isinf(rest[n]):
            assert got[n] == rest[n]
        else:
            tol = ref.rest_tolerance(float(rest[n]), float(vals[n, 0]), T, x.shape[-1])
            assert abs(float(got[n] - rest[n])) <= tol
    return r


TOP = [(300, 151936, BF, 128), (100, 60007, F32, 64), (64, 1, BF, 2), (70, 17, F32, 128), (1, 1, BF, 1), (2, 5, F32, 3), (3, 17, BF, 128), (4, 1000, BF, 7), (3, 4099, F32, 128),
       (2, 50021, BF, 64), (1, 128256, BF, 128), (2, 262144, F32, 100), (40, 8191, BF, 33),
       (350, 9000, BF, 16), (7, 151936, BF, 1)]


@pytest.mark.parametrize("N,V,dtype,k", TOP)
@pytest.mark.parametrize("T", [1.0, 0.3])
def test_top_logits(dev, N, V, dtype, k, T):
    _check_top(_logits((N, V), dtype, N + V), k, T, dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [1, 60, 128])
def test_top_logits_shapes_of_rows(dev, dtype, k):
    V = 40009
    i = torch.arange(V)
    q = (i // (8 if dtype == BF else 4)) % 512
    small = torch.randn(V, generator=_g(1))
    rows = [
        torch.zeros(V),                                   # all equal: the lowest indices
        i.float() / 300, -i.float() / 300,                # sorted either way
        torch.where(i % 2 == 0, -math.inf, small),        # every other place masked
        torch.full((V,), -math.inf),                      # nothing left
        torch.where(i == 12345, 3.0, -math.inf),          # one place left
        torch.where(i < 100, small, -math.inf),           # fewer left than kept
        torch.where(q < 2 * (k - 1), 50 + small, small),  # k - 1 groups hold nearly all large ones
        torch.where(i > V - 3000, 50 + small, small),     # large ones side by side
        torch.full((V,), torch.finfo(dtype).min),         # masked by the type's lowest value
        torch.where(i % 7 == 0, -0.0, 0.0),               # zeros of both signs are equal
    ]
    rows.append(torch.where(i < V // 2, -math.inf, small))   # nothing in the first half
    x = torch.stack(rows).to(dtype)
    _check_top(x, k, 1.0, dev)
    # many rows are taken differently: every copy of a row comes out as the definition's,
    # and bit for bit alike where the copies lie alike on the 16-byte grid (the sums of the
    # others are shared out by vectors of that grid)
    vals, ids, rest = ref.top(x, k, 2.0)
    r = sd.top_logits(x.to(dev).repeat(31, 1), k, temperature=2.0)
    alike = {}
    for b in range(31):
        part = slice(b * len(rows), (b + 1) * len(rows))
        assert torch.equal(r.ids[part].cpu(), ids) and torch.equal(r.vals[part].cpu(), vals)
        first = alike.setdefault(b * len(rows) * V * x.element_size() % 16, r.rest[part])
        assert torch.equal(r.rest[part], first)
        for n, e in enumerate(rest):
            got = float(r.rest[part][n])
            if math.isinf(e):
                assert got == float(e)
            else:
                tol = ref.rest_tolerance(float(e), float(vals[n, 0]), 2.0, V)
                assert abs(got - float(e)) <= tol


def test_top_logits_nan_and_inf(dev):
    x = _logits((3, 3001), F32, 9)
    x[0, 17] = math.nan
    x[1, 5] = math.inf
    x[2, 100:103] = -math.nan
    r = _check_top(x, 4, 1.0, dev)
    assert int(r.ids[1, 0]) == 5 and not bool(torch.isnan(r.vals).any())
    many = sd.top_logits(x.to(dev).repeat(100, 1), 4)
    assert torch.equal(many.ids, r.ids.repeat(100, 1)) and torch.equal(many.vals, r.vals.repeat(100, 1))
    assert bool(torch.isnan(many.rest.view(100, 3)[:, 0]).all()) and bool(torch.isfinite(many.rest.view(100, 3)[:, 1]).all())


def test_top_logits_views(dev):
    x = _logits((6, 5, 2003), BF, 10)
    big = torch.zeros((6, 5, 2048), dtype=BF, device=dev)
    big[..., 3:2006] = x.to(dev)
    a = _check_top(x, 9, 1.0, dev)
    b = _check_top(x, 9, 1.0, dev, big[..., 3:2006])
    assert a.ids.shape == (6, 5, 9) and torch.equal(a.ids, b.ids)
    assert _check_top(x[:, 2], 9, 1.0, dev, big[:, 2, 3:2006]).ids.shape == (6, 9)


# ------------------------------------------------------------------ distill --
def _distill_case(N, V, dtype, k, seed, T=1.0, rest=True):
    teacher = _logits((N, V), F32, seed)
    x = (teacher + torch.randn((N, V), generator=_g(seed + 1))).to(dtype)
    vals, ids = teacher.topk(min(k, V), 1)
    pad = k - vals.shape[1]
    if pad > 0:
        vals = torch.cat([vals, torch.full((N, pad), -math.inf)], 1)
        ids = torch.cat([ids, torch.full((N, pad), -1)], 1)
    left = teacher.scatter(1, ids.clamp(min=0), -math.inf)
    r = torch.logsumexp(left.double() / T, 1).float() if rest else None
    w = torch.rand(N, generator=_g(seed + 2)) + 0.5
    return x, ids.to(torch.int32), vals, r, w


def _want_distill(x, ids, vals, rest, T, w):
    loss, grad, shares = ref.distill(x, ids, vals, rest, T, w)
    return (loss, grad, *ref.distill_tolerance(x, shares, T, w, x.shape[1]))


def _near_distill(l, g, want):
    """A loss [N] and, where there is one, a gradient [N][V] against the definition's."""
    loss, grad, lt, gt = want
    l = l.cpu().to(ref.D)
    fin = torch.isfinite(loss)
    assert torch.equal(l[~fin], loss[~fin])
    off = (l - loss).abs() - lt - ref.U * loss.abs()
    assert bool((off[fin] <= 0).all()), (l - loss, lt)
    if g is None:
        return
    tol = gt + ref.half_step(g.dtype) * (grad.abs() + gt)
    off = ((g.cpu().to(ref.D) - grad).abs() - tol)[fin[:, None].expand_as(grad)]
    assert not off.numel() or float(off.max()) <= 0, float(off.max())


def _check_distill(dev, x, ids, vals, rest, T, w):
    up = lambda t: None if t is None else t.to(dev)
    want = _want_distill(x, ids, vals, rest, T, w)
    only = sd.distill_loss(up(x), up(ids), up(vals), up(rest), temperature=T, weight=up(w))
    both = sd.distill_grad(up(x), up(ids), up(vals), up(rest), temperature=T, weight=up(w))
    assert both[1].dtype == x.dtype and both[1].shape == x.shape
    _near_distill(only, None, want)
    _near_distill(*both, want)
    return both


DISTILL = [(1, 1, F32, 1), (3, 2, BF, 1), (2, 17, F32, 20), (5, 1000, BF, 16), (4, 4099, BF, 128),
           (3, 4099, F32, 7), (2, 50021, BF, 64), (1, 128256, BF, 32), (2, 262144, F32, 100),
           (330, 5003, BF, 8), (2, 300, F32, 0)]


def test_distill_many_rows(dev):
    # batches that are streamed, several rows to a CTA where rows are short: every copy of
    # a few rows against the definition (copies lie differently on the 16-byte grid)
    for V, dtype, k, times in ((1, F32, 1, 131), (5003, BF, 128, 131), (40001, F32, 33, 131),
                               (128256, BF, 64, 13)):
        x, ids, vals, r, w = _distill_case(5, V, dtype, k, V, 1.5)
        w[3] = 0.0
        x[3, 0] = math.nan
        more = lambda t: t.repeat(*((times,) + (1,) * (t.dim() - 1)))
        want = [more(t) for t in _want_distill(x, ids, vals, r, 1.5, w)]
        a = [more(t).to(dev) for t in (x, ids, vals, r, w)]
        only = sd.distill_loss(*a[:4], temperature=1.5, weight=a[4])
        loss, grad = sd.distill_grad(*a[:4], temperature=1.5, weight=a[4])
        _near_distill(only, None, want)
        _near_distill(loss, grad, want)


@pytest.mark.parametrize("N,V,dtype,k", DISTILL)
@pytest.mark.parametrize("T,rest", [(1.0, True), (4.0, True), (0.7, False)])
def test_distill(dev, N, V, dtype, k, T, rest):
    x, ids, vals, r, w = _distill_case(N, V, dtype, k, N + V + k, T, rest)
    _check_distill(dev, x, ids, vals, r, T, w)
    _check_distill(dev, x, ids, vals, r, T, None)


def test_distill_near_and_equal_to_the_teacher(dev):
    # the student is the teacher, or hardly off it: nothing may cancel
    for off, T in ((0.0, 1.0), (1e-3, 1.0), (1e-2, 4.0), (0.1, 2.0)):
        g = _g(int(off * 1e4))
        teacher = torch.randn((6, 3001), generator=g) * 2
        x = teacher + off * torch.randn(teacher.shape, generator=g)
        vals, ids = teacher.topk(20, 1)
        left = teacher.scatter(1, ids, -math.inf)
        rest = torch.logsumexp(left.double() / T, 1).float()
        loss, _ = _check_distill(dev, x, ids.to(torch.int32), vals, rest, T, None)
        assert bool((loss >= 0).all())


def test_distill_gradient_against_differences(dev):
    # the loss of the definition, in 64 bits, moved by h either way: off by h^2 / 6 times its
    # third derivative, which is below 1 / T^3 for shares of at most one
    N, V, k, T, h = 2, 40, 5, 1.3, 1e-3
    x, ids, vals, r, w = _distill_case(N, V, F32, k, 77, T)
    _, grad = sd.distill_grad(x.to(dev), ids.to(dev), vals.to(dev), r.to(dev), temperature=T,
                              weight=w.to(dev))
    _, _, shares = ref.distill(x, ids, vals, r, T, w)
    _, gt = ref.distill_tolerance(x, shares, T, w, V)
    for v in range(V):
        up, down = x.double(), x.double()
        up[:, v] += h
        down[:, v] -= h
        d = (ref.distill(up, ids, vals, r, T, w)[0] - ref.distill(down, ids, vals, r, T, w)[0]) / (2 * h)
        tol = gt[:, v] + w.double() * h * h / 6 / T ** 3 + ref.U * d.abs() + 1e-11
        assert bool(((grad[:, v].cpu().double() - d).abs() <= tol).all())


def test_distill_rows_with_nothing_to_learn(dev):
    N, V, k = 6, 1003, 4
    for dtype in (BF, F32):
        x, ids, vals, r, w = _distill_case(N, V, dtype, k, 31)
        w[0] = 0.0
        x[0, 5] = math.nan            # a row of weight 0 is not read
        ids[1], vals[1], r[1] = -1, -math.inf, -math.inf   # a teacher row of only -inf
        ids[2, 1] = -1                # an empty slot
        vals[3, 2] = -math.inf        # a named token of no mass
        r[4] = -math.inf              # no mass beside the named tokens
        loss, grad = _check_distill(dev, x, ids, vals, r, 1.0, w)
        assert float(loss[0]) == float(loss[1]) == 0
        assert float(grad[:2].abs().max()) == 0


def test_distill_student_without_mass(dev):
    V, k = 2005, 6
    x, ids, vals, r, w = _distill_case(5, V, F32, k, 55)
    x[0, ids[0, 3].long()] = -math.inf       # masked where the teacher has mass: infinite loss
    others = torch.ones(V, dtype=torch.bool)
    others[ids[1].long()] = False
    x[1, others] = -math.inf                 # and in the bucket of all others
    x[2, :] = -math.inf
    x[2, ids[2].long()] = 1.0
    r[2] = -math.inf                         # there without mass: finite
    x[3, others.nonzero()[::2, 0]] = -math.inf
    x[4, 9] = math.nan
    loss, grad = sd.distill_grad(x.to(dev), ids.to(dev), vals.to(dev), r.to(dev), weight=w.to(dev))
    assert float(loss[0]) == float(loss[1]) == math.inf
    assert bool(torch.isnan(loss[4])) and bool(torch.isnan(grad[4]).any())
    assert not bool(torch.isnan(grad[:4]).any())
    # the gradients of the infinite losses: q - p at named tokens all the same
    p = torch.softmax(torch.cat([vals[:2], r[:2, None]], 1).double(), 1)
    q = torch.softmax(x[:2].double(), 1)
    for n in range(2):
        e = w[n].double() * (q[n, ids[n].long()] - p[n, :k])
        assert bool(((grad[n].cpu().double()[ids[n].long()] - e).abs() <= 1e-6 * w[n]).all())
    keep = [2, 3]
    _check_distill(dev, x[keep], ids[keep], vals[keep], r[keep], 1.0, w[keep])


def test_distill_others_far_below(dev):
    # the others' share of the student is far below fp32's smallest: gradients stay finite
    V, k = 999, 3
    x, ids, vals, r, w = _distill_case(2, V, F32, k, 66)
    others = torch.ones(V, dtype=torch.bool)
    others[ids[0].long()] = False
    x[0] = 0.0
    x[0, others] = -200.0
    loss, grad = sd.distill_grad(x.to(dev), ids.to(dev), vals.to(dev), r.to(dev))
    want = ref.distill(x, ids, vals, r, 1.0, None)
    assert abs(float(loss[0]) - float(want[0][0])) <= 1e-5 * float(want[0][0])
    e = (grad[0].cpu().double() - want[1][0]).abs()
    assert float(e.max()) <= 1e-5 * float(want[1][0].abs().max())


def test_distill_bad_ids(dev):
    N, V = 5, 700
    x, ids, vals, r, w = _distill_case(N, V, BF, 6, 91)
    ids[0, 2], ids[1, 0], ids[2, 5] = V, -2, ids[2, 1]
    st = _zero(dev)
    loss, grad = sd.distill_grad(x.to(dev), ids.to(dev), vals.to(dev), r.to(dev),
                                 weight=w.to(dev), status=st)
    assert int(st) == sd.SD_STATUS_BAD_TOKEN
    assert float(loss[:3].abs().max()) == 0 and float(grad[:3].abs().max()) == 0
    _check_distill(dev, x[3:], ids[3:], vals[3:], r[3:], 1.0, w[3:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [3, 400])
def test_distill_views_and_in_place(dev, dtype, N):
    V, k = 1501, 9
    x, ids, vals, r, w = _distill_case(N, V, dtype, k, 13)
    a = [t.to(dev) for t in (ids, vals, r)]
    want = _want_distill(x, ids, vals, r, 1.0, w)
    pad = torch.zeros((N, V + 27), dtype=dtype, device=dev)
    for off, goff in ((0, 0), (3, 3), (3, 4), (8, 0)):
        pad.zero_()
        view = pad[:, off:off + V]
        view.copy_(x.to(dev))
        buf = torch.full((N, V + 27), 99.0, dtype=dtype, device=dev)
        g = buf[:, goff:goff + V]
        l2, g2 = sd.distill_grad(view, *a, weight=w.to(dev), grad=g)
        assert g2 is g
        _near_distill(l2, g2, want)
        assert bool((buf[:, :goff] == 99).all()) and bool((buf[:, goff + V:] == 99).all())
        l3, g3 = sd.distill_grad(view, *a, weight=w.to(dev), grad=view)
        assert g3 is not None and torch.equal(l3, l2) and torch.equal(view, g2)
        assert float(pad[:, :off].abs().sum()) == 0 and float(pad[:, off + V:].abs().sum()) == 0


# ---------------------------------------------------------- streams, graphs --
def _all_ops(dev, seed=1):
    x, k = _process_case(4, 3, 9001, BF, seed)
    k = _to(k, dev)
    xd = x.to(dev)
    h = torch.randint(0, 9001, (4, 500), generator=_g(seed), dtype=torch.int32).to(dev)
    n = torch.tensor([500, 3, 77, 0], dtype=torch.int32, device=dev)
    w = torch.full((4, 3), 1 / 12, device=dev)

    def call(stream=None):
        c = sd.token_counts(h, n, 9001, stream=stream)
        sd.token_counts_add(c, k["prev"], n.clamp(max=2), stream=stream)
        y = sd.process_logits(xd, **{**k, "counts": c}, stream=stream)
        t = sd.top_logits(xd, 12, stream=stream)
        loss, grad = sd.distill_grad(y, t.ids, t.vals, t.rest, weight=w, stream=stream)
        return c, y, t.ids, t.vals, t.rest, loss, grad
    return call


def _same(a, b):
    return all(torch.equal(torch.nan_to_num(x.float()), torch.nan_to_num(y.float()))
               for x, y in zip(a, b))


def test_same_bits_on_every_call_and_stream(dev):
    call = _all_ops(dev)
    first = call()
    torch.cuda.synchronize()
    for _ in range(3):
        assert _same(call(), first)
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    r = call(stream=s)
    s.synchronize()
    assert _same(r, first)


def test_graph_capture(dev):
    call = _all_ops(dev, 2)
    want = call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    for _ in range(2):
        for t in got[1:]:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert _same(got, want)
