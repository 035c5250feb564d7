"""Beam search's step (selection, reordering of states) against its definitions in 64 bits."""
import math

import pytest
import torch

from tests import beam_ref as ref

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


def _logits(shape, dtype, seed):
    g = _g(seed)
    x = torch.randn(shape, generator=g) * 3
    x[torch.rand(shape, generator=g) < 0.002] += 8
    return x.to(dtype)


def _scores(B, W, seed):
    return -20 * torch.rand((B, 1), generator=_g(seed)) - 4 * torch.rand((B, W), generator=_g(seed + 1))


def _run(dev, x, scores, k, status=0, **more):
    """Runs the call on copies on the device and holds it to the definition."""
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    there = {n: v.to(dev) if isinstance(v, torch.Tensor) else v for n, v in more.items()}
    beams = sd.beam_select(x if x.is_cuda else x.to(dev), scores.to(dev), k, status=st, **there)
    names = {"temperature": "T"}
    want = ref.select(x.cpu(), scores, k, **{names.get(n, n): v for n, v in more.items()})
    ref.check_select(beams, want, k, more.get("norm"))
    assert int(st) == want[2] == status
    return beams


# ------------------------------------------------------------------- select --
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,W,V,k", [
    (1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 1, 4), (3, 1, 7, 7), (2, 2, 33, 128), (1, 4, 1000, 4),
    (5, 7, 4099, 14), (3, 32, 517, 128), (1, 32, 32000, 32), (2, 4, 50021, 8), (4, 8, 128256, 16),
    (1, 1, 262144, 128), (40, 3, 32000, 6), (200, 3, 700, 9), (170, 17, 2000, 40)])
def test_select(dev, dtype, B, W, V, k):
    x = _logits((B, W, V), dtype, B + W + V + k)
    _run(dev, x, _scores(B, W, V), k, eos=V // 2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0.3, 0.7, 2.5])
def test_select_finished_dead_and_normed(dev, dtype, T):
    B, W, V, k = 9, 6, 3001, 12
    x, s = _logits((B, W, V), dtype, 3), _scores(B, W, 4)
    g = _g(5)
    fin = (torch.rand((B, W), generator=g) < 0.3).to(torch.uint8)
    s[torch.rand((B, W), generator=g) < 0.3] = -math.inf
    s[7] = -math.inf               # a sequence without a beam
    fin[8], s[8] = 1, -torch.rand(W, generator=g)   # and one of finished beams only
    norm = 1 + 3 * torch.rand((B, W), generator=g)
    for more in (dict(finished=fin, eos=5), dict(norm=norm), dict(finished=fin, eos=0, norm=norm),
                 dict(eos=V - 1)):
        _run(dev, x, s, k, temperature=T, **more)


def test_select_first_step_and_equal_beams(dev):
    # one live beam; beams alike to the bit tie in the order of beams, then tokens
    V = 700
    x = _logits((2, 4, V), BF, 8)
    s = torch.full((2, 4), -math.inf)
    s[:, 0] = 0.0
    _run(dev, x, s, 9)
    x[:, 1:] = x[:, :1]
    b = _run(dev, x, torch.full((2, 4), -1.5), 9)
    assert b.parents[0, :8].tolist() == [0, 1, 2, 3] * 2


@pytest.mark.parametrize("V", [1, 2, 701, 40000])
def test_select_beams_that_are_sure_tie_in_their_order(dev, V):
    # one token has all of the probability: its score is the beam's own, to the bit
    g = _g(V)
    for dtype, T in ((BF, 1.0), (F32, 0.3), (F32, 7.0)):
        B, W = 3, 9
        x = torch.randn((B, W, V), generator=g) - 900.0
        at = torch.randint(0, V, (B, W, 1), generator=g)
        x = x.scatter(2, at, 20 + 20 * torch.rand((B, W, 1), generator=g)).to(dtype)
        s = torch.tensor([0.0, -1.25, 3.0])[:, None].expand(B, W).contiguous()
        b = sd.beam_select(x.to(dev), s.to(dev), W, temperature=T)
        assert torch.equal(b.scores.cpu(), s) and torch.equal(b.tokens.cpu().long(), at[..., 0])
        assert b.parents.tolist() == [list(range(W))] * B


def test_select_masked_rows(dev):
    # rows of which a mask leaves nothing, one token, and fewer tokens than slots
    for dtype in (BF, F32):
        B, W, V, k = 3, 4, 2113, 16
        x = _logits((B, W, V), dtype, 9)
        x[0, 0] = -math.inf
        x[0, 1, 5:] = -math.inf
        x[0, 2, :] = -math.inf
        x[0, 2, V - 1] = 2.0
        x[1] = -math.inf                       # nothing in the whole sequence
        x[2, :, 3:] = -math.inf
        _run(dev, x, _scores(B, W, 10), k)


@pytest.mark.parametrize("fill", ["lowest", -1e10, -1e4])
def test_select_rows_masked_with_finite_values(dev, fill):
    # finite stand-ins for -inf are logits like others: fewer tokens than slots lie above them
    for dtype in (BF, F32):
        B, W, V, k = 2, 3, 20011, 16
        low = torch.finfo(dtype).min if fill == "lowest" else fill
        x = torch.full((B, W, V), low, dtype=dtype)
        x[0, 0, 100:103] = torch.tensor([1.0, 2.0, 0.5], dtype=dtype)
        x[0, 1, V - 2:] = 1.5
        x[1, 2, 7] = 3.0                       # the other rows of this one hold the fill alone
        for T in (1.0, 0.5):
            _run(dev, x, _scores(B, W, 11), k, temperature=T)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [513, 5000, 151936])
def test_select_many_equal_logits(dev, dtype, V):
    # thousands of equal logits at the k-th place, a few above them, at either end of the row
    B, W, k = 3, 4, 40
    x = torch.zeros((B, W, V), dtype=dtype)
    x[1, :, V // 2:V // 2 + 5] = 1.0
    x[1, :, -3:] = 2.0
    x[2] = torch.where(torch.rand((W, V), generator=_g(12)) < 0.5, 1.0, -1.0).to(dtype)
    x[2, 1, :] = 7.0
    x[2, 3, : V // 2] = -1.0
    fin = torch.zeros((B, W), dtype=torch.uint8)
    fin[1, 2] = 1
    s = torch.zeros((B, W)) - torch.arange(W) * 0.25
    s[1, 1] = -math.inf
    _run(dev, x, s, k, finished=fin, eos=1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_select_many_sequences_of_every_kind(dev, dtype):
    # more sequences than SMs: ordinary, equal, masked and crowded ones in turn
    B, W, V, k = 180, 4, 9000, 24
    x = _logits((B, W, V), dtype, 40)
    x[1::6] = 0.5
    x[2::6] = torch.finfo(dtype).min
    x[2::6, :, 5:8] = 1.0
    x[3::6, :, :3000] += 20
    x[4::6, 1] = -math.inf
    _run(dev, x, _scores(B, W, 41), k, eos=6)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_select_more_large_logits_than_the_list_holds(dev, dtype):
    # the large logits fill a few groups: more of them than there is room for, all different
    V, k = 60000, 128
    n = 256 if dtype == BF else 4000
    big = torch.arange(n, dtype=torch.float32) / (1 if dtype == BF else 7) + 1
    x = _logits((2, 2, V), dtype, 13) * 0.1
    x[0, 0, 3:3 + n] = big.to(dtype)
    x[0, 1, V - n:] = big.flip(0).to(dtype)
    x[1, :, 20000:20000 + 3000] = 5.0
    _run(dev, x, _scores(2, 2, 14), k)


def test_select_extreme_logits(dev):
    V, k = 3000, 8
    x = _logits((4, 3, V), F32, 15)
    x[0] += 1e6
    x[1] -= 1e6
    x[2] *= 1e-3
    x[3, 0, 17], x[3, 1, 4], x[3, 2] = 3e38, -3e38, x[3, 2] * 1e30
    for T in (1.0, 0.5):
        _run(dev, x, _scores(4, 3, 16), k, temperature=T)


def test_select_scores_that_tie_where_logits_do_not(dev):
    # differences of logits that no 64-bit score sees (below 2^-58 of it; between that and 2^-51 two
    # ways of rounding tie different ones): ties go to the lowest token
    for V, k in ((900, 12), (40000, 40)):
        x = torch.randn((2, 3, V), generator=_g(34)) * 1e-30
        x[1, 0, 5:50] = 1.0
        x[1, 1, V - 30:] = 2e-15
        _run(dev, x, _scores(2, 3, 35), k)
        _run(dev, _logits((2, 3, V), F32, 36), _scores(2, 3, 37), k, temperature=1e18)


def test_select_scales_that_pass_fp32(dev):
    # temperatures and norms at the ends of the type's range: scores over norm beyond fp32
    x, s = _logits((2, 4, 700), F32, 32), _scores(2, 4, 33)
    s[1] = -s[1]
    norm = torch.ones((2, 4))
    norm[0, 1], norm[0, 3], norm[1, 0], norm[1, 2] = 1e-38, 1e38, 2e-37, 3e38
    for T in (1.2e-38, 1e-20, 1.0, 1e20, 3e38):
        for n in (None, norm):
            _run(dev, x, s, 7, temperature=T, **({} if n is None else {"norm": n}))


def test_select_nonfinite_rows_and_scores(dev):
    V, k = 4001, 8
    for bad in (math.nan, math.inf):
        x, s = _logits((3, 4, V), BF, 17), _scores(3, 4, 18)
        x[0, 1, V - 1] = bad
        x[1, :, 0] = bad
        s[2, 3] = bad
        _run(dev, x, s, k, status=sd.SD_STATUS_NONFINITE)
    # rows that are not read may hold anything
    x, s = _logits((2, 3, V), BF, 19), _scores(2, 3, 20)
    x[0, 1], x[1, 2] = math.nan, math.inf
    s[0, 1] = -math.inf
    fin = torch.zeros((2, 3), dtype=torch.uint8)
    fin[1, 2] = 7
    _run(dev, x, s, k, finished=fin, eos=0)
    norm = torch.ones((2, 3))
    norm[0, 0], norm[0, 2], norm[1, 1], norm[1, 2] = 0.0, -1.0, math.nan, math.inf
    _run(dev, x, s, k, finished=fin, eos=0, norm=norm, status=sd.SD_STATUS_BAD_PENALTY)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_select_strided_rows(dev, dtype):
    B, W, V, k = 3, 5, 1777, 10
    buf = _logits((W, B + 1, V + 37), dtype, 21).to(dev)
    for off in (0, 1, 3):
        x = buf[:, :B, off:off + V].transpose(0, 1)
        _run(dev, x, _scores(B, W, 22), k)
    # one row for all beams
    _run(dev, buf[:1, :B, :V].transpose(0, 1).expand(B, W, V), _scores(B, W, 23), k)


def test_select_offsets_past_32_bits(dev):
    V = 40000
    buf = torch.empty(2 * 1_300_000_000 + V, dtype=BF, device=dev)
    x = torch.as_strided(buf, (2, 2, V), (1_300_000_000, 1_200_000_000, 1))
    x.copy_(_logits((2, 2, V), BF, 24))
    _run(dev, x, _scores(2, 2, 25), 6)


def test_select_into_given_outputs(dev):
    B, W, V, k = 4, 3, 900, 6
    x, s = _logits((B, W, V), F32, 26).to(dev), _scores(B, W, 27).to(dev)
    want = sd.beam_select(x, s, k, eos=3)
    out = sd.Beams(*(torch.empty_like(t) for t in want))
    before = [t._version for t in out]
    got = sd.beam_select(x, s, k, eos=3, out=out)
    assert got is out and all(torch.equal(a, b) for a, b in zip(got, want))
    assert [t._version for t in out] == [v + 1 for v in before]
    for twice in (dict(tokens=out.parents), dict(parents=out.tokens)):
        with pytest.raises(ValueError, match="overlap"):
            sd.beam_select(x, s, k, out=out._replace(**twice))
    with pytest.raises(ValueError, match="overlaps"):
        sd.beam_select(x, s, W, out=sd.Beams(s, *(t[:, :W].contiguous() for t in want[1:])))
    assert sd.beam_select(x[:0], s[:0], k).scores.shape == (0, k)


def test_select_same_bits_streams_and_graphs(dev):
    B, W, V, k = 6, 8, 32000, 16
    x, s = _logits((B, W, V), BF, 28).to(dev), _scores(B, W, 29).to(dev)
    call = lambda **m: sd.beam_select(x, s, k, eos=9, **m)
    want = call()
    same = lambda a: all(torch.equal(p, q) for p, q in zip(a, want))
    for _ in range(3):
        assert same(call())
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    got = call(stream=side)
    side.synchronize()
    assert same(got)
    graphs, outs = [], []
    for _ in range(2):   # two graphs, replayed side by side: they share no scratch
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert same(outs[0]) and same(outs[1])


def test_select_refusals(dev):
    x, s = torch.zeros((2, 3, 50), device=dev), torch.zeros((2, 3), device=dev)
    fin = torch.zeros((2, 3), dtype=torch.uint8, device=dev)
    for call in (lambda: sd.beam_select(x.half(), s, 3), lambda: sd.beam_select(x, s.double(), 3)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: sd.beam_select(x[0], s, 3), lambda: sd.beam_select(x, s[:1], 3),
                 lambda: sd.beam_select(x.transpose(1, 2), s, 3), lambda: sd.beam_select(x, s.cpu(), 3),
                 lambda: sd.beam_select(x, s, 3, finished=fin[:1], eos=0),
                 lambda: sd.beam_select(x, s, 3, norm=s[:1])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sd.beam_select(x, s, 0), lambda: sd.beam_select(x, s, 129),
                 lambda: sd.beam_select(x, s, 3, temperature=0.0),
                 lambda: sd.beam_select(x, s, 3, eos=50), lambda: sd.beam_select(x, s, 3, finished=fin)):
        with pytest.raises((ValueError, sd.SDError)):
            call()


# ------------------------------------------------------------------ reorder --
_TYPES = [torch.int32, torch.int16, torch.uint8, torch.float32, torch.bfloat16, torch.int64]


def _state(shape, dtype, seed):
    return torch.randint(0, 100, shape, generator=_g(seed)).to(dtype)


@pytest.mark.parametrize("dtype", _TYPES)
@pytest.mark.parametrize("B,W,row", [(1, 1, (1,)), (3, 4, (7,)), (2, 8, (513, 3)), (4, 5, (2048,)),
                                     (2, 17, (33,)), (1, 32, (1000,)), (2, 3, ()), (2, 3, (0,))])
def test_reorder(dev, dtype, B, W, row):
    x = _state((B, W, *row), dtype, W)
    p = torch.randint(-1, W, (B, W), generator=_g(B), dtype=torch.int32)
    want, _ = ref.reorder(x, p)
    xd, pd = x.to(dev), p.to(dev)
    assert torch.equal(sd.beam_reorder(xd, pd).cpu(), want) and torch.equal(xd.cpu(), x)
    version = xd._version
    assert sd.beam_reorder(xd, pd, out=xd) is xd and torch.equal(xd.cpu(), want)
    assert xd._version == version + 1


def test_reorder_several_states_strides_and_slots(dev):
    B, W, k = 3, 6, 4
    g = _g(31)
    p = torch.randint(0, W, (B, k), generator=g, dtype=torch.int32)
    xs = [_state((B, W, 50), torch.int32, 1), _state((B, W, 8, 16), BF, 2), _state((B, W), F32, 3),
          _state((B, W, 1001), torch.uint8, 4)]
    got = sd.beam_reorder([x.to(dev) for x in xs], p.to(dev))
    for x, y in zip(xs, got):
        assert torch.equal(y.cpu(), ref.reorder(x, p)[0])
    # rows inside larger buffers: what lies around them stays
    buf = torch.full((W, B, 80), -7, dtype=torch.int32, device=dev)
    rows = buf[:, :, 13:63].transpose(0, 1)
    rows.copy_(xs[0].to(dev))
    full = torch.randint(0, W, (B, W), generator=g, dtype=torch.int32)
    sd.beam_reorder(rows, full.to(dev), out=rows)
    assert torch.equal(rows.cpu(), ref.reorder(xs[0], full)[0])
    assert int((buf[:, :, :13] + 7).abs().sum() + (buf[:, :, 63:] + 7).abs().sum()) == 0
    # more slots than rows: those that name no parent stay as they are
    more = torch.tensor([[0, 5, -1, 2, 1, 1, -1, 3]] * B, dtype=torch.int32)
    out = torch.full((B, 8, 50), 99, dtype=torch.int32, device=dev)
    sd.beam_reorder(xs[0].to(dev), more.to(dev), out=out)
    want, _ = ref.reorder(xs[0], more)
    want[:, 6] = 99
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("W", [2, 8, 9, 13, 32])
@pytest.mark.parametrize("row", [1, 15, 16, 17, 4096, 4097, 9001, 20000])
def test_reorder_rows_at_every_place_of_the_grid(dev, W, row):
    # rows and their neighbours: bytes around the rows stay as they are
    g = _g(row + W)
    B, gap = 2, 16 + row % 7
    for place in (0, 5):
        buf = torch.randint(0, 256, (place + B * W * (row + gap),), generator=g, dtype=torch.uint8)
        views = lambda t: t[place:].view(B, W, row + gap)[:, :, :row]
        p = torch.randint(-1, W, (B, W), generator=g, dtype=torch.int32)
        want, _ = ref.reorder(views(buf), p)
        there = buf.to(dev)
        assert torch.equal(sd.beam_reorder(views(there), p.to(dev)).cpu(), want)
        sd.beam_reorder(views(there), p.to(dev), out=views(there))
        left = buf.clone()
        views(left).copy_(want)
        assert torch.equal(there.cpu(), left)


def test_reorder_bad_parents(dev):
    x = _state((2, 3, 5), torch.int32, 5)
    p = torch.tensor([[3, 0, -2], [1, 1, 2]], dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    y = sd.beam_reorder(x.to(dev), p.to(dev), status=st)
    assert torch.equal(y.cpu(), ref.reorder(x, p)[0]) and int(st) == sd.SD_STATUS_BAD_PARENT


def test_reorder_into_rows_between_the_states(dev):
    B, W, V = 3, 5, 37
    x = _state((B, W, V), torch.int32, 7).to(dev)
    p = torch.randint(0, W, (B, W), generator=_g(8), dtype=torch.int32).to(dev)
    buf = torch.zeros((B, W, 2 * V), dtype=torch.int32, device=dev)
    buf[..., :V] = x
    got = sd.beam_reorder(buf[..., :V], p, out=buf[..., V:])
    assert torch.equal(got, sd.beam_reorder(x, p)) and torch.equal(buf[..., :V], x)
    with pytest.raises(ValueError, match="overlaps"):
        sd.beam_reorder(buf[..., :V], p, out=buf[..., V - 1:2 * V - 1])


def test_under_inference_mode(dev):
    with torch.inference_mode():
        x, s = _logits((2, 3, 500), F32, 30).to(dev), _scores(2, 3, 31).to(dev)
        b = sd.beam_select(x, s, 3)
        state = _state((2, 3, 9), torch.int32, 9).to(dev)
        want, _ = ref.reorder(state.cpu(), b.parents.cpu())
        assert torch.equal(sd.beam_reorder(state, b.parents, out=state).cpu(), want)


def test_reorder_offsets_past_32_bits(dev):
    n = 1_200_000_000
    x = torch.zeros((1, 3, n), dtype=torch.uint8, device=dev)
    for w in range(3):
        x[0, w, -5:] = w + 1
        x[0, w, 0] = 10 * w
    sd.beam_reorder(x, torch.tensor([[2, 0, 0]], dtype=torch.int32, device=dev), out=x)
    assert x[0, :, -1].tolist() == [3, 1, 1] and x[0, :, 0].tolist() == [20, 0, 0]


def test_reorder_refusals(dev):
    x = torch.zeros((2, 3, 10), dtype=torch.int32, device=dev)
    p = torch.zeros((2, 3), dtype=torch.int32, device=dev)
    for call in (lambda: sd.beam_reorder(x, p[:1]), lambda: sd.beam_reorder(x, p[0]),
                 lambda: sd.beam_reorder(x.transpose(1, 2), p), lambda: sd.beam_reorder(x[:, :, ::2], p),
                 lambda: sd.beam_reorder(x, p, out=x[:, :2]), lambda: sd.beam_reorder(x, p, out=x.flip(1)[:, :, :5]),
                 lambda: sd.beam_reorder([x] * 17, p), lambda: sd.beam_reorder([x, x], p, out=[x, x]),
                 lambda: sd.beam_reorder(x, torch.zeros((2, 4), dtype=torch.int32, device=dev)),
                 lambda: sd.beam_reorder(x[:, :, 1:], p, out=x[:, :, :-1])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        sd.beam_reorder(x, p, out=x[:, :1].expand(2, 3, 10))
    assert sd.beam_reorder([], p) == []
