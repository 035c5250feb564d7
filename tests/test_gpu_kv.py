"""The page operators of a shared cache (fork, extend, free, compact, copy) against their
definitions, and a run of them together."""
import pytest
import torch

from tests import beam_ref as ref

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_logits_gb300")

I32 = torch.int32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _g(seed):
    return torch.Generator().manual_seed(seed)


def _ints(lo, hi, shape, g):
    return torch.randint(lo, hi, shape, generator=g, dtype=I32)


def _tables(B, W, M, page, g, free=20, reserve=0):
    """Tables of B groups of W rows that share a prefix, refs that count them, lengths."""
    rows = B * W
    t = torch.full((rows, M), -1, dtype=I32)
    n = torch.zeros(rows, dtype=I32)
    ids = iter(torch.randperm(rows * M + free, generator=g).tolist())
    for b in range(B):
        pre = int(_ints(0, max(M // 2, 1), (1,), g))
        shared = [next(ids) for _ in range(pre)]
        for w in range(W):
            r = b * W + w
            own = int(_ints(0, M - pre + 1, (1,), g))
            for j, p in enumerate(shared + [next(ids) for _ in range(own)]):
                t[r, j] = p
            held = pre + own
            used = max(held - reserve, pre)
            part = int(_ints(0, page, (1,), g)) if used > pre else 0
            n[r] = max(used * page - part, 0)
            if reserve == 0 and used > pre and part:
                continue
    N = rows * M + free
    refs = torch.bincount(t[t >= 0].long(), minlength=N).to(I32)
    return t, n, refs


def _check_fork(dev, t, n, parents, refs, page, **more):
    td, nd, rd = t.to(dev), n.to(dev), refs.to(dev)
    st = torch.zeros(1, dtype=I32, device=dev)
    f = sd.kv_fork(td, nd, parents.to(dev), rd, page, status=st, **more)
    groups = parents.shape[0] if parents.dim() == 2 else 0
    want = ref.fork(t, n, parents, refs, page, groups=groups, **more)
    for name, a, b in zip((*f._fields, "refs"), (*f, rd), want):
        assert torch.equal(a.cpu(), b), name
    assert int(st) == want[-1]
    assert torch.equal(td.cpu(), t) and torch.equal(nd.cpu(), n)
    return f, rd, want


# --------------------------------------------------------------------- fork --
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("B,W,M,page,append", [
    (1, 1, 1, 1, 0), (1, 4, 5, 16, 1), (3, 4, 7, 4, 0), (2, 8, 33, 16, 1), (5, 3, 64, 2, 9),
    (16, 4, 130, 16, 33), (1, 32, 20, 8, 70), (300, 8, 12, 16, 1)])
def test_fork(dev, keep, B, W, M, page, append):
    for seed, reserve in ((1, 0), (2, 2)):
        g = _g(seed + M)
        t, n, refs = _tables(B, W, M, page, g, free=4 * B * W + 40, reserve=reserve)
        _check_fork(dev, t, n, _ints(0, W, (B, W), g), refs, page, append=append, keep=keep)
        rows = B * W
        for R in (1, rows, rows + 3):
            _check_fork(dev, t, n, _ints(-1, rows, (R,), g), refs, page, append=append, keep=keep)


def test_fork_other_widths_of_groups(dev):
    g = _g(4)
    t, n, refs = _tables(6, 1, 9, 4, g, free=80)
    _check_fork(dev, t, n, torch.zeros((6, 5), dtype=I32), refs, 4, append=1, keep=True)
    t, n, refs = _tables(6, 5, 9, 4, g, free=80)
    _check_fork(dev, t, n, _ints(-1, 5, (6, 2), g), refs, 4, append=1)


def test_fork_identity_changes_nothing(dev):
    g = _g(5)
    t, n, refs = _tables(4, 3, 10, 4, g)
    f, rd, _ = _check_fork(dev, t, n, torch.arange(12, dtype=I32), refs, 4)
    assert torch.equal(f.block_table.cpu(), t) and torch.equal(rd.cpu(), refs) and int(f.count) == 0


def test_fork_with_too_few_pages_and_full_tables(dev):
    g = _g(6)
    for free in (0, 1, 3):
        t, n, refs = _tables(3, 4, 6, 4, g, free=0)
        zero = (refs == 0).nonzero().flatten()
        refs[zero[free:]] = 1   # pages that others hold
        p = _ints(0, 4, (3, 4), g)
        _, _, want = _check_fork(dev, t, n, p, refs, 4, append=5)
        _check_fork(dev, t, n, p, refs, 4, append=100, keep=True)
        assert want[-1] & sd.SD_STATUS_NO_PAGE


def test_fork_bad_parents_pages_and_lengths(dev):
    g = _g(7)
    t, n, refs = _tables(3, 4, 6, 4, g, free=60)
    _check_fork(dev, t, n, torch.tensor([-5, 0, 12, 3, -1, 2 ** 31 - 1], dtype=I32), refs, 4)
    _check_fork(dev, t, n, torch.tensor([[0, 4, 1], [-2, 3, 3], [-1, -1, 0]], dtype=I32), refs, 4)
    n2 = n.clone()
    n2[0], n2[1], n2[2] = -9, 10 ** 6, 2 ** 31 - 1
    _check_fork(dev, t, n2, _ints(0, 12, (12,), g), refs, 4, append=2, keep=True)
    t2 = t.clone()
    t2[1, 0], t2[3, 1], t2[5, 0] = 10 ** 9, -7, -1
    for keep in (False, True):
        _check_fork(dev, t2, n, _ints(0, 12, (12,), g), refs, 4, append=2, keep=keep)


def test_fork_shared_partial_pages(dev):
    # rows that share a partly filled page (a rollback past a fork leaves them): all go their own way
    t = torch.tensor([[4, 2, -1], [4, 2, 7], [4, 3, -1]], dtype=I32)
    n = torch.tensor([6, 5, 8], dtype=I32)
    refs = torch.bincount(t[t >= 0].long(), minlength=40).to(I32)
    for p in ([0, 1, 2], [1, 0, 0], [2, 2, 1]):
        for keep in (False, True):
            _check_fork(dev, t, n, torch.tensor(p, dtype=I32), refs, 4, append=1, keep=keep)


def test_fork_of_a_large_pool_and_a_long_row(dev):
    # many chunks of the pool, free pages far apart, a row that needs hundreds of pages
    g = _g(8)
    N, M = 200_003, 1300
    refs = (torch.rand(N, generator=g) < 0.997).to(I32)
    refs[:70_000] = 1
    t = torch.full((3, M), -1, dtype=I32)
    held = refs.nonzero().flatten()[:200].to(I32)
    t[0, :100], t[1, :100] = held[:100], held[100:]
    n = torch.tensor([100 * 16 - 3, 100 * 16, 0], dtype=I32)
    for keep in (False, True):
        _check_fork(dev, t, n, torch.tensor([0, 1, 0, 2], dtype=I32), refs, 16, append=2000, keep=keep)
        _check_fork(dev, t, n, torch.tensor([1], dtype=I32), refs, 16, append=20000, keep=keep)


def test_fork_many_rows(dev):
    g = _g(9)
    rows, M, page = 16384, 3, 4
    t = torch.randperm(rows * M, generator=g).to(I32).reshape(rows, M)
    t[:, 2] = -1
    n = _ints(1, 2 * page + 1, (rows,), g)
    t[n <= page, 1] = -1
    refs = torch.bincount(t[t >= 0].long(), minlength=2 * rows * M).to(I32)
    _check_fork(dev, t, n, _ints(0, rows, (rows,), g), refs, page, append=1)


@pytest.mark.parametrize("append", [0, 1, 9, 40])
def test_extend(dev, append):
    g = _g(10 + append)
    for reserve in (0, 2):
        t, n, refs = _tables(4, 3, 30, 4, g, free=200, reserve=reserve)
        td, rd = t.to(dev), refs.to(dev)
        st = torch.zeros(1, dtype=I32, device=dev)
        m = sd.kv_extend(td, n.to(dev), rd, 4, append, status=st)
        want = ref.fork(t, n, None, refs, 4, append=append)
        for a, b in zip((td, *m, rd), (want[0], *want[2:7])):
            assert torch.equal(a.cpu(), b)
        assert int(st) == want[-1]


def test_extend_prompts_and_a_shared_last_page(dev):
    t = torch.full((3, 600), -1, dtype=I32)
    t[1, :2] = torch.tensor([5, 9])
    t[2, :2] = torch.tensor([5, 9])
    n, refs = torch.tensor([0, 20, 30], dtype=I32), torch.zeros(3000, dtype=I32)
    refs[5] = refs[9] = 2
    td, rd = t.to(dev), refs.to(dev)
    m = sd.kv_extend(td, n.to(dev), rd, 16, 8192)
    want = ref.fork(t, n, None, refs, 16, append=8192)
    for a, b in zip((td, *m, rd), (want[0], *want[2:7])):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("rows", [12, 600])
def test_extend_rows_that_share_their_last_pages(dev, rows):
    # every row copies its last page in place while its old one is given back
    g = _g(rows)
    M, page = 40, 8
    t = torch.full((rows, M), -1, dtype=I32)
    ids = torch.randperm(4000 + rows * 8, generator=g).to(I32)
    n = torch.zeros(rows, dtype=I32)
    for r in range(0, rows, 3):
        held = int(_ints(1, 30, (1,), g))
        t[r:r + 3, :held] = ids[r * 10 % 3000:][:held]
        n[r:r + 3] = held * page - int(_ints(0, page, (1,), g))
    refs = torch.bincount(t[t >= 0].long(), minlength=len(ids)).to(I32)
    want = ref.fork(t, n, None, refs, page, append=9)
    assert int(want[5]) > rows // 3
    for _ in range(20):
        td, rd = t.to(dev), refs.to(dev)
        m = sd.kv_extend(td, n.to(dev), rd, page, 9)
        for a, b in zip((td, *m, rd), (want[0], *want[2:7])):
            assert torch.equal(a.cpu(), b)


def test_fork_given_outputs_and_refusals(dev):
    g = _g(11)
    t, n, refs = _tables(2, 3, 5, 4, g)
    td, nd, rd = t.to(dev), n.to(dev), refs.to(dev)
    p = _ints(0, 6, (4,), g).to(dev)
    want = sd.kv_fork(td, nd, p, rd.clone(), 4, append=1)
    out = sd.KVFork(*(torch.full_like(x, 77) for x in want))
    r2 = rd.clone()
    v = [x._version for x in (*out, r2)]
    got = sd.kv_fork(td, nd, p, r2, 4, append=1, out=out)
    assert got is out and all(torch.equal(a, b) for a, b in zip(got, want))
    assert [x._version for x in (*out, r2)] == [x + 1 for x in v]
    for bad in (lambda: sd.kv_fork(td, nd, p, rd, 4, out=out._replace(block_table=td[:4])),
                lambda: sd.kv_fork(td, nd, p, rd, 4, out=out._replace(src=out.dst)),
                lambda: sd.kv_fork(td, nd, p, rd, 4, out=out._replace(fill=p)),
                lambda: sd.kv_fork(td, nd, p.view(2, 2)[:, :0], rd, 4),
                lambda: sd.kv_fork(td[:5], nd[:5], p.view(2, 2), rd, 4),
                lambda: sd.kv_fork(td, nd[:3], p, rd, 4), lambda: sd.kv_fork(td[0], nd, p, rd, 4),
                lambda: sd.kv_fork(td, nd, p, rd[:0], 4)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sd.kv_fork(td, nd, p, rd, 4, append=2 ** 32 + 1),
                lambda: sd.kv_extend(td, nd, rd, 2 ** 32 + 4, 1)):
        with pytest.raises(ValueError, match="out of range"):
            bad()
    for bad in (lambda: sd.kv_fork(td.long(), nd, p, rd, 4), lambda: sd.kv_fork(td, nd, p.long(), rd, 4),
                lambda: sd.kv_fork(td, nd, p, rd.float(), 4)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: sd.kv_fork(td, nd, p, rd, 0), lambda: sd.kv_fork(td, nd, p, rd, 4, append=-1)):
        with pytest.raises(sd.SDError):
            bad()


def test_fork_of_no_rows_no_slots_and_no_entries(dev):
    i = lambda *s: torch.zeros(s, dtype=I32, device=dev)
    refs = torch.ones(3, dtype=I32, device=dev)
    refs[1] = 0
    # from an empty table: empty rows, or bad parents
    st = i(1)
    f = sd.kv_fork(i(0, 4), i(0), torch.tensor([-1, 0], dtype=I32, device=dev), refs, 4, append=3,
                   status=st)
    assert f.block_table.tolist() == [[-1] * 4] * 2 and f.kv_len.tolist() == [0, 0]
    assert int(st) == sd.SD_STATUS_BAD_PARENT and refs.tolist() == [1, 0, 1]
    # tables without slots
    f = sd.kv_fork(i(2, 0), i(2) + 7, i(3), refs, 4)
    assert f.block_table.shape == (3, 0) and f.kv_len.tolist() == [0, 0, 0]
    # extending nothing, and empty rows
    m = sd.kv_extend(i(0, 4), i(0), refs, 4, 5)
    assert m.count.tolist() == [0] and m.src.numel() == 0
    t = i(1, 4) - 1
    sd.kv_extend(t, i(1), refs, 4, 1)
    assert t.tolist() == [[1, -1, -1, -1]] and refs.tolist() == [1, 1, 1]
    assert sd.kv_free(i(0, 4), refs, which=torch.zeros(0, dtype=torch.uint8, device=dev)) is refs
    one = torch.ones(1, dtype=I32, device=dev)
    c = sd.kv_compact(one)
    assert c.src.numel() == 0 and c.live.tolist() == [1] and c.new_ids.tolist() == [0]


# --------------------------------------------------------------------- free --
@pytest.mark.parametrize("rows,M", [(1, 1), (3, 7), (64, 513), (200, 1025)])
def test_free_rows_and_lists(dev, rows, M):
    g = _g(rows + M)
    N = rows * M + 5
    t = _ints(-1, N, (rows, M), g)
    refs = torch.bincount(t[t >= 0].long(), minlength=N).to(I32)
    which = _ints(0, 2, (rows,), g).to(torch.uint8)
    for more in (dict(which=which), dict(which=which, clear=True), dict(clear=True), dict(),
                 dict(count=torch.tensor([rows * M // 2], dtype=I32)),
                 dict(count=torch.tensor([rows * M // 2], dtype=I32), which=which, clear=True),
                 dict(count=torch.tensor([-4], dtype=I32)),
                 dict(count=torch.tensor([10 ** 9], dtype=I32), clear=True)):
        td, rd = t.to(dev), refs.to(dev)
        st = torch.zeros(1, dtype=I32, device=dev)
        there = {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in more.items()}
        assert sd.kv_free(td, rd, status=st, **there) is rd
        r, left, status = ref.free(t, refs, **more)
        assert torch.equal(rd.cpu(), r) and torch.equal(td.cpu(), left) and int(st) == status == 0


def test_free_twice_and_foreign_ids(dev):
    t = torch.tensor([3, 3, 3, 1, -1, 9, 4, 4, 2 ** 31 - 1, -2], dtype=I32)
    refs = torch.tensor([1, 0, 1, 2, 2], dtype=I32)
    rd, st = refs.to(dev), torch.zeros(1, dtype=I32, device=dev)
    sd.kv_free(t.to(dev), rd, status=st)
    want, _, status = ref.free(t[None], refs)
    assert torch.equal(rd.cpu(), want) and int(st) == status == sd.SD_STATUS_BAD_PAGE
    assert want.tolist() == [1, 0, 1, 0, 0]


def test_free_takes_the_list_of_a_rollback(dev):
    g = _g(12)
    B, M, page, K = 7, 12, 4, 9
    t, n, refs = _tables(1, B, M, page, g)
    n = n + K + 1
    td, nd, rd = t.to(dev), n.to(dev), refs.to(dev)
    m = sd.kv_extend(td, (n - K - 1).to(dev), rd, page, K + 1)
    held = td.clone()
    tau = _ints(1, K + 2, (B,), g)
    _, freed, off = sd.kv_rollback(td, nd, tau.to(dev), page, K + 1)
    sd.kv_free(freed, rd, count=off[-1:])
    left = td.cpu()
    assert torch.equal(rd.cpu(), torch.bincount(left[left >= 0].long(), minlength=len(refs)).to(I32))
    assert int((held >= 0).sum()) > int((left >= 0).sum()) and int(m.count) >= 0


def test_free_refusals(dev):
    t, r = torch.zeros((2, 3), dtype=I32, device=dev), torch.ones(4, dtype=I32, device=dev)
    w = torch.ones(2, dtype=torch.uint8, device=dev)
    for bad in (lambda: sd.kv_free(t, r, which=w[:1]), lambda: sd.kv_free(t.flatten(), r, which=w),
                lambda: sd.kv_free(t, r, count=r[:2]), lambda: sd.kv_free(t, r.view(2, 2)),
                lambda: sd.kv_free(r, r), lambda: sd.kv_free(t.t(), r)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        sd.kv_free(t, r, which=w.bool())


# ------------------------------------------------------------------ compact --
@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 1000, 8191, 8192, 8193, 50000, 200_001])
def test_compact(dev, N):
    for live in (0.0, 0.3, 0.97, 1.0):
        g = _g(N + int(10 * live))
        refs = (torch.rand(N, generator=g) < live).to(I32) * _ints(1, 5, (N,), g)
        used = refs.nonzero().flatten().to(I32)
        t = torch.full((6, 11), -1, dtype=I32)
        if len(used):
            t = used[torch.randint(0, len(used), (6, 11), generator=g)]
            t[torch.rand((6, 11), generator=g) < 0.2] = -1
        rd, td = refs.to(dev), t.to(dev)
        st = torch.zeros(1, dtype=I32, device=dev)
        c = sd.kv_compact(rd, td, status=st)
        *want, r, left, status = ref.compact(refs, t)
        for name, a, b in zip(c._fields, c, want):
            assert torch.equal(a.cpu(), b), name
        assert torch.equal(rd.cpu(), r) and torch.equal(td.cpu(), left) and int(st) == status == 0
        again = sd.kv_compact(rd, td)     # what is compact stays as it is
        assert int(again.count) == 0 and torch.equal(rd.cpu(), r) and torch.equal(td.cpu(), left)


def test_compact_bad_tables_and_no_table(dev):
    refs = torch.tensor([0, 2, 0, 0, 1, 3, 0], dtype=I32)
    t = torch.tensor([5, 0, 99, -3, 4, -1, 2 ** 31 - 1, 1], dtype=I32)
    rd, td, st = refs.to(dev), t.to(dev), torch.zeros(1, dtype=I32, device=dev)
    sd.kv_compact(rd, td, status=st)
    *_, r, left, status = ref.compact(refs, t)
    assert torch.equal(td.cpu(), left) and int(st) == status == sd.SD_STATUS_BAD_PAGE
    rd = refs.to(dev)
    sd.kv_compact(rd)
    assert torch.equal(rd.cpu(), r)
    with pytest.raises(ValueError):
        sd.kv_compact(rd, rd)


# --------------------------------------------------------------------- copy --
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("dtype,dim", [(torch.bfloat16, 64), (torch.float32, 33), (torch.uint8, 80),
                                       (torch.uint8, 7), (torch.bfloat16, 5), (torch.float64, 3)])
def test_copy(dev, dtype, dim, heads_first):
    g = _g(dim)
    L, N, H, page, n = 3, 40, 2, 16, 12
    shape = (L, N, H, page, dim) if heads_first else (L, N, page, H, dim)
    c = torch.randint(0, 200, shape, generator=g).to(dtype)
    ids = torch.randperm(N, generator=g).to(I32)
    src, dst = ids[:n].clone(), ids[n:2 * n].clone()
    src[2] = src[3]                    # one page to two places
    src[5] = dst[5] = -1
    fill = _ints(-2, page + 4, (n,), g)
    for count in (None, 0, 7, 100):
        for f in (None, fill):
            cd = c.to(dev)
            there = dict(count=None if count is None else torch.tensor([count], dtype=I32, device=dev),
                         fill=None if f is None else f.to(dev), heads_first=heads_first)
            v = cd._version
            sd.kv_copy(cd, src.to(dev), dst.to(dev), **there)
            want, _ = ref.copy(c, src, dst, count=count, fill=f, heads_first=heads_first)
            assert torch.equal(cd.cpu(), want) and cd._version == v + 1
            parts = [x.to(dev) for x in c]     # the layers as tensors of their own
            sd.kv_copy(parts, src.to(dev), dst.to(dev), **there)
            assert torch.equal(torch.stack(parts).cpu(), want)


@pytest.mark.parametrize("page,entry", [(16, 1), (16, 33), (7, 16), (3, 5), (16, 66), (64, 1040)])
def test_copy_of_entries_that_end_inside_a_vector(dev, page, entry):
    g = _g(page * entry)
    c = torch.randint(0, 256, (2, 30, page, entry), generator=g, dtype=torch.uint8)
    ids = torch.randperm(30, generator=g).to(I32)
    src, dst = ids[:15], ids[15:]
    fill = torch.arange(15, dtype=I32) % (page + 1)
    cd = c.to(dev)
    sd.kv_copy(cd, src.to(dev), dst.to(dev), fill=fill.to(dev))
    assert torch.equal(cd.cpu(), ref.copy(c, src, dst, fill=fill)[0])


def test_extend_many_rows(dev):
    g = _g(77)
    t, n, refs = _tables(75, 4, 11, 4, g, free=3000, reserve=1)
    refs[:] = torch.bincount(t[t >= 0].long(), minlength=len(refs)).to(I32)
    td, rd = t.to(dev), refs.to(dev)
    st = torch.zeros(1, dtype=I32, device=dev)
    m = sd.kv_extend(td, n.to(dev), rd, 4, 6, status=st)
    want = ref.fork(t, n, None, refs, 4, append=6)
    for a, b in zip((td, *m, rd), (want[0], *want[2:7])):
        assert torch.equal(a.cpu(), b)
    assert int(st) == want[-1]


def test_copy_strides_bad_ids_and_large_pages(dev):
    g = _g(14)
    buf = torch.randint(0, 99, (30, 5, 16, 24), generator=g, dtype=torch.int16).to(dev)
    before = buf.clone()
    view = buf[:, 1:4].transpose(0, 1)          # [layers][N], pages of all layers side by side
    src, dst = torch.tensor([3, 30, 7, -1, -2], dtype=I32), torch.tensor([9, 1, -1, -1, 0], dtype=I32)
    st = torch.zeros(1, dtype=I32, device=dev)
    sd.kv_copy(view, src.to(dev), dst.to(dev), status=st)
    want, status = ref.copy(before[:, 1:4].transpose(0, 1).cpu(), src, dst)
    assert torch.equal(view.cpu(), want) and int(st) == status == sd.SD_STATUS_BAD_PAGE
    assert torch.equal(buf[:, 0], before[:, 0]) and torch.equal(buf[:, 4], before[:, 4])
    big = torch.randint(0, 99, (1, 6, 64, 8, 1024), generator=g, dtype=torch.int32).to(dev)
    src, dst = torch.tensor([5, 0], dtype=I32, device=dev), torch.tensor([2, 1], dtype=I32, device=dev)
    want, _ = ref.copy(big.cpu(), src, dst, fill=torch.tensor([63, 17]))
    sd.kv_copy(big, src, dst, fill=torch.tensor([63, 17], dtype=I32, device=dev))
    assert torch.equal(big.cpu(), want)


def test_copy_offsets_past_32_bits(dev):
    c = torch.zeros((2, 70_000, 16, 2048), dtype=torch.uint8, device=dev)   # 4.6 GB
    c[:, 69_998], c[1, 5] = 3, 9
    i = lambda *v: torch.tensor(v, dtype=I32, device=dev)
    sd.kv_copy(c, i(69_998, 5), i(1, 69_999))
    assert int(c[0, 1].sum()) == 3 * 16 * 2048 and int(c[1, 69_999].sum()) == 9 * 16 * 2048
    assert int(c[0, 69_999].sum()) == 0


def test_copy_refusals(dev):
    c = torch.zeros((2, 5, 16, 4), device=dev)
    i = torch.zeros(2, dtype=I32, device=dev)
    for bad in (lambda: sd.kv_copy(c.transpose(2, 3), i, i), lambda: sd.kv_copy(c[0, 0], i, i),
                lambda: sd.kv_copy([c[0], c[1, :4]], i, i), lambda: sd.kv_copy(c, i, i[:1]),
                lambda: sd.kv_copy(c, i.view(2, 1), i.view(2, 1)), lambda: sd.kv_copy(c, i, i, count=i),
                lambda: sd.kv_copy(c, i, i, fill=i[:1]), lambda: sd.kv_copy(c[:, :1].expand(2, 5, 16, 4), i, i),
                lambda: sd.kv_copy([c[0, :, 0, 0]], i, i), lambda: sd.kv_copy([c[0]] * 257, i, i),
                lambda: sd.kv_copy([c[0, :, :, 0].contiguous()], i, i, fill=i, heads_first=True)):
        with pytest.raises(ValueError):
            bad()
    assert sd.kv_copy([], i, i) is None and sd.kv_copy(c[:0], i, i) is None


# ----------------------------------------------------------------- together --
def test_graph_of_the_page_operators(dev):
    g = _g(15)
    t, n, refs = _tables(3, 4, 9, 4, g, free=70)
    p = _ints(0, 4, (3, 4), g)
    cache = torch.randint(0, 99, (2, len(refs), 4, 8), generator=g, dtype=I32)
    td, nd, pd, rd, cd = (x.to(dev) for x in (t, n, p, refs, cache))

    def step():
        f = sd.kv_fork(td, nd, pd, rd, 4, append=1)
        sd.kv_copy(cd, f.src, f.dst, count=f.count, fill=f.fill)
        sd.kv_free(f.block_table, rd, which=which)
        c = sd.kv_compact(rd)
        sd.kv_copy(cd, c.src, c.dst, count=c.count)
        return f, c

    which = torch.zeros(12, dtype=torch.uint8, device=dev)
    which[3] = 1
    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (rd, cd)]
    rd.copy_(refs)
    cd.copy_(cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, c = step()
    for _ in range(2):
        rd.copy_(refs)
        cd.copy_(cache)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rd, want[0]) and torch.equal(cd, want[1])
        assert torch.equal(f.block_table.cpu(), ref.fork(t, n, p, refs, 4, append=1, groups=3)[0])


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_rows_keep_their_texts_through_a_life_of_forks(dev, seed):
    """Rows of a shared cache, written one entry at a time: whatever is forked, rolled back, given
    back and moved, each row reads the text that it should hold."""
    g = _g(seed)
    B, W, M, page, N = 3, 4, 24, 4, 400
    rows = B * W
    cache = torch.full((2, N, page, 3), -1, dtype=I32, device=dev)
    refs = torch.zeros(N, dtype=I32, device=dev)
    table = torch.full((rows, M), -1, dtype=I32, device=dev)
    n = torch.zeros(rows, dtype=I32, device=dev)
    texts = [[] for _ in range(rows)]
    st = torch.zeros(1, dtype=I32, device=dev)

    def write(k):
        m = sd.kv_extend(table, n, refs, page, k, status=st)
        sd.kv_copy(cache, m.src, m.dst, count=m.count, fill=m.fill)
        tok = _ints(0, 10 ** 6, (rows, k), g)
        for i in range(k):
            at = n.long() + i
            pg = table.gather(1, (at // page)[:, None])[:, 0].long()
            cache[:, pg, at % page] = tok[:, i].to(dev)[None, :, None]
        n.add_(k)
        for r in range(rows):
            texts[r] += tok[r].tolist()

    def read():
        pos = torch.arange(M * page, device=dev)
        pg = table.long().clamp(min=0).repeat_interleave(page, 1)
        have = cache[:, pg, (pos % page).expand_as(pg)]
        for r in range(rows):
            k = int(n[r])
            assert k == len(texts[r])
            want = torch.tensor(texts[r], dtype=I32, device=dev)
            assert torch.equal(have[:, r, :k], want[None, :, None].expand(2, k, 3))
        live = table[table >= 0]
        assert torch.equal(refs, torch.bincount(live.long(), minlength=N).to(I32))
        assert int(st) == 0

    for step in range(12):
        write(int(_ints(1, 5, (1,), g)))
        read()
        if step % 3 != 2:      # beams go on from their parents
            p = _ints(0, W, (B, W), g)
            f = sd.kv_fork(table, n, p.to(dev), refs, page, append=1, status=st)
            sd.kv_copy(cache, f.src, f.dst, count=f.count, fill=f.fill)
            table, n = f.block_table.clone(), f.kv_len.clone()
            texts = [list(texts[b * W + int(p[b, w])]) for b in range(B) for w in range(W)]
            read()
        else:                  # a round's drafts, of which some are taken back
            tau = _ints(1, 4, (rows,), g)
            write(3)
            n2, freed, off = sd.kv_rollback(table, n, tau.to(dev), page, 3)
            sd.kv_free(freed, refs, count=off[-1:], status=st)
            texts = [t[:len(t) - 3 + int(tau[r])] for r, t in enumerate(texts)]
            n = n2
            read()
        if step % 4 == 3:      # requests end, others start
            which = _ints(0, 2, (rows,), g).to(torch.uint8)
            sd.kv_free(table, refs, which=which.to(dev), clear=True, status=st)
            n[which.to(dev) > 0] = 0
            texts = [[] if int(which[r]) else t for r, t in enumerate(texts)]
            read()
            c = sd.kv_compact(refs, table, status=st)
            sd.kv_copy(cache, c.src, c.dst, count=c.count, status=st)
            assert int(refs[int(c.live):].sum()) == 0
            read()
