"""Pools that run out, and tables that name pages which are not theirs any more: what the page calls
leave and say then does not depend on the order in which the GPU's threads run."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import pool_ref  # noqa: E402

sd = pytest.importorskip("speculative_decoding_verification_logits_gb300")

I32 = torch.int32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _sharing(rows, full, M, page, free):
    """Rows of `full` pages of their own and, in pairs, a shared and partly filled last one; a pool
    with `free` pages left: (table, kv_len, refs)."""
    ids = torch.arange(rows * full + rows, dtype=I32)
    t = torch.full((rows, M), -1, dtype=I32)
    t[:, :full] = ids[:rows * full].view(rows, full)
    t[:, full] = ids[rows * full:][torch.arange(rows) // 2]
    refs = torch.bincount(t[t >= 0].long(), minlength=len(ids)).to(I32)
    refs = torch.cat([refs[refs > 0], torch.zeros(free, dtype=I32)])
    return t, torch.full((rows,), full * page + 1, dtype=I32), refs


@pytest.mark.parametrize("rows,full", [(2, 0), (6, 3), (6, 600), (300, 5), (60, 700)])
@pytest.mark.parametrize("free", [0, 1, 3])
def test_extend_without_pages_says_so_alone(dev, rows, full, free):
    # the copies of shared last pages find no page: the tables are sound, so the status says no more
    M, page = full + 2, 4
    t, n, refs = _sharing(rows, full, M, page, free)
    for _ in range(10):
        td, rd, st = t.to(dev), refs.to(dev), torch.zeros(1, dtype=I32, device=dev)
        m = sd.kv_extend(td, n.to(dev), rd, page, 1, status=st)
        assert int(st) == (sd.SD_STATUS_NO_PAGE if free < rows else 0)
        assert torch.equal(td[:, :full].cpu(), t[:, :full])
        assert int(m.count) == rows and int((m.src >= 0).sum()) == min(free, rows)
        got = td[:min(free, rows), full].cpu()
        assert got.tolist() == list(range(len(refs) - free, len(refs)))[:rows]


def _check(dev, t, n, parents, refs, page, times=1, **more):
    """kv_fork (or kv_extend, without parents) held to the definition, the status too."""
    want = pool_ref.fork(t, n, parents, refs, page, **more)
    for _ in range(times):
        td, nd, rd = t.to(dev), n.to(dev), refs.to(dev)
        st = torch.zeros(1, dtype=I32, device=dev)
        if parents is None:
            m = sd.kv_extend(td, nd, rd, page, more["append"], status=st)
            got = (td, nd, *m, rd)
        else:
            got = (*sd.kv_fork(td, nd, parents.to(dev), rd, page, status=st, **more), rd)
            assert torch.equal(td.cpu(), t) and torch.equal(nd.cpu(), n)
        names = ("table", "len", "src", "dst", "fill", "count", "refs")
        for name, a, b in zip(names, got, want if parents is not None else (want[0], n, *want[2:])):
            assert torch.equal(a.cpu(), b), name
        assert int(st) == want[-1]
    return want


@pytest.mark.parametrize("rows,full", [(2, 0), (6, 3), (6, 600), (300, 5), (60, 700)])
@pytest.mark.parametrize("free", [0, 1, 2, 3, 7])
def test_rows_keep_last_pages_that_they_cannot_copy(dev, rows, full, free):
    page = 4
    t, n, refs = _sharing(rows, full, full + 4, page, free)
    for append in (0, 1, 9):
        want = _check(dev, t, n, None, refs, page, times=3, append=append)
        if free < rows:
            assert want[-1] == sd.SD_STATUS_NO_PAGE
            assert bool((want[0][:, full] >= 0).all())
            held = want[0][want[0] >= 0].long()
            assert torch.equal(torch.bincount(held, minlength=len(refs)).to(I32), want[6])
    g = torch.Generator().manual_seed(rows + free)
    for R in (1, rows, rows + 5):
        p = torch.randint(-1, rows, (R,), generator=g, dtype=I32)
        for keep in (False, True):
            _check(dev, t, n, p, refs, page, append=2, keep=keep)


def test_extend_again_after_pages_come_free(dev):
    # the entries of shared last pages outlast a pool that is full, and a later call copies them
    rows, full, page = 8, 2, 4
    t, n, refs = _sharing(rows, full, full + 2, page, 1)
    n += 1
    spare = torch.arange(len(refs), len(refs) + 12, dtype=I32)[None]
    refs = torch.cat([refs, torch.ones(12, dtype=I32)])
    td, nd, rd, sp = t.to(dev), n.to(dev), refs.to(dev), spare.to(dev)
    cache = torch.randint(0, 99, (1, len(refs), page, 3), dtype=I32, device=dev)
    read = lambda: cache[0, td.long().clamp(min=0)].flatten(1, 2)[:, :full * page + 2]
    before = read()
    st = torch.zeros(1, dtype=I32, device=dev)
    for status in (sd.SD_STATUS_NO_PAGE, 0):
        st.zero_()
        m = sd.kv_extend(td, nd, rd, page, 3, status=st)
        sd.kv_copy(cache, m.src, m.dst, count=m.count, fill=m.fill)
        assert int(st) == status and torch.equal(read(), before)
        if status:
            sd.kv_free(sp, rd)           # another request ends
            sd.kv_free(td[7:], rd)       # and one of the rows
            td, nd, before = td[:7].contiguous(), nd[:7].contiguous(), before[:7]
    # every row now writes into pages of its own
    for j in (full, full + 1):
        own = td[:, j]
        assert len(set(own.tolist())) == 7 and bool((rd[own.long()] == 1).all())


@pytest.mark.parametrize("groups,M", [(3, 5), (16, 20), (60, 9), (130, 300)])
@pytest.mark.parametrize("free", [0, 4, 60])
def test_fork_leaves_out_rows_that_were_given_back(dev, groups, M, free):
    # rows given back without clear name pages that are free by then, or that only others hold
    page, W = 4, 4
    g = torch.Generator().manual_seed(groups + free)
    shared = M // 2
    own = torch.randperm(groups * (shared + W * (M - 1 - shared)), generator=g).to(I32)
    t = torch.full((groups, W, M), -1, dtype=I32)
    t[:, :, :shared] = own[:groups * shared].view(groups, 1, shared)
    t[:, :, shared:M - 1] = own[groups * shared:].view(groups, W, -1)
    t = t.view(groups * W, M)
    n = torch.full((groups * W,), (M - 1) * page - 1, dtype=I32)
    refs = torch.bincount(t[t >= 0].long(), minlength=len(own)).to(I32)
    gone = torch.zeros(groups * W, dtype=torch.uint8)
    gone[torch.randperm(groups * W, generator=g)[:groups * W // 3]] = 1
    gone[0], gone[1] = 1, 0
    rd = torch.cat([refs, torch.zeros(free, dtype=I32)]).to(dev)
    sd.kv_free(t.to(dev), rd, which=gone.to(dev))
    refs = rd.cpu()
    left = (gone == 0).nonzero().flatten()
    for R in (len(left), groups * W):   # pages that were given back come into use again, or run out
        p = left[torch.randint(0, len(left), (R,), generator=g)].to(I32)
        want = _check(dev, t, n, p, refs, page, times=10, append=2)
        assert want[-1] & sd.SD_STATUS_BAD_PAGE
        new = want[0]
        taken = new[(new >= 0) & (refs[new.clamp(min=0).long()] == 0)].long()
        assert bool((want[6][taken] >= 1).all())
    _check(dev, t, n, p, refs, page, append=2, keep=True)


@pytest.mark.parametrize("rows", [6, 40, 900])
def test_fork_gives_back_more_than_is_held(dev, rows):
    # one page in every row, counted once: it gains holders and loses more of them, in any order
    t = torch.zeros((rows, 3), dtype=I32)
    t[:, 1:] = 1 + torch.arange(2 * rows, dtype=I32).view(rows, 2) // 4
    n = torch.full((rows,), 12, dtype=I32)
    refs = torch.ones(10 + rows, dtype=I32)
    g = torch.Generator().manual_seed(rows)
    for R in (1, rows // 2, rows, rows + 5):
        for held in (1, 2, rows // 2):
            refs[0] = held
            p = torch.randint(0, max(1, rows // 3), (R,), generator=g, dtype=I32)
            _check(dev, t, n, p, refs, 4, times=10)
