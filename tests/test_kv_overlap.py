"""Calls refuse arguments that they write and that share memory with others (the counts of pages above
all: they change while tables and lengths are read), and memory whose rows or pages overlap."""
import pytest
import torch

import speculative_decoding_verification_logits_gb300 as sd
from speculative_decoding_verification_logits_gb300 import kv


def test_which_addresses_overlap():
    for at, n, other, size in ((100, 4, 96, 5), (100, 4, 115, 1), (100, 4, 104, 4), (100, 4, 0, 1000)):
        with pytest.raises(ValueError, match="refs overlaps"):
            kv._apart("refs", at, n, (None, 50), (other, size))
    for at, n, other, size in ((100, 4, 96, 4), (100, 4, 116, 1), (100, 4, 108, 0), (100, 0, 96, 8),
                               (None, 4, 0, 1000), (100, 4, None, 8)):
        kv._apart("refs", at, n, (other, size))


def test_whether_pieces_lie_apart():
    g = torch.Generator().manual_seed(1)
    seen = set()
    for _ in range(3000):
        size, *dims = torch.randint(0, 9, (7,), generator=g).tolist()
        dims = list(zip(dims[:3], dims[3:]))
        used = [i * dims[0][1] + j * dims[1][1] + k * dims[2][1] + b for i in range(dims[0][0])
                for j in range(dims[1][0]) for k in range(dims[2][0]) for b in range(size)]
        want = len(set(used)) == len(used)
        assert kv._lie_apart(size, *dims) == want, (size, dims)
        seen.add(want)
    assert len(seen) == 2 and kv._lie_apart(4, (2, 8), (2, 12)) and not kv._lie_apart(4, (2, 8), (3, 4))


@pytest.mark.gpu
def test_refusals_of_rows_and_pages_that_overlap():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    buf = torch.arange(600, dtype=torch.int32, device="cuda:0")
    p = torch.tensor([[1, 0, 1], [2, 2, 0]], dtype=torch.int32, device="cuda:0")
    x = buf[300:330].view(2, 3, 5)
    before = buf.clone()
    for strides in ((30, 4, 1), (4, 30, 1), (15, 0, 1), (0, 5, 1), (12, 5, 1), (8, 6, 1)):
        y = torch.as_strided(buf, (2, 3, 5), strides)
        for call in (lambda: sd.beam_reorder(x, p, out=y), lambda: sd.beam_reorder(y, p, out=y)):
            with pytest.raises(ValueError, match="overlap"):
                call()
    i = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda:0")
    for shape, strides in (((2, 3, 4, 2), (30, 7, 2, 1)), ((2, 3, 4, 2), (8, 0, 2, 1)),
                           ((2, 3, 4, 2), (8, 8, 2, 1))):
        with pytest.raises(ValueError, match="overlap"):
            sd.kv_copy(torch.as_strided(buf, shape, strides), i(0), i(1))
    assert torch.equal(buf, before)
    # rows of one sequence between those of another, pages of one layer between another's
    y = torch.as_strided(buf, (2, 3, 5), (5, 11, 1))
    sd.beam_reorder(x, p, out=y)
    assert torch.equal(y, x.gather(1, p.long()[..., None].expand(2, 3, 5)))
    c = torch.as_strided(buf, (2, 3, 4, 2), (8, 17, 2, 1))
    want = c.clone()
    want[:, 2] = want[:, 0]
    sd.kv_copy(c, i(0), i(2))
    assert torch.equal(c, want)


@pytest.mark.gpu
def test_refusals():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    buf = torch.zeros(200, dtype=torch.int32, device="cuda:0")
    t, n, p, r, st = buf[:12].view(4, 3), buf[12:16], buf[16:20], buf[20:60], buf[60:61]
    flags = buf[100:101].view(torch.uint8)
    pool = lambda x: torch.as_strided(buf, (40,), (1,), x)   # counts that begin at place x
    for call in (lambda r=r, st=st, n=n, p=p: sd.kv_fork(t, n, p, r, 4, append=1, status=st),
                 lambda r=r, st=st, n=n: sd.kv_extend(t, n, r, 4, 1, status=st),
                 lambda r=r, st=st, n=n: sd.kv_free(t, r, which=flags, count=n[:1], clear=True, status=st),
                 lambda r=r, st=st: sd.kv_compact(r, t, status=st)):
        names = call.__code__.co_varnames[:call.__code__.co_argcount]
        bad = [dict(r=pool(11)), dict(r=pool(60)), dict(st=r[3:4]),
               dict(st=t[1, 1:2])]
        if "n" in names:
            bad += [dict(r=pool(12)), dict(st=n[:1]), dict(n=r[:4])]
        if "p" in names:
            bad += [dict(r=pool(19)), dict(st=p[1:2]), dict(p=r[:4])]
        elif "n" in names:   # the table is written
            bad += [dict(n=t.view(-1)[2:6])]
        for change in bad:
            with pytest.raises(ValueError, match="overlaps"):
                call(**change)
        call()               # apart, though of one block
    with pytest.raises(ValueError, match="overlaps"):
        sd.kv_free(t, pool(80), which=flags)
    assert sd.kv_free(t, r, count=r.new_zeros(1)) is r
