"""The definition of forks in pools that run out: by hand, and against the other definition where no
pool runs out."""
import torch

from tests import beam_ref, pool_ref

i32 = lambda v: torch.tensor(v, dtype=torch.int32)


def test_by_hand():
    # two rows of 6 entries share a last page of size 4; two pages, then one, then none are free
    t, n = i32([[2, 3, -1], [2, 3, -1]]), i32([6, 6])
    want = ([[2, 0, -1], [2, 1, -1]], [(3, 0, 2), (3, 1, 2)], [1, 1, 2, 0], 0), \
           ([[2, 0, -1], [2, 3, -1]], [(3, 0, 2), (-1, -1, 2)], [1, 1, 2, 1], pool_ref.NO_PAGE), \
           ([[2, 3, -1], [2, 3, -1]], [(-1, -1, 2)] * 2, [1, 1, 2, 2], pool_ref.NO_PAGE)
    for used, (table, pairs, refs, status) in enumerate(want):
        before = i32([used > 1, used > 0, 2, 2])
        got = pool_ref.fork(t, n, None, before, 4, append=1)
        assert got[0].tolist() == table and list(zip(*(v.tolist() for v in got[2:5]))) == pairs
        assert got[5].tolist() == [2] and got[6].tolist() == refs and got[7] == status
    # forked: the heir keeps what it cannot copy, another row of the parent has no such page to keep
    got = pool_ref.fork(t, n, i32([0, 0, 1]), i32([1, 1, 2, 2]), 4)
    assert got[0].tolist() == [[2, 3, -1], [2, -1, -1], [2, 3, -1]] and got[6].tolist() == [1, 1, 3, 2]
    # a row that ends gives its own back
    got = pool_ref.fork(t, n, i32([1]), i32([1, 1, 2, 2]), 4)
    assert got[0].tolist() == [[2, 3, -1]] and got[6].tolist() == [1, 1, 1, 1]


def test_definitions_agree_while_pages_last():
    for seed in range(300):
        g = torch.Generator().manual_seed(seed)
        ints = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.int32)
        rows, M, page = (int(ints(1, 9, 1)) for _ in range(3))
        N = 3 * rows * M + 20
        t = ints(0, max(1, rows * M), rows, M)
        if seed % 2:
            t[1:, :M // 2] = t[:1, :M // 2]
        n = ints(0, M * page + 1, rows)
        t[torch.arange(M) >= (n[:, None] + page - 1) // page] = -1
        refs = torch.bincount(t[t >= 0].long(), minlength=N).to(torch.int32)
        app = int(ints(0, 9, 1))
        for parents in (None, ints(-1, rows, int(ints(1, 2 * rows + 1, 1)))):
            for keep in (False,) if parents is None else (False, True):
                a = beam_ref.fork(t, n, parents, refs, page, append=app, keep=keep)
                b = pool_ref.fork(t, n, parents, refs, page, append=app, keep=keep)
                assert a[7] == b[7] and all(torch.equal(x, y) for x, y in zip(a[:7], b)), seed


def test_tables_that_name_pages_of_others_by_hand():
    # row 0 was given back and not cleared: page 4 is free, page 3 is row 1's alone
    t, n = i32([[3, 4], [3, 5]]), i32([8, 6])
    got = pool_ref.fork(t, n, i32([1, 1]), i32([1, 1, 1, 1, 0, 1]), 4)
    # page 4 is handed out by this call and stays held, page 3 is shared and given back once
    assert got[0].tolist() == [[3, 5], [3, 4]] and got[6].tolist() == [1, 1, 1, 1, 1, 1]
    assert got[7] == pool_ref.BAD_PAGE
    # counts end at zero
    got = pool_ref.fork(i32([[3], [3], [3]]), i32([4, 4, 4]), i32([-1]), i32([0, 0, 0, 1]), 4)
    assert got[6].tolist() == [0, 0, 0, 0] and got[7] == pool_ref.BAD_PAGE
