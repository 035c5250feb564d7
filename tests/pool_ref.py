"""Forks and extensions of block tables from their definition, in plain Python: also of pools that run
out, where a row that goes on keeps a shared last page that it cannot copy, and of tables that name
pages which they do not hold: what is added to the counts comes first, then what is given back."""
import torch

BAD_PAGE, NO_PAGE = 0x20, 0x40


def fork(table, kv_len, parents, refs, page, append=0, keep=False):
    """(table, len, src, dst, fill, count, refs, status) of kv_fork for parents [R] within the rows
    or -1; parents None: kv_extend."""
    T, M, N = table.tolist(), table.shape[1], refs.numel()
    parents = list(range(len(T))) if parents is None else parents.tolist()
    before, more, less, status = refs.tolist(), [0] * N, [0] * N, 0
    free = iter([p for p in range(N) if before[p] == 0])
    heirs, out, lens, pairs = {}, [], [], []
    for r, p in enumerate(parents):
        row, n = [-1] * M, 0
        heir = p >= 0 and not keep and heirs.setdefault(p, r) == r
        if p >= 0:
            n = min(max(int(kv_len[p]), 0), M * page)
            need = -(-(n + append) // page)
            status |= NO_PAGE if need > M else 0
        for j in range(M if p >= 0 else 0):
            old, has = T[p][j], 0 <= T[p][j] < N
            held = min(max(n - j * page, 0), page)      # entries of the slot
            status |= BAD_PAGE if held and not has else 0
            copy = 0 < held < page and has and not (heir and before[old] == 1)
            if copy or not held and j < need and not (heir and has):
                status |= BAD_PAGE if not held and heir and old != -1 else 0
                row[j] = next(free, -1)
                got = row[j] >= 0
                status |= 0 if got else NO_PAGE
                if copy:
                    pairs.append((old, row[j], held) if got else (-1, -1, held))
                    if heir and got:
                        less[old] += before[old] != 0
                        status |= 0 if before[old] else BAD_PAGE
                    elif heir:
                        row[j] = old
                if got:
                    more[row[j]] += 1
            elif held or heir:
                row[j] = old
                more[old if has else 0] += 1 if has and held and not heir else 0
        out.append(row)
        lens.append(n)
    for p in range(len(T)):
        if not keep and p not in heirs:
            for e in T[p]:
                if 0 <= e < N and before[e]:
                    less[e] += 1
                elif e != -1:   # none, or one that was free before the call
                    status |= BAD_PAGE
    after = [before[p] + more[p] - less[p] for p in range(N)]
    status |= BAD_PAGE if min(after) < 0 else 0
    i = lambda v: torch.tensor(v, dtype=torch.int32)
    R = len(parents)
    pad = [(-1, -1, 0)] * (R - len(pairs))
    src, dst, fill = i(pairs + pad).view(R, 3).unbind(1)
    return (i(out).view(R, M), i(lens), src, dst, fill, i([len(pairs)]),
            i([max(v, 0) for v in after]), status)
