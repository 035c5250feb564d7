"""Beam search's step and the pages of a shared cache from their definitions, in 64 bits or whole
numbers on the CPU (plain torch and Python): what the CUDA kernels are tested against, and
how far scores may be off.  U = 2^-24 is fp32's half step."""
import math

import torch

D = torch.float64
U = 2.0 ** -24

NONFINITE, BAD_PENALTY, BAD_PARENT, BAD_PAGE, NO_PAGE = 0x4, 0x8, 0x10, 0x20, 0x40


# ------------------------------------------------------------------- select --
def select(x, scores, k, T=1.0, finished=None, eos=-1, norm=None):
    """Per sequence the ranked candidates (rank, beam, token, score, ended), every beam's k + 1 best,
    with how far the device's score may be off; and the status."""
    B, W, V = x.shape
    T = torch.tensor(T, dtype=torch.float32).item()   # an fp32 argument of the call
    out, tol, status = [], [], 0
    for b in range(B):
        found, off = [], 0.0
        for w in range(W):
            s = float(scores[b, w])
            n = 1.0 if norm is None else float(norm[b, w])
            if s == -math.inf:
                continue
            if not math.isfinite(s):
                status |= NONFINITE
                continue
            if not (n > 0 and math.isfinite(n)):
                status |= BAD_PENALTY
                continue
            if finished is not None and int(finished[b, w]):
                found.append((s / n, w, eos, s, 1))
                continue
            row = x[b, w].to(D) / T
            if torch.isnan(row).any() or (row == math.inf).any():
                status |= NONFINITE
                continue
            if (row == -math.inf).all():
                continue
            m = row.max()
            q = torch.softmax(row, 0)
            far = (m - row).masked_fill(row == -math.inf, 0.0)
            # terms: 2^-22 of the device's power and 4 U of the exponent's rounding for each unit
            # of it, twice (within a piece of the row and between pieces); at most 45 fp32
            # additions above one another; at most 1024 pieces in whole units of 2^-31
            off = max(off, (4 + 4 + 45 + 4) * U + 4 * U * float((q * far).sum()))
            lp = s + torch.log_softmax(row, 0)
            y, i = torch.sort(lp, descending=True, stable=True)
            keep = min(V, k + 1)
            found += [(c / n, w, v, c, int(v == eos))
                      for c, v in zip(y[:keep].tolist(), i[:keep].tolist()) if c > -math.inf]
        found.sort(key=lambda f: (-f[0], f[1], f[2]))
        out.append(found)
        tol.append(off)
    return out, tol, status


def check_select(beams, want, k, norm=None):
    """Holds the device's beams to the ranked candidates: nothing that was left out lies further
    above what was taken than the two may be off, the order is theirs but for candidates as close
    as that, and a beam's own candidates come in the order of their logits, then tokens."""
    found, tol, _ = want
    for b, cand in enumerate(found):
        n = min(k, len(cand))
        scores, parents, tokens, ended = (t[b].tolist() for t in beams)
        assert all(g == (-math.inf, -1, -1, 0)
                   for g in zip(scores[n:], parents[n:], tokens[n:], ended[n:]))
        at = {(w, v): i for i, (_, w, v, _, _) in enumerate(cand)}
        over = lambda w: tol[b] / (1.0 if norm is None else float(norm[b, w]))
        near = lambda p, q: over(p[1]) + over(q[1]) + abs(p[0]) * 2.0 ** -50
        places = [at.get((w, v)) for w, v in zip(parents[:n], tokens[:n])]
        assert None not in places and len(set(places)) == n, (b, places)
        for p, q in zip(places, places[1:]):
            assert cand[p][0] >= cand[q][0] - near(cand[p], cand[q]), (b, cand[p], cand[q])
        for w in set(parents[:n]):
            own = [p for p in places if cand[p][1] == w]
            assert own == sorted(own), (b, w, own)
        for i in sorted(set(range(n)) - set(places)):   # left out: as good as what came instead
            worst = cand[max(places)]
            assert cand[i][0] <= worst[0] + near(cand[i], worst), (b, cand[i], worst)
        for score, p, e in zip(scores, places, ended):
            c = cand[p][3]
            assert e == cand[p][4]
            f = torch.tensor(c, dtype=D).to(torch.float32).item()
            if math.isinf(f):
                assert score == f
            else:
                assert abs(score - c) <= tol[b] + U * abs(c) + U * tol[b], (b, score, cand[p])


# ------------------------------------------------------------------ reorder --
def reorder(x, parents):
    B, k = parents.shape
    W = x.shape[1]
    y = torch.zeros((B, k, *x.shape[2:]), dtype=x.dtype)
    status = 0
    for b in range(B):
        for i in range(k):
            p = int(parents[b, i])
            if not 0 <= p < W:
                status |= BAD_PARENT if p != -1 else 0
                p = i
            if p < W:
                y[b, i] = x[b, p]
    return y, status


# -------------------------------------------------------------------- pages --
class Pool:
    """refs with the calls' checks."""

    def __init__(self, refs):
        self.refs = [int(v) for v in refs]
        self.N = len(self.refs)
        self.status = 0

    def ok(self, p):
        return 0 <= p < self.N

    def give_back(self, p):
        if not self.ok(p):
            self.status |= BAD_PAGE
        elif self.refs[p] <= 0:
            self.status |= BAD_PAGE
        else:
            self.refs[p] -= 1


def fork(table, kv_len, parents, refs, page, append=0, keep=False, groups=0):
    """(table, len, src, dst, fill, count, refs, status) of kv_fork; parents None: kv_extend."""
    rows, M = table.shape
    T = table.tolist()
    before = [int(v) for v in refs]
    P = Pool(refs)
    R = rows if parents is None else parents.numel()
    flat = list(range(R)) if parents is None else parents.reshape(-1).tolist()
    who = []
    for r, p in enumerate(flat):
        per = rows // groups if groups else rows
        if not 0 <= p < per:
            P.status |= BAD_PARENT if p != -1 else 0
            who.append(-1)
        else:
            who.append(p + (r // (R // groups) * per if groups else 0))
    free = iter([p for p in range(P.N) if before[p] == 0])
    out, lens, pairs, held = [], [], [], []

    def take():
        p = next(free, None)
        if p is None:
            P.status |= NO_PAGE
            return -1
        held.append(p)
        return p

    heirs = set()
    for r, p in enumerate(who):
        if p < 0:
            out.append([-1] * M)
            lens.append(0)
            continue
        heir = not keep and p not in heirs
        if heir:
            heirs.add(p)
        old = T[p]
        n = min(max(int(kv_len[p]), 0), M * page)
        full, part = divmod(n, page)
        used = full + (part > 0)
        need = -(-(n + append) // page)
        if need > M:
            P.status |= NO_PAGE
            need = M
        row = [-1] * M
        for j in range(M):
            e = old[j]
            if j < full:
                row[j] = e
                if not P.ok(e):
                    P.status |= BAD_PAGE
                elif not heir:
                    held.append(e)
            elif j < used:
                row[j] = e
                if not P.ok(e):
                    P.status |= BAD_PAGE
                elif not (heir and before[e] == 1):
                    if heir:
                        held.append(("back", e))
                    row[j] = take()
                    pairs.append((e, row[j], part) if row[j] >= 0 else (-1, -1, part))
            elif j < need:
                if heir and P.ok(e):
                    row[j] = e
                else:
                    if heir and e != -1:
                        P.status |= BAD_PAGE
                    row[j] = take()
            elif heir:
                row[j] = e
        out.append(row)
        lens.append(n)
    for h in held:
        if not isinstance(h, tuple):
            P.refs[h] += 1
    for h in held:
        if isinstance(h, tuple):
            P.give_back(h[1])
    if not keep:
        for p in range(rows):
            if p not in heirs:
                for e in T[p]:
                    if e != -1:
                        P.give_back(e)
    pad = R - len(pairs)
    i = lambda v: torch.tensor(v, dtype=torch.int32)
    src, dst, fill = (i([q[c] for q in pairs] + [d] * pad) for c, d in ((0, -1), (1, -1), (2, 0)))
    return (i(out).reshape(R, M), i(lens), src, dst, fill, i([len(pairs)]), i(P.refs), P.status)


def free(pages, refs, which=None, count=None, clear=False):
    P = Pool(refs)
    flat = pages.reshape(-1).tolist()
    cols = pages.shape[-1]
    for i, e in enumerate(flat):
        if e == -1 or (which is not None and not int(which[i // cols])):
            continue
        if count is not None and i >= int(count):
            continue
        P.give_back(e)
        if clear:
            flat[i] = -1
    return (torch.tensor(P.refs, dtype=torch.int32),
            torch.tensor(flat, dtype=torch.int32).reshape(pages.shape), P.status)


def compact(refs, table=None):
    N = refs.numel()
    r = refs.tolist()
    used = [p for p in range(N) if r[p] > 0]
    L = len(used)
    src = [p for p in used if p >= L]
    dst = [p for p in range(L) if r[p] <= 0]
    new = [-1] * N
    for p in used:
        new[p] = p
    for s, d in zip(src, dst):
        new[s], r[d], r[s] = d, r[s], 0
    status, t = 0, None
    if table is not None:
        t = table.clone().reshape(-1)
        for i, e in enumerate(t.tolist()):
            if e == -1:
                continue
            if not 0 <= e < N or new[e] < 0:
                status |= BAD_PAGE
            else:
                t[i] = new[e]
        t = t.reshape(table.shape)
    pad = N // 2 - len(src)
    i = lambda v: torch.tensor(v, dtype=torch.int32)
    return i(src + [-1] * pad), i(dst + [-1] * pad), i([len(src)]), i(new), i([L]), i(r), t, status


def copy(cache, src, dst, count=None, fill=None, heads_first=False):
    """cache [layers][N][...]: a copy of it with the pairs' pages copied; and the status."""
    y = cache.clone()
    N, status = cache.shape[1], 0
    for i in range(src.numel() if count is None else min(max(int(count), 0), src.numel())):
        s, d = int(src[i]), int(dst[i])
        if s == -1 and d == -1:
            continue
        if not (0 <= s < N and 0 <= d < N):
            status |= BAD_PAGE
            continue
        at = 3 if heads_first else 2
        n = cache.shape[at] if fill is None else min(max(int(fill[i]), 0), cache.shape[at])
        if fill is None:
            y[:, d] = cache[:, s]
        elif heads_first:
            y[:, d, :, :n] = cache[:, s, :, :n]
        else:
            y[:, d, :n] = cache[:, s, :n]
    return y, status
