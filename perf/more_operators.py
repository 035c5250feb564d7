"""Cases of beam search next to the verify step: the selection of the next beams over beams and
vocabulary, the reordering of what is kept per beam, and the pages of a paged KV cache that
beams and requests share: forking rows (with the copies of their last, partly filled pages),
giving pages back, and moving the pages in use to the front of the pool.

Layouts are those of the library: logits [B][W][V], block tables [rows][max_pages] of int32 page
ids (-1: none), kv_len [rows].  refs [N] counts the table entries that hold each page; a page of
count 0 is free.  Caches are [layers][N][page_size][heads][dim] (or [layers][N][heads][page_size]
[dim]); only their bytes matter here.  The plain forms are the definitions in elementary torch
operations."""
import math

import torch

own = False

# Vocabularies of the library's workloads (32000, 128256, 151936) and of its tests (50021);
# 16-entry pages and tables of 8192 + 16 entries (513 pages) as its paged workload has them.
_V = (32000, 50021, 128256, 151936)


def listed():
    return [
        # one request, four beams, one step: latency
        dict(name="select_one_f32", op="select", B=1, W=4, V=32000, dtype="f32", k=4, T=1.0,
             finished=0.0, norm=False, dead=0.0),
        # a small batch that ranks by normalised scores and keeps 2 W candidates
        dict(name="select_batch", op="select", B=16, W=4, V=128256, dtype="bf16", k=8, T=1.0,
             finished=0.2, norm=True, dead=0.0),
        # a large batch of eight beams, some of them finished
        dict(name="select_large", op="select", B=64, W=8, V=151936, dtype="bf16", k=16, T=1.0,
             finished=0.1, norm=False, dead=0.0),
        # an odd vocabulary (rows off the 16-byte grid), the step after the first: dead beams
        dict(name="select_odd_f32", op="select", B=5, W=7, V=50021, dtype="f32", k=14, T=0.7,
             finished=0.0, norm=False, dead=0.4),
        # what one batch keeps per beam beside its cache: texts only
        dict(name="reorder_texts", op="reorder", B=4, W=4, L=2047, V=0),
        # texts and the token counts that penalties read
        dict(name="reorder_counts", op="reorder", B=32, W=8, L=8208, V=151936),
        # a prompt forked into eight rows: n-best sampling begins
        dict(name="fork_prompt", op="fork", B=1, W=8, pages=513, prefix=250, own=0, page=16,
             layers=8, heads=8, dim=128, dtype="bf16", heads_first=False, keep=True, append=1,
             slack=64),
        # a step of beam search over a batch: survivors fork, the others' pages are given back
        dict(name="fork_beams", op="fork", B=64, W=8, pages=513, prefix=400, own=20, page=16,
             layers=8, heads=1, dim=128, dtype="bf16", heads_first=False, keep=False, append=1,
             slack=1024),
        # the pages that a round's rollback of 64 rows lists
        dict(name="free_round", op="free", rows=64, pages=4, N=16384, kind="list", share=0.0),
        # a third of a batch's requests end: their whole tables, much of them shared
        dict(name="free_requests", op="free", rows=512, pages=513, N=135168, kind="rows", share=0.5),
        # a small pool of which a part is left in use
        dict(name="compact_small", op="compact", N=2000, rows=16, pages=65, live=0.5, page=16,
             layers=4, heads=2, dim=64, dtype="bf16"),
        # a pool after its peak: half of the pages are free, all over it
        dict(name="compact_pool", op="compact", N=65536, rows=64, pages=513, live=0.5, page=16,
             layers=4, heads=1, dim=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["select", "select", "select", "reorder", "fork", "fork", "free", "compact"])
    if op == "select":
        f32 = rng.random() < 1 / 3
        V = rng.choice(_V + (_log(rng, 500, 151936),))
        W = rng.randint(1, 16)
        B = _log(rng, 1, max(1, min(256, (38_000_000 if f32 else 77_000_000) // (W * V))))
        return dict(op=op, B=B, W=W, V=V, dtype="f32" if f32 else "bf16",
                    k=min(64, rng.choice([W, W, 2 * W, _log(rng, 1, 64)])),
                    T=rng.choice([0.7, 1.0, 1.0, 1.3]), finished=rng.choice([0.0, 0.0, 0.2]),
                    norm=rng.random() < 0.4, dead=rng.choice([0.0, 0.0, 0.3]))
    if op == "reorder":
        W = rng.randint(2, 16)
        V = rng.choice((0, 0) + _V)
        B = _log(rng, 1, max(1, min(128, 39_000_000 // (W * max(V, 2000)))))
        return dict(op=op, B=B, W=W, L=_log(rng, 17, 8208), V=V)
    if op == "fork":
        keep = rng.random() < 0.3
        W = rng.randint(2, 16)
        page = rng.choice([16, 16, 32, 64])
        prefix, mine = _log(rng, 1, 400), 0 if keep else _log(rng, 1, 40)
        B = _log(rng, 1, max(1, min(64, 64 * 560 // (prefix + W * (mine + 3)))))
        return dict(op=op, B=B, W=W, pages=prefix + mine + rng.randint(3, 80), prefix=prefix,
                    own=mine, page=page, layers=rng.randint(1, 8),
                    heads=rng.choice([1, 1, 2]), dim=rng.choice([64, 80, 128]) * 16 // page,
                    dtype=rng.choice(["bf16", "f32", "u8"]), heads_first=rng.random() < 0.4,
                    keep=keep, append=rng.choice([0, 1, 1, 9, 33]), slack=_log(rng, 1, 300))
    if op == "free":
        rows, pages = _log(rng, 1, 512), _log(rng, 1, 513)
        return dict(op=op, rows=rows, pages=pages, N=rows * pages + _log(rng, 1, 4096),
                    kind=rng.choice(["list", "rows"]), share=rng.choice([0.0, 0.5, 0.9]))
    rows, pages = _log(rng, 1, 64), _log(rng, 1, 513)
    N = max(_log(rng, 100, 65536), 2 * rows)
    return dict(op=op, N=N, rows=rows, pages=pages, live=rng.choice([0.1, 0.5, 0.9]),
                page=rng.choice([16, 32]), layers=rng.randint(1, 4), heads=1,
                dim=rng.choice([33, 64]), dtype=rng.choice(["bf16", "u8"]))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _caches(case, N, g):
    """Caches of random bytes (finite values in every type)."""
    p, h, d = case["page"], case["heads"], case["dim"]
    shape = (N, h, p, d) if case.get("heads_first") else (N, p, h, d)
    shape = (case["layers"], *shape)
    if case["dtype"] == "u8":   # eight-bit caches, as the bytes that they are
        return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    return torch.randn(shape, generator=g, device="cuda", dtype=dt)


def _spread(free, n, N, g):
    """n page ids out of N, in no order."""
    return torch.randperm(N, generator=g, device="cuda")[:n].to(torch.int32)


def _prepare_select(case, s, g):
    B, W, V = case["B"], case["W"], case["V"]
    x = torch.randn((B * W, V), generator=g, device="cuda").mul_(3.0)
    ids = torch.randint(0, V, (B * W, 20), generator=g, device="cuda")
    x.scatter_(1, ids, x.gather(1, ids) + 8.0)
    s["logits"] = x.view(B, W, V).to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    # beams of one request lie a few nats apart
    r = torch.rand((4, B, W), generator=g, device="cuda")
    s["scores"] = -40.0 * r[0, :, :1] - 4.0 * r[1]
    dead = r[2] < case["dead"]
    dead[:, 0] = False
    s["scores"] = s["scores"].masked_fill(dead, -math.inf).contiguous()
    s["fin"] = s["len_norm"] = None
    s["eos"] = 2 % V
    if case["finished"]:
        s["fin"] = (r[3] < case["finished"]).to(torch.uint8)
    if case["norm"]:   # ((5 + length) / 6) ^ 0.6; finished beams are of several lengths
        n = torch.randint(20, 60, (B, W), generator=g, device="cuda").float()
        s["len_norm"] = ((5.0 + n) / 6.0) ** 0.6


def _prepare_fork(case, s, g):
    B, W, page = case["B"], case["W"], case["page"]
    rows = B if case["keep"] else B * W
    own_pages = case["own"] + 1           # and the page that is being filled
    # the whole prefix of a group is shared by its rows, the rest is each row's own
    used = B * case["prefix"] + rows * own_pages
    more = B * W * (2 + -(-case["append"] // page))
    N = used + more + case["slack"]
    ids = _spread(None, used, N, g)
    pre = ids[:B * case["prefix"]].view(B, case["prefix"]).repeat_interleave(rows // B, 0)
    mine = ids[B * case["prefix"]:].view(rows, own_pages)
    t = torch.full((rows, case["pages"]), -1, dtype=torch.int32, device="cuda")
    have = case["prefix"] + own_pages
    t[:, :case["prefix"]] = pre
    t[:, case["prefix"]:have] = mine
    # rows of a group are of one length, as beams are; some end with a full page
    n = torch.randint(0, page, (B,), generator=g, device="cuda", dtype=torch.int32)
    n = (have - 1) * page + 1 + n
    s["kv_len"] = n.repeat_interleave(rows // B).contiguous()
    s["refs"] = torch.zeros(N, dtype=torch.int32, device="cuda").scatter_add_(
        0, t[:, :have].reshape(-1).long(), torch.ones(rows * have, dtype=torch.int32, device="cuda"))
    s["table"] = t
    w = rows // B
    s["parents"] = torch.randint(0, w, (B, W), generator=g, device="cuda", dtype=torch.int32)
    s["caches"] = _caches(case, N, g)


def _prepare_free(case, s, g):
    rows, pages, N = case["rows"], case["pages"], case["N"]
    shared = int(pages * case["share"])
    ids = _spread(None, shared + rows * (pages - shared), N, g)
    t = torch.cat([ids[:shared].expand(rows, shared), ids[shared:].view(rows, pages - shared)], 1)
    t = t.contiguous()
    # rows are of several lengths
    n = torch.randint(1, pages + 1, (rows, 1), generator=g, device="cuda")
    t[torch.arange(pages, device="cuda") >= n] = -1
    one = (t >= 0).reshape(-1)
    s["refs"] = torch.zeros(N, dtype=torch.int32, device="cuda").scatter_add_(
        0, t.reshape(-1).clamp(min=0).long(), one.to(torch.int32))
    s["table"] = t
    s["which"] = s["n_list"] = None
    if case["kind"] == "rows":
        s["which"] = (torch.rand(rows, generator=g, device="cuda") < 1 / 3).to(torch.uint8)
        s["which"][0] = 1
    else:              # a list of ids, then a tail that is not part of it, as a rollback writes it
        flat = t.reshape(-1)
        order = torch.argsort((flat < 0).to(torch.int8), stable=True)
        s["table"] = flat[order].contiguous()
        s["n_list"] = one.sum().to(torch.int32).view(1)


def _prepare_compact(case, s, g):
    rows, pages, N = case["rows"], case["pages"], case["N"]
    n_live = max(1, int(N * case["live"]))
    ids = _spread(None, n_live, N, g)
    at = torch.randint(0, n_live, (rows, pages), generator=g, device="cuda")
    t = ids[at]
    n = torch.randint(1, pages + 1, (rows, 1), generator=g, device="cuda")
    t[torch.arange(pages, device="cuda") >= n] = -1
    # pages that no row of this table holds belong to a cache of prefixes
    s["refs"] = torch.zeros(N, dtype=torch.int32, device="cuda")
    s["refs"][ids.long()] = 1
    s["refs"].scatter_add_(0, t.reshape(-1).clamp(min=0).long(),
                           (t >= 0).reshape(-1).to(torch.int32))
    s["table"] = t.contiguous()
    s["caches"] = _caches(case, N, g)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "select":
        _prepare_select(case, s, g)
    elif case["op"] == "reorder":
        B, W = case["B"], case["W"]
        s["states"] = [torch.randint(0, 151936, (B, W, case["L"]), generator=g, device="cuda",
                                     dtype=torch.int32)]
        if case["V"]:
            s["states"].append(torch.randint(-32768, 32768, (B, W, case["V"]), generator=g,
                                             device="cuda", dtype=torch.int16))
        s["parents"] = torch.randint(0, W, (B, W), generator=g, device="cuda", dtype=torch.int32)
    elif case["op"] == "fork":
        _prepare_fork(case, s, g)
    elif case["op"] == "free":
        _prepare_free(case, s, g)
    else:
        _prepare_compact(case, s, g)
    return s


# ---------------------------------------------------------------- plain forms --
def _plain_select(s):
    x = s["logits"].float()
    B, W, V = x.shape
    k, T = s["k"], s["T"]
    kr = min(k, V)
    live = torch.isfinite(s["scores"])
    fin = torch.zeros_like(live) if s["fin"] is None else s["fin"] > 0
    # the best of each row: one integer key per place, larger value first, then the lower index
    u = (x + 0.0).view(torch.int32)
    u = torch.where(u < 0, u ^ 0x7FFFFFFF, u).long()
    key = u * (1 << 32) + (V - 1 - torch.arange(V, device="cuda"))
    ids = (V - 1) - (key.topk(kr, dim=2).values & 0xFFFFFFFF)
    del u, key
    vals = x.gather(2, ids)
    # candidates of different beams may lie next to one another: their scores in 64 bits
    m = vals[:, :, :1]
    lse = m.double() / T + torch.log(torch.exp((x - m) / T).sum(2, keepdim=True,
                                                                dtype=torch.float64))
    c = s["scores"].double()[:, :, None] + vals.double() / T - lse
    c = c.masked_fill(~(live & ~fin)[:, :, None], -math.inf)
    first = (torch.arange(kr, device="cuda") == 0)
    c = torch.where((live & fin)[:, :, None] & first, s["scores"].double()[:, :, None], c)
    ids = torch.where(fin[:, :, None], torch.full_like(ids, s["eos"]), ids)
    rank = c if s["len_norm"] is None else c / s["len_norm"].double()[:, :, None]
    # in the order of beams and tokens, so that a stable sort leaves ties with the lowest index
    order = torch.argsort(rank.view(B, W * kr), dim=1, descending=True, stable=True)
    if W * kr < k:
        order = torch.nn.functional.pad(order, (0, k - W * kr))
    order = order[:, :k]
    none = torch.arange(k, device="cuda") >= W * kr
    score = c.view(B, -1).gather(1, order)
    none = none | (score == -math.inf)
    parents = torch.where(none, -1, order // kr).to(torch.int32)
    tokens = torch.where(none, -1, ids.view(B, -1).gather(1, order)).to(torch.int32)
    ended = fin.gather(1, parents.clamp(min=0).long()) | (tokens == s["eos"])
    return (score.masked_fill(none, -math.inf).float(), parents, tokens,
            (ended & ~none).to(torch.uint8))


def _plain_copy(caches, src, dst, fill, heads_first):
    """The first `fill` entries of each page (all of them without it)."""
    if src.numel() == 0:
        return
    a = caches[:, src.long()]
    if fill is not None:
        shape = (1, -1, 1, caches.shape[3], 1) if heads_first else (1, -1, caches.shape[2], 1, 1)
        entry = torch.arange(shape[3] if heads_first else shape[2], device="cuda")
        use = (entry < fill[:, None]).view([d if d > 0 else src.numel() for d in shape])
        a = torch.where(use, a, caches[:, dst.long()])
    caches[:, dst.long()] = a


def _plain_fork(s):
    refs = s["refs"].clone()
    table, page, append = s["table"], s["page"], s["append"]
    rows, M = table.shape
    B, W = s["parents"].shape
    R = B * W
    p = (s["parents"].long() + torch.arange(B, device="cuda")[:, None] * (rows // B)).view(-1)
    r = torch.arange(R, device="cuda")
    col = torch.arange(M, device="cuda")
    first = torch.full((rows,), R, device="cuda").scatter_reduce_(0, p, r, "amin")
    heir = (first[p] == r) & (not s["keep"])
    n = s["kv_len"][p]
    full, part = n // page, n % page
    used, need = (n + page - 1) // page, (n + append + page - 1) // page
    old = table[p]
    last = old.gather(1, full.clamp(max=M - 1).long()[:, None])[:, 0]
    copy = (part > 0) & ~(heir & (refs[last.clamp(min=0).long()] == 1))
    # entries that need a page, in the order of rows and places
    want = (col >= used[:, None]) & (col < need[:, None]) & ~(heir[:, None] & (old >= 0))
    want |= copy[:, None] & (col == full[:, None])
    order = torch.argsort((refs != 0).to(torch.int8), stable=True).to(torch.int32)
    rank = torch.cumsum(want.view(-1), 0).view(R, M) - 1
    kept = (col < full[:, None]) | heir[:, None] | ((col == full[:, None]) & (part > 0)[:, None])
    out = torch.where(kept, old, -1)
    out = torch.where(want, order[rank.clamp(min=0)], out)
    # counts: what the new rows hold, less what the old ones held
    flat = out.view(-1)
    refs.scatter_add_(0, flat.clamp(min=0).long(), (flat >= 0).to(torch.int32))
    if not s["keep"]:
        flat = table.view(-1)
        refs.scatter_add_(0, flat.clamp(min=0).long(), -(flat >= 0).to(torch.int32))
    at = torch.argsort((~copy).to(torch.int8), stable=True)
    got = out.gather(1, full.clamp(max=M - 1).long()[:, None])[:, 0]
    some = copy[at]
    src = torch.where(some, last[at], -1)
    dst = torch.where(some, got[at], -1)
    fill = torch.where(some, part[at], 0)
    count = copy.sum().to(torch.int32).view(1)
    c = int(count)
    _plain_copy(s["caches"], src[:c], dst[:c], fill[:c], s["heads_first"])
    return out, n, src, dst, fill, count, refs, s["caches"]


def _plain_free(s):
    refs, t = s["refs"].clone(), s["table"].clone()
    if s["which"] is not None:
        gone = (t >= 0) & (s["which"] > 0)[:, None]
    else:
        gone = (t >= 0) & (torch.arange(t.numel(), device="cuda") < s["n_list"])
    refs.scatter_add_(0, t.view(-1).clamp(min=0).long(), -gone.view(-1).to(torch.int32))
    refs.clamp_(min=0)
    if s["which"] is not None:   # rows that end hold nothing afterwards
        t = torch.where((s["which"] > 0)[:, None], -1, t)
    return refs, t


def _plain_compact(s):
    refs, t = s["refs"].clone(), s["table"]
    N = refs.numel()
    page = torch.arange(N, device="cuda")
    used = refs > 0
    live = used.sum()
    move, hole = used & (page >= live), ~used & (page < live)
    src = torch.argsort((~move).to(torch.int8), stable=True)[:N // 2]
    dst = torch.argsort((~hole).to(torch.int8), stable=True)[:N // 2]
    count = move.sum()
    some = torch.arange(N // 2, device="cuda") < count
    to = torch.where(used, page, -1)
    c = int(count)
    to[src[:c]] = dst[:c]
    refs[dst[:c]] = refs[src[:c]]
    refs[src[:c]] = 0
    t = torch.where(t >= 0, to[t.clamp(min=0).long()].to(torch.int32), t)
    src = torch.where(some, src, -1).to(torch.int32)
    dst = torch.where(some, dst, -1).to(torch.int32)
    _plain_copy(s["caches"], src[:c], dst[:c], None, False)
    return (src, dst, count.to(torch.int32).view(1), to.to(torch.int32),
            live.to(torch.int32).view(1), refs, t, s["caches"])


def run(state):
    s = state
    op = s["op"]
    if not own:
        if op == "select":
            return _plain_select(s)
        if op == "reorder":
            at = s["parents"].long()
            return [x.gather(1, at[:, :, None].expand_as(x)) for x in s["states"]]
        if op == "fork":
            return _plain_fork(s)
        return _plain_free(s) if op == "free" else _plain_compact(s)
    import speculative_decoding_verification_logits_gb300 as sd
    if op == "select":
        b = sd.beam_select(s["logits"], s["scores"], s["k"], temperature=s["T"],
                           finished=s["fin"], eos=s["eos"], norm=s["len_norm"])
        return b.scores, b.parents, b.tokens, b.finished
    if op == "reorder":
        return sd.beam_reorder(s["states"], s["parents"])
    refs = s["refs"].clone()   # the calls change the counts where they are
    if op == "fork":
        f = sd.kv_fork(s["table"], s["kv_len"], s["parents"], refs, s["page"],
                       append=s["append"], keep=s["keep"])
        sd.kv_copy(s["caches"], f.src, f.dst, count=f.count, fill=f.fill,
                   heads_first=s["heads_first"])
        return f.block_table, f.kv_len, f.src, f.dst, f.fill, f.count, refs, s["caches"]
    t = s["table"].clone()
    if op == "free":
        sd.kv_free(t, refs, which=s["which"], count=s["n_list"], clear=s["which"] is not None)
        return refs, t
    c = sd.kv_compact(refs, t)
    sd.kv_copy(s["caches"], c.src, c.dst, count=c.count)
    return c.src, c.dst, c.count, c.new_ids, c.live, refs, t, s["caches"]


def work(case):
    op = case["op"]
    if op == "select":
        B, W, V, k = case["B"], case["W"], case["V"], case["k"]
        es = 2 if case["dtype"] == "bf16" else 4
        read = 1.0 - case["finished"] * (1 - case["dead"] * (W - 1) / W)   # rows that count
        read -= case["dead"] * (W - 1) / W
        return {"bytes": int(B * W * V * es * read) + B * W * 9 + B * k * 13,
                "flops": int(4 * B * W * V * read)}
    if op == "reorder":
        B, W = case["B"], case["W"]
        row = 4 * case["L"] + 2 * case["V"]
        # rows that some beam goes on from are read, all are written
        read = W * (1.0 - (1.0 - 1.0 / W) ** W)
        return {"bytes": int(B * row * (read + W)) + 4 * B * W, "flops": B * W}
    es = {"bf16": 2, "f32": 4, "u8": 1}.get(case.get("dtype"), 0)
    if op == "fork":
        B, W, M = case["B"], case["W"], case["pages"]
        rows = B if case["keep"] else B * W
        page = case["page"] * case["heads"] * case["dim"] * es * case["layers"]
        # parents that some row goes on from; on average half of a page is filled
        taken = 1 if case["keep"] else W * (1.0 - (1.0 - 1.0 / W) ** W)
        copies = B * (W - (0 if case["keep"] else taken)) * (1.0 - 1.0 / case["page"])
        return {"bytes": int(copies * page) + 4 * (rows * M + B * W * M) + B * W * 24,
                "flops": B * W * M}
    if op == "free":
        n = case["rows"] * case["pages"]
        part = 0.5 if case["kind"] == "list" else 1 / 6
        return {"bytes": int(n * part * 12), "flops": n}
    N, live = case["N"], case["live"]
    moved = N * live * (1.0 - live)
    page = case["page"] * case["heads"] * case["dim"] * es * case["layers"]
    return {"bytes": int(2 * moved * page) + 16 * N + 8 * case["rows"] * case["pages"],
            "flops": N}


# ------------------------------------------------- the definitions, in 64 bits --
def exact(case, seed):
    if case["op"] != "select":
        return None   # whole numbers and copies: the plain form has them exactly
    s = prepare(case, seed)
    B, W, V = s["logits"].shape
    k, eos = case["k"], s["eos"]
    scores = torch.full((B, k), -math.inf, dtype=torch.float64)
    parents = torch.full((B, k), -1, dtype=torch.int32)
    tokens, ended = parents.clone(), torch.zeros((B, k), dtype=torch.uint8)
    for b in range(B):
        found = []
        for w in range(W):
            s0 = float(s["scores"][b, w])
            norm = 1.0 if s["len_norm"] is None else float(s["len_norm"][b, w])
            if s0 == -math.inf:
                continue
            if s["fin"] is not None and int(s["fin"][b, w]):
                found.append((-s0 / norm, w, eos, s0, 1))
                continue
            lp = torch.log_softmax(s["logits"][b, w].to(torch.float64) / case["T"], 0) + s0
            y, i = torch.sort(lp, descending=True, stable=True)
            found += [(-c / norm, w, v, c, int(v == eos))
                      for c, v in zip(y[:k].tolist(), i[:k].tolist())]
        for j, (_, w, v, c, e) in enumerate(sorted(found)[:k]):
            scores[b, j], parents[b, j], tokens[b, j], ended[b, j] = c, w, v, e
    out = scores, parents, tokens, ended
    return tuple(t.to(s["logits"].device) for t in out)
