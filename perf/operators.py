"""Cases of the logit operators around the verify step: what a serving loop does to the
target's and the drafter's logits before it verifies a round (token counts, penalties, biases,
grammar masks), and what a training loop takes from the target's logits to train the drafter
on (the top logits of each row, the distillation loss over them and its gradient).

Layouts are those of the library: logits [B][R][V] or [N][V], histories [B][L] with lengths,
int32 token ids.  The plain forms are the formulas in elementary torch operations, in fp32."""
import math

import torch

own = False

# Vocabularies of the library's workloads (32000, 128256, 151936) and of its tests (an odd
# one, 50021); batches, drafts per round and history lengths of the same workloads.
_V = (32000, 50021, 128256, 151936)


def listed():
    return [
        # one chat stream, one token at a time, every penalty and a bias list: latency
        dict(name="process_one_token_f32", op="process", B=1, R=1, V=32000, dtype="f32", base=0,
             P=0, bias=32, mask="none"),
        # a verify round's target rows under penalties and a per-position grammar mask
        dict(name="process_round_masked", op="process", B=64, R=9, V=151936, dtype="bf16", base=0,
             P=8, bias=16, mask="half"),
        # an odd vocabulary (rows off the 16-byte grid), a grammar that allows few tokens
        dict(name="process_grammar_odd", op="process", B=13, R=7, V=50021, dtype="bf16", base=0,
             P=6, bias=300, mask="tight"),
        # a large batch of short rounds, penalties only
        dict(name="process_large_batch", op="process", B=256, R=5, V=128256, dtype="bf16", base=0,
             P=4, bias=0, mask="none"),
        # counts of a whole batch joining with its histories
        dict(name="counts_batch", op="counts", B=256, L=16384, V=128256),
        # a few long contexts
        dict(name="counts_long", op="counts", B=3, L=131071, V=151936),
        # the teacher's rows of one sequence's round: latency
        dict(name="top_one_round", op="top", N=7, V=128256, dtype="bf16", k=32, T=1.0),
        # a batch's rounds
        dict(name="top_batch", op="top", N=576, V=151936, dtype="bf16", k=64, T=2.0),
        # fp32 rows of an odd vocabulary, many tokens kept
        dict(name="top_odd_f32", op="top", N=33, V=50021, dtype="f32", k=128, T=1.0),
        # evaluating a drafter: the loss alone
        dict(name="distill_loss_eval", op="loss", N=576, V=151936, dtype="bf16", k=64, T=1.0,
             rest=True),
        # an online step on a few rounds' rows, fp32 logits, the top tokens renormalised
        dict(name="distill_grad_small_f32", op="grad", N=48, V=32000, dtype="f32", k=16, T=2.0,
             rest=False),
        # a training step's rows
        dict(name="distill_grad_train", op="grad", N=2048, V=128256, dtype="bf16", k=64, T=1.0,
             rest=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["process", "process", "counts", "top", "loss", "grad"])
    V = rng.choice(_V + (_log(rng, 1000, 151936),))
    if op == "process":
        R = rng.randint(1, 16)
        B = _log(rng, 1, max(1, min(256, 164_000_000 // (R * V))))
        base = rng.randint(0, 4)
        return dict(op=op, B=B, R=R, V=V, dtype=rng.choice(["bf16", "bf16", "f32"]), base=base,
                    P=min(32, base + R - 1), bias=rng.choice([0, 1, 17, 300]),
                    mask=rng.choice(["none", "half", "tight"]))
    if op == "counts":
        B = _log(rng, 1, max(1, min(256, 32_000_000 // V)))
        return dict(op=op, B=B, L=_log(rng, 17, min(131071, 4_000_000 // B)), V=V)
    f32 = rng.random() < 1 / 3
    most = {"top": 87_000_000, "loss": 87_000_000, "grad": 262_000_000}[op] // (2 if f32 else 1)
    case = dict(op=op, N=_log(rng, 1, max(1, min(4096, most // V))), V=V,
                dtype="f32" if f32 else "bf16", k=_log(rng, 1, 128),
                T=rng.choice([0.7, 1.0, 2.0, 4.0]))
    if op != "top":
        case["rest"] = rng.random() < 0.7
    return case


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _tokens(shape, V, g):
    """Token ids as text has them: a few of them very often."""
    u = torch.rand(shape, generator=g, device="cuda")
    return (torch.exp(u * math.log(V)) - 1).to(torch.int32).clamp_(0, V - 1)


def _rows(n, V, g):
    """Logits of n rows: N(0, 3^2), 20 places of each raised by 8."""
    x = torch.randn((n, V), generator=g, device="cuda").mul_(3.0)
    ids = torch.randint(0, V, (n, 20), generator=g, device="cuda")
    x.scatter_(1, ids, x.gather(1, ids) + 8.0)
    return x


def _pack(bits):
    """bool [..., V] -> int32 words [..., ceil(V / 32)], bit v % 32 of word v / 32."""
    V = bits.shape[-1]
    W = (V + 31) // 32
    bits = torch.nn.functional.pad(bits, (0, W * 32 - V)).view(*bits.shape[:-1], W, 32)
    w = (bits.to(torch.int64) << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    V = case["V"]
    if op == "counts":
        B, L = case["B"], case["L"]
        s["history"] = _tokens((B, L), V, g)
        s["lengths"] = torch.randint(L // 2, L + 1, (B,), generator=g, device="cuda",
                                     dtype=torch.int32)
        s["prompt_lengths"] = s["lengths"] // 2
        return s
    if op == "process":
        B, R, P = case["B"], case["R"], case["P"]
        s["logits"] = _rows(B * R, V, g).view(B, R, V).to(_dt(case))
        hist = _tokens((B, 600), V, g).long()
        c = torch.zeros((B, V), dtype=torch.int32, device="cuda")
        c.scatter_add_(1, hist, torch.ones_like(hist, dtype=torch.int32))
        c.scatter_(1, _tokens((B, 2000), V, g).long(), 0x8000, reduce="add")
        # the prompt's tokens carry bit 15, however often they occur
        c = (c & 0x7FFF) | torch.where(c >= 0x8000, 0x8000, 0)
        s["counts"] = torch.where(c >= 0x8000, c - 0x10000, c).to(torch.int16)
        s["prev"] = _tokens((B, P), V, g)
        r = torch.rand((3, B), generator=g, device="cuda")
        s["repetition"] = 1.0 + 0.5 * r[0]
        s["presence"] = r[1].clone()
        s["frequency"] = 0.5 * r[2]
        s["bias_ids"] = s["bias_vals"] = s["bits"] = None
        if case["bias"]:
            ids = torch.rand((B, V), generator=g, device="cuda").argsort(1)[:, :case["bias"]]
            s["bias_ids"] = ids.to(torch.int32).contiguous()
            s["bias_vals"] = torch.randn(ids.shape, generator=g, device="cuda") * 5.0
        if case["mask"] != "none":
            keep = 0.5 if case["mask"] == "half" else 50.0 / V
            bits = torch.rand((B, R, V), generator=g, device="cuda") < keep
            bits[..., V // 2] = True
            s["bits"] = _pack(bits)
        return s
    teacher = _rows(case["N"], V, g)
    if op == "top":
        s["logits"] = teacher.to(_dt(case))
        return s
    noise = torch.randn((case["N"], V), generator=g, device="cuda")
    s["student"] = (teacher + noise).to(_dt(case))
    del noise
    vals, ids = teacher.topk(case["k"], dim=1)
    s["vals"], s["ids"] = vals, ids.to(torch.int32)
    s["rest_mass"] = None
    if case["rest"]:
        s["rest_mass"] = torch.logsumexp(
            teacher.scatter_(1, ids, -math.inf).div_(case["T"]), dim=1)
    s["weight"] = torch.randint(1, 4, (case["N"],), generator=g, device="cuda").float() / case["N"]
    return s


# ---------------------------------------------------------------- plain forms --
def _plain_counts(s):
    B, L = s["history"].shape
    at = torch.arange(L, device="cuda")
    h = s["history"].long()
    out = (at >= s["prompt_lengths"][:, None]) & (at < s["lengths"][:, None])
    pro = at < s["prompt_lengths"][:, None]
    c = torch.zeros((B, s["V"]), dtype=torch.int32, device="cuda")
    p = torch.zeros_like(c)
    c.scatter_add_(1, h, out.to(torch.int32))
    p.scatter_add_(1, h, pro.to(torch.int32))
    return torch.where(p > 0, c.clamp(max=32767) - 32768, c.clamp(max=32767)).to(torch.int16)


def _plain_process(s):
    x0 = s["logits"]
    B, R, V = x0.shape
    x = x0.float()
    w = s["counts"].to(torch.int32) & 0xFFFF
    c = (w & 0x7FFF).float()[:, None, :].expand(B, R, V)
    P = s["P"]
    if P:
        i = torch.arange(P, device="cuda")
        r = torch.arange(R, device="cuda")
        before = (i[None, :] < s["base"] + r[:, None]).float()
        c = c.contiguous().scatter_add_(2, s["prev"].long()[:, None, :].expand(B, R, P),
                                        before[None].expand(B, R, P))
    some = c > 0
    seen = some | ((w >> 15) > 0)[:, None, :]
    th = s["repetition"][:, None, None]
    x = torch.where(seen, torch.where(x > 0, x / th, x * th), x)
    x = x - s["frequency"][:, None, None] * c - s["presence"][:, None, None] * some.float()
    if s["bias_ids"] is not None:
        b = torch.zeros((B, V), device="cuda").scatter_add_(1, s["bias_ids"].long(),
                                                            s["bias_vals"])
        x = x + b[:, None, :]
    if s["bits"] is not None:
        v = torch.arange(V, device="cuda")
        ok = ((s["bits"][..., v // 32] >> (v % 32)) & 1) > 0
        x = torch.where(ok, x, torch.full_like(x, -math.inf))
    return x.to(x0.dtype)


def _plain_top(s):
    x = s["logits"].float()
    N, V = x.shape
    # one integer key per place: larger value first, then the lower index
    u = (x + 0.0).view(torch.int32)
    u = torch.where(u < 0, u ^ 0x7FFFFFFF, u).long()
    key = u * (1 << 32) + (V - 1 - torch.arange(V, device="cuda"))
    ids = (V - 1) - (key.topk(s["k"], dim=1).values & 0xFFFFFFFF)
    vals = x.gather(1, ids)
    m = vals[:, :1]
    e = torch.exp((x - m) / s["T"]).scatter(1, ids, 0.0)
    rest = m[:, 0] / s["T"] + torch.log(e.sum(1))
    return vals, ids.to(torch.int32), rest


def _plain_distill(s, grad):
    T = s["T"]
    x = s["student"].float()
    ids = s["ids"].long()
    t = s["vals"]
    mt = t[:, :1]
    if s["rest_mass"] is not None:   # one more bucket: all the others
        r = s["rest_mass"][:, None].double() * T
        mt = torch.maximum(mt, r.float())
        t = torch.cat([(t - mt) / T, ((r - mt) / T).float()], 1)
    else:
        t = (t - mt) / T
    et = torch.exp(t)
    zt = et.sum(1, keepdim=True)
    p = et / zt
    m = x.max(1, keepdim=True).values
    e = torch.exp((x - m) / T)
    xs = (x.gather(1, ids) - m) / T
    es = e.gather(1, ids)
    rs = e.scatter(1, ids, 0.0).sum(1, keepdim=True)
    z = es.sum(1, keepdim=True) + rs
    q = es / z
    if s["rest_mass"] is not None:
        q = torch.cat([q, rs / z], 1)
        xs = torch.cat([xs, torch.log(rs)], 1)
    # p and q both sum to one, so the loss is also the sum of p log(p/q) - p + q, whose terms
    # are not negative: for p near q, p (d - 1 + exp(-d)) by its series, d = log(p/q)
    d = (t - xs) - (torch.log(zt) - torch.log(z))
    near = 1 / 5040 - d / 40320
    near = 1 / 24 - d * (1 / 120 - d * (1 / 720 - d * near))
    near = d * d * (0.5 - d * (1 / 6 - d * near))
    loss = torch.where(d.abs() < 0.5, p * near, p * d - p + q).sum(1, keepdim=True)
    if s["rest_mass"] is None:   # the others have p = 0: of p log(p/q) - p + q stays q
        loss = loss + rs / z
    w = s["weight"][:, None]
    loss = (w * loss)[:, 0]
    if not grad:
        return loss
    k = s["k"]
    gr = (w / T) * (e / z)
    if s["rest_mass"] is not None:
        # 1 - p/q of the others; where they have most of the mass, from the named tokens' sums
        named = (p[:, :k].sum(1, keepdim=True) - q[:, :k].sum(1, keepdim=True)) / q[:, k:]
        gr = gr * torch.where(q[:, k:] > 0.5, named, -torch.expm1(d[:, k:]))
    gr = gr.scatter(1, ids, (w / T) * (q - p)[:, :k])
    return loss, gr.to(s["student"].dtype)


def run(state):
    s = state
    op = s["op"]
    if not own:
        if op == "counts":
            return _plain_counts(s)
        if op == "process":
            return _plain_process(s)
        if op == "top":
            return _plain_top(s)
        return _plain_distill(s, op == "grad")
    import speculative_decoding_verification_logits_gb300 as sd
    if op == "counts":
        return sd.token_counts(s["history"], s["lengths"], s["V"],
                               prompt_lengths=s["prompt_lengths"])
    if op == "process":
        return sd.process_logits(s["logits"], counts=s["counts"], prev=s["prev"], base=s["base"],
                                 repetition=s["repetition"], presence=s["presence"],
                                 frequency=s["frequency"], bias_ids=s["bias_ids"],
                                 bias_vals=s["bias_vals"], mask=s["bits"])
    if op == "top":
        return sd.top_logits(s["logits"], s["k"], temperature=s["T"])
    if op == "loss":
        return sd.distill_loss(s["student"], s["ids"], s["vals"], s["rest_mass"],
                               temperature=s["T"], weight=s["weight"])
    return sd.distill_grad(s["student"], s["ids"], s["vals"], s["rest_mass"],
                           temperature=s["T"], weight=s["weight"])


def work(case):
    op, V = case["op"], case["V"]
    if op == "counts":
        B, L = case["B"], case["L"]
        return {"bytes": B * (3 * L // 4) * 4 + 8 * B + 2 * B * V, "flops": B * L}
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "process":
        B, R = case["B"], case["R"]
        n = 2 * B * R * V * es + 2 * B * V + 4 * B * case["P"] + 12 * B + 8 * B * case["bias"]
        if case["mask"] != "none":
            n += B * R * 4 * ((V + 31) // 32)
        return {"bytes": n, "flops": 6 * B * R * V}
    N, k = case["N"], case["k"]
    if op == "top":
        return {"bytes": N * V * es + N * (8 * k + 4), "flops": 4 * N * V}
    small = N * (8 * k + 4 + 4 + (4 if case["rest"] else 0))
    if op == "loss":
        return {"bytes": N * V * es + small, "flops": 4 * N * V}
    return {"bytes": 2 * N * V * es + small, "flops": 8 * N * V}


# ------------------------------------------------- the definitions, in 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "counts":
        return None   # whole numbers: the plain form has them exactly
    D = torch.float64
    if op == "process":
        out = torch.empty(s["logits"].shape, dtype=D, device="cuda")
        B, R, V = out.shape
        v = torch.arange(V, device="cuda")
        for b in range(B):
            word = s["counts"][b].long()
            n0 = torch.remainder(word, 32768).to(D)
            th, al, ph = (float(s[n][b]) for n in ("repetition", "presence", "frequency"))
            add = torch.zeros(V, dtype=D, device="cuda")
            if s["bias_ids"] is not None:
                add[s["bias_ids"][b].long()] = s["bias_vals"][b].to(D)
            for r in range(R):
                n = n0 + torch.bincount(s["prev"][b, :case["base"] + r].long(), minlength=V)
                y = s["logits"][b, r].to(D)
                # with a penalty of 1 or more, dividing what is positive and multiplying the
                # rest both come to the smaller of the two
                y = torch.where((n > 0) | (word < 0), torch.minimum(y / th, y * th), y)
                y = y - n * ph - torch.sign(n) * al + add
                if s["bits"] is not None:
                    y[torch.bitwise_right_shift(s["bits"][b, r].long()[v >> 5], v & 31) % 2 == 0] \
                        = -math.inf
                out[b, r] = y
        return out
    if op == "top":
        vals, rest = [], []
        ids = []
        for x in s["logits"]:
            x = x.to(D)
            y, i = torch.sort(x, descending=True, stable=True)
            vals.append(y[:case["k"]])
            ids.append(i[:case["k"]].to(torch.int32))
            rest.append(torch.logsumexp(y[case["k"]:] / case["T"], 0))
        return torch.stack(vals), torch.stack(ids), torch.stack(rest)
    losses, grads = [], []   # one bucket for each named token, one for all others
    for a in range(0, case["N"], 64):
        x = s["student"][a:a + 64].to(D).requires_grad_(op == "grad")
        ids = s["ids"][a:a + 64].long()
        lt = s["vals"][a:a + 64].to(D) / case["T"]
        if case["rest"]:
            lt = torch.cat([lt, s["rest_mass"][a:a + 64, None].to(D)], 1)
        lt = torch.log_softmax(lt, 1)
        lq = torch.log_softmax(x / case["T"], 1)
        named = lq.gather(1, ids)
        if case["rest"]:
            others = torch.logsumexp(lq.scatter(1, ids, -math.inf), 1, keepdim=True)
            named = torch.cat([named, others], 1)
        loss = (lt.exp() * (lt - named)).sum(1) * s["weight"][a:a + 64].to(D)
        losses.append(loss.detach())
        if op == "grad":
            grads.append(torch.autograd.grad(loss.sum(), x)[0])
    if op == "loss":
        return torch.cat(losses)
    return torch.cat(losses), torch.cat(grads)
