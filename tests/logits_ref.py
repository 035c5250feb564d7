"""The logit operators from their definitions, in 64 bits on the CPU (plain torch and
Python): what the CUDA kernels are tested against, and how far they may be off.

A rounding to type t is off by at most half a step: eps(t) / 2 relative.  The device's
2^x is good to 2^-22 relative.  U = 2^-24 is fp32's half step."""
import math

import torch

D = torch.float64
U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------- counts --
def token_counts(history, lengths, V, prompt_lengths=None):
    B, L = history.shape
    out = torch.zeros((B, V), dtype=torch.int16)
    for b in range(B):
        n = min(max(int(lengths[b]), 0), L)
        p = min(max(int(prompt_lengths[b]), 0), n) if prompt_lengths is not None else 0
        ok = lambda h: h[(h >= 0) & (h < V)].long()
        c = torch.bincount(ok(history[b, p:n]), minlength=V).clamp(max=32767)
        prompt = torch.bincount(ok(history[b, :p]), minlength=V) > 0
        out[b] = torch.where(prompt, c - 32768, c).to(torch.int16)
    return out


def token_counts_add(counts, tokens, n):
    out = counts.clone()
    B, V = counts.shape
    for b in range(B):
        for t in tokens[b, :min(max(int(n[b]), 0), tokens.shape[1])].tolist():
            if 0 <= t < V and (int(out[b, t]) & 0x7FFF) < 0x7FFF:
                out[b, t] += 1
    return out


# ------------------------------------------------------------------ process --
def process(x, counts=None, prev=None, base=0, repetition=None, presence=None, frequency=None,
            bias_ids=None, bias_vals=None, mask=None):
    """(y in 64 bits, the sum of the magnitudes that entered it, whether it was touched)."""
    B, R, V = x.shape
    x64 = x.to(D)
    y, size = x64.clone(), torch.zeros_like(x64)
    touched = torch.zeros(x.shape, dtype=torch.bool)
    for b in range(B):
        word = counts[b].long() if counts is not None else torch.zeros(V, dtype=torch.long)
        th = float(repetition[b]) if repetition is not None else 1.0
        al = float(presence[b]) if presence is not None else 0.0
        ph = float(frequency[b]) if frequency is not None else 0.0
        add = torch.zeros(V, dtype=D)
        mag = torch.zeros(V, dtype=D)
        biased = torch.zeros(V, dtype=torch.bool)
        if bias_ids is not None:
            for t, z in zip(bias_ids[b].tolist(), bias_vals[b].tolist()):
                if 0 <= t < V:
                    add[t] += z
                    mag[t] += abs(z)
                    biased[t] = True
        if not (0 < th < math.inf) or not math.isfinite(al) or not math.isfinite(ph):
            y[b] = math.nan
            touched[b] = True
            continue
        for r in range(R):
            n = word & 0x7FFF
            if prev is not None:
                for t in prev[b, :base + r].tolist():
                    if 0 <= t < V:
                        n = n.index_add(0, torch.tensor([t]), torch.tensor([1]))
            n = n.to(D)
            row = x64[b, r]
            seen = (n > 0) | (word < 0)
            z = torch.where(seen, torch.where(row > 0, row / th, row * th), row)
            w = z - ph * n - al * (n > 0) + add
            y[b, r] = torch.where(row == -math.inf, row, w)
            size[b, r] = z.abs() + abs(ph) * n + abs(al) + mag
            touched[b, r] = (seen | biased) & (row != -math.inf)
            if mask is not None:
                v = torch.arange(V)
                m = mask[b, r] if mask.dim() == 3 else mask[b]
                ok = ((m.long()[v // 32] >> (v % 32)) & 1) == 1
                y[b, r][~ok] = -math.inf
                touched[b, r][~ok] = False
    return y, size, touched


def process_tolerance(y, size, dtype):
    """At most eight fp32 roundings of values no larger than `size` (penalty, product, two
    differences, the biases' sum), then the rounding to the logits' type."""
    return 8 * U * size + half_step(dtype) * (y.abs() + 8 * U * size)


# ---------------------------------------------------------------------- top --
def top(x, k, T):
    N, V = x.shape
    vals = torch.full((N, k), -math.inf)
    ids = torch.full((N, k), -1, dtype=torch.int32)
    rest = torch.full((N,), -math.inf, dtype=D)
    for n in range(N):
        row = x[n].to(D)
        able = torch.where(torch.isnan(row), torch.full_like(row, -math.inf), row)
        o = torch.sort(able, descending=True, stable=True).indices
        o = o[able[o] > -math.inf][:k]
        vals[n, :len(o)] = row[o].float()
        ids[n, :len(o)] = o.to(torch.int32)
        left = torch.ones(V, dtype=torch.bool)
        left[o] = False
        if left.any():
            rest[n] = torch.logsumexp(row[left] / T, 0)
    return vals, ids, rest


def lse_error(V):
    """How far (absolute) the logarithm of a softmax's fp32 sum over V terms may be off: each
    term's 2^x (2^-22) and its argument's two roundings, where the terms that matter lie
    within log2(V) + 8 of the largest; the sum's roundings over a thread's terms, the warp, the
    block and the cluster (at most V / 512 + 64 in a chain); the offsets' rescaling."""
    return 2.0 ** -22 + (math.log2(V + 1) + 8) * 2 * U + (V / 512 + 64) * U + 8 * 2.0 ** -22


def rest_tolerance(rest, top_val, T, V):
    return lse_error(V) + 4 * U * (abs(rest) + abs(top_val / T))


# ------------------------------------------------------------------ distill --
def distill(x, ids, vals, rest, T, weight):
    """loss [N] and its gradient [N][V] by automatic differentiation of the definition, and
    the buckets' shares: dicts p, q ([N][k + 1], 64 bits)."""
    N, V = x.shape
    k = ids.shape[1]
    loss = torch.zeros(N, dtype=D)
    grad = torch.zeros((N, V), dtype=D)
    shares = []
    for n in range(N):
        w = float(weight[n]) if weight is not None else 1.0
        own = ids[n].long()
        some = [(int(i), float(t)) for i, t in zip(own, vals[n]) if i >= 0]
        r = float(rest[n]) if rest is not None else -math.inf
        bad = any(i >= V or i < -1 for i in own.tolist()) or len({i for i, _ in some}) < len(some)
        if w == 0 or bad or (r == -math.inf and all(t == -math.inf for _, t in some)):
            shares.append(None)
            continue
        named = torch.tensor([i for i, _ in some], dtype=torch.long)
        lt = torch.tensor([t / T for _, t in some] + [r], dtype=D)
        lp = lt - torch.logsumexp(lt, 0)
        s = x[n].to(D).requires_grad_(True)
        ls = s / T - torch.logsumexp(s / T, 0)
        others = torch.ones(V, dtype=torch.bool)
        others[named] = False
        # a bucket without teacher mass is no part of the loss: kept out of the graph (the
        # derivative of the logarithm of no mass at all is undefined)
        part = ls[others] if float(lp[-1]) > -math.inf else ls[others].detach()
        lr = torch.logsumexp(part, 0) if others.any() else torch.tensor(-math.inf, dtype=D)
        lq = torch.cat([ls[named], lr.reshape(1)])
        p = lp.exp()
        held = p > 0
        one = (p[held] * (lp[held] - lq[held])).sum() * w
        loss[n] = one.detach()
        if one.requires_grad and math.isfinite(float(one.detach())):
            grad[n] = torch.autograd.grad(one, s)[0]
        shares.append((p.detach(), lq.detach().exp(), lp.detach() - lq.detach(), named,
                       ls.detach()))
    return loss, grad, shares


def distill_tolerance(x, shares, T, weight, V):
    """(loss [N], gradient [N][V]) tolerances before the gradient's rounding to its type.

    E bounds the error of d = ln(p / q): both logarithms of sums and the terms' own 2^x and
    arguments.  The loss sum(p d - p + q) moves by sum |p - q| E to first order and by E^2 to
    second, and rounds each term; a gradient entry moves by E relative to the shares that it
    is made of (the entry of a token far below the row's largest by its argument's roundings
    too)."""
    N = x.shape[0]
    E = 2 * lse_error(V) + 2.0 ** -21
    lt, gt = torch.zeros(N, dtype=D), torch.zeros((N, V), dtype=D)
    for n in range(N):
        if shares[n] is None:
            continue
        p, q, d, named, ls = shares[n]
        w = abs(float(weight[n])) if weight is not None else 1.0
        held = p > 0
        term = torch.where(held, p * d.abs() + p + q, q)
        term = torch.where(held & (d.abs() < 0.4), p * d * d, term)   # by the series
        lt[n] = w * (E * (p - q).abs().sum() + E * E + 2.0 ** -21 * term.sum())
        e = ls.exp()
        far = E + (-ls.clamp(min=-200) / math.log(2)) * 4 * U
        other = q[-1]
        ratio = p[-1] / other if other > 0 else torch.tensor(0.0, dtype=D)
        gt[n] = (w / T) * far * (e + ratio * e)
        gt[n, named] = (w / T) * (E * (p + q))[:-1]
        gt[n] += 2.0 ** -126
    return lt, gt
