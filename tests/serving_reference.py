"""Plain definitions of the serving operators (CPU, 64 bits where numbers are
computed), and how far the kernels may be off them.

Attention.  The products' operands are exact (codes, and q up to a power of
two), sums are fp32: a score of `dim` products is off by at most dim + 8 half
steps of its terms' sizes, (dim + 8) * 2^-24 * sum |q k|, twice that where the
tensor cores cut off instead of rounding; dz is that, plus 2^-21 of the score's
own size for the factors (four roundings of 2^-24 and the exponential's 2^-22).
A weight is then off by a share of 2 dz + 2^-11 (its rounding to fp16, with the
sum's 2^-20 below it), and the output by as much of sum p |v|, plus half a step
of its own type: relative to the value, but below the type's smallest normal
number the steps are all alike, 2^-24 for fp16 (2^-14, ten fraction bits), so
that half a step is 2^-25 there whatever the value.
"""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
LEAST_HALF_STEP = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- slots --

def slots(cached, added, held, free, count, table, page, capacity):
    """(table, held, lengths, offsets, slots, left), by one loop over the requests."""
    cols = table.shape[1]
    table = table.clone()
    n = len(cached)
    taken, row = 0, 0
    held_out, lengths, offsets, slot = [], [], [0], [-1] * capacity
    count = min(max(count, 0), len(free))
    for b in range(n):
        c, a, h = max(int(cached[b]), 0), max(int(added[b]), 0), min(max(int(held[b]), 0), cols)
        need = max(0, min(-(-(c + a) // page), cols) - h)
        got = 0
        for j in range(need):
            at = count - 1 - taken
            taken += 1
            table[b, h + j] = int(free[at]) if at >= 0 else -1
            got += at >= 0
        held_out.append(h + got)
        lengths.append(min(c + a, 2 ** 31 - 1))
        for i in range(a):
            if row + i >= capacity:
                break
            pos = c + i
            if pos // page < cols and int(table[b, pos // page]) >= 0:
                slot[row + i] = int(table[b, pos // page]) * page + pos % page
        row += a
        offsets.append(min(row, capacity))
    return table, held_out, lengths, offsets, slot, count - taken


# ------------------------------------------------------------------- write --

def _codes(x):
    """e4m3 of fp32 values, to nearest even; NaN for what is not finite."""
    return torch.where(x.isfinite(), x.clamp(-448.0, 448.0), torch.full_like(x, math.nan)).to(F8)


def write(x, slot, cache, scale):
    """The cache [pages, heads, page, dim] and scales [pages, heads] after x [rows, heads, dim], in fp32 as specified."""
    cache, scale = cache.clone(), scale.clone()
    pages, heads, page, _ = cache.shape
    rows, t = x.shape[0], 0
    slot = slot.tolist()
    while t < rows:
        s = slot[t]
        if s < 0 or s >= pages * page:
            t += 1
            continue
        n = 1
        while t + n < rows and slot[t + n] == s + n and (s + n) % page:
            n += 1
        p, o = s // page, s % page
        run = x[t:t + n].float()
        size = torch.where(run.isfinite(), run.abs(), torch.zeros_like(run)).amax(dim=(0, 2))
        new = torch.maximum(size / torch.full_like(size, 448.0), torch.full_like(size, 2.0 ** -126))
        old = scale[p].clone()
        if o:
            new = torch.maximum(old, new)
        inv = torch.ones_like(new) / new
        if o:
            grown = new > old
            before = cache[p, :, :o].float()
            again = _codes(before * (old * inv)[:, None, None])
            cache[p, :, :o] = torch.where(grown[:, None, None], again.float(), before).to(F8)
        cache[p, :, o:o + n] = _codes(run * inv[None, :, None]).transpose(0, 1)
        scale[p] = new
        t += n
    return cache, scale


# --------------------------------------------------------------- attention --

def attention(q, k_cache, v_cache, k_scale, v_scale, table, offsets, lengths, scale):
    """(out, lse, bar of out, bar of lse) in 64 bits; rows of no request are NaN."""
    rows, q_heads, dim = q.shape
    pages, heads, page, _ = k_cache.shape
    group, half = q_heads // heads, HALF_STEP[q.dtype]
    out = torch.full((rows, q_heads, dim), math.nan, dtype=torch.float64)
    lse = torch.full((rows, q_heads), math.nan, dtype=torch.float64)
    out_bar, lse_bar = torch.zeros_like(out), torch.zeros_like(lse)
    for b, length in enumerate(lengths):
        lo, hi = offsets[b], offsets[b + 1]
        n = hi - lo
        length = min(length, table.shape[1] * page)
        at = table[b, :-(-length // page)].long()
        there = ((at >= 0) & (at < pages)).repeat_interleave(page)[:length]
        at = at.clamp(0, pages - 1)
        for h in range(q_heads):
            kv = h // group
            k = (k_cache.view(torch.uint8)[at, kv].view(F8).double() * k_scale[at, kv].double()[:, None, None]).reshape(-1, dim)[:length]
            v = (v_cache.view(torch.uint8)[at, kv].view(F8).double() * v_scale[at, kv].double()[:, None, None]).reshape(-1, dim)[:length]
            for i in range(n):
                sees = there & (torch.arange(length) < length - n + i + 1)
                x = q[lo + i, h].double()
                if not bool(sees.any()):
                    out[lo + i, h], lse[lo + i, h] = 0.0, -math.inf
                    continue
                ks, vs = k[sees], v[sees]
                z = ks @ x * scale
                lse[lo + i, h] = torch.logsumexp(z, 0)
                p = torch.softmax(z, 0)
                out[lo + i, h] = p @ vs
                terms = (ks.abs() @ x.abs()).max() * scale
                dz = float(2 * (dim + 8) * 2.0 ** -24 * terms + 2.0 ** -21 * z.abs().max())
                out_bar[lo + i, h] = (2 * dz + 2.0 ** -11 + 2.0 ** -20) * (p @ vs.abs()) + \
                    (half * out[lo + i, h].abs()).clamp(min=LEAST_HALF_STEP[q.dtype])
                lse_bar[lo + i, h] = dz + 2.0 ** -20 + 2.0 ** -22 * lse[lo + i, h].abs()
    if q.dtype == torch.float16:  # above the middle of 65504 and the step behind it a value rounds to infinity
        out = torch.where(out.abs() >= 65520.0, torch.sign(out) * math.inf, out)
    return out, lse, out_bar, lse_bar


# ------------------------------------------------------------------ verify --

def verify(target, draft, drafted, offsets, uniform, noise, scale):
    """(tokens, accepted, logp) in 64 bits; `scale` as fp32 has it."""
    scale = float(torch.tensor(scale, dtype=torch.float32))
    rows, cols = target.shape
    requests = len(offsets) - 1
    tokens, logp = [-1] * rows, [0.0] * rows

    def logs(z):
        z = z.double() * scale
        return z - torch.logsumexp(z, 0)

    def first_of_most(key):
        key = torch.where(key > 0, key, torch.zeros_like(key))
        top = float(key.max())
        return int((key == top).nonzero()[0]) if top > 0 else -1

    accepted = []
    for b in range(requests):
        lo, hi = offsets[b], offsets[b + 1]
        a = 0
        while a < hi - lo:
            x, row = int(drafted[lo + a]), lo + a + b
            if not 0 <= x < cols:
                break
            lp = float(logs(target[row])[x])
            q = 1.0 if draft is None else math.exp(float(logs(draft[lo + a])[x]))
            if not float(uniform[lo + a]) * q < math.exp(lp):
                break
            tokens[row], logp[row] = x, lp
            a += 1
        row = lo + a + b
        lp = logs(target[row])
        p = lp.exp()
        r = p
        if a < hi - lo:
            if draft is None:
                r = p.clone()
                if 0 <= int(drafted[lo + a]) < cols:
                    r[int(drafted[lo + a])] = 0.0
            else:
                r = (p - logs(draft[lo + a]).exp()).clamp(min=0)
        y = first_of_most(r / noise[b].double())
        if y < 0:
            y = first_of_most(p / noise[b].double())
        tokens[row] = y
        logp[row] = float(lp[y]) if y >= 0 else 0.0
        accepted.append(a)
    return tokens, accepted, logp
