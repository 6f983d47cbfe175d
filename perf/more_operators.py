"""The operators of a serving step over a cache held in 8 bits, as cases that can be timed.

Four operators, in the order in which a step runs them:

  slots      block tables and slot maps from request lengths
  write      new keys and values into the cache's pages, one scale for each page and head
  attention  of new tokens (one, a few drafted ones, a prompt) over the cache
  verify     drafted tokens against the target's probabilities, from given random numbers

With ``own`` false, ``run`` computes the plain form in elementary torch
operations; with ``own`` true it calls the library's entry points.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_F8 = torch.float8_e4m3fn
_TOP = 448.0  # the largest e4m3 value
_LEAST = 2.0 ** -126  # the smallest scale


# --------------------------------------------------------------- the cases --

def listed():
    return [
        # every request decodes one token: nothing but latency
        dict(name="slots_step", op="slots", requests=256, new=256, cached=250_000, page=64, ragged=False),
        # a million tokens of new prompts are laid out at once, small pages
        dict(name="slots_prompts", op="slots", requests=500, new=1_000_003, cached=100_000, page=16, ragged=True),
        # one token for each of 128 requests, into pages that are partly full
        dict(name="write_step_bf16", op="write", requests=128, new=128, cached=100_000, heads=8, dim=128, page=64,
             dtype="bf16", ragged=False),
        # the keys and values of prompts, most of them whole pages
        dict(name="write_prompts_f16", op="write", requests=24, new=65_521, cached=5_000, heads=8, dim=128, page=64,
             dtype="f16", ragged=True),
        # a few short requests of a small model: nothing but latency
        dict(name="attention_few_f16", op="attention", requests=4, new=4, total=1_501, heads=8, group=1, dim=64,
             page=16, dtype="f16", ragged=True),
        # one request with a long context: the work of a head has to be split along the cache
        dict(name="attention_long_bf16", op="attention", requests=1, new=1, total=131_071, heads=8, group=4, dim=128,
             page=64, dtype="bf16", ragged=False),
        # a batch that decodes, ragged lengths
        dict(name="attention_step_bf16", op="attention", requests=64, new=64, total=300_007, heads=8, group=4, dim=128,
             page=64, dtype="bf16", ragged=True),
        # five drafted tokens a request are checked in one pass; more query heads a key head
        dict(name="attention_drafts_f16", op="attention", requests=48, new=240, total=150_001, heads=8, group=8,
             dim=128, page=32, dtype="f16", ragged=True),
        # parts of prompts over what is cached of them
        dict(name="attention_prompts_bf16", op="attention", requests=4, new=8_191, total=16_381, heads=8, group=4,
             dim=128, page=64, dtype="bf16", ragged=True),
        # one request with four drafts: few rows, so a row has to spread over the chip
        dict(name="verify_few_f32", op="verify", requests=1, drafts=4, cols=32_000, dtype="f32", onehot=False,
             scale=1.0),
        # a batch with four drafts a request over a large vocabulary
        dict(name="verify_step_bf16", op="verify", requests=64, drafts=256, cols=128_000, dtype="bf16", onehot=False,
             scale=1.25),
        # drafts looked up in retrieved text (no probabilities of their own), ragged, an odd vocabulary
        dict(name="verify_odd_f16", op="verify", requests=37, drafts=101, cols=50_001, dtype="f16", onehot=True,
             scale=0.8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "write", "attention", "attention", "verify"])
    if op == "slots":
        requests = _log_int(rng, 1, 2000)
        new = rng.choice([requests, _log_int(rng, requests, 1_000_000)])
        return dict(op=op, requests=requests, new=new, cached=_log_int(rng, 10, 300_000),
                    page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7)
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "write":
        requests = _log_int(rng, 1, 256)
        new = rng.choice([requests, _log_int(rng, requests, 60_000)])
        return dict(op=op, requests=requests, new=new, cached=_log_int(rng, 10, 50_000), heads=rng.choice([1, 2, 4, 8]),
                    dim=rng.choice([64, 80, 96, 128]), page=rng.choice([16, 32, 64, 128]), dtype=dtype,
                    ragged=rng.random() < 0.7)
    if op == "attention":
        requests = _log_int(rng, 1, 64)
        heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 7, 8])
        case = dict(op=op, heads=heads, group=group, dim=rng.choice([64, 80, 96, 128]),
                    page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["f16", "bf16"]), ragged=rng.random() < 0.7)
        kind = rng.choice(["step", "drafts", "prompts"])
        if kind == "prompts":
            requests = min(requests, 8)
            new = requests * _log_int(rng, 20, 2000)
            total = new + _log_int(rng, 1, 10_000)
            while new * (total / requests) * heads * group > 5e8:
                new = max(requests, new // 2)
                total = max(new, total // 2)
        else:
            new = requests if kind == "step" else requests * rng.randint(2, 8)
            total = max(2 * new, _log_int(rng, 100, 250_000))
        return dict(case, requests=requests, new=new, total=total)
    cols = _log_int(rng, 16, 131_072)
    requests = _log_int(rng, 1, 64)
    drafts = min(requests * rng.randint(0, 6), 256, max(1, 30_000_000 // cols))
    return dict(op=op, requests=requests, drafts=drafts, cols=cols, dtype=dtype, onehot=rng.random() < 0.4,
                scale=rng.choice([0.7, 1.0, 1.25]))


# -------------------------------------------------------------- the inputs --

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _split(gen, total, parts, ragged):
    """`total` things over `parts` requests: one each first (as far as they go), the rest at random or evenly."""
    least = 1 if total >= parts else 0
    rest = total - least * parts
    if ragged:  # from a fifth to 5 times an even share
        w = 0.2 + 0.8 * torch.rand(parts, generator=gen, device="cuda", dtype=torch.float64)
        ends = (w.cumsum(0) / w.sum() * rest).round().long()
        ends[-1] = rest
    else:
        ends = torch.arange(1, parts + 1, device="cuda") * rest // parts
    got = ends.clone()
    got[1:] -= ends[:-1]
    return got + least


def _pages(n, page):
    return (n + page - 1) // page


def _width(total, requests, page):
    """Columns of a table that holds any request of _split's, whatever the seed."""
    return _pages(min(total, 5 * -(-total // requests)) + 2, page)


def _prefix(n):
    return torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), n.cumsum(0)])


def _table(gen, held, width, pool):
    """Rows of distinct random pages, `held` of them each, -1 behind; and the pages that are left."""
    order = torch.randperm(pool, generator=gen, device="cuda")
    col = torch.arange(width, device="cuda")
    at = _prefix(held)[:-1, None] + col
    table = torch.where(col < held[:, None], order[at.clamp(max=pool - 1)], torch.full_like(at, -1))
    return table.int(), order[int(held.sum()):].int().contiguous()


def _prepare_slots(case, gen):
    requests, page = case["requests"], case["page"]
    cached = _split(gen, case["cached"], requests, True)
    added = _split(gen, case["new"], requests, case["ragged"])
    # a request whose drafts were turned down holds a page more than its tokens fill
    held = _pages(cached, page) + (torch.rand(requests, generator=gen, device="cuda") < 0.1).long()
    width = _width(case["cached"], requests, page) + _width(case["new"], requests, page) + 4
    pool = _pages(case["cached"] + case["new"], page) + 3 * requests + 64
    table, free = _table(gen, held, width, pool)
    i32 = dict(dtype=torch.int32, device="cuda")
    # the slot map has room for a fixed number of tokens, as a captured graph needs it
    return dict(cached=cached.int(), added=added.int(), held=held.int(), free=free,
                count=torch.tensor([free.numel()], **i32), table=table, held_out=torch.empty(requests, **i32),
                lengths=torch.empty(requests, **i32), offsets=torch.empty(requests + 1, **i32),
                slots=torch.empty(case["new"] + 8, dtype=torch.int64, device="cuda"), left=torch.empty(1, **i32))


def _codes(gen, pool, heads, page, dim):
    x = torch.randn(pool, heads, page, dim, generator=gen, device="cuda", dtype=torch.float16) * 110.0
    return x.clamp_(-_TOP, _TOP).to(_F8)


def _scales(gen, pool, heads):
    return torch.exp(0.5 * torch.randn(pool, heads, generator=gen, device="cuda")) * 0.009


def _prepare_write(case, gen):
    requests, page, heads, dim = case["requests"], case["page"], case["heads"], case["dim"]
    cached = _split(gen, case["cached"], requests, True)
    added = _split(gen, case["new"], requests, case["ragged"])
    held = _pages(cached + added, page)
    pool = _pages(case["cached"] + case["new"], page) + requests + 16
    table, _ = _table(gen, held, int(held.max()), pool)
    offsets = _prefix(added)
    rows = case["new"] + 8  # rows of padding behind the last token
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(offsets[1:], t, right=True).clamp(max=requests - 1)
    pos = cached[b] + t - offsets[b]
    slots = table.long()[b, (pos // page).clamp(max=table.shape[1] - 1)] * page + pos % page
    slots = torch.where(t < case["new"], slots, torch.full_like(slots, -1))
    # heads differ in size, and now and then a token stands out
    size = torch.exp(torch.randn(heads, 1, generator=gen, device="cuda"))
    out = 1.0 + 5.0 * (torch.rand(rows, 1, 1, generator=gen, device="cuda") < 0.02).float()
    k, v = ((torch.randn(rows, heads, dim, generator=gen, device="cuda") * size * out).to(_DT[case["dtype"]])
            for _ in range(2))
    return dict(k=k, v=v, slots=slots, k_cache=_codes(gen, pool, heads, page, dim),
                v_cache=_codes(gen, pool, heads, page, dim), k_scale=_scales(gen, pool, heads),
                v_scale=_scales(gen, pool, heads))


def _prepare_attention(case, gen):
    requests, page, heads, dim = case["requests"], case["page"], case["heads"], case["dim"]
    added = _split(gen, case["new"], requests, case["ragged"] and case["new"] > 8 * requests)
    lengths = added + _split(gen, case["total"] - case["new"], requests, case["ragged"])
    held = _pages(lengths, page)
    pool = _pages(case["total"], page) + requests + 16
    table, _ = _table(gen, held, int(held.max()) + 2, pool)
    rows, q_heads = case["new"], heads * case["group"]
    q = (torch.randn(rows, q_heads, dim, generator=gen, device="cuda") * 2.0).to(_DT[case["dtype"]])
    return dict(q=q, k_cache=_codes(gen, pool, heads, page, dim), v_cache=_codes(gen, pool, heads, page, dim),
                k_scale=_scales(gen, pool, heads), v_scale=_scales(gen, pool, heads), table=table,
                offsets=_prefix(added).int(), lengths=lengths.int(), most=int(added.max()), out=torch.empty_like(q),
                lse=torch.empty(rows, q_heads, device="cuda"), scale=1.0 / math.sqrt(dim))


def _prepare_verify(case, gen):
    requests, n, cols, dt = case["requests"], case["drafts"], case["cols"], _DT[case["dtype"]]
    offsets = _prefix(_split(gen, n, requests, n > 8 * requests or n % requests > 0))
    rows = n + requests
    b = torch.searchsorted(offsets[1:], torch.arange(n, device="cuda"), right=True)
    target_row = torch.arange(n, device="cuda") + b
    # a broad bulk with a few dozen likely columns; the draft model has learnt most of it
    target = torch.randn(rows, cols, generator=gen, device="cuda") * 1.5
    likely = torch.randint(0, cols, (rows, 40), generator=gen, device="cuda")
    peak = 7.0 + 2.0 * torch.randn(rows, 40, generator=gen, device="cuda")
    target.scatter_add_(1, likely, peak)
    if cols > 64:  # columns that the sampler has ruled out
        target[:, cols // 3] = float("-inf")
    draft = target[target_row] + 0.6 * torch.randn(n, cols, generator=gen, device="cuda")
    target, draft = target.to(dt), draft.to(dt)
    gumbel = -torch.log(torch.empty(n, cols, device="cuda").exponential_(generator=gen).clamp_(min=1e-20))
    tokens = (draft.float() * case["scale"] + gumbel).argmax(dim=1) if n else torch.zeros(0, dtype=torch.long)
    noise = torch.empty(requests, cols, device="cuda").exponential_(generator=gen)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(target=target, draft=None if case["onehot"] else draft, drafted=tokens.to(**i32),
                offsets=offsets.int(), uniform=torch.rand(n, generator=gen, device="cuda"), noise=noise,
                tokens=torch.empty(rows, **i32), accepted=torch.empty(requests, **i32),
                logp=torch.empty(rows, device="cuda"))


_PREPARE = {"slots": _prepare_slots, "write": _prepare_write, "attention": _prepare_attention,
            "verify": _prepare_verify}


def prepare(case, seed):
    return dict(_PREPARE[case["op"]](case, _generator(seed)), case=dict(case))


# -------------------------------------------------------------- the passes --

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_slots(s):
    from late_interaction_retrieval_gb300 import binding
    binding.lik_cache_slots(s["cached"], s["added"], s["held"], s["free"], s["count"], s["table"], s["held_out"],
                            s["lengths"], s["offsets"], s["slots"], s["left"], page_size=s["case"]["page"])
    return {"table": s["table"], "held": s["held_out"], "lengths": s["lengths"], "offsets": s["offsets"],
            "slots": s["slots"], "left": s["left"]}


def _own_write(s):
    from late_interaction_retrieval_gb300 import binding
    binding.lik_cache_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _own_attention(s):
    from late_interaction_retrieval_gb300 import binding
    if "workspace" not in s:  # kept from pass to pass, as a serving loop keeps it
        need = binding.lik_cache_attention_workspace_bytes(s["q"], s["k_cache"], s["table"], max_added=s["most"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    binding.lik_cache_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                s["offsets"], s["lengths"], s["out"], s["lse"], workspace=s["workspace"],
                                max_added=s["most"], scale=s["scale"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_verify(s):
    from late_interaction_retrieval_gb300 import binding
    if "workspace" not in s:
        need = binding.lik_verify_drafts_workspace_bytes(s["target"], s["accepted"].numel())
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    binding.lik_verify_drafts(s["target"], s["draft"], s["drafted"], s["offsets"], s["uniform"], s["noise"],
                              s["tokens"], s["accepted"], s["logp"], workspace=s["workspace"],
                              scale=s["case"]["scale"])
    return {"tokens": s["tokens"], "accepted": s["accepted"], "logp": s["logp"]}


_OWN = {"slots": _own_slots, "write": _own_write, "attention": _own_attention, "verify": _own_verify}


def _plain_slots(s):
    page, room = s["case"]["page"], s["slots"].numel()
    cached, added, held, count = s["cached"].long(), s["added"].long(), s["held"].long(), s["count"].long()
    requests, width = s["table"].shape
    total = cached + added
    need = (_pages(total, page).clamp(max=width) - held).clamp(min=0)
    first = need.cumsum(0) - need
    col = torch.arange(width, device="cuda")
    rank = first[:, None] + col - held[:, None]
    taken = s["free"].long()[(count - 1 - rank).clamp(0, s["free"].numel() - 1)]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    table = torch.where(fresh, torch.where(rank < count, taken, torch.full_like(rank, -1)), s["table"].long())
    s["table"].copy_(table)
    held_out = held + torch.minimum(need, count - first).clamp(min=0)
    offsets = _prefix(added).clamp(max=room)
    t = torch.arange(room, device="cuda")
    b = torch.searchsorted(offsets[1:], t, right=True).clamp(max=requests - 1)
    pos = cached[b] + t - offsets[b]
    at = table[b, (pos // page).clamp(max=width - 1)]
    there = (t < offsets[-1]) & (pos // page < width) & (at >= 0)
    slots = torch.where(there, at * page + pos % page, torch.full_like(at, -1))
    return {"table": s["table"], "held": held_out.int(), "lengths": total.int(), "offsets": offsets.int(),
            "slots": slots, "left": (count - need.sum()).int()}


def _to_codes(x):
    """e4m3 of values in units of their scale; what is not finite becomes NaN."""
    return torch.where(x.isfinite(), x.clamp(-_TOP, _TOP), torch.full_like(x, math.nan)).to(_F8)


def _plain_write_one(x, slots, cache, scale):
    pool, heads, page, dim = cache.shape
    live = slots >= 0
    x = x.float()
    # pages of tokens that are not written: one behind the last
    at = torch.where(live, slots // page, torch.full_like(slots, pool))
    offset = torch.where(live, slots % page, torch.full_like(slots, page))
    size = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(dim=2)
    most = torch.zeros(pool + 1, heads, device="cuda").scatter_reduce_(0, at[:, None].expand_as(size), size, "amax")
    first = torch.full((pool + 1,), page, device="cuda").scatter_reduce_(0, at, offset, "amin")
    most, first = most[:pool], first[:pool]
    fresh = (most / _TOP).clamp(min=_LEAST)
    grown = torch.where(first[:, None] == 0, fresh, torch.maximum(scale, fresh))
    new = torch.where(first[:, None] < page, grown, scale)
    inverse = 1.0 / new
    held = torch.arange(page, device="cuda") < first[:, None]
    again = held[:, None, :, None] & (new > scale)[:, :, None, None]
    codes = torch.where(again, _to_codes(cache.float() * (scale * inverse)[:, :, None, None]).float(), cache.float())
    owner = torch.full((pool * page + 1,), -1, dtype=torch.long, device="cuda")
    owner.scatter_(0, torch.where(live, slots, torch.full_like(slots, pool * page)),
                   torch.arange(slots.numel(), device="cuda"))
    owner = owner[:pool * page].view(pool, page)
    token = _to_codes(x * inverse[at.clamp(max=pool - 1)][:, :, None]).float()
    written = token[owner.clamp(min=0)].transpose(1, 2)  # [pool, heads, page, dim]
    codes = torch.where((owner >= 0)[:, None, :, None], written, codes)
    cache.copy_(codes.to(_F8))
    scale.copy_(new)


def _plain_write(s):
    _plain_write_one(s["k"], s["slots"], s["k_cache"], s["k_scale"])
    _plain_write_one(s["v"], s["slots"], s["v_cache"], s["v_scale"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _gathered(cache, scale, table, there):
    """The cache's values [requests, heads, tokens, dim]; what is not there is 0."""
    pool, heads, page, dim = cache.shape
    at = table.clamp(min=0)
    x = cache.view(torch.uint8)[at].view(_F8).float() * scale[at][:, :, :, None, None]
    x = x.transpose(1, 2).reshape(table.shape[0], heads, -1, dim)
    return torch.where(there[:, None, :, None], x, torch.zeros_like(x))


def _plain_attention(s):
    c, table = s["case"], s["table"].long()
    page, heads, group, dim, most = c["page"], c["heads"], c["group"], c["dim"], s["most"]
    requests, rows = table.shape[0], s["q"].shape[0]
    lengths, offsets = s["lengths"].long(), s["offsets"].long()
    added = offsets[1:] - offsets[:-1]
    pos = torch.arange(table.shape[1] * page, device="cuda")
    there = (pos < lengths[:, None]) & (table >= 0).repeat_interleave(page, dim=1)
    k = _gathered(s["k_cache"], s["k_scale"], table, there)
    v = _gathered(s["v_cache"], s["v_scale"], table, there)
    i = torch.arange(most, device="cuda")
    q = s["q"].float()[(offsets[:-1, None] + i).clamp(max=rows - 1)]  # [requests, most, q heads, dim]
    q = q.view(requests, most, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(requests, heads, most * group, dim)
    z = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    sees = (pos < (lengths - added)[:, None, None] + i[:, None] + 1) & there[:, None]
    sees = sees.repeat_interleave(group, dim=1)[:, None]  # [requests, 1, most * group, tokens]
    z = torch.where(sees, z, torch.full_like(z, -math.inf))
    m = z.amax(dim=3, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(z - m)
    total = e.sum(dim=3, keepdim=True)
    out = torch.matmul(e, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (m + torch.log(total))[..., 0]
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(offsets[1:], t, right=True)
    at = t - offsets[b]
    out = out.view(requests, heads, most, group, dim)[b, :, at].reshape(rows, heads * group, dim)
    lse = lse.view(requests, heads, most, group)[b, :, at].reshape(rows, heads * group)
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _softmax64(z, scale):
    """Probabilities and their logarithms in 64 bits: a draw next to a border needs them."""
    z = z.double() * scale
    m = z.amax(dim=1, keepdim=True)
    z = z - torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(z)
    total = e.sum(dim=1, keepdim=True)
    return e / total, z - torch.log(total)


def _lowest_of_most(key):
    """Each row's column of the largest positive key (the lowest of equals), -1 where there is none."""
    cols = key.shape[1]
    key = torch.where(key > 0, key, torch.zeros_like(key))
    top = key.amax(dim=1, keepdim=True)
    at = torch.where((key == top) & (key > 0), torch.arange(cols, device="cuda"), torch.full_like(key, cols).long())
    at = at.amin(dim=1)
    return torch.where(at < cols, at, torch.full_like(at, -1))


def _plain_verify(s):
    scale, offsets, drafted = s["case"]["scale"], s["offsets"].long(), s["drafted"].long()
    requests, rows, n = offsets.numel() - 1, s["target"].shape[0], s["drafted"].numel()
    # a scale is 32 bits wide at the operator
    scale = float(torch.tensor(scale, dtype=torch.float32))
    p, log_p = _softmax64(s["target"], scale)
    t = torch.arange(n, device="cuda")
    b = torch.searchsorted(offsets[1:], t, right=True)
    px = p[t + b, drafted]
    q = None if s["draft"] is None else _softmax64(s["draft"], scale)[0]
    qx = torch.ones_like(px) if q is None else q[t, drafted]
    passed = s["uniform"].double() * qx < px
    counts = offsets[1:] - offsets[:-1]
    stops = torch.where(passed, counts[b], t - offsets[b])
    accepted = counts.clone().scatter_reduce_(0, b, stops, "amin")
    row = offsets[:-1] + torch.arange(requests, device="cuda") + accepted
    short = accepted < counts
    pr = p[row]
    at = (offsets[:-1] + accepted).clamp(max=max(n - 1, 0))
    if n == 0:
        residual = pr
    elif q is None:
        residual = torch.where(short[:, None] & (torch.arange(pr.shape[1], device="cuda") == drafted[at][:, None]),
                               torch.zeros_like(pr), pr)
    else:
        residual = torch.where(short[:, None], (pr - q[at]).clamp(min=0), pr)
    noise = s["noise"].double()
    token = _lowest_of_most(residual / noise)
    token = torch.where(token < 0, _lowest_of_most(pr / noise), token)
    # rows of the target: the drafts that passed, the drawn token, -1 behind it
    r = torch.arange(rows, device="cuda")
    rb = torch.searchsorted(offsets[1:] + torch.arange(1, requests + 1, device="cuda"), r, right=True)
    inside = r - offsets[rb] - rb
    kept = torch.full((rows,), -1, dtype=torch.long, device="cuda")
    kept[t + b] = drafted
    tokens = torch.where(inside < accepted[rb], kept, torch.where(inside == accepted[rb], token[rb], -1))
    logp = log_p.gather(1, tokens.clamp(min=0)[:, None])[:, 0]
    logp = torch.where(tokens >= 0, logp, torch.zeros_like(logp))
    return {"tokens": tokens.int(), "accepted": accepted.int(), "logp": logp.float()}


_PLAIN = {"slots": _plain_slots, "write": _plain_write, "attention": _plain_attention, "verify": _plain_verify}


# ---------------------------------------------------------------- the work --

def _bytes_of(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    """Each input that a pass cannot do without read once, each output written once."""
    op, requests = case["op"], case["requests"]
    if op == "slots":
        pages = case["new"] // case["page"] + requests
        # three numbers of a request in and out, its new pages read and written, 64-bit slots
        return {"bytes": 24 * requests + 8 * pages + 8 * (case["new"] + 8), "flops": case["new"] * 4}
    if op == "write":
        elements = 2 * case["new"] * case["heads"] * case["dim"]
        pages = case["new"] // case["page"] + requests
        return {"bytes": elements * (_bytes_of(case["dtype"]) + 1) + 16 * pages * case["heads"] + 8 * case["new"],
                "flops": elements * 3}
    if op == "attention":
        new, total, q_heads = case["new"], case["total"], case["heads"] * case["group"]
        each = new / requests
        pairs = new * (total / requests - each) + new * (each + 1) / 2
        pages = total // case["page"] + requests
        return {"bytes": 2 * total * case["heads"] * case["dim"] + pages * (4 + 8 * case["heads"]) +
                new * q_heads * (2 * _bytes_of(case["dtype"]) * case["dim"] + 4),
                "flops": int(4 * case["dim"] * q_heads * pairs)}
    rows = case["drafts"] + requests + (0 if case["onehot"] else case["drafts"])
    elements = rows * case["cols"]
    # subtract, scale, exponential, add; a quotient and a comparison in the row that is drawn from
    return {"bytes": elements * _bytes_of(case["dtype"]) + 4 * requests * case["cols"] + 20 * rows,
            "flops": elements * 4 + 4 * requests * case["cols"]}


# ---------------------------------------------------- the definition, fp64 --

def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers only
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, s)


def _exact_write(case, s):
    page, pool = case["page"], s["k_cache"].shape[0]
    slots = s["slots"]
    live = slots[slots >= 0]
    at, offset = live // page, live % page
    out = {}
    for name in ("k", "v"):
        x = s[name][slots >= 0].double()
        codes, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
        size = x.abs().amax(dim=2)
        top = torch.zeros_like(scale).index_reduce_(0, at, size, "amax")
        low = torch.full((pool,), page, device="cuda").index_reduce_(0, at, offset, "amin")
        hit = low < page
        after = (top / _TOP).clamp(min=_LEAST)
        after[low > 0] = torch.maximum(after, scale)[low > 0]
        after[~hit] = scale[~hit]
        ratio = torch.where(hit[:, None] & (low > 0)[:, None], scale / after, torch.ones_like(scale))
        codes = codes * ratio[:, :, None, None]
        # what stands behind a page's new tokens is no token: left as it was
        behind = torch.arange(page, device="cuda")[None, :] >= low[:, None]
        before = s[name + "_cache"].double()
        codes = torch.where(behind[:, None, :, None], before, codes)
        codes[at, :, offset] = x / after[at][:, :, None]
        out[name + "_cache"], out[name + "_scale"] = codes, after
    return {key: out[key] for key in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _exact_attention(case, s):
    new, q_heads = s["q"].shape[:2]
    heads, group, dim, page = case["heads"], case["group"], case["dim"], case["page"]
    out = torch.zeros(new, q_heads, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((new, q_heads), -math.inf, dtype=torch.float64, device="cuda")
    cuts, lengths = s["offsets"].tolist(), s["lengths"].tolist()
    if sum((b - a) * n for a, b, n in zip(cuts, cuts[1:], lengths)) * q_heads * dim > 2e11:
        return None
    for b, length in enumerate(lengths):
        lo, hi = cuts[b], cuts[b + 1]
        pages = s["table"][b, :_pages(length, page)].long()
        last = torch.arange(lo, hi, device="cuda") - hi + length  # the last position that a row sees
        hidden = torch.arange(length, device="cuda")[None, :] > last[:, None]
        for h in range(heads):
            k = (s["k_cache"][:, h][pages].double() * s["k_scale"][pages, h].double()[:, None, None]).reshape(-1, dim)
            v = (s["v_cache"][:, h][pages].double() * s["v_scale"][pages, h].double()[:, None, None]).reshape(-1, dim)
            for g in range(h * group, (h + 1) * group):
                z = (s["q"][lo:hi, g].double() @ k[:length].T) * s["scale"]
                z = z.masked_fill(hidden, -math.inf)
                lse[lo:hi, g] = torch.logsumexp(z, dim=1)
                out[lo:hi, g] = torch.softmax(z, dim=1) @ v[:length]
    return {"out": out, "lse": lse}


def _exact_verify(case, s):
    scale = float(torch.tensor(case["scale"], dtype=torch.float32))
    rows = s["target"].shape[0]
    cuts, uniform, drafted = s["offsets"].tolist(), s["uniform"].tolist(), s["drafted"].tolist()
    logp = torch.zeros(rows, dtype=torch.float64, device="cuda")
    for b in range(case["requests"]):
        lo, hi = cuts[b], cuts[b + 1]
        logs = torch.log_softmax(s["target"][lo + b:hi + b + 1].double() * scale, dim=1)
        own_logs = None if s["draft"] is None else torch.log_softmax(s["draft"][lo:hi].double() * scale, dim=1)
        n = 0
        while n < hi - lo:
            x = drafted[lo + n]
            chance = 1.0 if own_logs is None else float(own_logs[n, x].exp())
            if not uniform[lo + n] * chance < float(logs[n, x].exp()):
                break
            logp[lo + b + n] = logs[n, x]
            n += 1
        mass = logs[n].exp()
        if n < hi - lo:
            if own_logs is None:
                mass[drafted[lo + n]] = 0.0
            else:
                mass = torch.clamp(mass - own_logs[n].exp(), min=0.0)
        pick = int(torch.argmax(mass / s["noise"][b].double()))
        logp[lo + b + n] = logs[n, pick]
    return {"tokens": None, "accepted": None, "logp": logp}


_EXACT = {"write": _exact_write, "attention": _exact_attention, "verify": _exact_verify}
