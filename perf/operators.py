"""The training objectives over rows of logits, as cases that can be timed.

Three operators, each a loss with its gradient in the logits:

  distill     Kullback-Leibler divergence from a teacher's top logits
  policy      clipped policy loss with a KL term to a reference model
  preference  paired log ratios over ragged chosen / rejected sequences

A row of logits is a query's candidate scores or a token's vocabulary.  With
``own`` false, ``run`` computes the plain form in elementary 32-bit torch
operations; with ``own`` true it calls the library's entry points.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_NEG = float("-inf")


# --------------------------------------------------------------- the cases --

def listed():
    return [
        # a query's 17 candidates (256 queries): the per-query candidate head distilled from a reranker's
        # 16 best; nothing but latency
        dict(name="distill_candidates_f32", op="distill", rows=256, cols=17, k=16, dtype="f32", teacher="f32",
             full=False, masked=0.0, padded=0.1, scale=1.0, grad=True),
        # 128 queries against 4096 documents, distilled from the 64 documents a teacher ranked first
        dict(name="distill_corpus_f32", op="distill", rows=128, cols=4096, k=64, dtype="f32", teacher="f32",
             full=False, masked=0.0, padded=0.1, scale=2.0, grad=True),
        # a training batch of answer tokens over a large vocabulary
        dict(name="distill_vocab_bf16", op="distill", rows=4096, cols=128000, k=64, dtype="bf16", teacher="bf16",
             full=False, masked=0.0, padded=0.0, scale=0.5, grad=True),
        # an odd vocabulary (rows start at any 2-byte address), the teacher's true probabilities, masked rows
        dict(name="distill_odd_f16", op="distill", rows=1021, cols=50001, k=33, dtype="f16", teacher="f16",
             full=True, masked=0.2, padded=0.2, scale=1.0, grad=True),
        # the evaluation loss: forward only
        dict(name="distill_eval_bf16", op="distill", rows=2048, cols=128000, k=128, dtype="bf16", teacher="f32",
             full=True, masked=0.0, padded=0.0, scale=1.0, grad=False),
        # a handful of sampled tokens: few rows, so a row has to spread over the chip
        dict(name="policy_few_bf16", op="policy", rows=16, cols=32000, dtype="bf16", masked=0.0, kl=0.05,
             scale=1.0, grad=True),
        # a rollout batch, its prompt rows masked
        dict(name="policy_rollout_bf16", op="policy", rows=8192, cols=64000, dtype="bf16", masked=0.25, kl=0.02,
             scale=1.0, grad=True),
        # fp32 logits of an odd vocabulary, sampled at a temperature
        dict(name="policy_odd_f32", op="policy", rows=777, cols=100003, dtype="f32", masked=0.1, kl=0.0,
             scale=1.25, grad=True),
        # log-probabilities and loss of fixed rollouts: forward only, odd vocabulary
        dict(name="policy_eval_f16", op="policy", rows=3001, cols=32003, dtype="f16", masked=0.0, kl=0.1,
             scale=1.0, grad=False),
        # two short pairs
        dict(name="preference_few_f16", op="preference", pairs=2, rows=61, cols=32000, dtype="f16", prompt=0.25,
             average=False, smoothing=0.0, margin=0.0, reference=True, scale=1.0, grad=True),
        # eight pairs of long answers over a large vocabulary
        dict(name="preference_long_bf16", op="preference", pairs=8, rows=8192, cols=128000, dtype="bf16",
             prompt=0.25, average=False, smoothing=0.0, margin=0.0, reference=True, scale=1.0, grad=True),
        # length-averaged, without a reference, with a margin and smoothed labels; fp32, odd vocabulary
        dict(name="preference_odd_f32", op="preference", pairs=24, rows=1501, cols=20011, dtype="f32", prompt=0.4,
             average=True, smoothing=0.1, margin=0.5, reference=False, scale=1.0, grad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["distill", "policy", "preference"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    cols = _log_int(rng, 16, 131072)
    most = 1_000_000_000 // (cols * (4 if dtype == "f32" else 2))
    rows = max(1, min(_log_int(rng, 16, 8192), most))
    case = dict(op=op, rows=rows, cols=cols, dtype=dtype, scale=rng.choice([0.5, 1.0, 1.25]),
                grad=rng.random() < 0.8)
    if op == "distill":
        case.update(k=min(cols, _log_int(rng, 4, 256)), teacher=rng.choice([dtype, "f32"]),
                    full=rng.random() < 0.5, masked=rng.choice([0.0, 0.3]), padded=rng.choice([0.0, 0.2]))
    elif op == "policy":
        case.update(masked=rng.choice([0.0, 0.3]), kl=rng.choice([0.0, 0.05]))
    else:
        case.update(pairs=max(1, min(_log_int(rng, 1, 32), rows // 8)), prompt=rng.choice([0.0, 0.3]),
                    average=rng.random() < 0.5, smoothing=rng.choice([0.0, 0.1]), margin=rng.choice([0.0, 0.5]),
                    reference=rng.random() < 0.5)
    return case


# -------------------------------------------------------------- the inputs --

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _chunks(rows, cols):
    step = max(1, 200_000_000 // cols)
    return [(a, min(rows, a + step)) for a in range(0, rows, step)]


def _logits(gen, rows, cols, dtype):
    """Logits as a model gives them: a broad bulk, to which callers add the peaks of likely columns."""
    out = torch.empty(rows, cols, dtype=_DT[dtype], device="cuda")
    for a, b in _chunks(rows, cols):
        out[a:b] = torch.randn(b - a, cols, generator=gen, device="cuda") * 2.0 - 1.0
    return out


def _row_lse(logits, scale):
    parts = [torch.logsumexp(logits[a:b].float() * scale, dim=1) for a, b in _chunks(*logits.shape)]
    return torch.cat(parts)


def _keep(gen, rows, share):
    """A mask of rows that leaves out int(rows * share) of them."""
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[torch.randperm(rows, generator=gen, device="cuda")[:int(rows * share)]] = False
    return keep


def _loss_scale(dtype):
    """fp16 gradients are kept in range by a loss scale, folded into the weights."""
    return 1024.0 if dtype == "f16" else 1.0


def _plant_targets(gen, logits):
    """A sampled column per row, raised to where a model's own samples stand."""
    rows, cols = logits.shape
    target = torch.randint(0, cols, (rows,), generator=gen, device="cuda")
    at = torch.arange(rows, device="cuda")
    bump = 4.0 + 10.0 * torch.rand(rows, generator=gen, device="cuda")
    logits[at, target] = (logits[at, target].float() + bump).to(logits.dtype)
    return target


def prepare(case, seed):
    gen = _generator(seed)
    rows, cols, dtype = case["rows"], case["cols"], case["dtype"]
    logits = _logits(gen, rows, cols, dtype)
    dev = "cuda"
    s = dict(case=dict(case), logits=logits,
             grad=torch.empty_like(logits) if case["grad"] else None,
             loss=torch.empty(1, device=dev),
             row_state=torch.empty(rows, 4, device=dev))
    if case["op"] == "distill":
        k = case["k"]
        # distinct columns per row: a random start, then steps of a fixed stride without wrap-around repeats
        stride = max(1, cols // k)
        start = torch.randint(0, cols, (rows, 1), generator=gen, device=dev)
        index = (start + stride * torch.arange(k, device=dev)) % cols
        # a teacher's ranked logits: a falling ladder with noise; the student has learnt part of it
        teacher = 12.0 - 6.0 * torch.log1p(torch.arange(k, device=dev) * 0.5) + \
            torch.randn(rows, k, generator=gen, device=dev)
        teacher = teacher.sort(dim=1, descending=True).values.to(_DT[case["teacher"]])
        at = torch.arange(rows, device=dev)[:, None]
        learnt = logits[at, index].float() + 0.6 * teacher.float()
        logits[at, index] = learnt.to(logits.dtype)
        lse = None
        if case["full"]:  # the teacher's own normaliser: what is listed carries most of the mass
            lse = torch.logsumexp(teacher.float() * case["scale"], dim=1) + \
                0.2 * torch.rand(rows, generator=gen, device=dev)
        if case["padded"] > 0:
            kept = torch.randint(max(1, int(k * (1 - 2 * case["padded"]))), k + 1, (rows, 1), generator=gen,
                                 device=dev)
            index = torch.where(torch.arange(k, device=dev) < kept, index, torch.full_like(index, -1))
        weight = None
        if case["masked"] > 0 or dtype == "f16":
            keep = _keep(gen, rows, case["masked"])
            weight = keep.float() * (_loss_scale(dtype) / keep.sum())
        s.update(index=index.to(torch.int32).contiguous(), teacher=teacher, lse=lse, weight=weight,
                 row_loss=torch.empty(rows, device=dev))
        return s
    target = _plant_targets(gen, logits)
    lse = _row_lse(logits, case["scale"])
    logp = logits.gather(1, target[:, None])[:, 0].float() * case["scale"] - lse
    if case["op"] == "policy":
        # the policy has moved a little since it sampled, and a little more from its reference
        old = logp + 0.25 * torch.randn(rows, generator=gen, device=dev)
        ref = logp + 0.5 * torch.randn(rows, generator=gen, device=dev) if case["kl"] > 0 else None
        advantage = torch.randn(rows, generator=gen, device=dev)
        weight = None
        if case["masked"] > 0 or dtype == "f16":
            keep = _keep(gen, rows, case["masked"])
            weight = keep.float() * (_loss_scale(dtype) / keep.sum())
        s.update(target=target.to(torch.int32), old=old, ref=ref, advantage=advantage, weight=weight,
                 row_loss=torch.empty(rows, device=dev), row_logp=torch.empty(rows, device=dev))
        return s
    pairs = case["pairs"]
    # ragged sequences that fill the rows; the first tokens of each belong to its prompt (no target)
    cuts = torch.randperm(rows - 1, generator=gen, device=dev)[:2 * pairs - 1].sort().values + 1
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), cuts,
                         torch.full((1,), rows, dtype=torch.long, device=dev)])
    lengths = offsets[1:] - offsets[:-1]
    seq = torch.repeat_interleave(torch.arange(2 * pairs, device=dev), lengths, output_size=rows)
    inside = torch.arange(rows, device=dev) - offsets[seq]
    counted = inside >= (lengths[seq] * case["prompt"]).long()
    target = torch.where(counted, target, torch.full_like(target, -100))
    ref = None
    if case["reference"]:
        ref = torch.zeros(2 * pairs, dtype=torch.float64, device=dev)
        ref.index_add_(0, seq, torch.where(counted, logp, torch.zeros_like(logp)).double())
        if case["average"]:
            n = torch.zeros(2 * pairs, dtype=torch.float64, device=dev).index_add_(0, seq, counted.double())
            ref = ref / n.clamp(min=1.0)
        ref = (ref + 5.0 * torch.randn(2 * pairs, generator=gen, device=dev)).float()
    weight = None
    if dtype == "f16":
        weight = torch.full((pairs,), _loss_scale(dtype) / pairs, device=dev)
    s.update(target=target.to(torch.int32), offsets=offsets.to(torch.int32), ref=ref, weight=weight,
             pair_loss=torch.empty(pairs, device=dev), seq_logp=torch.empty(2 * pairs, device=dev))
    return s


_BETA = 0.1
_CLIP = (0.2, 0.28)


# -------------------------------------------------------------- the passes --

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_distill(s):
    from late_interaction_retrieval_gb300 import binding
    c = s["case"]
    if c["grad"]:
        binding.lik_distill_topk_step(s["logits"], s["index"], s["teacher"], s["loss"], s["row_loss"], s["grad"],
                                      teacher_lse=s["lse"], row_weight=s["weight"], scale=c["scale"])
    else:
        binding.lik_distill_topk_fwd(s["logits"], s["index"], s["teacher"], s["loss"], s["row_loss"],
                                     teacher_lse=s["lse"], row_weight=s["weight"], scale=c["scale"])
    return {"loss": s["loss"], "row_loss": s["row_loss"], "grad": s["grad"]}


def _own_policy(s):
    from late_interaction_retrieval_gb300 import binding
    c = s["case"]
    if c["grad"]:
        binding.lik_policy_loss_step(s["logits"], s["target"], s["old"], s["advantage"], s["loss"], s["row_loss"],
                                     s["row_logp"], s["grad"], ref_logp=s["ref"], row_weight=s["weight"],
                                     clip_low=_CLIP[0], clip_high=_CLIP[1], kl_coef=c["kl"], scale=c["scale"])
    else:
        binding.lik_policy_loss_fwd(s["logits"], s["target"], s["old"], s["advantage"], s["loss"], s["row_loss"],
                                    s["row_logp"], ref_logp=s["ref"], row_weight=s["weight"], clip_low=_CLIP[0],
                                    clip_high=_CLIP[1], kl_coef=c["kl"], scale=c["scale"])
    return {"loss": s["loss"], "row_loss": s["row_loss"], "row_logp": s["row_logp"], "grad": s["grad"]}


def _own_preference(s):
    from late_interaction_retrieval_gb300 import binding
    c = s["case"]
    if c["grad"]:
        binding.lik_preference_loss_step(s["logits"], s["target"], s["offsets"], s["loss"], s["pair_loss"],
                                         s["seq_logp"], s["row_state"], s["grad"], ref_logp=s["ref"],
                                         pair_weight=s["weight"], beta=_BETA, margin=c["margin"],
                                         smoothing=c["smoothing"], average=c["average"], scale=c["scale"])
    else:
        binding.lik_preference_loss_fwd(s["logits"], s["target"], s["offsets"], s["loss"], s["pair_loss"],
                                        s["seq_logp"], s["row_state"], ref_logp=s["ref"], pair_weight=s["weight"],
                                        beta=_BETA, margin=c["margin"], smoothing=c["smoothing"],
                                        average=c["average"], scale=c["scale"])
    return {"loss": s["loss"], "pair_loss": s["pair_loss"], "seq_logp": s["seq_logp"], "grad": s["grad"]}


_OWN = {"distill": _own_distill, "policy": _own_policy, "preference": _own_preference}


def _softmax(z, scale):
    """exp(scale (z - max)), its row sum, and the max; a row of -inf alone gives zeros and sum 1."""
    m = z.amax(dim=1, keepdim=True)
    m = torch.where(m == _NEG, torch.zeros_like(m), m)
    e = torch.exp((z - m) * scale)
    total = e.sum(dim=1, keepdim=True)
    return e, torch.where(total == 0, torch.ones_like(total), total), m


def _plain_distill(s):
    c, index = s["case"], s["index"].long()
    scale = c["scale"]
    z = s["logits"].float()
    rows, cols = z.shape
    e, total, m = _softmax(z, scale)
    inside = (index >= 0) & (index < cols)
    t = torch.where(inside, s["teacher"].float(), torch.full_like(index, 0).float().fill_(_NEG))
    if s["lse"] is None:
        et, tt, mt = _softmax(t, scale)
        p = et / tt
        log_p = (t - mt) * scale - torch.log(tt)
    else:
        log_p = t * scale - s["lse"][:, None]
        p = torch.exp(log_p)
    at = index.clamp(0, cols - 1)
    log_q = (z.gather(1, at) - m) * scale - torch.log(total)
    live = (z.amax(dim=1) > _NEG) & (p.sum(dim=1) > 0)
    if s["weight"] is None:
        w = torch.full((rows,), 1.0 / rows, device=z.device)
    else:
        w = s["weight"]
        live = live & (w != 0)
    p = torch.where(live[:, None] & inside, p, torch.zeros_like(p))
    row_loss = torch.where(p > 0, p * (log_p - log_q), torch.zeros_like(p)).sum(dim=1)
    loss = torch.where(live, w * row_loss, torch.zeros_like(w)).sum().reshape(1)
    grad = None
    if c["grad"]:
        g = e / total * p.sum(dim=1, keepdim=True)
        g.scatter_add_(1, at, -p)
        g = g * (w * scale)[:, None]
        grad = torch.where(live[:, None], g, torch.zeros_like(g)).to(s["logits"].dtype)
    return {"loss": loss, "row_loss": row_loss, "grad": grad}


def _target_logp(z, target, scale):
    """log softmax at the target, the softmax, and which rows count."""
    e, total, m = _softmax(z, scale)
    cols = z.shape[1]
    live = (target >= 0) & (target < cols) & (z.amax(dim=1) > _NEG)
    at = target.clamp(0, cols - 1).long()[:, None]
    lp = ((z.gather(1, at) - m) * scale - torch.log(total))[:, 0]
    return lp, e / total, at, live


def _target_grad(prob, at, coef, live, dtype):
    g = -prob * coef[:, None]
    g.scatter_add_(1, at, coef[:, None])
    return torch.where(live[:, None], g, torch.zeros_like(g)).to(dtype)


def _plain_policy(s):
    c = s["case"]
    scale = c["scale"]
    z = s["logits"].float()
    rows = z.shape[0]
    lp, prob, at, live = _target_logp(z, s["target"], scale)
    if s["weight"] is None:
        w = torch.full((rows,), 1.0 / rows, device=z.device)
    else:
        w = s["weight"]
        live = live & (w != 0)
    adv = s["advantage"]
    rho = torch.exp(lp - s["old"])
    clipped = torch.clamp(rho, 1.0 - _CLIP[0], 1.0 + _CLIP[1])
    row_loss = -torch.minimum(rho * adv, clipped * adv)
    d = torch.where(rho * adv <= clipped * adv, -rho * adv, torch.zeros_like(rho))
    if s["ref"] is not None:
        x = s["ref"] - lp
        row_loss = row_loss + c["kl"] * (torch.exp(x) - x - 1.0)
        d = d + c["kl"] * (1.0 - torch.exp(x))
    zero = torch.zeros_like(lp)
    row_loss = torch.where(live, row_loss, zero)
    loss = torch.where(live, w * row_loss, zero).sum().reshape(1)
    grad = _target_grad(prob, at, w * scale * d, live, s["logits"].dtype) if c["grad"] else None
    return {"loss": loss, "row_loss": row_loss, "row_logp": torch.where(live, lp, zero), "grad": grad}


def _plain_preference(s):
    c = s["case"]
    scale, pairs = c["scale"], c["pairs"]
    z = s["logits"].float()
    rows = z.shape[0]
    lp, prob, at, live = _target_logp(z, s["target"], scale)
    offsets = s["offsets"].long()
    seq = torch.repeat_interleave(torch.arange(2 * pairs, device=z.device), offsets[1:] - offsets[:-1],
                                  output_size=rows)
    counts = (seq[None, :] == torch.arange(2 * pairs, device=z.device)[:, None]) & live[None, :]
    sums = torch.where(counts, lp[None, :], torch.zeros_like(lp)[None, :]).sum(dim=1)
    share = torch.ones(2 * pairs, device=z.device)
    if c["average"]:
        share = 1.0 / counts.sum(dim=1).float().clamp(min=1.0)
        sums = sums * share
    gain = sums if s["ref"] is None else sums - s["ref"]
    x = _BETA * (gain[:pairs] - gain[pairs:]) - c["margin"]
    eps = c["smoothing"]
    tail = torch.log1p(torch.exp(-x.abs()))
    pair_loss = (1.0 - eps) * ((-x).clamp(min=0) + tail) + eps * (x.clamp(min=0) + tail)
    w = torch.full((pairs,), 1.0 / pairs, device=z.device) if s["weight"] is None else s["weight"]
    loss = (w * pair_loss).sum().reshape(1)
    grad = None
    if c["grad"]:
        g = w * _BETA * (1.0 / (1.0 + torch.exp(-x)) - (1.0 - eps))
        coef = (torch.cat([g, -g]) * share)[seq] * scale
        grad = _target_grad(prob, at, coef, live, s["logits"].dtype)
    return {"loss": loss, "pair_loss": pair_loss, "seq_logp": sums, "grad": grad}


_PLAIN = {"distill": _plain_distill, "policy": _plain_policy, "preference": _plain_preference}


# ---------------------------------------------------------------- the work --

def work(case):
    """Logits of the rows that count read once, every row's gradient written once; entries beside them."""
    es = 4 if case["dtype"] == "f32" else 2
    rows, cols = case["rows"], case["cols"]
    out = case.get("masked", case.get("prompt", 0.0))
    counted = rows - int(rows * out)
    elements = counted * cols
    moved = elements * es + rows * 24
    if case["grad"]:
        moved += rows * cols * es
    if case["op"] == "distill":
        moved += counted * case["k"] * (4 + (4 if case["teacher"] == "f32" else 2))
    # subtract, scale, exponential, add; for the gradient the first three again, and a product
    return {"bytes": moved, "flops": elements * (8 if case["grad"] else 4)}


# ---------------------------------------------------- the definition, fp64 --

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, s)


def _double_rows(s, body, out_grad):
    """body(z fp64 rows a..b, a, b) -> fp64 gradient rows, over chunks that fit."""
    rows, cols = s["logits"].shape
    step = max(1, 100_000_000 // cols)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        g = body(s["logits"][a:b].double(), a, b)
        if out_grad is not None:
            out_grad[a:b] = g


def _grad_like(case, s):
    return torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda") if case["grad"] else None


def _exact_distill(case, s):
    rows, cols = s["logits"].shape
    index, scale = s["index"].long(), float(case["scale"])
    weight = torch.full((rows,), 1.0 / rows, dtype=torch.float64, device="cuda")
    if s["weight"] is not None:
        weight = s["weight"].double()
    row_loss = torch.zeros(rows, dtype=torch.float64, device="cuda")
    grad = _grad_like(case, s)

    def body(z, a, b):
        idx = index[a:b]
        pad = (idx < 0) | (idx >= cols)
        t = s["teacher"][a:b].double().masked_fill(pad, _NEG) * scale
        norm = torch.logsumexp(t, 1) if s["lse"] is None else s["lse"][a:b].double()
        p = torch.exp(t - norm[:, None])
        log_q = torch.log_softmax(z * scale, 1)
        on = weight[a:b] != 0
        pick = log_q.gather(1, idx.clamp(0, cols - 1))
        term = torch.special.xlogy(p, p) - p * pick
        row_loss[a:b] = term.masked_fill(pad, 0.0).sum(1) * on
        if grad is None:
            return None
        p = p.masked_fill(pad, 0.0)
        dense = torch.zeros_like(z).scatter_add_(1, idx.clamp(0, cols - 1), p)
        return (weight[a:b] * scale)[:, None] * (p.sum(1, keepdim=True) * log_q.exp() - dense)

    _double_rows(s, body, grad)
    return {"loss": (weight * row_loss).sum().reshape(1), "row_loss": row_loss, "grad": grad}


def _one_hot_minus(log_q, target, coef):
    g = log_q.exp() * -coef[:, None]
    at = target.clamp(0, log_q.shape[1] - 1)[:, None]
    return g.scatter_add(1, at, coef[:, None])


def _exact_logp(case, s):
    rows, cols = s["logits"].shape
    target = s["target"].long()
    lp = torch.zeros(rows, dtype=torch.float64, device="cuda")

    def body(z, a, b):
        pick = torch.log_softmax(z * float(case["scale"]), 1).gather(1, target[a:b].clamp(0, cols - 1)[:, None])
        lp[a:b] = pick[:, 0]

    _double_rows(s, body, None)
    return lp, (target >= 0) & (target < cols), target


def _exact_grad(case, s, target, coef):
    grad = _grad_like(case, s)
    if grad is not None:
        _double_rows(s, lambda z, a, b: _one_hot_minus(torch.log_softmax(z * float(case["scale"]), 1), target[a:b],
                                                       coef[a:b]), grad)
    return grad


def _exact_policy(case, s):
    lp, on, target = _exact_logp(case, s)
    rows = lp.numel()
    weight = torch.full((rows,), 1.0 / rows, dtype=torch.float64, device="cuda")
    if s["weight"] is not None:
        weight = s["weight"].double()
    on = on & (weight != 0)
    ratio = (lp - s["old"].double()).exp()
    adv = s["advantage"].double()
    lo, hi = 1.0 - _CLIP[0], 1.0 + _CLIP[1]
    inner, outer = ratio * adv, ratio.clamp(lo, hi) * adv
    loss = -torch.minimum(inner, outer)
    slope = torch.where(inner <= outer, -inner, torch.zeros_like(inner))
    if s["ref"] is not None:
        gap = s["ref"].double() - lp
        loss = loss + case["kl"] * (torch.expm1(gap) - gap)
        slope = slope - case["kl"] * torch.expm1(gap)
    row_loss = torch.where(on, loss, torch.zeros_like(loss))
    coef = torch.where(on, weight * float(case["scale"]) * slope, torch.zeros_like(slope))
    return {"loss": (weight * row_loss).sum().reshape(1), "row_loss": row_loss,
            "row_logp": torch.where(on, lp, torch.zeros_like(lp)), "grad": _exact_grad(case, s, target, coef)}


def _exact_preference(case, s):
    lp, on, target = _exact_logp(case, s)
    pairs = case["pairs"]
    cuts = s["offsets"].tolist()
    sums, per = [], torch.zeros_like(lp)
    spans = list(zip(cuts[:-1], cuts[1:]))
    for a, b in spans:
        v = lp[a:b][on[a:b]]
        n = max(1, v.numel()) if case["average"] else 1
        sums.append(v.sum() / n)
        per[a:b] = 1.0 / n
    sums = torch.stack(sums)
    ref = torch.zeros_like(sums) if s["ref"] is None else s["ref"].double()
    gain = sums - ref
    x = _BETA * (gain[:pairs] - gain[pairs:]) - case["margin"]
    eps = float(case["smoothing"])
    softplus = torch.nn.functional.softplus
    pair_loss = (1.0 - eps) * softplus(-x, threshold=1000.0) + eps * softplus(x, threshold=1000.0)
    weight = torch.full((pairs,), 1.0 / pairs, dtype=torch.float64, device="cuda")
    if s["weight"] is not None:
        weight = s["weight"].double()
    slope = weight * _BETA * (eps * torch.sigmoid(x) - (1.0 - eps) * torch.sigmoid(-x))
    coef = torch.zeros_like(lp)
    for i, (a, b) in enumerate(spans):
        coef[a:b] = (slope[i] if i < pairs else -slope[i - pairs]) * per[a:b]
    coef = torch.where(on, coef * float(case["scale"]), torch.zeros_like(coef))
    return {"loss": (weight * pair_loss).sum().reshape(1), "pair_loss": pair_loss, "seq_logp": sums,
            "grad": _exact_grad(case, s, target, coef)}


_EXACT = {"distill": _exact_distill, "policy": _exact_policy, "preference": _exact_preference}
