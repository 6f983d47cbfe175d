"""The training objectives over logits in fp64, from their definitions.

Plain torch, row by row statements over whole tensors, no library code.
Every function returns its outputs as fp64 CPU tensors; ``left_out`` rows have
zero loss and zero gradient whatever they hold.

Bars (fixed from the arithmetic, not from runs).  A gradient element is a sum
of two fp32 products, each within a few 2^-22 of its value relative to the
row's largest, and is rounded to its dtype once: half an ulp is 2^-9 (bf16),
2^-12 (fp16, 2^-25 absolute below its normal range).  The bars allow twice
the rounding plus 1e-5 of the largest element, the library's fp32 bar.
Losses and log-probabilities are fp32: 1e-5 of max(1, largest).
"""
import torch

ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -24}
NEG = float("-inf")


def assert_grad(got, want, dtype, scale=None):
    got, want = got.detach().cpu().double(), want.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "NaN in other places"
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    got, want = got[fine], want[fine]
    if want.numel() == 0:
        return
    top = float(want.abs().max()) if scale is None else scale
    bar = ROUND[dtype] * want.abs() + 1e-5 * top + TINY[dtype]
    worst = float(((got - want).abs() / bar.clamp(min=1e-300)).max())
    assert ((got - want).abs() <= bar).all(), f"gradient is {worst:.2f} times its bar off"


def assert_loss(got, want):
    got, want = torch.as_tensor(got).detach().cpu().double().reshape(-1), want.cpu().double().reshape(-1)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "NaN in other places"
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    if fine.any():
        top = max(1.0, float(want[fine].abs().max()))
        assert float((got[fine] - want[fine]).abs().max()) <= 1e-5 * top


def _log_softmax(z, scale):
    """fp64 log-softmax of scale * z; rows of -inf alone are reported empty."""
    m = z.max(dim=1, keepdim=True).values
    empty = (m == NEG).squeeze(1)
    m = torch.where(m == NEG, torch.zeros_like(m), m)
    y = (z - m) * scale
    return y - torch.log(torch.exp(y).sum(dim=1, keepdim=True)), empty


def distill(logits, index, teacher, lse=None, weight=None, scale=1.0):
    z, t = logits.detach().cpu().double(), teacher.detach().cpu().double()
    index = index.detach().cpu().long()
    rows, cols = z.shape
    w = torch.full((rows,), 1.0 / max(rows, 1), dtype=torch.float64) if weight is None else weight.cpu().double()
    row_loss, grad = torch.zeros(rows, dtype=torch.float64), torch.zeros(rows, cols, dtype=torch.float64)
    for r in range(rows):
        if float(w[r]) == 0.0:
            continue
        on = (index[r] >= 0) & (index[r] < cols) & (t[r] != NEG)
        idx, tr = index[r][on], t[r][on]
        log_q, empty = _log_softmax(z[r:r + 1], scale)
        if bool(empty[0]) or idx.numel() == 0:
            continue
        log_q = log_q[0]
        norm = torch.logsumexp((tr - tr.max()) * scale, 0) + tr.max() * scale if lse is None else lse[r].cpu().double()
        if lse is None:
            log_p = (tr - tr.max()) * scale - torch.log(torch.exp((tr - tr.max()) * scale).sum())
        else:
            log_p = tr * scale - norm
        p = torch.exp(log_p)
        if float(p.sum()) == 0.0:
            continue
        some = p != 0
        row_loss[r] = (p[some] * (log_p[some] - log_q[idx[some]])).sum()
        g = p.sum() * torch.exp(log_q)
        g = g.index_add(0, idx, -p)
        grad[r] = float(w[r]) * scale * g
    loss = torch.where(row_loss == 0, torch.zeros_like(row_loss), w * row_loss).sum()
    return loss, row_loss, grad


def _targets(logits, target, scale):
    z, y = logits.detach().cpu().double(), target.detach().cpu().long()
    cols = z.shape[1]
    log_q, empty = _log_softmax(z, scale)
    on = (y >= 0) & (y < cols) & ~empty
    at = y.clamp(0, cols - 1)[:, None]
    lp = torch.where(on, log_q.gather(1, at)[:, 0], torch.zeros(z.shape[0], dtype=torch.float64))
    return log_q, lp, on, at


def _target_grad(log_q, at, coef, on):
    g = -torch.exp(log_q) * coef[:, None]
    g = g.scatter_add(1, at, coef[:, None])
    return torch.where(on[:, None], g, torch.zeros_like(g))


def policy(logits, target, old, adv, ref=None, weight=None, clip_low=0.2, clip_high=0.2, kl=0.0, scale=1.0):
    log_q, lp, on, at = _targets(logits, target, scale)
    rows = lp.numel()
    w = torch.full((rows,), 1.0 / max(rows, 1), dtype=torch.float64) if weight is None else weight.cpu().double()
    on = on & (w != 0)
    old, adv = old.cpu().double(), adv.cpu().double()
    ratio = torch.exp(lp - old)
    a, b = ratio * adv, ratio.clamp(1.0 - clip_low, 1.0 + clip_high) * adv
    loss = -torch.minimum(a, b)
    d = torch.where(a <= b, -a, torch.where(a > b, torch.zeros_like(a), torch.full_like(a, float("nan"))))
    if ref is not None:
        x = ref.cpu().double() - lp
        loss = loss + kl * (torch.exp(x) - x - 1.0)
        d = d + kl * (1.0 - torch.exp(x))
    zero = torch.zeros_like(lp)
    row_loss, lp = torch.where(on, loss, zero), torch.where(on, lp, zero)
    total = torch.where(row_loss == 0, zero, w * row_loss).sum()
    return total, row_loss, lp, _target_grad(log_q, at, w * scale * d, on)


def preference(logits, target, offsets, ref=None, weight=None, beta=0.1, margin=0.0, smoothing=0.0, average=False,
               scale=1.0):
    log_q, lp, on, at = _targets(logits, target, scale)
    rows, cuts = lp.numel(), offsets.cpu().tolist()
    pairs = len(cuts) // 2
    w = torch.full((pairs,), 1.0 / max(pairs, 1), dtype=torch.float64) if weight is None else weight.cpu().double()
    sums, share = torch.zeros(2 * pairs, dtype=torch.float64), torch.ones(2 * pairs, dtype=torch.float64)
    coef = torch.zeros(rows, dtype=torch.float64)
    for i in range(2 * pairs):
        a, b = cuts[i], cuts[i + 1]
        sums[i] = lp[a:b][on[a:b]].sum()
        n = int(on[a:b].sum())
        if average and n:
            sums[i], share[i] = sums[i] / n, 1.0 / n
    gain = sums if ref is None else sums - ref.cpu().double()
    x = beta * (gain[:pairs] - gain[pairs:]) - margin
    soft = lambda v: torch.logaddexp(torch.zeros_like(v), v)  # noqa: E731
    pair_loss = (1.0 - smoothing) * soft(-x) + smoothing * soft(x)
    slope = w * beta * (smoothing * torch.sigmoid(x) - (1.0 - smoothing) * torch.sigmoid(-x))
    out = w == 0
    pair_loss, slope = pair_loss.masked_fill(out, 0.0), slope.masked_fill(out, 0.0)
    for i in range(2 * pairs):
        coef[cuts[i]:cuts[i + 1]] = (slope[i] if i < pairs else -slope[i - pairs]) * share[i]
    total = torch.where(pair_loss == 0, torch.zeros_like(w), w * pair_loss).sum()
    return total, pair_loss, sums, _target_grad(log_q, at, coef * scale, on)
