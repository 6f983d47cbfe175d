"""Autograd layers over liblik: MaxSim, MaxSimPairwise, MaxSimKD.

Call shapes follow the Late Interaction Kernels README ("Scoring interface"
table) and, for the per-query candidate layout, the colpali PR "Add support
for late-interaction-kernels (LIK)" (Design section):

  MaxSim          Q [Nq, Lq, dim], D [Nd, Ld, dim]     -> [Nq, Nd]
  MaxSimPairwise  Q [B, Lq, dim],  D [B, Ld, dim]      -> [B]
  MaxSimKD        Q [B, Lq, dim],  D [B, N, Ld, dim]   -> [B, N]

Masks are bool, True = valid, or None.  Scores are fp32.  The forward saves
only the int32 argmax [pairs, Lq] (linear in the number of pairs; no
[pairs, Lq, Ld] similarity grid exists anywhere).  For fp16/bf16 inputs with
dim % 8 == 0 and dim <= 256 the backward asks liblik for gradients in the
input dtype directly (summed in fp32, rounded once); otherwise it asks for
fp32 gradients and casts them.  This module only allocates tensors and calls
the binding.  With recompute=True the forward saves no argmax: the
backward re-runs the forward into a transient workspace.

Training objectives over logits [..., cols] (a query's candidate scores, a
token's vocabulary), each a scalar fp32 loss differentiable once, in the logits:

  distill_topk     divergence from a teacher's top logits
  policy_loss      clipped policy loss with a KL term to a reference
  preference_loss  paired log ratios of chosen and rejected sequences

Their forward saves four floats per row; the backward writes the gradient in
the logits' dtype from the logits and those.
"""
from __future__ import annotations

import torch

from . import binding


def _contig(t):
    return None if t is None else t.contiguous()


def _score_shape(kind, Q, D):
    if kind == "allpairs":
        return (Q.shape[0], D.shape[0])
    if kind == "pairwise":
        return (Q.shape[0],)
    return (Q.shape[0], D.shape[1])


class _MaxSimFn(torch.autograd.Function):
    """MaxSim of layout `kind`.  With `recompute`, the forward keeps only the
    scores (and the inputs it already needs); the backward re-runs the
    forward into a transient argmax workspace (lik_maxsim_*_bwd_recompute)."""

    @staticmethod
    def forward(ctx, kind, recompute, Q, D, qmask, dmask):
        Q, D, qmask, dmask = Q.contiguous(), D.contiguous(), _contig(qmask), _contig(dmask)
        Lq = Q.shape[1]
        shape = _score_shape(kind, Q, D)
        scores = torch.empty(shape, dtype=torch.float32, device=Q.device)
        need = ctx.needs_input_grad[2] or ctx.needs_input_grad[3]
        argmax = (torch.empty((*shape, Lq), dtype=torch.int32, device=Q.device)
                  if need and not recompute else None)
        getattr(binding, f"lik_maxsim_{kind}_fwd")(Q, D, qmask, dmask, scores, argmax)
        ctx.kind, ctx.recompute = kind, recompute
        if recompute:
            ctx.save_for_backward(Q, D, qmask, dmask)
        else:
            ctx.save_for_backward(Q, D, argmax)
        return scores

    @staticmethod
    def backward(ctx, g):
        kind = ctx.kind
        g = g.contiguous().float()
        want_q, want_d = ctx.needs_input_grad[2], ctx.needs_input_grad[3]
        if ctx.recompute:
            Q, D, qmask, dmask = ctx.saved_tensors
            ws = torch.empty((*_score_shape(kind, Q, D), Q.shape[1]), dtype=torch.int32, device=Q.device)
            gQ = torch.empty(Q.shape, dtype=torch.float32, device=Q.device) if want_q else None
            gD = torch.empty(D.shape, dtype=torch.float32, device=D.device) if want_d else None
            getattr(binding, f"lik_maxsim_{kind}_bwd_recompute")(Q, D, qmask, dmask, g, ws, gQ, gD)
        else:
            Q, D, argmax = ctx.saved_tensors
            same = Q.dtype != torch.float32 and Q.shape[-1] % 8 == 0 and Q.shape[-1] <= 256
            gdt = Q.dtype if same else torch.float32
            gQ = torch.empty(Q.shape, dtype=gdt, device=Q.device) if want_q else None
            gD = torch.empty(D.shape, dtype=gdt, device=D.device) if want_d else None
            getattr(binding, f"lik_maxsim_{kind}_bwd" + ("_same_dtype" if same else ""))(Q, D, g, argmax, gQ, gD)
        return (None, None, None if gQ is None else gQ.to(Q.dtype), None if gD is None else gD.to(D.dtype),
                None, None)


def maxsim(Q, D, qmask=None, dmask=None, recompute=False):
    """All-pairs MaxSim scores [Nq, Nd] (fp32), differentiable in Q and D.
    recompute=True keeps no argmax between forward and backward."""
    return _MaxSimFn.apply("allpairs", recompute, Q, D, qmask, dmask)


def maxsim_pairwise(Q, D, qmask=None, dmask=None, recompute=False):
    """Pairwise MaxSim scores [B] (fp32), differentiable in Q and D."""
    return _MaxSimFn.apply("pairwise", recompute, Q, D, qmask, dmask)


def maxsim_kd(Q, D, qmask=None, dmask=None, recompute=False):
    """Per-query candidate MaxSim scores [B, N] (fp32), differentiable in Q and D."""
    return _MaxSimFn.apply("kd", recompute, Q, D, qmask, dmask)


class MaxSim(torch.nn.Module):
    def __init__(self, recompute: bool = False):
        super().__init__()
        self.recompute = recompute

    def forward(self, Q, D, qmask=None, dmask=None):
        return maxsim(Q, D, qmask, dmask, self.recompute)


class MaxSimPairwise(torch.nn.Module):
    def __init__(self, recompute: bool = False):
        super().__init__()
        self.recompute = recompute

    def forward(self, Q, D, qmask=None, dmask=None):
        return maxsim_pairwise(Q, D, qmask, dmask, self.recompute)


class MaxSimKD(torch.nn.Module):
    def __init__(self, recompute: bool = False):
        super().__init__()
        self.recompute = recompute

    def forward(self, Q, D, qmask=None, dmask=None):
        return maxsim_kd(Q, D, qmask, dmask, self.recompute)


# ------------------------------------ training objectives over logits --

def _logit_rows(logits):
    """logits [..., cols] as [rows, cols] with contiguous rows that do not overlap (a view where possible)."""
    rows = logits if logits.dim() == 2 else logits.reshape(-1, logits.shape[-1])
    n, cols = rows.shape
    whole = rows.stride(1) == 1 or cols <= 1
    apart = rows.stride(0) >= cols or n <= 1
    return rows if whole and apart else rows.contiguous()


def _flat(t, dtype):
    return None if t is None else t.detach().reshape(-1).to(dtype).contiguous()


def _int32(t):
    """Columns or offsets as int32.  Values beyond it stay out of range: none wraps into a valid one."""
    if t.dtype == torch.int64:
        t = t.clamp(-1, 2 ** 31 - 1)
    return t.detach().to(torch.int32).contiguous()


def _fp32(like, *shape):
    return torch.empty(shape, dtype=torch.float32, device=like.device)


def _grad_buffer(rows):
    """A gradient with the logits' row stride where that carries no more than
    padding.  Rows of logits that start on a 16-byte boundary are then written
    with 16-byte stores; of logits at another address, or with wider gaps, the
    gradient's rows may lie otherwise and are written by elements."""
    n, cols = rows.shape
    if n > 1 and cols < rows.stride(0) <= cols + cols // 8:
        return torch.empty((n, rows.stride(0)), dtype=rows.dtype, device=rows.device)[:, :cols]
    return torch.empty((n, cols), dtype=rows.dtype, device=rows.device)


def _upstream(g):
    return g.detach().reshape(1).to(torch.float32).contiguous()


class _OnceFn(torch.autograd.Function):
    """A gradient as it is, which depends on its logits and on what is upstream but cannot be differentiated."""

    @staticmethod
    def forward(ctx, grad, z, g):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("the losses over logits have no second derivative")


def _once(grad, z, g):
    return _OnceFn.apply(grad, z, g) if torch.is_grad_enabled() else grad  # enabled: create_graph


class _DistillFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, index, teacher, teacher_lse, weight, scale):
        n, k = z.shape[0], teacher.shape[-1]
        index = _int32(index.reshape(n, k))
        teacher = teacher.detach().reshape(n, k).contiguous()
        teacher_lse, weight = _flat(teacher_lse, torch.float32), _flat(weight, torch.float32)
        loss = _fp32(z, 1)
        row_loss = _fp32(z, n)
        state = _fp32(z, n, 4) if ctx.needs_input_grad[0] else None
        binding.lik_distill_topk_fwd(z, index, teacher, loss, row_loss, state, teacher_lse=teacher_lse,
                                     row_weight=weight, scale=scale)
        ctx.scale = scale
        ctx.save_for_backward(z, index, teacher, teacher_lse, state)
        ctx.mark_non_differentiable(row_loss)
        return loss.view(()), row_loss

    @staticmethod
    def backward(ctx, g, _):
        z, index, teacher, teacher_lse, state = ctx.saved_tensors
        grad = _grad_buffer(z)
        binding.lik_distill_topk_bwd(z, index, teacher, state, grad, grad_loss=_upstream(g), teacher_lse=teacher_lse,
                                     scale=ctx.scale)
        return (_once(grad, z, g),) + (None,) * 5


class _PolicyFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, target, old_logp, advantage, ref_logp, weight, clip_low, clip_high, kl_coef, scale):
        n, f32 = z.shape[0], torch.float32
        target = _int32(target.reshape(-1))
        loss = _fp32(z, 1)
        row_loss, row_logp = _fp32(z, n), _fp32(z, n)
        state = _fp32(z, n, 4) if ctx.needs_input_grad[0] else None
        binding.lik_policy_loss_fwd(z, target, _flat(old_logp, f32), _flat(advantage, f32), loss, row_loss, row_logp,
                                    state, ref_logp=_flat(ref_logp, f32), row_weight=_flat(weight, f32),
                                    clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef, scale=scale)
        ctx.scale = scale
        ctx.save_for_backward(z, target, state)
        ctx.mark_non_differentiable(row_loss, row_logp)
        return loss.view(()), row_loss, row_logp

    @staticmethod
    def backward(ctx, g, *_):
        z, target, state = ctx.saved_tensors
        grad = _grad_buffer(z)
        binding.lik_policy_loss_bwd(z, target, state, grad, grad_loss=_upstream(g), scale=ctx.scale)
        return (_once(grad, z, g),) + (None,) * 9


class _PreferenceFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, target, offsets, ref_logp, weight, beta, margin, smoothing, average, scale):
        n, f32 = z.shape[0], torch.float32
        target, offsets = _int32(target.reshape(-1)), _int32(offsets.reshape(-1))
        pairs = offsets.numel() // 2
        loss = _fp32(z, 1)
        pair_loss, seq_logp = _fp32(z, pairs), _fp32(z, 2 * pairs)
        state = _fp32(z, n, 4)
        binding.lik_preference_loss_fwd(z, target, offsets, loss, pair_loss, seq_logp, state,
                                        ref_logp=_flat(ref_logp, f32), pair_weight=_flat(weight, f32), beta=beta,
                                        margin=margin, smoothing=smoothing, average=average, scale=scale)
        ctx.scale = scale
        ctx.save_for_backward(z, target, state)
        ctx.mark_non_differentiable(pair_loss, seq_logp)
        return loss.view(()), pair_loss, seq_logp

    @staticmethod
    def backward(ctx, g, *_):
        z, target, state = ctx.saved_tensors
        grad = _grad_buffer(z)
        binding.lik_preference_loss_bwd(z, target, state, grad, grad_loss=_upstream(g), scale=ctx.scale)
        return (_once(grad, z, g),) + (None,) * 9


def distill_topk(logits, teacher_index, teacher_logits, teacher_lse=None, row_weight=None, scale=1.0,
                 return_rows=False):
    """Kullback-Leibler divergence of softmax(scale * logits) [..., cols] from a
    teacher known at its top columns (teacher_index, teacher_logits [..., k];
    indices outside [0, cols) are padding), summed with row_weight [...] (None:
    the mean over rows).  teacher_lse [...] makes the teacher's probabilities
    exp(scale * teacher_logits - teacher_lse) instead of normalising them over
    the k entries.  Differentiable in the logits only.  With return_rows also
    the row losses (no gradient)."""
    loss, row_loss = _DistillFn.apply(_logit_rows(logits), teacher_index, teacher_logits, teacher_lse, row_weight,
                                      scale)
    return (loss, row_loss.view(logits.shape[:-1])) if return_rows else loss


def policy_loss(logits, target, old_logp, advantage, ref_logp=None, row_weight=None, clip_low=0.2, clip_high=0.2,
                kl_coef=0.0, scale=1.0, return_rows=False):
    """Clipped policy loss of the sampled tokens target [...] under logits
    [..., cols], with kl_coef times the KL term to ref_logp; summed with
    row_weight (None: the mean over rows).  A target outside [0, cols) leaves
    its token out.  Differentiable in the logits only: advantage, ref_logp and
    row_weight get no gradient.  With return_rows also the token losses and the
    tokens' log-probabilities (no gradient)."""
    loss, row_loss, row_logp = _PolicyFn.apply(_logit_rows(logits), target, old_logp, advantage, ref_logp, row_weight,
                                               clip_low, clip_high, kl_coef, scale)
    shape = logits.shape[:-1]
    return (loss, row_loss.view(shape), row_logp.view(shape)) if return_rows else loss


def preference_loss(logits, target, offsets, ref_logp=None, pair_weight=None, beta=0.1, margin=0.0, smoothing=0.0,
                    average=False, scale=1.0, return_rows=False):
    """Preference loss over pairs of sequences packed along the rows of logits
    [rows, cols]: sequence i holds the rows offsets[i]..offsets[i + 1], pair p
    sets sequence p (chosen) against sequence pairs + p (rejected).
    Differentiable in the logits only.  With return_rows also the pair losses and
    the sequences' log-probabilities (no gradient)."""
    out = _PreferenceFn.apply(_logit_rows(logits), target, offsets, ref_logp, pair_weight, beta, margin, smoothing,
                              average, scale)
    return out if return_rows else out[0]


class DistillTopK(torch.nn.Module):
    def __init__(self, scale: float = 1.0):
        super().__init__()
        self.scale = scale

    def forward(self, logits, teacher_index, teacher_logits, teacher_lse=None, row_weight=None):
        return distill_topk(logits, teacher_index, teacher_logits, teacher_lse, row_weight, self.scale)


class PolicyLoss(torch.nn.Module):
    def __init__(self, clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0, scale: float = 1.0):
        super().__init__()
        self.clip_low, self.clip_high, self.kl_coef, self.scale = clip_low, clip_high, kl_coef, scale

    def forward(self, logits, target, old_logp, advantage, ref_logp=None, row_weight=None):
        return policy_loss(logits, target, old_logp, advantage, ref_logp, row_weight, self.clip_low, self.clip_high,
                           self.kl_coef, self.scale)


class PreferenceLoss(torch.nn.Module):
    def __init__(self, beta: float = 0.1, margin: float = 0.0, smoothing: float = 0.0, average: bool = False,
                 scale: float = 1.0):
        super().__init__()
        self.beta, self.margin, self.smoothing, self.average, self.scale = beta, margin, smoothing, average, scale

    def forward(self, logits, target, offsets, ref_logp=None, pair_weight=None):
        return preference_loss(logits, target, offsets, ref_logp, pair_weight, self.beta, self.margin, self.smoothing,
                               self.average, self.scale)
