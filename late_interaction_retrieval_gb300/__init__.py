"""GB300-native late-interaction MaxSim.

The operator (Late Interaction Kernels README, "What does it compute?"):
score(q, d) = sum over valid query tokens i of max over valid document
tokens j of Q_i . D_j, in three layouts (all-pairs, pairwise, per-query
candidates) with a backward for each; and training objectives over rows of
logits (distillation from a teacher's top logits, a clipped policy loss, a
preference loss), each with its gradient; and a serving step of an answer model
over a cache in 8 bits (``serving``).  All arithmetic runs in the CUDA
library ``liblik`` (C ABI in ``include/lik.h``); this package only builds it,
loads it and marshals torch tensors into its calls.

``workloads`` (seeded synthetic inputs) imports without the CUDA library.
The binding and the autograd layers load it on first use and fail loudly
when it is missing.
"""
import importlib

__all__ = ["binding", "layers", "serving", "workloads", "MaxSim", "MaxSimPairwise", "MaxSimKD",
           "maxsim", "maxsim_pairwise", "maxsim_kd", "DistillTopK", "PolicyLoss", "PreferenceLoss",
           "distill_topk", "policy_loss", "preference_loss", "TokenCache",
           "cache_slots", "cache_write", "cache_attention", "verify_drafts", "LIKError"]

_LAZY = {
    "binding": ("late_interaction_retrieval_gb300.binding", None),
    "layers": ("late_interaction_retrieval_gb300.layers", None),
    "MaxSim": ("late_interaction_retrieval_gb300.layers", "MaxSim"),
    "MaxSimPairwise": ("late_interaction_retrieval_gb300.layers", "MaxSimPairwise"),
    "MaxSimKD": ("late_interaction_retrieval_gb300.layers", "MaxSimKD"),
    "maxsim": ("late_interaction_retrieval_gb300.layers", "maxsim"),
    "maxsim_pairwise": ("late_interaction_retrieval_gb300.layers", "maxsim_pairwise"),
    "maxsim_kd": ("late_interaction_retrieval_gb300.layers", "maxsim_kd"),
    "DistillTopK": ("late_interaction_retrieval_gb300.layers", "DistillTopK"),
    "PolicyLoss": ("late_interaction_retrieval_gb300.layers", "PolicyLoss"),
    "PreferenceLoss": ("late_interaction_retrieval_gb300.layers", "PreferenceLoss"),
    "distill_topk": ("late_interaction_retrieval_gb300.layers", "distill_topk"),
    "policy_loss": ("late_interaction_retrieval_gb300.layers", "policy_loss"),
    "preference_loss": ("late_interaction_retrieval_gb300.layers", "preference_loss"),
    "serving": ("late_interaction_retrieval_gb300.serving", None),
    "TokenCache": ("late_interaction_retrieval_gb300.serving", "TokenCache"),
    "cache_slots": ("late_interaction_retrieval_gb300.serving", "cache_slots"),
    "cache_write": ("late_interaction_retrieval_gb300.serving", "cache_write"),
    "cache_attention": ("late_interaction_retrieval_gb300.serving", "cache_attention"),
    "verify_drafts": ("late_interaction_retrieval_gb300.serving", "verify_drafts"),
    "LIKError": ("late_interaction_retrieval_gb300.binding", "LIKError"),
}


def __getattr__(name):
    if name == "workloads":
        return importlib.import_module("late_interaction_retrieval_gb300.workloads")
    if name not in _LAZY:
        raise AttributeError(name)
    mod, attr = _LAZY[name]
    m = importlib.import_module(mod)
    return m if attr is None else getattr(m, attr)
