"""Argument errors of the training objectives that are found before any CUDA
call, and the fp64 definitions the GPU tests compare with (CPU only)."""
import pytest
import torch

import loss_reference as ref
from late_interaction_retrieval_gb300 import binding
from late_interaction_retrieval_gb300 import build as lik_build

N = None


@pytest.fixture(scope="module")
def lib():
    return binding.load(lik_build.build())


def _distill(lib, dtype=2, rows=4, cols=100, stride=100, tdtype=0, k=8, scale=1.0, g_stride=100):
    return lib.lik_distill_topk_step(N, dtype, rows, cols, stride, N, N, tdtype, k, N, N, scale, N, N, N, g_stride, N)


@pytest.mark.parametrize("bad,status", [(dict(dtype=9), 1), (dict(rows=-1), 1), (dict(cols=0), 1), (dict(cols=-3), 1),
                                        (dict(stride=99), 1), (dict(g_stride=99), 1), (dict(tdtype=-1), 1),
                                        (dict(k=-1), 1), (dict(k=1025), 2), (dict(scale=0.0), 1),
                                        (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
                                        (dict(rows=2 ** 31), 2),
                                        (dict(cols=2 ** 30 + 1, stride=2 ** 30 + 1, g_stride=2 ** 30 + 1), 2),
                                        (dict(stride=2 ** 31 + 1), 2), (dict(rows=2 ** 20, stride=2 ** 31), 2),
                                        (dict(rows=2 ** 20, g_stride=2 ** 31), 2)])
def test_distill_refusals(lib, bad, status):
    assert _distill(lib, **bad) == status
    assert lib.lik_last_error_message()


@pytest.mark.parametrize("bad", [(-0.1, 0.2, 0.0), (1.1, 0.2, 0.0), (0.2, -0.2, 0.0), (0.2, float("inf"), 0.0),
                                 (0.2, 0.2, float("nan"))])
def test_policy_refusals(lib, bad):
    assert lib.lik_policy_loss_step(N, 0, 4, 10, 10, N, N, N, N, N, *bad, 1.0, N, N, N, N, 10, N) == 1


@pytest.mark.parametrize("pairs,beta,margin,smoothing,status", [(-1, 0.1, 0.0, 0.0, 1), (2 ** 20 + 1, 0.1, 0.0, 0.0, 2),
                                                                (1, float("inf"), 0.0, 0.0, 1),
                                                                (1, 0.1, float("nan"), 0.0, 1), (1, 0.1, 0.0, 1.5, 1),
                                                                (1, 0.1, 0.0, -0.5, 1)])
def test_preference_refusals(lib, pairs, beta, margin, smoothing, status):
    assert lib.lik_preference_loss_fwd(N, 0, 4, 10, 10, N, N, pairs, N, N, beta, margin, smoothing, 0, 1.0, N, N, N,
                                       N, N) == status


def test_definitions_agree_with_autograd():
    """The reference's gradients are those of its losses (fp64 autograd of the textbook forms)."""
    gen = torch.Generator().manual_seed(0)
    z = torch.randn(6, 20, generator=gen, dtype=torch.float64, requires_grad=True)
    index = torch.stack([torch.randperm(20, generator=gen)[:5] for _ in range(6)])
    t = torch.randn(6, 5, generator=gen, dtype=torch.float64)
    loss, rows, grad = ref.distill(z, index, t, scale=0.7)
    p = torch.softmax(t * 0.7, 1)
    mine = (p * (torch.log(p) - torch.log_softmax(z * 0.7, 1).gather(1, index))).sum(1).mean()
    (g,) = torch.autograd.grad(mine, z)
    assert abs(float(mine - loss)) < 1e-12 and float((g - grad).abs().max()) < 1e-12

    y = torch.randint(0, 20, (6,), generator=gen)
    old = torch.log_softmax(z.detach(), 1).gather(1, y[:, None])[:, 0] + 0.3 * torch.randn(6, generator=gen)
    adv, other = torch.randn(6, generator=gen).double(), old + 0.2
    lp = torch.log_softmax(z, 1).gather(1, y[:, None])[:, 0]
    ratio = (lp - old).exp()
    mine = (-torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv) + 0.1 * ((other - lp).exp() - (other - lp) - 1)).mean()
    (g,) = torch.autograd.grad(mine, z)
    loss, _, _, grad = ref.policy(z, y, old, adv, other, kl=0.1)
    assert abs(float(mine - loss)) < 1e-12 and float((g - grad).abs().max()) < 1e-12

    cuts = torch.tensor([0, 2, 3, 5, 6])
    lp = torch.log_softmax(z, 1).gather(1, y[:, None])[:, 0]
    s = torch.stack([lp[0:2].mean(), lp[2:3].mean(), lp[3:5].mean(), lp[5:6].mean()])
    x = 0.4 * (s[:2] - s[2:]) - 0.1
    mine = -(0.9 * torch.nn.functional.logsigmoid(x) + 0.1 * torch.nn.functional.logsigmoid(-x)).mean()
    (g,) = torch.autograd.grad(mine, z)
    loss, _, _, grad = ref.preference(z, y, cuts, beta=0.4, margin=0.1, smoothing=0.1, average=True)
    assert abs(float(mine - loss)) < 1e-12 and float((g - grad).abs().max()) < 1e-12
