"""Training objectives over logits (GPU) against their fp64 definitions
(loss_reference.py, which also derives the bars)."""
import gc

import numpy as np
import pytest
import torch

import loss_reference as ref
from late_interaction_retrieval_gb300 import binding, layers

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NEG, NAN, INF = float("-inf"), float("nan"), float("inf")
# one column, fewer than a warp, odd sizes around a vector, a chunk, a tile of
# every kernel, an odd vocabulary, a large one
SIZES = [(1, 1), (3, 2), (5, 17), (9, 128), (4, 1000), (3, 1025), (2, 4096), (7, 8191), (3, 32003), (2, 50001),
         (2, 131072), (300, 33), (1, 70000), (40, 2050)]


@pytest.fixture(scope="module", autouse=True)
def _leave_no_garbage():
    """No device memory of these tests is left to be freed inside another."""
    yield
    gc.collect()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _weights(gen, rows, dtype):
    w = torch.rand(rows, generator=gen) + 0.25
    if rows > 2:
        w[1] = 0.0
    return w * (256.0 if dtype == "f16" else 1.0)


def _logits(gen, rows, cols, dtype):
    return (torch.randn(rows, cols, generator=gen) * 2.5).to(DT[dtype])


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _out(*shape, dtype=torch.float32):
    return torch.full(shape, NAN, dtype=dtype, device="cuda")


# ------------------------------------------------------------------ runners --

def run_distill(z, index, teacher, lse=None, weight=None, scale=1.0, up=None, inplace=False, grad=None):
    """All three forms: (loss, row_loss, grad of the step, grad of fwd + bwd)."""
    z, index, teacher, lse, weight = _cuda(z, index, teacher, lse, weight)
    rows = z.shape[0]
    loss, row_loss, state = _out(1), _out(rows), _out(rows, 4)
    kw = dict(teacher_lse=lse, scale=scale)
    binding.lik_distill_topk_fwd(z, index, teacher, loss, row_loss, state, row_weight=weight, **kw)
    g2 = torch.full_like(z, NAN)
    binding.lik_distill_topk_bwd(z, index, teacher, state, g2, grad_loss=None if up is None else up.cuda(), **kw)
    loss2, row_loss2 = _out(1), _out(rows)
    binding.lik_distill_topk_fwd(z, index, teacher, loss2, row_loss2, row_weight=weight, **kw)
    assert torch.equal(loss.view(torch.int32), loss2.view(torch.int32)), "the loss depends on the saved state"
    g = z if inplace else grad if grad is not None else torch.full_like(z, NAN)
    loss3, row_loss3 = _out(1), _out(rows)
    binding.lik_distill_topk_step(z, index, teacher, loss3, row_loss3, g, row_weight=weight, **kw)
    binding.lik_check_device_error()
    return [(loss, row_loss), (loss3, row_loss3)], g, g2


def check_distill(z, index, teacher, lse=None, weight=None, scale=1.0, **kw):
    want = ref.distill(z, index, teacher, lse, weight, scale)
    up = torch.tensor([1.75])
    forms, g, g2 = run_distill(z, index, teacher, lse, weight, scale, up=up, **kw)
    for loss, row_loss in forms:
        ref.assert_loss(loss, want[0])
        ref.assert_loss(row_loss, want[1])
    ref.assert_grad(g, want[2], z.dtype)
    ref.assert_grad(g2, want[2] * 1.75, z.dtype)
    return want


def run_policy(z, target, old, adv, refp=None, weight=None, up=None, inplace=False, **kw):
    z, target, old, adv, refp, weight = _cuda(z, target, old, adv, refp, weight)
    rows = z.shape[0]
    kw = dict(kw, ref_logp=refp, row_weight=weight)
    a = (_out(1), _out(rows), _out(rows))
    state, g2 = _out(rows, 4), torch.full_like(z, NAN)
    binding.lik_policy_loss_fwd(z, target, old, adv, *a, state, **kw)
    binding.lik_policy_loss_bwd(z, target, state, g2, grad_loss=None if up is None else up.cuda(),
                                scale=kw.get("scale", 1.0))
    b = (_out(1), _out(rows), _out(rows))
    binding.lik_policy_loss_fwd(z, target, old, adv, *b, **kw)
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.int32), y.view(torch.int32)), "outputs depend on the saved state"
    g = z if inplace else torch.full_like(z, NAN)
    c = (_out(1), _out(rows), _out(rows))
    binding.lik_policy_loss_step(z, target, old, adv, *c, g, **kw)
    binding.lik_check_device_error()
    return [a, c], g, g2


def check_policy(z, target, old, adv, refp=None, weight=None, clip=(0.2, 0.2), kl=0.0, scale=1.0, **kw):
    want = ref.policy(z, target, old, adv, refp, weight, clip[0], clip[1], kl, scale)
    up = torch.tensor([-0.5])
    forms, g, g2 = run_policy(z, target, old, adv, refp, weight, up=up, clip_low=clip[0], clip_high=clip[1],
                              kl_coef=kl, scale=scale, **kw)
    for form in forms:
        for got, w in zip(form, want):
            ref.assert_loss(got, w)
    ref.assert_grad(g, want[3], z.dtype)
    ref.assert_grad(g2, want[3] * -0.5, z.dtype)
    return want


def run_preference(z, target, offsets, refp=None, weight=None, up=None, inplace=False, **kw):
    z, target, offsets, refp, weight = _cuda(z, target, offsets, refp, weight)
    rows, pairs = z.shape[0], offsets.numel() // 2
    kw = dict(kw, ref_logp=refp, pair_weight=weight)
    a = (_out(1), _out(pairs), _out(2 * pairs))
    state, g2 = _out(rows, 4), torch.full_like(z, NAN)
    binding.lik_preference_loss_fwd(z, target, offsets, *a, state, **kw)
    binding.lik_preference_loss_bwd(z, target, state, g2, grad_loss=None if up is None else up.cuda(),
                                    scale=kw.get("scale", 1.0))
    g = z if inplace else torch.full_like(z, NAN)
    c = (_out(1), _out(pairs), _out(2 * pairs))
    binding.lik_preference_loss_step(z, target, offsets, *c, _out(rows, 4), g, **kw)
    binding.lik_check_device_error()
    return [a, c], g, g2


def check_preference(z, target, offsets, refp=None, weight=None, scale=1.0, inplace=False, **kw):
    want = ref.preference(z, target, offsets, refp, weight, scale=scale, **kw)
    up = torch.tensor([3.0])
    forms, g, g2 = run_preference(z, target, offsets, refp, weight, up=up, scale=scale, inplace=inplace, **kw)
    for form in forms:
        for got, w in zip(form, want):
            ref.assert_loss(got, w)
    ref.assert_grad(g, want[3], z.dtype)
    ref.assert_grad(g2, want[3] * 3.0, z.dtype)
    return want


# -------------------------------------------------------------------- inputs --

def distill_inputs(rows, cols, dtype, k, seed, teacher="f32", padded=True, full=False, weighted=True, scale=1.0):
    gen = _gen(seed)
    z = _logits(gen, rows, cols, dtype)
    k = min(k, cols)
    index = torch.stack([torch.randperm(cols, generator=gen)[:k] for _ in range(rows)]).to(torch.int32)
    t = (torch.randn(rows, k, generator=gen) * 2.0).to(DT[teacher])
    lse = torch.logsumexp(t.float() * scale, 1) + torch.rand(rows, generator=gen) if full else None
    if padded and k > 2:
        index[torch.rand(rows, k, generator=gen) < 0.2] = -1
        index[0, 1] = cols  # also padding
    return z, index, t, lse, _weights(gen, rows, dtype) if weighted else None


def policy_inputs(rows, cols, dtype, seed, weighted=True, kl=True, scale=1.0):
    gen = _gen(seed)
    z = _logits(gen, rows, cols, dtype)
    target = torch.randint(0, cols, (rows,), generator=gen)
    lp = torch.log_softmax(z.double() * scale, 1).gather(1, target[:, None])[:, 0].float()
    old = lp + 0.3 * torch.randn(rows, generator=gen)
    refp = lp + 0.5 * torch.randn(rows, generator=gen) if kl else None
    adv = torch.randn(rows, generator=gen)
    target = target.to(torch.int32)
    if rows > 3:
        target[2], target[3] = -100, cols
    return z, target, old, adv, refp, _weights(gen, rows, dtype) if weighted else None


def preference_inputs(rows, cols, dtype, pairs, seed, reference=True):
    gen = _gen(seed)
    z = _logits(gen, rows, cols, dtype)
    target = torch.randint(0, cols, (rows,), generator=gen).to(torch.int32)
    target[torch.rand(rows, generator=gen) < 0.2] = -100
    cuts = torch.randint(0, rows + 1, (2 * pairs + 1,), generator=gen).sort().values.to(torch.int32)
    refp = torch.randn(2 * pairs, generator=gen) * 3 - 10 if reference else None
    w = (torch.rand(pairs, generator=gen) + 0.5) * (256.0 if dtype == "f16" else 1.0)
    return z, target, cuts, refp, w


# --------------------------------------------------------------- sizes, types --

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_distill_sizes(rows, cols, dtype):
    full = rows % 2 == 1
    z, i, t, lse, w = distill_inputs(rows, cols, dtype, 24, rows * 100 + cols, teacher=dtype if rows % 3 else "f32",
                                     full=full, scale=0.75)
    check_distill(z, i, t, lse, w, scale=0.75)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_policy_sizes(rows, cols, dtype):
    z, y, old, adv, refp, w = policy_inputs(rows, cols, dtype, rows * 100 + cols, kl=rows % 2 == 1, scale=1.25)
    check_policy(z, y, old, adv, refp, w, clip=(0.2, 0.28), kl=0.07, scale=1.25)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_preference_sizes(rows, cols, dtype):
    pairs = max(1, min(5, rows // 2))
    z, y, cuts, refp, w = preference_inputs(rows, cols, dtype, pairs, rows * 100 + cols, reference=rows % 2 == 1)
    check_preference(z, y, cuts, refp, w, average=rows % 3 == 0, smoothing=0.1 * (rows % 2), margin=0.25)


@pytest.mark.parametrize("teacher", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("k", [0, 1, 31, 257, 1024])
def test_distill_teacher_sizes_and_types(k, teacher):
    z, i, t, lse, w = distill_inputs(6, 5000, "bf16", k, 11 + k, teacher=teacher, full=k == 31)
    if k == 0:
        i, t = i[:, :0].contiguous(), t[:, :0].contiguous()
    check_distill(z, i, t, lse, w)
    check_distill(z, i, t, lse, None)


def test_more_rows_than_one_wave():
    """Rows enough that every block takes several."""
    z, i, t, lse, w = distill_inputs(5000, 70, "bf16", 8, 3)
    check_distill(z, i, t, lse, w)
    z, y, old, adv, refp, w = policy_inputs(2600, 1300, "f16", 4)
    check_policy(z, y, old, adv, refp, w, kl=0.1)


# -------------------------------------------------------------------- layouts --

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols,stride,offset", [(1000, 1024, 0), (1001, 1007, 3), (37, 61, 5), (33000, 33003, 1),
                                                (33000, 33280, 8)])
def test_strided_rows(cols, stride, offset, dtype):
    """Rows at any element address and stride; the gaps of the gradient stay as they were."""
    rows = 5
    z, y, old, adv, refp, w = policy_inputs(rows, cols, dtype, cols + stride)
    want = ref.policy(z, y, old, adv, refp, w, kl=0.1)
    buf = torch.full((offset + rows * stride + 9,), 777.0, dtype=DT[dtype], device="cuda")
    zv = buf[offset:offset + rows * stride].view(rows, stride)[:, :cols]
    zv.copy_(z)
    for g_stride, g_offset in ((cols, 0), (stride, offset), (stride + 1, 7)):
        gbuf = torch.full((g_offset + rows * g_stride + 9,), 555.0, dtype=DT[dtype], device="cuda")
        gv = gbuf[g_offset:g_offset + rows * g_stride].view(rows, g_stride)[:, :cols]
        out = (_out(1), _out(rows), _out(rows))
        binding.lik_policy_loss_step(zv, *_cuda(y, old, adv), *out, gv, ref_logp=refp.cuda(), row_weight=w.cuda(),
                                     kl_coef=0.1)
        ref.assert_grad(gv, want[3], DT[dtype])
        ref.assert_loss(out[1], want[1])
        mark = torch.ones_like(gbuf, dtype=torch.bool)
        mark[g_offset:g_offset + rows * g_stride].view(rows, g_stride)[:, :cols] = False
        assert (gbuf[mark] == 555.0).all(), "wrote outside the rows"
        dz, di, dt, dlse, dw = distill_inputs(rows, cols, dtype, 16, 5)
        dwant = ref.distill(z, di, dt, dlse, dw)
        gbuf.fill_(555.0)
        binding.lik_distill_topk_step(zv, di.cuda(), dt.cuda(), _out(1), _out(rows), gv, row_weight=dw.cuda())
        ref.assert_grad(gv, dwant[2], DT[dtype])
        assert (gbuf[mark] == 555.0).all(), "wrote outside the rows"
    assert (buf[offset:offset + rows * stride].view(rows, stride)[:, cols:] == 777.0).all()


@pytest.mark.parametrize("rows,cols,dtype", [(5, 77, "bf16"), (6, 3001, "f32"), (4, 40001, "f16"), (3, 131072, "bf16")])
def test_gradient_in_place_of_the_logits(rows, cols, dtype):
    z, i, t, lse, w = distill_inputs(rows, cols, dtype, 20, 21)
    check_distill(z, i, t, lse, w, inplace=True)
    z, y, old, adv, refp, w = policy_inputs(rows, cols, dtype, 22)
    check_policy(z, y, old, adv, refp, w, kl=0.1, inplace=True)
    z, y, cuts, refp, w = preference_inputs(rows, cols, dtype, 2, 23)
    check_preference(z, y, cuts, refp, w, inplace=True)


# --------------------------------------------------------- values and masks --

LOWEST = {"f32": torch.finfo(torch.float32).min, "f16": torch.finfo(torch.float16).min,
          "bf16": torch.finfo(torch.bfloat16).min}


def _awkward(cols, dtype):
    """Rows: plain, half masked by -inf, half by the type's lowest value, one live column, all lowest, all -inf,
    NaN, one +inf, large offsets, equal values."""
    gen = _gen(cols)
    z = _logits(gen, 10, cols, dtype).float()
    half = cols // 2
    z[1, half:] = NEG
    z[2, half:] = LOWEST[dtype]
    z[3, 1:] = NEG
    z[4] = LOWEST[dtype]
    z[5] = NEG
    z[6, cols - 1] = NAN
    z[7, cols // 3] = INF
    z[8] += 3e4
    z[9] = 1.5
    return z.to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [40, 1500, 20001])
def test_masked_columns_and_awkward_values(cols, dtype):
    z = _awkward(cols, dtype)
    live = [0, 1, 2, 3, 4, 5, 8, 9]
    target = torch.zeros(10, dtype=torch.int32)
    old, adv = torch.full((10,), -3.0), torch.linspace(-1, 1, 10)
    index = torch.arange(4, dtype=torch.int32).repeat(10, 1)
    index[3, 1:] = -1  # its only unmasked column
    t = torch.randn(10, 4, generator=_gen(1))
    w = torch.ones(10)
    # without the NaN rows: exact comparisons
    sel = torch.tensor(live)
    check_policy(z[sel], target[sel], old[sel], adv[sel], None, w[sel], scale=2.0)
    check_distill(z[sel], index[sel], t[sel], None, w[sel], scale=2.0)
    cuts = torch.tensor([0, 2, 4, 6, 8], dtype=torch.int32)
    check_preference(z[sel], target[sel], cuts, None, torch.ones(2), average=True)
    # a NaN or +inf logit makes its own row NaN, and no other
    forms, g, g2 = run_policy(z, target, old, adv, None, w)
    for f in forms:
        assert torch.isnan(f[1][6:8]).all() and torch.isfinite(f[1][live]).all() and torch.isnan(f[0])
    for x in (g, g2):
        assert torch.isnan(x[6:8]).all() and torch.isfinite(x[live].float()).all()
    forms, g, g2 = run_distill(z, index, t, None, w)
    for f in forms:
        assert torch.isnan(f[1][6:8]).all() and torch.isfinite(f[1][live]).all()
    for x in (g, g2):
        assert torch.isnan(x[6:8]).all() and torch.isfinite(x[live].float()).all()
    # and left out, by weight or by target, it gives zeros
    w[6:8] = 0.0
    old[6:8], adv[6:8] = NAN, INF
    forms, g, g2 = run_policy(z, target, old, adv, old, w)
    for f in forms:
        assert (f[1][6:8] == 0).all() and (f[2][6:8] == 0).all() and torch.isfinite(f[0])
    assert (g[6:8] == 0).all() and (g2[6:8] == 0).all()
    forms, g, g2 = run_distill(z, index, t, None, w)
    assert all((f[1][6:8] == 0).all() and torch.isfinite(f[0]) for f in forms)
    assert (g[6:8] == 0).all() and (g2[6:8] == 0).all()
    target[6:8] = -1
    forms, g, g2 = run_preference(z, target, torch.tensor([0, 5, 10], dtype=torch.int32))
    assert all(torch.isfinite(f[0]) and torch.isfinite(f[2]).all() for f in forms)
    assert (g[6:8] == 0).all() and (g2[6:8] == 0).all()


@pytest.mark.parametrize("cols", [50, 9000])
def test_distill_teacher_corners(cols):
    gen = _gen(cols)
    z = _logits(gen, 8, cols, "f32")
    index = torch.stack([torch.randperm(cols, generator=gen)[:12] for _ in range(8)]).to(torch.int32)
    t = torch.randn(8, 12, generator=gen)
    index[0] = -1  # no teacher: left out
    t[1] = NEG  # no mass: left out
    t[2, 3:] = NEG
    index[3, :] = index[3, 0]  # one column twelve times
    index[4, 5] = index[4, 2]  # a column twice
    index[5, 0], index[5, 1] = 2 ** 31 - 1, -2 ** 31
    t[6] = torch.finfo(torch.float32).min  # equal lowest values: uniform
    want = check_distill(z, index, t)
    assert (want[1][:2] == 0).all()
    check_distill(z, index, t, lse=torch.logsumexp(t.double(), 1).clamp(min=-50).float() + 0.5)
    # the teacher asks for a masked column: infinite loss, finite gradient
    z[7, index[7, 0].long()] = NEG
    want = check_distill(z, index, t)
    assert torch.isinf(want[1][7])


def test_policy_clipping_sides():
    """Both signs of the advantage on both sides of the clip range, at its edges, and without a gradient."""
    z = torch.zeros(8, 30)
    y = torch.arange(8, dtype=torch.int32)
    lp = -float(np.log(30.0))
    shift = torch.tensor([0.5, 0.5, -0.5, -0.5, 0.0, 0.0, 0.1, -0.1])
    adv = torch.tensor([1.0, -1.0, 1.0, -1.0, 1.0, -1.0, 0.0, 2.0])
    want = check_policy(z, y, lp - shift, adv, None, None)
    zero = (want[3].abs().sum(1) == 0)
    assert zero.tolist() == [True, False, False, True, False, False, True, False]


def test_preference_sequences():
    """Empty sequences, sequences without a counted token, rows outside every sequence, a pair of weight 0,
    saturated pairs."""
    z, y, _, _, _ = preference_inputs(30, 700, "bf16", 3, 8)
    y[10:14] = -100
    cuts = torch.tensor([2, 7, 7, 10, 14, 20, 28], dtype=torch.int32)
    for average in (False, True):
        check_preference(z, y, cuts, None, torch.tensor([1.0, 0.0, 2.0]), average=average, margin=-0.5)
        check_preference(z, y, cuts, torch.tensor([900.0, 0, 0, 0, -900.0, 5.0]), None, average=average, beta=2.0)
    check_preference(z, y, torch.zeros(3, dtype=torch.int32), None, None)
    w = check_preference(z, y, torch.tensor([0], dtype=torch.int32), None, None)
    assert float(w[0]) == 0.0


def test_preference_offsets_out_of_range_are_clamped():
    z, y, _, _, _ = preference_inputs(12, 64, "f32", 1, 9)
    a, _, _ = run_preference(z, y, torch.tensor([-5, 6, 99], dtype=torch.int32))
    b, _, _ = run_preference(z, y, torch.tensor([0, 6, 12], dtype=torch.int32))
    assert torch.equal(a[0][2], b[0][2])


def test_no_rows():
    for dtype in (torch.float32, torch.bfloat16):
        z = torch.empty(0, 50, dtype=dtype)
        forms, _, _ = run_distill(z, torch.empty(0, 4, dtype=torch.int32), torch.empty(0, 4))
        assert all(f[0].item() == 0.0 for f in forms)
        e = torch.empty(0)
        forms, _, _ = run_policy(z, torch.empty(0, dtype=torch.int32), e, e)
        assert all(f[0].item() == 0.0 for f in forms)
        forms, _, _ = run_preference(z, torch.empty(0, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
        assert all(abs(f[0].item() - np.log(2.0)) < 1e-6 for f in forms)


# --------------------------------------------- what only large calls come to --

@pytest.mark.parametrize("rows,cols,dtype", [(3000, 2500, "bf16"), (700, 21000, "f16"), (1300, 5003, "f32")])
def test_many_masked_rows(rows, cols, dtype):
    """Left-out rows lie in runs and alone."""
    gen = _gen(rows)
    off = (torch.arange(rows) // 37 % 3 == 1) | (torch.rand(rows, generator=gen) < 0.3)
    z, y, old, adv, refp, w = policy_inputs(rows, cols, dtype, 101)
    w[off] = 0.0
    check_policy(z, y, old, adv, refp, w, kl=0.1)
    z, i, t, lse, w = distill_inputs(rows, cols, dtype, 40, 102)
    w[off] = 0.0
    t[::29] = NEG
    check_distill(z, i, t, lse, w)
    z, y, cuts, refp, w = preference_inputs(rows, cols, dtype, 9, 103)
    y[off] = -100
    check_preference(z, y, cuts, refp, w)


def test_thousands_of_left_out_rows():
    """Many short-lived blocks, half of them over rows that are left out."""
    rows, cols = 16500, 2100
    z, y, old, adv, refp, w = policy_inputs(rows, cols, "bf16", 111)
    w[torch.rand(rows, generator=_gen(1)) < 0.5] = 0.0
    check_policy(z, y, old, adv, refp, w, kl=0.1)


@pytest.mark.parametrize("inplace", [False, True])
def test_rows_longer_than_the_chip_holds(inplace):
    """800 KB a row: many batches a thread, from the largest blocks."""
    rows, cols = 9, 200003
    z, i, t, lse, w = distill_inputs(rows, cols, "f32", 50, 121, full=True)
    check_distill(z, i, t, lse, w, inplace=inplace)
    z, y, old, adv, refp, w = policy_inputs(rows, cols, "f32", 122)
    check_policy(z, y, old, adv, refp, w, kl=0.1, inplace=inplace)


@pytest.mark.parametrize("rows,cols,dtype", [(3000, 2501, "bf16"), (900, 20001, "bf16"), (700, 9003, "f32")])
def test_gradient_rows_at_other_alignments(rows, cols, dtype):
    """Logits on 16-byte boundaries, gradient rows on any."""
    pad = (-cols) % 8
    z, y, old, adv, refp, w = policy_inputs(rows, cols, dtype, 131)
    w[torch.rand(rows, generator=_gen(2)) < 0.4] = 0.0
    want = ref.policy(z, y, old, adv, refp, w, kl=0.1)
    zv = torch.zeros(rows, cols + pad, dtype=DT[dtype], device="cuda")[:, :cols]
    zv.copy_(z)
    y, old, adv, refp, w = _cuda(y, old, adv, refp, w)
    state = _out(rows, 4)
    binding.lik_policy_loss_fwd(zv, y, old, adv, _out(1), _out(rows), _out(rows), state, ref_logp=refp, row_weight=w,
                                kl_coef=0.1)
    g, g2 = (torch.full((rows, cols), NAN, dtype=DT[dtype], device="cuda") for _ in range(2))
    binding.lik_policy_loss_bwd(zv, y, state, g, scale=1.0)
    binding.lik_policy_loss_step(zv, y, old, adv, _out(1), _out(rows), _out(rows), g2, ref_logp=refp, row_weight=w,
                                 kl_coef=0.1)
    binding.lik_check_device_error()
    ref.assert_grad(g, want[3], DT[dtype])
    ref.assert_grad(g2, want[3], DT[dtype])
    z, i, t, lse, w = distill_inputs(rows, cols, dtype, 40, 132)
    want = ref.distill(z, i, t, lse, w)
    zv.copy_(z)
    i, t, w = _cuda(i, t, w)
    binding.lik_distill_topk_fwd(zv, i, t, _out(1), _out(rows), state, row_weight=w)
    binding.lik_distill_topk_bwd(zv, i, t, state, g)
    binding.lik_distill_topk_step(zv, i, t, _out(1), _out(rows), g2, row_weight=w)
    binding.lik_check_device_error()
    ref.assert_grad(g, want[2], DT[dtype])
    ref.assert_grad(g2, want[2], DT[dtype])


@pytest.mark.parametrize("cols,dtype", [(4500, "f32"), (40000, "bf16"), (131072, "f32")])
def test_many_teacher_entries_over_long_rows(cols, dtype):
    z, i, t, lse, w = distill_inputs(170, cols, dtype, 1024, 141, teacher="bf16")
    check_distill(z, i, t, lse, w)


# ---------------------------------------------------------------- gradients --

@pytest.mark.parametrize("op", ["distill", "policy", "preference"])
@pytest.mark.parametrize("rows,cols", [(6, 40), (5, 3001)])
def test_gradient_against_differences(op, rows, cols):
    """(L(z + h v) - L(z - h v)) / 2h of the fp64 definition along random
    directions v against <grad, v>: the truncation is O(h^2) of a smooth loss
    (h = 1e-4, third derivatives below about 10), the fp32 gradient's own bar
    1e-5 of its norm."""
    gen = _gen(cols)
    if op == "distill":
        z, i, t, lse, w = distill_inputs(rows, cols, "f32", 10, 31)
        f = lambda x: ref.distill(x, i, t, lse, w)[0]  # noqa: E731
        _, g, _ = run_distill(z, i, t, lse, w)
    elif op == "policy":
        z, y, old, adv, refp, w = policy_inputs(rows, cols, "f32", 32)
        # keep ratios off the kinks of the clip
        old = old + 0.05 * torch.sign(old - old.mean())
        f = lambda x: ref.policy(x, y, old, adv, refp, w, kl=0.2)[0]  # noqa: E731
        _, g, _ = run_policy(z, y, old, adv, refp, w, kl_coef=0.2)
    else:
        z, y, cuts, refp, w = preference_inputs(rows, cols, "f32", 2, 33)
        f = lambda x: ref.preference(x, y, cuts, refp, w, smoothing=0.1)[0]  # noqa: E731
        _, g, _ = run_preference(z, y, cuts, refp, w, smoothing=0.1)
    g = g.cpu().double()
    for _ in range(4):
        v = torch.randn(rows, cols, generator=gen, dtype=torch.float64)
        h = 1e-4
        diff = float(f(z.double() + h * v) - f(z.double() - h * v)) / (2 * h)
        assert abs(diff - float((g * v).sum())) <= 1e-5 * float(g.norm() * v.norm()) + 1e-6


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layers_backward(dtype):
    """The autograd layers over [..., cols] logits give the step's gradient, scaled by what is upstream."""
    z, i, t, lse, w = distill_inputs(12, 900, dtype, 16, 41, full=True)
    leaf = z.cuda().view(3, 4, 900).requires_grad_()
    loss, rows = layers.distill_topk(leaf, i.cuda().long().view(3, 4, 16), t.cuda().view(3, 4, 16),
                                     lse.cuda().view(3, 4), w.cuda().view(3, 4), return_rows=True)
    (loss * 2.0).backward()
    want = ref.distill(z, i, t, lse, w)
    ref.assert_loss(loss, want[0])
    assert rows.shape == (3, 4) and not rows.requires_grad
    ref.assert_grad(leaf.grad.view(12, 900), want[2] * 2.0, DT[dtype])

    z, y, old, adv, refp, w = policy_inputs(12, 901, dtype, 42)
    leaf = z.cuda().view(3, 4, 901).requires_grad_()
    mod = layers.PolicyLoss(0.2, 0.3, 0.1)
    mod(leaf, y.cuda().long().view(3, 4), old.cuda().view(3, 4), adv.cuda().view(3, 4), refp.cuda().view(3, 4),
        w.cuda().view(3, 4)).backward()
    want = ref.policy(z, y, old, adv, refp, w, 0.2, 0.3, 0.1)
    ref.assert_grad(leaf.grad.view(12, 901), want[3], DT[dtype])

    z, y, cuts, refp, w = preference_inputs(12, 902, dtype, 2, 43)
    wide = torch.zeros(12, 928, dtype=DT[dtype], device="cuda")
    wide[:, :902] = z.cuda()
    leaf = wide.requires_grad_()
    loss, pair, seq = layers.preference_loss(leaf[:, :902], y.cuda(), cuts.cuda(), refp.cuda(), w.cuda(),
                                             smoothing=0.1, return_rows=True)
    loss.backward()
    want = ref.preference(z, y, cuts, refp, w, smoothing=0.1)
    ref.assert_loss(seq, want[2])
    ref.assert_grad(leaf.grad[:, :902], want[3], DT[dtype])
    assert (leaf.grad[:, 902:] == 0).all()
    with torch.no_grad():
        assert not layers.DistillTopK()(z.cuda(), *(x.cuda() for x in distill_inputs(12, 902, dtype, 5, 1)[1:3])
                                        ).requires_grad


def test_layers_padding_beyond_int32():
    """int64 columns and targets that do not fit in 32 bits are padding, whatever their low bits say."""
    z, i, t, lse, w = distill_inputs(6, 300, "f32", 8, 91, padded=False)
    wide = i.long()
    wide[:, 3], wide[:, 5], wide[1, 0] = -2 ** 63, 2 ** 32 + 7, 2 ** 63 - 1
    i[:, 3], i[:, 5], i[1, 0] = -1, -1, -1
    loss = layers.distill_topk(z.cuda(), wide.cuda(), t.cuda(), None, w.cuda())
    ref.assert_loss(loss, ref.distill(z, i, t, None, w)[0])
    z, y, old, adv, refp, w = policy_inputs(6, 300, "f32", 92)
    wide = y.long()
    wide[0], wide[1], wide[4] = -2 ** 63, 2 ** 32, 2 ** 63 - 1
    y[0], y[1], y[4] = -1, -1, -1
    loss = layers.policy_loss(z.cuda(), wide.cuda(), old.cuda(), adv.cuda(), None, torch.ones(6).cuda())
    ref.assert_loss(loss, ref.policy(z, y, old, adv, None, torch.ones(6))[0])
    z, y, _, _, _ = preference_inputs(12, 64, "f32", 1, 93)
    far = layers.preference_loss(z.cuda(), y.cuda(), torch.tensor([-2 ** 63, 6, 2 ** 63 - 1]).cuda())
    near = layers.preference_loss(z.cuda(), y.cuda(), torch.tensor([0, 6, 12]).cuda())
    assert torch.equal(far, near)


@pytest.mark.parametrize("default", [torch.float64, torch.bfloat16])
def test_layers_under_another_default_dtype(default):
    z, i, t, lse, w = distill_inputs(6, 300, "bf16", 8, 94)
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        leaf = z.cuda().requires_grad_()
        loss = layers.distill_topk(leaf, i.cuda(), t.cuda(), None, w.cuda())
        loss.backward()
    finally:
        torch.set_default_dtype(before)
    want = ref.distill(z, i, t, None, w)
    assert loss.dtype == torch.float32
    ref.assert_loss(loss, want[0])
    ref.assert_grad(leaf.grad, want[2], torch.bfloat16)


# -------------------------------------------------------- streams, repetition --

def test_repeated_calls_are_bit_identical():
    z, i, t, lse, w = distill_inputs(700, 3333, "bf16", 40, 51)
    a, ga, ga2 = run_distill(z, i, t, lse, w)
    b, gb, gb2 = run_distill(z, i, t, lse, w)
    assert torch.equal(a[0][0], b[0][0]) and torch.equal(a[1][1], b[1][1])
    assert torch.equal(ga, gb) and torch.equal(ga2, gb2)
    z, y, cuts, refp, w = preference_inputs(600, 3333, "f32", 7, 52)
    a, ga, _ = run_preference(z, y, cuts, refp, w)
    b, gb, _ = run_preference(z, y, cuts, refp, w)
    assert torch.equal(a[1][0], b[1][0]) and torch.equal(ga, gb)


def test_calls_run_on_the_given_stream():
    """Inputs written on a side stream, the call on it, no other synchronisation."""
    z, y, old, adv, refp, w = policy_inputs(400, 20000, "bf16", 61)
    want, g_want, _ = run_policy(z, y, old, adv, refp, w, kl_coef=0.1)
    side = torch.cuda.Stream()
    zc, yc, oc, ac, rc, wc = _cuda(z, y, old, adv, refp, w)
    late, out = torch.zeros_like(zc), (_out(1), _out(400), _out(400))
    g = torch.empty_like(zc)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(zc)
        binding.lik_policy_loss_step(late, yc, oc, ac, *out, g, ref_logp=rc, row_weight=wc, kl_coef=0.1)
    side.synchronize()
    assert torch.equal(out[1], want[1][1]) and torch.equal(g, g_want)
    # and the same by argument
    out2, g2 = (_out(1), _out(400), _out(400)), torch.empty_like(zc)
    torch.cuda.synchronize()
    binding.lik_policy_loss_step(zc, yc, oc, ac, *out2, g2, ref_logp=rc, row_weight=wc, kl_coef=0.1, stream=side)
    side.synchronize()
    assert torch.equal(g2, g_want)


def test_step_in_a_cuda_graph():
    z, i, t, lse, w = _cuda(*distill_inputs(64, 5001, "bf16", 32, 71))
    out, g = (_out(1), _out(64)), torch.empty_like(z)
    call = lambda: binding.lik_distill_topk_step(z, i, t, *out, g, row_weight=w)  # noqa: E731
    call()
    want = g.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    g.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g, want)


@pytest.mark.slow
def test_offsets_past_32_bits():
    """More than 2^31 logits: the last rows give what the same rows give alone."""
    rows, cols = 16900, 128000
    z = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    z.normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    tail = z[-40:].clone()
    y = torch.randint(0, cols, (rows,), device="cuda", dtype=torch.int32)
    old, adv = torch.full((rows,), -12.0, device="cuda"), torch.ones(rows, device="cuda")
    w = torch.ones(rows, device="cuda")
    out = (_out(1), _out(rows), _out(rows))
    binding.lik_policy_loss_step(z, y, old, adv, *out, z, row_weight=w)
    small, g = (_out(1), _out(40), _out(40)), torch.empty_like(tail)
    binding.lik_policy_loss_step(tail, y[-40:].contiguous(), old[-40:], adv[-40:], *small, g, row_weight=w[-40:])
    ref.assert_loss(out[1][-40:], small[1].cpu().double())
    ref.assert_grad(z[-40:], g.cpu().double(), torch.bfloat16)


# ------------------------------------------------------------------ refusals --

def test_refusals():
    z, i, t, lse, w = _cuda(*distill_inputs(4, 100, "f32", 8, 81))
    loss, rl, g = _out(1), _out(4), torch.empty_like(z)
    step = binding.lik_distill_topk_step
    with pytest.raises(ValueError):
        step(z.double(), i, t, loss, rl, g)
    with pytest.raises(ValueError):
        step(z.t().contiguous().t(), i, t, loss, rl, g)
    with pytest.raises(ValueError):
        step(z, i.long(), t, loss, rl, g)
    with pytest.raises(ValueError):
        step(z, i[:3], t, loss, rl, g)
    with pytest.raises(ValueError):
        step(z, i, t, loss, rl, g.bfloat16())
    with pytest.raises(ValueError):
        step(z.cpu(), i, t, loss, rl, g)
    with pytest.raises(ValueError):
        step(z, i, t, loss, rl, None)
    for scale in (0.0, -1.0, NAN, INF):
        with pytest.raises(binding.LIKError) as e:
            step(z, i, t, loss, rl, g, scale=scale)
        assert e.value.status == 1
    with pytest.raises(binding.LIKError) as e:  # an overlap that is not the logits buffer itself
        buf = torch.zeros(1000, device="cuda")
        step(buf[:400].view(4, 100), i, t, loss, rl, buf[100:500].view(4, 100))
    assert e.value.status == 1
    with pytest.raises(binding.LIKError) as e:  # rows that overlap each other
        step(z[:1].expand(4, 100), i, t, loss, rl, g)
    assert e.value.status == 1
    with pytest.raises(binding.LIKError) as e:
        big = torch.zeros(4, 1025, device="cuda")
        step(z, big.int(), big, loss, rl, g)
    assert e.value.status == 2
    y = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.zeros(4, device="cuda")
    for bad in (dict(clip_low=-0.1), dict(clip_low=1.5), dict(clip_high=-1.0), dict(kl_coef=NAN)):
        with pytest.raises(binding.LIKError) as e:
            binding.lik_policy_loss_step(z, y, f, f, loss, rl, _out(4), g, **bad)
        assert e.value.status == 1
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for bad in (dict(smoothing=1.5), dict(smoothing=-0.1), dict(beta=INF), dict(margin=NAN)):
        with pytest.raises(binding.LIKError) as e:
            binding.lik_preference_loss_fwd(z, y, off, loss, _out(1), _out(2), _out(4, 4), **bad)
        assert e.value.status == 1
    with pytest.raises(ValueError):
        binding.lik_preference_loss_fwd(z, y, off[:2].contiguous(), loss, _out(1), _out(2), _out(4, 4))
    with pytest.raises(ValueError):
        binding.lik_preference_loss_bwd(z, y, _out(3, 4), g)
    torch.cuda.synchronize()
