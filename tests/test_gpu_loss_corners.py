"""Corners of the training objectives over logits (GPU).  Where a finite row is
compared, it is with the fp64 definitions and bars of loss_reference.py; what
is infinite or left out has its value written down here."""
import gc
import sys
import threading

import pytest
import torch

import loss_reference as ref
from late_interaction_retrieval_gb300 import binding, layers
from test_gpu_losses import (DT, INF, NAN, NEG, _cuda, _gen, _out, check_distill, check_preference, distill_inputs,
                             policy_inputs, preference_inputs, run_distill, run_policy, run_preference)


pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _leave_no_garbage():
    """No device memory of these tests is left to be freed inside another."""
    yield
    gc.collect()


# ------------------------------------------------ terms whose factor is 0 --

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [60, 3001])
def test_preference_of_a_masked_answer(cols, dtype):
    """One pair's sequence counts a token on a masked column, so its x is +inf (rejected) or -inf (chosen).  Without
    smoothing -log sigma(+inf) is 0 and -log sigma(-inf) is inf; all smoothing exchanges the two; with some of both
    either is inf.  The slopes are finite."""
    rows = 12
    z, y, _, _, _ = preference_inputs(rows, cols, dtype, 2, 201)
    y = y.clamp(min=0)
    cuts = torch.tensor([0, 3, 6, 9, 12], dtype=torch.int32)  # pair 0 is rows 0..2 and 6..8, pair 1 3..5 and 9..11
    other = torch.tensor([1.0, 0.0])
    for row, sign in ((10, 1), (4, -1)):
        zm = z.clone()
        zm[row, int(y[row])] = NEG
        for smoothing in (0.0, 1.0, 0.25):
            beta, want = 0.1, [0.0, INF] if sign > 0 else [INF, 0.0]
            want = INF if 0.0 < smoothing < 1.0 else want[int(smoothing)]
            # the other pair alone, by its weight
            alone = ref.preference(zm, y, cuts, None, other, beta=beta, smoothing=smoothing)
            up = torch.tensor([2.0])
            forms, g, g2 = run_preference(zm, y, cuts, None, torch.ones(2), up=up, smoothing=smoothing, beta=beta)
            for loss, pair, seq in forms:
                ref.assert_loss(pair[:1], alone[1][:1])
                assert float(pair[1]) == want
                ref.assert_loss(loss, alone[0] + want)
                assert float(seq[3 if sign > 0 else 1]) == NEG
            # d loss / d x is -(1 - smoothing) at x = -inf and smoothing at +inf
            slope = beta * (smoothing if sign > 0 else smoothing - 1.0)
            log_q, _, on, at = ref._targets(zm, y, 1.0)
            coef = torch.zeros(rows, dtype=torch.float64)
            coef[3:6], coef[9:12] = slope, -slope
            grad = alone[3] + ref._target_grad(log_q, at, coef, on)
            ref.assert_grad(g, grad, DT[dtype])
            ref.assert_grad(g2, grad * 2.0, DT[dtype])


@pytest.mark.parametrize("cols", [60, 3001])
def test_policy_kl_term_without_a_coefficient(cols):
    """kl_coef 0 with a reference given: no term, however far (or masked, or not a number) the reference is."""
    z, y, old, adv, refp, w = policy_inputs(9, cols, "f32", 211)
    z[5, int(y[5])] = NEG  # its ratio is 0
    refp = refp + torch.tensor([0.0, 0.0, 0.0, 0.0, 95.0, 0.0, 1e6, INF, NAN])
    want = ref.policy(z, y, old, adv, None, w)
    forms, g, g2 = run_policy(z, y, old, adv, refp, w, kl_coef=0.0)
    for form in forms:
        for got, x in zip(form, want):
            ref.assert_loss(got, x)
    ref.assert_grad(g, want[3], torch.float32)
    ref.assert_grad(g2, want[3], torch.float32)


@pytest.mark.parametrize("cols", [60, 3001])
def test_policy_kl_term_of_a_masked_target(cols):
    """lp = -inf with a coefficient: exp(x) - x - 1 at x = +inf is +inf; the other rows are as without it."""
    z, y, old, adv, refp, w = policy_inputs(9, cols, "f32", 212)
    zm = z.clone()
    zm[5, int(y[5])] = NEG
    want = ref.policy(z, y, old, adv, refp, w, kl=0.1)
    forms, g, g2 = run_policy(zm, y, old, adv, refp, w, kl_coef=0.1)
    rest = [0, 1, 2, 3, 4, 6, 7, 8]
    for loss, row_loss, row_logp in forms:
        assert float(row_loss[5]) == INF and float(row_logp[5]) == NEG and float(loss) == INF
        ref.assert_loss(row_loss[rest], want[1][rest])
    ref.assert_grad(g[rest], want[3][rest], torch.float32)
    ref.assert_grad(g2[rest], want[3][rest], torch.float32)


@pytest.mark.parametrize("cols", [60, 3001])
def test_policy_without_advantage_at_any_ratio(cols):
    """Advantage 0 at a ratio past fp32's range (log ratios of 100 and +inf): no term, no gradient."""
    z, y, old, adv, refp, w = policy_inputs(9, cols, "f32", 213)
    far = old.clone()
    far[4], far[5], far[6] = old[4] - 100.0, NEG, old[6] - 100.0
    adv[4:7] = torch.tensor([0.0, -0.0, 0.0])
    near = torch.where(adv == 0, old, far)  # of a row without advantage, the old log-probability is of no account
    want = ref.policy(z, y, near, adv, refp, w, kl=0.1)
    forms, g, g2 = run_policy(z, y, far, adv, refp, w, kl_coef=0.1)
    for form in forms:
        for got, x in zip(form, want):
            ref.assert_loss(got, x)
    ref.assert_grad(g, want[3], torch.float32)
    ref.assert_grad(g2, want[3], torch.float32)


# ---------------------------------------------------------- the teacher's --

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [50, 9000])
def test_teacher_without_an_entry_and_any_normaliser(cols, dtype):
    """Rows of padding alone and of -inf alone are left out whatever their log-sum-exp is (-inf is what a fully
    masked teacher row gives)."""
    z, index, t, _, w = distill_inputs(8, cols, dtype, 12, 221, padded=False, weighted=False)
    index[0], index[3] = -1, cols
    t[1], t[4], t[6] = NEG, NEG, NEG
    lse = torch.logsumexp(t.double(), 1).float() + 0.5
    lse[0], lse[1], lse[3], lse[4], lse[6] = NEG, NEG, NAN, NAN, INF
    want = check_distill(z, index, t, lse=lse)
    assert (want[1][[0, 1, 3, 4, 6]] == 0).all() and (want[1][[2, 5, 7]] != 0).all()


@pytest.mark.parametrize("scale", [1.0, 0.75])
@pytest.mark.parametrize("level", [1000.0, -4000.0])
@pytest.mark.parametrize("cols", [200, 3001, 70000])
def test_teacher_far_from_zero(cols, level, scale):
    """A level common to the teacher's logits and their log-sum-exp cancels.  An entry's log p is one fused
    multiply-add, rounded once from the inputs, so the bars are the ordinary ones."""
    z, index, t, _, w = distill_inputs(5, cols, "f32", 64, 231)
    t = t + level
    lse = (torch.logsumexp(t.double() * scale, 1) + 0.25).float()
    check_distill(z, index, t, lse, w, scale=scale)


@pytest.mark.parametrize("cols", [300, 5000])
def test_duplicate_columns_across_warps(cols):
    """Hundreds of entries over a few columns, padding and -inf among them."""
    gen = _gen(cols)
    for k, of in ((40, 5), (300, 20), (1000, 50), (1024, 1), (700, 290)):
        z = (torch.randn(5, cols, generator=gen) * 2.5)
        pool = torch.randperm(cols, generator=gen)[:of]
        index = pool[torch.randint(0, of, (5, k), generator=gen)].to(torch.int32)
        t = torch.randn(5, k, generator=gen) * 2.0
        index[torch.rand(5, k, generator=gen) < 0.1] = -1
        t[torch.rand(5, k, generator=gen) < 0.1] = NEG
        check_distill(z, index, t)
        check_distill(z, index, t, lse=torch.logsumexp(t, 1) + 0.5)
        first = run_distill(z, index, t)
        again = run_distill(z, index, t)
        assert torch.equal(first[1], again[1]) and torch.equal(first[2], again[2])


# ------------------------------------------------------------ long sequences --

@pytest.mark.parametrize("average", [False, True])
def test_preference_of_long_sequences(average):
    """Sums of thousands of log-probabilities, some 30000, in a difference of about 10: the fp32 of a returned sum has
    steps of 2^-9 there, 2e-4 of beta * gap.  The loss has its ordinary bar: a row's log-probability is rounded at
    2^-20 or less, and 3000 such roundings add up to some 1e-5 of a sum, 1e-6 of beta times it."""
    gen = _gen(281)
    rows, cols, pairs = 24000, 37, 4
    z = torch.randn(rows, cols, generator=gen) * 4.0
    y = torch.randint(0, cols, (rows,), generator=gen).to(torch.int32)
    cuts = torch.arange(0, rows + 1, rows // (2 * pairs)).to(torch.int32)
    seq = ref.preference(z, y, cuts, average=average)[2]
    refp = (seq + torch.randn(2 * pairs, generator=gen) * 5.0).float()
    check_preference(z, y, cuts, refp, torch.ones(pairs), average=average, beta=0.1)


# -------------------------------------------------------------------- layers --

@pytest.mark.parametrize("cols", [40, 3001])
def test_layers_over_rows_that_overlap(cols):
    """An expanded row of logits, and windows over a line of scores: gradients add up where rows share elements."""
    z, i, t, _, w = distill_inputs(4, cols, "f32", 10, 251)
    leaf = z[:1].cuda().requires_grad_()
    loss = layers.distill_topk(leaf.expand(4, cols), i.cuda(), t.cuda(), None, w.cuda())
    loss.backward()
    want = ref.distill(z[:1].repeat(4, 1), i, t, None, w)
    ref.assert_loss(loss, want[0])
    ref.assert_grad(leaf.grad, want[2].sum(0, keepdim=True), torch.float32)
    z, y, old, adv, refp, w = policy_inputs(4, cols, "f32", 252)
    line = torch.randn(cols + 3, generator=_gen(3)) * 2.5
    leaf = line.cuda().requires_grad_()
    windows = leaf.unfold(0, cols, 1)
    assert windows.shape == (4, cols) and windows.stride() == (1, 1)
    loss = layers.policy_loss(windows, y.cuda(), old.cuda(), adv.cuda(), refp.cuda(), w.cuda(), kl_coef=0.1)
    loss.backward()
    want = ref.policy(line.unfold(0, cols, 1), y, old, adv, refp, w, kl=0.1)
    total = torch.zeros(cols + 3, dtype=torch.float64)
    for r in range(4):
        total[r:r + cols] += want[3][r]
    ref.assert_loss(loss, want[0])
    ref.assert_grad(leaf.grad, total, torch.float32)


def test_layers_refuse_a_second_derivative():
    """create_graph keeps the first gradient as it is; differentiating that one is an error, not a constant."""
    z, i, t, _, w = distill_inputs(4, 300, "f32", 10, 261)
    _, y, old, adv, _, _ = policy_inputs(4, 300, "f32", 262)
    i, t, w, y, old, adv = _cuda(i, t, w, y, old, adv)
    cuts = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    calls = [lambda x: layers.distill_topk(x, i, t, None, w), lambda x: layers.policy_loss(x, y, old, adv, None, w),
             lambda x: layers.preference_loss(x, y, cuts)]
    for call in calls:
        a = z.cuda().requires_grad_()
        (first,) = torch.autograd.grad(call(a), a)
        loss = call(a)
        (g,) = torch.autograd.grad(loss, a, create_graph=True)
        assert torch.equal(g, first)
        with pytest.raises(RuntimeError, match="second derivative"):
            (loss + g.square().sum()).backward()
        inner = z.cuda().view(2, 2, 300).requires_grad_()  # through what comes before the layer
        loss = call(torch.tanh(inner.reshape(4, 300)))
        (g,) = torch.autograd.grad(loss, inner, create_graph=True)
        with pytest.raises(RuntimeError, match="second derivative"):
            torch.autograd.grad(g.square().sum(), inner)


# ------------------------------------------------------------------ in place --

@pytest.mark.parametrize("rows,cols,dtype", [(70, 17, "f32"), (5, 77, "bf16"), (6, 3001, "f32"), (4, 40001, "f16"),
                                             (3, 131072, "bf16")])
def test_backward_in_place_of_the_logits(rows, cols, dtype):
    """The gradient from a saved state, written over the logits it is taken from, is the one written elsewhere."""
    z, i, t, lse, w = _cuda(*distill_inputs(rows, cols, dtype, 20, 241, full=True))
    state, apart = _out(rows, 4), torch.empty_like(z)
    binding.lik_distill_topk_fwd(z, i, t, _out(1), _out(rows), state, teacher_lse=lse, row_weight=w)
    binding.lik_distill_topk_bwd(z, i, t, state, apart, teacher_lse=lse)
    binding.lik_distill_topk_bwd(z, i, t, state, z, teacher_lse=lse)
    assert torch.equal(z, apart)
    z, y, old, adv, refp, w = _cuda(*policy_inputs(rows, cols, dtype, 242))
    binding.lik_policy_loss_fwd(z, y, old, adv, _out(1), _out(rows), _out(rows), state, ref_logp=refp, row_weight=w,
                                kl_coef=0.1)
    binding.lik_policy_loss_bwd(z, y, state, apart)
    binding.lik_policy_loss_bwd(z, y, state, z)
    assert torch.equal(z, apart)
    z, y, cuts, refp, w = _cuda(*preference_inputs(rows, cols, dtype, 1, 243))
    binding.lik_preference_loss_fwd(z, y, cuts, _out(1), _out(1), _out(2), state, ref_logp=refp, pair_weight=w)
    binding.lik_preference_loss_bwd(z, y, state, apart)
    binding.lik_preference_loss_bwd(z, y, state, z)
    assert torch.equal(z, apart)
    binding.lik_check_device_error()


# ------------------------------------------------------------------- callers --

def test_calls_from_several_threads():
    """Steps of two row lengths at once, whose blocks need 50 and 64 KB of shared memory: no call lowers what another's
    launch may use.  The library's entry is called directly, so that the threads meet inside it."""
    step = binding.load().lik_distill_topk_step
    refused = []

    def work(cols):
        torch.cuda.set_device(0)
        stream = torch.cuda.Stream()
        z, i, t, _, _ = _cuda(*distill_inputs(1, cols, "bf16", 4, cols, weighted=False))
        loss, row_loss, g = _out(1), _out(1), torch.empty_like(z)
        stream.wait_stream(torch.cuda.current_stream())
        args = (z.data_ptr(), binding.LIK_BF16, 1, cols, cols, i.data_ptr(), t.data_ptr(), binding.LIK_F32, 4, None,
                None, 1.0, loss.data_ptr(), row_loss.data_ptr(), g.data_ptr(), cols, stream.cuda_stream)
        refused.append(sum(step(*args) != 0 for _ in range(20000)))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(cols,)) for cols in (512, 385) * 3]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert refused == [0] * 6


# --------------------------------------------------------- the longest calls --

@pytest.mark.slow
def test_sequences_that_end_at_the_last_row_there_can_be():
    """2^31 - 1 rows of two columns; the only pair's sequences are the last 300 rows."""
    rows = 2 ** 31 - 1
    z = torch.zeros(rows, 2, dtype=torch.bfloat16, device="cuda")
    target = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    tail_z = torch.randn(300, 2, generator=_gen(271)).bfloat16()
    tail_y = torch.randint(0, 2, (300,), generator=_gen(272)).to(torch.int32)
    z[-300:], target[-300:] = tail_z.cuda(), tail_y.cuda()
    state = torch.zeros(rows, 4, device="cuda")
    cuts = torch.tensor([rows - 300, rows - 140, rows], dtype=torch.int32)
    loss, pair, seq = _out(1), _out(1), _out(2)
    binding.lik_preference_loss_step(z, target, cuts.cuda(), loss, pair, seq, state, z)
    binding.lik_check_device_error()
    want = ref.preference(tail_z, tail_y, torch.tensor([0, 160, 300]))
    ref.assert_loss(loss, want[0])
    ref.assert_loss(seq, want[2])
    ref.assert_grad(z[-300:], want[3], torch.bfloat16)
    assert not z[:-300].any()
    del z, target, state
    torch.cuda.empty_cache()
