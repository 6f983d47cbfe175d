"""Draft verification (GPU) where probabilities are hard to take: columns that
are ruled out by a finite number, temperatures near 0, logits far from 0.

What log p may be off by (derived, no run behind it).  With e_c = exp(scale *
(z_c - max)) and p_c = e_c / sum:
  scale * (z - max): three roundings of 2^-24 of its size, which is at most
    |log p| + log(cols);
  the sum: each term's exponent t has the same three roundings, so that the
    sum is off by a share of at most 3 * 2^-24 * sum p_c |t_c|, and sum p_c
    |t_c| <= log(cols); the exponential's 2^-22; fp32 additions of the terms,
    which are a few dozen in a row before they are joined: 2^-18 with room;
  its logarithm: 2^-23 of its size.
Together below 2^-17 + 2^-21 |log p| for any number of columns here.
"""
import math

import pytest
import torch

import serving_reference as ref
import test_gpu_serving as one

pytestmark = pytest.mark.gpu

DT, NAN, INF = one.DT, float("nan"), float("inf")


def _from_largest(z):
    """Rows in 64 bits, less their largest: the same distribution, and a logarithm of the sum that 64 bits hold next to
    the logits whatever their size (3.4e38 + log(cols) is 3.4e38 there)."""
    return None if z is None else z.double() - z.double().amax(dim=1, keepdim=True)


def definition(target, draft, drafted, offsets, uniform, noise, scale=1.0):
    return ref.verify(_from_largest(target), _from_largest(draft), drafted, offsets, uniform, noise, scale)


def check(case, scale=1.0, want=None):
    """Tokens and counts are equal, log p within its bar; `want`: from other inputs than the call's."""
    tokens, accepted, logp = one.run_verify(*case, scale=scale)
    want = definition(*case, scale) if want is None else want
    assert accepted == want[1] and tokens == want[0]
    w = torch.tensor(want[2], dtype=torch.float64)
    off, bar = (logp.double() - w).abs(), 2.0 ** -17 + 2.0 ** -21 * w.abs()
    assert bool((off <= bar).all()), f"log p is off by {float((off / bar).max()):.2f} bars"
    return tokens, accepted


def _rows(offsets):
    return [t + b for b in range(len(offsets) - 1) for t in range(offsets[b], offsets[b + 1])]


def _drawn(gen, draft, scale):
    """A token of each draft row, from its own distribution."""
    noise = torch.empty(draft.shape).exponential_(generator=gen).double()
    return ((draft.double() * scale) - noise.log()).argmax(1).int()


# ------------------------------------------------- ruled out by a finite number --

LEAST = [("f32", torch.finfo(torch.float32).min), ("f32", -1e10), ("f32", -1e30), ("f16", torch.finfo(torch.float16).min),
         ("bf16", torch.finfo(torch.bfloat16).min), ("bf16", -1e10)]


def _masked(gen, counts, cols, dtype, low, keep, where):
    """Rows of which all but `keep` columns hold `low`; `where`: target, draft or both."""
    target, draft, _, offsets, uniform, noise = one._drafts(gen, counts, cols, dtype)
    for b, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        # a request's sampler keeps the same columns in all of its rows
        out = torch.ones(cols, dtype=torch.bool)
        out[torch.randperm(cols, generator=gen)[:keep]] = False
        if where != "draft":
            target[lo + b:hi + b + 1, out] = low
        if where != "target":
            draft[lo:hi, out] = low
    return target, draft, _drawn(gen, draft, 1.0) if sum(counts) else torch.zeros(0, dtype=torch.int32), offsets, uniform, noise


@pytest.mark.parametrize("dtype,low", LEAST)
@pytest.mark.parametrize("where", ["target", "draft", "both"])
@pytest.mark.parametrize("keep", [0, 1, 50])
def test_columns_ruled_out_by_a_finite_number(dtype, low, where, keep):
    """All columns but some hold the type's lowest value (or another far one): they have no probability."""
    gen = one._gen(keep + 7)
    for counts, cols in (([2, 0, 3], 4096), ([1, 2], 4099), ([1], 32003)):
        case = _masked(gen, counts, cols, dtype, low, keep, where)
        check(case)
        check((case[0], None) + case[2:])
        # uniforms of 0: a draft passes where its row and the target's both have it
        check(case[:4] + (torch.zeros_like(case[4]),) + case[5:])


def test_plain_sampling_from_masked_rows():
    """No drafts at all; the columns that are left lie together, so that most threads see none of them."""
    gen = one._gen(3)
    target = torch.full((4, 128_000), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16)
    for r, at in enumerate((0, 63_990, 127_950, 5)):
        target[r, at:at + 50] = torch.randn(50, generator=gen).to(torch.bfloat16)
    noise = torch.empty(4, 128_000).exponential_(generator=gen)
    none = torch.zeros(0, dtype=torch.int32)
    tokens, _ = check((target, None, none, [0] * 5, none.float(), noise))
    assert all(at <= t < at + 50 for t, at in zip(tokens, (0, 63_990, 127_950, 5)))


# ------------------------------------------------------------- low temperatures --

def _sharp(gen, counts, cols, dtype, scale, at):
    """Rows whose best columns lie within a few temperatures of one another, near `at`, above a bulk far below."""
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    rows = offsets[-1] + len(counts)
    target = at - 8.0 - torch.rand(rows, cols, generator=gen) * 4.0
    best = torch.stack([torch.randperm(cols, generator=gen)[:6] for _ in range(rows)])
    target.scatter_(1, best, at + 2.0 * torch.randn(rows, 6, generator=gen) / scale)
    target = target.to(DT[dtype])
    draft = target[_rows(offsets)].float()
    draft.scatter_add_(1, best[_rows(offsets)], torch.randn(offsets[-1], 6, generator=gen) / scale)
    draft = draft.to(DT[dtype])
    noise = torch.empty(len(counts), cols).exponential_(generator=gen)
    return target, draft, _drawn(gen, draft, scale), offsets, torch.rand(offsets[-1], generator=gen), noise


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale", [1e3, 1e4, 1e5, 1e6, 1e7, 1e8, 1e30])
def test_low_temperatures(dtype, scale):
    """1 / temperature far above 1: near-greedy and greedy sampling."""
    gen = one._gen(int(math.log10(scale)))
    for counts, cols in (([2, 3, 0], 4096), ([1, 4], 4099)):
        for at in (10.3, 17.77, 29.9):
            check(_sharp(gen, counts, cols, dtype, scale, at), scale)


@pytest.mark.parametrize("dtype,shift", [("f32", 1e6), ("f32", -1e6), ("f32", 3e8), ("f16", 6e4), ("bf16", 1e6)])
def test_logits_far_from_zero(dtype, shift):
    """A number added to a whole row changes nothing but what its rounding does to the logits."""
    gen = one._gen(9)
    for counts, cols in (([2, 0, 3], 4096), ([4], 4099)):
        target, draft, drafted, offsets, uniform, noise = one._drafts(gen, counts, cols, "f32")
        target, draft = ((t + shift).to(DT[dtype]) for t in (target, draft))
        case = (target, draft, _drawn(gen, draft, 1.0), offsets, uniform, noise)
        check(case)
        check(case, 0.25)


# -------------------------------------------------------- draft rows without mass --

@pytest.mark.parametrize("bad", [-INF, NAN, INF])
@pytest.mark.parametrize("cols", [100, 4096])
def test_draft_rows_that_are_no_distribution(bad, cols):
    """A draft row of -inf alone, or with a NaN or +inf logit: its draft does not pass, and p replaces it."""
    target, draft, drafted, offsets, _, noise = one._drafts(one._gen(cols), [3, 2, 1, 0], cols, "f32")
    uniform = torch.zeros(6)
    broken, none = draft.clone(), draft.clone()
    for r in (0, 4, 5):
        none[r] = NAN
        if bad == -INF:
            broken[r] = bad
        else:
            broken[r, (int(drafted[r]) + 7) % cols] = bad
    want = definition(target, none, drafted, offsets, uniform, noise)
    _, accepted = check((target, broken, drafted, offsets, uniform, noise), want=want)
    assert accepted == [0, 1, 0, 0]
