"""Attention over the 8-bit cache (GPU) at the ends of its range: scores far
from 0, references that move at every tile, many short requests, requests that
are longer than their table.  Definitions and bars: serving_reference.py."""
import math

import pytest
import torch

import serving_reference as ref
import test_gpu_serving as one

pytestmark = pytest.mark.gpu

F8, NAN = torch.float8_e4m3fn, float("nan")


# ----------------------------------------------------------- scores far from 0 --

FAR = 12  # dimensions that make a score far from 0


def _far(seed, lengths, added, heads, group, dim, page, dtype, levels):
    """Scores of whole numbers: `levels` (one a page, in turn) times 256 * 448 * FAR, and a few units.

    They are exact in 32 bits (below 2^24, of whole numbers), and so are their differences; the values' scales are
    powers of two.  What is left of the bars: a weight's 2^-11, the factor scale * log2(e) (off by 2^-22 of itself at
    most), which scales the differences of scores, up to `span`, and the log-sum-exp's own 2^-21.  And the step of the
    smallest weights: 2^-24 in fp16, half of it 2^-25, where a row's largest weight is at least 2^6 (with its page's
    scale in it), so that each of its tokens is off by up to 2^-31 of the largest weight times its own code: 448 at
    most, of scales up to 2^-5.  A dimension in which the likely tokens are 0 shows it."""
    gen = one._gen(seed)
    q, kc, vc, ks, vs, table, offsets, lengths = one._requests(gen, lengths, added, heads, group, dim, page, dtype)
    pages = kc.shape[0]
    unused = ks[:, 0].isnan()
    small = torch.randint(-2, 3, kc.shape, generator=gen).float()
    level = torch.zeros(pages)
    for row in table:
        for j, p in enumerate(row.tolist()):
            if p >= 0:
                level[p] = levels[j % len(levels)]
    small[..., :FAR] = 448.0 * level[:, None, None, None]
    hidden = (kc.view(torch.uint8) & 0x7F) == 0x7F
    kc = torch.where(hidden, kc.float(), small).to(F8)
    q = torch.randint(-2, 3, q.shape, generator=gen).to(q.dtype)
    q[..., :FAR] = 256.0
    ks, vs = torch.ones_like(ks), 2.0 ** torch.randint(-9, -4, vs.shape, generator=gen).float()
    ks[unused], vs[unused] = NAN, NAN
    return q, kc, vc, ks, vs, table, offsets, lengths


def _check_far(case, span=8 * 128.0, **kw):
    out, lse, _, _ = ref.attention(*case, 1.0)
    q, _, vc, _, vs, table, offsets, lengths = case
    # sum p |v|: the same attention over the values' sizes
    size = ref.attention(*case[:2], vc.float().abs().to(F8), *case[3:], 1.0)[0]
    bar = (2.0 ** -11 + 2.0 ** -20 + 2.0 ** -21 * span) * size + (ref.HALF_STEP[q.dtype] * out.abs()).clamp(
        min=ref.LEAST_HALF_STEP[q.dtype]) + 2.0 ** -31 * 2.0 ** -5 * 448 * max(lengths)
    got = one.run_attention(*case, 1.0, **kw)
    one.assert_attention(got, (out, lse, bar, 2.0 ** -18 + 2.0 ** -21 * lse.abs()))


BATCHES = [([40, 300], [1, 1], 4), ([700], [1], 1), ([33, 90], [2, 1], 8), ([300, 70], [5, 3], 8), ([260, 3], [130, 3], 4),
           ([600], [300], 2)]
# 12 * 256 * 448 = 1376256 below and above 0 (1985508 in powers of two), in all pages or some
LEVELS = [[-1.0], [1.0], [-1.0, -0.625], [-0.625, -1.0], [-1.0, 0.0], [0.0, -1.0], [-1.0, -1.0, -1.0, 1.0], [1.0, -1.0]]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("levels", LEVELS)
def test_scores_far_from_zero(dtype, levels):
    for i, (lengths, added, group) in enumerate(BATCHES):
        for page in (16, 64):
            _check_far(_far(i, lengths, added, 1, group, 64, page, dtype, levels))
    _check_far(_far(9, [300, 40], [5, 1], 2, 4, 128, 32, dtype, levels))


@pytest.mark.parametrize("levels", [[-1.0], [-1.0, -0.625]])
def test_scores_far_from_zero_split_along_the_cache(levels):
    """Pieces whose rows have seen such scores only, and pieces that have seen nothing, joined."""
    case = _far(3, [20011], [1], 1, 4, 16, 64, "bf16", levels)
    case[5][0, 40:100] = -1
    _check_far(case)
    case = _far(4, [9000], [40], 1, 4, 64, 64, "f16", levels)
    case[5][0, :70] = -1
    _check_far(case)


# -------------------------------------------- references that move at every tile --

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("added,group", [(300, 4), (40, 2), (20, 2)])
def test_references_that_move_at_every_tile(dtype, added, group):
    """Scores and values' scales that grow along the cache: the sums are rescaled at every tile, in every run alike."""
    q, kc, vc, ks, vs, table, offsets, lengths = case = one._requests(one._gen(added), [2500, 1800], [added, added // 2], 2,
                                                                      group, 64, 64, dtype)
    for row in table:
        for j, p in enumerate(row.tolist()):
            if p >= 0:
                ks[p] = 0.004 * (1.0 + 0.5 * j)
                vs[p] = 2.0 ** (j - 30)
    got = one.run_attention(*case, 0.125)
    for _ in range(30):
        again = one.run_attention(*case, 0.125)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    some = [0, 1, added // 2, added - 1, added, added + added // 2 - 1]
    out, lse, bar, lse_bar = ref.attention(*case, 0.125)
    # Where the likely tokens' values are small, what the unlikely ones' weights lose shows: half a step of the smallest
    # fp16 numbers, 2^-25, where a row's largest weight is 2^6 at least (its page's scale in it).  So each token is off by
    # at most 2^-31 of that weight, sum p v_scale at most, times a code, 448 at most.
    unit = ref.attention(*case[:2], torch.ones(vc.shape).to(F8), *case[3:], 0.125)[0]
    bar = bar + 2.0 ** -31 * 448 * max(lengths) * unit
    one.assert_attention([t[some] for t in got], [t[some] for t in (out, lse, bar, lse_bar)])


# -------------------------------------------------------- many short requests --

@pytest.mark.parametrize("group", [2, 10])
def test_many_short_requests(group):
    """More requests than a block has warps' chunks for, of a unit or two each: the same bits in every run."""
    gen = one._gen(group)
    n = 700
    lengths = [int(x) for x in torch.randint(1, 40, (n,), generator=gen)]
    added = [int(i % 5 != 0) for i in range(n)]
    case = one._requests(gen, lengths, added, 1, group, 16, 16, "bf16")
    got = one.check_attention(case)
    for _ in range(40):
        again = one.run_attention(*case, 0.25)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


# ----------------------------------------------- requests longer than their table --

def _cut(case, cols):
    """The same batch with tables of `cols` columns, and with tables whose further entries are no pages."""
    q, kc, vc, ks, vs, table, offsets, lengths = case
    wide = table.clone()
    wide[:, cols:] = -1
    return (q, kc, vc, ks, vs, table[:, :cols].contiguous(), offsets, lengths), (q, kc, vc, ks, vs, wide, offsets, lengths)


@pytest.mark.parametrize("page,group", [(16, 1), (16, 4), (64, 8), (128, 2)])
def test_requests_that_pass_their_table(page, group):
    """A row sees what it would with a longer table, without the tokens that have no place in it."""
    for seed, (lengths, added) in enumerate([([3 * page + 3, 7], [5, 2]), ([3 * page + 1, 4 * page], [1, 1]),
                                             ([4 * page, 3 * page + 9], [page + 4, 12]), ([5 * page, 2 * page], [page, 3])]):
        case = one._requests(one._gen(seed), lengths, added, 2, group, 64, page, "bf16")
        for cols in (3, 1):
            narrow, wide = _cut(case, cols)
            for hint in (1, 1000):  # both kernels
                got = one.run_attention(*narrow, 0.125, max_added=hint)
                one.assert_attention(got, ref.attention(*wide, 0.125))


def test_lengths_out_of_range():
    """The largest and negative lengths: all of the table is seen, or nothing."""
    case = one._requests(one._gen(5), [48, 48, 48], [3, 2, 1], 1, 2, 32, 16, "f16")
    narrow, wide = _cut(case, 3)
    q, kc, vc, ks, vs, table, offsets, _ = narrow
    for hint in (1, 1000):
        out, lse = one.run_attention(q, kc, vc, ks, vs, table, offsets, [2 ** 31 - 1, -7, 2 ** 31 - 1], 0.2, max_added=hint)
        want = ref.attention(q, kc, vc, ks, vs, wide[5], offsets, [51, 0, 49], 0.2)
        one.assert_attention((out, lse), want)
        assert bool((out[3:5] == 0).all()) and bool((lse[3:5] == -math.inf).all())


@pytest.mark.parametrize("hint", [1, 1000])
def test_no_columns_no_pages(hint):
    """Tables without a column, a cache without a page: rows that see nothing."""
    q, kc, vc, ks, vs, table, offsets, lengths = one._requests(one._gen(6), [20, 5], [3, 1], 2, 4, 32, 16, "bf16")
    for case in ((q, kc, vc, ks, vs, table[:, :0], offsets, lengths), (q, kc[:0], vc[:0], ks[:0], vs[:0], table, offsets, lengths)):
        out, lse = one.run_attention(*case, 0.2, max_added=hint)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())
