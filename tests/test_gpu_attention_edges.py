"""Attention over the 8-bit cache (GPU) at the ends of its range: references
that move at every tile, many short requests.  Definitions and bars: serving_reference.py."""
import pytest
import torch

import serving_reference as ref
import test_gpu_serving as one

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


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
