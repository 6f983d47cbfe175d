"""TokenCache (GPU) where a batch does not go as planned: places without a
request, steps that do not fit into the pages, the table or the rows."""
import pytest
import torch

import serving_reference as ref
import test_gpu_serving as one
import test_gpu_serving_step as steps
from late_interaction_retrieval_gb300 import TokenCache, binding, serving

pytestmark = pytest.mark.gpu

_dev = steps._dev


def _cache(pages=8, requests=2, max_tokens=64, heads=1, dim=16, page_size=16):
    return TokenCache(1, heads, dim, pages=pages, requests=requests, max_tokens=max_tokens, page_size=page_size)


# ------------------------------------------------------ places without a request --

@pytest.mark.parametrize("kept", [[4, 1], 4, [9, 9], 9])
def test_keep_takes_no_more_than_was_planned(kept):
    """An idle place (no new token) keeps none, whatever the verification of its neighbours' drafts gave it."""
    cache = _cache()
    cache.plan(_dev([4, 0]), 6)
    cache.keep(_dev(kept) if isinstance(kept, list) else kept)
    assert cache.cached.tolist() == [4, 0]
    cache.plan(_dev([2, 0]), 6)
    cache.keep(torch.tensor([1, 1], device="cuda"))  # of 64 bits
    assert cache.cached.tolist() == [5, 0] and cache.held.tolist() == [1, 0]
    cache.release(0)
    cache.plan(_dev([0, 3]), 6)
    cache.keep(_dev([1, 2]))
    assert cache.cached.tolist() == [0, 2]


# ------------------------------------------------------------ steps that do not fit --

def _same_state(cache, state):
    assert cache.cached.tolist() == state


def test_a_step_without_pages_is_not_kept():
    cache = _cache(pages=3)
    cache.plan(_dev([20, 5]), 25)
    assert int(cache.missing) == 0
    cache.keep(_dev([20, 5]))
    cache.plan(_dev([14, 2]), 25)
    assert int(cache.missing) == 1
    cache.keep(_dev([14, 2]))
    _same_state(cache, [20, 5])
    cache.plan(_dev([12, 11]), 25)  # the same pages hold these
    assert int(cache.missing) == 0
    cache.keep(_dev([12, 11]))
    _same_state(cache, [32, 16])


def test_a_request_that_outgrows_its_table_is_missing_pages():
    """max_tokens is passed although pages are free: counted, and not kept."""
    cache = _cache(pages=8, max_tokens=32)
    cache.plan(_dev([33, 4]), 40)
    assert int(cache.missing) == 1 and int(cache.free_count) == 5
    assert cache.slots.tolist()[32] == -1 and min(cache.slots.tolist()[33:37]) >= 0
    cache.keep(_dev([33, 4]))
    _same_state(cache, [0, 0])
    cache.plan(_dev([32, 0]), 40)
    assert int(cache.missing) == 0
    cache.keep(32)
    _same_state(cache, [32, 0])
    cache.plan(_dev([60, 40]), 100)  # 4 and 1 pages behind the tables
    assert int(cache.missing) == 5
    cache.keep(60)
    _same_state(cache, [32, 0])


def test_a_step_of_more_tokens_than_rows_is_not_kept():
    cache = _cache()
    cache.plan(_dev([6, 7]), 10)
    assert int(cache.missing) > 0 and cache.offsets.tolist() == [0, 6, 10]
    cache.keep(_dev([6, 4]))
    _same_state(cache, [0, 0])
    cache.plan(_dev([6, 4]), 10)
    assert int(cache.missing) == 0
    cache.keep(_dev([6, 4]))
    _same_state(cache, [6, 4])


def test_a_captured_step_that_does_not_fit_is_not_kept():
    """Nobody can look between the plan and the keep of a captured step: it looks itself."""
    cache, added, tokens = _cache(pages=4, max_tokens=48), _dev([1, 1]), _dev([1, 1])
    cache.plan(added, 40)
    cache.keep(tokens)
    cache.release(0)
    cache.release(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.plan(added, 40)
        cache.keep(tokens)
    state = [0, 0]
    # pages held, of 4 in all and 3 a request: 2 and 1; 3 (the one that was left) and 1, where 2 were wanted; so it stays
    for n, fits in (([20, 3], True), ([20, 17], False), ([0, 30], False), ([9, 0], True), ([8, 12], True), ([1, 0], True),
                    ([0, 0], True), ([30, 20], False)):
        added.copy_(_dev(n))
        tokens.copy_(_dev(n))
        graph.replay()
        if fits:
            state = [s + a for s, a in zip(state, n)]
        assert cache.cached.tolist() == state and (int(cache.missing) == 0) == fits, n


@pytest.mark.parametrize("most", [1, 40])
def test_rows_that_are_left_out_shift_nobody(most):
    """More new tokens than rows: those that have a row see what they would have seen."""
    gen = one._gen(most)
    heads, dim, page = 2, 64, 16
    cached, added, rows = [40, 9, 3], [5, 30, 4], 12
    case = one._requests(gen, cached, [0] * 3, heads, 4, dim, page, "bf16", spare=12)
    _, kc, vc, ks, vs, table, _, _ = case
    used = set(table[table >= 0].tolist())
    free = _dev([p for p in range(kc.shape[0]) if p not in used])
    table = torch.cat([table, torch.full((3, 4), -1, dtype=torch.int32)], 1).cuda()
    held = _dev([-(-c // page) for c in cached])
    kc, vc, ks, vs = (t.cuda() for t in (kc, vc, ks, vs))
    held, lengths, offsets, slots, _ = serving.cache_slots(_dev(cached), _dev(added), held, free, _dev([free.shape[0]]), table,
                                                           page, rows)
    assert offsets.tolist() == [0, 5, 12, 12] and lengths.tolist() == [45, 16, 3]
    x, y = (torch.randn(rows, heads, dim, generator=gen).bfloat16().cuda() for _ in range(2))
    serving.cache_write(x, y, slots, kc, vc, ks, vs)
    q = torch.randn(rows, 4 * heads, dim, generator=gen).bfloat16().cuda()
    got = serving.cache_attention(q, kc, vc, ks, vs, table, offsets, lengths, return_lse=True, max_added=most)
    binding.lik_check_device_error()
    want = ref.attention(q.cpu(), kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu(), table.cpu(), [0, 5, 12, 12], [45, 16, 3], dim ** -0.5)
    one.assert_attention(got, want)
