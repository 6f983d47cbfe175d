"""TokenCache (GPU) where a batch does not go as planned: places without a
request, steps that do not fit into the pages, the table or the rows, and a
whole step of requests that come and go, as the documentation shows it."""
import os

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


# ------------------------------------------------------------- whether a batch fits --

def _fit(cached, added, held, free, count, table, page, capacity):
    """lik_cache_slots_fit beside lik_cache_slots, which it has to equal in all but the lengths; most, missing, lengths."""
    n = len(cached)
    plain = one.run_slots(cached, added, held, free, count, table, page, capacity)
    held_out, lengths, most = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for _ in range(3))
    offsets, left, missing = (torch.full((k,), -9, dtype=torch.int32, device="cuda") for k in (n + 1, 1, 1))
    slots, own = torch.full((capacity,), -9, dtype=torch.int64, device="cuda"), table.cuda()
    binding.lik_cache_slots_fit(_dev(cached), _dev(added), _dev(held), _dev(free), _dev([count]), own, held_out, lengths,
                                offsets, slots, left, most, missing, page_size=page)
    assert torch.equal(own.cpu(), plain[0]) and held_out.tolist() == plain[1] and offsets.tolist() == plain[3]
    assert slots.tolist() == plain[4] and int(left) == plain[5]
    # by the definition: a token has its place if it has a slot, as long as no page that is held is missing in the table
    has = [max(c, 0) for c in cached]
    want = [min(c + b - a, 2 ** 31 - 1) for c, a, b in zip(has, plain[3], plain[3][1:])]
    lost = sum(max(a, 0) for a in added) - sum(s >= 0 for s in plain[4])
    short = max(-plain[5], -(-lost // page))
    assert lengths.tolist() == want and int(missing) == min(short, 2 ** 31 - 1)
    assert most.tolist() == (has if short else want)
    return short


@pytest.mark.parametrize("n,page", [(1, 16), (7, 64), (33, 32), (513, 16), (1500, 128), (8192, 16)])
def test_whether_a_batch_fits(n, page):
    """Batches that fit, and the same ones with fewer pages, columns or rows."""
    gen = one._gen(n)
    cols = -(-(90 + 40) // page) + 1
    cached, added, held, free, table = one._batch(gen, n, 90, 40, page, cols, extra=0.3)
    rows = sum(added)
    assert _fit(cached, added, held, free, len(free), table, page, rows + 5) == 0
    assert _fit(cached, added, held, free, len(free), table, page, rows) == 0
    assert _fit(cached, added, held, free, 2, table, page, rows + 5) == max(0, sum(
        max(0, -(-(c + a) // page) - h) for c, a, h in zip(cached, added, held)) - 2)
    _fit(cached, added, held, free, len(free), table, page, max(rows - 7, 0))
    _fit(cached, added, held, free, len(free), table, page, rows // 3)
    few = max(1, cols // 2)
    _fit(cached, added, [min(h, few) for h in held], free, len(free), table[:, :few].contiguous(), page, rows + 3)


def test_whether_odd_batches_fit():
    """No request, no row, no page, no column; negative numbers; lengths next to 2^31."""
    assert _fit([], [], [], [3, 4], 2, torch.zeros((0, 4), dtype=torch.int32), 16, 5) == 0
    table = torch.arange(20, dtype=torch.int32).reshape(4, 5)
    assert _fit([3, 0, 0, 9], [0, 0, 0, 0], [1, 0, 0, 1], [50], 1, table, 16, 0) == 0
    assert _fit([3, 0, 0, 9], [1, 0, 0, 0], [1, 0, 0, 1], [50], 1, table, 16, 0) == 1
    assert _fit([0, 0], [3, 20], [0, 0], [], 0, table[:2], 16, 30) == 3
    assert _fit([0, 0], [3, 20], [0, 0], [5], 1, torch.zeros((2, 0), dtype=torch.int32), 16, 30) == 2
    assert _fit([-5, 40, 70, 3], [10, 30, 40, -2], [0, 5, 9, -1], [90, 91, 92], 7, table, 16, 200) == 2
    _fit([2 ** 31 - 1, 4], [2 ** 31 - 1, 2 ** 31 - 1], [0, 0], [1], 1, table[:2].clone(), 256, 300)


def test_fit_refusals():
    i = _dev([1, 2])
    one_, table, slots = _dev([1]), torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int64,
                                                                                                  device="cuda")

    def call(most=None, missing=None, page=16):
        binding.lik_cache_slots_fit(i, i, i, i, one_, table, i.clone(), i.clone(), _dev([0, 0, 0]), slots, one_.clone(),
                                    i.clone() if most is None else most, one_.clone() if missing is None else missing,
                                    page_size=page)

    call()
    both = i.clone()
    for bad in (dict(page=24), dict(most=i), dict(missing=one_), dict(most=both, missing=both[1:]),
                dict(most=table.view(-1)[2:4])):
        with pytest.raises(binding.LIKError):
            call(**bad)
    for bad in (dict(most=i.long()), dict(most=_dev([1])), dict(missing=i), dict(missing=one_.cpu())):
        with pytest.raises(ValueError):
            call(**bad)


# ------------------------------------------------- requests that come and go --

def test_rows_of_the_logits():
    """Which rows of a step a verification wants: the newest token's and the drafts' of a request that decodes, the last
    of a prompt; a place without a request has a row of no meaning."""
    cache = _cache(pages=40, requests=5, max_tokens=64)
    cache.plan(_dev([3, 0, 20, 1, 0]), 30)
    rows, offsets = cache.verify_rows(_dev([2, 0, 0, 0, 0]), 4)
    assert rows.dtype == torch.int64 and offsets.dtype == torch.int32
    assert offsets.tolist() == [0, 2, 2, 2, 2, 2] and rows.shape == (9,)
    got = rows.tolist()
    assert got[:3] == [0, 1, 2] and got[4:6] == [22, 23]
    assert all(0 <= r < 30 for r in got)
    # more drafts than a request planned: what it planned but for its newest token
    rows, offsets = cache.verify_rows(_dev([9, 4, 2, 1, -1]), 6)
    assert offsets.tolist() == [0, 2, 2, 4, 4, 4] and rows.tolist()[:3] == [0, 1, 2] and rows.tolist()[4:8] == [20 + 0, 21, 22, 23]


@pytest.mark.parametrize("captured", [False, True])
def test_requests_come_and_go(captured):
    """The documented step over places of which some are empty: each request's rows, tokens and cache are those that it
    would have alone."""
    gen = one._gen(4)
    model = steps.Model(gen, heads=2, group=2, dim=32, cols=97)
    places, rows, total = 3, 24, 9
    cache = TokenCache(1, 2, 32, pages=30, requests=places, max_tokens=96, page_size=16)
    i32 = dict(dtype=torch.int32, device="cuda")
    b = dict(tokens=torch.zeros(rows, **i32), added=torch.zeros(places, **i32), drafts=torch.zeros(places, **i32),
             drafted=torch.zeros(total, **i32), uniform=torch.zeros(total, device="cuda"),
             noise=torch.ones(places, 97, device="cuda"))

    def step():
        q, k, v = model.qkv(b["tokens"])
        cache.plan(b["added"], rows)
        cache.write(0, k, v)
        x = cache.attention(0, q, max_added=4, out=torch.zeros_like(q))
        logits = model.logits(x)
        at, offsets = cache.verify_rows(b["drafts"], total)
        got = serving.verify_drafts(logits[at], b["drafted"], offsets, b["uniform"], b["noise"])
        cache.keep(b["added"] - b["drafts"] + got[1])
        return q, k, v, x, logits, got

    if captured:
        step()  # nobody is there yet
        assert cache.cached.tolist() == [0, 0, 0] and cache.held.tolist() == [0, 0, 0]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
    place, alone, prompt, newest = [None] * places, {}, {}, {}
    # what happens before each step: a request's name in its place, "-" where one ends
    for event in ({0: "a"}, {2: "b"}, {}, {0: "-"}, {1: "c"}, {2: "-", 0: "d"}, {}, {1: "-"}, {}):
        for p, name in event.items():
            if name == "-":
                cache.release(p)
                place[p] = None
                continue
            place[p] = name
            prompt[name] = torch.randint(0, 97, (int(torch.randint(1, 9, (1,), generator=gen)),), generator=gen).tolist()
            alone[name] = TokenCache(1, 2, 32, pages=6, requests=1, max_tokens=96, page_size=16)
        packed, added, drafts, drafted = [], [], [], []
        for name in place:
            d = []
            if name in newest:  # the newest token and what a draft model adds to it
                d = torch.randint(0, 97, (int(torch.randint(0, 4, (1,), generator=gen)),), generator=gen).tolist()
            new = [] if name is None else [newest[name]] + d if name in newest else prompt[name]
            packed, drafted = packed + new, drafted + d
            added.append(len(new))
            drafts.append(len(d))
        uniform = torch.rand(total, generator=gen) * 0.05
        noise = torch.empty(places, 97).exponential_(generator=gen)
        for key, value in (("tokens", packed + [5] * (rows - len(packed))), ("added", added), ("drafts", drafts),
                           ("drafted", drafted + [3] * (total - len(drafted)))):
            b[key].copy_(torch.tensor(value, dtype=torch.int32))
        b["uniform"].copy_(uniform)
        b["noise"].copy_(noise)
        if captured:
            graph.replay()
            q, k, v, x, logits, (tokens, accepted, logp) = held
        else:
            q, k, v, x, logits, (tokens, accepted, logp) = step()
        assert int(cache.missing) == 0
        first = cut = 0
        for p, name in enumerate(place):
            if name is None:
                assert int(cache.cached[p]) == 0 and int(cache.held[p]) == 0
                continue
            own, end, d = alone[name], first + added[p], drafts[p]
            own.plan(_dev([added[p]]), added[p])
            own.write(0, k[first:end], v[first:end])
            y = own.attention(0, q[first:end], max_added=4)
            # either is off by half a step of bf16 and 2^-11 of the values' sizes
            size = float(own.v_scale.max()) * 448
            assert float((y.float() - x[first:end].float()).abs().max()) <= 2 * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -14) * size
            want = ref.verify(logits[end - d - 1:end].cpu(), None, torch.tensor(drafted[cut:cut + d]), [0, d],
                              uniform[cut:cut + d], noise[p:p + 1], 1.0)
            assert tokens[cut + p:cut + p + d + 1].tolist() == want[0] and int(accepted[p]) == want[1][0]
            own.keep(added[p] - d + want[1][0])
            n = int(own.cached)
            assert int(cache.cached[p]) == n and int(cache.held[p]) == int(own.held)
            here, there = ([c.block_table[r][:int(c.held[r])].long() for c, r in ((cache, p), (own, 0))])
            assert torch.equal(cache.k_scale[0][here], own.k_scale[0][there])
            for codes, same in ((cache.k, own.k), (cache.v, own.v)):
                a, c = (t.view(torch.uint8)[0][at].transpose(1, 2).flatten(0, 1)[:n] for t, at in ((codes, here), (same, there)))
                assert torch.equal(a, c)
            newest[name] = want[0][want[1][0]]
            first, cut = end, cut + d
    binding.lik_check_device_error()


# ---------------------------------------------------------- as it is documented --

def test_the_documented_step():
    """README's step, as it stands there, on a small model: a request with drafts, an empty place, a prompt."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        text = f.read()
    code = text[text.index("**A serving step.**"):]
    code = code[code.index("```python\n") + 10:]
    gen = one._gen(6)
    model = [steps.Model(gen, heads=2, group=2, dim=128, cols=83) for _ in range(2)]
    caches = []

    class Layer:
        def __init__(self, weights):
            self.project, self.finish = weights.qkv, lambda out: weights.logits(out).argmax(1)

    def small(**sizes):
        caches.append(TokenCache(**dict(sizes, layers=2, heads=2, pages=12, requests=3, max_tokens=64)))
        return caches[0]

    added, drafts, drafted = [3, 0, 6], [2, 0, 0], [7, 11]
    target, draft = one._logits(gen, 12, 83, "f32"), one._logits(gen, 2, 83, "f32")
    uniform, noise = torch.full((2,), 1e-6), torch.empty(3, 83).exponential_(generator=gen)
    seen = []
    names = dict(TokenCache=small, verify_drafts=serving.verify_drafts, model=[Layer(m) for m in model], rows=12, total=2,
                 x=torch.randint(0, 83, (12,), generator=gen).cuda(), added=_dev(added), drafts=_dev(drafts),
                 drafted=_dev(drafted), uniform=uniform.cuda(), noise=noise.cuda(), draft_logits=draft.cuda(),
                 head=lambda x: seen.append(x) or target.cuda()[:5])
    exec(code[:code.index("```")], names)
    # verify_drafts has 2 + 1 rows of the first request, one of the empty place, one of the prompt
    assert seen[0].shape == (5,) and torch.equal(seen[0][[0, 1, 2, 4]], names["x"][[0, 1, 2, 8]])
    want = ref.verify(target[:5], draft, torch.tensor(drafted), [0, 2, 2, 2], uniform, noise, 1.0)
    assert names["tokens"].tolist() == want[0] and names["accepted"].tolist() == want[1]
    assert caches[0].cached.tolist() == [1 + want[1][0], 0, 6] and int(caches[0].missing) == 0
