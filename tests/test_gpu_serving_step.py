"""The serving operators together, as a model's step runs them (GPU): through
the public functions, captured and replayed, on two streams, and at their
largest and smallest sizes.  Definitions and bars: serving_reference.py."""
import gc

import pytest
import torch

import serving_reference as ref
import test_gpu_serving as one
from late_interaction_retrieval_gb300 import TokenCache, binding, layers, serving

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _leave_no_garbage():
    yield
    gc.collect()


def _dev(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Model:
    """One layer and a vocabulary: embeddings to keys, values and queries, attention to logits."""

    def __init__(self, gen, heads=2, group=4, dim=64, cols=515, dtype=torch.bfloat16):
        def weight(*shape):
            return (torch.randn(*shape, generator=gen) / shape[0] ** 0.5).cuda().to(dtype)

        self.heads, self.group, self.dim, self.cols = heads, group, dim, cols
        self.embed = (torch.randn(cols, 48, generator=gen)).cuda().to(dtype)
        self.k, self.v = weight(48, heads * dim), weight(48, heads * dim)
        self.q, self.head = weight(48, heads * group * dim), weight(heads * group * dim, cols)

    def qkv(self, tokens):
        x = self.embed[tokens.clamp(min=0).long()]
        return ((x @ self.q).view(-1, self.heads * self.group, self.dim), (x @ self.k).view(-1, self.heads, self.dim),
                (x @ self.v).view(-1, self.heads, self.dim))

    def logits(self, out):
        return (out.flatten(1) @ self.head) * 4.0


def _snapshot(cache):
    return {n: getattr(cache, n).clone().cpu() for n in ("cached", "held", "free_count", "block_table", "k", "v", "k_scale",
                                                         "v_scale", "_free")}


def _check_step(model, before, cache, added, rows, q, k, v, out, lse):
    """One plan, write and attention against the definitions, from what the cache held before."""
    page = cache.page_size
    table, held, lengths, offsets, slots, left = ref.slots(
        before["cached"].tolist(), added, before["held"].tolist(), before["_free"][:-1].tolist(), int(before["free_count"]),
        before["block_table"], page, rows)
    assert torch.equal(cache.block_table.cpu(), table) and cache.held.tolist() == held
    assert cache.lengths.tolist() == lengths and cache.offsets.tolist() == offsets and cache.slots.tolist() == slots
    assert int(cache.free_count) == max(left, 0) and int(cache.missing) == max(-left, 0)
    for x, codes, scale in ((k, "k", "k_scale"), (v, "v", "v_scale")):
        want_c, want_s = ref.write(x.cpu(), torch.tensor(slots), before[codes][0], before[scale][0])
        got_c, got_s = getattr(cache, codes)[0].cpu(), getattr(cache, scale)[0].cpu()
        assert torch.equal(got_s, want_s) and one._same_codes(got_c, want_c)
    n = offsets[-1]
    want = ref.attention(q.cpu()[:n], *(getattr(cache, c)[0].cpu() for c in ("k", "v", "k_scale", "v_scale")), table, offsets,
                         lengths, model.dim ** -0.5)
    one.assert_attention((out[:n], lse[:n]), want)


@pytest.mark.parametrize("dtype,page,dim", [(torch.bfloat16, 16, 64), (torch.float16, 64, 128), (torch.float32, 32, 48)])
def test_a_model_answers_and_learns(dtype, page, dim):
    """Prompts, drafts, a request that ends and one that takes its place; then a policy step on what was sampled."""
    gen = torch.Generator().manual_seed(page)
    half = torch.bfloat16 if dtype == torch.float32 else dtype  # q is 16 bits wide
    model = Model(gen, dim=dim, dtype=dtype)
    requests, cols = 3, model.cols
    cache = TokenCache(1, model.heads, model.dim, pages=40, requests=requests, max_tokens=160, page_size=page)

    def forward(tokens, added, rows):
        before = _snapshot(cache)
        q, k, v = model.qkv(tokens)
        q = q.to(half)
        cache.plan(_dev(added), rows)
        cache.write(0, k, v)
        out, lse = cache.attention(0, q, return_lse=True, max_added=max(added))
        _check_step(model, before, cache, added, rows, q, k, v, out, lse)
        return model.logits(out.to(dtype))

    prompts = [37, 0, 70]
    tokens = torch.randint(0, cols, (sum(prompts) + 5,), generator=gen).cuda()  # 5 rows of padding
    logits = forward(tokens, prompts, tokens.shape[0])
    cache.keep(_dev(prompts))
    last = torch.tensor([36, 0, 106]).cuda()
    noise = torch.empty(requests, cols).exponential_(generator=gen).cuda()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    first, accepted, logp = serving.verify_drafts(logits[last].contiguous(), none, _dev([0, 0, 0, 0]), none.float(), noise)
    assert accepted.tolist() == [0, 0, 0]
    newest, sampled = first.clone(), []
    drafts = [3, 0, 5]
    for step in range(4):
        if step == 2:  # request 0 has ended; another takes its place with one token
            free = int(cache.free_count) + int(cache.held[0])
            cache.release(0)
            assert int(cache.free_count) == free and cache.cached.tolist()[0] == 0
            pool = cache._free[:free].tolist() + [p for p in cache.block_table.flatten().tolist() if p >= 0]
            assert sorted(pool) == list(range(40))
        n = sum(drafts)
        drafted = torch.randint(0, cols, (n,), generator=gen, dtype=torch.int32).cuda()
        draft_logits = torch.randn(n, cols, generator=gen).cuda().to(dtype)
        at = [0, 0, 0]
        packed = []
        cut = [0]
        for b in range(requests):  # each request's newest token, then its drafts
            packed += [newest[b:b + 1], drafted[cut[-1]:cut[-1] + drafts[b]]]
            cut.append(cut[-1] + drafts[b])
            at[b] = cut[b] + b
        tokens = torch.cat(packed)
        added = [d + 1 for d in drafts]
        logits = forward(tokens, added, n + requests)
        uniform = torch.rand(n, generator=gen).cuda() * (0.02 if step % 2 else 1.0)  # small: some drafts pass
        noise = torch.empty(requests, cols).exponential_(generator=gen).cuda()
        got = serving.verify_drafts(logits, drafted, _dev(cut), uniform, noise, draft_logits)
        want = ref.verify(logits.cpu(), draft_logits.cpu(), drafted.cpu(), cut, uniform.cpu(), noise.cpu(), 1.0)
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
        cache.keep(got[1] + 1)
        newest = torch.stack([got[0][at[b] + want[1][b]] for b in range(requests)])
        sampled.append((logits, got[0], got[2]))
    logits, target, old = (torch.cat(t) for t in zip(*sampled))
    logits.requires_grad_(True)
    advantage = torch.randn(target.shape[0], generator=gen).cuda()
    loss, _, logp = layers.policy_loss(logits, target, old, advantage, return_rows=True)
    loss.backward()
    there = target >= 0
    # the same logits: the ratio is 1 up to the roundings of log p = z - max - log(sum) on either side
    assert float((logp - old)[there].abs().max()) <= 2.0 ** -16
    assert bool(logits.grad.isfinite().all()) and float(logits.grad[there].abs().sum()) > 0
    assert bool((logits.grad[~there] == 0).all())


def _step_buffers(gen, requests, cols, heads=2, group=4, dim=64, page=16, rows=24):
    cache = TokenCache(1, heads, dim, pages=80, requests=requests, max_tokens=200, page_size=page)
    b = dict(q=torch.empty(rows, heads * group, dim, dtype=torch.bfloat16, device="cuda"),
             k=torch.empty(rows, heads, dim, dtype=torch.bfloat16, device="cuda"),
             v=torch.empty(rows, heads, dim, dtype=torch.bfloat16, device="cuda"),
             added=torch.zeros(requests, dtype=torch.int32, device="cuda"),
             logits=torch.empty(rows, cols, device="cuda"), draft=torch.empty(rows - requests, cols, device="cuda"),
             drafted=torch.zeros(rows - requests, dtype=torch.int32, device="cuda"),
             cut=torch.zeros(requests + 1, dtype=torch.int32, device="cuda"),
             uniform=torch.empty(rows - requests, device="cuda"), noise=torch.ones(requests, cols, device="cuda"))
    return cache, b


def _fill(gen, b, added):
    rows, requests = b["q"].shape[0], len(added)
    for n in ("q", "k", "v", "logits", "draft"):
        b[n].copy_(torch.randn(b[n].shape, generator=gen))
    b["noise"].copy_(torch.empty(b["noise"].shape).exponential_(generator=gen))
    b["uniform"].copy_(torch.rand(b["uniform"].shape, generator=gen))
    b["drafted"].copy_(torch.randint(0, b["logits"].shape[1], b["drafted"].shape, generator=gen))
    b["added"].copy_(torch.tensor(added, dtype=torch.int32))
    b["cut"].copy_(torch.tensor([0] + [a - 1 for a in added]).cumsum(0))
    assert sum(added) <= rows and min(added) >= 1 and requests == b["noise"].shape[0]


def _run(cache, b, most):
    cache.plan(b["added"], b["q"].shape[0])
    cache.write(0, b["k"], b["v"])
    out, lse = cache.attention(0, b["q"], return_lse=True, max_added=most, out=b["q"].new_zeros(b["q"].shape))
    tokens, accepted, logp = serving.verify_drafts(b["logits"], b["drafted"], b["cut"], b["uniform"], b["noise"], b["draft"])
    cache.keep(accepted + 1)
    return out, lse, tokens, accepted, logp


@pytest.mark.parametrize("most", [2, 40])  # the kernel for few rows and the one for many
def test_a_captured_step_is_replayed_with_other_lengths(most):
    requests, cols = 4, 301
    steps = [[1, 1, 1, 1], [6, 1, 9, 8], [1, 20, 2, 1], [2, 2, 3, 1], [3, 3, 3, 3]]
    results = []
    for captured in (False, True):
        gen = torch.Generator().manual_seed(5)
        cache, b = _step_buffers(gen, requests, cols)
        if captured:  # on an empty step first: what capture needs once is done
            _fill(gen, b, steps[0])
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            state = _snapshot(cache)
            with torch.cuda.stream(side):
                _run(cache, b, most)
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                held = _run(cache, b, most)
            for n, t in state.items():
                getattr(cache, n).view(torch.uint8).copy_(t.view(torch.uint8))
            gen = torch.Generator().manual_seed(5)
        got = []
        for added in steps:
            _fill(gen, b, added)
            if captured:
                graph.replay()
                result = held
            else:
                result = _run(cache, b, most)
            n = sum(added)
            got.append([t[:n].clone() if t.shape[0] == b["q"].shape[0] else t.clone() for t in result])
        binding.lik_check_device_error()
        got.append([cache.k.view(torch.uint8).clone(), cache.k_scale.clone(), cache.block_table.clone(), cache.cached.clone()])
        results.append(got)
    for eager, replayed in zip(*results):
        for x, y in zip(eager, replayed):
            assert torch.equal(x, y)


@pytest.mark.parametrize("added", [[1] * 9, [5, 1, 2, 130, 1, 1, 7, 1, 64]])
def test_two_streams_with_a_workspace_each(added):
    gen = torch.Generator().manual_seed(11)
    lengths = [a + 17 * i for i, a in enumerate(added)]
    cases = [one._requests(gen, lengths, added, 2, 4, 128, 64, "bf16") for _ in range(2)]
    alone = [one.run_attention(*c, 0.1) for c in cases]
    verify = [one._drafts(gen, [3, 0, 2], 4099, "bf16") for _ in range(2)]
    alone_v = [one.run_verify(*c) for c in verify]
    args = []
    for q, kc, vc, ks, vs, table, offsets, length in cases:
        args.append([t.cuda() for t in (q, kc, vc, ks, vs, table)] + [_dev(offsets), _dev(length)])
    v_args = [[t.cuda() for t in (c[0], c[2])] + [_dev(c[3])] + [t.cuda() for t in (c[4], c[5], c[1])] for c in verify]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append((serving.cache_attention(*args[i], scale=0.1, max_added=max(added)),
                                serving.verify_drafts(*v_args[i])))
    torch.cuda.synchronize()
    binding.lik_check_device_error()
    for i in range(2):
        for out, (tokens, accepted, logp) in outs[i]:
            assert torch.equal(out, alone[i][0])
            assert tokens.tolist() == alone_v[i][0] and torch.equal(logp.cpu(), alone_v[i][2])


def test_most_requests():
    """8192 requests: single tokens, some of them empty, over a page or none."""
    gen = torch.Generator().manual_seed(3)
    n = 8192
    added = [int(i % 97 != 0) for i in range(n)]
    lengths = [int(x) for x in torch.randint(1, 20, (n,), generator=gen)]
    case = one._requests(gen, lengths, added, 1, 2, 16, 16, "f16")
    q, kc, vc, ks, vs, table, offsets, _ = case
    got = one.run_attention(*case, 0.25)
    some = sorted({0, 1, 2, 96, 97, 98, 4095, 4096, 8190, 8191} | set(torch.randint(0, n, (150,), generator=gen).tolist()))
    for b in some:
        lo, hi = offsets[b], offsets[b + 1]
        want = ref.attention(q[lo:hi], kc, vc, ks, vs, table[b:b + 1], [0, hi - lo], [lengths[b]], 0.25)
        one.assert_attention((got[0][lo:hi], got[1][lo:hi]), want)
    assert bool(got[0].isfinite().all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,group,dim,page,lengths,added", [
    (1, 4, 64, 64, [200, 300, 3], [200, 150, 3]), (2, 1, 128, 128, [260, 129, 1], [257, 129, 1]),
    (1, 8, 128, 64, [150, 64, 65], [150, 1, 17]), (1, 128, 64, 256, [70, 2], [3, 1]), (1, 3, 96, 64, [400], [390])])
def test_prompts_of_many_rows(dtype, heads, group, dim, page, lengths, added):
    gen = torch.Generator().manual_seed(dim + page)
    one.check_attention(one._requests(gen, lengths, added, heads, group, dim, page, dtype))


@pytest.mark.parametrize("seed,dtype", [(0, "bf16"), (1, "f16"), (2, "bf16")])
def test_ragged_batches(seed, dtype):
    """Prompts, drafts, single and no tokens in one batch, which no two blocks cut alike."""
    gen = torch.Generator().manual_seed(100 + seed)
    heads, group, dim, page = [(2, 5, 64, 64), (1, 7, 128, 32), (3, 2, 48, 128)][seed]
    added = [int(x) for x in torch.randint(0, 70, (11,), generator=gen)] + [1, 0, 1, 5]
    lengths = [a + int(x) for a, x in zip(added, torch.randint(0, 400, (15,), generator=gen))]
    one.check_attention(one._requests(gen, lengths, added, heads, group, dim, page, dtype))


@pytest.mark.parametrize("dtype,heads,dim,page", [("f32", 1, 128, 256), ("f32", 2, 80, 128), ("bf16", 1, 128, 256),
                                                  ("f16", 1, 112, 256)])
@pytest.mark.parametrize("apart", [False, True])
def test_write_long_runs(dtype, heads, dim, page, apart):
    """Runs longer than what a block's shared memory holds, and rows that allow no 16-byte loads."""
    gen = torch.Generator().manual_seed(dim)
    slot = [2 * page + i for i in range(page)] + [page + 7 + i for i in range(page - 7)] + [-1] + [3 * page + i for i in range(130)]
    shape = (len(slot), heads, dim + 1) if apart else (len(slot), heads, dim)
    x, y = ((torch.randn(shape, generator=gen) * 3).to(one.DT[dtype]).cuda()[..., :dim] for _ in range(2))
    y[::9, :, ::7] = float("inf")
    x[5] = NAN
    one.check_write(x, y, slot, *one._pair(gen, 5, heads, page, dim))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_write_many_short_runs(dtype):
    """A large batch of single tokens and drafts: more rows than a block of its own each."""
    gen = torch.Generator().manual_seed(8)
    page, pages = 16, 4000
    order = torch.randperm(pages, generator=gen).tolist()
    slot = []
    while len(slot) < 9000:
        p, o = order.pop(), int(torch.randint(0, page, (1,), generator=gen))
        slot += [p * page + o + i for i in range(min(page - o, 1 + len(order) % 7))]
    x, y = (torch.randn(len(slot), 1, 32, generator=gen).to(one.DT[dtype]) for _ in range(2))
    one.check_write(x, y, slot, *one._pair(gen, pages, 1, page, 32))


@pytest.mark.parametrize("onehot", [False, True])
def test_many_drafts_of_a_request(onehot):
    gen = torch.Generator().manual_seed(21)
    case = list(one._drafts(gen, [130, 0, 66, 1], 211, "f32", onehot))
    case[4] = case[4] * 0.01  # long runs of drafts pass
    _, accepted = one.check_verify(tuple(case))
    assert max(accepted) > 64 or onehot


def test_pages_that_run_out():
    cache = TokenCache(1, 1, 16, pages=3, requests=2, max_tokens=64, page_size=16)
    cache.plan(_dev([40, 30]), 70)
    assert int(cache.missing) == 2 and int(cache.free_count) == 0 and cache.held.tolist() == [3, 0]
    assert cache.slots.tolist()[40:] == [-1] * 30
    k = torch.ones(70, 1, 16, device="cuda", dtype=torch.float16)
    cache.write(0, k, k)
    out, lse = cache.attention(0, k, return_lse=True, max_added=40)
    assert bool((out[40:] == 0).all()) and bool((lse[40:] == -float("inf")).all())
    assert float((out[:40].float() - 1).abs().max()) <= 2.0 ** -10
    cache.release(0)
    assert int(cache.free_count) == 3 and sorted(cache._free[:3].tolist()) == [0, 1, 2]


def test_calls_that_are_refused():
    cache = TokenCache(1, 2, 32, pages=4, requests=2, max_tokens=32, page_size=16)
    added = _dev([1, 1])
    cache.plan(added, 2)
    q = torch.zeros(2, 4, 32, device="cuda", dtype=torch.bfloat16)
    for bad in (q.cpu(), q[..., :16], q[:, :3], q.float(), q.to(torch.float64), q[0], q.transpose(0, 2)):
        with pytest.raises((ValueError, binding.LIKError)):
            cache.attention(0, bad)
    with pytest.raises(binding.LIKError):
        cache.attention(0, q, out=q)
    with pytest.raises(binding.LIKError):
        cache.attention(0, q, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        cache.write(0, q[:, :2], q[:, :2].float())
    with pytest.raises(ValueError):
        cache.write(0, q[:1, :2], q[:1, :2])  # slots were planned for two rows
    with pytest.raises(ValueError):
        cache.plan(added.long(), 2)
    with pytest.raises(ValueError):
        serving.verify_drafts(torch.zeros(3, 8, device="cuda"), added[:0], _dev([0, 0]), torch.zeros(0, device="cuda"),
                              torch.ones(1, 8, device="cuda"))
