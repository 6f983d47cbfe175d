"""The serving operators over the 8-bit cache (GPU) against their plain
definitions (serving_reference.py, which also derives the bars)."""
import gc
import math

import pytest
import torch

import serving_reference as ref
from late_interaction_retrieval_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _leave_no_garbage():
    yield
    gc.collect()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


# ------------------------------------------------------------------- slots --

def run_slots(cached, added, held, free, count, table, page, capacity):
    n = len(cached)
    d = dict(device="cuda")
    full = torch.full((table.shape[0], table.shape[1] + 3), -77, dtype=torch.int32, **d)  # rows further apart
    full[:, :table.shape[1]] = table.cuda()
    held_out, lengths = (torch.full((n,), -9, dtype=torch.int32, **d) for _ in range(2))
    offsets, left = torch.full((n + 1,), -9, dtype=torch.int32, **d), torch.full((1,), -9, dtype=torch.int32, **d)
    slots = torch.full((capacity,), -9, dtype=torch.int64, **d)
    view = full[:, :table.shape[1]]
    binding.lik_cache_slots(_i32(cached).cuda(), _i32(added).cuda(), _i32(held).cuda(), _i32(free).cuda(),
                            _i32([count]).cuda(), view, held_out, lengths, offsets, slots, left, page_size=page)
    assert bool((full[:, table.shape[1]:] == -77).all()), "the gap between the table's rows was written"
    return view.cpu(), held_out.tolist(), lengths.tolist(), offsets.tolist(), slots.tolist(), int(left)


def check_slots(cached, added, held, free, count, table, page, capacity):
    got = run_slots(cached, added, held, free, count, table, page, capacity)
    want = ref.slots(cached, added, held, free, count, table, page, capacity)
    assert torch.equal(got[0], want[0])
    assert list(got[1:]) == list(want[1:])


def _batch(gen, n, most_cached, most_added, page, cols, extra=0.2):
    cached = torch.randint(0, most_cached + 1, (n,), generator=gen).tolist()
    added = torch.randint(0, most_added + 1, (n,), generator=gen).tolist()
    held = [-(-c // page) + int(torch.rand(1, generator=gen) < extra) for c in cached]
    pool = torch.randperm(8 * n * cols + 64, generator=gen).tolist()
    table = torch.full((n, cols), -1, dtype=torch.int32)
    for b in range(n):
        for j in range(min(held[b], cols)):
            table[b, j] = pool.pop()
    return cached, added, held, pool[:4 * n * cols + 16], table


@pytest.mark.parametrize("n,most_cached,most_added,page", [(1, 0, 1, 16), (1, 100, 100, 16), (7, 300, 1, 64),
                                                           (33, 50, 40, 32), (512, 90, 5, 16), (513, 90, 5, 16),
                                                           (1500, 20, 3, 128), (3, 5000, 9000, 256)])
def test_slots(n, most_cached, most_added, page):
    gen = _gen(n + page)
    cols = -(-(most_cached + most_added) // page) + 2
    cached, added, held, free, table = _batch(gen, n, most_cached, most_added, page, cols)
    check_slots(cached, added, held, free, len(free), table, page, sum(added) + 11)


def test_slots_most_requests():
    gen = _gen(5)
    cached, added, held, free, table = _batch(gen, 8192, 40, 2, 16, 5)
    check_slots(cached, added, held, free, len(free), table, 16, sum(added))


def test_slots_no_request():
    got = run_slots([], [], [], [3, 4], 2, torch.zeros((0, 4), dtype=torch.int32), 16, 5)
    assert got[3] == [0] and got[4] == [-1] * 5 and got[5] == 2


def test_slots_out_of_pages():
    """The list runs out inside a request: what is there is given in order, the rest is -1 and counted."""
    table = torch.full((4, 8), -1, dtype=torch.int32)
    check_slots([0, 0, 0, 0], [40, 40, 1, 40], [0, 0, 0, 0], [10, 11, 12, 13, 14], 5, table, 16, 130)
    check_slots([0, 0], [33, 1], [0, 0], [10, 11], 0, table[:2].clone(), 16, 40)


def test_slots_clamped():
    """Lengths below 0, tables that are too narrow, more pages held than columns, a list length out of range, fewer
    slots than tokens, a page that was never given."""
    table = torch.arange(20, dtype=torch.int32).reshape(4, 5)
    table[1, 2] = -1
    check_slots([-5, 40, 70, 3], [10, 30, 40, -2], [0, 4, 9, -1], [90, 91, 92], 7, table, 16, 60)
    check_slots([-5, 40, 70, 3], [10, 30, 40, -2], [0, 4, 9, -1], [90, 91, 92], -3, table, 16, 200)
    check_slots([2 ** 31 - 1, 4], [2 ** 31 - 1, 2 ** 31 - 1], [0, 0], [1], 1, table[:2].clone(), 256, 300)


def test_slots_refusals():
    i = _i32([1, 2]).cuda()
    one, table, slots = _i32([1]).cuda(), torch.zeros((2, 4), dtype=torch.int32, device="cuda"), \
        torch.zeros(4, dtype=torch.int64, device="cuda")

    def call(cached=i, held_out=None, page=16, left=None, free=i):
        binding.lik_cache_slots(cached, i, i, free, one, table, i.clone() if held_out is None else held_out, i.clone(),
                                _i32([0, 0, 0]).cuda(), slots, one.clone() if left is None else left, page_size=page)

    call()
    for bad in (dict(page=24), dict(page=512), dict(held_out=i), dict(left=one), dict(held_out=table.view(-1)[2:4])):
        with pytest.raises(binding.LIKError):
            call(**bad)
    with pytest.raises(ValueError):
        call(cached=i.long())
    with pytest.raises(ValueError):
        call(free=i.cpu())


# ------------------------------------------------------------------- write --

def _cache(gen, pages, heads, page, dim, nan=True):
    raw = torch.randint(0, 256, (pages, heads, page, dim), generator=gen, dtype=torch.uint8)
    if not nan:
        raw = torch.where((raw & 127) == 127, raw - 1, raw)
    return raw.view(F8), (torch.rand(pages, heads, generator=gen) + 0.01) * 0.02


def _same_codes(x, y):
    """Codes are equal, bit for bit; a NaN code of either sign is a NaN."""
    x, y = x.view(torch.uint8), y.view(torch.uint8)
    nan = ((x & 127) == 127) & ((y & 127) == 127)
    return bool(((x == y) | nan).all())


def check_write(x, y, slot, kc, vc, ks, vs):
    dev = [t.cuda() for t in (kc, vc, ks, vs)]
    binding.lik_cache_write(x.cuda() if not x.is_cuda else x, y.cuda() if not y.is_cuda else y,
                            torch.tensor(slot, dtype=torch.int64).cuda(), *dev)
    slot = torch.tensor(slot, dtype=torch.int64)
    for t, c, s, got_c, got_s in ((x.cpu(), kc, ks, dev[0], dev[2]), (y.cpu(), vc, vs, dev[1], dev[3])):
        want_c, want_s = ref.write(t, slot, c, s)
        assert torch.equal(got_s.cpu(), want_s)
        assert _same_codes(got_c.cpu(), want_c)


def _runs(gen, pages, page, count, full):
    """Slots of runs in distinct pages: from any offset, or whole pages of one long sequence."""
    order = torch.randperm(pages, generator=gen).tolist()
    slot = []
    for p in order[:count]:
        o = 0 if full else int(torch.randint(0, page, (1,), generator=gen))
        n = page if full else int(torch.randint(1, page - o + 1, (1,), generator=gen))
        slot += [p * page + o + i for i in range(n)]
        if not full and torch.rand(1, generator=gen) < 0.3:
            slot += [-1]
    return slot


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,dim,page,count,full", [(1, 16, 16, 3, False), (8, 128, 64, 5, False), (2, 80, 32, 9, True),
                                                       (3, 96, 128, 4, False), (1, 128, 256, 3, True),
                                                       (2, 64, 16, 600, True)])
def test_write(dtype, heads, dim, page, count, full):
    gen = _gen(dim + page)
    pages = count + 3
    slot = _runs(gen, pages, page, count, full)
    x, y = ((torch.randn(len(slot), heads, dim, generator=gen) * 3).to(DT[dtype]) for _ in range(2))
    y[::5] *= 8
    check_write(x, y, slot, *_pair(gen, pages, heads, page, dim))


def _pair(gen, pages, heads, page, dim):
    kc, ks = _cache(gen, pages, heads, page, dim)
    vc, vs = _cache(gen, pages, heads, page, dim)
    return kc, vc, ks, vs


def test_write_single_tokens():
    """One token a request, into every offset; scales that grow and scales that do not."""
    gen = _gen(3)
    slot = [p * 32 + p for p in range(32)]
    x = torch.randn(32, 4, 64, generator=gen) * torch.exp(2 * torch.randn(32, 4, 1, generator=gen))
    check_write(x, -x, slot, *_pair(gen, 32, 4, 32, 64))


def test_write_step_after_step():
    """A page filled token by token holds what one filled at once does, up to its requantisations."""
    gen = _gen(4)
    x = torch.randn(16, 2, 32, generator=gen)
    kc, vc, ks, vs = (t.cuda() for t in _pair(gen, 2, 2, 16, 32))
    for t in range(16):
        binding.lik_cache_write(x[t:t + 1].cuda(), x[t:t + 1].cuda(), torch.tensor([16 + t]).cuda(), kc, vc, ks, vs)
    size = x.abs().amax(dim=(0, 2))
    assert torch.equal(ks.cpu()[1], size / torch.full_like(size, 448.0))
    got = kc.cpu()[1].float() * ks.cpu()[1][:, None, None]
    # each requantisation is off by half a step (2^-4 of the value, 2^-10 of the scale below the normal codes);
    # at most 16 of them, one for each step
    off = (got - x.transpose(0, 1)).abs()
    assert bool((off <= 16 * (2.0 ** -4 * x.transpose(0, 1).abs() + 2.0 ** -10 * ks.cpu()[1][:, None, None])).all())
    assert torch.equal(kc.cpu()[1].view(torch.uint8), vc.cpu()[1].view(torch.uint8))


def test_write_values():
    """Zeros, the smallest and largest values, infinities and NaN (as NaN codes, no part of the scale)."""
    gen = _gen(6)
    x = torch.randn(16, 2, 16, generator=gen)
    x[0], x[1, 0, 3], x[2, 1, 5], x[3, 0, 0] = 0.0, INF, NAN, -INF
    x[8:12, :, :] = 1e-44
    y = torch.zeros(16, 2, 16)
    y[5] = 3.4e38
    slot = list(range(16, 24)) + list(range(48, 56))
    check_write(x, y, slot, *_pair(gen, 4, 2, 16, 16))


def test_write_no_slot():
    """Slots outside the cache write nothing."""
    gen = _gen(7)
    x = torch.randn(9, 2, 16, generator=gen)
    check_write(x, x, [-1, 64, 5, 6, 2 ** 40, -2 ** 60, 63, 64, 65], *_pair(gen, 4, 2, 16, 16))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_write_strides(dtype):
    """Keys and values as slices of one projection; heads before rows; rows at any address."""
    gen = _gen(8)
    slot = list(range(3, 16)) + list(range(32, 48)) + [-1]
    n = len(slot)
    fused = torch.randn(n, 3, 4, 32, generator=gen).to(DT[dtype]).cuda()
    check_write(fused[:, 1, :2], fused[:, 2, :2], slot, *_pair(gen, 4, 2, 16, 32))
    swapped = torch.randn(2, n, 32, generator=gen).to(DT[dtype]).cuda()
    check_write(swapped.transpose(0, 1), swapped.transpose(0, 1), slot, *_pair(gen, 4, 2, 16, 32))
    odd = torch.randn(n, 2, 33, generator=gen).to(DT[dtype]).cuda()
    check_write(odd[:, :, 1:], odd[:, :, :32], slot, *_pair(gen, 4, 2, 16, 32))
    check_write(odd[:, :1, 1:].expand(n, 2, 32), odd[:, :, :32], slot, *_pair(gen, 4, 2, 16, 32))


def test_write_refusals():
    gen = _gen(9)
    kc, vc, ks, vs = (t.cuda() for t in _pair(gen, 4, 2, 16, 16))
    x, slot = torch.randn(3, 2, 16, device="cuda"), torch.tensor([0, 1, 2], device="cuda")
    binding.lik_cache_write(x, x, slot, kc, vc, ks, vs)
    for bad in ((kc, kc, ks, vs), (kc, vc, ks, ks)):
        with pytest.raises(binding.LIKError):
            binding.lik_cache_write(x, x, slot, *bad)
    with pytest.raises(ValueError):
        binding.lik_cache_write(x, x, slot.int(), kc, vc, ks, vs)
    with pytest.raises(ValueError):
        binding.lik_cache_write(x[:, :1], x[:, :1], slot, kc, vc, ks, vs)
    with pytest.raises(ValueError):
        binding.lik_cache_write(x, x.half(), slot, kc, vc, ks, vs)
    small = torch.randn(3, 2, 24, device="cuda")
    with pytest.raises(binding.LIKError):
        binding.lik_cache_write(small, small, slot, *(torch.zeros(4, 2, 16, 24, device="cuda").to(F8) for _ in range(2)),
                                ks, vs)


# --------------------------------------------------------------- attention --

def _requests(gen, lengths, added, heads, group, dim, page, dtype, spare=3):
    """Tables, packed rows and a cache whose unused codes and scales are NaN."""
    n = len(lengths)
    held = [-(-x // page) for x in lengths]
    pages, cols = sum(held) + spare, max(held + [0]) + 1
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((n, cols), -1, dtype=torch.int32)
    kc, ks = _cache(gen, pages, heads, page, dim, nan=False)
    vc, vs = _cache(gen, pages, heads, page, dim, nan=False)
    kr, vr = kc.view(torch.uint8), vc.view(torch.uint8)
    used = set()
    for b in range(n):
        for j in range(held[b]):
            p = order.pop()
            table[b, j] = p
            used.add(p)
            tail = lengths[b] - j * page
            if tail < page:
                kr[p, :, tail:], vr[p, :, tail:] = 0x7F, 0xFF
    for p in range(pages):
        if p not in used:
            kr[p], vr[p], ks[p], vs[p] = 0x7F, 0x7F, NAN, NAN
    offsets = [0]
    for a in added:
        offsets.append(offsets[-1] + a)
    q = (torch.randn(offsets[-1], heads * group, dim, generator=gen) * 1.5).to(DT[dtype])
    return q, kc, vc, ks, vs, table, offsets, list(lengths)


def run_attention(q, kc, vc, ks, vs, table, offsets, lengths, scale, max_added=None, out=None, lse=True, ws=None):
    d = [t.cuda() for t in (kc, vc, ks, vs)]
    q = q if q.is_cuda else q.cuda()
    table = table if table.is_cuda else table.cuda()
    out = torch.full_like(q, NAN) if out is None else out
    l = torch.full(q.shape[:2], NAN, device="cuda") if lse else None
    if max_added is None:
        max_added = max([b - a for a, b in zip(offsets, offsets[1:])] + [0])
    need = binding.lik_cache_attention_workspace_bytes(q, d[0], table, max_added=max_added)
    ws = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
    binding.lik_cache_attention(q, *d, table, _i32(offsets).cuda(), _i32(lengths).cuda(), out, l, workspace=ws,
                                max_added=max_added, scale=scale)
    binding.lik_check_device_error()
    assert bool((ws[need:] == 0xFF).all()), "written behind the workspace"
    return out, l


def assert_attention(got, want):
    out, lse = got
    w_out, w_lse, out_bar, lse_bar = want
    out = out.cpu().double()
    assert torch.equal(out.isnan(), w_out.isnan())
    fine = w_out.isfinite()  # where it is not, the value itself is expected (and has no bar)
    assert torch.equal(out == INF, w_out == INF) and torch.equal(out == -INF, w_out == -INF)
    off, bar = (out - w_out)[fine].abs(), out_bar[fine]
    assert bool((off <= bar).all()), f"out is off by {float((off / bar.clamp(min=1e-300)).max()):.2f} bars"
    if lse is not None:
        lse = lse.cpu().double()
        assert torch.equal(lse.isnan(), w_lse.isnan()) and torch.equal(lse == -INF, w_lse == -INF)
        fine = w_lse.isfinite()
        off = (lse - w_lse)[fine].abs()
        assert bool((off <= lse_bar[fine]).all()), f"lse is off by {float((off / lse_bar[fine]).max()):.2f} bars"


def check_attention(case, scale=None, **kw):
    scale = case[0].shape[2] ** -0.5 if scale is None else scale
    got = run_attention(*case, scale, **kw)
    assert_attention(got, ref.attention(*case, scale))
    return got


# one token; lengths around a unit and a page; empty requests; several units a warp
ONE = [([1], [1]), ([31, 32, 33], [1, 1, 1]), ([0, 5, 64], [0, 1, 1]), ([600, 17, 1, 255, 256, 257], [1] * 6),
       ([1300], [1]), ([9, 0, 40], [1, 1, 1])]
# drafts and prompts: rows that fill a tile of 16 and pass it
MANY = [([5], [5]), ([40, 7], [5, 3]), ([100, 0, 33], [17, 0, 33]), ([300], [130]), ([64, 64, 64], [64, 1, 2]),
        ([3, 260], [5, 9])]
SHAPES = [(1, 1, 16, 16), (2, 4, 128, 64), (4, 1, 64, 16), (2, 7, 80, 32), (1, 8, 128, 256), (1, 16, 96, 16),
          (1, 20, 48, 128)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,group,dim,page", SHAPES)
def test_attention_single_tokens(dtype, heads, group, dim, page):
    for i, (lengths, added) in enumerate(ONE):
        check_attention(_requests(_gen(i + dim), lengths, added, heads, group, dim, page, dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,group,dim,page", SHAPES)
def test_attention_several_tokens(dtype, heads, group, dim, page):
    for i, (lengths, added) in enumerate(MANY):
        check_attention(_requests(_gen(i + 7 * dim), lengths, added, heads, group, dim, page, dtype))


@pytest.mark.parametrize("hint", [0, 1, 5, 1000])
def test_attention_hint_changes_nothing_but_time(hint):
    case = _requests(_gen(1), [50, 300, 4, 0], [5, 40, 1, 0], 2, 4, 64, 16, "bf16")
    check_attention(case, max_added=hint)


def test_attention_split_along_the_cache():
    """One request over every block of the chip: cut at any unit, joined in order; twice the same bits."""
    case = _requests(_gen(2), [20011], [1], 1, 4, 64, 64, "f16")
    a, b = (run_attention(*case, 0.125) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert_attention(a, ref.attention(*case, 0.125))
    check_attention(_requests(_gen(3), [15000, 3, 9000, 1], [1, 1, 1, 1], 2, 2, 128, 16, "bf16"))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_strides(dtype):
    """q as a slice of a fused projection at an odd address, out with heads before rows, a wide table."""
    q, kc, vc, ks, vs, table, offsets, lengths = case = _requests(_gen(4), [70, 33], [3, 1], 2, 3, 48, 16, dtype)
    want = ref.attention(*case, 0.2)
    for pad, wide in ((1, 0), (3, 1), (16, 8)):
        big = torch.full((4, 6, 48 + pad), NAN, dtype=DT[dtype], device="cuda")
        big[:, :, pad:] = q.cuda()
        out = torch.full((6, 4, 48 + wide), NAN, dtype=DT[dtype], device="cuda")
        t = torch.full((2, table.shape[1] + 5), 10 ** 9, dtype=torch.int32, device="cuda")
        t[:, :table.shape[1]] = table.cuda()
        got = run_attention(big[:, :, pad:], kc, vc, ks, vs, t[:, :table.shape[1]], offsets, lengths, 0.2,
                            out=out[:, :, :48].transpose(0, 1))
        assert_attention(got, want)
        assert bool(out[:, :, 48:].isnan().all())
    assert_attention(run_attention(*case, 0.2, lse=False), want)


def test_attention_rows_of_no_request_stay():
    q, kc, vc, ks, vs, table, offsets, lengths = case = _requests(_gen(5), [20, 9], [2, 1], 1, 2, 32, 16, "bf16")
    padded = torch.cat([q, torch.full((5, 2, 32), NAN, dtype=q.dtype)])
    out, lse = run_attention(padded, kc, vc, ks, vs, table, offsets, lengths, 0.3)
    assert bool(out[3:].isnan().all()) and bool(lse[3:].isnan().all())
    assert_attention((out[:3], lse[:3]), ref.attention(*case, 0.3))


@pytest.mark.parametrize("page", [16, 32, 128])
def test_attention_hidden_pages(page):
    """Entries outside the pool hide their tokens, at the front, inside and behind."""
    case = _requests(_gen(6), [300, 200, 40], [1, 4, 2], 2, 2, 64, page, "f16")
    table = case[5]
    table[0, 0] = -1
    table[0, -2] = 2 ** 31 - 1
    table[1, 1] = case[1].shape[0]
    table[2] = -5
    check_attention(case)


def test_attention_nan_of_tokens_that_a_row_does_not_see():
    """Rows before a drafted token are not touched by its NaN codes or its page's scale; rows behind have them."""
    for page, group in ((16, 2), (64, 8), (64, 1)):
        q, kc, vc, ks, vs, table, offsets, lengths = case = _requests(_gen(7), [48 + 5, 30], [5, 2], 1, group, 64, page,
                                                                      "bf16")
        p, o = int(table[0, 50 // page]), 50 % page
        vc.view(torch.uint8)[p, 0, o, 7] = 0x7F
        kc.view(torch.uint8)[p, 0, o + 1, 9] = 0xFF
        want = ref.attention(*case, 0.125)
        assert not bool(want[0][:2].isnan().any()) and bool(want[0][4].isnan().all())
        got = run_attention(*case, 0.125)
        assert_attention((got[0], None), want)
    # the last token opens a page whose scales are not finite
    for bad, group in ((NAN, 2), (INF, 2), (NAN, 20), (INF, 20)):
        q, kc, vc, ks, vs, table, offsets, lengths = case = _requests(_gen(8), [33, 12], [2, 1], 1, group, 64, 16, "f16")
        vs[int(table[0, 2]), 0] = bad
        got = run_attention(*case, 0.125)
        want = ref.attention(*case, 0.125)
        assert_attention((got[0][[0, 2]], got[1]), (want[0][[0, 2]], want[1], want[2][[0, 2]], want[3]))
        assert not bool(got[0][1].isfinite().any())


def test_attention_sizes_of_numbers():
    """Queries far from 1, scales that differ between pages by many powers of two, sharp and flat softmaxes."""
    for i, (size, spread, scale) in enumerate([(1e-6, 0.0, 1e3), (3e4, 0.0, 1e-4), (1.0, 12.0, 0.1), (1.0, 3.0, 30.0),
                                               (2.0, 0.0, 1e-20)]):
        q, kc, vc, ks, vs, table, offsets, lengths = case = _requests(_gen(9 + i), [500, 90], [1, 3], 2, 3, 64, 16,
                                                                      "f16" if size < 1e5 else "bf16")
        case = list(case)
        case[0] = (q.float() * size / 4).to(q.dtype)
        case[4] = vs * torch.exp(spread * torch.randn(vs.shape, generator=_gen(1)))
        check_attention(case, scale=scale)
    # a zero row, a page of zero scale, all scales 0
    q, kc, vc, ks, vs, table, offsets, lengths = case = _requests(_gen(20), [100, 20], [1, 1], 1, 2, 32, 16, "bf16")
    q[0, 0] = 0.0
    vs[int(table[0, 2])] = 0.0
    ks[int(table[0, 3])] = 0.0
    check_attention(case)
    vs[:] = 0.0
    got = run_attention(*case, 0.1)
    assert bool((got[0] == 0).all())


def test_attention_long_tail():
    """A hundred thousand tokens that together weigh as much as one peak: none of them is lost to rounding."""
    n = 100_000
    q, kc, vc, ks, vs, table, offsets, lengths = case = _requests(_gen(30), [n], [1], 1, 1, 16, 256, "f16")
    kr, vr = kc.view(torch.uint8), vc.view(torch.uint8)
    ks[:], vs[:] = 1.0, 1.0
    kc.copy_(torch.zeros(kc.shape).to(F8))
    vc.copy_(torch.ones(vc.shape).to(F8))
    p = int(table[0, 100])
    kc[p, 0, 5] = torch.full((16,), 1.0).to(F8)
    vc[p, 0, 5] = torch.full((16,), -1.0).to(F8)
    kr[int(table[0, -2]), :, n % 256:], vr[int(table[0, -2]), :, n % 256:] = 0x7F, 0x7F
    case = (torch.full((1, 1, 16), math.log(n) / 16, dtype=torch.float16),) + case[1:]
    check_attention(case, scale=1.0)


def test_attention_far_pages():
    """Pages whose codes lie beyond 2^32 bytes of the cache's start."""
    pages, heads, page, dim = 70_000, 8, 64, 128
    kc = torch.zeros(pages, heads, page, dim, dtype=torch.uint8, device="cuda").view(F8)
    vc = torch.zeros_like(kc)
    ks, vs = (torch.full((pages, heads), 0.01, device="cuda") for _ in range(2))
    gen = _gen(31)
    far = [69_999, 0, 35_000, 65_537]
    small = [_cache(gen, 4, heads, page, dim, nan=False)[0] for _ in range(2)]
    at = torch.tensor(far, device="cuda")
    kc.view(torch.uint8)[at], vc.view(torch.uint8)[at] = (x.view(torch.uint8).cuda() for x in small)
    q = torch.randn(2, 16, dim, generator=gen).half()
    out, lse = torch.full_like(q, NAN).cuda(), torch.empty(2, 16, device="cuda")
    table = _i32([far[:3], [far[3], 0, 0]]).cuda()
    ws = torch.empty(binding.lik_cache_attention_workspace_bytes(q.cuda(), kc, table, 1), dtype=torch.uint8, device="cuda")
    binding.lik_cache_attention(q.cuda(), kc, vc, ks, vs, table, _i32([0, 1, 2]).cuda(), _i32([180, 64]).cuda(), out, lse,
                                workspace=ws, max_added=1, scale=0.09)
    binding.lik_check_device_error()
    one = torch.full((4, heads), 0.01)
    assert_attention((out, lse), ref.attention(q, *small, one, one, _i32([[0, 1, 2], [3, 0, 0]]), [0, 1, 2], [180, 64], 0.09))
    slot = torch.tensor([69_998 * 64 + i for i in range(64)], device="cuda")
    x = torch.randn(64, heads, dim, generator=gen).cuda()
    binding.lik_cache_write(x, x, slot, kc, vc, ks, vs)
    want = ref.write(x.cpu(), torch.arange(64), torch.zeros(1, heads, page, dim).to(F8), torch.ones(1, heads))
    assert torch.equal(kc[69_998].cpu().view(torch.uint8), want[0][0].view(torch.uint8))
    assert torch.equal(ks[69_998].cpu(), want[1][0])


def test_attention_refusals():
    q, kc, vc, ks, vs, table, offsets, lengths = _requests(_gen(40), [20], [1], 2, 2, 32, 16, "f16")
    d = dict(q=q.cuda(), kc=kc.cuda(), vc=vc.cuda(), ks=ks.cuda(), vs=vs.cuda(), table=table.cuda(), scale=0.1)
    off, n = _i32(offsets).cuda(), _i32(lengths).cuda()
    ws = torch.empty(1 << 23, dtype=torch.uint8, device="cuda")

    def call(out=None, ws=ws, **kw):
        e = dict(d, **kw)
        out = torch.empty_like(e["q"]) if out is None else out
        binding.lik_cache_attention(e["q"], e["kc"], e["vc"], e["ks"], e["vs"], e["table"], off, n, out, workspace=ws,
                                    scale=e["scale"])

    call()
    for bad in (dict(ws=None), dict(ws=ws[:64]), dict(ws=ws[1:]), dict(scale=0.0), dict(scale=NAN), dict(q=d["q"].float()),
                dict(q=d["q"][:, :3]), dict(out=d["q"])):
        with pytest.raises(binding.LIKError):
            call(**bad)
    for bad in (dict(q=d["q"].double()), dict(kc=d["kc"].float()), dict(ks=d["ks"].half()), dict(table=d["table"].long()),
                dict(out=torch.empty(1, 4, 31, device="cuda").half()), dict(q=d["q"].cpu())):
        with pytest.raises(ValueError):
            call(**bad)


# ------------------------------------------------------------------ verify --

def _logits(gen, rows, cols, dtype, peak=6.0):
    z = torch.randn(rows, cols, generator=gen) * 1.5
    z.scatter_add_(1, torch.randint(0, cols, (rows, 8), generator=gen), peak + torch.randn(rows, 8, generator=gen))
    return z.to(DT[dtype])


def _drafts(gen, counts, cols, dtype, onehot=False):
    n, requests = sum(counts), len(counts)
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    target = _logits(gen, n + requests, cols, dtype)
    row = [t + b for b in range(requests) for t in range(offsets[b], offsets[b + 1])]
    draft = (target[row].float() + 0.5 * torch.randn(n, cols, generator=gen)).to(DT[dtype])
    noise = torch.empty(requests, cols).exponential_(generator=gen)
    gumbel = -torch.log(torch.empty(n, cols).exponential_(generator=gen))
    drafted = (draft.float() + gumbel).argmax(1).int() if n else torch.zeros(0, dtype=torch.int32)
    return target, None if onehot else draft, drafted, offsets, torch.rand(n, generator=gen), noise


def run_verify(target, draft, drafted, offsets, uniform, noise, scale=1.0):
    c = [None if t is None else t if t.is_cuda else t.cuda() for t in (target, draft, drafted, uniform, noise)]
    rows, requests = target.shape[0], len(offsets) - 1
    tokens = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    accepted = torch.full((requests,), -9, dtype=torch.int32, device="cuda")
    logp = torch.full((rows,), NAN, device="cuda")
    need = binding.lik_verify_drafts_workspace_bytes(target, requests)
    ws = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    binding.lik_verify_drafts(c[0], c[1], c[2], _i32(offsets).cuda(), c[3], c[4], tokens, accepted, logp, workspace=ws,
                              scale=scale)
    assert bool((ws[need:] == 0xFF).all()), "written behind the workspace"
    return tokens.tolist(), accepted.tolist(), logp.cpu()


def check_verify(case, scale=1.0):
    tokens, accepted, logp = run_verify(*case, scale=scale)
    want = ref.verify(*(t.cpu() if torch.is_tensor(t) else t for t in case), scale)
    assert tokens == want[0] and accepted == want[1]
    # log p = scale * (z - max) - log(sum): a few roundings of numbers up to the logits' scaled span; the sum's
    # relative error is under 2^-18 for any vocabulary here (fp32 partial sums of a few thousand terms, joined)
    span = float((case[0].float()[case[0].float().isfinite()].abs().max() * 2 * scale).clamp(min=1.0))
    assert float((logp.double() - torch.tensor(want[2], dtype=torch.float64)).abs().max()) <= 2.0 ** -22 * span + 2.0 ** -18
    return tokens, accepted


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("onehot", [False, True])
@pytest.mark.parametrize("counts,cols", [([0], 1), ([1], 2), ([3, 0, 2], 17), ([4], 1000), ([0, 0, 5, 1, 9], 4099),
                                         ([2, 2], 32003), ([1] * 70, 301), ([20, 3], 8192)])
def test_verify(dtype, onehot, counts, cols):
    check_verify(_drafts(_gen(cols + len(counts)), counts, cols, dtype, onehot), scale=1.0)
    check_verify(_drafts(_gen(cols + 1), counts, cols, dtype, onehot), scale=0.7)


def test_verify_everything_and_nothing_passes():
    target, draft, drafted, offsets, _, noise = _drafts(_gen(1), [3, 2], 500, "f32")
    t, a = check_verify((target, draft, drafted, offsets, torch.zeros(5), noise))
    assert a == [3, 2]
    same = torch.cat([target[0:3], target[4:6]])
    t, a = check_verify((target, same, drafted, offsets, torch.full((5,), 1 - 2.0 ** -24), noise))
    assert a == [3, 2]  # the draft is the target: u < 1 passes
    far = torch.full((5, 500), -40.0)
    far[torch.arange(5), drafted.long()] = 40.0
    t, a = check_verify((target, far, drafted, offsets, torch.full((5,), 0.9999), noise))
    assert a == [0, 0]


def test_verify_masked_columns_and_rows_without_mass():
    gen = _gen(2)
    target, draft, drafted, offsets, uniform, noise = _drafts(gen, [3, 2, 1, 0], 100, "f32")
    target[:, ::3] = -INF
    draft[:, 1::3] = -INF
    check_verify((target, draft, drafted, offsets, uniform, noise))
    # a drafted token that the target has ruled out, one that the draft had ruled out, tokens outside the row
    drafted[0], drafted[3], drafted[5] = 3, 4, 100
    check_verify((target, draft, drafted, offsets, torch.zeros(6), noise))
    drafted[0] = -1
    check_verify((target, draft, drafted, offsets, torch.zeros(6), noise))
    check_verify((target, None, drafted, offsets, torch.zeros(6), noise))
    for bad in (-INF, NAN, INF):
        broken = target.clone()
        if bad == -INF:
            broken[0], broken[6] = bad, bad
        else:
            broken[0, 50], broken[6, 11] = bad, bad
        tokens, accepted, logp = run_verify(broken, draft, drafted, offsets, torch.zeros(6), noise)
        assert accepted[0] == 0 and tokens[:4] == [-1] * 4 and logp[0] == 0
        assert tokens[4 + 2] == -1 or accepted[1] != 2
        want = ref.verify(target, draft, drafted, offsets, torch.zeros(6), noise, 1.0)
        assert tokens[8:] == want[0][8:]


def test_verify_ties_go_to_the_lowest_column():
    target, noise = torch.zeros(2, 3000), torch.ones(2, 3000)
    tokens, accepted, _ = run_verify(target, None, torch.zeros(0, dtype=torch.int32), [0, 0, 0], torch.zeros(0), noise)
    assert tokens == [0, 0] and accepted == [0, 0]
    target[0, 1234:] = 2.0
    noise[1, 700:] = 0.5
    assert run_verify(target, None, torch.zeros(0, dtype=torch.int32), [0, 0, 0], torch.zeros(0), noise)[0] == [1234, 700]


def test_verify_residual_without_mass_draws_from_the_target():
    """Draft and target agree but for a token that the target has ruled out: p <= q everywhere else."""
    target = torch.tensor([[1.0, 2.0, -INF, 0.5], [0.0, 0.0, 0.0, 0.0]])
    draft = torch.tensor([[1.0, 2.0, -INF, 0.5]])
    noise = torch.tensor([[0.2, 5.0, 0.001, 3.0]])
    check_verify((target, draft, _i32([2]), [0, 1], torch.tensor([0.5]), noise))


def test_verify_unusual_noise():
    """Entries that are 0 or not numbers; a column whose quotient is infinite wins, the lowest of equals."""
    target = torch.zeros(1, 600)
    noise = torch.ones(1, 600)
    noise[0, 3], noise[0, 4], noise[0, 300], noise[0, 301] = NAN, -1.0, 0.0, 0.0
    assert run_verify(target, None, _i32([]), [0, 0], torch.zeros(0), noise)[0] == [300]
    noise[0] = INF
    assert run_verify(target, None, _i32([]), [0, 0], torch.zeros(0), noise)[0] == [-1]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_strides_and_padding(dtype):
    target, draft, drafted, offsets, uniform, noise = case = _drafts(_gen(5), [2, 3], 333, dtype)
    wide = torch.full((7, 340), NAN, dtype=DT[dtype], device="cuda")
    wide[:, 3:336] = target.cuda()
    wd = torch.full((5, 401), NAN, dtype=DT[dtype], device="cuda")
    wd[:, 1:334] = draft.cuda()
    check_verify((wide[:, 3:336], wd[:, 1:334], drafted, offsets, uniform, noise))
    # rows behind the last request's: not read, written as -1 and 0
    more = torch.cat([target, torch.full((4, 333), NAN).to(DT[dtype])])
    md = torch.cat([draft, torch.full((4, 333), NAN).to(DT[dtype])])
    tokens, accepted, logp = run_verify(more, md, torch.cat([drafted, _i32([999] * 4)]), offsets,
                                        torch.cat([uniform, torch.full((4,), NAN)]), noise)
    want = ref.verify(*case, 1.0)
    assert tokens == want[0] + [-1] * 4 and accepted == want[1] and bool((logp[7:] == 0).all())


def test_verify_distribution():
    """Tokens drawn with drafts from another distribution are distributed as the target's (20000 draws of 8 columns:
    a share is off by more than 5 standard deviations once in millions)."""
    gen, n, cols = _gen(6), 20_000, 8
    target, draft = torch.randn(cols, generator=gen), torch.randn(cols, generator=gen)
    q = torch.softmax(draft, 0)
    drafted = torch.multinomial(q, n, replacement=True, generator=gen).int()
    counts, first = 4000, torch.zeros(cols, dtype=torch.int64)
    for a in range(0, n, counts):
        tokens, _, _ = run_verify(target.repeat(2 * counts, 1), draft.repeat(counts, 1), drafted[a:a + counts],
                                  list(range(counts + 1)), torch.rand(counts, generator=gen),
                                  torch.empty(counts, cols).exponential_(generator=gen))
        first += torch.bincount(torch.tensor(tokens[::2]), minlength=cols)
    p = torch.softmax(target, 0)
    assert bool(((first / n - p).abs() <= 5 * torch.sqrt(p * (1 - p) / n)).all())


def test_verify_refusals():
    target, draft, drafted, offsets, uniform, noise = _drafts(_gen(7), [2], 64, "f32")
    t, d, x, u, e = (v.cuda() for v in (target, draft, drafted, uniform, noise))
    off = _i32(offsets).cuda()
    out = (torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
           torch.zeros(3, device="cuda"))
    ws = torch.empty(binding.lik_verify_drafts_workspace_bytes(t, 1), dtype=torch.uint8, device="cuda")
    binding.lik_verify_drafts(t, d, x, off, u, e, *out, workspace=ws)
    for bad in (dict(workspace=None), dict(workspace=ws[:16]), dict(workspace=ws, scale=0.0),
                dict(workspace=ws, scale=INF)):
        with pytest.raises(binding.LIKError):
            binding.lik_verify_drafts(t, d, x, off, u, e, *out, **bad)
    for args in ((t[:2], d, x, off, u, e), (t, d.half(), x, off, u, e), (t, d[:, :32], x, off, u, e),
                 (t, d, x.long(), off, u, e), (t, d, x, off, u[:1], e), (t, d, x, off, u, e.half())):
        with pytest.raises(ValueError):
            binding.lik_verify_drafts(*args, *out, workspace=ws)
    with pytest.raises(binding.LIKError):  # an output inside an input
        binding.lik_verify_drafts(t, d, x, off, u, e, out[0], out[1], t[0, :3], workspace=ws)
