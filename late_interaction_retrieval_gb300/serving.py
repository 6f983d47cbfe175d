"""A serving step of an answer model over keys and values held in 8 bits.

  cache_slots      block tables and slot maps of a batch, from its requests' lengths
  cache_write      a layer's new keys and values into the cache
  cache_attention  the new tokens' attention over the cache
  verify_drafts    drafted tokens against the target model's probabilities
  TokenCache       pages, scales and the requests' table of a model, on which
                   the first three work together

Prompts, single tokens and drafts go through the same calls: a batch packs the
new tokens of its requests along one axis, request b those of the rows
offsets[b] .. offsets[b + 1].  Nothing is read back from the device, so that a
step can be captured into a CUDA graph and replayed with other lengths; rows
behind the last request's are padding.  The log-probabilities that
verify_drafts returns are the old ones that layers.policy_loss wants.

These functions run on the current stream, allocate what is not given and call
the binding (argument checks and errors are its); none has a gradient.
"""
from __future__ import annotations

import torch

from . import binding


def _buffer(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def cache_slots(cached, added, held, free_pages, free_count, block_table, page_size, rows):
    """(held, lengths, offsets, slots, free_left) of a batch whose request b
    holds held[b] pages with cached[b] tokens in them and gets added[b] more;
    all int32, block_table [requests, most pages] gets its new entries in
    place.  Pages come from the end of free_pages[:free_count]; free_left below
    zero says how many were missing.  slots [rows] (int64, -1: none) says where
    each row's token goes; lengths are the requests' tokens with the new ones
    that have a row: where `rows` are too few, the last tokens are left out."""
    most, missing = (torch.empty(n, dtype=torch.int32, device=cached.device) for n in (cached.shape[0], 1))
    return _slots(cached, added, held, free_pages, free_count, block_table, page_size, rows, most, missing)


def _slots(cached, added, held, free_pages, free_count, block_table, page_size, rows, most, missing):
    """cache_slots, with the buffers for what the requests may have after the step and for what is missing."""
    def int32(n):
        return torch.empty(n, dtype=torch.int32, device=cached.device)

    n = cached.shape[0]
    held_out, lengths, offsets, left = int32(n), int32(n), int32(n + 1), int32(1)
    slots = torch.empty(rows, dtype=torch.int64, device=cached.device)
    binding.lik_cache_slots_fit(cached, added, held, free_pages, free_count, block_table, held_out, lengths, offsets,
                                slots, left, most, missing, page_size)
    return held_out, lengths, offsets, slots, left


def cache_write(k, v, slots, k_cache, v_cache, k_scale, v_scale):
    """New keys and values [rows, heads, dim] (fp32, fp16, bf16; any strides of
    rows and heads) into the slots of the cache [pages, heads, page, dim], in
    place.  A page and head share one scale [pages, heads], which grows with
    their largest value; slots outside the cache write nothing."""
    binding.lik_cache_write(k, v, slots, k_cache, v_cache, k_scale, v_scale)


def cache_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, offsets, lengths, scale=None, max_added=None,
                    out=None, return_lse=False, workspace=None):
    """Attention of the rows q [rows, q_heads, dim], the last tokens of their
    requests, over all tokens up to their own: q head h reads head h // (q_heads
    // heads).  scale: dim ** -0.5 unless given.  max_added: the most rows of a
    request, if known (time depends on it, results do not).  Rows that see
    nothing are 0; rows of no request keep what `out` held.  With return_lse
    also log sum exp of the scores [rows, q_heads] fp32."""
    rows, q_heads, dim = q.shape
    requests = block_table.shape[0]
    if scale is None:
        scale = dim ** -0.5
    if max_added is None:
        max_added = -(-rows // requests) if requests else 0
    if out is None:
        out = torch.empty((rows, q_heads, dim), dtype=q.dtype, device=q.device)
    lse = torch.empty((rows, q_heads), dtype=torch.float32, device=q.device) if return_lse else None
    if workspace is None:
        workspace = _buffer(binding.lik_cache_attention_workspace_bytes(q, k_cache, block_table, max_added), q.device)
    binding.lik_cache_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, offsets, lengths, out, lse,
                                workspace, max_added, scale)
    return (out, lse) if return_lse else out


def verify_drafts(target_logits, drafted, offsets, uniform, noise, draft_logits=None, scale=1.0, workspace=None):
    """(tokens, accepted, logp) of drafts under the target's logits.  Request b
    drafted drafted[offsets[b] .. offsets[b + 1]] (none: plain sampling) from
    draft_logits [drafts, cols] (None: looked up, not drawn); its rows of
    target_logits [drafts + requests, cols], tokens and logp begin at
    offsets[b] + b and are one more (offsets count drafts alone: not a plan's,
    see TokenCache.verify_rows).  The accepted[b] drafts that pass come
    first, then one token drawn where they end, then -1.  uniform [drafts] in
    [0, 1) and noise [requests, cols] from the exponential distribution make the
    tokens the target's own; logp are their log-probabilities."""
    dev, rows, requests = target_logits.device, target_logits.shape[0], noise.shape[0]
    tokens = torch.empty(rows, dtype=torch.int32, device=dev)
    accepted = torch.empty(requests, dtype=torch.int32, device=dev)
    logp = torch.empty(rows, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _buffer(binding.lik_verify_drafts_workspace_bytes(target_logits, requests), dev)
    binding.lik_verify_drafts(target_logits, draft_logits, drafted, offsets, uniform, noise, tokens, accepted, logp,
                              workspace, scale)
    return tokens, accepted, logp


class TokenCache:
    """The 8-bit cache of a model's layers, and the requests that share its pages.

      plan(added, rows)     a step's new tokens: lengths, offsets and slots
      write(layer, k, v)    their keys and values
      attention(layer, q)   their attention over the cache
      verify_rows(drafts, total)  the rows and offsets that verify_drafts wants of them
      keep(tokens)          so many of them stay; drafts that were turned down leave
      release(request)      a finished request's pages go back

    A step is one plan, each layer's write and attention, one keep, on one
    stream at a time.  A place without a request (none yet, or released) plans
    no token.  All lengths stay on the device and every buffer where it is: a
    captured step can be replayed.  missing [1] (int32, device) is how many
    pages the last plan lacked: beyond those that were free, behind the table's
    columns (max_tokens), or for tokens beyond its rows.  0: the step fits.
    Tokens without a place are neither written nor seen, and keep() keeps
    nothing of a step that does not fit.
    """

    def __init__(self, layers, heads, dim, pages, requests, max_tokens, page_size=64, device="cuda"):
        def full(shape, value, dtype=torch.int32):
            return torch.full(shape, value, dtype=dtype, device=device)

        codes, scales = (layers, pages, heads, page_size, dim), (layers, pages, heads)
        self.page_size, self.pages = page_size, pages
        self.k, self.v = (full(codes, 0, torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
        self.k_scale, self.v_scale = (full(scales, 0.0, torch.float32) for _ in range(2))
        self.block_table = full((requests, -(-max_tokens // page_size)), -1)
        self.cached, self.held = full((requests,), 0), full((requests,), 0)
        # one entry behind the pages, where release() puts what is no page
        self._free = torch.arange(pages + 1, dtype=torch.int32, device=device)
        self.free_count, self.missing = full((1,), pages), full((1,), 0)
        self._most = full((requests,), 0)  # what a request may have after the step that was planned last
        self.lengths = self.offsets = self.slots = None

    def plan(self, added, rows):
        """Places for added[b] (int32 [requests], device) new tokens of request b, at most `rows` together."""
        held, self.lengths, self.offsets, self.slots, left = _slots(
            self.cached, added, self.held, self._free[:self.pages], self.free_count, self.block_table, self.page_size,
            rows, self._most, self.missing)
        self.held.copy_(held)
        torch.clamp(left, min=0, out=self.free_count)
        return self.lengths, self.offsets, self.slots

    def write(self, layer, k, v):
        cache_write(k, v, self.slots, self.k[layer], self.v[layer], self.k_scale[layer], self.v_scale[layer])

    def attention(self, layer, q, **options):
        """cache_attention of the planned tokens' rows q [rows, q_heads, dim]."""
        return cache_attention(q, self.k[layer], self.v[layer], self.k_scale[layer], self.v_scale[layer],
                               self.block_table, self.offsets, self.lengths, **options)

    def verify_rows(self, drafts, total):
        """(rows, offsets) with which verify_drafts follows a plan whose request b's last drafts[b] (int32 [requests],
        device) tokens are drafts, at most `total` together; 0 for a prompt, of which the last row is wanted.  rows
        [total + requests] (int64) are the batch's rows that target_logits is made of: verify_drafts has one more than
        drafts for every request.  A place without a request has one too, of no meaning, and so are the token that is
        drawn there and the rows behind the last: offsets count drafts alone and are not the plan's."""
        ends = self.offsets[1:]
        drafts = torch.minimum(drafts, ends - self.offsets[:-1] - 1).clamp(min=0)
        offsets = torch.zeros_like(self.offsets)
        torch.cumsum(drafts, 0, dtype=torch.int32, out=offsets[1:])
        first = offsets[:-1] + torch.arange(drafts.shape[0], dtype=torch.int32, device=offsets.device)
        at = torch.arange(total + drafts.shape[0], dtype=torch.int32, device=offsets.device)
        b = torch.searchsorted(first, at, right=True) - 1
        rows = (ends - 1 - drafts - first)[b] + at
        return rows.clamp(min=0, max=max(self.slots.shape[0] - 1, 0)).long(), offsets

    def keep(self, tokens):
        """The first tokens[b] (device, or one number for all) of request b's planned ones stay: no more than were
        planned, and none in a place without a request, which planned none.  Of a step that did not fit nothing does:
        `missing` says so, also behind a captured step, which can be run again once there is room."""
        self.cached.add_(tokens)
        torch.minimum(self.cached, self._most, out=self.cached)

    def release(self, request):
        """Request number `request` has ended: its pages are free, its place is empty."""
        row, held = self.block_table[request], self.held[request]
        place = torch.arange(row.shape[0], device=row.device)
        taken = (place < held) & (row >= 0)
        to = torch.where(taken, self.free_count + taken.cumsum(0) - 1, self.pages)
        self._free.index_copy_(0, to, row)
        self.free_count.add_(taken.sum())
        row.fill_(-1)
        self.held[request] = 0
        self.cached[request] = 0
        self._most[request] = 0
