"""One decoding step of a softmax-attention layer over a paged cache, captured
once in a CUDA graph and replayed: the counterpart, for the attention layers of a
hybrid decoder, of ``spec_step.SpeculativeStep`` for its gated-delta-rule layers.

The step is three kernels in two C-ABI calls with arguments built once:

  1. gdn_kv_cache_write: the new tokens' queries and keys rotated by their
     positions, keys and values written (quantised, for an 8-bit cache) to
     their slots;
  2. gdn_paged_attention: every new token over its sequence's cache.

Everything that changes from step to step is device memory read at replay time
(queries, keys, values, positions, slots, block table, lengths), so one graph
serves every step.  The caller fills the buffers (``place`` computes positions
and slots for tokens appended to the sequences), replays, and reads ``out``.
"""
from __future__ import annotations

import torch

from .attention import KVCacheWriteCall, PagedAttentionCall


class AttentionStep:
    """``seqs`` sequences, ``tokens`` new tokens each (1: decode; more: the
    verification of drafted tokens, causal among themselves), over ``cache`` (a
    ``PagedKVCache``) with at most ``pages_per_seq`` pages a sequence.

    Buffers, all device tensors owned by this object: ``q`` [seqs * tokens, Hq,
    d], ``k``, ``v`` [seqs * tokens, Hkv, d] (unrotated), ``block_table`` [seqs,
    pages_per_seq], ``kv_lens`` [seqs] (cached tokens, the new ones included),
    ``positions`` and ``slots`` [seqs * tokens].  ``table`` is a rotary table
    (``rotary_table``).  Outputs: ``out`` [seqs * tokens, Hq, d] and the rotated
    queries ``q_rotated``; the cache is written in place.
    """

    def __init__(self, cache, table, *, seqs, num_q_heads, pages_per_seq, tokens=1, dtype=torch.float16,
                 interleaved=False, scale=0.0, window=0):
        if pages_per_seq < 1:
            raise ValueError("pages_per_seq must be at least 1")
        dev, (_, page, heads, d) = cache.device, cache.k.shape
        self.cache, self.seqs, self.tokens, self.page = cache, seqs, tokens, page
        T = seqs * tokens
        new = lambda *s: torch.zeros(s, dtype=dtype, device=dev)  # noqa: E731
        idx = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
        self.q, self.k, self.v = new(T, num_q_heads, d), new(T, heads, d), new(T, heads, d)
        self.block_table, self.kv_lens = idx(seqs, pages_per_seq), idx(seqs)
        self.positions, self.slots = idx(T), idx(T) - 1
        self.status = idx(1)
        self._offsets = torch.arange(-tokens, 0, device=dev)  # of the new tokens' positions from the lengths
        cu = torch.arange(0, T + 1, tokens, dtype=torch.int32, device=dev) if tokens > 1 else None
        self._write = KVCacheWriteCall(self.k, self.v, cache, self.slots, positions=self.positions, table=table,
                                       interleaved=interleaved, q=self.q, status=self.status)
        self.q_rotated = self._write.outputs
        self._attend = PagedAttentionCall(self.q_rotated, cache, self.block_table, self.kv_lens, cu_seqlens=cu,
                                          scale=scale, window=window, max_seqlen=tokens, status=self.status)
        self.out = self._attend.outputs
        self.graph = None

    def place(self):
        """Positions and slots of the new tokens, from ``kv_lens`` and ``block_table`` (device operations only).  A token
        before a sequence's first position (an idle row: ``kv_lens`` 0, or fewer than the new tokens) is not stored: slot -1.
        One past the table's last page, or in a page that the pool does not have, gets a slot outside the pool, so that
        it is flagged and not written."""
        capacity, pool = self.block_table.shape[1] * self.page, self.cache.args.num_pages * self.page
        at = self.kv_lens[:, None] + self._offsets  # (64 bits, for the sums below)
        self.positions.view_as(at).copy_(at.clamp(min=0))
        inside = at.clamp(0, capacity - 1)
        page = self.block_table.gather(1, inside // self.page)
        slot = (inside % self.page).add_(page, alpha=self.page)
        slot.masked_fill_(slot < 0, pool).clamp_(max=pool)
        # at - inside is 0 for a token inside the table, negative before it and positive past it
        slot.add_(at.sub_(inside), alpha=1 << 31)
        self.slots.view_as(slot).copy_(slot.clamp_(-1, pool))

    def launch(self, stream=None):
        """The step's two calls on ``stream`` (default: the current one)."""
        self._write.launch(stream)
        return self._attend.launch(stream)

    def capture(self):
        """Records the step into a CUDA graph.  The warm-up before it stores no token and attends to nothing."""
        slots, lens = self.slots.clone(), self.kv_lens.clone()
        self.slots.fill_(-1)
        self.kv_lens.zero_()
        self.launch()
        torch.cuda.current_stream(self.slots.device).synchronize()
        self.slots.copy_(slots)
        self.kv_lens.copy_(lens)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.launch()
        return self

    def replay(self):
        if self.graph is None:
            self.capture()
        self.graph.replay()
        return self.out
