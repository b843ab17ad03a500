"""One layer's GAAC compressed KV cache held in torch device memory.

Allocation and argument marshalling only: the calibration, encoding, append,
attention and decompression themselves run in the library's kernels.
"""
from __future__ import annotations

import torch

from . import (BLOCK, _DTYPES, FP8_E4M3, HEAD_DIM, Kv8, Pools, _call, _made_for, _stream_object, append,
               attention_workspace, beam_workspace, calibrate,
               decode_attention, decode_attention_bf16, decompress, encode_blocks, entry_fields, kv8_append,
               kv8_attention_workspace, kv8_compact, kv8_decode_attention, kv8_fork, kv8_release, kv8_reorder,
               kv8_reserve, new_stats, new_table)


class LayerCache:
    """Slot table, pools, window bases and counters of one layer.

    slot_ids: int32 [batch, max_blocks, n_kv_heads, 2]: the slot each block is
    encoded (or sealed) into.  Default: a dense map (one slot per table position).
    n_raw: raw tiles available for tails and fallbacks (default: one per
    (sequence, kv-head, K|V) plus one per table position, i.e. never exhausted).
    open_compressed: keep each sequence's open block compressed in its slot
    (prefill and append), instead of as a BF16 tail.
    """

    def __init__(self, batch: int, n_kv_heads: int, max_blocks: int, device="cuda", slot_ids=None, n_slots=None,
                 n_raw=None, raw_free=None, open_compressed: bool = False):
        self.batch, self.n_kv_heads, self.max_blocks = batch, n_kv_heads, max_blocks
        self.open_compressed = open_compressed
        self.device = torch.device(device)
        positions = batch * max_blocks * n_kv_heads * 2
        if slot_ids is None:
            slot_ids = torch.arange(positions, dtype=torch.int32, device=device).view(batch, max_blocks, n_kv_heads, 2)
            n_slots = positions if n_slots is None else n_slots
        elif n_slots is None:
            n_slots = int(slot_ids.max().item()) + 1
        self.slot_ids = slot_ids.to(torch.int32).contiguous()
        if n_raw is None:
            n_raw = positions + batch * n_kv_heads * 2
        self.pools = Pools(n_slots, n_raw, device=device, raw_free=raw_free)
        self.table = new_table(batch, max_blocks, n_kv_heads, device=device)
        self.base3 = torch.zeros((2, n_kv_heads, HEAD_DIM), dtype=torch.uint8, device=device)
        self.base4 = torch.zeros((2, n_kv_heads, HEAD_DIM), dtype=torch.uint8, device=device)
        self.stats = new_stats(device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self._ws = None
        self.all_raw = False  # encoded with raw=True: every block a raw tile, appends keep it so

    # -- building
    def calibrate(self, k_cal: torch.Tensor, v_cal: torch.Tensor, stream=None):
        """k_cal, v_cal: BF16 [n_tok, kv_heads, 128] calibration tokens."""
        calibrate(k_cal, self.base3[0], self.base4[0], self.status, stream)
        calibrate(v_cal, self.base3[1], self.base4[1], self.status, stream)

    def encode(self, k: torch.Tensor, v: torch.Tensor, seq_lens: torch.Tensor, stream=None, raw: bool = False):
        """Prefill: k, v BF16 [batch, tokens, kv_heads, 128]; seq_lens int32 [batch].
        raw=True stores every block as BF16 (the uncompressed baseline cache)."""
        with torch.cuda.stream(_stream_object(stream, self.device)):
            self.seq_lens.copy_(seq_lens)
        self.all_raw = raw
        encode_blocks(k, v, self.seq_lens, self.max_blocks, self.base3, self.base4, self.table,
                      None if raw else self.slot_ids, self.pools, self.stats, self.status, stream,
                      open_compressed=self.open_compressed and not raw)

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None):
        """Decode step: one token per sequence, k_new/v_new BF16 [batch, kv_heads, 128]."""
        append(k_new, v_new, self.seq_lens, self.max_blocks, self.base3, self.base4, self.table,
               None if self.all_raw else self.slot_ids, self.pools, self.stats, self.status, stream,
               open_compressed=self.open_compressed)

    # -- reading
    def auto_splits(self) -> int:
        from . import auto_splits

        return auto_splits(self.batch, self.n_kv_heads, self.max_blocks)

    def workspace(self, n_splits: int = 0, stream=None) -> torch.Tensor:
        need = attention_workspace(self.batch, self.n_kv_heads, self.max_blocks, n_splits)
        if self._ws is None or self._ws.numel() < need:
            self._ws = _made_for(stream, self.device,
                                 lambda: torch.zeros(max(need, 16), dtype=torch.uint8, device=self.device))
        if stream is not None:  # a larger one may take its place
            self._ws.record_stream(_stream_object(stream, self.device))
        return self._ws

    def attention(self, q: torch.Tensor, scale: float, out: torch.Tensor | None = None, n_splits: int = 0,
                  stream=None, bf16: bool = False) -> torch.Tensor:
        """q: BF16 [batch, q_heads, 128] -> fp32 [batch, q_heads, 128].  bf16=True: the uncompressed BF16
        kernel (the cache must have been encoded with raw=True)."""
        if out is None:
            out = _made_for(stream, q.device, lambda: torch.empty(q.shape, dtype=torch.float32, device=q.device))
        if bf16:
            decode_attention_bf16(q, self.seq_lens, self.table, self.pools, scale, out,
                                  self.workspace(n_splits, stream), n_splits, self.status, stream)
        else:
            decode_attention(q, self.seq_lens, self.table, self.pools, self.base3, self.base4, scale, out,
                             self.workspace(n_splits, stream), n_splits, self.status, stream)
        return out

    def decompress(self, n_tok: int | None = None, stream=None):
        """BF16 (k, v) [batch, n_tok, kv_heads, 128] rebuilt from the cache (tokens past a sequence: 0)."""
        n_tok = self.max_blocks * BLOCK if n_tok is None else n_tok
        shape = (self.batch, n_tok, self.n_kv_heads, HEAD_DIM)
        k, v = (_made_for(stream, self.device, lambda: torch.zeros(shape, dtype=torch.bfloat16, device=self.device))
                for _ in range(2))
        decompress(self.table, self.seq_lens, self.pools, self.base3, self.base4, k, v, self.status, stream)
        return k, v

    def fields(self):
        return entry_fields(self.table)

    def resident_bytes(self) -> dict:
        """Bytes held by the cache's blocks: slots, raw tiles, table entries."""
        _, _, mode, _ = entry_fields(self.table)
        n_slot = int((mode == 0).sum().item())
        n_raw = int((mode == 1).sum().item())
        return {"slot_tiles": n_slot, "raw_tiles": n_raw, "slot_bytes": n_slot * 12032, "raw_bytes": n_raw * 16384,
                "table_bytes": self.table.numel() * 8}


class Kv8Cache(Kv8):
    """One layer's 8-bit paged KV cache: FP8 pages of 64 tokens with a scale for each (page, kv-head, K|V), the open
    block of every sequence in the model's type, and counted pages that sequences share.

    Calls on one cache share its workspaces, attention too: they are ordered on the GPU (one stream, or events), and
    after whatever made the cache.  Attentions that run beside one another take kv8_decode_attention with a workspace
    each.

    dtype: BF16 or FP16, the type of k, v, q and the open block.  Faults that only the device sees (no page left, a
    length past the table, offsets out of order) are recorded in `status`, as by the calls of the lossless cache; such
    a call leaves the sequence's tokens as they were, with the pages that could be reserved for it.
    """

    def __init__(self, n_pages: int, batch: int, n_kv_heads: int, max_blocks: int, fmt: int = FP8_E4M3,
                 dtype: torch.dtype = torch.bfloat16, device="cuda"):
        self._over(torch.zeros((n_pages, n_kv_heads, 2, BLOCK, HEAD_DIM), dtype=torch.uint8, device=device),
                   torch.ones((n_pages, n_kv_heads, 2), dtype=torch.float32, device=device),
                   torch.zeros((batch, n_kv_heads, 2, BLOCK, HEAD_DIM), dtype=dtype, device=device),
                   torch.full((batch, max_blocks), -1, dtype=torch.int32, device=device),
                   torch.zeros(n_pages, dtype=torch.int32, device=device),
                   torch.zeros(batch, dtype=torch.int32, device=device), fmt)

    @classmethod
    def over(cls, pages, scales, tail, table, refs, seq_lens, fmt: int = FP8_E4M3) -> "Kv8Cache":
        """A cache around existing tensors (the shapes are Kv8's)."""
        self = cls.__new__(cls)
        self._over(pages, scales, tail, table, refs, seq_lens, fmt)
        return self

    def _over(self, *args):
        Kv8.__init__(self, *args)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._own_status = (self.status, self.status.data_ptr())
        with torch.cuda.device(self.device):
            self._ws = torch.zeros(kv8_attention_workspace(), dtype=torch.uint8, device=self.device)

    def append(self, k: torch.Tensor, v: torch.Tensor, cu_tokens: torch.Tensor | None = None, reserve: bool = True,
               stream=None):
        """Tokens behind the sequences: rows cu_tokens[b] .. cu_tokens[b + 1] of k, v [n, kv_heads, 128] for sequence
        b, or one row for each, a released one included (cu_tokens passes over it).  reserve=False: the pages of blocks
        that fill have been reserved before."""
        kv8_append(self, k, v, cu_tokens, self.status, stream, reserve)

    def attention(self, q: torch.Tensor, scale: float, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """q: [batch, q_heads, 128] -> the same shape and type (or `out`'s: fp32 is allowed)."""
        if out is None:
            out = _made_for(stream, q.device, lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device))
        kv8_decode_attention(self, q, scale, out, self._ws, self.status, stream)
        return out

    def reserve(self, cu_tokens: torch.Tensor | None = None, stream=None):
        kv8_reserve(self, cu_tokens, self.status, stream)

    def release(self, seqs: torch.Tensor, stream=None):
        kv8_release(self, seqs, self.status, stream)

    def fork(self, src: torch.Tensor, dst: torch.Tensor, stream=None):
        kv8_fork(self, src, dst, self.status, stream)

    def reorder(self, parents: torch.Tensor, stream=None):
        """The beams of each search follow its choice: sequence g * beams + i becomes what g * beams + parents[g, i] was
        (int32 [groups, beams], as Beams.select gives them)."""
        kv8_reorder(self, parents, self.status, stream)

    def compact(self, stream=None) -> torch.Tensor:
        """int32 [n_pages]: where each page has gone, -1 for free ones."""
        moved_to = _made_for(stream, self.device, lambda: torch.empty_like(self.refs))
        kv8_compact(self, moved_to, stream)
        return moved_to


class Beams:
    """The choice of `batch` beam searches of `beams` beams over a vocabulary, with its workspace: beam i of search b is
    row b * beams + i of the logits, and sequence b * beams + i of a cache.

    n_out: candidates that are chosen (default: beams).  end_token: what ended beams go on with.  Calls on one object
    share its workspace: they are ordered on the GPU, and after whatever made it."""

    def __init__(self, batch: int, beams: int, vocab: int, n_out: int | None = None, end_token: int = 0, device="cuda"):
        self.batch, self.beams, self.vocab, self.end_token = batch, beams, vocab, end_token
        self.n_out = beams if n_out is None else n_out
        need = beam_workspace(batch, beams, vocab, self.n_out)
        if need == 0:
            raise ValueError("batch >= 1, 1 <= beams <= 32, 1 <= n_out <= 64 and 1 <= vocab <= 2^20 are wanted")
        self._ws = torch.zeros(need, dtype=torch.uint8, device=device)
        self.device, self._index = self._ws.device, self._ws.get_device()
        self._rows, self._scores = (batch * beams, vocab), (batch, beams)
        self._like = tuple(torch.empty((batch, self.n_out), dtype=t, device=device) for t in (torch.float32, torch.int32))

    def select(self, logits: torch.Tensor, scores: torch.Tensor, ended: torch.Tensor | None = None, stream=None):
        """logits [batch * beams, vocab], scores fp32 [batch, beams], ended bool or uint8 [batch, beams] -> (scores fp32,
        parents int32, tokens int32), each [batch, n_out], as beam_select says."""
        code, index = _DTYPES.get(logits.dtype), self._index
        if code is None or logits.shape != self._rows or logits.get_device() != index or \
                (logits.stride(1) != 1 and self.vocab > 1):
            raise ValueError("logits must be BF16, FP16 or FP32 [batch * beams, vocab] on the workspace's device, tokens contiguous")
        if scores.shape != self._scores or scores.dtype != torch.float32 or scores.get_device() != index or \
                not scores.is_contiguous():
            raise ValueError("scores must be contiguous fp32 [batch, beams] on the logits' device")
        if (logits.requires_grad or scores.requires_grad) and torch.is_grad_enabled():
            raise ValueError("autograd does not see select: call it under torch.no_grad()")
        if ended is not None and (ended.dtype not in (torch.bool, torch.uint8) or ended.shape != self._scores or
                                  ended.get_device() != index or not ended.is_contiguous()):
            raise ValueError("ended must be contiguous bool or uint8 [batch, beams] on the logits' device")

        like, like_whole = self._like  # empty_like takes half of empty's microseconds
        if stream is None:
            best, parents, tokens = torch.empty_like(like), torch.empty_like(like_whole), torch.empty_like(like_whole)
        else:
            best, parents, tokens = (_made_for(stream, self.device, lambda t=t: torch.empty_like(t))
                                     for t in (like, like_whole, like_whole))
        # what beam_select would do, whose checks of the results and the workspace are met here
        _call("gaac_beam_select", index, stream, logits.data_ptr(), code,
              logits.stride(0) if self._rows[0] > 1 else self.vocab, scores.data_ptr(), 0 if ended is None else ended.data_ptr(),
              self.end_token, self.batch, self.beams, self.vocab, self.n_out, best.data_ptr(), parents.data_ptr(),
              tokens.data_ptr(), self._ws.data_ptr(), self._ws.nbytes)
        return best, parents, tokens
