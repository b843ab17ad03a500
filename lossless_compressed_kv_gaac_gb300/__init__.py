"""Python binding of the GAAC compressed-KV decode-attention library.

Thin marshalling over the C ABI declared in ``include/gaac.h`` (ctypes): every
function below passes torch device pointers, sizes and the current CUDA stream
to the library and raises on a nonzero status.  All computation happens in the
library's CUDA kernels; there is no CPU fallback.  If ``libgaac.so`` has not been
built, the first call raises.

Method: "GAAC: Lossless KV Compression for Bandwidth-Efficient LLM Inference on
Personal Devices" (sections 3.1-3.3).  Tile format v3 is described in gaac.h.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

import torch

HEAD_DIM = 128
BLOCK = 64
TILE_ELEMS = 8192
SLOT_BYTES = 12032
ESC_CAPACITY = 496
RAW_TILE_BYTES = 16384
MAX_GQA = 8

OK, EINVAL, EPOOL, EFORMAT, ECUDA, ETIMEOUT = range(6)
MODE_SLOT, MODE_RAW, MODE_NONE = 0, 1, 255
OPEN_COMPRESSED = 1  # flag of encode_blocks / append: keep the open block compressed in its slot

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgaac.so")
_lock = threading.Lock()
_lib = None


class GaacError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {strerror(status) if _lib is not None else status} (status {status})")


class gaac_pools(ctypes.Structure):
    _fields_ = [
        ("slot_pool", ctypes.c_void_p),
        ("n_slots", ctypes.c_int64),
        ("raw_pool", ctypes.c_void_p),
        ("n_raw", ctypes.c_int64),
        ("raw_free", ctypes.c_void_p),
        ("n_raw_free", ctypes.c_int64),
        ("raw_cursor", ctypes.c_void_p),
    ]


STATS_FIELDS = ("groups0", "groups1", "groups2", "groups3", "escape_bytes", "slot_tiles", "raw_tiles", "tail_tiles")


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it was not built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"GAAC CUDA library not found at {LIB_PATH}; build it with "
                    "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
            L = ctypes.CDLL(LIB_PATH)
            P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
            L.gaac_strerror.argtypes = [i32]
            L.gaac_strerror.restype = ctypes.c_char_p
            L.gaac_format_version.argtypes = []
            L.gaac_format_version.restype = i32
            L.gaac_calibrate.argtypes = [P, i64, i64, i32, P, P, P, P]
            L.gaac_calibrate.restype = i32
            L.gaac_encode_blocks.argtypes = [P, P, i64, i64, i64, P, i32, i32, i32, P, P, P, P, P, P, P, P]
            L.gaac_encode_blocks.restype = i32
            L.gaac_append.argtypes = [P, P, P, i32, i32, i32, P, P, P, P, P, P, P, P]
            L.gaac_append.restype = i32
            L.gaac_encode_blocks_ex.argtypes = [P, P, i64, i64, i64, P, i32, i32, i32, P, P, P, P, P, P,
                                                ctypes.c_uint, P, P]
            L.gaac_encode_blocks_ex.restype = i32
            L.gaac_append_ex.argtypes = [P, P, P, i32, i32, i32, P, P, P, P, P, P, ctypes.c_uint, P, P]
            L.gaac_append_ex.restype = i32
            L.gaac_attention_workspace.argtypes = [i32, i32, i32, i32]
            L.gaac_attention_workspace.restype = sz
            L.gaac_attention_auto_splits.argtypes = [i32, i32, i32]
            L.gaac_attention_auto_splits.restype = i32
            L.gaac_decode_attention.argtypes = [P, i32, i32, i32, i32, P, P, P, P, P, ctypes.c_float, i32, P, P, sz,
                                                P, P]
            L.gaac_decode_attention.restype = i32
            L.gaac_decode_attention_bf16.argtypes = [P, i32, i32, i32, i32, P, P, P, ctypes.c_float, i32, P, P, sz,
                                                     P, P]
            L.gaac_decode_attention_bf16.restype = i32
            L.gaac_decode_attention_hd256.argtypes = L.gaac_decode_attention.argtypes
            L.gaac_decode_attention_hd256.restype = i32
            L.gaac_decompress.argtypes = [P, P, i32, i32, i32, P, P, P, P, P, i64, i64, i64, P, P]
            L.gaac_decode_attention_noalloc.argtypes = [P, i32, i32, i32, i32, P, P, P, P, P, ctypes.c_float, i32, P,
                                                        P, P]
            L.gaac_decode_attention_noalloc.restype = i32
            L.gaac_decompress.restype = i32
            L.gaac_encode_tiles.argtypes = [P, i64, P, P, i32, P, P, P, P, P, P, P]
            L.gaac_encode_tiles.restype = i32
            L.gaac_decode_tiles.argtypes = [P, P, i64, P, P, i32, P, P, P, P, P]
            L.gaac_decode_tiles.restype = i32
            L.gaac_nested_calibrate.argtypes = [P, i64, i64, i32, P, P, P]
            L.gaac_nested_calibrate.restype = i32
            L.gaac_nested_encode_tiles.argtypes = [P, i64, P, P, i32, P, P, P, P, P, P, P]
            L.gaac_nested_encode_tiles.restype = i32
            L.gaac_nested_decode_tiles.argtypes = [P, P, i64, P, P, i32, P, P, P, P, P, P]
            L.gaac_nested_decode_tiles.restype = i32
            L.gaac_fp8_slot_bytes.argtypes = [i32]
            L.gaac_fp8_slot_bytes.restype = i32
            L.gaac_fp8_calibrate.argtypes = [P, i64, i64, i32, i32, P, P, P, P]
            L.gaac_fp8_calibrate.restype = i32
            L.gaac_fp8_encode_tiles.argtypes = [P, i64, i32, P, P, i32, P, P, P, P, P, P, P]
            L.gaac_fp8_encode_tiles.restype = i32
            L.gaac_fp8_decompress_tiles.argtypes = [P, P, i64, i32, P, P, i32, P, P, P, P, P]
            L.gaac_fp8_decompress_tiles.restype = i32
            L.gaac_rope.argtypes = [P, i32, i32, i64, i64, i32, i32, P, i32, i64, i64, P, ctypes.c_float,
                                    ctypes.c_uint, P]
            L.gaac_rope.restype = i32
            L.gaac_prompt_attention.argtypes = [P, i32, i64, i32, i32, P, i32, ctypes.c_float, P, P]
            L.gaac_prompt_attention.restype = i32
            L.gaac_qk_norm_rope_workspace.argtypes = [i32]
            L.gaac_qk_norm_rope_workspace.restype = sz
            L.gaac_qk_norm_rope.argtypes = [P, i32, i32, i32, i64, i64, i32, i32, P, i32, i64, i64, P, ctypes.c_float,
                                            ctypes.c_float, ctypes.c_uint, P]
            L.gaac_qk_norm_rope.restype = i32
            L.gaac_qk_norm_rope_gradient.argtypes = L.gaac_qk_norm_rope.argtypes[:-1] + [P, sz, P]
            L.gaac_qk_norm_rope_gradient.restype = i32
            L.gaac_kv8_workspace.argtypes = [i32, i64]
            L.gaac_kv8_workspace.restype = sz
            L.gaac_kv8_append.argtypes = [P, P, P, i64, i64, i64, P, P, P]
            L.gaac_kv8_append.restype = i32
            L.gaac_kv8_reserve_append.argtypes = L.gaac_kv8_append.argtypes
            L.gaac_kv8_reserve_append.restype = i32
            L.gaac_kv8_attention_workspace.argtypes = []
            L.gaac_kv8_attention_workspace.restype = sz
            L.gaac_kv8_decode_attention.argtypes = [P, P, i32, i64, ctypes.c_float, P, i32, P, sz, P, P]
            L.gaac_kv8_decode_attention.restype = i32
            L.gaac_kv8_reserve.argtypes = [P, P, P, P]
            L.gaac_kv8_reserve.restype = i32
            L.gaac_kv8_release.argtypes = [P, P, i32, P, P]
            L.gaac_kv8_release.restype = i32
            L.gaac_kv8_fork.argtypes = [P, P, P, i32, P, P]
            L.gaac_kv8_fork.restype = i32
            L.gaac_kv8_reorder.argtypes = [P, P, i32, P, P]
            L.gaac_kv8_reorder.restype = i32
            L.gaac_beam_workspace.argtypes = [i32, i32, i32, i32]
            L.gaac_beam_workspace.restype = sz
            L.gaac_beam_select.argtypes = [P, i32, i64, P, P, i32, i32, i32, i32, i32, P, P, P, P, sz, P]
            L.gaac_beam_select.restype = i32
            L.gaac_kv8_compact.argtypes = [P, P, P]
            L.gaac_kv8_compact.restype = i32
            _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().gaac_strerror(status).decode()


def format_version() -> int:
    return lib().gaac_format_version()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _check(fn: str, status: int):
    if status != OK:
        raise GaacError(fn, status)


def _cuda(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


class Pools:
    """Caller-owned storage of one layer's compressed cache.

    slot_pool: uint8 [n_slots, 12032]; raw_pool: int16 [n_raw, 8192] (BF16 bits);
    raw_free: optional int32 list of free raw-tile indices (None = 0..n_raw-1);
    raw_cursor: int32 [1] device counter of popped raw tiles."""

    def __init__(self, n_slots: int, n_raw: int, device="cuda", raw_free: torch.Tensor | None = None):
        self.slot_pool = torch.zeros((max(n_slots, 1), SLOT_BYTES), dtype=torch.uint8, device=device)
        self.raw_pool = torch.zeros((max(n_raw, 1), TILE_ELEMS), dtype=torch.int16, device=device)
        self.n_slots, self.n_raw = n_slots, n_raw
        self.raw_free = raw_free
        self.raw_cursor = torch.zeros(1, dtype=torch.int32, device=device)

    def c(self) -> gaac_pools:
        n_free = self.raw_free.numel() if self.raw_free is not None else self.n_raw
        return gaac_pools(self.slot_pool.data_ptr(), self.n_slots, self.raw_pool.data_ptr(), self.n_raw,
                          _ptr(self.raw_free), n_free, self.raw_cursor.data_ptr())


def new_table(batch: int, max_blocks: int, n_kv_heads: int, device="cuda") -> torch.Tensor:
    """Slot table of one layer: int64 [batch, max_blocks, n_kv_heads, 2], one gaac_entry per element
    (bits 0-31 index, 32-47 esc_len, 48-55 mode, 56-63 n_tok)."""
    t = torch.zeros((batch, max_blocks, n_kv_heads, 2), dtype=torch.int64, device=device)
    t.fill_(MODE_NONE << 48)
    return t


def entry_fields(table: torch.Tensor):
    """(index, esc_len, mode, n_tok) tensors of a table."""
    return table & 0xFFFFFFFF, (table >> 32) & 0xFFFF, (table >> 48) & 0xFF, (table >> 56) & 0xFF


def new_stats(device="cuda") -> torch.Tensor:
    return torch.zeros(len(STATS_FIELDS), dtype=torch.int64, device=device)


def stats_dict(stats: torch.Tensor) -> dict:
    return dict(zip(STATS_FIELDS, stats.tolist()))


def _kv_strides(x: torch.Tensor, name: str):
    if x.dtype not in (torch.bfloat16, torch.int16) or x.dim() != 4 or x.shape[-1] != HEAD_DIM:
        raise ValueError(f"{name} must be a [batch, tokens, kv_heads, 128] BF16 tensor")
    if x.stride(3) != 1 or x.stride(2) != HEAD_DIM:
        raise ValueError(f"{name}: heads and channels must be contiguous")
    return x.stride(0), x.stride(1)


def calibrate(x: torch.Tensor, base3: torch.Tensor, base4: torch.Tensor, status: torch.Tensor | None = None,
              stream=None) -> None:
    """x: BF16 [n_tok, kv_heads, 128] (token stride free); writes uint8 base3/base4 [kv_heads, 128]."""
    _cuda(x, "x")
    if x.dim() != 3 or x.shape[-1] != HEAD_DIM or x.stride(2) != 1 or x.stride(1) != HEAD_DIM:
        raise ValueError("x must be [n_tok, kv_heads, 128] with contiguous heads and channels")
    _check("gaac_calibrate", lib().gaac_calibrate(x.data_ptr(), x.shape[0], x.stride(0), x.shape[1], base3.data_ptr(),
                                                   base4.data_ptr(), _ptr(status), _stream(stream)))


def encode_blocks(k, v, seq_lens, max_blocks, base3, base4, table, slot_ids, pools: Pools, stats=None, status=None,
                  stream=None, open_compressed: bool = False) -> None:
    """Prefill encode of a layer.  k, v: BF16 [batch, tokens, kv_heads, 128]; seq_lens int32 [batch];
    base3/base4 uint8 [2, kv_heads, 128]; table from new_table(); slot_ids int32 shaped like the table,
    or None to store every block as a raw BF16 tile (the uncompressed baseline).  open_compressed keeps
    each sequence's incomplete last block in its slot (GAAC_OPEN_COMPRESSED)."""
    for t, n in ((k, "k"), (v, "v"), (seq_lens, "seq_lens"), (table, "table")):
        _cuda(t, n)
    ss, ts = _kv_strides(k, "k")
    if _kv_strides(v, "v") != (ss, ts):
        raise ValueError("k and v must share strides")
    pc = pools.c()
    _check("gaac_encode_blocks_ex", lib().gaac_encode_blocks_ex(
        k.data_ptr(), v.data_ptr(), ss, ts, min(k.shape[1], v.shape[1]), seq_lens.data_ptr(), k.shape[0], k.shape[2],
        max_blocks,
        base3.data_ptr(), base4.data_ptr(), table.data_ptr(), _ptr(slot_ids), ctypes.byref(pc), _ptr(stats),
        OPEN_COMPRESSED if open_compressed else 0, _ptr(status), _stream(stream)))


def append(k_new, v_new, seq_lens, max_blocks, base3, base4, table, slot_ids, pools: Pools, stats=None,
           status=None, stream=None, open_compressed: bool = False) -> None:
    """Append one token per sequence.  k_new, v_new: BF16 [batch, kv_heads, 128]; slot_ids shaped like the
    table (the slot a block is sealed into, or kept open in with open_compressed), or None for a cache of
    raw tiles only (full tails stay raw); seq_lens is incremented."""
    pc = pools.c()
    _check("gaac_append_ex", lib().gaac_append_ex(
        k_new.data_ptr(), v_new.data_ptr(), seq_lens.data_ptr(), k_new.shape[0], k_new.shape[1], max_blocks,
        base3.data_ptr(), base4.data_ptr(), table.data_ptr(), _ptr(slot_ids), ctypes.byref(pc),
        _ptr(stats), OPEN_COMPRESSED if open_compressed else 0, _ptr(status), _stream(stream)))


def attention_workspace(batch: int, n_kv_heads: int, max_blocks: int, n_splits: int = 0) -> int:
    return lib().gaac_attention_workspace(batch, n_kv_heads, max_blocks, n_splits)


def auto_splits(batch: int, n_kv_heads: int, max_blocks: int) -> int:
    return lib().gaac_attention_auto_splits(batch, n_kv_heads, max_blocks)


def decode_attention(q, seq_lens, table, pools: Pools, base3, base4, scale: float, out, workspace, n_splits: int = 0,
                     status=None, stream=None) -> None:
    """q: BF16 [batch, q_heads, 128]; out: fp32 [batch, q_heads, 128]; workspace: uint8 device buffer."""
    batch, hq = q.shape[0], q.shape[1]
    max_blocks, hkv = table.shape[1], table.shape[2]
    pc = pools.c()
    _check("gaac_decode_attention", lib().gaac_decode_attention(
        q.data_ptr(), batch, hq, hkv, max_blocks, seq_lens.data_ptr(), table.data_ptr(), ctypes.byref(pc),
        base3.data_ptr(), base4.data_ptr(), float(scale), n_splits, out.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)))


def decode_attention_bf16(q, seq_lens, table, pools: Pools, scale: float, out, workspace, n_splits: int = 0,
                          status=None, stream=None) -> None:
    """decode_attention over an uncompressed BF16 cache (every entry a raw tile): the same kernel specialised
    to raw tiles, with no decode path."""
    batch, hq = q.shape[0], q.shape[1]
    max_blocks, hkv = table.shape[1], table.shape[2]
    pc = pools.c()
    _check("gaac_decode_attention_bf16", lib().gaac_decode_attention_bf16(
        q.data_ptr(), batch, hq, hkv, max_blocks, seq_lens.data_ptr(), table.data_ptr(), ctypes.byref(pc),
        float(scale), n_splits, out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream)))


def decompress(table, seq_lens, pools: Pools, base3, base4, k_out, v_out, status=None, stream=None) -> None:
    """Rebuild BF16 k_out/v_out [batch, tokens, kv_heads, 128] for tokens < seq_lens."""
    ss, ts = _kv_strides(k_out, "k_out")
    if _kv_strides(v_out, "v_out") != (ss, ts):
        raise ValueError("k_out and v_out must share strides")
    pc = pools.c()
    _check("gaac_decompress", lib().gaac_decompress(
        table.data_ptr(), seq_lens.data_ptr(), table.shape[0], table.shape[2], table.shape[1], ctypes.byref(pc),
        base3.data_ptr(), base4.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), ss, ts,
        min(k_out.shape[1], v_out.shape[1]), _ptr(status), _stream(stream)))


STATIC_SCRATCH_BYTES = 4 << 20


def decode_attention_noalloc(q, seq_lens, table, pools: Pools, base3, base4, scale: float, out, n_splits: int = 0,
                             status=None, stream=None) -> None:
    """decode_attention without a workspace: for callers that cannot allocate device memory at call time.
    The split partials use the library's own fixed scratch array (STATIC_SCRATCH_BYTES per device), so
    calls must not overlap on the GPU, and the first call on a device must come before any stream capture."""
    batch, hq = q.shape[0], q.shape[1]
    max_blocks, hkv = table.shape[1], table.shape[2]
    pc = pools.c()
    _check("gaac_decode_attention_noalloc", lib().gaac_decode_attention_noalloc(
        q.data_ptr(), batch, hq, hkv, max_blocks, seq_lens.data_ptr(), table.data_ptr(), ctypes.byref(pc),
        base3.data_ptr(), base4.data_ptr(), float(scale), n_splits, out.data_ptr(), _ptr(status), _stream(stream)))


# ---------------------------------------------------------------- FP8 variant of the codec
FP8_E4M3, FP8_E5M2 = 0, 1
FP8_NO_SLOT = 0xFFFF  # esc_len of a tile that stays FP8


def fp8_slot_bytes(fmt: int) -> int:
    return lib().gaac_fp8_slot_bytes(fmt)


def fp8_calibrate(x: torch.Tensor, fmt: int, base3: torch.Tensor, base4: torch.Tensor, status=None,
                  stream=None) -> None:
    """x: uint8 FP8 bits [n_tok, kv_heads, 128] (token stride free); writes uint8 base3/base4 [kv_heads, 128]."""
    _cuda(x, "x")
    if x.dtype != torch.uint8 or x.dim() != 3 or x.shape[-1] != HEAD_DIM or x.stride(2) != 1 or x.stride(1) != HEAD_DIM:
        raise ValueError("x must be uint8 [n_tok, kv_heads, 128] with contiguous heads and channels")
    _check("gaac_fp8_calibrate", lib().gaac_fp8_calibrate(x.data_ptr(), x.shape[0], x.stride(0), x.shape[1], fmt,
                                                           base3.data_ptr(), base4.data_ptr(), _ptr(status),
                                                           _stream(stream)))


def _tile_batch(tiles, slots, esc_len, tile_kind, tile_row, bases, elem_bytes: int, slot_bytes: int) -> int:
    """Checks a tile batch's tensors (device, contiguity, shapes, element sizes) and returns n."""
    n = tiles.shape[0] if tiles.dim() == 3 else -1
    for t, name in ((tiles, "tiles"), (slots, "slots"), (esc_len, "esc_len"), (tile_kind, "tile_kind"),
                    (tile_row, "tile_row"), *((b, "base") for b in bases)):
        _cuda(t, name)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if tiles.dim() != 3 or tuple(tiles.shape[1:]) != (BLOCK, HEAD_DIM) or tiles.element_size() != elem_bytes:
        raise ValueError(f"tiles must be [n, {BLOCK}, {HEAD_DIM}] of {elem_bytes}-byte elements")
    if tuple(slots.shape) != (n, slot_bytes) or slots.element_size() != 1:
        raise ValueError(f"slots must be uint8 [n, {slot_bytes}]")
    if esc_len.numel() != n or esc_len.element_size() != 2:
        raise ValueError("esc_len must hold n 16-bit values")
    if tile_kind.numel() != n or tile_kind.element_size() != 1 or tile_row.numel() != n or tile_row.dtype != torch.int32:
        raise ValueError("tile_kind must be uint8 [n] and tile_row int32 [n]")
    for b in bases:
        if b.dim() != 2 or b.shape[1] != HEAD_DIM or b.element_size() != 1 or b.shape[0] != bases[0].shape[0]:
            raise ValueError("bases must be uint8 [rows, 128], all with the same rows")
    return n


def fp8_encode_tiles(tiles, fmt: int, tile_kind, tile_row, base3, base4, slots, esc_len, stats=None, status=None,
                     stream=None) -> None:
    """tiles: uint8 [n, 64, 128]; tile_kind: uint8 [n] (0 K, 1 V); tile_row: int32 [n] (row of base3/base4
    [rows, 128]); slots: uint8 [n, fp8_slot_bytes(fmt)]; esc_len: int16 [n] (0xFFFF = stays FP8)."""
    n = _tile_batch(tiles, slots, esc_len, tile_kind, tile_row, (base3, base4), 1, fp8_slot_bytes(fmt))
    _check("gaac_fp8_encode_tiles", lib().gaac_fp8_encode_tiles(
        tiles.data_ptr(), n, fmt, tile_kind.data_ptr(), tile_row.data_ptr(), base3.shape[0], base3.data_ptr(),
        base4.data_ptr(), slots.data_ptr(), esc_len.data_ptr(), _ptr(stats), _ptr(status), _stream(stream)))


def fp8_decompress_tiles(slots, esc_len, fmt: int, tile_kind, tile_row, base3, base4, tiles, status=None,
                         stream=None) -> None:
    n = _tile_batch(tiles, slots, esc_len, tile_kind, tile_row, (base3, base4), 1, fp8_slot_bytes(fmt))
    _check("gaac_fp8_decompress_tiles", lib().gaac_fp8_decompress_tiles(
        slots.data_ptr(), esc_len.data_ptr(), n, fmt, tile_kind.data_ptr(), tile_row.data_ptr(), base3.shape[0],
        base3.data_ptr(), base4.data_ptr(), tiles.data_ptr(), _ptr(status), _stream(stream)))


def encode_tiles(tiles, tile_kind, tile_row, base3, base4, slots, esc_len, stats=None, status=None,
                 stream=None) -> None:
    """Format v3 tile batch.  tiles: BF16 [n, 64, 128] token-major; tile_kind: uint8 [n] (0 K, 1 V);
    tile_row: int32 [n] (row of base3/base4 [rows, 128]); slots: uint8 [n, SLOT_BYTES]; esc_len: int16 [n]
    (0xFFFF: does not fit, slot untouched)."""
    n = _tile_batch(tiles, slots, esc_len, tile_kind, tile_row, (base3, base4), 2, SLOT_BYTES)
    _check("gaac_encode_tiles", lib().gaac_encode_tiles(
        tiles.data_ptr(), n, tile_kind.data_ptr(), tile_row.data_ptr(), base3.shape[0],
        base3.data_ptr(), base4.data_ptr(), slots.data_ptr(), esc_len.data_ptr(), _ptr(stats), _ptr(status),
        _stream(stream)))


def decode_tiles(slots, esc_len, tile_kind, tile_row, base3, base4, tiles, status=None, stream=None) -> None:
    n = _tile_batch(tiles, slots, esc_len, tile_kind, tile_row, (base3, base4), 2, SLOT_BYTES)
    _check("gaac_decode_tiles", lib().gaac_decode_tiles(
        slots.data_ptr(), esc_len.data_ptr(), n, tile_kind.data_ptr(), tile_row.data_ptr(),
        base3.shape[0], base3.data_ptr(), base4.data_ptr(), tiles.data_ptr(), _ptr(status), _stream(stream)))


NESTED_SLOT_BYTES = 12048


def nested_calibrate(x: torch.Tensor, base2: torch.Tensor, status=None, stream=None) -> None:
    """x: BF16 [n_tok, kv_heads, 128] -> base2 uint8 [kv_heads, 128] (best 4-exponent window)."""
    _cuda(x, "x")
    if x.dim() != 3 or x.shape[-1] != HEAD_DIM or x.stride(2) != 1 or x.stride(1) != HEAD_DIM:
        raise ValueError("x must be [n_tok, kv_heads, 128] with contiguous heads and channels")
    _check("gaac_nested_calibrate", lib().gaac_nested_calibrate(x.data_ptr(), x.shape[0], x.stride(0), x.shape[1],
                                                                 base2.data_ptr(), _ptr(status), _stream(stream)))


def nested_encode_tiles(tiles, tile_kind, tile_row, base2, base3, base4, slots, esc_len, status=None,
                        stream=None) -> None:
    """Nested 2-bit-mode ablation format; arguments as encode_tiles, slots [n, NESTED_SLOT_BYTES]."""
    n = _tile_batch(tiles, slots, esc_len, tile_kind, tile_row, (base2, base3, base4), 2, NESTED_SLOT_BYTES)
    _check("gaac_nested_encode_tiles", lib().gaac_nested_encode_tiles(
        tiles.data_ptr(), n, tile_kind.data_ptr(), tile_row.data_ptr(), base3.shape[0],
        base2.data_ptr(), base3.data_ptr(), base4.data_ptr(), slots.data_ptr(), esc_len.data_ptr(), _ptr(status),
        _stream(stream)))


def nested_decode_tiles(slots, esc_len, tile_kind, tile_row, base2, base3, base4, tiles, status=None,
                        stream=None) -> None:
    n = _tile_batch(tiles, slots, esc_len, tile_kind, tile_row, (base2, base3, base4), 2, NESTED_SLOT_BYTES)
    _check("gaac_nested_decode_tiles", lib().gaac_nested_decode_tiles(
        slots.data_ptr(), esc_len.data_ptr(), n, tile_kind.data_ptr(), tile_row.data_ptr(),
        base3.shape[0], base2.data_ptr(), base3.data_ptr(), base4.data_ptr(), tiles.data_ptr(), _ptr(status),
        _stream(stream)))


def decode_attention_hd256(q, seq_lens, table, pools: Pools, base3, base4, scale: float, out, workspace,
                           n_splits: int = 0, status=None, stream=None) -> None:
    """Attention over 256-channel heads stored as two 128-channel half-heads: q BF16 [batch, n_q_heads, 256],
    table [batch, max_blocks, 2 * n_kv_heads, 2], base3/base4 [2, 2 * n_kv_heads, 128], out fp32
    [batch, n_q_heads, 256]; workspace >= attention_workspace(batch, 2 * n_kv_heads, max_blocks, n_splits)."""
    B, Hq, d = q.shape
    if d != 256 or out.shape != (B, Hq, 256):
        raise ValueError("q and out must be [batch, n_q_heads, 256]")
    n_kv = table.shape[2] // 2
    pc = pools.c()
    _check("gaac_decode_attention_hd256", lib().gaac_decode_attention_hd256(
        q.data_ptr(), B, Hq, n_kv, table.shape[1], seq_lens.data_ptr(), table.data_ptr(), ctypes.byref(pc),
        base3.data_ptr(), base4.data_ptr(), float(scale), n_splits, out.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)))


def _stream_object(stream, device) -> torch.cuda.Stream | None:
    """The torch stream of a call's `stream` argument: a stream, a raw handle or None, which stays None."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle in (0, 1, 2):  # the default stream, or a thread's, which keeps its order with that
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(handle, device=device)


def _made_for(stream, device, make) -> torch.Tensor:
    """make()'s tensor for a call on `stream` (None: the current one).  It is made on that stream, so its memory is not
    what the current stream's pending work still uses, and not given out again before the current stream, where it
    may be read, is past its use."""
    if stream is None:
        return make()
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(_stream_object(stream, device)):
        t = make()
    t.record_stream(current)
    return t


# ---------------------------------------------------------------- rotary positions
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # GAAC_BF16, GAAC_F16, GAAC_F32
ROPE_INTERLEAVED, ROPE_INVERSE = 1, 2


class gaac_rope_tensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n_heads", ctypes.c_int32),
                ("x_seq", ctypes.c_int64), ("x_tok", ctypes.c_int64), ("x_head", ctypes.c_int64),
                ("out_seq", ctypes.c_int64), ("out_tok", ctypes.c_int64), ("out_head", ctypes.c_int64)]


_ROPE_TENSOR = struct.Struct("@PPi6q")  # gaac_rope_tensor packed in one go
assert _ROPE_TENSOR.size == ctypes.sizeof(gaac_rope_tensor)


def rope_frequencies(rot_dim: int, theta: float = 1e4, scaling: str | None = None, factor: float = 1.0,
                     original_len: int | None = None, fast: float = 32.0, slow: float = 1.0):
    """(w, mscale): the angular frequencies w_j = theta^(-2j/rot_dim) as a float64 tensor [rot_dim/2], scaled for
    a context `factor` times the trained one, and the multiplier of the rotated channels that goes with them.

    scaling None: as they are.  "linear": w / factor (positions interpolated).  "base": theta stretched to
    theta * factor^(rot_dim/(rot_dim-2)), which leaves the fastest pair alone and slows the slowest by factor.
    "bands": by how often a pair turns within original_len tokens: `fast` turns and more keep w, `slow` and fewer
    get w / factor, linear in the pair's index between; mscale = 0.1 ln(factor) + 1.  That is YaRN's scaling (Peng et
    al., 2023) with the ramp over indices in common use: from that of `fast` turns, rounded down and at least 0, to
    that of `slow`, rounded up, which may lie behind the last pair."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    if not theta > 0 or not factor > 0:
        raise ValueError("theta and factor must be positive")
    j = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError("base scaling needs rot_dim >= 4")
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    w = theta ** (-2.0 * j / rot_dim)
    if scaling in (None, "base"):
        return w, 1.0
    if scaling == "linear":
        return w / factor, 1.0
    if scaling != "bands":
        raise ValueError("scaling must be None, 'linear', 'base' or 'bands'")
    if not original_len or original_len <= 0 or not fast > slow > 0 or not theta > 1:
        raise ValueError("band scaling needs original_len > 0, fast > slow > 0 and theta > 1")

    def pair_of(turns):  # the (real) index of the pair that turns so often within original_len
        return rot_dim * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(theta))

    lo = max(0.0, math.floor(pair_of(fast)))
    hi = math.ceil(pair_of(slow))
    keep = 1.0 - ((j - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
    return w * keep + w / factor * (1.0 - keep), (0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0)


def rope_turns(w: torch.Tensor, device=None) -> torch.Tensor:
    """The angular frequencies w (radians per position) as fractions of a turn in 64-bit fixed point, the form
    rope() takes: int64 tensor of round(w / (2 pi) * 2^64) modulo 2^64, on `device` (default: w's)."""
    if w.dim() != 1:
        raise ValueError("w must be one-dimensional")
    values = w.double().tolist()
    if not all(math.isfinite(x) for x in values):
        raise ValueError("frequencies must be finite")
    fixed = [round(x / (2 * math.pi) * 2.0 ** 64) & (2 ** 64 - 1) for x in values]
    return torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in fixed], dtype=torch.int64,
                        device=w.device if device is None else device)


def _gpu(*tensors) -> int:
    """The index of the CUDA device that all of them are on."""
    index = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != index or index < 0:
            raise ValueError("tensors must be on one CUDA device")
    return index


# The current stream's handle, without the stream object that torch.cuda.current_stream() makes (2 us a call), and
# the current device.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(fn: str, index: int, stream, *args):
    """Calls the library with device `index` current and the stream (default: the device's current one) last."""
    if index != _current_device():
        with torch.cuda.device(index):
            return _call(fn, index, stream, *args)
    if stream is None:
        s = _raw_stream(index)
    else:
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    status = getattr(_lib or lib(), fn)(*args, s)
    if status != OK:
        raise GaacError(fn, status)


def _rope_pair(x, out, dtype, index, name):
    """gaac_rope_tensor of an input [tokens, heads, dim] or [batch, tokens, heads, dim] and its output (None: in place),
    and the input's shape."""
    shape, st = x.shape, x.stride()
    n = len(shape)
    if n != 3 and n != 4:
        raise ValueError(f"{name} must be [tokens, heads, dim] or [batch, tokens, heads, dim]")
    if x.dtype != dtype or x.get_device() != index or (st[-1] != 1 and shape[-1] > 1):
        raise ValueError(f"{name} must be of q's type and device, channels contiguous")
    at = x.data_ptr()
    if out is None:
        out_at, so = at, st
    else:
        out_at, so = out.data_ptr(), out.stride()
        if out.shape != shape or out.dtype != dtype or out.get_device() != index or (so[-1] != 1 and shape[-1] > 1):
            raise ValueError(f"{name}_out must have {name}'s shape, type and device, channels contiguous")
    if n == 3:
        return _ROPE_TENSOR.pack(at, out_at, shape[1], 0, st[0], st[1], 0, so[0], so[1]), shape
    return _ROPE_TENSOR.pack(at, out_at, shape[2], st[0], st[1], st[2], so[0], so[1], so[2]), shape


def rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, turns: torch.Tensor, q_out=None, k_out=None,
         interleaved: bool = False, mscale: float = 1.0, inverse: bool = False, stream=None) -> None:
    """Rotary positions of q and, if given, k in one launch.  q, k: [tokens, heads, dim] or [batch, tokens, heads,
    dim], BF16, FP16 or FP32, channels contiguous, other strides free; positions: int32 or int64, [tokens] or
    [batch, tokens]; turns: rope_turns(...), one for each pair of the rotated channels (the first
    2 * turns.numel() of a head; the others are copied).  Pairs are (j, j + half) or, interleaved, (2j, 2j + 1).
    q_out, k_out: default in place; q and k share no elements, nor do their outputs with the other's.  inverse turns
    the other way: the gradient of the call without it.  Autograd does not see either, so tensors that require a
    gradient are refused while it records: call it under torch.no_grad() or from a torch.autograd.Function, with
    inverse in its backward."""
    if (q.requires_grad or (k is not None and k.requires_grad) or (q_out is not None and q_out.requires_grad) or
            (k_out is not None and k_out.requires_grad)) and torch.is_grad_enabled():
        raise ValueError("autograd does not see rope: call it under torch.no_grad() or from an autograd.Function")
    dtype, index = q.dtype, q.get_device()
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("q must be BF16, FP16 or FP32")
    if index < 0 or positions.get_device() != index or turns.get_device() != index:
        raise ValueError("tensors must be on one CUDA device")
    desc, shape = _rope_pair(q, q_out, dtype, index, "q")
    count = 1
    if k is not None:
        more, k_shape = _rope_pair(k, k_out, dtype, index, "k")
        if k_shape[:-2] != shape[:-2] or k_shape[-1] != shape[-1]:
            raise ValueError("k must have q's tokens and width")
        desc += more
        count = 2
    elif k_out is not None:
        raise ValueError("k_out without k")
    turns_shape = turns.shape
    if turns.dtype != torch.int64 or len(turns_shape) != 1 or not turns.is_contiguous():
        raise ValueError("turns must be a contiguous int64 tensor [pairs]")
    pos_type = positions.dtype
    if pos_type != torch.int32 and pos_type != torch.int64:
        raise ValueError("positions must be int32 or int64")
    n_seq, n_tok = (1, shape[0]) if len(shape) == 3 else shape[:2]
    pos_shape, ps = positions.shape, positions.stride()
    if len(pos_shape) == 1 and pos_shape[0] == n_tok:
        ps = (0, ps[0])
    elif len(shape) != 4 or pos_shape != shape[:2]:
        raise ValueError("positions must be [tokens] or [batch, tokens]")
    _call("gaac_rope", index, stream, desc, count, code, n_seq, n_tok, shape[-1], 2 * turns_shape[0], positions.data_ptr(),
          32 if pos_type == torch.int32 else 64, *ps, turns.data_ptr(), mscale,
          (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_INVERSE if inverse else 0))


class gaac_norm_tensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("dz", ctypes.c_void_p), ("out", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("dweight", ctypes.c_void_p), ("n_heads", ctypes.c_int32),
                ("x_seq", ctypes.c_int64), ("x_tok", ctypes.c_int64), ("x_head", ctypes.c_int64),
                ("dz_seq", ctypes.c_int64), ("dz_tok", ctypes.c_int64), ("dz_head", ctypes.c_int64),
                ("out_seq", ctypes.c_int64), ("out_tok", ctypes.c_int64), ("out_head", ctypes.c_int64)]


_NORM_TENSOR = struct.Struct("@5Pi9q")  # gaac_norm_tensor packed in one go
assert _NORM_TENSOR.size == ctypes.sizeof(gaac_norm_tensor)


def _norm_input(x, dz, out, weight, dweight, dtype, index, name):
    """gaac_norm_tensor of an input, its result's gradient (None in the forward pass), the output (None: in place of dz,
    else of x) and the weights; the input's shape and the weights' type (None without them)."""
    shape, st = x.shape, x.stride()
    n = len(shape)
    if (n != 3 and n != 4) or x.dtype != dtype or x.get_device() != index or (st[-1] != 1 and shape[-1] > 1):
        raise ValueError(f"{name} must be [tokens, heads, dim] or [batch, tokens, heads, dim] of q's type and device, "
                         "channels contiguous")
    at = out_at = x.data_ptr()
    so, z_at, zs = st, 0, (0, 0, 0)
    if dz is not None:
        z_at, zs = dz.data_ptr(), dz.stride()
        if dz.shape != shape or dz.dtype != dtype or dz.get_device() != index or (zs[-1] != 1 and shape[-1] > 1):
            raise ValueError(f"d{name} must have {name}'s shape, type and device, channels contiguous")
        out_at, so = z_at, zs
    if out is not None:
        out_at, so = out.data_ptr(), out.stride()
        if out.shape != shape or out.dtype != dtype or out.get_device() != index or (so[-1] != 1 and shape[-1] > 1):
            raise ValueError(f"{name}'s output must have its shape, type and device, channels contiguous")
    w_at, w_type, d_at = 0, None, 0
    if weight is not None:
        w_at, w_type, ws = weight.data_ptr(), weight.dtype, weight.shape
        if len(ws) != 1 or ws[0] != shape[-1] or (w_type != dtype and w_type != torch.float32) or \
                weight.get_device() != index or not weight.is_contiguous():
            raise ValueError(f"{name}'s weights must be contiguous [dim] on its device, of its type or fp32")
    if dweight is not None:
        d_at, ws = dweight.data_ptr(), dweight.shape
        if len(ws) != 1 or ws[0] != shape[-1] or dweight.dtype != torch.float32 or dweight.get_device() != index or \
                not dweight.is_contiguous():
            raise ValueError(f"the gradient of {name}'s weights must be contiguous fp32 [dim] on its device")
    if n == 3:
        return _NORM_TENSOR.pack(at, z_at, out_at, w_at, d_at, shape[1], 0, st[0], st[1], 0, zs[0], zs[1], 0, so[0],
                                 so[1]), shape, w_type
    return _NORM_TENSOR.pack(at, z_at, out_at, w_at, d_at, shape[2], st[0], st[1], st[2], zs[0], zs[1], zs[2], so[0], so[1],
                             so[2]), shape, w_type


def _norm_rope(fn, q, k, dq, dk, q_out, k_out, q_weight, k_weight, dq_weight, dk_weight, positions, turns, interleaved,
               mscale, eps, stream, *more):
    if (q.requires_grad or (k is not None and k.requires_grad) or (q_weight is not None and q_weight.requires_grad) or
            (k_weight is not None and k_weight.requires_grad) or (q_out is not None and q_out.requires_grad) or
            (k_out is not None and k_out.requires_grad) or (dq is not None and dq.requires_grad) or
            (dk is not None and dk.requires_grad) or (dq_weight is not None and dq_weight.requires_grad) or
            (dk_weight is not None and dk_weight.requires_grad)) and torch.is_grad_enabled():
        raise ValueError("autograd does not see qk_norm_rope: call it under torch.no_grad() or from an autograd.Function")
    dtype, index = q.dtype, q.get_device()
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("q must be BF16, FP16 or FP32")
    if index < 0 or positions.get_device() != index or turns.get_device() != index:
        raise ValueError("tensors must be on one CUDA device")
    desc, shape, w_type = _norm_input(q, dq, q_out, q_weight, dq_weight, dtype, index, "q")
    count = 1
    if k is not None:
        second, k_shape, k_type = _norm_input(k, dk, k_out, k_weight, dk_weight, dtype, index, "k")
        if k_shape[:-2] != shape[:-2] or k_shape[-1] != shape[-1]:
            raise ValueError("k must have q's tokens and width")
        if w_type is None:
            w_type = k_type
        elif k_type is not None and k_type != w_type:
            raise ValueError("the weights of q and k must be of one type")
        desc += second
        count = 2
    elif k_out is not None or k_weight is not None or dk_weight is not None:
        raise ValueError("k's output or weights without k")
    turns_shape = turns.shape
    if turns.dtype != torch.int64 or len(turns_shape) != 1 or not turns.is_contiguous():
        raise ValueError("turns must be a contiguous int64 tensor [pairs]")
    pos_type = positions.dtype
    if pos_type != torch.int32 and pos_type != torch.int64:
        raise ValueError("positions must be int32 or int64")
    n_seq, n_tok = (1, shape[0]) if len(shape) == 3 else shape[:2]
    pos_shape, ps = positions.shape, positions.stride()
    if len(pos_shape) == 1 and pos_shape[0] == n_tok:
        ps = (0, ps[0])
    elif len(shape) != 4 or pos_shape != shape[:2]:
        raise ValueError("positions must be [tokens] or [batch, tokens]")
    _call(fn, index, stream, desc, count, code, code if w_type is None else _DTYPES[w_type], n_seq, n_tok, shape[-1],
          2 * turns_shape[0], positions.data_ptr(), 32 if pos_type == torch.int32 else 64, *ps, turns.data_ptr(), mscale,
          eps, ROPE_INTERLEAVED if interleaved else 0, *more)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, q_weight: torch.Tensor | None, k_weight: torch.Tensor | None,
                 positions: torch.Tensor, turns: torch.Tensor, eps: float = 1e-6, q_out=None, k_out=None,
                 interleaved: bool = False, mscale: float = 1.0, stream=None) -> None:
    """Norms of every head of q and, if given, k, x / sqrt(mean(x^2) + eps) * weight, and their rotary positions, in
    one pass.  q_weight, k_weight: [dim] of q's type or fp32, None for ones; dim is at most 256.  Everything else as
    in rope: in place by default, and not seen by autograd (qk_norm_rope_gradient is its backward)."""
    _norm_rope("gaac_qk_norm_rope", q, k, None, None, q_out, k_out, q_weight, k_weight, None, None, positions, turns,
               interleaved, mscale, eps, stream)


def qk_norm_rope_workspace(dim: int) -> int:
    """Bytes of qk_norm_rope_gradient's workspace, of any contents."""
    return lib().gaac_qk_norm_rope_workspace(dim)


def qk_norm_rope_gradient(dq: torch.Tensor, dk: torch.Tensor | None, q: torch.Tensor, k: torch.Tensor | None,
                          q_weight: torch.Tensor | None, k_weight: torch.Tensor | None, positions: torch.Tensor,
                          turns: torch.Tensor, dq_weight: torch.Tensor | None, dk_weight: torch.Tensor | None,
                          workspace: torch.Tensor, eps: float = 1e-6, dq_out=None, dk_out=None, interleaved: bool = False,
                          mscale: float = 1.0, stream=None) -> None:
    """The backward pass of qk_norm_rope: dq, dk are the gradients of its results, q and k what it was given (not
    its results).  dq_out, dk_out receive the gradients of q and k (default: in place of dq and dk), dq_weight and
    dk_weight, fp32 [dim] or None, those of the weights.  workspace: qk_norm_rope_workspace(dim) bytes, not shared by
    calls that may overlap on the GPU."""
    if (dk is None) != (k is None) or dq is None:
        raise ValueError("q and k each go with their gradient")
    if workspace.get_device() != q.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on q's device")
    _norm_rope("gaac_qk_norm_rope_gradient", q, k, dq, dk, dq_out, dk_out, q_weight, k_weight, dq_weight, dk_weight,
               positions, turns, interleaved, mscale, eps, stream, workspace.data_ptr(), workspace.nbytes)


# ---------------------------------------------------------------- attention of prompts
class gaac_prompt(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "out", "lse")] + \
        [(n, ctypes.c_int64) for n in ("q_tok", "q_head", "k_tok", "k_head", "v_tok", "v_head", "out_tok", "out_head")]


_PROMPT = struct.Struct("@5P8q")  # gaac_prompt packed in one go
assert _PROMPT.size == ctypes.sizeof(gaac_prompt)


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_tokens: torch.Tensor, scale: float,
                     out: torch.Tensor | None = None, lse: torch.Tensor | None = None, status=None,
                     stream=None) -> torch.Tensor:
    """Causal attention of whole prompts, packed: rows cu_tokens[b] .. cu_tokens[b + 1] (int32 [batch + 1]) are the tokens
    of sequence b, and a token attends to itself and those before it in its sequence.  q: [n, q_heads, 128]; k, v:
    [n, kv_heads, 128], at most 8 query heads to a kv-head; BF16 or FP16, channels contiguous, other strides free
    (multiples of 8 elements, 16-byte aligned: slices of one projection will do).  out: of q's shape and type (made,
    contiguous, if not given; rows of no sequence are not written), with no element of an input's (another slice of the
    projection will do); lse: fp32 [n, q_heads], contiguous, memory of its own, receives the
    logarithm of each row's sum of exponentials.  Offsets that are not valid leave out as it was, and like everything that
    only the device sees they are reported in status (int32), if it is given."""
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or
                                    (out is not None and out.requires_grad) or (lse is not None and lse.requires_grad)):
        raise ValueError("autograd does not see prompt_attention: call it under torch.no_grad()")
    dtype, index = q.dtype, q.get_device()
    if dtype not in (torch.bfloat16, torch.float16) or index < 0:
        raise ValueError("q must be BF16 or FP16 on a CUDA device")
    n, hq = q.shape[:2] if q.dim() == 3 else (-1, -1)
    hkv = k.shape[1] if k.dim() == 3 else -1
    if out is None:
        out = _made_for(stream, q.device, lambda: torch.empty(q.shape, dtype=dtype, device=q.device))
    for t, shape, name in ((q, (n, hq, HEAD_DIM), "q"), (k, (n, hkv, HEAD_DIM), "k"), (v, (n, hkv, HEAD_DIM), "v"),
                           (out, (n, hq, HEAD_DIM), "out")):
        if t.shape != shape or t.dtype != dtype or t.get_device() != index or t.stride(2) != 1:
            raise ValueError(f"{name} must be [tokens, heads, {HEAD_DIM}] of q's type and device, channels contiguous")
    if cu_tokens.dtype != torch.int32 or cu_tokens.dim() != 1 or cu_tokens.shape[0] < 1 or not cu_tokens.is_contiguous() or \
            cu_tokens.get_device() != index:
        raise ValueError("cu_tokens must be a contiguous int32 tensor [batch + 1] on q's device")
    if lse is not None and (lse.shape != (n, hq) or lse.dtype != torch.float32 or not lse.is_contiguous() or
                            lse.get_device() != index):
        raise ValueError("lse must be contiguous fp32 [tokens, q_heads] on q's device")
    if status is not None and (status.get_device() != index or status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status must be an int32 tensor on q's device")
    desc = _PROMPT.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(lse) or 0, *q.stride()[:2],
                        *k.stride()[:2], *v.stride()[:2], *out.stride()[:2])
    _call("gaac_prompt_attention", index, stream, desc, _DTYPES[dtype], n, hq, hkv, cu_tokens.data_ptr(),
          cu_tokens.shape[0] - 1, scale, _ptr(status))
    return out


# ---------------------------------------------------------------- 8-bit paged cache
class gaac_kv8(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tail", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("work", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("max_blocks", ctypes.c_int32), ("fmt", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class Kv8:
    """Storage of one layer's 8-bit paged cache around the caller's tensors, which stay the ones it was made with.

    pages: uint8 [n_pages, kv_heads, 2, 64, 128]; scales: fp32 [n_pages, kv_heads, 2]; tail: BF16 or FP16
    [batch, kv_heads, 2, 64, 128]; table: int32 [batch, max_blocks]; refs: int32 [n_pages]; seq_lens: int32
    [batch].  fmt: FP8_E4M3 or FP8_E5M2."""

    def __init__(self, pages, scales, tail, table, refs, seq_lens, fmt: int):
        self._index = _gpu(pages, scales, tail, table, refs, seq_lens)
        self.device = pages.device
        if pages.dim() != 5 or tuple(pages.shape[2:]) != (2, BLOCK, HEAD_DIM) or pages.dtype != torch.uint8:
            raise ValueError(f"pages must be uint8 [n_pages, kv_heads, 2, {BLOCK}, {HEAD_DIM}]")
        n_pages, heads = pages.shape[:2]
        if tuple(scales.shape) != (n_pages, heads, 2) or scales.dtype != torch.float32:
            raise ValueError("scales must be fp32 [n_pages, kv_heads, 2]")
        if table.dim() != 2 or table.dtype != torch.int32:
            raise ValueError("table must be int32 [batch, max_blocks]")
        batch, max_blocks = table.shape
        if tuple(tail.shape) != (batch, heads, 2, BLOCK, HEAD_DIM) or tail.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"tail must be BF16 or FP16 [batch, kv_heads, 2, {BLOCK}, {HEAD_DIM}]")
        if tuple(refs.shape) != (n_pages,) or refs.dtype != torch.int32:
            raise ValueError("refs must be int32 [n_pages]")
        if tuple(seq_lens.shape) != (batch,) or seq_lens.dtype != torch.int32:
            raise ValueError("seq_lens must be int32 [batch]")
        if fmt not in (FP8_E4M3, FP8_E5M2):
            raise ValueError("fmt must be FP8_E4M3 or FP8_E5M2")
        for t, name in ((pages, "pages"), (scales, "scales"), (tail, "tail"), (table, "table"), (refs, "refs"),
                        (seq_lens, "seq_lens")):
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        self.batch, self.max_blocks, self.n_pages, self.n_kv_heads, self.fmt = batch, max_blocks, n_pages, heads, fmt
        self.dtype = tail.dtype
        work = torch.zeros(max(4, lib().gaac_kv8_workspace(batch, n_pages) // 4), dtype=torch.int32, device=self.device)
        self._tensors = (pages, scales, tail, table, refs, seq_lens, work)
        self._c = gaac_kv8(*(t.data_ptr() for t in self._tensors), n_pages, batch, heads, max_blocks, fmt,
                           _DTYPES[tail.dtype])
        self._ref = ctypes.byref(self._c)
        self._own_status = (None, 0)  # a status tensor made with the cache, and its address

    pages = property(lambda s: s._tensors[0])
    scales = property(lambda s: s._tensors[1])
    tail = property(lambda s: s._tensors[2])
    table = property(lambda s: s._tensors[3])
    refs = property(lambda s: s._tensors[4])
    seq_lens = property(lambda s: s._tensors[5])


def _index_list(t, name, cache):
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.get_device() != cache._index:
        raise ValueError(f"{name} must be a contiguous int32 tensor on the cache's device")
    return t.shape[0]


def _kv8_cu(cache: Kv8, cu_tokens):
    if cu_tokens is None:
        return 0
    if _index_list(cu_tokens, "cu_tokens", cache) != cache.batch + 1:
        raise ValueError("cu_tokens must hold batch + 1 offsets")
    return cu_tokens.data_ptr()


def _kv8_rows(cache: Kv8, t, heads, name):
    """Row stride of t [n, heads (any if None), 128] of the cache's type, heads and channels contiguous; n."""
    shape, st = t.shape, t.stride()
    if t.dtype != cache.dtype or t.get_device() != cache._index or len(shape) != 3 or shape[2] != HEAD_DIM or \
            (heads is not None and shape[1] != heads) or st[2] != 1 or (st[1] != HEAD_DIM and shape[1] > 1):
        raise ValueError(f"{name} must be [n, heads, {HEAD_DIM}] of the cache's type and device, heads and channels "
                         "contiguous")
    return shape[0], (st[0] if shape[0] > 1 else shape[1] * HEAD_DIM)


def _kv8_status(cache: Kv8, status):
    own, at = cache._own_status
    if status is own:
        return at
    if status is None:
        return 0
    if status.get_device() != cache._index or status.dtype != torch.int32 or status.numel() < 1:
        raise ValueError("status must be an int32 tensor on the cache's device")
    return status.data_ptr()


def kv8_append(cache: Kv8, k: torch.Tensor, v: torch.Tensor, cu_tokens: torch.Tensor | None = None, status=None,
               stream=None, reserve: bool = False) -> None:
    """Appends rows cu_tokens[b] .. cu_tokens[b + 1] of k and v ([n, kv_heads, 128] of the cache's type, heads and
    channels contiguous) to sequence b; without cu_tokens (int32 [batch + 1]) one row for each sequence.  The pages
    of blocks that fill must have been reserved, or are with reserve=True."""
    cu = _kv8_cu(cache, cu_tokens)
    n, k_row = _kv8_rows(cache, k, cache.n_kv_heads, "k")
    n_v, v_row = _kv8_rows(cache, v, cache.n_kv_heads, "v")
    if n_v != n or (cu == 0 and n != cache.batch):
        raise ValueError("k and v must hold the same rows: one for each sequence without cu_tokens")
    _call("gaac_kv8_reserve_append" if reserve else "gaac_kv8_append", cache._index, stream, cache._ref, k.data_ptr(),
          v.data_ptr(), n, k_row, v_row, cu, _kv8_status(cache, status))


def kv8_attention_workspace() -> int:
    """Bytes of decode attention's workspace on the current device; zero them before the first call."""
    return lib().gaac_kv8_attention_workspace()


def kv8_decode_attention(cache: Kv8, q: torch.Tensor, scale: float, out: torch.Tensor, workspace: torch.Tensor,
                         status=None, stream=None) -> None:
    """q: [batch, q_heads, 128] of the cache's type (rows may be strided); out: the same shape, contiguous, of the
    cache's type or fp32; workspace: kv8_attention_workspace() bytes, zero before the first call."""
    n, row = _kv8_rows(cache, q, None, "q")
    code = _DTYPES.get(out.dtype)
    if n != cache.batch or out.shape != q.shape or (out.dtype != cache.dtype and code != 2) or \
            out.get_device() != cache._index or not out.is_contiguous():
        raise ValueError("q must have a row for each sequence, and out must be contiguous, of q's shape and device, in "
                         "the cache's type or fp32")
    if workspace.get_device() != cache._index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the cache's device")
    _call("gaac_kv8_decode_attention", cache._index, stream, cache._ref, q.data_ptr(), q.shape[1], row, scale,
          out.data_ptr(), code, workspace.data_ptr(), workspace.nbytes, _kv8_status(cache, status))


def kv8_reserve(cache: Kv8, cu_tokens: torch.Tensor | None = None, status=None, stream=None) -> None:
    """Pages for the blocks that appending these tokens fills: the lowest free ones, in order of sequence and block.
    When they run out, sequences keep what they have got."""
    _call("gaac_kv8_reserve", cache._index, stream, cache._ref, _kv8_cu(cache, cu_tokens), _kv8_status(cache, status))


def kv8_release(cache: Kv8, seqs: torch.Tensor, status=None, stream=None) -> None:
    """Empties the listed sequences (int32); pages that no other sequence holds become free."""
    n = _index_list(seqs, "seqs", cache)
    _call("gaac_kv8_release", cache._index, stream, cache._ref, seqs.data_ptr(), n, _kv8_status(cache, status))


def kv8_fork(cache: Kv8, src: torch.Tensor, dst: torch.Tensor, status=None, stream=None) -> None:
    """Empty sequences dst (int32) become copies of src, sharing their full blocks."""
    n = _index_list(src, "src", cache)
    if _index_list(dst, "dst", cache) != n:
        raise ValueError("src and dst must have the same length")
    _call("gaac_kv8_fork", cache._index, stream, cache._ref, src.data_ptr(), dst.data_ptr(), n, _kv8_status(cache, status))


def kv8_reorder(cache: Kv8, parents: torch.Tensor, status=None, stream=None) -> None:
    """parents: int32 [groups, beams], groups * beams sequences: sequence g * beams + i becomes what
    g * beams + parents[g, i] was, all at once.  Full blocks are shared, open blocks copied, reserved pages of the
    sequences that change given back."""
    if parents.dtype != torch.int32 or parents.dim() != 2 or not parents.is_contiguous() or \
            parents.get_device() != cache._index or parents.numel() != cache.batch:
        raise ValueError("parents must be a contiguous int32 tensor [groups, beams] of the cache's sequences and device")
    _call("gaac_kv8_reorder", cache._index, stream, cache._ref, parents.data_ptr(), parents.shape[1], _kv8_status(cache, status))


def kv8_compact(cache: Kv8, moved_to: torch.Tensor, stream=None) -> None:
    """Moves the held pages to the front of the pool; moved_to (int32 [n_pages]) gets each page's new place, -1 for
    free ones."""
    if _index_list(moved_to, "moved_to", cache) != cache.n_pages:
        raise ValueError("moved_to must hold n_pages values")
    _call("gaac_kv8_compact", cache._index, stream, cache._ref, moved_to.data_ptr())


# ---------------------------------------------------------------- beam search
def beam_workspace(batch: int, beams: int, vocab: int, n_out: int) -> int:
    """Bytes of beam_select's workspace, which is zero before the first call and serves calls of these sizes; 0 for sizes
    that it does not take."""
    return lib().gaac_beam_workspace(batch, beams, vocab, n_out)


def beam_select(logits: torch.Tensor, scores: torch.Tensor, out_scores: torch.Tensor, parents: torch.Tensor,
                tokens: torch.Tensor, workspace: torch.Tensor, ended: torch.Tensor | None = None, end_token: int = 0,
                stream=None) -> None:
    """The n_out largest of scores[b, i] + log_softmax(logits[b * beams + i])[t] over beams i and tokens t, for each
    search b, in descending order, equal ones by i, then t.  logits: [batch * beams, vocab], BF16, FP16 or FP32, tokens
    contiguous (rows may be strided); scores: fp32 [batch, beams].  out_scores (fp32), parents (the beam i) and tokens
    (int32): [batch, n_out].  ended: bool or uint8 [batch, beams]; such a beam has one candidate, end_token, at its score.
    A beam whose score or sum of exponentials is not finite has none; where there are too few, the lowest of the others
    follow at -infinity.  workspace: beam_workspace(...) bytes, zero before the first call, for calls of the same sizes that do
    not overlap on the GPU."""
    index = logits.get_device()
    code = _DTYPES.get(logits.dtype)
    if torch.is_grad_enabled() and (logits.requires_grad or scores.requires_grad or out_scores.requires_grad):
        raise ValueError("autograd does not see beam_select: call it under torch.no_grad()")
    if code is None or logits.dim() != 2 or index < 0 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be BF16, FP16 or FP32 [batch * beams, vocab] on a CUDA device, tokens contiguous")
    if scores.dim() != 2 or scores.dtype != torch.float32 or not scores.is_contiguous() or scores.get_device() != index or \
            scores.numel() != logits.shape[0]:
        raise ValueError("scores must be contiguous fp32 [batch, beams] on the logits' device")
    batch, beams = scores.shape
    shape = out_scores.shape
    if len(shape) != 2 or shape[0] != batch or parents.shape != shape or tokens.shape != shape:
        raise ValueError("out_scores, parents and tokens must be [batch, n_out]")
    for t, dtype, name in ((out_scores, torch.float32, "out_scores"), (parents, torch.int32, "parents"),
                           (tokens, torch.int32, "tokens")):
        if t.dtype != dtype or t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous on the logits' device, of {dtype}")
    if ended is not None and (ended.dtype not in (torch.bool, torch.uint8) or ended.shape != scores.shape or
                              not ended.is_contiguous() or ended.get_device() != index):
        raise ValueError("ended must be contiguous bool or uint8 [batch, beams] on the logits' device")
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the logits' device")
    _call("gaac_beam_select", index, stream, logits.data_ptr(), code, max(logits.stride(0), logits.shape[1]) if
          logits.shape[0] <= 1 else logits.stride(0), scores.data_ptr(), 0 if ended is None else ended.data_ptr(), end_token,
          batch, beams, logits.shape[1], shape[1], out_scores.data_ptr(), parents.data_ptr(), tokens.data_ptr(),
          workspace.data_ptr(), workspace.nbytes)
