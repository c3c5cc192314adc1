"""Binding of the indexer's paged key cache (include/indexer_paged.h).

Argument marshalling only, as in the package's other calls: every step runs in
the library's HIP kernels, on `stream` (default: torch's current stream of the
tensors' device), and a call that cannot be made raises.  Outputs that the caller
does not pass come from torch's allocator on that stream.  With `stream`, the caller
keeps the inputs (and orders their producers) until the call is done there,
as for any work on another stream than a tensor's own.
"""
from __future__ import annotations

import ctypes
from typing import Tuple

from . import latent as _l

INDEXER_ROPE_DIM = 64
_HEADS, _DIM = 32, 128
_BF16, _FP32 = 0, 1

EXPORTED_INDEXER_PAGED = ("indexer_cache_store", "indexer_queries", "indexer_cache_load_paged", "indexer_logits_paged")


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the library's entry points."""
    i32, i64, vp, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
    turn = [vp, vp, i64, i32, i32]   # positions, cos_sin, its rows, interleaved, hadamard
    types = {
        "indexer_cache_store": [vp, i64, vp, vp, i32, f32] + turn + [vp, vp, i64, vp, vp, i64, i64],
        "indexer_queries": [vp, i64, i64, vp, i64, i32, f32] + turn + [vp, vp, vp, i64],
        "indexer_cache_load_paged": [vp, vp, i32, vp, i64, vp, vp, vp, vp, i32, i64, i64, i64],
        "indexer_logits_paged": [vp, vp, vp, i64, vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, i64, i64, i64],
    }
    for name, args in types.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


def _keys(keys, key_scale, at: int):
    """The cache arguments of a call, and the number of slots."""
    shape, strides = keys.shape, keys.stride()
    if not (len(shape) == 2 and shape[1] == _DIM and keys.dtype is _l._UINT8 and strides[1] == 1 and keys.get_device() == at):
        raise ValueError(f"keys must be a (slots, {_DIM}) uint8 (fp8 E4M3 codes) tensor with contiguous rows on device {at}")
    slots = shape[0]
    if not _l._is(key_scale, _l._FLOAT32, (slots,), at):
        raise ValueError("key_scale must be a contiguous (slots,) float32 tensor on keys' device")
    return (keys.data_ptr(), strides[0] if slots > 1 else _DIM, key_scale.data_ptr()), slots


def _turn(positions, cos_sin, interleaved, hadamard, tokens: int, at: int):
    """The arguments of the rotation and the mixing."""
    if cos_sin is None:
        if positions is not None:
            raise ValueError("positions and cos_sin go together")
        return None, None, 0, 0, int(bool(hadamard))
    if positions is None:
        raise ValueError("positions and cos_sin go together")
    _l._int32("positions", positions, (tokens,), at)
    if not (cos_sin.dim() == 2 and _l._is(cos_sin, _l._FLOAT32, (cos_sin.shape[0], INDEXER_ROPE_DIM), at)):
        raise ValueError(f"cos_sin must be a contiguous (positions, {INDEXER_ROPE_DIM}) float32 tensor")
    return positions.data_ptr(), cos_sin.data_ptr(), cos_sin.shape[0], int(bool(interleaved)), int(bool(hadamard))


def _float_type(name: str, t) -> int:
    if t.dtype is _l._BFLOAT16:
        return _BF16
    if t.dtype is _l._FLOAT32:
        return _FP32
    raise ValueError(f"{name} must be bfloat16 or float32")


def _table(page_table, at: int):
    if page_table.dim() != 2:
        raise ValueError("page_table must be (requests, pages)")
    _l._int32("page_table", page_table, page_table.shape, at)
    return page_table.shape


def indexer_cache_store(k, slot_map, keys, key_scale, norm_weight=None, norm_bias=None, eps: float = 1e-6,
                        positions=None, cos_sin=None, interleaved: bool = True, hadamard: bool = False,
                        stream=None) -> None:
    """Stores tokens' index keys in their paged cache: layer norm (with norm_weight
    and norm_bias), rotation of the first 64 values (with positions and cos_sin),
    mixing by Hadamard's matrix (with hadamard), 8-bit codes and a scale per
    token, in one pass.

    k (T, 128) bfloat16, rows that do not overlap; slot_map (T,) int32 (paged_append_plan's): tokens
    with a slot outside the cache are skipped, and no two may name one slot; keys (slots,
    128) uint8 codes and key_scale (slots,) float32; norm_weight, norm_bias
    (128,) bfloat16 or float32; positions (T,) int32; cos_sin (positions, 64)
    float32: cosines, then sines, of a position's 32 angles.
    """
    dev, at = _l._gpu(k, "k")
    shape, strides = k.shape, k.stride()
    if not (len(shape) == 2 and shape[1] == _DIM and k.dtype is _l._BFLOAT16 and strides[1] == 1):
        raise ValueError(f"k must be a (tokens, {_DIM}) bfloat16 tensor with contiguous rows")
    T = shape[0]
    _l._int32("slot_map", slot_map, (T,), at)
    cache, slots = _keys(keys, key_scale, at)
    if (norm_weight is None) != (norm_bias is None):
        raise ValueError("norm_weight and norm_bias go together")
    weight, bias, kind = None, None, _BF16
    if norm_weight is not None:
        kind = _float_type("norm_weight", norm_weight)
        for name, t in (("norm_weight", norm_weight), ("norm_bias", norm_bias)):
            if not _l._is(t, norm_weight.dtype, (_DIM,), at):
                raise ValueError(f"{name} must be a contiguous tensor of shape ({_DIM},) on k's device, of one type with the other")
        weight, bias = norm_weight.data_ptr(), norm_bias.data_ptr()
    turn = _turn(positions, cos_sin, interleaved, hadamard, T, at)
    _l._call("indexer_cache_store", dev, stream, lambda handle: (
        k.data_ptr(), strides[0] if T > 1 else _DIM, weight, bias, kind, float(eps), *turn, slot_map.data_ptr(), *cache,
        handle, T, slots))


def indexer_queries(q, weights, weight_scale: float = 1.0, positions=None, cos_sin=None, interleaved: bool = True,
                    hadamard: bool = False, out_q=None, out_weights=None, stream=None) -> Tuple[object, object]:
    """A step's queries and head weights in the form the scores take.

    q (T, 32, 128) bfloat16 with any token and head strides that leave heads apart; weights (T,
    32) bfloat16 or float32.  Rotation, mixing and codes as in
    indexer_cache_store.  Returns (T, 32, 128) uint8 codes and (T, 32) float32:
    weights * weight_scale * the scale of the head's codes.  Tokens with a position
    outside cos_sin are padding, and their rows are left as they are.
    """
    dev, at = _l._gpu(q, "q")
    shape, strides = q.shape, q.stride()
    if not (len(shape) == 3 and shape[1] == _HEADS and shape[2] == _DIM and q.dtype is _l._BFLOAT16
            and (strides[2] == 1 or q.numel() == 0)):
        raise ValueError(f"q must be a (tokens, {_HEADS}, {_DIM}) bfloat16 tensor whose last dimension is contiguous")
    T = shape[0]
    kind = _float_type("weights", weights)
    if not (weights.shape == (T, _HEADS) and (weights.stride(1) == 1 or T == 0) and weights.get_device() == at):
        raise ValueError(f"weights must be a (tokens, {_HEADS}) tensor with contiguous rows on q's device")
    turn = _turn(positions, cos_sin, interleaved, hadamard, T, at)
    if out_q is not None and not _l._is(out_q, _l._UINT8, (T, _HEADS, _DIM), at):
        raise ValueError(f"out_q must be a contiguous uint8 tensor of shape ({T}, {_HEADS}, {_DIM})")
    if out_weights is not None and not _l._is(out_weights, _l._FLOAT32, (T, _HEADS), at):
        raise ValueError(f"out_weights must be a contiguous float32 tensor of shape ({T}, {_HEADS})")
    got = []

    def args(handle):
        torch = _l.torch
        got.append(torch.empty((T, _HEADS, _DIM), dtype=_l._UINT8, device=dev) if out_q is None else out_q)
        got.append(torch.empty((T, _HEADS), dtype=_l._FLOAT32, device=dev) if out_weights is None else out_weights)
        return (q.data_ptr(), strides[0] if T > 1 else _HEADS * _DIM, strides[1] if T > 0 else _DIM, weights.data_ptr(),
                weights.stride(0) if T > 1 else _HEADS, kind, float(weight_scale), *turn, got[0].data_ptr(),
                got[1].data_ptr(), handle, T)

    _l._call("indexer_queries", dev, stream, args)
    return got[0], got[1]


def indexer_cache_load_paged(page_table, kv_starts, page_size: int, num_rows: int, keys, key_scale, out_keys=None,
                             out_scale=None, stream=None) -> Tuple[object, object]:
    """The cached keys of whole requests in a row, as indexer_topk takes them (kv and
    kv_scale): rows [kv_starts[b], kv_starts[b + 1]) are positions 0, 1, ... of
    request b.  page_table (B, P) int32, kv_starts (B + 1,) int32; num_rows is
    the length of the outputs, and rows past kv_starts[B] are left as they are."""
    dev, at = _l._gpu(page_table, "page_table")
    B, P = _table(page_table, at)
    _l._int32("kv_starts", kv_starts, (B + 1,), at)
    rows = int(num_rows)
    if rows < 0:
        raise ValueError("num_rows must be >= 0")
    cache, slots = _keys(keys, key_scale, at)
    if out_keys is not None and not _l._is(out_keys, _l._UINT8, (rows, _DIM), at):
        raise ValueError(f"out_keys must be a contiguous uint8 tensor of shape ({rows}, {_DIM})")
    if out_scale is not None and not _l._is(out_scale, _l._FLOAT32, (rows,), at):
        raise ValueError(f"out_scale must be a contiguous float32 tensor of shape ({rows},)")
    got = []

    def args(handle):
        torch = _l.torch
        got.append(torch.empty((rows, _DIM), dtype=_l._UINT8, device=dev) if out_keys is None else out_keys)
        got.append(torch.empty((rows,), dtype=_l._FLOAT32, device=dev) if out_scale is None else out_scale)
        return (page_table.data_ptr(), kv_starts.data_ptr(), int(page_size), *cache, got[0].data_ptr(),
                got[1].data_ptr(), handle, B, P, rows, slots)

    _l._call("indexer_cache_load_paged", dev, stream, args)
    return got[0], got[1]


def indexer_logits_paged(q, weights, keys, key_scale, page_table, seq_lens, q_starts, page_size: int, width=None,
                         out=None, lens=None, stream=None) -> Tuple[object, object]:
    """Scores of a step's new tokens against their requests' cached keys.

    q (T, 32, 128) uint8 codes and weights (T, 32) float32 (indexer_queries'); keys, key_scale: the cache;
    page_table (B, P) int32; seq_lens (B,) int32: cached positions, the new
    tokens' own included; q_starts (B + 1,) int32: request b's tokens are rows
    [q_starts[b], q_starts[b + 1]).  The i-th of n sees L = seq_lens[b] - n + i +
    1 positions (at most width and P * page_size).  Returns logits (T, width) float32, whose
    entries from L on are left as they are, and lens (T,) int32: L, and 0 for rows past
    q_starts[B].  Both go to topk_transform as scores and seq_lens, with each token's
    row of the page table.  width: out's, or else P * page_size.
    """
    dev, at = _l._gpu(q, "q")
    T = q.shape[0] if q.dim() == 3 else -1
    if T < 0 or not _l._is(q, _l._UINT8, (T, _HEADS, _DIM), at):
        raise ValueError(f"q must be a contiguous uint8 (fp8 E4M3 codes) tensor of shape (tokens, {_HEADS}, {_DIM})")
    if not _l._is(weights, _l._FLOAT32, (T, _HEADS), at):
        raise ValueError(f"weights must be a contiguous float32 tensor of shape (tokens, {_HEADS}) on q's device")
    cache, slots = _keys(keys, key_scale, at)
    B, P = _table(page_table, at)
    _l._int32("seq_lens", seq_lens, (B,), at)
    _l._int32("q_starts", q_starts, (B + 1,), at)
    if width is None:
        width = P * int(page_size) if out is None or out.dim() != 2 else out.shape[1]
    width = int(width)
    if width < 0:
        raise ValueError("width must be >= 0")
    if out is not None and not _l._is(out, _l._FLOAT32, (T, width), at):
        raise ValueError(f"out must be a contiguous float32 tensor of shape ({T}, {width})")
    if lens is not None:
        _l._int32("lens", lens, (T,), at)
    got = []

    def args(handle):
        torch = _l.torch
        got.append(torch.empty((T, width), dtype=_l._FLOAT32, device=dev) if out is None else out)
        got.append(torch.empty((T,), dtype=_l._INT32, device=dev) if lens is None else lens)
        return (q.data_ptr(), weights.data_ptr(), *cache, page_table.data_ptr(), seq_lens.data_ptr(), q_starts.data_ptr(),
                int(page_size), got[0].data_ptr(), got[1].data_ptr(), handle, T, B, P, width, slots)

    _l._call("indexer_logits_paged", dev, stream, args)
    return got[0], got[1]
