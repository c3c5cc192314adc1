"""Binding of the paged latent cache and of latent attention (include/latent_attention.h).

Argument marshalling only, as in the package's other calls: every step runs in
the library's HIP kernels, on `stream` (default: torch's current stream of the
tensors' device), and a call that cannot be made raises.  Outputs and
workspaces that the caller does not pass come from torch's allocator on that
stream, so captured graphs and concurrent streams share none.  With `stream`, the caller
keeps the inputs (and orders their producers) until the call is done there,
as for any work on another stream than a tensor's own.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import NamedTuple, Optional, Tuple

LATENT_DIM = 512
LATENT_ROPE_DIM = 64
LATENT_HEAD_DIM = 128
_QUERY = LATENT_DIM + LATENT_ROPE_DIM
_BF16, _E4M3 = 0, 1

EXPORTED_LATENT = ("paged_append_plan", "latent_cache_store", "latent_cache_load", "latent_cache_load_paged",
                   "latent_attention", "latent_attention_paged", "latent_attention_workspace",
                   "latent_attention_expanded", "latent_attention_expanded_workspace")


class AppendPlan(NamedTuple):
    """What paged_append_plan writes beside the page table."""
    seq_lens: object     # (requests,) int32: cached tokens after the step
    q_starts: object     # (requests + 1,) int32: each request's first token
    slot_map: object     # (num_tokens,) int32: each token's slot, -1 for none
    positions: object    # (num_tokens,) int32: each token's position, -1 past the last
    free_used: object    # (1,) int32: entries of free_pages taken so far


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the library's entry points."""
    i32, i64, vp, f32, size = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    cache = [vp, i64, vp, i64, vp, i32]   # latent, stride, rope, stride, scale, type
    types = {
        "paged_append_plan": [vp] * 5 + [i32] + [vp] * 5 + [vp, i32, i64, i64, i64],
        "latent_cache_store": [vp, i64, vp, f32, vp, vp, i64, i32, vp] + cache + [vp, i64, i64],
        "latent_cache_load": [vp] + cache + [vp, vp, vp, i64, i64],
        "latent_cache_load_paged": [vp, vp, i32] + cache + [vp, vp, vp, i32, i64, i64, i64],
        "latent_attention": [vp, i64, i64] + cache + [vp, f32, vp, vp, vp, size, vp, i32, i32, i64, i64],
        "latent_attention_paged": [vp, i64, i64] + cache + [vp, vp, vp, i32, f32, vp, vp, vp, size, vp, i32, i32, i32,
                                                            i64, i64],
        "latent_attention_workspace": [i32, i32, i64, ctypes.POINTER(size)],
        "latent_attention_expanded": [vp, i64, i64, vp, i64, i64, vp, i64, vp, vp, f32, i32, vp, vp, vp, size, vp, i32,
                                      i64, i32, i32],
        "latent_attention_expanded_workspace": [i32, i32, i64, i32, ctypes.POINTER(size)],
    }
    for name, args in types.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


package = torch = None   # this package and torch, once a call has needed them
_INT32 = _BFLOAT16 = _FLOAT32 = _UINT8 = _current_device = None


def _modules() -> None:
    """Binds the names above (they are not imported with this module: the
    package loads without torch, and imports this module)."""
    global package, torch, _INT32, _BFLOAT16, _FLOAT32, _UINT8, _current_device
    import torch as torch_module

    import sparse_attention_indexer_fp32_amd as this_package
    _INT32, _BFLOAT16 = torch_module.int32, torch_module.bfloat16
    _FLOAT32, _UINT8 = torch_module.float32, torch_module.uint8
    # without the check that CUDA is initialised: a tensor is on the device already
    _current_device = getattr(torch_module._C, "_cuda_getDevice", torch_module.cuda.current_device)
    torch, package = torch_module, this_package


@contextlib.contextmanager
def _on(dev, stream):
    """The tensors' device made current and, for allocations, the call's stream."""
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream must be one of {dev}, the tensors' device")
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _call(name: str, dev, stream, make_args):
    """Calls an entry point on its device; make_args(stream handle) gives its
    arguments and allocates what the caller did not pass."""
    fn = getattr(package.load(), name)
    if stream is None and dev.index == _current_device():
        st = fn(*make_args(package._stream_handle(None, dev)))
    else:
        with _on(dev, stream):
            st = fn(*make_args(package._stream_handle(stream, dev)))
    if st:
        package._check(st)


# The checks below run before every launch, and launches here take
# microseconds: they read each property of a tensor once (a tenth of a
# microsecond each), and compare device numbers rather than devices.

def _is(t, dtype, shape, at: int) -> bool:
    """Whether t is a contiguous tensor of this type and shape on device `at`."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == at


def _int32(name: str, t, shape, at: int) -> None:
    if not (t.dtype is _INT32 and t.shape == shape and t.is_contiguous() and t.get_device() == at):
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on device {at}")


def _gpu(t, name: str):
    """t's device, and its number."""
    if torch is None:
        _modules()
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    return t.device, t.get_device()


def _cache(latent, rope, scale, at: int):
    """The cache arguments of a call, and the number of slots."""
    shape, strides = latent.shape, latent.stride()
    if not (len(shape) == 2 and shape[1] == LATENT_DIM and strides[1] == 1 and latent.get_device() == at):
        raise ValueError(f"latent must be a (slots, {LATENT_DIM}) tensor with contiguous rows on device {at}")
    slots, rope_strides = shape[0], rope.stride()
    if not (rope.shape == (slots, LATENT_ROPE_DIM) and rope.dtype is _BFLOAT16 and rope_strides[1] == 1
            and rope.get_device() == at):
        raise ValueError(f"rope must be a (slots, {LATENT_ROPE_DIM}) bfloat16 tensor with contiguous rows on latent's device")
    if scale is None:
        if latent.dtype is not _BFLOAT16:
            raise ValueError("latent must be bfloat16, or uint8 (fp8 E4M3 codes) with scale")
        kind, sp = _BF16, None
    else:
        if not (latent.dtype is _UINT8 and _is(scale, _FLOAT32, (slots,), at)):
            raise ValueError("an 8-bit cache is latent uint8 (fp8 E4M3 codes) and scale, a contiguous (slots,) float32 tensor on its device")
        kind, sp = _E4M3, scale.data_ptr()
    # a single row has no stride to speak of
    ls, rs = (strides[0], rope_strides[0]) if slots > 1 else (LATENT_DIM, LATENT_ROPE_DIM)
    return (latent.data_ptr(), ls, rope.data_ptr(), rs, sp, kind), slots


def _queries(q, width: int):
    shape, strides = q.shape, q.stride()
    if not (len(shape) == 3 and shape[2] == width and q.dtype is _BFLOAT16 and (strides[2] == 1 or q.numel() == 0)):
        raise ValueError(f"q must be a (tokens, heads, {width}) bfloat16 tensor whose last dimension is contiguous")
    tokens, heads = shape[0], shape[1]
    return tokens, heads, (q.data_ptr(), strides[0] if tokens > 1 else heads * width, strides[1] if heads > 1 else width)


def _outputs(out, lse, tokens: int, heads: int, width: int, at: int):
    """Checks the outputs that are passed; those that are not are made by _made."""
    if out is not None and not _is(out, _BFLOAT16, (tokens, heads, width), at):
        raise ValueError(f"out must be a contiguous bfloat16 tensor of shape ({tokens}, {heads}, {width})")
    if lse is not None and not _is(lse, _FLOAT32, (tokens, heads), at):
        raise ValueError(f"lse must be a contiguous float32 tensor of shape ({tokens}, {heads})")


def _made(out, lse, tokens: int, heads: int, width: int, dev):
    if out is None:
        out = torch.empty((tokens, heads, width), dtype=_BFLOAT16, device=dev)
    if lse is None:
        lse = torch.empty((tokens, heads), dtype=_FLOAT32, device=dev)
    return out, lse


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(device_index: int, query: str, *sizes: int) -> int:
    n = ctypes.c_size_t(0)
    package._check(getattr(package.load(), query)(*sizes, ctypes.byref(n)))
    return n.value


def _workspace(dev, query: str, *sizes: int):
    """The workspace of a call as (tensor to hold on to, pointer, bytes)."""
    n = _workspace_bytes(dev.index, query, *sizes)
    if n == 0:
        return None, None, 0
    w = torch.empty(n, dtype=torch.uint8, device=dev)
    return w, w.data_ptr(), n


def paged_append_plan(kv_lens, new_lens, page_table, free_pages, page_size: int, num_tokens: int, free_used=None,
                      stream=None) -> AppendPlan:
    """Pages and slots of the tokens a step appends, from request lengths.

    kv_lens, new_lens (B,) int32: cached and new tokens of each request;
    page_table (B, P) int32, whose fresh entries are filled in place from
    free_pages (F,) int32, starting at free_used (1,) int32 (None: 0).
    num_tokens is the length of the token buffers; entries past the step's
    tokens are -1.  Returns AppendPlan; free_used above F says that pages ran
    out (their entries and slots are -1).
    """
    dev, at = _gpu(kv_lens, "kv_lens")
    B = kv_lens.numel()
    _int32("kv_lens", kv_lens, (B,), at)
    _int32("new_lens", new_lens, (B,), at)
    if not (page_table.dim() == 2 and page_table.shape[0] == B):
        raise ValueError("page_table must be (requests, pages)")
    _int32("page_table", page_table, page_table.shape, at)
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be 1-D")
    _int32("free_pages", free_pages, free_pages.shape, at)
    if free_used is not None:
        _int32("free_used", free_used, (1,), at)
    num_tokens = int(num_tokens)
    if num_tokens < 0:
        raise ValueError("num_tokens must be >= 0")
    plan = []

    def args(handle):
        # one allocation for all: these calls take microseconds
        whole = torch.empty(2 * B + 2 + 2 * num_tokens, dtype=_INT32, device=dev)
        plan.append(AppendPlan(*whole.split_with_sizes((B, B + 1, num_tokens, num_tokens, 1))))
        to = whole.data_ptr()
        return (kv_lens.data_ptr(), new_lens.data_ptr(), page_table.data_ptr(), free_pages.data_ptr(),
                free_used.data_ptr() if free_used is not None else None, int(page_size), to, to + 4 * B,
                to + 4 * (2 * B + 1), to + 4 * (2 * B + 1 + num_tokens), to + 4 * (2 * B + 1 + 2 * num_tokens), handle,
                B, page_table.shape[1], free_pages.shape[0], num_tokens)

    _call("paged_append_plan", dev, stream, args)
    return plan[0]


def latent_cache_store(kv, slot_map, latent, rope, scale=None, norm_weight=None, eps: float = 1e-6, positions=None,
                       cos_sin=None, interleaved: bool = True, stream=None) -> None:
    """Stores tokens in the cache: RMS norm of the latent (with norm_weight),
    rotation of the rotary key (with positions and cos_sin), 8-bit codes and a
    scale per token (with scale), in one pass.

    kv (T, 512 + 64) bfloat16, rows that do not overlap; slot_map (T,) int32: tokens
    with a slot outside the cache are skipped, and no two may name one slot;
    latent (slots, 512) bfloat16, or uint8 codes with scale (slots,) float32;
    rope (slots, 64) bfloat16; norm_weight (512,) bfloat16; positions (T,)
    int32; cos_sin (positions, 64) float32: cosines, then sines, of a
    position's 32 angles.
    """
    dev, at = _gpu(kv, "kv")
    shape, strides = kv.shape, kv.stride()
    if not (len(shape) == 2 and shape[1] == _QUERY and kv.dtype is _BFLOAT16 and strides[1] == 1):
        raise ValueError(f"kv must be a (tokens, {_QUERY}) bfloat16 tensor with contiguous rows")
    T = shape[0]
    _int32("slot_map", slot_map, (T,), at)
    cache, slots = _cache(latent, rope, scale, at)
    if norm_weight is not None:
        if not _is(norm_weight, _BFLOAT16, (LATENT_DIM,), at):
            raise ValueError(f"norm_weight must be a contiguous bfloat16 tensor of shape ({LATENT_DIM},)")
    if (positions is None) != (cos_sin is None):
        raise ValueError("positions and cos_sin go together")
    if cos_sin is not None:
        _int32("positions", positions, (T,), at)
        if not (cos_sin.dim() == 2 and _is(cos_sin, _FLOAT32, (cos_sin.shape[0], LATENT_ROPE_DIM), at)):
            raise ValueError(f"cos_sin must be a contiguous (positions, {LATENT_ROPE_DIM}) float32 tensor")
    rotate = cos_sin is not None
    _call("latent_cache_store", dev, stream, lambda handle: (
        kv.data_ptr(), strides[0] if T > 1 else _QUERY, norm_weight.data_ptr() if norm_weight is not None else None,
        float(eps), positions.data_ptr() if rotate else None, cos_sin.data_ptr() if rotate else None,
        cos_sin.shape[0] if rotate else 0, int(bool(interleaved)), slot_map.data_ptr(), *cache, handle, T, slots))


def _load_outputs(out_latent, out_rope, rows: int, at: int):
    for name, t, width in (("out_latent", out_latent, LATENT_DIM), ("out_rope", out_rope, LATENT_ROPE_DIM)):
        if not (t is None or _is(t, _BFLOAT16, (rows, width), at)):
            raise ValueError(f"{name} must be a contiguous bfloat16 tensor of shape ({rows}, {width})")


def _load_made(out_latent, out_rope, rows: int, dev):
    if out_latent is None:
        out_latent = torch.empty((rows, LATENT_DIM), dtype=_BFLOAT16, device=dev)
    if out_rope is None:
        out_rope = torch.empty((rows, LATENT_ROPE_DIM), dtype=_BFLOAT16, device=dev)
    return out_latent, out_rope


def latent_cache_load(slots, latent, rope, scale=None, out_latent=None, out_rope=None,
                      stream=None) -> Tuple[object, object]:
    """Rows of the cache by slot, as contiguous bfloat16: (rows, 512) and (rows,
    64).  slots (rows,) int32; a slot outside the cache gives zeros."""
    dev, at = _gpu(slots, "slots")
    if slots.dim() != 1:
        raise ValueError("slots must be 1-D")
    rows = slots.shape[0]
    _int32("slots", slots, (rows,), at)
    cache, n = _cache(latent, rope, scale, at)
    _load_outputs(out_latent, out_rope, rows, at)
    got = []

    def args(handle):
        got.extend(_load_made(out_latent, out_rope, rows, dev))
        return (slots.data_ptr(), *cache, got[0].data_ptr(), got[1].data_ptr(), handle, rows, n)

    _call("latent_cache_load", dev, stream, args)
    return got[0], got[1]


def latent_cache_load_paged(page_table, kv_starts, page_size: int, num_rows: int, latent, rope, scale=None,
                            out_latent=None, out_rope=None, stream=None) -> Tuple[object, object]:
    """The cached rows of whole requests, as contiguous bfloat16: rows
    [kv_starts[b], kv_starts[b + 1]) are positions 0, 1, ... of request b.
    page_table (B, P) int32, kv_starts (B + 1,) int32; num_rows is the length
    of the outputs, and rows past kv_starts[B] are left as they are."""
    dev, at = _gpu(page_table, "page_table")
    if page_table.dim() != 2:
        raise ValueError("page_table must be (requests, pages)")
    B = page_table.shape[0]
    _int32("page_table", page_table, page_table.shape, at)
    _int32("kv_starts", kv_starts, (B + 1,), at)
    rows = int(num_rows)
    if rows < 0:
        raise ValueError("num_rows must be >= 0")
    cache, n = _cache(latent, rope, scale, at)
    _load_outputs(out_latent, out_rope, rows, at)
    got = []

    def args(handle):
        got.extend(_load_made(out_latent, out_rope, rows, dev))
        return (page_table.data_ptr(), kv_starts.data_ptr(), int(page_size), *cache, got[0].data_ptr(),
                got[1].data_ptr(), handle, B, page_table.shape[1], rows, n)

    _call("latent_cache_load_paged", dev, stream, args)
    return got[0], got[1]


def latent_attention(q, latent, rope, indices, softmax_scale: float, scale=None, out=None, lse=None,
                     stream=None) -> Tuple[object, object]:
    """Latent attention, absorbed form, over selected slots.

    q (T, H, 512 + 64) bfloat16 with any token stride, heads that do not overlap; indices (T, k)
    int32 slots in any order (topk_transform's out; -1 selects nothing);
    latent, rope, scale: the cache.  Returns out (T, H, 512) bfloat16 and lse
    (T, H) float32, the natural logarithm of the softmax's sum.  A token that
    selects nothing gets zeros and -inf, a head with a score of NaN or +inf NaN in both.
    """
    dev, at = _gpu(q, "q")
    T, H, qargs = _queries(q, _QUERY)
    if indices.dim() != 2:
        raise ValueError("indices must be (tokens, k)")
    k = indices.shape[1]
    _int32("indices", indices, (T, k), at)
    cache, slots = _cache(latent, rope, scale, at)
    _outputs(out, lse, T, H, LATENT_DIM, at)
    got = []

    def args(handle):
        got.extend(_made(out, lse, T, H, LATENT_DIM, dev))
        got.extend(_workspace(dev, "latent_attention_workspace", T, H, k))
        return (*qargs, *cache, indices.data_ptr(), float(softmax_scale), got[0].data_ptr(), got[1].data_ptr(), got[3],
                got[4], handle, T, H, k, slots)

    _call("latent_attention", dev, stream, args)
    return got[0], got[1]


def latent_attention_paged(q, latent, rope, page_table, seq_lens, q_starts, page_size: int, softmax_scale: float,
                           scale=None, out=None, lse=None, stream=None) -> Tuple[object, object]:
    """Latent attention, absorbed form, over whole cached sequences.

    Request b's tokens are rows [q_starts[b], q_starts[b + 1]) of q; the i-th
    of n attends positions [0, seq_lens[b] - n + i + 1) of the request, found
    through page_table (B, P) int32.  Rows of q past q_starts[B] are padding
    and their outputs are left as they are.  Other arguments and the return
    value as in latent_attention.
    """
    dev, at = _gpu(q, "q")
    T, H, qargs = _queries(q, _QUERY)
    if page_table.dim() != 2:
        raise ValueError("page_table must be (requests, pages)")
    B, P = page_table.shape
    _int32("page_table", page_table, (B, P), at)
    _int32("seq_lens", seq_lens, (B,), at)
    _int32("q_starts", q_starts, (B + 1,), at)
    cache, slots = _cache(latent, rope, scale, at)
    _outputs(out, lse, T, H, LATENT_DIM, at)
    got = []

    def args(handle):
        got.extend(_made(out, lse, T, H, LATENT_DIM, dev))
        got.extend(_workspace(dev, "latent_attention_workspace", T, H, P * int(page_size)))
        return (*qargs, *cache, page_table.data_ptr(), seq_lens.data_ptr(), q_starts.data_ptr(), int(page_size),
                float(softmax_scale), got[0].data_ptr(), got[1].data_ptr(), got[3], got[4], handle, T, H, B, P, slots)

    _call("latent_attention_paged", dev, stream, args)
    return got[0], got[1]


def latent_attention_expanded(q, kv_up, rope, q_starts, kv_starts, softmax_scale: float, causal: bool = True, out=None,
                              lse=None, stream=None) -> Tuple[object, object]:
    """Latent attention, expanded form, over a ragged batch.

    q (Tq, H, 128 + 64) bfloat16; kv_up (Tk, H, 256) bfloat16: each head's key
    (128), then its value (128); rope (Tk, 64) bfloat16, the rotary keys all
    heads share; q_starts, kv_starts (B + 1,) int32: each request's rows.
    Causal: the i-th of nq queries attends keys [0, nk - nq + i + 1).  Returns
    out (Tq, H, 128) bfloat16 and lse (Tq, H) float32; a query with no key
    gets zeros and -inf, rows past q_starts[B] are left as they are.
    """
    dev, at = _gpu(q, "q")
    T, H, qargs = _queries(q, LATENT_HEAD_DIM + LATENT_ROPE_DIM)
    if not (kv_up.dim() == 3 and tuple(kv_up.shape[1:]) == (H, 2 * LATENT_HEAD_DIM) and kv_up.dtype == torch.bfloat16
          and (kv_up.stride(2) == 1 or kv_up.numel() == 0) and kv_up.device == dev):
        raise ValueError(f"kv_up must be a (keys, {H}, {2 * LATENT_HEAD_DIM}) bfloat16 tensor whose last dimension is contiguous")
    K = kv_up.shape[0]
    if not (tuple(rope.shape) == (K, LATENT_ROPE_DIM) and rope.dtype == torch.bfloat16 and rope.stride(1) == 1
          and rope.device == dev):
        raise ValueError(f"rope must be a ({K}, {LATENT_ROPE_DIM}) bfloat16 tensor with contiguous rows")
    if not (q_starts.dim() == 1 and q_starts.shape[0] >= 1):
        raise ValueError("q_starts must be (requests + 1,)")
    B = q_starts.shape[0] - 1
    _int32("q_starts", q_starts, (B + 1,), at)
    _int32("kv_starts", kv_starts, (B + 1,), at)
    _outputs(out, lse, T, H, LATENT_HEAD_DIM, at)
    got = []

    def args(handle):
        got.extend(_made(out, lse, T, H, LATENT_HEAD_DIM, dev))
        got.extend(_workspace(dev, "latent_attention_expanded_workspace", T, H, K, B))
        return (*qargs, kv_up.data_ptr(), kv_up.stride(0) if K > 1 else H * 2 * LATENT_HEAD_DIM,
                kv_up.stride(1) if H > 1 else 2 * LATENT_HEAD_DIM, rope.data_ptr(),
                rope.stride(0) if K > 1 else LATENT_ROPE_DIM, q_starts.data_ptr(), kv_starts.data_ptr(),
                float(softmax_scale), int(bool(causal)), got[0].data_ptr(), got[1].data_ptr(), *got[3:5],
                handle, T, K, H, B)

    _call("latent_attention_expanded", dev, stream, args)
    return got[0], got[1]
