"""CPU oracle of the paged latent cache and of latent attention: the definitions
of include/latent_attention.h in float64 (numpy), one row at a time, and the
error bounds the GPU results are held to.

Shares no code with the library.  bf16 arrays come in as float64 values.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import numpy as np

LATENT = 512
ROPE = 64
HEAD = 128
U32 = 2.0 ** -24          # half a step of fp32, relative
U16 = 2.0 ** -8           # of bf16


def e4m3_value(codes: np.ndarray) -> np.ndarray:
    """Values of OCP E4M3 codes (bias 7, 0x7F / 0xFF are NaN)."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9.0)
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


# ---- plan -------------------------------------------------------------------------------------

class Plan(NamedTuple):
    page_table: np.ndarray
    seq_lens: np.ndarray
    q_starts: np.ndarray
    slot_map: np.ndarray
    positions: np.ndarray
    free_used: int


def append_plan(kv_lens, new_lens, page_table, free_pages, free_used, page_size, num_tokens) -> Plan:
    table = np.array(page_table, np.int64)
    pages_per_row = table.shape[1]
    slot_map = np.full(num_tokens, -1, np.int64)
    positions = np.full(num_tokens, -1, np.int64)
    starts, seq = [0], []
    used = int(free_used)
    for b, (kv, new) in enumerate(zip(kv_lens, new_lens)):
        kv, new = max(0, int(kv)), max(0, int(new))
        for col in range(-(-kv // page_size), -(-(kv + new) // page_size)):
            if col < pages_per_row:
                table[b, col] = free_pages[used] if 0 <= used < len(free_pages) else -1
                used += 1
        for i in range(new):
            t, pos = starts[-1] + i, kv + i
            if t >= num_tokens:
                break
            positions[t] = pos
            col = pos // page_size
            if col < pages_per_row and table[b, col] >= 0:
                slot = int(table[b, col]) * page_size + pos % page_size
                slot_map[t] = slot if slot < 2 ** 31 else -1
        seq.append(kv + new)
        starts.append(starts[-1] + new)
    return Plan(table, np.array(seq, np.int64), np.array(starts, np.int64), slot_map, positions, used)


# ---- store ------------------------------------------------------------------------------------

def normed(c: np.ndarray, weight: Optional[np.ndarray], eps: float) -> np.ndarray:
    if weight is None:
        return c
    return c / np.sqrt(np.mean(c * c) + eps) * weight


def rotated(r: np.ndarray, cos_sin: Optional[np.ndarray], interleaved: bool) -> np.ndarray:
    if cos_sin is None:
        return r
    out = r.copy()
    for i in range(ROPE // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + ROPE // 2)
        cs, sn = cos_sin[i], cos_sin[ROPE // 2 + i]
        out[a], out[b] = r[a] * cs - r[b] * sn, r[b] * cs + r[a] * sn
    return out


# The norm: a sum of 512 squares (each sum and product one rounding, halved by
# the root), the root, the division, two products.
NORM_ERROR = (LATENT / 2 + 8) * U32


# ---- attention --------------------------------------------------------------------------------

class Attended(NamedTuple):
    out: np.ndarray
    lse: float
    out_bound: np.ndarray
    lse_bound: float


def attend(q: np.ndarray, keys: np.ndarray, values: np.ndarray, scale: float) -> Attended:
    """One head's query against its keys (n, d) and values (n, e).

    The bounds count the roundings of an fp32 evaluation whose weights are
    rounded to bf16 and whose result is rounded to bf16:
      * a score: d products summed in fp32, its scaling, the subtraction of the
        reference and exp2 (2 units): dz, relative on the weight;
      * the sum of n weights, in any order and rescaled at most n times;
      * the weight's own rounding to bf16, the products and sums of the result,
        the division, and the result's rounding to bf16.
    """
    n, d = keys.shape
    if n == 0:
        return Attended(np.zeros(values.shape[1]), -np.inf, np.zeros(values.shape[1]), 0.0)
    z = scale * (keys @ q)
    top = z.max()
    p = np.exp(z - top)
    total = p.sum()
    p /= total
    lse = top + np.log(total)
    out = p @ values
    size = np.abs(p) @ np.abs(values)
    magnitude = abs(scale) * (np.abs(keys) @ np.abs(q))
    # weights of keys far below the top do not count: their error is taken
    # times their share
    dz = (d + 2) * U32 * magnitude + 4 * U32 * (np.abs(z) + abs(top) + 16.0) + 4 * U32
    weight = float(p @ dz)
    sums = 3 * n * U32 + 8 * U32
    worst = (p * dz) @ np.abs(values)
    out_bound = U16 * np.abs(out) + (1 + U16) * (worst + (weight + U16 + 2 * sums) * size)
    lse_bound = weight + sums + 4 * U32 * (1 + abs(lse) + abs(top))
    return Attended(out, float(lse), out_bound + 1e-30, float(lse_bound))


def causal_keys(i: int, nq: int, nk: int, causal: bool = True) -> int:
    """Keys the i-th of nq queries attends, of nk."""
    return max(0, min(nk, nk - nq + i + 1)) if causal else nk


def page_slots(row: np.ndarray, page_size: int, n: int, num_slots: int) -> np.ndarray:
    """Slots of positions [0, n) of a page table row that have a page."""
    pos = np.arange(min(n, len(row) * page_size))
    page = row.astype(np.int64)[pos // page_size]
    slot = page * page_size + pos % page_size
    return slot[(page >= 0) & (slot < num_slots)]


def check(name: str, got: np.ndarray, want: np.ndarray, bound) -> Optional[str]:
    """A message where got is further than bound from want (or not finite alike)."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    if not np.array_equal(np.isfinite(got), np.isfinite(want)):
        return f"{name}: not finite in the same places"
    fin = np.isfinite(want)
    if not np.array_equal(got[~fin], want[~fin]):
        return f"{name}: infinities differ"
    over = np.where(fin, np.abs(np.where(fin, got, 0) - np.where(fin, want, 0)) - bound, -1.0)
    if (over > 0).any():
        at = np.unravel_index(int(np.argmax(over)), over.shape)
        return f"{name}: {got[at]!r} for {want[at]!r} at {at}, {over[at]:.3g} over its bound"
    return None
