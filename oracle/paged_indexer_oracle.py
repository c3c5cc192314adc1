"""CPU oracle of the indexer's 8-bit keys and queries: the definitions of
include/indexer_paged.h in float64 (numpy), one row at a time, and the error
bounds the GPU results are held to.  The scores' own are indexer_oracle's.

Shares no code with the library.  bf16 arrays come in as float64 values.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import numpy as np

DIM = 128
ROPE = 64
U32 = 2.0 ** -24          # half a step of fp32, relative
U8 = 2.0 ** -4            # of E4M3
TINY8 = 2.0 ** -10        # half a step of its subnormal numbers


class Row(NamedTuple):
    y: np.ndarray         # the row before its codes
    slack: np.ndarray     # how far an fp32 evaluation may be from it


def normed(x: np.ndarray, weight: Optional[np.ndarray], bias: Optional[np.ndarray], eps: float) -> Row:
    """The layer norm.  Roundings: the mean is a sum of 128 values (one each) and a
    product; a deviation is one subtraction; the mean of squares has 128 sums and
    products, the root and the division halve and add few; two products and a sum
    follow.  The mean's own error moves every deviation by as much, and the spread
    by less than its share of it."""
    if weight is None:
        return Row(x, np.zeros(DIM))
    mean = x.mean()
    d = x - mean
    inv = 1.0 / np.sqrt(np.mean(d * d) + eps)
    moved = 130 * U32 * np.mean(np.abs(x))
    y = d * inv * weight + bias
    rel = (DIM / 2 + 10) * U32 + moved * inv
    slack = np.abs(weight) * inv * (np.abs(d) * rel + moved) + 4 * U32 * (np.abs(d * inv * weight) + np.abs(bias))
    return Row(y, slack)


def rotated(r: Row, cos_sin: Optional[np.ndarray], interleaved: bool) -> Row:
    if cos_sin is None:
        return r
    y, slack = r.y.copy(), r.slack.copy()
    for i in range(ROPE // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + ROPE // 2)
        cs, sn = float(cos_sin[i]), float(cos_sin[ROPE // 2 + i])
        y[a], y[b] = r.y[a] * cs - r.y[b] * sn, r.y[b] * cs + r.y[a] * sn
        slack[a] = abs(cs) * r.slack[a] + abs(sn) * r.slack[b] + 3 * U32 * (abs(cs * r.y[a]) + abs(sn * r.y[b]))
        slack[b] = abs(cs) * r.slack[b] + abs(sn) * r.slack[a] + 3 * U32 * (abs(cs * r.y[b]) + abs(sn * r.y[a]))
    return Row(y, slack)


def hadamard() -> np.ndarray:
    """Entry (i, j) is -1 to the number of ones that i and j have in common."""
    return np.array([[(-1.0) ** bin(i & j).count("1") for j in range(DIM)] for i in range(DIM)])


_H = hadamard()


def mixed(r: Row, on: bool) -> Row:
    """Seven rounds of sums, then a product by a rounded constant."""
    if not on:
        return r
    root = np.sqrt(DIM)
    return Row(_H @ r.y / root, (r.slack.sum() + 10 * U32 * (np.abs(r.y).sum())) / root * np.ones(DIM))


def row(x, weight=None, bias=None, eps=0.0, cos_sin=None, interleaved=True, mix=False) -> Row:
    return mixed(rotated(normed(x, weight, bias, eps), cos_sin, interleaved), mix)


def scale_of(r: Row) -> Tuple[float, float]:
    """The row's scale, and how far it may be off."""
    top = np.abs(r.y).max()
    if top == 0 and r.slack.max() == 0:
        return 1.0, 0.0
    return top / 448.0, (r.slack.max() + 4 * U32 * top) / 448.0


def value_bound(r: Row, scale: float) -> np.ndarray:
    """Code * scale against y: half a step of the code on what was rounded, and the
    roundings of the quotient and of the product."""
    return U8 * (np.abs(r.y) + r.slack) + TINY8 * scale + r.slack + 8 * U32 * np.abs(r.y) + 1e-30
