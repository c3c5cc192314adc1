"""CPU tests of the indexer's paged cache: the oracle's own pins, and the refusals of
the C entry points, which fail before a device is touched."""
import os
import re

import numpy as np
import pytest

import sparse_attention_indexer_fp32_amd as topk
from oracle import paged_indexer_oracle as po

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ---- pins of the oracle -----------------------------------------------------------------------

def test_hadamard_is_the_doubled_square():
    h = np.ones((1, 1))
    while len(h) < 128:
        h = np.block([[h, h], [h, -h]])
    np.testing.assert_array_equal(po.hadamard(), h)
    np.testing.assert_array_equal(h @ h.T, 128 * np.eye(128))


def test_norm_closed_forms():
    x = np.arange(128.0)
    one, zero = np.ones(128), np.zeros(128)
    y = po.normed(x, one, zero, 0.0).y
    assert abs(y.mean()) < 1e-12 and abs((y * y).mean() - 1) < 1e-12
    np.testing.assert_allclose(y, (x - 63.5) / np.sqrt((128 ** 2 - 1) / 12))
    np.testing.assert_array_equal(po.normed(one, 3 * one, x, 1e-6).y, x)      # a constant row: the bias
    assert po.normed(x, None, None, 0.0).y is x


def test_rotation_closed_forms():
    x = np.zeros(128)
    x[0], x[100] = 2.0, 5.0
    cs = np.concatenate([np.zeros(32), np.ones(32)])      # a quarter turn
    pairs, halves = po.rotated(po.Row(x, 0 * x), cs, True).y, po.rotated(po.Row(x, 0 * x), cs, False).y
    assert pairs[1] == 2.0 and halves[32] == 2.0 and pairs[100] == halves[100] == 5.0
    assert abs(pairs).sum() == abs(halves).sum() == 7.0


def test_bounds_notice_a_wrong_row():
    """A wrong bias, angle, sign or scale is far outside the bounds."""
    rng = np.random.default_rng(0)
    x, w, b = rng.standard_normal(128), 1 + 0.1 * rng.standard_normal(128), 0.1 * rng.standard_normal(128)
    cs = np.concatenate([np.cos(np.arange(32.0)), np.sin(np.arange(32.0))])
    good = po.row(x, w, b, 1e-6, cs, True, True)
    scale, off = po.scale_of(good)
    bound = po.value_bound(good, scale)
    for bad in (po.row(x, w, 0 * b, 1e-6, cs, True, True), po.row(x, w, b, 1e-6, cs, False, True),
                po.row(x, w, b, 1e-6, np.roll(cs, 32), True, True), po.row(x, w, b, 1e-6, cs, True, False)):
        assert (np.abs(bad.y - good.y) > bound).any()
    assert abs(scale * 1.001 - scale) > off


# ---- the C entry points -----------------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(topk.LIB_PATH):
        pytest.fail("libtopk_transform.so is not built (run __graft_entry__.build())")
    return topk.load()


def test_exports_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "indexer_paged.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(indexer_[a-z_]+)\s*\(", text))
    assert names == set(topk.EXPORTED_INDEXER_PAGED)
    for name in names:
        assert hasattr(lib, name), name


A = 4096   # a pointer that is never followed: the calls below fail their checks first
BAD_KEYS = [dict(keys=None), dict(keys=A + 8), dict(ks=127), dict(ks=136), dict(ks=2 ** 31 + 16), dict(scale=None),
            dict(slots=-1), dict(slots=2 ** 31)]
BAD_TURN = [dict(cs=A), dict(cs=A + 4, pos=A), dict(cs=A, pos=A, maxpos=-1)]
BAD_PAGES = [dict(ps=0), dict(ps=-16), dict(ps=24), dict(B=-1), dict(P=-1), dict(P=2 ** 31), dict(table=None)]


def _store(lib, **kw):
    a = dict(k=A, kst=128, w=None, b=None, kind=0, pos=None, cs=None, maxpos=0, map=A, keys=A, ks=128, scale=A, T=3, slots=8)
    a.update(kw)
    return lib.indexer_cache_store(a["k"], a["kst"], a["w"], a["b"], a["kind"], 1e-6, a["pos"], a["cs"], a["maxpos"], 1, 0,
                                   a["map"], a["keys"], a["ks"], a["scale"], None, a["T"], a["slots"])


@pytest.mark.parametrize("kw", BAD_KEYS + BAD_TURN + [
    dict(T=-1), dict(T=2 ** 31), dict(k=None), dict(k=A + 2), dict(kst=120), dict(kst=132), dict(map=None), dict(w=A),
    dict(b=A), dict(w=A + 8, b=A), dict(w=A, b=A + 8), dict(kind=2), dict(kind=-1)])
def test_store_refusals(lib, kw):
    assert _store(lib, **kw) == 1 and topk.topk_last_error()


def _queries(lib, **kw):
    a = dict(q=A, ts=4096, hs=128, w=A, ws=32, kind=1, pos=None, cs=None, maxpos=0, out=A, outw=A, T=3)
    a.update(kw)
    return lib.indexer_queries(a["q"], a["ts"], a["hs"], a["w"], a["ws"], a["kind"], 1.0, a["pos"], a["cs"], a["maxpos"], 1,
                               0, a["out"], a["outw"], None, a["T"])


@pytest.mark.parametrize("kw", BAD_TURN + [
    dict(T=-1), dict(T=2 ** 26 + 1), dict(q=None), dict(q=A + 2), dict(ts=-8), dict(ts=4100), dict(hs=120), dict(hs=130),
    dict(w=None), dict(ws=-1), dict(kind=2), dict(out=None), dict(out=A + 4), dict(outw=None)])
def test_queries_refusals(lib, kw):
    assert _queries(lib, **kw) == 1 and topk.topk_last_error()


def _load(lib, **kw):
    a = dict(table=A, starts=A, ps=16, keys=A, ks=128, scale=A, out=A, outs=A, B=2, P=4, rows=5, slots=8)
    a.update(kw)
    return lib.indexer_cache_load_paged(a["table"], a["starts"], a["ps"], a["keys"], a["ks"], a["scale"], a["out"], a["outs"],
                                        None, a["B"], a["P"], a["rows"], a["slots"])


@pytest.mark.parametrize("kw", BAD_KEYS + BAD_PAGES + [
    dict(rows=-1), dict(rows=2 ** 31), dict(starts=None), dict(out=None), dict(outs=None), dict(out=A + 4)])
def test_load_refusals(lib, kw):
    assert _load(lib, **kw) == 1 and topk.topk_last_error()


def _logits(lib, **kw):
    a = dict(q=A, w=A, keys=A, ks=128, scale=A, table=A, seq=A, qs=A, ps=16, out=A, lens=A, T=2, B=2, P=4, width=64, slots=8)
    a.update(kw)
    return lib.indexer_logits_paged(a["q"], a["w"], a["keys"], a["ks"], a["scale"], a["table"], a["seq"], a["qs"], a["ps"],
                                    a["out"], a["lens"], None, a["T"], a["B"], a["P"], a["width"], a["slots"])


@pytest.mark.parametrize("kw", BAD_KEYS + BAD_PAGES + [
    dict(q=None), dict(q=A + 4), dict(w=None), dict(w=A + 4), dict(seq=None), dict(qs=None), dict(out=None), dict(T=-1),
    dict(width=-1), dict(width=2 ** 29, T=1), dict(width=2 ** 31), dict(T=2 ** 20, width=2 ** 20)])
def test_logits_refusals(lib, kw):
    assert _logits(lib, **kw) == 1 and topk.topk_last_error()


def test_nothing_to_do(lib):
    """Calls of no tokens or rows succeed without a device."""
    assert _store(lib, T=0, k=None, map=None) == 0
    assert _queries(lib, T=0, q=None, w=None, out=None, outw=None) == 0
    assert _load(lib, rows=0, out=None, outs=None) == 0 and _load(lib, B=0, table=None) == 0
    assert _logits(lib, T=0, q=None, w=None) == 0


def test_binding_refuses_host_tensors():
    import torch
    with pytest.raises(ValueError):
        topk.indexer_cache_store(torch.zeros((1, 128), dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32),
                                 torch.zeros((4, 128), dtype=torch.uint8), torch.zeros(4))
    with pytest.raises(ValueError):
        topk.indexer_logits_paged(torch.zeros((1, 32, 128), dtype=torch.uint8), torch.zeros((1, 32)),
                                  torch.zeros((4, 128), dtype=torch.uint8), torch.zeros(4),
                                  torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                                  torch.zeros(2, dtype=torch.int32), 4)
