"""CPU tests of the C entry point of latent attention behind shared prefixes: its
refusals, which come before a device is touched."""
import ctypes
import os

import pytest

import sparse_attention_indexer_fp32_amd as topk


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(topk.LIB_PATH):
        pytest.fail("libtopk_transform.so is not built (run __graft_entry__.build())")
    return topk.load()


A = 4096   # a pointer that is never followed: the calls below fail their checks first


def _shared(lib, **kw):
    a = dict(q=A, qts=4 * 576, qhs=576, lat=A, ls=512, rope=A, rs=64, scale=None, kind=0, table=A, seq=A, qs=A, gs=A, sl=A, ps=16,
             out=A, lse=A, ws=A, wsb=1 << 40, T=3, H=4, B=2, G=1, P=4, slots=8)
    a.update(kw)
    return lib.latent_attention_shared(a["q"], a["qts"], a["qhs"], a["lat"], a["ls"], a["rope"], a["rs"], a["scale"], a["kind"],
                                       a["table"], a["seq"], a["qs"], a["gs"], a["sl"], a["ps"], 0.1, a["out"], a["lse"], a["ws"],
                                       a["wsb"], None, a["T"], a["H"], a["B"], a["G"], a["P"], a["slots"])


@pytest.mark.parametrize("kw", [
    dict(kind=2), dict(kind=1), dict(scale=A), dict(lat=None), dict(rope=None), dict(lat=A + 8), dict(ls=500), dict(rs=63),
    dict(slots=-1), dict(q=None), dict(q=A + 2), dict(qts=-8), dict(qhs=575), dict(out=None), dict(out=A + 4), dict(ps=0),
    dict(ps=12), dict(T=-1), dict(H=-1), dict(B=-1), dict(G=-1), dict(P=-1), dict(P=2 ** 31), dict(table=None), dict(seq=None),
    dict(qs=None), dict(gs=None), dict(sl=None), dict(H=2 ** 24 + 1), dict(B=2 ** 31 - 1, G=2),
    dict(T=1, H=2 ** 24, P=2 ** 20, ps=64)])
def test_refusals(lib, kw):
    assert _shared(lib, **kw) == 1 and topk.topk_last_error()


def test_nothing_to_do_is_no_error(lib):
    assert _shared(lib, T=0) == 0 and _shared(lib, H=0) == 0 and _shared(lib, B=0) == 0


def test_workspace_refusals(lib):
    n = ctypes.c_size_t(7)
    assert lib.latent_attention_shared_workspace(-1, 4, ctypes.byref(n)) == 1
    assert lib.latent_attention_shared_workspace(4, -1, ctypes.byref(n)) == 1
    assert lib.latent_attention_shared_workspace(4, 4, None) == 1
    assert lib.latent_attention_shared_workspace(0, 4, ctypes.byref(n)) == 0 and n.value == 0
