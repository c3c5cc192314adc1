"""Pins of the latent oracle on the CPU: against hand-made results and against
torch's own operations in float64, and the refusals of the entry points that
need no device."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import sparse_attention_indexer_fp32_amd as topk
from oracle import latent_oracle as lo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_e4m3_values_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(lo.e4m3_value(codes), want)


def test_plan_by_hand():
    """Three requests, pages of 4: 3 + 2 tokens take one page behind a kept one, 0 + 0
    none, 4 + 5 two."""
    table = np.array([[7, -5, -5], [-5, -5, -5], [9, -5, -5]])
    p = lo.append_plan([3, 0, 4], [2, 0, 5], table, [20, 21, 22, 23], 1, 4, 9)
    assert p.page_table.tolist() == [[7, 21, -5], [-5, -5, -5], [9, 22, 23]]
    assert p.seq_lens.tolist() == [5, 0, 9] and p.q_starts.tolist() == [0, 2, 2, 7]
    assert p.slot_map.tolist() == [31, 84, 88, 89, 90, 91, 92, -1, -1]
    assert p.positions.tolist() == [3, 4, 4, 5, 6, 7, 8, -1, -1]
    assert p.free_used == 4


def test_plan_runs_out_of_pages():
    p = lo.append_plan([0, 0], [3, 2], np.full((2, 2), -9), [5], 0, 2, 5)
    assert p.page_table.tolist() == [[5, -1], [-1, -9]]
    assert p.slot_map.tolist() == [10, 11, -1, -1, -1] and p.free_used == 3


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(1)
    r, angle = rng.standard_normal(64), rng.uniform(0, 6, 32)
    cs = np.concatenate([np.cos(angle), np.sin(angle)])
    z = (r[0::2] + 1j * r[1::2]) * np.exp(1j * angle)
    got = lo.rotated(r, cs, True)
    np.testing.assert_allclose(got[0::2] + 1j * got[1::2], z)
    z = (r[:32] + 1j * r[32:]) * np.exp(1j * angle)
    got = lo.rotated(r, cs, False)
    np.testing.assert_allclose(got[:32] + 1j * got[32:], z)


def test_attend_matches_torch():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal(192), rng.standard_normal((37, 192)), rng.standard_normal((37, 128))
    a = lo.attend(q, k, v, 0.11)
    z = torch.from_numpy(k @ q * 0.11)
    np.testing.assert_allclose(a.out, (torch.softmax(z, 0) @ torch.from_numpy(v)).numpy())
    np.testing.assert_allclose(a.lse, float(torch.logsumexp(z, 0)))
    empty = lo.attend(q, k[:0], v[:0], 0.11)
    assert empty.lse == -np.inf and not empty.out.any()


def test_bounds_tell_a_wrong_result():
    """The bounds are far below what a dropped key, a wrong key or a missing
    rescale would change, and an honest bf16 evaluation stays inside them."""
    rng = np.random.default_rng(3)
    bf = lambda a: torch.from_numpy(a).bfloat16()  # noqa: E731
    q, k, v = (bf(rng.standard_normal(s)) for s in ((192,), (300, 192), (300, 128)))
    a = lo.attend(q.double().numpy(), k.double().numpy(), v.double().numpy(), 0.07)
    z = (k.float() @ q.float()) * 0.07
    p = torch.exp(z - z.max())
    out = ((p.bfloat16().float() @ v.float()) / p.sum()).bfloat16()
    assert lo.check("out", out.double().numpy(), a.out, a.out_bound) is None
    assert lo.check("lse", float(z.max() + p.sum().log()), a.lse, a.lse_bound) is None
    heavy = int(z.argmax())
    keep = np.arange(300) != heavy
    fewer = lo.attend(q.double().numpy(), k.double().numpy()[keep], v.double().numpy()[keep], 0.07)
    assert lo.check("out", fewer.out, a.out, a.out_bound) is not None
    assert lo.check("lse", fewer.lse, a.lse, a.lse_bound) is not None


# ---- the binding and the C entry points, without a device -------------------------------------------

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(topk.LIB_PATH):
        pytest.fail("libtopk_transform.so is not built (run __graft_entry__.build())")
    return topk.load()


def test_exports_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "latent_attention.h")).read(), flags=re.S)
    names = set(re.findall(r"\b((?:latent|paged)_[a-z_]+)\s*\(", text))
    assert names == set(topk.EXPORTED_LATENT)
    for name in names:
        assert hasattr(lib, name), name


A = 4096   # a pointer that is never followed: the calls below fail their checks first


def _plan(lib, **kw):
    a = dict(kv=A, new=A, table=A, free=A, used=None, ps=16, seq=A + 256, qs=A, slots=A, pos=A, out=A, B=2, P=2, F=2, T=4)
    a.update(kw)
    return lib.paged_append_plan(a["kv"], a["new"], a["table"], a["free"], a["used"], a["ps"], a["seq"], a["qs"],
                                 a["slots"], a["pos"], a["out"], None, a["B"], a["P"], a["F"], a["T"])


@pytest.mark.parametrize("kw", [dict(ps=0), dict(ps=-4), dict(ps=24), dict(B=-1), dict(P=-1), dict(F=-1), dict(T=-1),
                                dict(T=2 ** 31), dict(kv=None), dict(new=None), dict(table=None), dict(free=None),
                                dict(seq=None), dict(qs=None), dict(slots=None), dict(pos=None), dict(out=None),
                                dict(used=A),                   # free_used_out aliases free_used
                                dict(seq=A), dict(new=A + 256)])   # seq_lens aliases kv_lens, new_lens
def test_plan_refusals(lib, kw):
    assert _plan(lib, **kw) == 1 and topk.topk_last_error()


CACHE = dict(lat=A, ls=512, rope=A, rs=64, scale=None, kind=0)
BAD_CACHE = [dict(kind=2), dict(kind=-1), dict(kind=1), dict(scale=A), dict(lat=None), dict(rope=None), dict(lat=A + 8),
             dict(rope=A + 2), dict(ls=500), dict(ls=516), dict(rs=63), dict(rs=68), dict(slots=-1),
             dict(slots=2 ** 31)]


def _store(lib, **kw):
    a = dict(CACHE, kv=A, kvs=576, w=None, pos=None, cs=None, maxpos=0, map=A, T=3, slots=8)
    a.update(kw)
    return lib.latent_cache_store(a["kv"], a["kvs"], a["w"], 1e-6, a["pos"], a["cs"], a["maxpos"], 1, a["map"],
                                  a["lat"], a["ls"], a["rope"], a["rs"], a["scale"], a["kind"], None, a["T"],
                                  a["slots"])


@pytest.mark.parametrize("kw", BAD_CACHE + [dict(kv=None), dict(kv=A + 8), dict(kvs=570), dict(kvs=580), dict(map=None),
                                            dict(T=-1), dict(w=A + 2), dict(cs=A), dict(cs=A, pos=A, maxpos=-1)])
def test_store_refusals(lib, kw):
    assert _store(lib, **kw) == 1 and topk.topk_last_error()


def _load(lib, **kw):
    a = dict(CACHE, map=A, out=A, outr=A, rows=3, slots=8)
    a.update(kw)
    return lib.latent_cache_load(a["map"], a["lat"], a["ls"], a["rope"], a["rs"], a["scale"], a["kind"], a["out"],
                                 a["outr"], None, a["rows"], a["slots"])


def _load_paged(lib, **kw):
    a = dict(CACHE, table=A, starts=A, ps=16, out=A, outr=A, B=2, P=3, rows=3, slots=8)
    a.update(kw)
    return lib.latent_cache_load_paged(a["table"], a["starts"], a["ps"], a["lat"], a["ls"], a["rope"], a["rs"],
                                       a["scale"], a["kind"], a["out"], a["outr"], None, a["B"], a["P"], a["rows"],
                                       a["slots"])


@pytest.mark.parametrize("kw", BAD_CACHE + [dict(map=None), dict(out=None), dict(outr=None), dict(out=A + 4),
                                            dict(rows=-1)])
def test_load_refusals(lib, kw):
    assert _load(lib, **kw) == 1 and topk.topk_last_error()


@pytest.mark.parametrize("kw", BAD_CACHE + [dict(table=None), dict(starts=None), dict(ps=3), dict(B=-1), dict(P=-1),
                                            dict(out=None), dict(outr=A + 8), dict(rows=-1)])
def test_load_paged_refusals(lib, kw):
    assert _load_paged(lib, **kw) == 1 and topk.topk_last_error()


def _attention(lib, **kw):
    a = dict(CACHE, q=A, qts=8 * 576, qhs=576, idx=A, out=A, lse=A, T=2, H=8, k=4, slots=8)
    a.update(kw)
    return lib.latent_attention(a["q"], a["qts"], a["qhs"], a["lat"], a["ls"], a["rope"], a["rs"], a["scale"],
                                a["kind"], a["idx"], 0.1, a["out"], a["lse"], None, 0, None, a["T"], a["H"], a["k"],
                                a["slots"])


def _paged(lib, **kw):
    a = dict(CACHE, q=A, qts=8 * 576, qhs=576, table=A, seq=A, starts=A, ps=16, out=A, lse=A, T=2, H=8, B=2, P=3,
             slots=8)
    a.update(kw)
    return lib.latent_attention_paged(a["q"], a["qts"], a["qhs"], a["lat"], a["ls"], a["rope"], a["rs"], a["scale"],
                                      a["kind"], a["table"], a["seq"], a["starts"], a["ps"], 0.1, a["out"], a["lse"],
                                      None, 0, None, a["T"], a["H"], a["B"], a["P"], a["slots"])


BAD_Q = [dict(q=None), dict(q=A + 8), dict(qts=-8), dict(qts=4), dict(qhs=570), dict(qhs=580), dict(out=None),
         dict(out=A + 8), dict(T=-1), dict(H=-1)]


@pytest.mark.parametrize("kw", BAD_CACHE + BAD_Q + [dict(idx=None), dict(k=-1), dict(k=2 ** 31)])
def test_attention_refusals(lib, kw):
    assert _attention(lib, **kw) == 1 and topk.topk_last_error()


@pytest.mark.parametrize("kw", BAD_CACHE + BAD_Q + [dict(table=None), dict(seq=None), dict(starts=None), dict(ps=0),
                                                    dict(ps=48), dict(B=-1), dict(P=-1)])
def test_paged_refusals(lib, kw):
    assert _paged(lib, **kw) == 1 and topk.topk_last_error()


def _expanded(lib, **kw):
    a = dict(q=A, qts=4 * 192, qhs=192, kv=A, kts=4 * 256, khs=256, rope=A, rs=64, qst=A, kst=A, out=A, lse=A, T=5, K=7,
             H=4, B=2, ws=None, wsb=0)
    a.update(kw)
    return lib.latent_attention_expanded(a["q"], a["qts"], a["qhs"], a["kv"], a["kts"], a["khs"], a["rope"], a["rs"],
                                         a["qst"], a["kst"], 0.1, 1, a["out"], a["lse"], a["ws"], a["wsb"], None, a["T"],
                                         a["K"], a["H"], a["B"])


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=A + 2), dict(qhs=180), dict(qhs=196), dict(qts=-8), dict(kv=None),
                                dict(kv=A + 8), dict(khs=250), dict(khs=260), dict(kts=4), dict(rope=None),
                                dict(rope=A + 8), dict(rs=60), dict(rs=68), dict(qst=None), dict(kst=None),
                                dict(out=None), dict(T=-1), dict(K=-1), dict(H=-1), dict(H=70000), dict(B=-1),
                                dict(kts=1 << 24), dict(rs=1 << 24)])
def test_expanded_refusals(lib, kw):
    assert _expanded(lib, **kw) == 1 and topk.topk_last_error()


def test_nothing_to_do_is_no_error(lib):
    assert _store(lib, T=0) == 0 and _load(lib, rows=0) == 0 and _load_paged(lib, rows=0) == 0
    assert _attention(lib, T=0) == 0 and _paged(lib, T=0) == 0 and _paged(lib, B=0) == 0
    assert _expanded(lib, T=0) == 0 and _expanded(lib, B=0) == 0
    n = ctypes.c_size_t(5)
    assert lib.latent_attention_workspace(0, 8, 100, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.latent_attention_workspace(-1, 8, 100, ctypes.byref(n)) == 1
    assert lib.latent_attention_workspace(1, 8, 100, None) == 1
    n.value = 5
    assert lib.latent_attention_expanded_workspace(0, 8, 100, 2, ctypes.byref(n)) == 0 and n.value == 0
    for bad in [(-1, 8, 100, 2), (3, -1, 100, 2), (3, 8, -1, 2), (3, 8, 100, -1)]:
        assert lib.latent_attention_expanded_workspace(*bad, ctypes.byref(n)) == 1
    assert lib.latent_attention_expanded_workspace(3, 8, 100, 2, None) == 1


def test_binding_refuses_before_any_call():
    bf, i32 = torch.bfloat16, torch.int32
    z = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        topk.latent_attention(z(1, 2, 576), z(4, 512), z(4, 64), z(1, 3, dtype=i32), 0.1)
    with pytest.raises(ValueError, match="GPU"):
        topk.paged_append_plan(z(2, dtype=i32), z(2, dtype=i32), z(2, 2, dtype=i32), z(3, dtype=i32), 16, 4)
    cpu = torch.device("cpu")
    from sparse_attention_indexer_fp32_amd import latent as binding
    for latent, rope, scale in ((z(4, 500), z(4, 64), None), (z(4, 512), z(3, 64), None),
                                (z(4, 512, dtype=torch.float16), z(4, 64), None), (z(4, 512), z(4, 64), z(4, dtype=torch.float32)),
                                (z(4, 512, dtype=torch.uint8), z(4, 64), None),
                                (z(4, 512, dtype=torch.uint8), z(4, 64), z(3, dtype=torch.float32)),
                                (z(4, 512, dtype=torch.uint8), z(4, 64), z(4)), (z(512, 4).T, z(4, 64), None)):
        with pytest.raises(ValueError):
            binding._cache(latent, rope, scale, cpu)
    with pytest.raises(ValueError):
        binding._queries(z(2, 4, 570), 576)
    with pytest.raises(ValueError):
        binding._queries(z(2, 4, 576, dtype=torch.float32), 576)
    with pytest.raises(ValueError):
        binding._outputs(z(2, 4, 511), None, 2, 4, 512, cpu)
    with pytest.raises(ValueError):
        binding._outputs(None, z(2, 4), 2, 4, 512, cpu)


# ---- the binding's checks, each by its one defect ------------------------------------------------------

ON_CPU = -1   # the device number of CPU tensors


def _zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.fixture(scope="module")
def binding():
    from sparse_attention_indexer_fp32_amd import latent
    latent._modules()
    return latent


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("slots", [0, 1, 4])
def test_binding_takes_a_cache(binding, e4m3, slots):
    """A cache as it should be, and as a view of a wider buffer, is taken with its strides."""
    latent = _zeros(slots, 512, dtype=torch.uint8 if e4m3 else torch.bfloat16)
    scale = _zeros(slots, dtype=torch.float32) if e4m3 else None
    rope = _zeros(slots, 64)
    args, n = binding._cache(latent, rope, scale, ON_CPU)
    assert n == slots and args[1] == 512 and args[3] == 64 and args[5] == int(e4m3)
    wide = _zeros(slots, 640, dtype=latent.dtype)
    args, n = binding._cache(wide[:, :512], _zeros(slots, 128)[:, 64:], scale, ON_CPU)
    assert n == slots and (args[1], args[3]) == ((640, 128) if slots > 1 else (512, 64))


@pytest.mark.parametrize("name,match", [
    ("narrow", "latent must be"), ("transposed", "latent must be"), ("flat", "latent must be"), ("elsewhere", "latent must be"),
    ("rope_rows", "rope must be"), ("rope_width", "rope must be"), ("rope_type", "rope must be"), ("rope_transposed", "rope must be"),
    ("latent_type", "latent must be bfloat16"), ("codes_without_scale", "latent must be bfloat16"), ("scale_of_bf16", "an 8-bit cache"),
    ("scale_rows", "an 8-bit cache"), ("scale_type", "an 8-bit cache"), ("scale_strided", "an 8-bit cache"),
])
def test_binding_refuses_a_cache(binding, name, match):
    codes, f32 = _zeros(4, 512, dtype=torch.uint8), torch.float32
    latent, rope, scale, at = {
        "narrow": (_zeros(4, 500), _zeros(4, 64), None, ON_CPU),
        "transposed": (_zeros(512, 4).T, _zeros(4, 64), None, ON_CPU),
        "flat": (_zeros(512), _zeros(4, 64), None, ON_CPU),
        "elsewhere": (_zeros(4, 512), _zeros(4, 64), None, 0),
        "rope_rows": (_zeros(4, 512), _zeros(3, 64), None, ON_CPU),
        "rope_width": (_zeros(4, 512), _zeros(4, 65), None, ON_CPU),
        "rope_type": (_zeros(4, 512), _zeros(4, 64, dtype=f32), None, ON_CPU),
        "rope_transposed": (_zeros(4, 512), _zeros(64, 4).T, None, ON_CPU),
        "latent_type": (_zeros(4, 512, dtype=torch.float16), _zeros(4, 64), None, ON_CPU),
        "codes_without_scale": (codes, _zeros(4, 64), None, ON_CPU),
        "scale_of_bf16": (_zeros(4, 512), _zeros(4, 64), _zeros(4, dtype=f32), ON_CPU),
        "scale_rows": (codes, _zeros(4, 64), _zeros(3, dtype=f32), ON_CPU),
        "scale_type": (codes, _zeros(4, 64), _zeros(4), ON_CPU),
        "scale_strided": (codes, _zeros(4, 64), _zeros(8, dtype=f32)[::2], ON_CPU),
    }[name]
    with pytest.raises(ValueError, match=match):
        binding._cache(latent, rope, scale, at)


def test_binding_checks_queries_and_outputs(binding):
    f32 = torch.float32
    assert binding._queries(_zeros(2, 5, 600)[:, 1:, :576], 576)[:2] == (2, 4)
    assert binding._queries(_zeros(2, 4, 576), 576)[2][1:] == (4 * 576, 576)
    for bad in (_zeros(2, 4, 570), _zeros(2, 576), _zeros(2, 4, 576, dtype=f32), _zeros(576, 4, 2).permute(2, 1, 0)):
        with pytest.raises(ValueError, match="q must be"):
            binding._queries(bad, 576)
    good = (_zeros(2, 4, 512), _zeros(2, 4, dtype=f32))
    binding._outputs(*good, 2, 4, 512, ON_CPU)
    binding._outputs(None, None, 2, 4, 512, ON_CPU)
    for bad in (_zeros(2, 4, 511), _zeros(2, 3, 512), _zeros(2, 4, 512, dtype=f32), _zeros(4, 2, 512).transpose(0, 1)):
        with pytest.raises(ValueError, match="out must be"):
            binding._outputs(bad, good[1], 2, 4, 512, ON_CPU)
    for bad in (_zeros(2, 4), _zeros(2, 5, dtype=f32), _zeros(4, 2, dtype=f32).T):
        with pytest.raises(ValueError, match="lse must be"):
            binding._outputs(good[0], bad, 2, 4, 512, ON_CPU)
    with pytest.raises(ValueError, match="out must be"):
        binding._outputs(*good, 2, 4, 512, 0)
    rows = (_zeros(3, 512), _zeros(3, 64))
    binding._load_outputs(*rows, 3, ON_CPU)
    for bad in ((_zeros(3, 500), rows[1]), (rows[0], _zeros(2, 64)), (rows[0].float(), rows[1])):
        with pytest.raises(ValueError, match="must be a contiguous bfloat16"):
            binding._load_outputs(*bad, 3, ON_CPU)
    binding._int32("x", _zeros(3, dtype=torch.int32), (3,), ON_CPU)
    for bad in (_zeros(3, dtype=torch.int64), _zeros(4, dtype=torch.int32), _zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="x must be a contiguous int32"):
            binding._int32("x", bad, (3,), ON_CPU)


def test_binding_refuses_a_stream_of_another_device(binding):
    """A kernel launched on another device's stream would read memory that is not there."""
    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    with pytest.raises(ValueError, match="stream"):
        with binding._on(torch.device("cuda", 0), Stream()):
            raise AssertionError("the call is on its way")


@pytest.mark.parametrize("call,kw", [
    (_load, dict(rows=2 ** 29)), (_load_paged, dict(rows=2 ** 31 - 1)),
    (_attention, dict(T=2 ** 26, H=16)), (_attention, dict(T=2 ** 26, H=1)), (_attention, dict(T=2 ** 24, H=32)),
    (_attention, dict(T=2 ** 24, H=33)), (_attention, dict(T=2 ** 20, H=1024)), (_attention, dict(T=2 ** 31 - 1, H=2 ** 31 - 1)),
    (_paged, dict(T=2 ** 26, H=7)), (_expanded, dict(T=2 ** 20, B=2 ** 20, H=16)), (_expanded, dict(T=2 ** 31 - 1, H=128)),
])
def test_launches_of_too_many_threads_are_refused(lib, call, kw):
    """2^32 threads and more would be cut off without an error."""
    assert call(lib, **kw) == 1 and "threads" in topk.topk_last_error()
