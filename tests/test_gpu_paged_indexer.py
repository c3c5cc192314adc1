"""GPU tests of the indexer's paged key cache (store, queries, load, scores) against
the float64 oracles, through the binding.  The bounds are the oracles': roundings
counted from the formulas, none fitted."""
import numpy as np
import pytest

from gpu_util import note
from oracle import indexer_oracle as ix
from oracle import paged_indexer_oracle as po
from oracle.latent_oracle import check, e4m3_value

pytestmark = pytest.mark.gpu

GUARD = 77   # what outputs hold before a call that must leave them


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def _i32(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to(dev)


def _bf(rng, shape, dev, sigma=1.0, shift=0.0):
    """bf16 normals on the device, and their values in float64 on the host."""
    import torch
    t = (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) * sigma + shift).bfloat16()
    return t.to(dev), t.double().numpy()


def _finite_codes(rng, shape):
    codes = rng.integers(0, 256, shape, dtype=np.uint8)
    codes[(codes & 0x7F) == 0x7F] ^= 0x10
    return codes


def _angles(n):
    """Cosines and sines of n positions, in fp32."""
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def _check_row(name, x, codes, scale, **kw):
    r = po.row(x, **kw)
    want, off = po.scale_of(r)
    assert abs(float(scale) - want) <= off, (name, float(scale), want, off)
    err = check(name, e4m3_value(codes) * float(scale), r.y, po.value_bound(r, float(scale)))
    assert err is None, err


# ---- store ------------------------------------------------------------------------------------

@pytest.mark.parametrize("norm", [None, "bf16", "fp32"])
@pytest.mark.parametrize("rotate", [None, "pairs", "halves"])
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("tokens", [1, 7, 130])
def test_store(lib, dev, norm, rotate, mix, tokens):
    import torch
    rng = np.random.default_rng(tokens)
    slots_n, positions_n = 200, 50
    wide, wideh = _bf(rng, (tokens, 144), dev, sigma=2.0, shift=0.7)
    k, kh = wide[:, 8:136], wideh[:, 8:136].copy()        # rows of a larger buffer
    if tokens > 5:
        k[5], kh[5] = 0.0, 0.0                            # all zero (the norm's bias is left)
    kind = torch.float32 if norm == "fp32" else torch.bfloat16
    w = (1 + 0.2 * torch.randn(128, generator=torch.Generator().manual_seed(1))).to(kind)
    bias = (0.2 * torch.randn(128, generator=torch.Generator().manual_seed(2))).to(kind)
    buf = torch.from_numpy(_finite_codes(rng, (slots_n, 160))).to(dev)
    keys = buf[:, :128] if tokens == 7 else buf[:, :128].contiguous()     # a row stride of its own
    scale = torch.from_numpy(rng.uniform(0.5, 1, slots_n).astype(np.float32)).to(dev)
    slot_map, pos = rng.permutation(slots_n)[:tokens], rng.integers(0, positions_n, tokens)
    if tokens > 20:
        slot_map[3], slot_map[9] = -1, slots_n            # not stored
        pos[10], pos[11] = -1, positions_n                # nor these, when rotated
    before = keys.clone(), scale.clone()
    cs = _angles(positions_n)
    note(f"index store norm={norm} rotate={rotate} mix={mix} tokens={tokens}")
    lib.indexer_cache_store(k, _i32(slot_map, dev), keys, scale, norm_weight=w.to(dev) if norm else None,
                            norm_bias=bias.to(dev) if norm else None, eps=1e-5, interleaved=rotate == "pairs", hadamard=mix,
                            positions=_i32(pos, dev) if rotate else None,
                            cos_sin=torch.from_numpy(cs).to(dev) if rotate else None)
    torch.cuda.synchronize()
    got, gots = keys.cpu().numpy(), scale.cpu().numpy()
    stored = [t for t in range(tokens) if 0 <= slot_map[t] < slots_n and not (rotate and not 0 <= pos[t] < positions_n)]
    for t in stored:
        _check_row(f"token {t}", kh[t], got[slot_map[t]], gots[slot_map[t]], weight=w.double().numpy() if norm else None,
                   bias=bias.double().numpy() if norm else None, eps=1e-5, cos_sin=cs[pos[t]] if rotate else None,
                   interleaved=rotate == "pairs", mix=mix)
    left = np.setdiff1d(np.arange(slots_n), slot_map[stored])
    assert torch.equal(before[0].cpu()[left], keys.cpu()[left]) and torch.equal(before[1].cpu()[left], scale.cpu()[left])


def test_store_not_finite_and_tiny(lib, dev):
    """A NaN or an infinity makes its row's scale NaN, and leaves the other rows
    alone; rows far below 1 and far above keep their digits."""
    import torch
    rng = np.random.default_rng(5)
    k, kh = _bf(rng, (5, 128), dev)
    k[0, 100], k[2, 127] = float("inf"), float("nan")
    k[3], k[4] = k[3] * 1e-30, k[4] * 1e30
    kh[3], kh[4] = k[3].double().cpu().numpy(), k[4].double().cpu().numpy()
    keys, scale = torch.zeros((8, 128), dtype=torch.uint8, device=dev), torch.zeros(8, device=dev)
    lib.indexer_cache_store(k, _i32([4, 5, 6, 1, 2], dev), keys, scale)
    s = scale.cpu().numpy()
    assert np.isnan(s[[4, 6]]).all() and np.isfinite(s[[0, 1, 2, 3, 5, 7]]).all()
    for t, at in ((1, 5), (3, 1), (4, 2)):
        _check_row(f"token {t}", kh[t], keys.cpu().numpy()[at], s[at])


# ---- queries ----------------------------------------------------------------------------------

@pytest.mark.parametrize("rotate", [None, "pairs", "halves"])
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("tokens,fp32", [(1, True), (3, False), (37, True)])
def test_queries(lib, dev, rotate, mix, tokens, fp32):
    import torch
    rng = np.random.default_rng(tokens)
    q, qh = _bf(rng, (tokens, 33, 136), dev)
    q, qh = q[:, 1:, :128], qh[:, 1:, :128]               # strides of a larger buffer
    w = torch.from_numpy(rng.standard_normal((tokens, 40)).astype(np.float32))
    w = (w if fp32 else w.bfloat16()).to(dev)[:, 8:]
    pos = rng.integers(0, 50, tokens)
    if tokens > 10:
        pos[4], pos[7] = -1, 50                           # padding, when rotated
    out = torch.full((tokens, 32, 128), GUARD, dtype=torch.uint8, device=dev)
    outw = torch.full((tokens, 32), float(GUARD), device=dev)
    cs = _angles(50)
    note(f"queries rotate={rotate} mix={mix} tokens={tokens}")
    got, gotw = lib.indexer_queries(q, w, 0.25, positions=_i32(pos, dev) if rotate else None,
                                    cos_sin=torch.from_numpy(cs).to(dev) if rotate else None,
                                    interleaved=rotate == "pairs", hadamard=mix, out_q=out, out_weights=outw)
    assert got is out and gotw is outw
    codes, weights, wh = out.cpu().numpy(), outw.double().cpu().numpy(), w.double().cpu().numpy()
    for t in range(tokens):
        if rotate and not 0 <= pos[t] < 50:
            assert (codes[t] == GUARD).all() and (weights[t] == GUARD).all()
            continue
        for h in range(32):
            r = po.row(qh[t, h], cos_sin=cs[pos[t]] if rotate else None, interleaved=rotate == "pairs", mix=mix)
            s, off = po.scale_of(r)
            # two more products
            assert abs(weights[t, h] - 0.25 * wh[t, h] * s) <= 0.25 * abs(wh[t, h]) * (off + 3 * po.U32 * s), (t, h)
            err = check(f"{t} {h}", e4m3_value(codes[t, h]) * s, r.y, po.value_bound(r, s) + 448 * off)
            assert err is None, err


def test_queries_keep_products(lib, dev):
    """Rotation and mixing of query and key alike: the products of the values that
    the codes stand for are those of the rotated rows, to the codes' roundings."""
    import torch
    rng = np.random.default_rng(9)
    q, qh = _bf(rng, (4, 32, 128), dev)
    k, kh = _bf(rng, (4, 128), dev)
    cs = _angles(64)
    pos = [3, 60, 17, 0]
    keys, scale = torch.zeros((4, 128), dtype=torch.uint8, device=dev), torch.zeros(4, device=dev)
    kw = dict(positions=_i32(pos, dev), cos_sin=torch.from_numpy(cs).to(dev), hadamard=True)
    lib.indexer_cache_store(k, _i32(range(4), dev), keys, scale, **kw)
    codes, w = lib.indexer_queries(q, torch.ones((4, 32), device=dev), **kw)
    kv = e4m3_value(keys.cpu().numpy()) * scale.double().cpu().numpy()[:, None]
    qv = e4m3_value(codes.cpu().numpy()) * w.double().cpu().numpy()[..., None]
    for t in range(4):
        kr = po.row(kh[t], cos_sin=cs[pos[t]]).y
        for h in range(32):
            qr = po.row(qh[t, h], cos_sin=cs[pos[t]]).y
            # each code is off by 2^-4 of its value at most, or by a subnormal half step of its row's scale
            dq = 2.0 ** -4 * np.abs(_mixed(qr)) + 2.0 ** -10 * w[t, h].item()
            dk = 2.0 ** -4 * np.abs(_mixed(kr)) + 2.0 ** -10 * scale[t].item()
            bound = dq @ np.abs(_mixed(kr)) + dk @ np.abs(_mixed(qr)) + dq @ dk
            assert abs(qv[t, h] @ kv[t] - qr @ kr) <= bound * 1.0001


def _mixed(y):
    return po.hadamard() @ y / np.sqrt(128)


# ---- load -------------------------------------------------------------------------------------

@pytest.mark.parametrize("ps", [1, 16, 64])
@pytest.mark.parametrize("lens", [[5], [0, 0, 17, 0, 1, 64, 0], [1] * 200, [300, 2, 129], [0, 0]])
def test_load_paged(lib, dev, ps, lens):
    import torch
    rng = np.random.default_rng(len(lens))
    P = max(1, -(-max(lens) // ps))
    slots = ps * len(lens) * P + 3
    codes, sc = _finite_codes(rng, (slots, 144)), rng.uniform(0.5, 2, slots).astype(np.float32)
    keys = torch.from_numpy(codes).to(dev)[:, :128]
    table = rng.permutation(len(lens) * P).reshape(len(lens), P)
    table[0, 0] = -1
    table[-1, 0] = 10 ** 6      # beyond the cache
    starts = np.concatenate([[0], np.cumsum(lens)])
    n = int(starts[-1])
    out = torch.full((n + 9, 128), GUARD, dtype=torch.uint8, device=dev)
    outs = torch.full((n + 9,), float(GUARD), device=dev)
    note(f"load index keys ps={ps} {lens[:4]}")
    lib.indexer_cache_load_paged(_i32(table, dev), _i32(starts, dev), ps, n + 9, keys, torch.from_numpy(sc).to(dev),
                                 out_keys=out, out_scale=outs)
    k, s = out.cpu().numpy(), outs.cpu().numpy()
    assert (k[n:] == GUARD).all() and (s[n:] == GUARD).all()
    for b, L in enumerate(lens):
        for i in range(L):
            slot = table[b, i // ps] * ps + i % ps
            ok = table[b, i // ps] >= 0 and slot < slots
            assert (k[starts[b] + i] == (codes[slot, :128] if ok else 0)).all() and s[starts[b] + i] == (sc[slot] if ok else 0)
    fresh = lib.indexer_cache_load_paged(_i32(table, dev), _i32(starts, dev), ps, n, keys, torch.from_numpy(sc).to(dev))
    assert torch.equal(fresh[0], out[:n]) and torch.equal(fresh[1], outs[:n])


# ---- scores -----------------------------------------------------------------------------------

SCORES = {
    # cached lengths (new tokens included), new tokens, page size, width below the table's or None, rows of padding
    "one": ([300], [1], 64, None, 0),
    "decode": ([1, 500, 31, 32, 33, 128, 129, 2000], [1] * 8, 64, None, 0),
    "idle": ([77, 0, 500, 9], [1, 0, 0, 1], 16, None, 2),
    "two_each": ([130, 2, 700], [2, 2, 2], 1, None, 0),
    "chunks": ([300, 40, 0, 1000, 5], [70, 40, 0, 1, 5], 16, None, 3),
    "longer_than_cached": ([3, 400], [5, 3], 32, None, 0),       # tokens that see nothing
    "narrow": ([500, 60], [3, 2], 64, 200, 1),
    "narrow_decode": ([500, 60], [1, 1], 64, 130, 0),
    "many": ([1 + (i * 37) % 150 for i in range(700)], [1] * 700, 16, None, 0),
    "many_idle": ([20] * 600, [1 if i in (0, 299, 599) else 0 for i in range(600)], 16, None, 0),
    "none": ([], [], 16, None, 4),
}


def _scores_case(rng, name, dev):
    import torch
    lens, new, ps, width, pad = SCORES[name]
    B, T = len(lens), sum(new) + pad
    P = max([1] + [-(-n // ps) for n in lens])
    slots = ps * max(1, B) * P
    codes, sc = _finite_codes(rng, (slots, 128)), rng.uniform(0.5, 2, slots).astype(np.float32)
    table = rng.permutation(max(1, B) * P).reshape(max(1, B), P)[:B]
    if B > 2:
        table[2, 0] = -1
        table[0, -1] = 10 ** 7
    q, w = _finite_codes(rng, (T, 32, 128)), rng.standard_normal((T, 32)).astype(np.float32)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    return dict(lens=lens, new=new, ps=ps, width=width, B=B, T=T, P=P, slots=slots, codes=codes, sc=sc, table=table, q=q,
                w=w, starts=starts, dev=dict(q=torch.from_numpy(q).to(dev), w=torch.from_numpy(w).to(dev),
                                             keys=torch.from_numpy(codes).to(dev), scale=torch.from_numpy(sc).to(dev),
                                             table=_i32(table.reshape(B, P), dev), lens=_i32(lens, dev), starts=_i32(starts, dev)))


@pytest.mark.parametrize("name", sorted(SCORES))
def test_scores(lib, dev, name):
    import torch
    c = _scores_case(np.random.default_rng(sorted(SCORES).index(name)), name, dev)
    d, ps, P = c["dev"], c["ps"], c["P"]
    width = c["width"] or P * ps
    out = torch.full((c["T"], width), float(GUARD), device=dev)
    note(f"paged scores {name} T={c['T']}")
    got, lens = lib.indexer_logits_paged(d["q"], d["w"], d["keys"], d["scale"], d["table"], d["lens"], d["starts"], ps, out=out)
    assert got is out
    got, lens = out.cpu().numpy(), lens.cpu().numpy()
    assert (got[c["starts"][-1]:] == GUARD).all() and (lens[c["starts"][-1]:] == 0).all()
    for b in range(c["B"]):
        for i in range(c["new"][b]):
            t = int(c["starts"][b]) + i
            L = max(0, min(c["lens"][b] - c["new"][b] + i + 1, width, P * ps))
            assert lens[t] == L and (got[t, L:] == GUARD).all()
            if L == 0:
                continue
            pos = np.arange(L)
            page = c["table"][b].astype(np.int64)[pos // ps]
            slot = page * ps + pos % ps
            ok = (page >= 0) & (slot < c["slots"])
            slot = np.where(ok, slot, 0)
            row = c["codes"][slot], c["sc"][slot]
            want = np.where(ok, ix.indexer_scores_row(c["q"][t], c["w"][t], *row, range(L)), -np.inf)
            err = check(f"{b} {i}", got[t, :L], want, ix.fp32_error_bound(c["q"][t], c["w"][t], *row, range(L)))
            assert err is None, err


@pytest.mark.parametrize("new", [1, 5])
def test_scores_are_those_of_contiguous_keys(lib, dev, new):
    """The same fp32 values, bit by bit, as over the keys laid in a row."""
    import torch
    rng = np.random.default_rng(4)
    B, ps, lens = 6, 16, [40, 700, 129, 64, 6, 1000]
    P = -(-max(lens) // ps)
    table, n = _i32(rng.permutation(B * P).reshape(B, P), dev), _i32(lens, dev)
    keys = torch.from_numpy(_finite_codes(rng, (B * P * ps, 128))).to(dev)
    scale = torch.from_numpy(rng.uniform(0.5, 2, B * P * ps).astype(np.float32)).to(dev)
    q = torch.from_numpy(_finite_codes(rng, (B * new, 32, 128))).to(dev)
    w = torch.from_numpy(rng.standard_normal((B * new, 32)).astype(np.float32)).to(dev)
    starts, kv = np.arange(B + 1) * new, np.concatenate([[0], np.cumsum(lens)])
    got, rows = lib.indexer_logits_paged(q, w, keys, scale, table, n, _i32(starts, dev), ps)
    flat, fscale = lib.indexer_cache_load_paged(table, _i32(kv, dev), ps, int(kv[-1]), keys, scale)
    ks = np.repeat(kv[:-1], new)
    ke = ks + rows.cpu().numpy()
    want = lib.indexer_logits(q, w, flat, fscale, _i32(ks, dev), _i32(ke, dev), P * ps)
    for t in range(B * new):
        assert torch.equal(got[t, :int(rows[t])], want[t, :int(rows[t])])


@pytest.mark.parametrize("ps", [4, 32])
@pytest.mark.parametrize("new", [1, 2, 6])
def test_scores_of_pages_named_twice(lib, dev, new, ps):
    """Requests that name one page several times, their own and each other's, have its scores as often; the width is wider
    than what is cached."""
    import torch
    rng = np.random.default_rng(5)
    keys = torch.from_numpy(_finite_codes(rng, (4 * ps, 128))).to(dev)
    scale = torch.from_numpy(rng.uniform(0.5, 2, 4 * ps).astype(np.float32)).to(dev)
    q1, w1 = _finite_codes(rng, (new, 32, 128)), rng.standard_normal((new, 32)).astype(np.float32)
    q, w = torch.from_numpy(np.tile(q1, (2, 1, 1))).to(dev), torch.from_numpy(np.tile(w1, (2, 1))).to(dev)
    table = _i32([[3, 1, 3, 3, 0], [3, 3, 1, 3, 1]], dev)
    width = 5 * ps + 70
    got, lens = lib.indexer_logits_paged(q, w, keys, scale, table, _i32([5 * ps, 5 * ps], dev), _i32([0, new, 2 * new], dev), ps,
                                         width=width, out=torch.full((2 * new, width), float(GUARD), device=dev))
    got = got.cpu().numpy()
    assert lens.tolist() == [5 * ps - new + i + 1 for i in range(new)] * 2
    for i in range(new):
        a, b = got[i], got[new + i]
        n = 5 * ps - new + i + 1
        assert (a[n:] == GUARD).all() and (b[n:] == GUARD).all()
        page = lambda row, p: row[p * ps:min(n, (p + 1) * ps)]     # noqa: E731
        for row, p in ((a, 2), (b, 0), (b, 1), (b, 3)):
            np.testing.assert_array_equal(page(row, p), page(a, 0)[:len(page(row, p))])
        np.testing.assert_array_equal(page(a, 1), page(b, 2))
        rows = np.arange(ps) + 3 * ps
        want = ix.indexer_scores_row(q1[i], w1[i], keys.cpu().numpy()[rows], scale.cpu().numpy()[rows], range(ps))
        err = check(f"{i}", a[:ps], want, ix.fp32_error_bound(q1[i], w1[i], keys.cpu().numpy()[rows], scale.cpu().numpy()[rows], range(ps)))
        assert err is None, err


def test_scores_far_slots(lib, dev):
    """Slots whose bytes lie beyond 2^32 of the cache's start."""
    import torch
    rng = np.random.default_rng(3)
    slots, stride, ps = 70000, 65536, 16
    buf = torch.empty((slots, stride), dtype=torch.uint8, device=dev)
    keys, n = buf[:, :128], 40
    codes = _finite_codes(rng, (n, 128))
    pages = np.array([slots // ps - 1, slots // ps - 2, 4200])
    slot = (pages[np.arange(n) // ps] * ps + np.arange(n) % ps)
    keys[torch.from_numpy(slot).to(dev)] = torch.from_numpy(codes).to(dev)
    scale = torch.zeros(slots, device=dev)
    sc = rng.uniform(0.5, 2, n).astype(np.float32)
    scale[torch.from_numpy(slot).to(dev)] = torch.from_numpy(sc).to(dev)
    q, w = _finite_codes(rng, (1, 32, 128)), rng.standard_normal((1, 32)).astype(np.float32)
    got, _ = lib.indexer_logits_paged(torch.from_numpy(q).to(dev), torch.from_numpy(w).to(dev), keys, scale,
                                      _i32(pages[None], dev), _i32([n], dev), _i32([0, 1], dev), ps)
    err = check("far", got[0, :n].cpu().numpy(), ix.indexer_scores_row(q[0], w[0], codes, sc, range(n)),
                ix.fp32_error_bound(q[0], w[0], codes, sc, range(n)))
    assert err is None, err
    # and the store and the load that put them there and bring them back
    k, kh = _bf(rng, (n, 128), dev)
    lib.indexer_cache_store(k, _i32(slot, dev), keys, scale)
    flat, fs = lib.indexer_cache_load_paged(_i32(pages[None], dev), _i32([0, n], dev), ps, n, keys, scale)
    for t in range(n):
        _check_row(f"far {t}", kh[t], flat[t].cpu().numpy(), fs[t].item())


# ---- a step -----------------------------------------------------------------------------------

class Step:
    """A decode step through all calls: append plan, store, queries, scores, selection."""

    def __init__(self, lib, dev, seed, B=5, ps=16, k=64):
        import torch
        rng = np.random.default_rng(seed)
        self.lib, self.B, self.ps, self.k, P = lib, B, ps, k, 40
        self.kv = _i32(rng.integers(100, 500, B), dev)
        self.new = _i32(np.ones(B), dev)
        self.table = _i32(np.arange(B * P).reshape(B, P), dev)
        self.free = _i32(np.arange(B * P, B * P + 50), dev)
        slots = (B * P + 50) * ps
        self.keys = torch.from_numpy(_finite_codes(rng, (slots, 128))).to(dev)
        self.scale = torch.from_numpy(rng.uniform(0.5, 2, slots).astype(np.float32)).to(dev)
        self.cs = torch.from_numpy(_angles(1000)).to(dev)
        self.inputs(seed, dev)

    def inputs(self, seed, dev):
        rng = np.random.default_rng(seed + 100)
        k, self.kh = _bf(rng, (self.B, 128), dev)
        q, self.qh = _bf(rng, (self.B, 32, 128), dev)
        w, self.wh = _bf(rng, (self.B, 32), dev)
        if hasattr(self, "x"):
            for a, b in zip(self.x, (k, q, w)):
                a.copy_(b)
        else:
            self.x = (k, q, w)

    def run(self, stream=None):
        lib, (k, q, w) = self.lib, self.x
        plan = lib.paged_append_plan(self.kv, self.new, self.table, self.free, self.ps, self.B, stream=stream)
        turn = dict(positions=plan.positions, cos_sin=self.cs, hadamard=True, stream=stream)
        lib.indexer_cache_store(k, plan.slot_map, self.keys, self.scale, **turn)
        codes, weights = lib.indexer_queries(q, w, 0.5, **turn)
        logits, lens = lib.indexer_logits_paged(codes, weights, self.keys, self.scale, self.table, plan.seq_lens,
                                                plan.q_starts, self.ps, stream=stream)
        slots, raw = lib.topk_transform_sorted(logits, lens, self.table, self.k, self.ps, want_raw=True, stream=stream)
        return codes, weights, logits, lens, slots, raw, plan

    def check(self, got):
        codes, weights, logits, lens, slots, raw, plan = (x.cpu().numpy() if hasattr(x, "cpu") else x for x in got)
        kv, table = self.kv.cpu().numpy(), self.table.cpu().numpy()
        keys, scale = self.keys.cpu().numpy(), self.scale.cpu().numpy()
        for b in range(self.B):
            L = kv[b] + 1
            assert lens[b] == L
            pos = np.arange(L)
            at = table[b][pos // self.ps] * self.ps + pos % self.ps
            _check_row(f"key {b}", self.kh[b], keys[at[-1]], scale[at[-1]], cos_sin=self.cs.cpu().numpy()[kv[b]], mix=True)
            want = ix.indexer_scores_row(codes[b], weights[b], keys[at], scale[at], range(L))
            err = check(f"scores {b}", logits[b, :L], want, ix.fp32_error_bound(codes[b], weights[b], keys[at], scale[at], range(L)))
            assert err is None, err
            order = np.lexsort((pos, -logits[b, :L].astype(np.float64)))[:self.k]
            np.testing.assert_array_equal(raw[b], order)
            np.testing.assert_array_equal(slots[b], at[order])


def test_step(lib, dev):
    s = Step(lib, dev, 1)
    s.check(s.run())


def test_step_captured(lib, dev):
    """The same in a graph, replayed on other inputs, with eager work between."""
    import torch
    s = Step(lib, dev, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = s.run()
    for seed in (3, 4, 5):
        s.inputs(seed, dev)
        for x in got[:6]:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        s.check(got)
        (got[2].float() * 2).sum().item()      # eager work between the replays


def test_two_steps_on_streams(lib, dev):
    import torch
    steps = [Step(lib, dev, 10 + i) for i in range(3)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    got = [s.run(stream=st) for _ in range(4) for s, st in zip(steps, streams)][-3:]
    torch.cuda.synchronize()
    for s, g in zip(steps, got):
        s.check(g)


def test_refusals(lib, dev):
    """Tensors that do not fit are refused before anything is queued."""
    import torch
    t = lambda *shape, dtype=torch.uint8: torch.zeros(shape, dtype=dtype, device=dev)   # noqa: E731
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    keys, scale, table = t(64, 128), t(64, dtype=f32), t(2, 4, dtype=i32)
    store = dict(k=t(3, 128, dtype=bf), slot_map=t(3, dtype=i32), keys=keys, key_scale=scale)
    for bad in (dict(k=t(3, 128, dtype=f32)), dict(k=t(3, 120, dtype=bf)), dict(k=t(3, 256, dtype=bf)[:, ::2]), dict(slot_map=t(2, dtype=i32)),
                dict(slot_map=t(3, dtype=torch.int64)), dict(keys=t(64, 128, dtype=bf)), dict(keys=t(64, 136)[:, 4:132]),
                dict(key_scale=t(63, dtype=f32)), dict(key_scale=t(64, dtype=bf)), dict(norm_weight=t(128, dtype=bf)),
                dict(norm_weight=t(128, dtype=bf), norm_bias=t(128, dtype=f32)), dict(positions=t(3, dtype=i32)),
                dict(cos_sin=t(5, 64, dtype=f32)), dict(positions=t(3, dtype=i32), cos_sin=t(5, 32, dtype=f32)),
                dict(k=t(3, 128, dtype=bf).cpu())):
        with pytest.raises(ValueError):
            lib.indexer_cache_store(**{**store, **bad})
    qs = dict(q=t(3, 32, 128, dtype=bf), weights=t(3, 32, dtype=f32))
    for bad in (dict(q=t(3, 31, 128, dtype=bf)), dict(q=t(3, 32, 128, dtype=f32)), dict(weights=t(3, 31, dtype=f32)),
                dict(weights=t(3, 32, dtype=i32)), dict(out_q=t(3, 32, 128, dtype=bf)), dict(out_weights=t(3, 32, dtype=bf)),
                dict(q=t(3, 1, 128, dtype=bf).expand(3, 32, 128)), dict(positions=t(3, dtype=i32))):
        with pytest.raises(ValueError):
            lib.indexer_queries(**{**qs, **bad})
    load = dict(page_table=table, kv_starts=t(3, dtype=i32), page_size=16, num_rows=5, keys=keys, key_scale=scale)
    for bad in (dict(kv_starts=t(2, dtype=i32)), dict(page_size=12), dict(page_size=0), dict(num_rows=-1),
                dict(out_keys=t(4, 128)), dict(out_scale=t(4, dtype=f32)), dict(page_table=t(8, dtype=i32))):
        with pytest.raises(ValueError):
            lib.indexer_cache_load_paged(**{**load, **bad})
    score = dict(q=t(2, 32, 128), weights=t(2, 32, dtype=f32), keys=keys, key_scale=scale, page_table=table,
                 seq_lens=t(2, dtype=i32), q_starts=t(3, dtype=i32), page_size=16)
    for bad in (dict(q=t(2, 32, 128, dtype=bf)), dict(q=t(2, 32, 64)), dict(weights=t(2, 32, dtype=bf)), dict(seq_lens=t(3, dtype=i32)),
                dict(q_starts=t(2, dtype=i32)), dict(page_size=3), dict(width=-1), dict(out=t(2, 63, dtype=f32), width=64),
                dict(lens=t(3, dtype=i32)), dict(out=t(2, 64, dtype=bf))):
        with pytest.raises(ValueError):
            lib.indexer_logits_paged(**{**score, **bad})


# ---- rows at the ends of the range --------------------------------------------------------------

@pytest.mark.parametrize("mix", [False, True])
def test_rows_far_below_one(lib, dev, mix):
    """Down to values that are subnormal themselves, a row's scale is its maximum's part, 2^-126 at least, and its codes are
    within half a step of it.  (No absolute term in the bounds: a row of zeros would not pass.)"""
    import torch
    rng = np.random.default_rng(21)
    sizes = [1e-28, 1e-30, 1e-33, 1e-35, 3e-36, 3e-37, 1e-37, 1e-38, 1e-39, 2e-40]
    k = (torch.from_numpy(rng.standard_normal((len(sizes), 128))) * torch.tensor(sizes, dtype=torch.float64)[:, None]).bfloat16()
    kh = k.double().numpy()
    least, clamped = 2.0 ** -126, 0
    keys, scale = torch.zeros((16, 128), dtype=torch.uint8, device=dev), torch.zeros(16, device=dev)
    q = k[:, None].expand(-1, 32, -1).contiguous().to(dev)
    lib.indexer_cache_store(k.to(dev), _i32(range(len(sizes)), dev), keys, scale, hadamard=mix)
    qc, qw = lib.indexer_queries(q, torch.ones((len(sizes), 32), device=dev), hadamard=mix)
    codes, s = keys.cpu().numpy(), scale.double().cpu().numpy()
    assert torch.equal(qc[:, 31], keys[:len(sizes)]) and torch.equal(qw[:, 31], scale[:len(sizes)])
    for t in range(len(sizes)):
        r = po.row(kh[t], mix=mix)
        top = np.abs(r.y).max()
        want = max(top / 448.0, least)
        clamped += want == least
        # the row's own error, the quotient's rounding and, with mixing, the product's and the factor's
        off = r.slack.max() / 448.0 + 4 * po.U32 * want
        assert abs(s[t] - want) <= off, (t, s[t], want, off)
        bound = po.U8 * (np.abs(r.y) + r.slack) + po.TINY8 * s[t] + r.slack + 8 * po.U32 * np.abs(r.y)
        err = check(f"row {t}", e4m3_value(codes[t]) * s[t], r.y, bound)
        assert err is None, err
        if top > 0.01 * least:
            assert codes[t].any()
    assert clamped >= 3


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -10, 1.0, 2.0 ** 100])
def test_codes_of_ties(lib, dev, size):
    """Codes are the fp32 quotient by the step, rounded to nearest even: exactly, where many values lie on ties
    of the codes or one unit of fp32 beside one."""
    import torch
    rng = np.random.default_rng(22)
    top = (1 + np.arange(128) / 128.0).astype(np.float32)         # every bf16 mantissa as a row's maximum
    k = np.zeros((128, 128), np.float32)
    # the bf16 numbers around the ties (an odd number of sixteenths, 16 to 32 of them) of a row
    for t in range(128):
        ties = np.array([(16 + 2 * (i % 8) + 1) * 2.0 ** (4 - i // 8) for i in range(126)]) % 448 * top[t] / 448
        near = torch.from_numpy(ties).bfloat16().float().numpy()
        k[t] = np.concatenate([[top[t]], near, [0.75 * top[t]]])
    k = torch.from_numpy((k * rng.choice([-1, 1], k.shape) * size).astype(np.float32)).bfloat16()
    v = k.float()
    step = v.abs().amax(1) / 448                                  # fp32 divisions, as the definition's
    want = (v / step[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    keys, scale = torch.zeros((128, 128), dtype=torch.uint8, device=dev), torch.zeros(128, device=dev)
    lib.indexer_cache_store(k.to(dev), _i32(range(128), dev), keys, scale)
    assert torch.equal(scale.cpu(), step)
    assert torch.equal(keys.cpu(), want)
    codes, w = lib.indexer_queries(k[:, None].expand(-1, 32, -1).contiguous().to(dev), torch.ones((128, 32), device=dev))
    assert torch.equal(codes[:, 5].cpu(), want) and torch.equal(w[:, 31].cpu(), step)


@pytest.mark.parametrize("mix", [False, True])
def test_norm_of_large_values(lib, dev, mix):
    """The layer norm of rows up to the largest bf16 numbers, whose squares and sums do not fit fp32."""
    import torch
    rng = np.random.default_rng(23)
    sizes = [1e3, 1e15, 2e18, 1e19, 1e20, 1e30, 1e36, 8e37, 1e38, 1e38]
    k = (torch.from_numpy(rng.standard_normal((len(sizes), 128))).clamp(-3, 3)
         * torch.tensor(sizes, dtype=torch.float64)[:, None]).bfloat16()
    k[8] = k[8].abs()                                             # a sum beyond fp32
    k[9, 77] = float("inf")
    kh = k.double().numpy()
    w, bias = 1 + 0.2 * torch.randn(128, generator=torch.Generator().manual_seed(3)), torch.full((128,), 0.1)
    keys, scale = torch.zeros((16, 128), dtype=torch.uint8, device=dev), torch.zeros(16, device=dev)
    lib.indexer_cache_store(k.to(dev), _i32(range(len(sizes)), dev), keys, scale, norm_weight=w.to(dev), norm_bias=bias.to(dev),
                            eps=1e-6, hadamard=mix)
    codes, s = keys.cpu().numpy(), scale.cpu().numpy()
    for t in range(len(sizes) - 1):
        _check_row(f"row {t}", kh[t], codes[t], s[t], weight=w.double().numpy(), bias=bias.double().numpy(), eps=1e-6, mix=mix)
    assert np.isnan(s[len(sizes) - 1])


# ---- pages that are not there, in every form of the scores --------------------------------------

@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("new", [1, 2, 3, 9])
def test_scores_of_missing_pages(lib, dev, new, ps):
    """Negative pages and pages beyond the cache, where tokens see them: -inf whatever the weights, one token a request (of pages
    that hold whole tiles of keys and of others), two, and more; keys that are there have their scores."""
    import torch
    rng = np.random.default_rng(31)
    B, P = 7, 12
    slots = 50 * ps - (0 if 50 * ps % 32 == 0 else 50 * ps % 32)
    codes, sc = _finite_codes(rng, (slots, 128)), rng.uniform(0.5, 2, slots).astype(np.float32)
    table = rng.integers(0, slots // ps, (B, P))
    table[:, 0], table[:, 5], table[1:, 7] = -1, -2 ** 31, 10 ** 7
    table[:, 3], table[:, 9], table[0, 7] = slots // ps, 2 ** 31 - 1, -5
    lens = rng.integers(9 * ps + new, P * ps + 1, B)
    lens[2], lens[3] = new, P * ps
    q, w = _finite_codes(rng, (B * new, 32, 128)), rng.standard_normal((B * new, 32)).astype(np.float32)
    starts = np.arange(B + 1) * new
    d = dict(q=torch.from_numpy(q).to(dev), w=torch.from_numpy(w).to(dev), k=torch.from_numpy(codes).to(dev),
             s=torch.from_numpy(sc).to(dev), t=_i32(table, dev), n=_i32(lens, dev), b=_i32(starts, dev))
    wild = d["w"].clone()
    wild[:, 3], wild[:, 4], wild[::2, 5] = float("inf"), float("-inf"), float("nan")
    note(f"missing pages new={new} ps={ps}")
    got, rows = lib.indexer_logits_paged(d["q"], d["w"], d["k"], d["s"], d["t"], d["n"], d["b"], ps)
    other, _ = lib.indexer_logits_paged(d["q"], wild, d["k"], d["s"], d["t"], d["n"], d["b"], ps)
    got, other, seen = got.cpu().numpy(), other.cpu().numpy(), {"negative": 0, "beyond": 0}
    for b in range(B):
        for i in range(new):
            t, L = b * new + i, int(lens[b]) - new + i + 1
            assert int(rows[t]) == L
            pos = np.arange(L)
            page = table[b].astype(np.int64)[pos // ps]
            slot = page * ps + pos % ps
            ok = (page >= 0) & (slot < slots)
            seen["negative"] += int((page < 0).any())
            seen["beyond"] += int((slot >= slots).any())
            slot = np.where(ok, slot, 0)
            row = codes[slot], sc[slot]
            want = np.where(ok, ix.indexer_scores_row(q[t], w[t], *row, range(L)), -np.inf)
            err = check(f"{b} {i}", got[t, :L], want, ix.fp32_error_bound(q[t], w[t], *row, range(L)))
            assert err is None, err
            assert np.isneginf(other[t, :L][~ok]).all() and not np.isfinite(other[t, :L]).any()
    assert min(seen.values()) >= (B - 1) * new


# ---- many tiles to a workgroup, many requests to a workgroup ------------------------------------

LONG = {
    # cached lengths, new tokens: enough for several tiles (of 128 keys, with three tokens or more 64) to each of the workgroups, of
    # which there are four or two a CU; or for several requests to each
    "one_token": ([1_000_003], [1]),
    "two_tokens": ([700_001], [2]),
    "decode": ([3 + (i * 7919) % 65536 for i in range(64)], [1] * 64),
    "two_each": ([3 + (i * 7919) % 65536 for i in range(64)], [2] * 64),
    "chunk": ([16_391], [1003]),
    "chunks": ([9_000, 20_001, 70, 12_345], [300, 129, 70, 517]),
    "three_each": ([3 + (i * 7919) % 33333 for i in range(40)], [3] * 40),
    "short": ([1 + (i * 37) % 300 for i in range(3000)], [1] * 3000),
    "short_two_each": ([2 + (i * 37) % 300 for i in range(2000)], [2] * 2000),
    "short_some": ([9 + (i * 37) % 300 for i in range(1500)], [(i * 5) % 9 for i in range(1500)]),
    "mixed": ([40_000] + [2000 + (i * 7919) % 9000 for i in range(63)], [1500] + [1] * 63),
}


@pytest.mark.parametrize("ps", [8, 64])
@pytest.mark.parametrize("name", sorted(LONG))
def test_scores_of_long_shares(lib, dev, name, ps):
    """Loops that run many times in each workgroup and pass from request to request: every score is, bit by bit, that of
    the scan over the same keys in a row, and some are held against the oracle."""
    import torch
    lens, new = LONG[name]
    B, T, P = len(lens), sum(new), -(-max(lens) // ps)
    gen = torch.Generator(device=dev).manual_seed(sorted(LONG).index(name))
    pages = -(-np.asarray(lens) // ps)
    total = int(pages.sum())
    slots = (total + 8) // 8 * 8 * ps                     # a multiple of 32 or more
    keys = torch.randint(0, 256, (slots, 128), dtype=torch.uint8, device=dev, generator=gen)
    keys = torch.where((keys & 0x7F) == 0x7F, keys ^ 0x10, keys)
    scale = torch.rand(slots, device=dev, generator=gen) + 0.5
    q = torch.randint(0, 256, (T, 32, 128), dtype=torch.uint8, device=dev, generator=gen)
    q = torch.where((q & 0x7F) == 0x7F, q ^ 0x10, q)
    w = torch.randn((T, 32), device=dev, generator=gen)
    rng = np.random.default_rng(7)
    order, table, at = rng.permutation(total), np.full((B, P), -1, np.int64), 0
    for b in range(B):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
    for b, page in ((0, -3), (B - 1, 10 ** 7), (B // 2, -1)):
        table[b, pages[b] // 2] = page                    # not there, within what tokens see
    tab, n, starts = _i32(table, dev), _i32(lens, dev), np.concatenate([[0], np.cumsum(new)])
    width = P * ps
    out = torch.full((T, width), float(GUARD), device=dev)
    note(f"long shares {name} ps={ps} T={T} width={width}")
    got, rows = lib.indexer_logits_paged(q, w, keys, scale, tab, n, _i32(starts, dev), ps, out=out)
    want_rows = np.concatenate([[lens[b] - new[b] + i + 1 for i in range(new[b])] for b in range(B)]).clip(0)
    np.testing.assert_array_equal(rows.cpu().numpy(), want_rows)
    # the keys in a row, and which of them are there
    kv = np.concatenate([[0], np.cumsum(lens)])
    flat, fscale = lib.indexer_cache_load_paged(tab, _i32(kv, dev), ps, int(kv[-1]), keys, scale)
    first = torch.from_numpy(np.repeat(kv[:-1], new)).to(dev)
    ks, ke = first.int(), (first + rows).int()
    want = lib.indexer_logits(q, w, flat, fscale, ks, ke, width)
    owner = torch.from_numpy(np.repeat(np.arange(B), new)).to(dev)
    there = (tab >= 0) & (tab < slots // ps)
    for t0 in range(0, T, 512):                           # some rows at a time
        t = slice(t0, min(T, t0 + 512))
        inside = torch.arange(width, device=dev)[None, :] < rows[t, None]
        ok = there[owner[t]].repeat_interleave(ps, 1)
        full = torch.where(inside, torch.where(ok, want[t], float("-inf")), float(GUARD))
        same = got[t] == full
        assert bool(same.all()), [x[:4].tolist() for x in torch.nonzero(~same, as_tuple=True)]
    for t in rng.integers(0, T, 6):
        L, b = int(want_rows[t]), int(owner[t])
        if L == 0:
            continue
        pos = np.unique(np.concatenate([[0, L - 1], rng.integers(0, L, 200)]))
        page = table[b][pos // ps]
        slot = np.where((page >= 0) & (page < slots // ps), page * ps + pos % ps, -1)
        pos, slot = pos[slot >= 0], slot[slot >= 0]
        row = keys.cpu().numpy()[slot], scale.cpu().numpy()[slot]
        qt, wt = q[t].cpu().numpy(), w[t].cpu().numpy()
        err = check(f"token {t}", got[t].cpu().numpy()[pos], ix.indexer_scores_row(qt, wt, *row, range(len(pos))),
                    ix.fp32_error_bound(qt, wt, *row, range(len(pos))))
        assert err is None, err
