"""GPU tests of the paged latent cache and of latent attention against the
float64 oracle, through the binding.  The bounds are the oracle's: roundings
counted from the formulas, none fitted."""
import numpy as np
import pytest

from gpu_util import note
from oracle import latent_oracle as lo

pytestmark = pytest.mark.gpu

GUARD = -7   # what outputs hold before a call that must leave them


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def _i32(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to(dev)


def _bf(rng, shape, dev, sigma=1.0):
    """bf16 normals on the device, and their values in float64 on the host."""
    import torch
    t = (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) * sigma).bfloat16()
    return t.to(dev), t.double().numpy()


def _host(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """A filled cache and its float64 values.  joint: latent and rope share one
    buffer with a longer row stride."""

    def __init__(self, rng, slots, e4m3, dev, joint=False):
        import torch
        self.slots, self.e4m3 = slots, e4m3
        if e4m3:
            codes = rng.integers(0, 256, (slots, 512), dtype=np.uint8)
            codes[(codes & 0x7F) >= 0x78] &= 0x97   # finite, up to 30
            scale = rng.uniform(0.02, 0.05, slots).astype(np.float32)
            wide = torch.zeros((slots, 528 if joint else 512), dtype=torch.uint8, device=dev)
            wide[:, :512] = torch.from_numpy(codes).to(dev)
            self.latent, self.scale = wide[:, :512], torch.from_numpy(scale).to(dev)
            self.c = lo.e4m3_value(codes) * scale.astype(np.float64)[:, None]
            rope, self.r = _bf(rng, (slots, 64), dev)
            self.rope = rope
        else:
            latent, self.c = _bf(rng, (slots, 512), dev)
            rope, self.r = _bf(rng, (slots, 64), dev)
            self.scale = None
            if joint:
                both = torch.zeros((slots, 592), dtype=torch.bfloat16, device=dev)
                both[:, :512], both[:, 512:576] = latent, rope
                self.latent, self.rope = both[:, :512], both[:, 512:576]
            else:
                self.latent, self.rope = latent, rope

    def poison(self, slots):
        """NaN in slots that nothing may use (host values stay finite: they are not used either)."""
        idx = [int(s) for s in slots]
        if not idx:
            return
        if self.e4m3:
            self.latent[idx] = 0x7F
            self.scale[idx] = float("nan")
        else:
            self.latent[idx] = float("nan")
        self.rope[idx] = float("nan")


def _check_token(name, cache, q, slots, scale, out, lse, heads=None):
    keys = np.concatenate([cache.c[slots], cache.r[slots]], 1)
    for h in range(q.shape[0]) if heads is None else heads:
        a = lo.attend(q[h], keys, cache.c[slots], scale)
        for err in (lo.check(f"{name} head {h} out", out[h], a.out, a.out_bound),
                    lo.check(f"{name} head {h} lse", lse[h], a.lse, a.lse_bound)):
            assert err is None, err


# ---- plan -------------------------------------------------------------------------------------

PLANS = {
    # requests, longest cached, longest new, page size, pages per row or None, token buffer beyond the tokens, pages missing
    "one": (1, 100, 1, 16, None, 0, 0),
    "none": (0, 1, 1, 16, 3, 5, 0),
    "decode": (64, 5000, 1, 64, None, 0, 0),
    "mixed": (300, 900, 130, 16, None, 77, 0),
    "page_1": (37, 50, 9, 1, None, 3, 0),
    "tiles": (2500, 40, 7, 8, None, 0, 0),          # more requests than one scan tile
    "long_prompt": (3, 10, 9000, 64, None, 0, 0),   # one request's tokens over many workgroups
    "short_buffer": (40, 100, 20, 16, None, -50, 0),
    "short_rows": (20, 100, 90, 16, 6, 4, 0),       # tokens past the page table's row
    "out_of_pages": (50, 64, 40, 16, None, 10, 7),
}


@pytest.mark.parametrize("name", sorted(PLANS))
def test_plan(lib, dev, name):
    import torch
    B, kv_hi, new_hi, ps, P, extra, missing = PLANS[name]
    rng = np.random.default_rng(sorted(PLANS).index(name))
    kv, new = rng.integers(0, kv_hi + 1, B), rng.integers(0, new_hi + 1, B)
    if name == "decode":
        new[:] = 1
    if name == "long_prompt":
        new[1] = new_hi
    if B > 5:
        kv[2], new[3], new[4] = -4, -9, 0
    seq = np.maximum(kv, 0) + np.maximum(new, 0)
    P = P or (int(-(-seq.max() // ps)) if B else 1)
    table = rng.integers(0, 10 ** 6, (B, P))
    if B > 8:
        table[7, 0] = -1            # a kept page that is not there
        table[8, 0] = 2 ** 31 - 2   # and one whose slots do not fit int32 (page size above 1)
    used = 3
    need = lo.append_plan(kv, new, table, [], 0, ps, 0).free_used
    free = rng.permutation(10 ** 6)[:max(0, need + used - missing)]
    T = max(0, int(np.maximum(new, 0).sum()) + extra)
    want = lo.append_plan(kv, new, table, free, used, ps, T)
    t = _i32(table, dev).reshape(B, P)
    note(f"plan {name} B={B} T={T}")
    got = lib.paged_append_plan(_i32(kv, dev), _i32(new, dev), t, _i32(free, dev), ps, T, free_used=_i32([used], dev))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(t.cpu().numpy(), want.page_table.reshape(B, P))
    for field in ("seq_lens", "q_starts", "slot_map", "positions"):
        np.testing.assert_array_equal(getattr(got, field).cpu().numpy(), getattr(want, field), err_msg=field)
    assert int(got.free_used[0]) == want.free_used
    if name == "out_of_pages":
        assert want.free_used > len(free)


# ---- store and load ---------------------------------------------------------------------------

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("norm,rotate", [(True, "pairs"), (True, "halves"), (False, "pairs"), (True, None), (False, None)])
@pytest.mark.parametrize("tokens", [1, 7, 130])
def test_store(lib, dev, e4m3, norm, rotate, tokens):
    import torch
    rng = np.random.default_rng(tokens + 10 * norm)
    joint = tokens == 7
    cache = Cache(rng, 200, e4m3, dev, joint)
    kv, kvh = _bf(rng, (tokens, 600 if joint else 576), dev, 2.5)
    kv, kvh = kv[:, :576], kvh[:, :576]
    w, wh = _bf(rng, (512,), dev)
    angle = rng.uniform(0, 6.28, (50, 32))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos = rng.integers(0, 50, tokens)
    slots = rng.permutation(200)[:tokens]
    special = tokens > 20
    if special:
        kv[3, :512] = 0
        kvh[3, :512] = 0
        kv[5] *= 2.0 ** -100
        kvh[5] *= 2.0 ** -100
        slots[8], slots[9] = -1, 200          # not stored
        pos[10], pos[11] = -1, 50             # nor these, when rotated
    before = (cache.latent.clone(), cache.rope.clone(), cache.scale.clone() if e4m3 else None)
    note(f"store e4m3={e4m3} norm={norm} rotate={rotate} tokens={tokens}")
    lib.latent_cache_store(kv, _i32(slots, dev), cache.latent, cache.rope, scale=cache.scale,
                           norm_weight=w if norm else None, eps=1e-5, interleaved=rotate == "pairs",
                           positions=_i32(pos, dev) if rotate else None,
                           cos_sin=torch.from_numpy(cs).to(dev) if rotate else None)
    torch.cuda.synchronize()
    latent, rope = cache.latent.cpu(), _host(cache.rope)
    scale = cache.scale.double().cpu().numpy() if e4m3 else None
    stored = [t for t in range(tokens) if 0 <= slots[t] < 200 and not (rotate and not 0 <= pos[t] < 50)]
    for t in stored:
        s = slots[t]
        y = lo.normed(kvh[t, :512], wh if norm else None, 1e-5)
        slack = (lo.NORM_ERROR if norm else 0) * np.abs(y)
        if e4m3:
            top = np.abs(y).max()
            if top == 0:
                assert scale[s] == 1.0
            else:
                assert abs(scale[s] - top / 448) <= (lo.NORM_ERROR + 4 * lo.U32) * top / 448
            value = lo.e4m3_value(latent[s].numpy()) * scale[s]
            # half a step of the code (2^-4; 2^-10 of the scale where it is subnormal); the largest lands on 448 within its slack
            err = lo.check(f"token {t}", value, y, np.abs(y) * 2.0 ** -4 + 2.0 ** -10 * scale[s] + slack
                           + np.abs(y) * (lo.NORM_ERROR + 8 * lo.U32))
        else:
            err = lo.check(f"token {t}", latent[s].double().numpy(), y, lo.U16 * np.abs(y) * (1 + 2 * lo.NORM_ERROR) + slack)
        assert err is None, err
        r = lo.rotated(kvh[t, 512:], cs[pos[t]].astype(np.float64) if rotate else None, rotate == "pairs")
        size = lo.rotated(np.abs(kvh[t, 512:]), None, True)
        err = lo.check(f"token {t} rope", rope[s], r, lo.U16 * np.abs(r) + 4 * lo.U32 * 2 * size.max())
        assert err is None, err
    left = np.setdiff1d(np.arange(200), slots[stored])
    assert torch.equal(before[0].cpu()[left], latent[left])
    assert torch.equal(before[1].cpu()[left], cache.rope.cpu()[left])
    if e4m3:
        assert torch.equal(before[2].cpu()[left], cache.scale.cpu()[left])


def test_store_not_finite(lib, dev):
    """A NaN or an infinity makes its row read back as NaN in an 8-bit cache, and
    leaves the other rows alone."""
    import torch
    rng = np.random.default_rng(5)
    cache = Cache(rng, 8, True, dev)
    kv, _ = _bf(rng, (3, 576), dev)
    kv[0, 100], kv[2, 511] = float("inf"), float("nan")
    lib.latent_cache_store(kv, _i32([4, 5, 6], dev), cache.latent, cache.rope, scale=cache.scale)
    c, _ = lib.latent_cache_load(_i32([4, 5, 6], dev), cache.latent, cache.rope, scale=cache.scale)
    bad = torch.isnan(c).all(1).cpu().tolist()
    assert bad == [True, False, True] and not torch.isnan(c[1]).any()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", [1, 8, 61, 1000])
def test_load(lib, dev, e4m3, rows):
    import torch
    rng = np.random.default_rng(rows)
    cache = Cache(rng, 150, e4m3, dev, joint=rows == 61)
    slots = rng.integers(-2, 153, rows)
    note(f"load e4m3={e4m3} rows={rows}")
    c, r = lib.latent_cache_load(_i32(slots, dev), cache.latent, cache.rope, scale=cache.scale)
    ok = (slots >= 0) & (slots < 150)
    want = np.where(ok[:, None], cache.c[np.where(ok, slots, 0)], 0)
    # code * scale is one fp32 rounding, then one to bf16; bf16 rows come back as they are
    assert lo.check("latent", _host(c), want, (lo.U16 * np.abs(want) * (1 + lo.U16) if e4m3 else 0)) is None
    np.testing.assert_array_equal(_host(r), np.where(ok[:, None], cache.r[np.where(ok, slots, 0)], 0))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens", [[5], [0, 0, 17, 0, 1, 64, 0], [1] * 200, [300, 2, 129]])
def test_load_paged(lib, dev, e4m3, lens):
    import torch
    rng = np.random.default_rng(len(lens))
    ps = 16
    P = max(1, -(-max(lens) // ps))
    cache = Cache(rng, ps * (len(lens) * P + 1), e4m3, dev)
    table = rng.permutation(len(lens) * P).reshape(len(lens), P)
    table[0, 0] = -1
    table[-1, 0] = 10 ** 6      # beyond the cache
    starts = np.concatenate([[0], np.cumsum(lens)])
    n = starts[-1]
    out = torch.full((n + 9, 512), float(GUARD), dtype=torch.bfloat16, device=dev)
    outr = torch.full((n + 9, 64), float(GUARD), dtype=torch.bfloat16, device=dev)
    note(f"load paged e4m3={e4m3} {lens[:4]}")
    lib.latent_cache_load_paged(_i32(table, dev), _i32(starts, dev), ps, n + 9, cache.latent, cache.rope,
                                scale=cache.scale, out_latent=out, out_rope=outr)
    c, r = _host(out), _host(outr)
    assert (c[n:] == GUARD).all() and (r[n:] == GUARD).all()
    for b, L in enumerate(lens):
        for i in range(L):
            page = table[b, i // ps]
            slot = page * ps + i % ps
            ok = 0 <= page and slot < cache.slots
            want = cache.c[slot] if ok else np.zeros(512)
            assert lo.check(f"{b} {i}", c[starts[b] + i], want, lo.U16 * np.abs(want) * (1 + lo.U16) if e4m3 else 0) is None
            np.testing.assert_array_equal(r[starts[b] + i], cache.r[slot] if ok else np.zeros(64))


# ---- absorbed form over selected slots --------------------------------------------------------------

SELECTED = [
    # tokens, heads, k
    (1, 1, 1), (1, 32, 33), (2, 5, 64), (3, 33, 200), (1, 64, 2048), (5, 128, 100), (2, 70, 97), (4, 130, 65),
    (40, 8, 512), (300, 3, 40), (1100, 2, 31), (2, 16, 0), (350, 50, 70), (60, 24, 300),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,H,k", SELECTED)
def test_selected(lib, dev, e4m3, T, H, k):
    import torch
    rng = np.random.default_rng(T * 1000 + H * 10 + k)
    cache = Cache(rng, max(3 * k, 50), e4m3, dev, joint=H == 5)
    q, qh = _bf(rng, (T, H + 1, 600), dev)
    q, qh = q[:, 1:, :576], qh[:, 1:, :576]      # strides of a larger buffer
    idx = np.stack([rng.permutation(np.arange(1, cache.slots))[:k] for _ in range(T)]).reshape(T, k)
    for t in range(T):                           # masks: nothing, holes, a tail, slots outside, a slot twice
        kind = t % 6
        if kind == 1:
            idx[t] = -1
        elif kind == 2:
            idx[t, rng.random(k) < 0.4] = -1
        elif kind == 3:
            idx[t, k // 3:] = -1
        elif kind == 4 and k > 3:
            idx[t, 0], idx[t, 1], idx[t, 2] = cache.slots, 2 ** 31 - 1, idx[t, 3]
    used = np.unique(idx)
    cache.poison(np.setdiff1d(np.arange(cache.slots), used))     # slot 0 among them
    note(f"selected e4m3={e4m3} T={T} H={H} k={k}")
    out, lse = lib.latent_attention(q, cache.latent, cache.rope, _i32(idx, dev), 0.07, scale=cache.scale)
    out, lse = _host(out), _host(lse)
    heads = None if T * H <= 200 else sorted({0, H // 2, H - 1})
    for t in range(T) if T <= 40 else list(range(12)) + [T // 2, T - 1]:
        s = idx[t][(idx[t] >= 0) & (idx[t] < cache.slots)]
        _check_token(f"token {t}", cache, qh[t], s, 0.07, out[t], lse[t], heads)


def test_selected_large_scores(lib, dev):
    """Scores of hundreds, rising along the list: the reference moves at nearly every
    tile, and most weights vanish."""
    rng = np.random.default_rng(8)
    cache = Cache(rng, 500, False, dev)
    q, qh = _bf(rng, (2, 4, 576), dev)
    z = np.concatenate([cache.c, cache.r], 1) @ qh[0, 0]
    idx = np.stack([np.argsort(z), np.argsort(-z)])
    for scale in (1.0, 4.0, -1.0):
        out, lse = lib.latent_attention(q, cache.latent, cache.rope, _i32(idx, dev), scale)
        for t in range(2):
            _check_token(f"scale {scale} token {t}", cache, qh[t], idx[t], scale, _host(out)[t], _host(lse)[t])


@pytest.mark.parametrize("e4m3", [False, True])
def test_selected_long_list_of_few_slots(lib, dev, e4m3):
    """A list far longer than the cache, one slot many times: every naming counts,
    shared by as many workgroups as there are.  Also at scale 0, where all count alike."""
    rng = np.random.default_rng(10)
    cache = Cache(rng, 300, e4m3, dev)
    q, qh = _bf(rng, (3, 20, 576), dev)
    idx = rng.integers(0, 300, (3, 40000))
    idx[1, 100:] = 7
    idx[2, :39999] = -1                          # only the last entry
    for scale in (0.1, 0.0):
        out, lse = lib.latent_attention(q, cache.latent, cache.rope, _i32(idx, dev), scale, scale=cache.scale)
        for t in range(3):
            _check_token(f"scale {scale} token {t}", cache, qh[t], idx[t][idx[t] >= 0], scale, _host(out)[t], _host(lse)[t],
                         heads=(0, 19))


def test_selected_far_slots(lib, dev):
    """Slots whose byte offsets pass 2^32 (a cache of 9 GB)."""
    import torch
    rng = np.random.default_rng(9)
    small = Cache(rng, 64, False, dev)
    slots = 8_000_000
    latent = torch.empty((slots, 512), dtype=torch.bfloat16, device=dev)
    rope = torch.empty((slots, 64), dtype=torch.bfloat16, device=dev)
    at = np.concatenate([rng.integers(0, slots, 62), [slots - 1, 2_097_152]])
    at = np.unique(at)
    latent[_i32(at, dev).long()] = small.latent[:len(at)]
    rope[_i32(at, dev).long()] = small.rope[:len(at)]
    q, qh = _bf(rng, (1, 8, 576), dev)
    out, lse = lib.latent_attention(q, latent, rope, _i32(at[None], dev), 0.1)
    _check_token("far", small, qh[0], np.arange(len(at)), 0.1, _host(out)[0], _host(lse)[0])
    c, r = lib.latent_cache_load(_i32(at, dev), latent, rope)
    assert torch.equal(c, small.latent[:len(at)]) and torch.equal(r, small.rope[:len(at)])


# ---- absorbed form over whole sequences ---------------------------------------------------------------

PAGED = {
    # lengths (new tokens included), new tokens, heads, page size, rows of padding
    "decode": ([1, 31, 32, 33, 64, 65, 500], [1] * 7, 8, 16, 0),
    "empty": ([0, 5, 0], [1, 1, 0], 3, 16, 2),
    "several": ([40, 3, 100, 7], [3, 2, 0, 7], 33, 16, 3),
    "more_new_than_cached": ([2, 1], [5, 3], 5, 64, 0),
    "page_1": ([70, 9], [1, 2], 12, 1, 0),
    "one_long": ([9001], [1], 32, 64, 0),
    "heads_64": ([200, 77, 300], [1, 1, 1], 64, 64, 0),
    "heads_128": ([150, 90], [2, 1], 128, 64, 1),
    "many": (list(range(1, 1150)), [1] * 1149, 2, 16, 0),     # more tokens than a split launch takes
    "one_prompt": ([700], [700], 2, 16, 5),
    "wide_many": ([1 + i % 67 for i in range(1030)], [1] * 1030, 20, 16, 0),
    "wide_64": ([3 + i % 90 for i in range(360)], [1] * 360, 50, 16, 1),
    "wide_prompts": ([300, 40, 100], [200, 0, 90], 24, 64, 4),
}


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("name", sorted(PAGED))
def test_paged(lib, dev, e4m3, name):
    import torch
    lens, new, H, ps, pad = PAGED[name]
    rng = np.random.default_rng(sorted(PAGED).index(name))
    B = len(lens)
    P = max(1, -(-max(lens) // ps)) + 1
    pages = B * P + 1
    cache = Cache(rng, pages * ps, e4m3, dev, joint=name == "several")
    table = (1 + rng.permutation(B * P)).reshape(B, P)
    if name == "several":
        table[0, 1], table[2, 2] = -1, 10 ** 6      # pages that are not there
    starts = np.concatenate([[0], np.cumsum(new)])
    T = starts[-1] + pad
    used = np.concatenate([lo.page_slots(table[b], ps, lens[b], cache.slots) for b in range(B)])
    cache.poison(np.setdiff1d(np.arange(cache.slots), used))     # the rest of last pages among them
    q, qh = _bf(rng, (T, H, 576), dev)
    out = torch.full((T, H, 512), float(GUARD), dtype=torch.bfloat16, device=dev)
    lse = torch.full((T, H), float(GUARD), dtype=torch.float32, device=dev)
    note(f"paged e4m3={e4m3} {name}")
    lib.latent_attention_paged(q, cache.latent, cache.rope, _i32(table, dev), _i32(lens, dev), _i32(starts, dev), ps,
                               0.08, scale=cache.scale, out=out, lse=lse)
    out, lse = _host(out), _host(lse)
    assert (out[starts[-1]:] == GUARD).all() and (lse[starts[-1]:] == GUARD).all()
    heads = None if H <= 12 else [0, H // 2, H - 1]
    for b in range(B) if B < 100 else (0, 1, 700 % B, B - 1):
        for i in range(new[b]) if new[b] < 100 else (0, 1, 33, new[b] - 1):
            n = lo.causal_keys(i, new[b], lens[b])
            s = lo.page_slots(table[b], ps, n, cache.slots)
            _check_token(f"request {b} token {i}", cache, qh[starts[b] + i], s, 0.08, out[starts[b] + i],
                         lse[starts[b] + i], heads)


# ---- expanded form ----------------------------------------------------------------------------------

EXPANDED = {
    # query lengths, key lengths, heads, causal, rows of padding
    "one": ([1], [1], 1, True, 0),
    "square": ([130], [130], 3, True, 0),
    "ragged": ([5, 0, 64, 129, 1], [5, 9, 200, 129, 300], 4, True, 3),
    "no_keys": ([3, 40], [0, 2], 2, True, 0),           # more queries than keys: the first see none
    "not_causal": ([33, 200], [70, 1], 2, False, 0),
    "single_tokens": ([1] * 70, list(range(1, 71)), 2, True, 1),
    "tiles": ([257], [1000], 9, True, 0),
    "long": ([700], [1500], 2, True, 0),
    # long key ranges and few queries: blocks are shared by several workgroups
    "tiles_split": ([1, 130, 0, 70, 5], [9000, 4000, 3000, 64, 2], 3, True, 2),
    "tiles_split_chunk": ([1000], [4100], 2, True, 0),
    "tiles_split_not_causal": ([33, 200], [5000, 1000], 2, False, 0),
    "tiles_split_one": ([1], [20001], 1, True, 0),
}


@pytest.mark.parametrize("name", sorted(EXPANDED))
def test_expanded(lib, dev, name):
    import torch
    nq, nk, H, causal, pad = EXPANDED[name]
    rng = np.random.default_rng(sorted(EXPANDED).index(name) + 50)
    qs, ks = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    T, K = qs[-1] + pad, ks[-1] + pad
    q, qh = _bf(rng, (T, H + 1, 200), dev)
    q, qh = q[:, :H, 8:], qh[:, :H, 8:]
    kv, kvh = _bf(rng, (K, H, 264), dev)
    kv, kvh = kv[:, :, :256], kvh[:, :, :256]
    rope, rh = _bf(rng, (K, 80), dev)
    rope, rh = rope[:, 16:], rh[:, 16:]
    if pad:
        kv[ks[-1]:], rope[ks[-1]:] = float("nan"), float("nan")
    out = torch.full((T, H, 128), float(GUARD), dtype=torch.bfloat16, device=dev)
    lse = torch.full((T, H), float(GUARD), dtype=torch.float32, device=dev)
    note(f"expanded {name}")
    lib.latent_attention_expanded(q, kv, rope, _i32(qs, dev), _i32(ks, dev), 0.09, causal=causal, out=out, lse=lse)
    out, lse = _host(out), _host(lse)
    assert (out[qs[-1]:] == GUARD).all() and (lse[qs[-1]:] == GUARD).all()
    for b in range(len(nq)):
        rows = range(nq[b]) if nq[b] <= 64 else sorted({0, 1, 31, 32, 63, 64, 127, 128, nq[b] // 2, nq[b] - 2, nq[b] - 1} & set(range(nq[b])))
        for i in rows:
            n = lo.causal_keys(i, nq[b], nk[b], causal)
            for h in range(H):
                up = kvh[ks[b]:ks[b] + n, h]
                keys = np.concatenate([up[:, :128], rh[ks[b]:ks[b] + n]], 1)
                a = lo.attend(qh[qs[b] + i, h], keys, up[:, 128:], 0.09)
                for err in (lo.check(f"{b} {i} {h} out", out[qs[b] + i, h], a.out, a.out_bound),
                            lo.check(f"{b} {i} {h} lse", lse[qs[b] + i, h], a.lse, a.lse_bound)):
                    assert err is None, err


@pytest.mark.parametrize("nq,nk", [(70, 333), (40, 4500)])      # one workgroup to a block, and several
@pytest.mark.parametrize("scale", [4.0, -1.0, 0.0])
def test_expanded_scales(lib, dev, nq, nk, scale):
    """Scores of hundreds, the largest products last, of both signs, and none."""
    rng = np.random.default_rng(62)
    q, qh = _bf(rng, (nq, 2, 192), dev)
    kv, kvh = _bf(rng, (nk, 2, 256), dev)
    rope, rh = _bf(rng, (nk, 64), dev)
    order = np.argsort(np.concatenate([kvh[:, 0, :128], rh], 1) @ qh[nq - 1, 0])
    at = _i32(order, dev).long()
    kv, rope, kvh, rh = kv[at].contiguous(), rope[at].contiguous(), kvh[order], rh[order]
    out, lse = lib.latent_attention_expanded(q, kv, rope, _i32([0, nq], dev), _i32([0, nk], dev), scale)
    out, lse = _host(out), _host(lse)
    for i in (0, 31, nq - 1):
        n = lo.causal_keys(i, nq, nk, True)
        for h in range(2):
            a = lo.attend(qh[i, h], np.concatenate([kvh[:n, h, :128], rh[:n]], 1), kvh[:n, h, 128:], scale)
            for err in (lo.check(f"{i} {h} out", out[i, h], a.out, a.out_bound), lo.check(f"{i} {h} lse", lse[i, h], a.lse, a.lse_bound)):
                assert err is None, err


def test_expanded_split_over_many_requests(lib, dev):
    """300 requests of one query and 2000 to 2200 keys; one key row (stride 0)
    serves all, so weights come from the rotary part."""
    import torch
    rng = np.random.default_rng(61)
    B = 300
    nk = 2000 + rng.integers(0, 200, B)
    nk[7], nk[8] = 0, 3000
    ks = np.concatenate([[0], np.cumsum(nk)])
    K = int(ks[-1])
    assert K >= 2048 * B
    q, qh = _bf(rng, (B, 1, 192), dev)
    row, rowh = _bf(rng, (1, 1, 256), dev)
    rope, rh = _bf(rng, (K, 64), dev)
    out, lse = lib.latent_attention_expanded(q, row.expand(K, 1, 256), rope, _i32(range(B + 1), dev), _i32(ks, dev), 0.2)
    out, lse = _host(out), _host(lse)
    for b in list(range(0, B, 23)) + [7, 8, B - 1]:
        n = int(nk[b])
        keys = np.concatenate([np.repeat(rowh[0, :, :128], n, 0), rh[ks[b]:ks[b] + n]], 1)
        a = lo.attend(qh[b, 0], keys, np.repeat(rowh[0, :, 128:], n, 0), 0.2)
        for err in (lo.check(f"{b} out", out[b, 0], a.out, a.out_bound), lo.check(f"{b} lse", lse[b, 0], a.lse, a.lse_bound)):
            assert err is None, err


def test_expanded_small_workspace_is_refused(lib, dev):
    import ctypes

    import torch
    n = ctypes.c_size_t(0)
    handle = lib.load()
    assert handle.latent_attention_expanded_workspace(1, 2, 9000, 1, ctypes.byref(n)) == 0 and n.value > 0
    x = torch.zeros((9000, 2, 256), dtype=torch.bfloat16, device=dev)
    starts, ends = _i32([0, 1], dev), _i32([0, 9000], dev)
    out = torch.full((1, 2, 128), float(GUARD), dtype=torch.bfloat16, device=dev)
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    for w, b in ((None, 0), (ws.data_ptr(), n.value - 1), (ws.data_ptr() + 8, n.value)):
        assert handle.latent_attention_expanded(x.data_ptr(), 384, 192, x.data_ptr(), 512, 256, x.data_ptr(), 64,
                                                starts.data_ptr(), ends.data_ptr(), 0.1, 1, out.data_ptr(), None, w, b,
                                                torch.cuda.current_stream().cuda_stream, 1, 9000, 2, 1) == 1
    torch.cuda.synchronize()
    assert (out == GUARD).all()


def test_expanded_not_finite_where_masked(lib, dev):
    """Keys and values that hold NaN or an infinity reach the queries that
    attend them and no other, also those of the same tile."""
    import torch
    rng = np.random.default_rng(60)
    n, H = 200, 2
    q, qh = _bf(rng, (n, H, 192), dev)
    kv, kvh = _bf(rng, (n, H, 256), dev)
    rope, rh = _bf(rng, (n, 64), dev)
    kv[100, 0, 130] = float("inf")          # head 0: a value column
    kv[150, 0, 3] = float("nan")            # head 0: a key
    rope[180, 5] = float("nan")             # every head's key
    out, lse = lib.latent_attention_expanded(q, kv, rope, _i32([0, n], dev), _i32([0, n], dev), 0.1)
    out, lse = _host(out), _host(lse)
    assert np.isfinite(lse[:150]).all() and np.isfinite(out[:100]).all() and np.isfinite(out[:180, 1]).all()
    assert np.isposinf(out[100:150, 0, 2]).all() and np.isfinite(np.delete(out[:150, 0], 2, axis=1)).all()
    assert np.isnan(out[150:, 0]).all() and np.isnan(out[180:, 1]).all() and np.isfinite(lse[:180, 1]).all()
    for i in (0, 63, 64, 99, 149):
        for h in range(H):
            v = kvh[:i + 1, h, 128:].copy()
            a = lo.attend(qh[i, h], np.concatenate([kvh[:i + 1, h, :128], rh[:i + 1]], 1), v, 0.1)
            keep = np.arange(128) != 2 if (h == 0 and i >= 100) else np.ones(128, bool)
            assert lo.check("out", out[i, h][keep], a.out[keep], a.out_bound[keep]) is None
            assert lo.check("lse", lse[i, h], a.lse, a.lse_bound) is None


# ---- together, captured, on other streams ------------------------------------------------------------------

def _forms_agree(lib, dev, stream=None):
    """A prompt through plan, store, load and both forms of attention, then a
    decode step over the slots that topk_transform selects: returns outputs."""
    import torch
    rng = np.random.default_rng(77)
    ps, H = 16, 4
    cache = Cache(rng, 40 * ps, False, dev)
    table = torch.full((2, 20), -1, dtype=torch.int32, device=dev)
    free = _i32(rng.permutation(40), dev)
    wk, wkh = _bf(rng, (H, 128, 512), dev, 512 ** -0.5)
    wv, wvh = _bf(rng, (H, 128, 512), dev, 512 ** -0.5)
    steps = [[37, 150], [1, 1]]
    held, used, results = _i32([0, 0], dev), None, []
    for new in steps:
        plan = lib.paged_append_plan(held, _i32(new, dev), table, free, ps, sum(new), free_used=used, stream=stream)
        kv, _ = _bf(rng, (sum(new), 576), dev)
        lib.latent_cache_store(kv, plan.slot_map, cache.latent, cache.rope, stream=stream)
        held, used = plan.seq_lens, plan.free_used
        qn, _ = _bf(rng, (sum(new), H, 128), dev)
        qr, _ = _bf(rng, (sum(new), H, 64), dev)
        qc = torch.stack([qn[:, h].float() @ wk[h].float() for h in range(H)], 1)
        q = torch.cat([qc.bfloat16(), qr], 2)
        results.append((plan, kv, qn, qr, q))
    return cache, table, wk, wv, results


def test_forms_together(lib, dev):
    """The absorbed form over the page table, over selected slots (all of them)
    and the expanded form over the loaded cache agree within their bounds: same
    rows, three ways.  topk_transform's slots feed latent_attention as they are."""
    import torch
    cache, table, wk, wv, results = _forms_agree(lib, dev)
    plan, kv, qn, qr, q = results[-1]      # the decode step: one token a request
    ps, H, scale = 16, 4, 192 ** -0.5
    lens = plan.seq_lens.cpu().tolist()
    assert lens == [38, 151]
    out_p, lse_p = lib.latent_attention_paged(q, cache.latent, cache.rope, table, plan.seq_lens, plan.q_starts, ps, scale)
    scores = torch.from_numpy(np.random.default_rng(4).standard_normal((2, 320)).astype(np.float32)).to(dev)
    slots, _ = lib.topk_transform(scores, plan.seq_lens, table, 160, ps)
    out_s, lse_s = lib.latent_attention(q, cache.latent, cache.rope, slots, scale)
    c, r, qh = _host(cache.latent), _host(cache.rope), _host(q)
    starts = _i32(np.concatenate([[0], np.cumsum(lens)]), dev)
    lat, rope = lib.latent_cache_load_paged(table, starts, ps, sum(lens), cache.latent, cache.rope)
    up = torch.cat([torch.stack([lat.float() @ w[h].float().T for h in range(H)], 1) for w in (wk, wv)], 2).bfloat16()
    out_e, lse_e = lib.latent_attention_expanded(torch.cat([qn, qr], 2), up, rope, plan.q_starts, starts, scale)
    for b in range(2):
        s = lo.page_slots(table[b].cpu().numpy(), ps, lens[b], cache.slots)
        assert set(slots[b].cpu().tolist()) - {-1} == set(s.tolist())
        np.testing.assert_array_equal(_host(lat)[sum(lens[:b]):sum(lens[:b + 1])], c[s])
        for h in range(H):
            a = lo.attend(qh[b, h], np.concatenate([c[s], r[s]], 1), c[s], scale)
            for out, lse in ((out_p, lse_p), (out_s, lse_s)):
                assert lo.check("out", _host(out)[b, h], a.out, a.out_bound) is None
                assert lo.check("lse", _host(lse)[b, h], a.lse, a.lse_bound) is None
            # the expanded form's own rows, and the two forms against each other: bf16 keys,
            # values and absorbed queries differ by half a step each
            uh = _host(up)[sum(lens[:b]):sum(lens[:b + 1]), h]
            e = lo.attend(np.concatenate([_host(qn)[b, h], _host(qr)[b, h]]), np.concatenate([uh[:, :128], r[s]], 1), uh[:, 128:], scale)
            assert lo.check("out", _host(out_e)[b, h], e.out, e.out_bound) is None
            assert lo.check("lse", _host(lse_e)[b, h], e.lse, e.lse_bound) is None
            through = a.out @ _host(wv)[h].T
            dz = scale * lo.U16 * 2 * (np.abs(uh[:, :128]) @ np.abs(_host(qn)[b, h]) + np.abs(c[s]) @ np.abs(qh[b, h, :512])).max()
            assert np.abs(through - e.out).max() <= (2 * dz + 2 * lo.U16) * np.abs(uh[:, 128:]).max()


def _attend_all(lib, x, out=None, stream=None):
    """The three attention calls on prepared inputs."""
    o = out or [(None, None)] * 3
    a = lib.latent_attention(x["q"], x["cache"].latent, x["cache"].rope, x["idx"], 0.1, scale=x["cache"].scale, out=o[0][0], lse=o[0][1], stream=stream)
    b = lib.latent_attention_paged(x["q"], x["cache"].latent, x["cache"].rope, x["table"], x["lens"], x["starts"], 16, 0.1,
                                   scale=x["cache"].scale, out=o[1][0], lse=o[1][1], stream=stream)
    c = lib.latent_attention_expanded(x["qe"], x["kv"], x["rope"], x["starts"], x["ks"], 0.1, out=o[2][0], lse=o[2][1], stream=stream)
    return [a, b, c]


def _prepared(seed, dev, e4m3):
    rng = np.random.default_rng(seed)
    B, H = 3, 40
    lens = np.array([700, 33, 450])
    cache = Cache(rng, 16 * 140, e4m3, dev)
    x = dict(cache=cache, q=_bf(rng, (B, H, 576), dev)[0], idx=_i32(rng.integers(-1, cache.slots, (B, 600)), dev),
             table=_i32(rng.permutation(140)[:132].reshape(3, 44), dev), lens=_i32(lens, dev),
             starts=_i32(np.arange(B + 1), dev), qe=_bf(rng, (B, H, 192), dev)[0], kv=_bf(rng, (90, H, 256), dev)[0],
             rope=_bf(rng, (90, 64), dev)[0], ks=_i32([0, 30, 31, 90], dev))
    return x


@pytest.mark.parametrize("e4m3", [False, True])
def test_captured(lib, dev, e4m3):
    """Captured once with the store in front, replayed on new inputs with eager
    work and synchronisations between: each replay equals the eager result bit
    for bit (no atomics, a fixed order of sums)."""
    import torch
    x = _prepared(1, dev, e4m3)
    want0 = _attend_all(lib, x)
    rng = np.random.default_rng(2)
    kv, slot_map = _bf(rng, (5, 576), dev)[0], _i32([3, 900, -1, 17, 2000], dev)
    held, new, table, free = _i32([5, 0], dev), _i32([2, 9], dev), torch.zeros((2, 4), dtype=torch.int32, device=dev), _i32(range(20), dev)
    store = lambda: lib.latent_cache_store(kv, slot_map, x["cache"].latent, x["cache"].rope, scale=x["cache"].scale)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = lib.paged_append_plan(held, new, table, free, 4, 16)
        store()
        got = _attend_all(lib, x)
        back = lib.latent_cache_load(slot_map, x["cache"].latent, x["cache"].rope, scale=x["cache"].scale)
    for rep in range(4):
        kv.copy_(_bf(rng, (5, 576), dev)[0])
        x["q"].copy_(_bf(rng, tuple(x["q"].shape), dev)[0])
        new.copy_(_i32([rep, 9 - rep], dev))
        x["cache"].latent[3] = 0
        graph.replay()
        torch.cuda.synchronize()
        got_copy = [(o.clone(), l.clone()) for o, l in got]
        back_copy, plan_copy = [t.clone() for t in back], [t.clone() for t in plan]
        want = _attend_all(lib, x)
        store()
        want_back = lib.latent_cache_load(slot_map, x["cache"].latent, x["cache"].rope, scale=x["cache"].scale)
        want_plan = lib.paged_append_plan(held, new, table.clone(), free, 4, 16)
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got_copy, want):
            assert torch.equal(o, wo) and torch.equal(l, wl), rep
        for a, b in zip((*back_copy, *plan_copy), (*want_back, *want_plan)):
            assert torch.equal(a, b), rep
    assert not torch.equal(want0[0][0], want[0][0])


def test_streams(lib, dev):
    """Calls on two streams at once, and on a stream that is not the current
    one, give the current stream's results."""
    import torch
    xs = [_prepared(s, dev, s % 2 == 1) for s in (11, 12)]
    want = [_attend_all(lib, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(5):
        got = [None, None]
        for _ in range(3):
            for i in (0, 1):
                got[i] = _attend_all(lib, xs[i], stream=streams[i])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for (o, l), (wo, wl) in zip(g, w):
                assert torch.equal(o, wo) and torch.equal(l, wl)


def test_two_graphs_do_not_share(lib, dev):
    """Two graphs captured one after the other on one stream, replayed at once on
    two streams: each has its own workspace."""
    import torch
    xs = [_prepared(s, dev, False) for s in (21, 22)]
    want = [_attend_all(lib, x) for x in xs]
    graphs, got = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(_attend_all(lib, x))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for (o, l), (wo, wl) in zip(g, w):
                assert torch.equal(o, wo) and torch.equal(l, wl)


def test_small_workspace_is_refused(lib, dev):
    import ctypes
    import torch
    x = _prepared(3, dev, False)
    n = ctypes.c_size_t(0)
    L = lib.load()
    assert L.latent_attention_workspace(3, 40, 600, ctypes.byref(n)) == 0 and n.value > 0
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    out = torch.full((3, 40, 512), float(GUARD), dtype=torch.bfloat16, device=dev)

    def call(ptr, size):
        c = x["cache"]
        return L.latent_attention(x["q"].data_ptr(), 40 * 576, 576, c.latent.data_ptr(), 512, c.rope.data_ptr(), 64, None, 0,
                                  x["idx"].data_ptr(), 0.1, out.data_ptr(), None, ptr, size,
                                  torch.cuda.current_stream().cuda_stream, 3, 40, 600, c.slots)

    assert call(ws.data_ptr(), n.value - 1) == 1 and call(None, 0) == 1 and call(ws.data_ptr() + 4, n.value) == 1
    torch.cuda.synchronize()
    assert bool((out == GUARD).all())
    assert call(ws.data_ptr(), n.value) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, lib.latent_attention(x["q"], x["cache"].latent, x["cache"].rope, x["idx"], 0.1)[0])


# ---- attended keys that are not finite ----------------------------------------------------------------------

# tokens, heads, keys: one workgroup a token; whole tokens shared among workgroups; parts joined by the second launch
SHAPES = {"own": (350, 8, 70), "shared": (5, 24, 90), "joined": (5, 40, 2000)}


def _both_absorbed(lib, dev, cache, q, idx, scale):
    """The absorbed form over the slots of idx, by list and as pages of one slot."""
    T, k = idx.shape
    yield "selected", *lib.latent_attention(q, cache.latent, cache.rope, _i32(idx, dev), scale, scale=cache.scale)
    yield "paged", *lib.latent_attention_paged(q, cache.latent, cache.rope, _i32(idx, dev), _i32([k] * T, dev),
                                               _i32(range(T + 1), dev), 1, scale, scale=cache.scale)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_absorbed_not_finite(lib, dev, e4m3, shape):
    """A NaN, or a score of +inf, among a token's keys makes out and lse NaN,
    not the zeros and -inf of a token without keys; a score of -inf weighs
    nothing.  Other tokens are as they would be without."""
    T, H, k = SHAPES[shape]
    rng = np.random.default_rng(31)
    cache = Cache(rng, 3000, e4m3, dev)
    q, qh = _bf(rng, (T, H, 576), dev)
    q[:, :, 512 + 9], q[:, :, 512 + 11] = 1, -1
    qh[:, :, 512 + 9], qh[:, :, 512 + 11] = 1, -1
    cache.rope[0, 5] = float("nan")
    if e4m3:
        cache.scale[1] = float("nan")
    else:
        cache.latent[1, 7] = float("nan")
    cache.rope[2, 9] = float("inf")
    cache.rope[3, 11] = float("inf")          # a score of -inf
    idx = np.stack([4 + rng.permutation(2996)[:k] for _ in range(T)])
    kind = np.arange(T) % 5                   # 0: no such key; 1 to 4: the slot before it
    for t in np.nonzero(kind)[0]:
        idx[t, rng.integers(k)] = kind[t] - 1
    for form, out, lse in _both_absorbed(lib, dev, cache, q, idx, 0.07):
        out, lse = _host(out), _host(lse)
        bad = (kind >= 1) & (kind <= 3)
        assert np.isnan(out[bad]).all() and np.isnan(lse[bad]).all(), form
        for t in np.nonzero(~bad)[0][:8]:
            _check_token(f"{form} token {t}", cache, qh[t], idx[t][idx[t] > 3], 0.07, out[t], lse[t], heads=(0, H // 2, H - 1))


@pytest.mark.parametrize("nq,nk", [(70, 333), (40, 4500)])      # one workgroup to a block, and several
def test_expanded_not_finite(lib, dev, nq, nk):
    """The same for the expanded form, query by query."""
    rng = np.random.default_rng(32)
    q, qh = _bf(rng, (nq, 2, 192), dev)
    q[:, :, 128 + 5], q[:, :, 128 + 7] = 1, -1
    qh[:, :, 128 + 5], qh[:, :, 128 + 7] = 1, -1
    kv, kvh = _bf(rng, (nk, 2, 256), dev)
    rope, rh = _bf(rng, (nk, 64), dev)
    rope[2, 7] = float("inf")                       # a score of -inf
    kv[nk - nq + 10, 0, 3] = float("nan")           # head 0, from query 10 on
    rope[nk - nq + 20, 5] = float("inf")            # a score of +inf, from query 20 on
    out, lse = lib.latent_attention_expanded(q, kv, rope, _i32([0, nq], dev), _i32([0, nk], dev), 0.1)
    out, lse = _host(out), _host(lse)
    for h, first in ((0, 10), (1, 20)):
        assert np.isnan(out[first:, h]).all() and np.isnan(lse[first:, h]).all()
        for i in (0, 5, first - 1):
            at = np.setdiff1d(np.arange(lo.causal_keys(i, nq, nk)), [2])
            a = lo.attend(qh[i, h], np.concatenate([kvh[at, h, :128], rh[at]], 1), kvh[at, h, 128:], 0.1)
            assert lo.check("out", out[i, h], a.out, a.out_bound) is None
            assert lo.check("lse", lse[i, h], a.lse, a.lse_bound) is None


# ---- scores of any finite size ------------------------------------------------------------------------------

def _size(t, h):
    """Of a score's unit: powers of two up to 2^118, of both signs."""
    a = (10, 22, 27, 31, 33, 40, 60, 100, 110, 118)[(t + 3 * h) % 10]
    return (-1.0) ** (t + h) * 2.0 ** a


def _check_largest(name, sizes, units, values, scale, out, lse):
    """Rows of scores scale * size * unit, whole units apart: the largest score's
    keys share all the weight.  out: their mean, rounded to bf16, as the weights
    and their products with a scale are; lse: fp32."""
    for at in np.ndindex(*sizes.shape):
        z = sizes[at] * units[at[0]]
        top = z == z.max()
        want = values[at][top].mean(0)
        size = np.abs(values[at][top]).mean(0)
        assert lo.check(f"{name} {at} out", out[at], want, lo.U16 * np.abs(want) + (lo.U16 * 1.01 + 64 * lo.U32) * size) is None
        want = scale * z.max() + np.log(top.sum())
        # a product of the scale, its conversion to and from base 2, a logarithm, a sum
        assert lo.check(f"{name} {at} lse", lse[at], want, 8 * lo.U32 * (abs(want) + abs(scale * z.max()) + 1)) is None


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_absorbed_scores_of_any_size(lib, dev, e4m3, shape):
    """Scores whose distance from the largest cannot be told within fp32 of their
    own size, or that all lie below any constant, still weigh at most 1."""
    import torch
    T, H, k = SHAPES[shape]
    rng = np.random.default_rng(33)
    cache = Cache(rng, 3000, e4m3, dev)
    units = rng.integers(2, 200, 3000)
    units[rng.permutation(3000)[:60]] = 200
    units[rng.permutation(3000)[:60]] = 1
    cache.rope[:, 5] = torch.from_numpy(units.astype(np.float32)).bfloat16().to(dev)
    sizes = np.array([[_size(t, h) for h in range(H)] for t in range(T)])
    q = torch.zeros((T, H, 576), dtype=torch.bfloat16, device=dev)
    q[:, :, 512 + 5] = torch.from_numpy(sizes).to(dev).bfloat16()
    idx = np.stack([rng.permutation(3000)[:k] for _ in range(T)])
    few = min(T, 10)
    for form, out, lse in _both_absorbed(lib, dev, cache, q, idx, 0.3):
        out, lse = _host(out), _host(lse)
        assert np.isfinite(out).all() and np.isfinite(lse).all(), form
        for t in range(few):
            for h in {0, 1, 2, H // 2, H - 1}:
                _check_largest(f"{form} token {t} head {h}", sizes[t:t + 1, h], units[idx[t]][None], cache.c[idx[t]][None], 0.3,
                               out[t:t + 1, h], lse[t:t + 1, h])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("nq,nk", [(70, 333), (40, 4500)])      # one workgroup to a block, and several
def test_expanded_scores_of_any_size(lib, dev, nq, nk, causal):
    import torch
    rng = np.random.default_rng(34)
    units = rng.integers(2, 200, nk)
    units[rng.permutation(nk)[:nk // 40]] = 200
    units[rng.permutation(nk)[:nk // 40]] = 1
    kv, kvh = _bf(rng, (nk, 3, 256), dev)
    rope = _bf(rng, (nk, 64), dev)[0]
    rope[:, 5] = torch.from_numpy(units.astype(np.float32)).bfloat16().to(dev)
    sizes = np.array([[_size(i, h) for h in range(3)] for i in range(nq)])
    q = torch.zeros((nq, 3, 192), dtype=torch.bfloat16, device=dev)
    q[:, :, 128 + 5] = torch.from_numpy(sizes).to(dev).bfloat16()
    out, lse = lib.latent_attention_expanded(q, kv, rope, _i32([0, nq], dev), _i32([0, nk], dev), 0.3, causal=causal)
    out, lse = _host(out), _host(lse)
    for i in range(nq):
        n = lo.causal_keys(i, nq, nk, causal)
        for h in range(3):
            _check_largest(f"query {i} head {h}", sizes[i:i + 1, h], units[None, :n], kvh[None, :n, h, 128:], 0.3, out[i:i + 1, h], lse[i:i + 1, h])


def test_expanded_many_keys_of_equal_weight(lib, dev):
    """131072 keys of weight 0.7 after one of weight 1, one workgroup to a block.
    The sum takes a tile of 64 keys at a time (32 to a lane), so 2048 additions
    to the running sum and 32 within a tile, each off by at most half a step,
    and 2 units for each weight; one addition a key would be off by 6e-4."""
    import torch
    K, H = 131072, 384
    rng = np.random.default_rng(35)
    q = torch.zeros((1, H, 192), dtype=torch.bfloat16, device=dev)
    q[:, :, 128] = 1
    row, rowh = _bf(rng, (1, H, 256), dev)
    rope = torch.zeros((K, 64), dtype=torch.bfloat16, device=dev)
    rope[1:, 0] = np.log(0.7)
    other = float(rope[1, 0])
    out, lse = lib.latent_attention_expanded(q, row.expand(K, H, 256), rope, _i32([0, 1], dev), _i32([0, K], dev), 1.0)
    want = np.log(1 + (K - 1) * np.exp(other))
    bound = (2048 + 32 + 4) * lo.U32 + 8 * lo.U32 * (1 + want)
    assert lo.check("lse", _host(lse)[0], np.full(H, want), bound) is None
    # every value is its head's row: weights and result rounded to bf16, the weighted sum of a tile at a time
    size = np.abs(rowh[0, :, 128:])
    assert lo.check("out", _host(out)[0], rowh[0, :, 128:], (2.02 * lo.U16 + 2 * K // 16 * lo.U32) * size) is None


def test_workspace_serves_smaller_calls(lib, dev):
    """A workspace of the size that is said for a step's largest call serves every
    call with fewer tokens and keys, also those that are split where the
    largest is not."""
    import ctypes

    import torch
    n = ctypes.c_size_t(0)
    L = lib.load()
    cache = Cache(np.random.default_rng(36), 64, False, dev)
    x = torch.zeros((600, 64, 576), dtype=torch.bfloat16, device=dev)
    idx = torch.zeros((600, 2048), dtype=torch.int32, device=dev)
    out = torch.empty((600, 64, 512), dtype=torch.bfloat16, device=dev)
    for H in (16, 32, 64):
        for T, k in ((512, 2048), (600, 700)):
            assert L.latent_attention_workspace(T, H, k, ctypes.byref(n)) == 0
            ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
            for t, kk in ((T, k), (300, k), (300, 64), (64, k), (5, 2 * k // 3), (1, k), (1, 1)):
                st = L.latent_attention(x.data_ptr(), 64 * 576, 576, cache.latent.data_ptr(), 512, cache.rope.data_ptr(), 64, None, 0,
                                        idx.data_ptr(), 0.1, out.data_ptr(), None, ws.data_ptr(), n.value,
                                        torch.cuda.current_stream().cuda_stream, t, H, kk, 64)
                assert st == 0, (H, T, k, t, kk, lib.topk_last_error())
            torch.cuda.synchronize()
    q_starts, kv_starts = _i32([0, 1, 2], dev), _i32([0, 2048, 6000], dev)
    kv = torch.zeros((6000, 64, 256), dtype=torch.bfloat16, device=dev)
    rope = torch.zeros((6000, 64), dtype=torch.bfloat16, device=dev)
    assert L.latent_attention_expanded_workspace(600, 64, 6000, 3, ctypes.byref(n)) == 0
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    for t, K, H, B in ((2, 6000, 64, 2), (2, 6000, 4, 2), (1, 2048, 64, 1), (600, 6000, 5, 2), (1, 1, 1, 1)):
        st = L.latent_attention_expanded(x.data_ptr(), 64 * 576, 192, kv.data_ptr(), 64 * 256, 256, rope.data_ptr(), 64, q_starts.data_ptr(),
                                         kv_starts.data_ptr(), 0.1, 1, out.data_ptr(), None, ws.data_ptr(), n.value,
                                         torch.cuda.current_stream().cuda_stream, t, K, H, B)
        assert st == 0, (t, K, H, B, lib.topk_last_error())
    torch.cuda.synchronize()


def test_store_more_tokens_than_a_launch_has_threads_for(lib, dev):
    """2^26 tokens, a wave each: 2^32 threads.  All but the ends are padding."""
    import torch
    T, ends = 2 ** 26 + 5, [0, 1, 2 ** 25 - 1, 2 ** 25, 2 ** 26 - 1, 2 ** 26, 2 ** 26 + 4]
    if torch.cuda.mem_get_info()[0] < 90e9:
        pytest.skip("needs 90 GB")
    rng = np.random.default_rng(37)
    small, _ = _bf(rng, (len(ends), 576), dev)
    at = torch.tensor(ends, device=dev)
    kv = torch.empty((T, 576), dtype=torch.bfloat16, device=dev)
    kv[at] = small
    slot_map = torch.full((T,), -1, dtype=torch.int32, device=dev)
    slot_map[at] = torch.arange(len(ends), dtype=torch.int32, device=dev)
    positions = torch.zeros(T, dtype=torch.int32, device=dev)
    positions[at] = torch.arange(len(ends), dtype=torch.int32, device=dev)
    cos_sin = torch.randn((len(ends), 64), device=dev)
    whole, few = ([torch.zeros((len(ends) + 1, n), dtype=torch.bfloat16, device=dev) for n in (512, 64)] for _ in range(2))
    lib.latent_cache_store(kv, slot_map, *whole, positions=positions, cos_sin=cos_sin)
    lib.latent_cache_store(small, slot_map[at], *few, positions=positions[at], cos_sin=cos_sin)
    torch.cuda.synchronize()
    assert torch.equal(whole[0], few[0]) and torch.equal(whole[1], few[1]) and bool(few[0][:-1].any(1).all())
    del kv, slot_map, positions
    torch.cuda.empty_cache()


@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_scale_of_zero(lib, dev, shape):
    """With scale 0 every key weighs the same, however large its product, and
    masked ones still nothing."""
    import torch
    T, H, k = SHAPES[shape]
    rng = np.random.default_rng(38)
    cache = Cache(rng, 3000, False, dev)
    q, _ = _bf(rng, (T, H, 576), dev)
    q[:, :, 512 + 5] = 2.0 ** 110
    idx = np.stack([rng.permutation(3000)[:k] for _ in range(T)])
    idx[:, ::7] = -1
    n = int((idx[0] >= 0).sum())
    for form, out, lse in _both_absorbed(lib, dev, cache, q, idx, 0.0):
        out, lse = _host(out), _host(lse)
        assert (np.abs(lse - np.log(n)) <= 2.0 ** -20 + (2 * k + 8) * lo.U32).all(), form
        for t in range(min(T, 6)):
            rows = cache.c[idx[t][idx[t] >= 0]]
            bound = lo.U16 * np.abs(rows.mean(0)) + (4 * k * lo.U32 + 2.0 ** -18) * np.abs(rows).mean(0)
            for h in (0, H - 1):
                assert lo.check(f"{form} token {t}", out[t, h], rows.mean(0), bound) is None
    kv, kvh = _bf(rng, (k, 2, 256), dev)
    rope = _bf(rng, (k, 64), dev)[0]
    qe = q[:3, :2, :192].contiguous()
    qe[:, :, 128 + 5] = 2.0 ** 110
    out, lse = lib.latent_attention_expanded(qe, kv, rope, _i32([0, 3], dev), _i32([0, k], dev), 0.0)
    for i in range(3):
        v = kvh[:k - 2 + i, :, 128:]
        assert (np.abs(_host(lse)[i] - np.log(len(v))) <= 2.0 ** -20 + (2 * k + 8) * lo.U32).all()
        bound = lo.U16 * np.abs(v.mean(0)) + (4 * k * lo.U32 + 2.0 ** -18) * np.abs(v).mean(0)
        assert lo.check(f"query {i}", _host(out)[i], v.mean(0), bound) is None


@pytest.mark.parametrize("e4m3", [False, True])
def test_norm_of_large_values(lib, dev, e4m3):
    """The norm of rows up to the largest bf16 numbers, whose squares do not fit fp32."""
    import torch
    rng = np.random.default_rng(71)
    sizes = [1e3, 1e15, 1e18, 2e19, 1e20, 1e30, 1e37, 1e38]
    kv = torch.from_numpy(np.clip(rng.standard_normal((len(sizes), 576)), -3, 3))
    kv[:, :512] *= torch.tensor(sizes, dtype=torch.float64)[:, None]
    kv = kv.bfloat16()
    kvh = kv.double().numpy()
    w, wh = _bf(rng, (512,), dev)
    cache = Cache(rng, 16, e4m3, dev)
    lib.latent_cache_store(kv.to(dev), _i32(range(len(sizes)), dev), cache.latent, cache.rope, scale=cache.scale, norm_weight=w,
                           eps=1e-6)
    latent = cache.latent.cpu()
    for t in range(len(sizes)):
        y = lo.normed(kvh[t, :512], wh, 1e-6)
        slack = lo.NORM_ERROR * np.abs(y)
        if e4m3:
            s = float(cache.scale[t])
            # as in the other tests of the store: half a step of the code, the norm's error, the quotient's and the product's
            err = lo.check(f"row {t}", lo.e4m3_value(latent[t].numpy()) * s, y, np.abs(y) * 2.0 ** -4 + 2.0 ** -10 * s + slack
                           + np.abs(y) * (lo.NORM_ERROR + 8 * lo.U32))
        else:
            err = lo.check(f"row {t}", latent[t].double().numpy(), y, lo.U16 * np.abs(y) * (1 + 2 * lo.NORM_ERROR) + slack)
        assert err is None, err
