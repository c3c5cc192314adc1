"""GPU tests of latent attention over sequences that share prefixes, against the
float64 oracle, through the binding.  The bounds are the oracle's."""
import numpy as np
import pytest

from gpu_util import note
from oracle import latent_oracle as lo
from test_gpu_latent import GUARD, Cache, _bf, _check_token, _host, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


CASES = {
    # requests' own lengths (new tokens included), new tokens, group starts, shared lengths, heads, page size, rows of padding
    "one": ([3], [1], [0, 1], [40], 4, 16, 0),
    "no_groups": ([5, 70, 33], [1, 1, 1], [0], [], 7, 16, 0),
    "decode": ([1, 31, 32, 33, 64, 65, 200, 2], [1] * 8, [0, 8], [100], 16, 16, 0),
    "groups": ([9, 1, 40, 7, 3, 100, 5, 2], [1] * 8, [1, 1, 4, 4, 7], [77, 130, 5, 64], 5, 16, 2),      # empty groups, requests of none
    "nothing_shared": ([9, 50, 40], [1, 1, 1], [0, 2, 3], [0, 33], 20, 16, 0),
    "several": ([40, 3, 100, 7, 2], [3, 2, 0, 7, 1], [0, 3, 5], [70, 200], 33, 16, 3),
    "no_keys": ([0, 0, 4], [1, 1, 1], [0, 2], [0], 3, 16, 0),
    "only_shared": ([0, 0, 6], [2, 1, 3], [0, 3], [90], 6, 16, 0),          # a prefix that reaches past the new tokens
    "page_1": ([70, 9, 30], [1, 2, 1], [0, 3], [45], 12, 1, 0),
    "page_64": ([70, 9, 300], [1, 2, 1], [0, 3], [1000], 24, 64, 0),
    "long": ([9, 40, 77], [1, 1, 2], [0, 3], [9001], 32, 64, 0),
    "long_own": ([5000, 40], [1, 1], [0, 2], [33], 32, 64, 0),
    "heads_128": ([50, 90, 3], [2, 1, 1], [0, 3], [150], 128, 64, 1),
    "prompts": ([300, 40, 100], [200, 0, 90], [0, 3], [130], 3, 16, 4),
    "wide_prompts": ([130, 70], [130, 70], [0, 2], [257], 40, 64, 0),
    "one_head": ([2 + i % 40 for i in range(200)], [1 + i % 2 for i in range(200)], [0, 50, 200], [300, 65], 1, 16, 0),
    "many": ([1 + i % 50 for i in range(700)], [1] * 700, list(range(0, 701, 2)), [3 * (i % 40) for i in range(350)], 2, 16, 3),
    "many_idle": ([20] * 1500, [1 if i in (0, 700, 1499) else 0 for i in range(1500)], [0, 1499, 1500], [64, 10], 8, 16, 0),
    "launches": ([4 + i % 9 for i in range(8500)], [1] * 8500, [0, 3000, 8500], [40, 100], 1, 16, 2),      # more tokens than a launch takes
    "launches_wide": ([1 + i % 30 for i in range(1000)], [1] * 1000, [0, 1000], [70], 128, 16, 0),
    "wider_prompts_in_two_launches": ([925, 40], [920, 30], [0, 2], [100], 128, 64, 1),      # of one request's tokens
}


class Batch:
    def __init__(self, name, e4m3, dev):
        own, new, starts, shared, H, ps, pad = CASES[name]
        self.rng = rng = np.random.default_rng(sorted(CASES).index(name))
        self.own, self.new, self.group_starts, self.shared, self.H, self.ps = own, new, starts, shared, H, ps
        B = self.B = len(own)
        self.group = np.full(B, -1)
        for g in range(len(shared)):
            self.group[starts[g]:starts[g + 1]] = g
        prefix = np.array([shared[g] if g >= 0 else 0 for g in self.group], np.int64)
        self.prefix, self.lens = prefix, prefix + np.asarray(own, np.int64)
        P = self.P = int(max(1, -(-self.lens.max() // ps))) + 1
        # every row has pages of its own, also where only the first request's are used
        pages = np.minimum(-(-self.lens // ps) + 1, P)
        order = 1 + rng.permutation(int(pages.sum()))
        self.table, at = np.full((B, P), -1, np.int64), 0
        for b in range(B):
            self.table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
        if name == "several":
            self.table[0, 1], self.table[2, 2], self.table[4, 13] = -1, 10 ** 6, -1    # pages that are not there
        self.cache = Cache(rng, (int(pages.sum()) + 1) * ps, e4m3, dev, joint=name == "several")
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.T = int(self.starts[-1]) + pad
        self.q, self.qh = _bf(rng, (self.T, H, 576), dev)
        self.dev = dev
        self.args = dict(page_table=_i32(self.table, dev), seq_lens=_i32(self.lens, dev), q_starts=_i32(self.starts, dev),
                         group_starts=_i32(starts, dev), shared_lens=_i32(shared, dev), page_size=ps)

    def slots(self, b, limit):
        """Slots that a token of request b attends whose positions end at limit."""
        n = int(self.prefix[b])
        first = self.table[self.group_starts[self.group[b]]] if self.group[b] >= 0 else self.table[b]
        pos = np.concatenate([np.arange(min(n, self.P * self.ps)), np.arange(n, max(n, min(limit, self.P * self.ps)))])
        row = np.where((pos < n)[:, None], first[None, :], self.table[b][None, :])
        page = row[np.arange(len(pos)), pos // self.ps] if len(pos) else np.zeros(0, np.int64)
        slot = page * self.ps + pos % self.ps
        return slot[(page >= 0) & (slot < self.cache.slots)]

    def run(self, lib, scale=0.08, **kw):
        return lib.latent_attention_shared(self.q, self.cache.latent, self.cache.rope, softmax_scale=scale, scale=self.cache.scale,
                                           **self.args, **kw)

    def tokens(self):
        for b in range(self.B) if self.B < 100 else sorted({0, 1, 2, 299, 300, self.B // 2, self.B - 1} & set(range(self.B)) | {700 % self.B, 910 % self.B, 8191 % self.B}):
            for i in range(self.new[b]) if self.new[b] < 100 else (0, 1, 33, self.new[b] - 1):
                yield b, i, int(self.starts[b]) + i, int(self.lens[b]) - self.new[b] + i + 1


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_shared(lib, dev, e4m3, name):
    import torch
    x = Batch(name, e4m3, dev)
    used = np.unique(np.concatenate([x.slots(b, int(x.lens[b])) for b in range(x.B) if x.new[b]]))
    # what nobody attends holds NaN: the other requests' copies of a prefix and the rest of last pages among it
    x.cache.poison(np.setdiff1d(np.arange(x.cache.slots), used))
    out = torch.full((x.T, x.H, 512), float(GUARD), dtype=torch.bfloat16, device=dev)
    lse = torch.full((x.T, x.H), float(GUARD), dtype=torch.float32, device=dev)
    note(f"shared e4m3={e4m3} {name} T={x.T} H={x.H}")
    x.run(lib, out=out, lse=lse)
    torch.cuda.synchronize()
    out, lse = _host(out), _host(lse)
    assert (out[x.starts[-1]:] == GUARD).all() and (lse[x.starts[-1]:] == GUARD).all()
    heads = None if x.H <= 12 else [0, x.H // 2, x.H - 1]
    for b, i, t, limit in x.tokens():
        _check_token(f"request {b} token {i}", x.cache, x.qh[t], x.slots(b, limit), 0.08, out[t], lse[t], heads)


@pytest.mark.parametrize("name", ["several", "prompts", "decode"])
@pytest.mark.parametrize("e4m3,what", [(False, "nan"), (False, "inf"), (True, "nan"), (True, "scale")])
def test_later_keys_that_are_not_finite(lib, dev, e4m3, name, what):
    """The last new token's row of a request holds a NaN or an infinity: the earlier
    tokens' results are as without it, its own are NaN (the request's alone)."""
    import torch
    x = Batch(name, e4m3, dev)
    clean = x.run(lib)
    hit = [b for b in range(x.B) if x.new[b] and x.own[b] and len(x.slots(b, int(x.lens[b])))]
    for b in hit:
        pos = int(x.lens[b]) - 1
        slot = int(x.table[b][pos // x.ps]) * x.ps + pos % x.ps
        if what == "scale":
            x.cache.scale[slot] = float("nan")
        elif what == "nan":
            x.cache.latent[slot, 100] = 0x7F if e4m3 else float("nan")
        else:
            x.cache.latent[slot, 100] = float("inf")
    note(f"not finite {what} e4m3={e4m3} {name}")
    out, lse = x.run(lib)
    torch.cuda.synchronize()
    for b in hit:
        a, z = int(x.starts[b]), int(x.starts[b + 1]) - 1
        if what != "inf":
            assert torch.equal(out[a:z], clean[0][a:z]) and torch.equal(lse[a:z], clean[1][a:z]), b
        # An infinite score moves the running reference of the 16 rows that a wave takes together, and weights
        # 2^(z - m) of another m are rounded elsewhere: to the oracle's bound, not bit by bit.
        for i, t in enumerate(range(a, z)):
            if i < 3 or t >= z - 3:
                _check_token(f"request {b} token {i}", x.cache, x.qh[t], x.slots(b, int(x.lens[b]) - x.new[b] + i + 1), 0.08,
                             _host(out[t]), _host(lse[t]), (0, x.H - 1))
        if what == "inf":
            # the score is +inf (NaN results) or -inf (the key weighs nothing): by head
            score = x.q[z, :, 100].float() * 0.08
            up = (score > 0).cpu()
            assert torch.isnan(out[z]).all(1).cpu()[up].all() and torch.isnan(lse[z]).cpu()[up].all()
            assert torch.isfinite(lse[z]).cpu()[~up].all()
        else:
            assert torch.isnan(out[z]).all() and torch.isnan(lse[z]).all(), b


@pytest.mark.parametrize("scale", [4.0, -1.0, 0.0])
def test_scales(lib, dev, scale):
    x = Batch("several", False, dev)
    out, lse = x.run(lib, scale)
    out, lse = _host(out), _host(lse)
    for b, i, t, limit in x.tokens():
        _check_token(f"scale {scale} request {b} token {i}", x.cache, x.qh[t], x.slots(b, limit), scale, out[t], lse[t], (0, 16, 32))


@pytest.mark.parametrize("e4m3", [False, True])
def test_shared_where_nothing_has_to_be(lib, dev, e4m3):
    """Requests whose rows of the page table agree on the prefix: what a call over
    whole sequences gives, to both's roundings; and lengths past the table's row are cut."""
    import torch
    rng = np.random.default_rng(4)
    B, ps, P, H, prefix = 6, 16, 40, 20, 256
    table = 1 + rng.permutation(B * P).reshape(B, P)
    table[:, :prefix // ps] = table[0, :prefix // ps]
    cache = Cache(rng, (B * P + 1) * ps, e4m3, dev)
    q, _ = _bf(rng, (B, H, 576), dev)
    lens = _i32([300, 257, 640, 1000, 256, 400], dev)       # one past the row, one without keys of its own
    args = (q, cache.latent, cache.rope, _i32(table, dev), lens, _i32(range(B + 1), dev))
    out, lse = lib.latent_attention_shared(*args, _i32([0, B], dev), _i32([prefix], dev), ps, 0.07, scale=cache.scale)
    want, wlse = lib.latent_attention_paged(*args, ps, 0.07, scale=cache.scale)
    # each is within the weights' (2^-8) and its own (2^-8) rounding of the same sums
    size = want.float().abs().amax(-1, keepdim=True)
    assert bool(((out.float() - want.float()).abs() <= 4 * 2.0 ** -8 * size).all())
    assert bool(((lse - wlse).abs() <= 1e-5 * (1 + wlse.abs())).all())
    whole, _ = lib.latent_attention_shared(*args, _i32([0, B], dev), _i32([10 ** 9], dev), ps, 0.07, scale=cache.scale)
    same, _ = lib.latent_attention_shared(*args, _i32([0, B], dev), _i32([P * ps], dev), ps, 0.07, scale=cache.scale)
    assert torch.equal(whole, same)


def test_strides_and_far_slots(lib, dev):
    """Queries in a larger buffer, slots whose bytes lie beyond 2^32."""
    import torch
    rng = np.random.default_rng(6)
    small = Cache(rng, 96, False, dev)
    slots, ps = 5_000_000, 32
    latent = torch.empty((slots, 512), dtype=torch.bfloat16, device=dev)
    rope = torch.empty((slots, 64), dtype=torch.bfloat16, device=dev)
    pages = np.array([slots // ps - 1, 140_000, slots // ps - 3])
    at = (pages[:, None] * ps + np.arange(ps)).reshape(-1)
    latent[torch.from_numpy(at).to(dev)], rope[torch.from_numpy(at).to(dev)] = small.latent, small.rope
    q, qh = _bf(rng, (2, 9, 600), dev)
    q, qh = q[:, 1:, :576], qh[:, 1:, :576]
    table = np.array([[pages[0], -1, -1], [0, pages[1], pages[2]]])     # the second reads its first page in the first's row
    out, lse = lib.latent_attention_shared(q, latent, rope, _i32(table, dev), _i32([32, 90], dev), _i32([0, 1, 2], dev),
                                           _i32([0, 2], dev), _i32([32], dev), ps, 0.1)
    _check_token("first", small, qh[0], np.arange(32), 0.1, _host(out)[0], _host(lse)[0])
    _check_token("second", small, qh[1], np.arange(90), 0.1, _host(out)[1], _host(lse)[1])


@pytest.mark.parametrize("slots,stride,rope_stride", [(70000, 65536, 32768), (300, 2 ** 24, 64), (300, 2 ** 24 + 16, 64), (2000, 512, 2 ** 20)])
def test_codes_in_wide_rows(lib, dev, slots, stride, rope_stride):
    """8-bit rows far apart, before and beyond the distance that offsets of 32 bits are used for."""
    import torch
    rng = np.random.default_rng(8)
    small, ps = Cache(rng, 96, True, dev), 16
    pages = np.array([slots // ps - 1, 2, slots // ps - 3, 0, 7, slots // ps - 2])
    at = torch.from_numpy((pages[:, None] * ps + np.arange(ps)).reshape(-1)).to(dev)
    latent = torch.empty((slots, stride), dtype=torch.uint8, device=dev)[:, :512]
    rope = torch.empty((slots, rope_stride), dtype=torch.bfloat16, device=dev)[:, :64]
    scale = torch.full((slots,), float("nan"), device=dev)
    latent[at], rope[at], scale[at] = small.latent, small.rope, small.scale
    q, qh = _bf(rng, (3, 20, 576), dev)
    table = np.array([[pages[0], pages[1], -1, -1, -1], [pages[0], pages[1], pages[2], pages[3], -1], [-1, -1, pages[4], pages[5], -1]])
    out, lse = lib.latent_attention_shared(q, latent, rope, _i32(table, dev), _i32([32, 64, 57], dev), _i32([0, 1, 2, 3], dev),
                                           _i32([0, 3], dev), _i32([27], dev), ps, 0.1, scale=scale)
    out, lse = _host(out), _host(lse)
    own = [np.arange(32), np.arange(64), np.r_[np.arange(27), 64:64 + 57 - 32]]      # the last one's second page is missing
    for b in range(3):
        _check_token(f"request {b}", small, qh[b], own[b], 0.1, out[b], lse[b], [0, 7, 19])


def test_captured_and_on_streams(lib, dev):
    """Replays on other inputs equal the eager result bit for bit (no atomics, a fixed
    order of sums); two graphs of one stream and calls on two streams share nothing."""
    import torch
    xs = [Batch("several", False, dev), Batch("groups", True, dev)]
    graphs, got = [], []
    for x in xs:
        x.run(lib)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(x.run(lib))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    rng = np.random.default_rng(1)
    for rep in range(4):
        for x in xs:
            x.q.copy_(_bf(rng, tuple(x.q.shape), dev)[0])
            x.args["seq_lens"].sub_(1 if rep == 2 else 0)
        want = [x.run(lib) for x in xs]
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        eager = [x.run(lib, stream=s) for _ in range(3) for x, s in zip(xs, streams)][-2:]
        torch.cuda.synchronize()
        for x, g, e, w in zip(xs, got, eager, want):
            n = int(x.starts[-1])
            for a, b, c in zip(g, e, w):
                assert torch.equal(a[:n], c[:n]) and torch.equal(b[:n], c[:n]), rep


def test_a_step_behind_a_prefix(lib, dev):
    """Plan, store and attention together: three requests branch off one cached
    prompt, whose pages they name but do not own."""
    import torch
    rng = np.random.default_rng(12)
    ps, prompt, H, B = 16, 100, 12, 3
    latent = torch.zeros((40 * ps, 512), dtype=torch.bfloat16, device=dev)
    rope = torch.zeros((40 * ps, 64), dtype=torch.bfloat16, device=dev)
    zero = lambda n: _i32([0] * n, dev)     # noqa: E731
    kv, kvh = _bf(rng, (prompt, 576), dev)
    table = torch.full((1, 10), -1, dtype=torch.int32, device=dev)
    free = _i32(rng.permutation(40), dev)
    plan = lib.paged_append_plan(zero(1), _i32([prompt], dev), table, free, ps, prompt)
    lib.latent_cache_store(kv, plan.slot_map, latent, rope)
    # the branches share the full pages and hold the rest of the prompt themselves
    shared = prompt // ps * ps
    tables = torch.full((B, 10), -1, dtype=torch.int32, device=dev)
    tables[:, :shared // ps] = table[:, :shared // ps]
    new = [5, 1, 9]
    rest = prompt - shared
    plan = lib.paged_append_plan(_i32([shared] * B, dev), _i32([rest + n for n in new], dev), tables, free, ps,
                                 B * rest + sum(new), free_used=plan.free_used)
    own, ownh = _bf(rng, (sum(new), 576), dev)
    rows, rowsh = [], []
    for b in range(B):
        a = sum(new[:b])
        rows += [kv[shared:], own[a:a + new[b]]]
        rowsh.append(np.concatenate([kvh, ownh[a:a + new[b]]]))
    lib.latent_cache_store(torch.cat(rows), plan.slot_map, latent, rope)
    q, qh = _bf(rng, (B * rest + sum(new), H, 576), dev)
    out, lse = lib.latent_attention_shared(q, latent, rope, tables, plan.seq_lens, plan.q_starts, _i32([0, B], dev),
                                           _i32([shared], dev), ps, 0.06)
    out, lse, t = _host(out), _host(lse), 0
    for b in range(B):
        for i in range(rest + new[b]):
            keys = rowsh[b][:shared + i + 1]
            for h in (0, 7, 11):
                a = lo.attend(qh[t, h], keys, keys[:, :512], 0.06)
                for err in (lo.check(f"{b} {i} {h}", out[t, h], a.out, a.out_bound), lo.check("lse", lse[t, h], a.lse, a.lse_bound)):
                    assert err is None, err
            t += 1


def test_refusals(lib, dev):
    import ctypes
    import torch
    x = Batch("groups", False, dev)
    for bad in (dict(group_starts=x.args["group_starts"][:-1].contiguous()), dict(shared_lens=x.args["shared_lens"].long()), dict(page_size=24),
                dict(seq_lens=x.args["seq_lens"][1:].contiguous()), dict(shared_lens=x.args["shared_lens"][None]),
                dict(group_starts=x.args["group_starts"].cpu()), dict(page_table=x.args["page_table"][0])):
        with pytest.raises(ValueError):
            lib.latent_attention_shared(x.q, x.cache.latent, x.cache.rope, softmax_scale=0.1, **{**x.args, **bad})
    with pytest.raises(ValueError):
        x.run(lib, out=torch.zeros((x.T, x.H, 511), dtype=torch.bfloat16, device=dev))
    n = ctypes.c_size_t(0)
    L = lib.load()
    assert L.latent_attention_shared_workspace(x.T, x.H, ctypes.byref(n)) == 0 and n.value > 0
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    out = torch.full((x.T, x.H, 512), float(GUARD), dtype=torch.bfloat16, device=dev)

    def call(ptr, size):
        c, a = x.cache, x.args
        return L.latent_attention_shared(x.q.data_ptr(), x.H * 576, 576, c.latent.data_ptr(), 512, c.rope.data_ptr(), 64, None, 0,
                                         a["page_table"].data_ptr(), a["seq_lens"].data_ptr(), a["q_starts"].data_ptr(),
                                         a["group_starts"].data_ptr(), a["shared_lens"].data_ptr(), x.ps, 0.08, out.data_ptr(), None,
                                         ptr, size, torch.cuda.current_stream().cuda_stream, x.T, x.H, x.B, len(x.shared), x.P, c.slots)

    assert call(ws.data_ptr(), n.value - 1) == 1 and call(None, 0) == 1 and call(ws.data_ptr() + 4, n.value) == 1
    torch.cuda.synchronize()
    assert bool((out == GUARD).all())
    assert call(ws.data_ptr(), n.value) == 0
    torch.cuda.synchronize()
    k = int(x.starts[-1])
    assert torch.equal(out[:k], x.run(lib)[0][:k])


def test_workspace_grows_with_tokens(lib, dev):
    import ctypes
    L, last = lib.load(), 0
    for t in (1, 7, 100, 900, 5000, 10 ** 6):
        n = ctypes.c_size_t(0)
        assert L.latent_attention_shared_workspace(t, 32, ctypes.byref(n)) == 0
        assert n.value >= last
        last = n.value
    assert last < 2 ** 30


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("prefix", [1, 32, 0])
def test_positions_up_to_the_last(lib, dev, e4m3, prefix):
    """A request of 2^31 - 1 positions, of which a few pages exist, at both ends.  Behind a prefix of one position its
    last tile reaches past 2^31; of its two tokens only the second attends the last position, which is not finite."""
    import torch
    rng = np.random.default_rng(14)
    ps, H, n = 1024, 16, 2 ** 31 - 1
    P = 2 ** 31 // ps
    cache = Cache(rng, 3 * ps, e4m3, dev)
    table = np.full((1, P), -1, np.int32)
    table[0, 0], table[0, P - 1] = 1, 2                    # slots 1024 to 2047, and from 2048 on
    last = 2 * ps + (n - 1) % ps                           # the last position's slot
    q, qh = _bf(rng, (2, H, 576), dev)
    note(f"far positions e4m3={e4m3} prefix={prefix}")
    args = (q, cache.latent, cache.rope, _i32(table, dev), _i32([n], dev), _i32([0, 2], dev), _i32([0, 1], dev),
            _i32([prefix], dev), ps, 0.05)
    out, lse = lib.latent_attention_shared(*args, scale=cache.scale)
    out, lse = _host(out), _host(lse)
    for i in range(2):
        _check_token(f"token {i}", cache, qh[i], np.arange(ps, last + i), 0.05, out[i], lse[i], (0, 7, 15))
    cache.poison([last])
    cache.poison(range(last + 1, 3 * ps))
    cache.poison(range(ps))
    out, lse = lib.latent_attention_shared(*args, scale=cache.scale)
    out, lse = _host(out), _host(lse)
    _check_token("before the last", cache, qh[0], np.arange(ps, last), 0.05, out[0], lse[0], (0, 7, 15))
    assert np.isnan(out[1]).all() and np.isnan(lse[1]).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("name", ["several", "prompts", "decode", "heads_128"])
def test_a_score_of_minus_infinity_weighs_nothing(lib, dev, e4m3, name):
    """An infinite value in the row of a request's last position, which some of its tokens attend, all, or one alone
    (bf16; an 8-bit row has it in its rotary part): heads whose score is -inf are as without the row, but for 0 times the infinity in
    its own element, whoever shares their tile; heads whose score is +inf are NaN, and tokens before it are as without."""
    import torch
    x = Batch(name, e4m3, dev)
    hit = [b for b in range(x.B) if x.new[b] and x.own[b] and len(x.slots(b, int(x.lens[b])))]
    column = 100
    for b in hit:
        pos = int(x.lens[b]) - 1
        slot = int(x.table[b][pos // x.ps]) * x.ps + pos % x.ps
        if e4m3:
            x.cache.rope[slot, 3] = float("inf")
        else:
            x.cache.latent[slot, column] = float("inf")
    note(f"minus infinity e4m3={e4m3} {name}")
    out, lse = x.run(lib)
    torch.cuda.synchronize()
    out, lse = _host(out), _host(lse)
    seen = 0
    for b in hit:
        n, first, z = int(x.lens[b]), int(x.starts[b]), int(x.starts[b + 1]) - 1
        up = x.qh[z, :, 515 if e4m3 else column] > 0
        assert np.isnan(out[z][up]).all() and np.isnan(lse[z][up]).all()
        heads = np.nonzero(~up)[0][:6]
        got = out[z].copy()
        if not e4m3:
            assert np.isnan(got[~up][:, column]).all()
        # the key's row counts for the weights of no head here; its own element is compared apart
        slots = x.slots(b, n - 1)
        for h in heads:
            keys = np.concatenate([x.cache.c[slots], x.cache.r[slots]], 1)
            a = lo.attend(x.qh[z, h], keys, x.cache.c[slots], 0.08)
            rest = np.ones(512, bool)
            rest[column] = e4m3
            for err in (lo.check(f"{b} {h} out", got[h, rest], a.out[rest], a.out_bound[rest]),
                        lo.check(f"{b} {h} lse", lse[z, h], a.lse, a.lse_bound)):
                assert err is None, err
            seen += 1
        for t in range(max(first, z - 3), z):
            _check_token(f"request {b} before", x.cache, x.qh[t], x.slots(b, n - (z - t)), 0.08, out[t], lse[t], (0, x.H - 1))
    assert seen > 0
    # and where nothing is shared, the results of the call over whole sequences
    none = dict(x.args, group_starts=_i32([0], dev), shared_lens=_i32([], dev))
    args = (x.q, x.cache.latent, x.cache.rope)
    a, al = lib.latent_attention_shared(*args, softmax_scale=0.08, scale=x.cache.scale, **none)
    none.pop("group_starts"), none.pop("shared_lens")
    w, wl = lib.latent_attention_paged(*args, softmax_scale=0.08, scale=x.cache.scale, **none)
    k = int(x.starts[-1])
    assert torch.equal(torch.isnan(a[:k]), torch.isnan(w[:k])) and torch.equal(torch.isnan(al[:k]), torch.isnan(wl[:k]))
    assert bool(torch.isnan(a[:k]).any())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,new,H,prefix,own", [(64, 1, 32, 7000, 900), (40, 3, 20, 12001, 333), (300, 1, 16, 2050, 60), (5, 2, 128, 20000, 4000)])
def test_many_tiles_to_a_workgroup(lib, dev, e4m3, B, new, H, prefix, own):
    """Parts of some tens of tiles, where the other cases have six at most: all tokens within the roundings of the call over
    whole sequences, which reads every request's own copy of the same page table, and some against the oracle."""
    import torch
    rng = np.random.default_rng(B)
    ps = 16
    lens = prefix + rng.integers(new, own + 1, B)
    shared = prefix // ps * ps
    pages = -(-lens // ps) - shared // ps
    total, P = shared // ps + int(pages.sum()), int((shared // ps + pages).max())
    order, at = rng.permutation(total), shared // ps
    table = np.full((B, P), -1, np.int64)
    for b in range(B):
        table[b, :shared // ps] = order[:shared // ps]
        table[b, shared // ps:shared // ps + pages[b]] = order[at:at + pages[b]]
        at += pages[b]
    cache = Cache(rng, total * ps, e4m3, dev)
    T = B * new
    q, qh = _bf(rng, (T, H, 576), dev)
    args = (q, cache.latent, cache.rope, _i32(table, dev), _i32(lens, dev), _i32(np.arange(B + 1) * new, dev))
    note(f"long parts e4m3={e4m3} B={B} H={H}")
    out, lse = lib.latent_attention_shared(*args, _i32([0, B], dev), _i32([shared], dev), ps, 0.06, scale=cache.scale)
    want, wlse = lib.latent_attention_paged(*args, ps, 0.06, scale=cache.scale)
    # a bf16 result's own rounding, and its weights', on either side (2^-8 each, of the row's largest element)
    size = want.float().abs().amax(-1, keepdim=True)
    assert bool(((out.float() - want.float()).abs() <= 4 * 2.0 ** -8 * size).all())
    assert bool(((lse - wlse).abs() <= 1e-5 * (1 + wlse.abs())).all())
    out, lse = _host(out), _host(lse)
    for b in sorted({0, B // 2, B - 1}):
        i = int(rng.integers(new))
        pos = np.arange(int(lens[b]) - new + i + 1)
        _check_token(f"request {b} token {i}", cache, qh[b * new + i], table[b][pos // ps] * ps + pos % ps, 0.06,
                     out[b * new + i], lse[b * new + i], (0, H // 2, H - 1))
