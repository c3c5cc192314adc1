"""The indexer's own cache and a batch's shared prefix: what each operator computes, on which sizes it is measured.

The append of index keys to their paged cache (norm, rotation, 8-bit codes), the indexer's queries in the same form, the
load of cached keys for the scan over a prompt, the scores of new tokens against the paged cache, and latent attention
for requests that share a long prefix.  `run` computes a case in plain torch operations, or, where `own` is set, through
the library's entry points.
"""
import math

import torch

own = False

HEADS = 32     # the indexer's heads
DIM = 128      # width of an index key, and of a head's query
TURNED = 64    # of these, the first that are rotated by position
LATENT = 512   # width of a token's latent vector
ROPE = 64      # width of its shared rotary key
E4M3_MAX = 448.0
EPS = 1e-6
FAR = 65536    # positions that the angles' table holds


# ---- the cases ------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 requests: a key each
        dict(name="keys_decode_64", op="keys", tokens=64, slots=16384, spare=0, hadamard=True, interleaved=False, wide=True),
        # a prompt chunk, some rows of the batch being padding
        dict(name="keys_prefill_16000", op="keys", tokens=16000, slots=65536, spare=37, hadamard=False, interleaved=True, wide=False),
        # the same decode step's queries, with the weights of their heads
        dict(name="queries_decode_64", op="queries", tokens=64, hadamard=True, interleaved=False, wide=False),
        # a whole prompt's
        dict(name="queries_prefill_8192", op="queries", tokens=8192, hadamard=True, interleaved=True, wide=True),
        # the cached keys of a few requests, in a row for the scan of a chunk
        dict(name="load_3", op="load", rows=5000, requests=3, page=16, slots=65536),
        # those of 16 long ones
        dict(name="load_16", op="load", rows=400000, requests=16, page=64, slots=524288),
        # one token of one request with a million cached ones
        dict(name="logits_decode_1", op="logits", requests=1, new_lo=1, new_hi=1, lo=1048576, hi=1048576, page=64),
        # one decode step of 64 requests, the benchmark's ragged lengths
        dict(name="logits_decode_64", op="logits", requests=64, new_lo=1, new_hi=1, lo=4096, hi=65536, page=64),
        # a prompt chunk: the last 1024 tokens of 65536
        dict(name="logits_chunk_1024", op="logits", requests=1, new_lo=1024, new_hi=1024, lo=65536, hi=65536, page=64),
        # a few answers to one question, as many heads as one GPU of several has
        dict(name="shared_decode_8", op="shared", requests=8, groups=1, new=1, shared_lo=4096, shared_hi=4096, lo=1, hi=300, heads=16, fp8=False, page=64),
        # one decode step of 64 requests behind one long document, each with a conversation of its own
        dict(name="shared_decode_64", op="shared", requests=64, groups=1, new=1, shared_lo=32768, shared_hi=32768, lo=100, hi=4000, heads=32, fp8=False, page=64),
        # two new tokens each of 150 requests behind five instructions of odd lengths, in an 8-bit cache
        dict(name="shared_groups_5", op="shared", requests=150, groups=5, new=2, shared_lo=1000, shared_hi=15000, lo=2, hi=1500, heads=20, fp8=True, page=16),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["keys", "queries", "load", "logits", "logits", "shared", "shared"])
    if op == "keys":
        tokens = _log_int(rng, 1, 16000)
        return dict(op=op, tokens=tokens, slots=tokens + _log_int(rng, 100, 49000), spare=rng.choice([0, 1, 5]), hadamard=rng.random() < 0.5, interleaved=rng.random() < 0.5, wide=rng.random() < 0.5)
    if op == "queries":
        return dict(op=op, tokens=_log_int(rng, 1, 8192), hadamard=rng.random() < 0.5, interleaved=rng.random() < 0.5, wide=rng.random() < 0.5)
    if op == "load":
        return dict(op=op, rows=_log_int(rng, 100, 400000), requests=_log_int(rng, 1, 60), page=rng.choice([1, 16, 64]), slots=524288)
    page = rng.choice([1, 16, 32, 64])
    if op == "logits":
        requests = _log_int(rng, 1, 200)
        new_hi = rng.choice([1, 1, 2, _log_int(rng, 1, max(1, 1000 // requests))])
        hi = _log_int(rng, max(16, 2 * new_hi), max(17, 2 * new_hi, min(1048576, 4000000 // requests, 60000000 // (requests * new_hi))))
        return dict(op=op, requests=requests, new_lo=rng.choice([0, 1]), new_hi=new_hi, lo=max(1, hi // 16), hi=hi, page=page)
    requests = _log_int(rng, 1, 200)
    groups = _log_int(rng, 1, min(8, requests))
    new = rng.choice([1, 1, 1, 2, 3])
    heads = rng.choice([1, 5, 8, 16, 20, 32, 64, 128])
    columns = requests * new * heads
    hi = _log_int(rng, 10, max(10, min(32768, 60000000 // columns)))
    own_hi = _log_int(rng, 10, max(10, min(4000, 8000000 // columns)))
    return dict(op=op, requests=requests, groups=groups, new=new, shared_lo=rng.choice([0, hi // 3]), shared_hi=hi, lo=new, hi=max(new, own_hi), heads=heads, fp8=rng.random() < 0.5, page=page)


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _even(lo, hi, n):
    """n lengths spread evenly from lo to hi: their sum is the case's own."""
    return torch.linspace(hi if n == 1 else lo, hi, n, device="cuda", dtype=torch.float64).long()


def _between(lo, hi, n, g):
    """The same in an order of the seed's."""
    return _even(lo, hi, n)[torch.randperm(n, generator=g, device="cuda")]


def _starts(lens):
    return torch.cat([lens.new_zeros(1), lens.cumsum(0)])


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _codes(shape, g):
    """8-bit codes of values as they are after scaling by a row's largest."""
    return (_normal(shape, g) * 112).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(n, g):
    return (torch.rand(n, generator=g, device="cuda") + 0.5) / 112


def _angles():
    """Cosines and sines of every position's angles."""
    angle = torch.arange(FAR, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, TURNED, 2, device="cuda", dtype=torch.float64) / TURNED)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _signs(dtype):
    """Hadamard's matrix of DIM rows, orthonormal: entry (i, j) is -1 to the number of ones that i and j have in common."""
    i = torch.arange(DIM, device="cuda")
    common = ((i[:, None] & i)[..., None] >> torch.arange(7, device="cuda") & 1).sum(-1)
    return (1 - 2 * (common % 2)).to(dtype) / math.sqrt(DIM)


def _pages(lens, page, g, kept=None, leader=None):
    """A page table over pages in random order, and the number of slots it spans; a request's first `kept` pages are those of `leader`."""
    need = (lens + page - 1) // page
    kept = torch.zeros_like(need) if kept is None else kept
    fresh = need - kept
    total, most = int(fresh.sum()), max(1, int(need.max()))
    order = torch.randperm(max(1, total), generator=g, device="cuda")
    col = torch.arange(most, device="cuda")
    at = _starts(fresh)[:-1, None] + col - kept[:, None]
    table = torch.where((col >= kept[:, None]) & (col < need[:, None]), order[at.clamp(0, max(0, total - 1))], -1)
    if leader is not None:
        table = torch.where(col < kept[:, None], table[leader], table)
    return table.int(), max(1, total) * page


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], dict(case)
    kind = torch.float32 if case.get("wide") else torch.bfloat16
    if op in ("keys", "queries"):
        n = case["tokens"]
        s.update(positions=torch.randint(0, FAR, (n,), generator=g, device="cuda").int(), cos_sin=_angles())
        if case["hadamard"]:
            s["signs"] = _signs(torch.float32)
    if op == "keys":
        slot_map = torch.randperm(case["slots"], generator=g, device="cuda")[:n].int()
        slot_map[n - case["spare"]:] = -1
        s.update(k=_normal((n, DIM), g) * 2 + 0.3, slot_map=slot_map, norm_weight=1 + 0.1 * _normal((DIM,), g, kind), norm_bias=0.1 * _normal((DIM,), g, kind),
                 keys=_codes((case["slots"], DIM), g), key_scale=_scales(case["slots"], g))
    elif op == "queries":
        s.update(q=_normal((n, HEADS, DIM), g) * 2, weights=_normal((n, HEADS), g, kind), weight_scale=(HEADS * DIM) ** -0.5)
    elif op == "load":
        lens = _between(0, 2 * case["rows"] // max(2, case["requests"]), case["requests"], g)
        s["page_table"], _ = _pages(lens, case["page"], g)
        s.update(keys=_codes((case["slots"], DIM), g), key_scale=_scales(case["slots"], g), kv_starts=_starts(lens).int(), num_rows=int(lens.sum()))
    elif op == "logits":
        new = _between(case["new_lo"], case["new_hi"], case["requests"], g)
        lens = torch.maximum(_between(case["lo"], case["hi"], case["requests"], g), new)
        s["page_table"], slots = _pages(lens, case["page"], g)
        n, width = int(new.sum()), s["page_table"].shape[1] * case["page"]
        s.update(q=_codes((n, HEADS, DIM), g), weights=_normal((n, HEADS), g, torch.float32) * 0.01, keys=_codes((slots, DIM), g), key_scale=_scales(slots, g),
                 seq_lens=lens.int(), q_starts=_starts(new).int(), most_new=case["new_hi"], out=torch.full((n, width), -math.inf, device="cuda"))
    else:
        b, groups, page = case["requests"], case["groups"], case["page"]
        # groups of different sizes, fixed by the case
        group_starts = (b * torch.linspace(0, 1, groups + 1, device="cuda", dtype=torch.float64) ** 1.5).round().long()
        shared = _even(case["shared_lo"], case["shared_hi"], groups)
        group = torch.searchsorted(group_starts[1:].contiguous(), torch.arange(b, device="cuda"), right=True)
        leader = group_starts[group]
        lens = shared[group] + _between(case["lo"], case["hi"], b, g).clamp_min(case["new"])
        kept = torch.where(leader == torch.arange(b, device="cuda"), 0, shared[group] // page)
        s["page_table"], slots = _pages(lens, page, g, kept, leader)
        tokens = b * case["new"]
        latent, s["scale"] = _normal((slots, LATENT), g), None
        if case["fp8"]:
            latent = (latent * 112).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
            s["scale"] = _scales(slots, g)
        s.update(latent=latent, rope=_normal((slots, ROPE), g), q=_normal((tokens, case["heads"], LATENT + ROPE), g), sm=(DIM + ROPE) ** -0.5,
                 seq_lens=lens.int(), q_starts=torch.arange(0, tokens + 1, case["new"], device="cuda", dtype=torch.int32),
                 group_starts=group_starts.int(), shared_lens=shared.int(), most_group=int(group_starts.diff().max()), most_shared=case["shared_hi"], most_own=int((lens - shared[group]).max()))
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_attention_indexer_fp32_amd as lib
    op = s["op"]
    if op == "keys":
        lib.indexer_cache_store(s["k"], s["slot_map"], s["keys"], s["key_scale"], norm_weight=s["norm_weight"], norm_bias=s["norm_bias"], eps=EPS,
                                positions=s["positions"], cos_sin=s["cos_sin"], interleaved=s["interleaved"], hadamard=s["hadamard"])
        return s["keys"].view(torch.float8_e4m3fn), s["key_scale"]
    if op == "queries":
        q, weights = lib.indexer_queries(s["q"], s["weights"], s["weight_scale"], positions=s["positions"], cos_sin=s["cos_sin"], interleaved=s["interleaved"], hadamard=s["hadamard"])
        return q.view(torch.float8_e4m3fn), weights
    if op == "load":
        keys, key_scale = lib.indexer_cache_load_paged(s["page_table"], s["kv_starts"], s["page"], s["num_rows"], s["keys"], s["key_scale"])
        return keys.view(torch.float8_e4m3fn), key_scale
    if op == "logits":
        return lib.indexer_logits_paged(s["q"], s["weights"], s["keys"], s["key_scale"], s["page_table"], s["seq_lens"], s["q_starts"], s["page"], out=s["out"])
    return lib.latent_attention_shared(s["q"], s["latent"], s["rope"], s["page_table"], s["seq_lens"], s["q_starts"], s["group_starts"], s["shared_lens"], s["page"], s["sm"], scale=s["scale"])


def _run_plain(s):
    return {"keys": _keys, "queries": _queries, "load": _load, "logits": _logits, "shared": _shared}[s["op"]](s)


def _turned(x, s, positions):
    """Rows whose first TURNED values are rotated by their position, then mixed."""
    cos, sin = s["cos_sin"][positions.long()].split(TURNED // 2, -1)
    cos, sin = (v.reshape(len(x), *[1] * (x.dim() - 2), TURNED // 2) for v in (cos, sin))
    r, rest = x[..., :TURNED], x[..., TURNED:]
    if s["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :TURNED // 2], r[..., TURNED // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    y = torch.cat([r, rest], -1)
    return y @ s["signs"] if s["hadamard"] else y


def _quantised(y):
    """8-bit codes of each row, and the row's scale."""
    scale = y.abs().amax(-1) / E4M3_MAX
    scale = torch.where(scale > 0, scale, 1.0)
    return (y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _keys(s):
    live = s["slot_map"] >= 0
    slot = s["slot_map"][live].long()
    x = s["k"][live].float()
    x = x - x.mean(1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["norm_weight"].float() + s["norm_bias"].float()
    codes, scale = _quantised(_turned(x, s, s["positions"][live]))
    s["keys"][slot] = codes.view(torch.uint8)
    s["key_scale"][slot] = scale
    return s["keys"].view(torch.float8_e4m3fn), s["key_scale"]


def _queries(s):
    codes, scale = _quantised(_turned(s["q"].float(), s, s["positions"]))
    return codes, s["weights"].float() * scale * s["weight_scale"]


def _owner(starts, n):
    """The request of each of n rows, and whether the row belongs to one."""
    t = torch.arange(n, device=starts.device, dtype=torch.int32)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    return t, b.clamp_max(len(starts) - 2), t < starts[-1]


def _load(s):
    t, b, live = _owner(s["kv_starts"], s["num_rows"])
    pos = t - s["kv_starts"][b]
    slot = (s["page_table"][b, (pos // s["page"]).long()] * s["page"] + pos % s["page"]).long()
    return s["keys"][slot].view(torch.float8_e4m3fn), s["key_scale"][slot]


def _logits(s):
    page, qs, lens = s["page"], s["q_starts"].long(), s["seq_lens"].long()
    width, n = s["page_table"].shape[1] * page, qs.diff()
    pos = torch.arange(width, device="cuda")
    slot = (s["page_table"][:, pos // page].long() * page + pos % page).clamp_min(0)
    i = torch.arange(s["most_new"], device="cuda")
    at = (qs[:-1, None] + i).clamp_max(len(s["q"]) - 1)
    q = s["q"].view(torch.float8_e4m3fn)[at].float()
    keys = s["keys"].view(torch.float8_e4m3fn)[slot].float()
    z = torch.bmm(q.flatten(1, 2), keys.mT).relu_().unflatten(1, (s["most_new"], HEADS))
    score = torch.matmul(s["weights"][at][:, :, None], z)[:, :, 0] * s["key_scale"][slot][:, None]
    most = lens[:, None] - n[:, None] + i + 1
    has = i < n[:, None]
    return torch.where(pos < most[..., None], score, -math.inf)[has], most[has].int()


def _rows(s, slot):
    """Cache rows of these slots as 32-bit values; a slot below zero gives zeros."""
    live, slot = (slot >= 0)[..., None], slot.clamp_min(0).long()
    c = s["latent"][slot]
    c = c.view(torch.float8_e4m3fn).float() * s["scale"][slot][..., None] if s["fp8"] else c.float()
    return torch.where(live, torch.cat([c, s["rope"][slot].float()], -1), 0.0)


def _part(s, q, rows, live):
    """Unscaled sums of one part of the keys, their largest score and the sum of their weights."""
    z = torch.where(live, s["sm"] * torch.bmm(q, rows.mT), -math.inf)
    top = z.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(z - top)
    return torch.bmm(p, rows[..., :LATENT]), top, p.sum(-1, keepdim=True)


def _shared(s):
    heads, new, page, b = s["heads"], s["new"], s["page"], s["requests"]
    starts, shared = s["group_starts"].long(), s["shared_lens"].long()
    group = torch.searchsorted(starts[1:].contiguous(), torch.arange(b, device="cuda"), right=True)
    q = s["q"].float()

    # the shared prefixes, each against all of its group's queries
    pos = torch.arange(max(1, s["most_shared"]), device="cuda")
    has = pos < shared[:, None]
    row = starts[:-1].clamp_max(b - 1)
    col = (pos // page).clamp_max(s["page_table"].shape[1] - 1)
    slot = torch.where(has, s["page_table"][row][:, col] * page + pos % page, -1)
    i = torch.arange(s["most_group"] * new, device="cuda")
    at = (starts[:-1, None] * new + i).clamp_max(len(q) - 1)
    o1, m1, l1 = _part(s, q[at].flatten(1, 2), _rows(s, slot), has[:, None])
    mine = i < (starts.diff() * new)[:, None]
    o1, m1, l1 = (v.unflatten(1, (-1, heads))[mine] for v in (o1, m1, l1))

    # every request's own keys
    pos = torch.arange(s["most_own"], device="cuda") + shared[group][:, None]
    has = pos < s["seq_lens"][:, None]
    slot = torch.where(has, s["page_table"].gather(1, (pos // page).clamp_max(s["page_table"].shape[1] - 1)) * page + pos % page, -1)
    last = s["seq_lens"][:, None] - new + torch.arange(new, device="cuda")
    live = (pos[:, None] <= last[..., None]).repeat_interleave(heads, 1)
    o2, m2, l2 = _part(s, q.reshape(b, new * heads, -1), _rows(s, slot), live)
    o2, m2, l2 = (v.reshape(b * new, heads, -1) for v in (o2, m2, l2))

    m = torch.maximum(m1, m2)
    w1, w2 = torch.exp(m1 - m), torch.exp(m2 - m)
    total = l1 * w1 + l2 * w2
    return ((o1 * w1 + o2 * w2) / total).bfloat16(), (m + total.log()).squeeze(-1)


# ---- what a pass cannot do without ----------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "keys":
        n = case["tokens"] - case["spare"]
        return {"bytes": n * (2 * DIM + 8 + 4 * TURNED + DIM + 4), "flops": n * DIM * (14 if case["hadamard"] else 7)}
    if op == "queries":
        n = case["tokens"] * HEADS
        return {"bytes": n * (3 * DIM + (4 if case["wide"] else 2) + 4) + case["tokens"] * (4 + 4 * TURNED), "flops": n * DIM * (11 if case["hadamard"] else 4)}
    if op == "load":
        return {"bytes": case["rows"] * 2 * (DIM + 4), "flops": 0}
    if op == "logits":
        b, new, mean = case["requests"], (case["new_lo"] + case["new_hi"]) / 2, (case["lo"] + case["hi"]) / 2
        tokens = b * case["new_hi"] if b == 1 else b * new
        mean = case["hi"] if b == 1 else mean
        pairs = tokens * max(1.0, mean - (tokens / b) / 2)
        return {"bytes": b * mean * (DIM + 4) + 4 * pairs + tokens * HEADS * (DIM + 4), "flops": pairs * HEADS * (2 * DIM + 3)}
    b, groups, heads = case["requests"], case["groups"], case["heads"]
    row = LATENT + 4 + 2 * ROPE if case["fp8"] else 2 * (LATENT + ROPE)
    starts = [round(b * (i / groups) ** 1.5) for i in range(groups + 1)]
    lens = [case["shared_hi"] if groups == 1 else case["shared_lo"] + (case["shared_hi"] - case["shared_lo"]) * i / (groups - 1) for i in range(groups)]
    mean = case["hi"] if b == 1 else (case["lo"] + case["hi"]) / 2
    tokens = b * case["new"]
    pairs = sum((starts[i + 1] - starts[i]) * case["new"] * lens[i] for i in range(groups)) + tokens * mean
    cached = sum(n for i, n in enumerate(lens) if starts[i + 1] > starts[i]) + b * mean
    return {"bytes": cached * row + tokens * heads * (2 * (LATENT + ROPE) + 2 * LATENT + 4), "flops": 2 * pairs * heads * (2 * LATENT + ROPE)}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"keys": _exact_keys, "queries": _exact_queries, "load": _exact_load, "logits": _exact_logits, "shared": _exact_shared}[case["op"]](s)


def _exact_turn(x, s, positions):
    angle = s["cos_sin"][positions.long()].double()
    turn = torch.complex(angle[:, :TURNED // 2], angle[:, TURNED // 2:])
    if x.dim() == 3:
        turn = turn[:, None]
    r = x[..., :TURNED]
    pairs = r.unflatten(-1, (TURNED // 2, 2)) if s["interleaved"] else r.unflatten(-1, (2, TURNED // 2)).transpose(-1, -2)
    done = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = torch.cat([(done if s["interleaved"] else done.transpose(-1, -2)).flatten(-2), x[..., TURNED:]], -1)
    if s["hadamard"]:
        for bit in range(7):   # sums and differences of the values whose places differ in one bit
            a, b = y.unflatten(-1, (DIM >> bit + 1, 2, 1 << bit)).unbind(-2)
            y = torch.stack([a + b, a - b], -2).flatten(-3)
        y = y / math.sqrt(DIM)
    return y


def _exact_codes(y):
    """The value nearest to each in four significand bits, subnormal below 2^-6, ties to even; and the row's step."""
    step = y.abs().amax(-1) / E4M3_MAX
    step = torch.where(step > 0, step, 1.0)
    y = y / step[..., None]
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / unit) * unit, step


def _exact_keys(s):
    rows = (s["slot_map"] >= 0).nonzero()[:, 0]
    x = s["k"][rows].double()
    x = (x - x.mean(1, keepdim=True)) / torch.sqrt(x.var(1, unbiased=False, keepdim=True) + EPS) * s["norm_weight"].double() + s["norm_bias"].double()
    keys, scale = s["keys"].view(torch.float8_e4m3fn).double(), s["key_scale"].double()
    keys[s["slot_map"][rows].long()], scale[s["slot_map"][rows].long()] = _exact_codes(_exact_turn(x, s, s["positions"][rows]))
    return keys, scale


def _exact_queries(s):
    codes, step = _exact_codes(_exact_turn(s["q"].double(), s, s["positions"]))
    return codes, s["weights"].double() * step * s["weight_scale"]


def _exact_load(s):
    starts, slots = s["kv_starts"].tolist(), []
    for b in range(len(starts) - 1):
        pos = torch.arange(starts[b + 1] - starts[b], device="cuda")
        slots.append(s["page_table"][b].long()[pos // s["page"]] * s["page"] + pos % s["page"])
    slots = torch.cat(slots)
    return s["keys"].view(torch.float8_e4m3fn).double()[slots], s["key_scale"].double()[slots]


def _exact_logits(s):
    out = torch.full(s["out"].shape, -math.inf, dtype=torch.float64, device="cuda")
    starts, lens, last = s["q_starts"].tolist(), s["seq_lens"].tolist(), []
    for b, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        slot = s["page_table"][b].long()[pos // s["page"]] * s["page"] + pos % s["page"]
        keys = s["keys"][slot].view(torch.float8_e4m3fn).double() * s["key_scale"][slot].double()[:, None]
        for t in range(starts[b], starts[b + 1]):
            most = n - (starts[b + 1] - t) + 1
            z = s["q"][t].view(torch.float8_e4m3fn).double() @ keys[:most].T
            out[t, :most] = s["weights"][t].double() @ z.clamp_min(0)
            last.append(most)
    return out, torch.tensor(last, device="cuda", dtype=torch.int32)


def _exact_shared(s):
    out = torch.zeros(len(s["q"]), s["heads"], LATENT, dtype=torch.float64, device="cuda")
    lse = torch.zeros(len(s["q"]), s["heads"], dtype=torch.float64, device="cuda")
    starts, shared, lens = s["group_starts"].tolist(), s["shared_lens"].tolist(), s["seq_lens"].tolist()
    for g in range(s["groups"]):
        for b in range(starts[g], starts[g + 1]):
            pos = torch.arange(lens[b], device="cuda")
            page = torch.where(pos < shared[g], s["page_table"][starts[g]].long()[pos // s["page"]], s["page_table"][b].long()[pos // s["page"]])
            slot = page * s["page"] + pos % s["page"]
            c = s["latent"][slot]
            c = c.view(torch.float8_e4m3fn).double() * s["scale"][slot].double()[:, None] if s["fp8"] else c.double()
            rows = torch.cat([c, s["rope"][slot].double()], 1)
            for i in range(s["new"]):
                t, most = b * s["new"] + i, lens[b] - s["new"] + i + 1
                z = s["sm"] * (s["q"][t].double() @ rows[:most].T)
                lse[t] = torch.logsumexp(z, 1)
                out[t] = torch.exp(z - lse[t][:, None]) @ c[:most]
    return out, lse
