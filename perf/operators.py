"""The serving operators around the top-k selection: what each computes, on which sizes it is measured.

The plan of an append (pages and slots of new tokens), the latent cache's store and load, latent attention in its
absorbed form (over selected slots, or over a whole paged cache) and in its expanded form (prefill).  `run` computes a
case in plain torch operations, or, where `own` is set, through the library's entry points.
"""
import math

import torch

own = False

LATENT = 512   # width of a token's latent vector
ROPE = 64      # width of its shared rotary key
HEAD = 128     # width of a head's expanded key (without its rotary part) and value
E4M3_MAX = 448.0
EPS = 1e-6


# ---- the cases ------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 requests: one new token each, the benchmark's ragged lengths
        dict(name="plan_decode_64", op="plan", requests=64, lo=4096, hi=65536, new_lo=1, new_hi=1, page=64, spare=0),
        # a step of 300 requests that mixes prompt chunks, single tokens and idle requests; the token buffers are longer
        # than the step's tokens, as those of a captured graph are
        dict(name="plan_chunks_300", op="plan", requests=300, lo=0, hi=16384, new_lo=0, new_hi=1024, page=16, spare=1000),
        # the same decode step's cache rows
        dict(name="store_decode_64", op="store", tokens=64, fp8=False, slots=16384, spare=0),
        # a prompt chunk into an 8-bit cache, some rows of the batch being padding
        dict(name="store_prefill_16000", op="store", tokens=16000, fp8=True, slots=65536, spare=37),
        # rows picked by slot
        dict(name="load_slots_1000", op="load", rows=1000, fp8=False, slots=65536, paged=False, requests=0, page=64),
        # the cached prefixes of 16 requests, before their keys and values are expanded
        dict(name="load_paged_16", op="load", rows=400000, fp8=True, slots=524288, paged=True, requests=16, page=64),
        # one token of one request with a million cached ones, over the 2048 that the indexer selected
        dict(name="sparse_decode_1", op="sparse", requests=1, new=1, lo=1048576, hi=1048576, k=2048, heads=32, fp8=False, page=64),
        # one decode step of 64 requests over their selected slots
        dict(name="sparse_decode_64", op="sparse", requests=64, new=1, lo=4096, hi=65536, k=2048, heads=64, fp8=True, page=64),
        # a prompt chunk: the last 1024 tokens of 65536, each over its own selected slots
        dict(name="sparse_prefill_1024", op="sparse", requests=1, new=1024, lo=65536, hi=65536, k=2048, heads=128, fp8=False, page=64),
        # one decode step over the whole cache
        dict(name="paged_decode_64", op="paged", requests=64, new=1, lo=4096, hi=65536, heads=32, fp8=False, page=64),
        # a whole prompt
        dict(name="prefill_8192", op="expanded", requests=1, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0, heads=32),
        # chunks of six prompts behind cached prefixes, odd lengths, as many heads as one GPU of several has
        dict(name="prefill_ragged_6", op="expanded", requests=6, new_lo=1, new_hi=1500, ctx_lo=0, ctx_hi=5000, heads=20),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["plan", "store", "load", "sparse", "sparse", "paged", "expanded"])
    if op == "plan":
        requests = _log_int(rng, 1, 2000)
        new_hi = _log_int(rng, 1, max(1, 200000 // requests))
        return dict(op=op, requests=requests, lo=0, hi=_log_int(rng, 10, 65536), new_lo=rng.choice([0, 1]), new_hi=new_hi, page=rng.choice([1, 16, 32, 64, 128]), spare=_log_int(rng, 1, 2000) - 1)
    if op == "store":
        tokens = _log_int(rng, 1, 16000)
        return dict(op=op, tokens=tokens, fp8=rng.random() < 0.5, slots=tokens + _log_int(rng, 100, 49000), spare=rng.choice([0, 1, 5]))
    if op == "load":
        paged = rng.random() < 0.5
        rows = _log_int(rng, 10, 400000)
        return dict(op=op, rows=rows, fp8=rng.random() < 0.5, slots=524288 if paged else _log_int(rng, 1000, 524288), paged=paged, requests=_log_int(rng, 1, 60) if paged else 0, page=rng.choice([16, 64]))
    fp8, page = rng.random() < 0.5, rng.choice([1, 16, 64])
    heads = rng.choice([5, 8, 12, 24, 32, 40, 64, 128])
    if op == "sparse":
        requests = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, max(1, 1000 // requests))
        lo = _log_int(rng, max(2, new), 32000)
        return dict(op=op, requests=requests, new=new, lo=lo, hi=_log_int(rng, lo, 65536), k=rng.choice([64, 500, 512, 1024, 2048]), heads=heads, fp8=fp8, page=page)
    if op == "paged":
        requests = _log_int(rng, 1, 200)
        hi = min(1048576, _log_int(rng, 16, 2000000) // requests + 2)
        return dict(op=op, requests=requests, new=rng.choice([1, 1, 2, 3]) if hi * requests < 400000 else 1, lo=max(1, hi // 16), hi=hi, heads=min(heads, 64) if hi * requests > 500000 else heads, fp8=fp8, page=page)
    requests = _log_int(rng, 1, 12)
    new_hi = _log_int(rng, 1, 4000) // requests + 1
    return dict(op=op, requests=requests, new_lo=rng.choice([0, 1]), new_hi=new_hi, ctx_lo=0, ctx_hi=rng.choice([0, _log_int(rng, 1, 3000)]), heads=rng.choice([1, 3, 8, 16, 32]))


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _between(lo, hi, n, g):
    """n lengths spread evenly from lo to hi, in an order of the seed's: their sum is the case's own."""
    return torch.linspace(hi if n == 1 else lo, hi, n, device="cuda", dtype=torch.float64).long()[torch.randperm(n, generator=g, device="cuda")]


def _starts(lens):
    return torch.cat([lens.new_zeros(1), lens.cumsum(0)])


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _cache(slots, fp8, g):
    """A cache that already holds tokens: normed latents, rotary keys; in 8 bits codes and a scale a token."""
    latent, rope, scale = _normal((slots, LATENT), g), _normal((slots, ROPE), g), None
    if fp8:
        latent = (latent * 112).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = (torch.rand(slots, generator=g, device="cuda") + 0.5) / 112
    return latent, rope, scale


def _pages(lens, page, g):
    """A page table over pages in random order, and the number of slots it spans."""
    need = (lens + page - 1) // page
    total, most = int(need.sum()), max(1, int(need.max()))
    order = torch.randperm(total, generator=g, device="cuda")
    at = _starts(need)[:-1, None] + torch.arange(most, device="cuda")
    table = torch.where(torch.arange(most, device="cuda") < need[:, None], order[at.clamp_max(total - 1)], -1)
    return table.int(), total * page


def _chosen(table, page, lengths, owner, k, g):
    """k distinct positions below each row's length, spread over it, as slots in no order; short rows end in -1."""
    j = torch.arange(k, device="cuda")
    n = lengths[:, None]
    pos = torch.where(n > k, ((j + torch.rand(len(owner), k, generator=g, device="cuda", dtype=torch.float64)) * n / k).long(), j)
    pos = torch.minimum(pos, (n - 1).clamp_min(0))
    slot = table[owner[:, None], pos // page].long() * page + pos % page
    slot = torch.where(j < n, slot, -1)
    return torch.where(n > k, slot[:, torch.randperm(k, generator=g, device="cuda")], slot).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], dict(case)
    if op == "plan":
        lens, new = _between(case["lo"], case["hi"], case["requests"], g), _between(case["new_lo"], case["new_hi"], case["requests"], g)
        new[new < case["new_hi"] // 8] = case["new_lo"]   # idle requests, or single tokens
        page = case["page"]
        had, need = (lens + page - 1) // page, (lens + new + page - 1) // page
        table, _ = _pages(lens, page, g)
        width = -(-(case["hi"] + case["new_hi"]) // page)
        table = torch.cat([table, table.new_full((len(lens), width - table.shape[1]), -1)], 1).contiguous()
        free = int(had.sum()) + torch.randperm(int((need - had).sum()) + 5, generator=g, device="cuda")
        s.update(kv_lens=lens.int(), new_lens=new.int(), page_table=table, free_pages=free.int(), free_used=torch.full((1,), 3, dtype=torch.int32, device="cuda"), num_tokens=int(new.sum()) + case["spare"])
    elif op == "store":
        n = case["tokens"]
        slot_map = torch.randperm(case["slots"], generator=g, device="cuda")[:n].int()
        slot_map[n - case["spare"]:] = -1
        angle = torch.arange(65536, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
        s["latent"], s["rope"], s["scale"] = _cache(case["slots"], case["fp8"], g)
        s.update(kv=_normal((n, LATENT + ROPE), g) * 3, slot_map=slot_map, positions=torch.randint(0, 65536, (n,), generator=g, device="cuda").int(),
                 norm_weight=1 + 0.1 * _normal((LATENT,), g), cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float())
    elif op == "load":
        s["latent"], s["rope"], s["scale"] = _cache(case["slots"], case["fp8"], g)
        if case["paged"]:
            lens = _between(0, 2 * case["rows"] // max(2, case["requests"]), case["requests"], g)
            s["page_table"], _ = _pages(lens, case["page"], g)
            s["kv_starts"], s["num_rows"] = _starts(lens).int(), int(lens.sum())
        else:
            s["slot_map"] = torch.randint(0, case["slots"], (case["rows"],), generator=g, device="cuda").int()
            s["slot_map"][::9] = -1
    elif op in ("sparse", "paged"):
        lens = _between(case["lo"], case["hi"], case["requests"], g).clamp_min(case["new"])
        s["page_table"], slots = _pages(lens, case["page"], g)
        s["latent"], s["rope"], s["scale"] = _cache(slots, case["fp8"], g)
        tokens = case["requests"] * case["new"]
        s["q"] = _normal((tokens, case["heads"], LATENT + ROPE), g)
        s["sm"] = (HEAD + ROPE) ** -0.5
        if op == "paged":
            s["seq_lens"], s["q_starts"] = lens.int(), torch.arange(0, tokens + 1, case["new"], device="cuda", dtype=torch.int32)
        else:
            owner = torch.arange(tokens, device="cuda") // case["new"]
            lengths = lens[owner] - case["new"] + 1 + torch.arange(tokens, device="cuda") % case["new"]
            s["indices"] = torch.cat([_chosen(s["page_table"], case["page"], n, o, case["k"], g) for n, o in zip(lengths.split(4096), owner.split(4096))])
    else:
        new, ctx = _between(case["new_lo"], case["new_hi"], case["requests"], g), _between(case["ctx_lo"], case["ctx_hi"], case["requests"], g)
        s["q_starts"], s["kv_starts"] = _starts(new).int(), _starts(new + ctx).int()
        s["most_q"], s["most_kv"] = int(new.max()), int((new + ctx).max())
        tq, tk = int(new.sum()), int((new + ctx).sum())
        s.update(q=_normal((tq, case["heads"], HEAD + ROPE), g), kv_up=_normal((tk, case["heads"], 2 * HEAD), g), rope=_normal((tk, ROPE), g), sm=(HEAD + ROPE) ** -0.5)
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_attention_indexer_fp32_amd as lib
    op = s["op"]
    if op == "plan":
        return lib.paged_append_plan(s["kv_lens"], s["new_lens"], s["page_table"], s["free_pages"], s["page"], s["num_tokens"], free_used=s["free_used"])._asdict() | {"page_table": s["page_table"]}
    if op == "store":
        lib.latent_cache_store(s["kv"], s["slot_map"], s["latent"], s["rope"], scale=s["scale"], norm_weight=s["norm_weight"], eps=EPS, positions=s["positions"], cos_sin=s["cos_sin"])
        if not s["fp8"]:
            return s["latent"], s["rope"]
        return (*lib.latent_cache_load(s["slot_map"], s["latent"], s["rope"], scale=s["scale"]), s["scale"])
    if op == "load" and s["paged"]:
        return lib.latent_cache_load_paged(s["page_table"], s["kv_starts"], s["page"], s["num_rows"], s["latent"], s["rope"], scale=s["scale"])
    if op == "load":
        return lib.latent_cache_load(s["slot_map"], s["latent"], s["rope"], scale=s["scale"])
    if op == "sparse":
        return lib.latent_attention(s["q"], s["latent"], s["rope"], s["indices"], s["sm"], scale=s["scale"])
    if op == "paged":
        return lib.latent_attention_paged(s["q"], s["latent"], s["rope"], s["page_table"], s["seq_lens"], s["q_starts"], s["page"], s["sm"], scale=s["scale"])
    return lib.latent_attention_expanded(s["q"], s["kv_up"], s["rope"], s["q_starts"], s["kv_starts"], s["sm"])


def _run_plain(s):
    return {"plan": _plan, "store": _store, "load": _load, "sparse": _sparse, "paged": _paged, "expanded": _expanded}[s["op"]](s)


def _owner(starts, n):
    """The request of each of n rows, and whether the row belongs to one."""
    t = torch.arange(n, device=starts.device, dtype=torch.int32)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    return t, b.clamp_max(len(starts) - 2), t < starts[-1]


def _plan(s):
    page, table, used = s["page"], s["page_table"], s["free_used"].long()
    kv, new = s["kv_lens"].long(), s["new_lens"].long()
    had, need = (kv + page - 1) // page, (kv + new + page - 1) // page
    first = _starts(need - had)
    col = torch.arange(table.shape[1], device="cuda")
    at = used + first[:-1, None] + col - had[:, None]
    fresh = torch.where(at < len(s["free_pages"]), s["free_pages"][at.clamp(0, len(s["free_pages"]) - 1)], -1)
    table.copy_(torch.where((col >= had[:, None]) & (col < need[:, None]), fresh, table))
    q_starts = _starts(new).int()
    t, b, live = _owner(q_starts, s["num_tokens"])
    pos = kv[b] + t - q_starts[b]
    held = table[b, (pos // page).clamp_max(table.shape[1] - 1)].long()
    slot = torch.where(live & (held >= 0), held * page + pos % page, -1)
    return {"seq_lens": (kv + new).int(), "q_starts": q_starts, "slot_map": slot.int(), "positions": torch.where(live, pos, -1).int(),
            "free_used": (used + first[-1]).int(), "page_table": table}


def _store(s):
    live = s["slot_map"] >= 0
    slot = s["slot_map"][live].long()
    x = s["kv"][live].float()
    c, r = x[:, :LATENT], x[:, LATENT:]
    y = c * torch.rsqrt(c.square().mean(1, keepdim=True) + EPS) * s["norm_weight"].float()
    cos, sin = s["cos_sin"][s["positions"][live].long()].split(ROPE // 2, 1)
    even, odd = r[:, 0::2], r[:, 1::2]
    s["rope"][slot] = torch.stack([even * cos - odd * sin, odd * cos + even * sin], 2).reshape(len(slot), ROPE).bfloat16()
    if not s["fp8"]:
        s["latent"][slot] = y.bfloat16()
        return s["latent"], s["rope"]
    scale = y.abs().amax(1) / E4M3_MAX
    scale = torch.where(scale > 0, scale, 1.0)
    s["scale"][slot] = scale
    s["latent"][slot] = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return (*_load(s), s["scale"])


def _rows(s, slot):
    """Cache rows of these slots as 32-bit values; a slot below zero gives zeros."""
    live, slot = (slot >= 0)[..., None], slot.clamp_min(0).long()
    c = s["latent"][slot]
    c = c.view(torch.float8_e4m3fn).float() * s["scale"][slot][..., None] if s["fp8"] else c.float()
    return torch.where(live, c, 0.0), torch.where(live, s["rope"][slot].float(), 0.0)


def _load(s):
    slot = s.get("slot_map")
    if slot is None:
        t, b, live = _owner(s["kv_starts"], s["num_rows"])
        pos = t - s["kv_starts"][b]
        slot = torch.where(live, s["page_table"][b, (pos // s["page"]).long()] * s["page"] + pos % s["page"], -1)
    c, r = _rows(s, slot)
    return c.bfloat16(), r.bfloat16()


def _softmax(z, live):
    """Weights and the logarithm of their sum; a row with nothing live weighs nothing."""
    z = torch.where(live, z, -math.inf)
    top = z.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p / total, 0.0), (top + total.log()).squeeze(-1)


def _sparse(s):
    q = s["q"].float()
    c, r = _rows(s, s["indices"])
    z = s["sm"] * (torch.bmm(q[..., :LATENT], c.mT) + torch.bmm(q[..., LATENT:], r.mT))
    p, lse = _softmax(z, (s["indices"] >= 0)[:, None])
    return torch.bmm(p, c).bfloat16(), lse


def _paged(s):
    b, new, page = s["requests"], s["new"], s["page"]
    pos = torch.arange(s["page_table"].shape[1] * page, device="cuda")
    slot = s["page_table"][:, pos // page] * page + pos % page
    c, r = _rows(s, torch.where(pos < s["seq_lens"][:, None], slot, -1))
    q = s["q"].float().reshape(b, new * s["heads"], LATENT + ROPE)
    z = s["sm"] * (torch.bmm(q[..., :LATENT], c.mT) + torch.bmm(q[..., LATENT:], r.mT))
    last = s["seq_lens"][:, None] - new + torch.arange(new, device="cuda")
    live = (pos <= last[..., None]).repeat_interleave(s["heads"], 1)
    p, lse = _softmax(z, live)
    return torch.bmm(p, c).reshape(b * new, s["heads"], LATENT).bfloat16(), lse.reshape(b * new, s["heads"])


def _expanded(s):
    qs, ks = s["q_starts"].long(), s["kv_starts"].long()
    nq, nk = qs.diff(), ks.diff()
    i, j = torch.arange(s["most_q"], device="cuda"), torch.arange(s["most_kv"], device="cuda")
    at_q = (qs[:-1, None] + i).clamp_max(len(s["q"]) - 1)
    at_k = (ks[:-1, None] + j).clamp_max(len(s["rope"]) - 1)
    q = s["q"][at_q].float().transpose(1, 2)
    up = s["kv_up"][at_k].float().transpose(1, 2)
    z = torch.matmul(q[..., :HEAD], up[..., :HEAD].mT) + torch.matmul(q[..., HEAD:], s["rope"][at_k].float()[:, None].mT)
    live = j <= (nk - nq)[:, None, None] + i[:, None]
    p, lse = _softmax(s["sm"] * z, (live & (j < nk[:, None, None]))[:, None])
    o = torch.matmul(p, up[..., HEAD:]).transpose(1, 2)
    has = i < nq[:, None]
    return o[has].bfloat16(), lse.transpose(1, 2)[has]


# ---- what a pass cannot do without ----------------------------------------------------------------------------------

def _row_bytes(fp8):
    return LATENT + 4 + 2 * ROPE if fp8 else 2 * (LATENT + ROPE)


def work(case):
    op = case["op"]
    if op == "plan":
        new = (case["new_lo"] + case["new_hi"]) / 2
        tokens = case["requests"] * new
        return {"bytes": 16 * case["requests"] + 8 * (tokens + case["spare"]) + 8 * (tokens / case["page"] + case["requests"] / 2), "flops": 0}
    if op == "store":
        n = case["tokens"] - case["spare"]
        rows = n * (2 * (LATENT + ROPE) + 8 + 4 * ROPE + _row_bytes(case["fp8"]))
        return {"bytes": rows + (n * (_row_bytes(True) + 2 * (LATENT + ROPE)) if case["fp8"] else 0), "flops": n * 6 * (LATENT + ROPE)}
    if op == "load":
        return {"bytes": case["rows"] * (_row_bytes(case["fp8"]) + 2 * (LATENT + ROPE)), "flops": 0}
    if op in ("sparse", "paged"):
        tokens, mean = case["requests"] * case["new"], (case["lo"] + case["hi"]) / 2
        pairs = tokens * (min(mean, case["k"]) if op == "sparse" else mean)
        cached = min(pairs, case["requests"] * mean)
        io = tokens * case["heads"] * (2 * (LATENT + ROPE) + 2 * LATENT + 4) + (4 * tokens * case["k"] if op == "sparse" else 0)
        return {"bytes": cached * _row_bytes(case["fp8"]) + io, "flops": 2 * pairs * case["heads"] * (2 * LATENT + ROPE)}
    new, ctx = (case["new_lo"] + case["new_hi"]) / 2, (case["ctx_lo"] + case["ctx_hi"]) / 2
    tq, tk = case["requests"] * new, case["requests"] * (new + ctx)
    pairs = tq * (ctx + new / 2)
    return {"bytes": 2 * case["heads"] * (tq * (2 * HEAD + ROPE + 2) + tk * 2 * HEAD) + 2 * tk * ROPE, "flops": 2 * pairs * case["heads"] * (2 * HEAD + ROPE)}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None   # whole numbers only
    if op in ("store", "load"):
        return _exact_store(s) if op == "store" else _exact_load(s)
    if op == "expanded":
        return _exact_expanded(s)
    out = torch.zeros(len(s["q"]), case["heads"], LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((len(s["q"]), case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for t in range(len(s["q"])):
        if op == "sparse":
            slot = s["indices"][t]
            slot = slot[slot >= 0].long()
        else:
            b, i = divmod(t, case["new"])
            pos = torch.arange(int(s["seq_lens"][b]) - case["new"] + i + 1, device="cuda")
            slot = s["page_table"][b].long()[pos // case["page"]] * case["page"] + pos % case["page"]
        if len(slot):
            c = s["latent"][slot]
            c = c.view(torch.float8_e4m3fn).double() * s["scale"][slot].double()[:, None] if case["fp8"] else c.double()
            z = s["q"][t].double() @ torch.cat([c, s["rope"][slot].double()], 1).T * s["sm"]
            lse[t] = torch.logsumexp(z, 1)
            out[t] = torch.exp(z - lse[t][:, None]) @ c
    return out, lse


def _exact_store(s):
    rows = (s["slot_map"] >= 0).nonzero()[:, 0]
    slot, x = s["slot_map"][rows].long(), s["kv"][rows].double()
    c = x[:, :LATENT]
    c = c / torch.sqrt((c * c).sum(1, keepdim=True) / LATENT + EPS) * s["norm_weight"].double()
    turn = torch.complex(*s["cos_sin"][s["positions"][rows].long()].double().split(ROPE // 2, 1))
    r = torch.view_as_real(torch.view_as_complex(x[:, LATENT:].reshape(-1, ROPE // 2, 2)) * turn).reshape(-1, ROPE)
    if not s["fp8"]:
        latent, rope = s["latent"].double(), s["rope"].double()
        latent[slot], rope[slot] = c, r
        return latent, rope
    scale = s["scale"].double()
    step = c.abs().max(1).values / E4M3_MAX
    scale[slot] = step
    # the value nearest to each in four significand bits, subnormal below 2^-6, ties to even
    y = c / step[:, None]
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    held = torch.zeros(len(s["kv"]), LATENT, dtype=torch.float64, device="cuda")
    turned = torch.zeros(len(s["kv"]), ROPE, dtype=torch.float64, device="cuda")
    held[rows] = torch.round(y / unit) * unit * step[:, None]
    turned[rows] = r
    return held, turned, scale


def _exact_load(s):
    if s["paged"]:
        starts = s["kv_starts"].tolist()
        slot = []
        for b in range(len(starts) - 1):
            pos = torch.arange(starts[b + 1] - starts[b], device="cuda")
            slot.append(s["page_table"][b].long()[pos // s["page"]] * s["page"] + pos % s["page"])
        slot = torch.cat(slot)
    else:
        slot = s["slot_map"].long()
    c = s["latent"][slot]
    c = c.view(torch.float8_e4m3fn).double() * s["scale"][slot].double()[:, None] if s["fp8"] else c.double()
    r = s["rope"][slot].double()
    c[slot < 0], r[slot < 0] = 0, 0
    return c, r


def _exact_expanded(s):
    heads = s["heads"]
    out = torch.zeros(len(s["q"]), heads, HEAD, dtype=torch.float64, device="cuda")
    lse = torch.full((len(s["q"]), heads), -math.inf, dtype=torch.float64, device="cuda")
    qs, ks = s["q_starts"].tolist(), s["kv_starts"].tolist()
    for b in range(len(qs) - 1):
        q, up, r = s["q"][qs[b]:qs[b + 1]].double(), s["kv_up"][ks[b]:ks[b + 1]].double(), s["rope"][ks[b]:ks[b + 1]].double()
        if len(q) == 0 or len(up) == 0:
            continue
        hidden = torch.ones(len(q), len(up), dtype=torch.bool, device="cuda").triu(len(up) - len(q) + 1)
        for h in range(heads):
            z = (q[:, h] @ torch.cat([up[:, h, :HEAD], r], 1).T * s["sm"]).masked_fill(hidden, -math.inf)
            lse[qs[b]:qs[b + 1], h] = torch.logsumexp(z, 1)
            out[qs[b]:qs[b + 1], h] = torch.softmax(z, 1) @ up[:, h, HEAD:]
    return out, lse
