"""Cases of the paged key-value cache: appending tokens, attention of one new token, eviction by accumulated weight.

A cache is a pool of pages, each holding `page` slots of every KV head; a table lists each sequence's pages, in any
order of the pool.  Slot s of sequence b is row s % page of page table[b, s // page].
"""

import math

import torch

own = False

ROPE_BASE = 1e6
SINKS, RECENT = 4, 64


# --------------------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------------------

def _case(name, op, batch, kv, group, d, n, page, dtype="bf16", **kw):
    c = {"op": op, "batch": batch, "kv": kv, "group": group, "d": d, "n": n, "page": page, "dtype": dtype,
         "ragged": False, "paired": False}
    c.update(kw)
    return {"name": name, **c} if name else c


def listed():
    return [
        # the start of a chat with one user: launch latency counts
        _case("decode 1 x 300", "decode", 1, 8, 4, 128, 300, 16),
        # the batch and context of the tiered workload, one token a sequence
        _case("decode 8 x 32768", "decode", 8, 8, 4, 128, 32768, 64),
        # one long document, the length split over the whole GPU
        _case("decode 1 x 131071", "decode", 1, 8, 4, 128, 131071, 64, paired=True),
        # a server's running batch: lengths from idle to 8K, small pages, K and V of a page side by side
        _case("decode 64 ragged", "decode", 64, 8, 4, 128, 8190, 16, ragged=True, paired=True),
        # a small float32 model: one query head a KV head, d = 64, odd length
        _case("decode f32 5 x 4099", "decode", 5, 4, 1, 64, 4099, 32, "f32"),
        # decoding that also tracks how much attention every cached token gets
        _case("weights 8 x 32768", "weights", 8, 8, 4, 128, 32768, 64),
        # the same for a small model with 8 query heads a KV head
        _case("weights 3 x 1000", "weights", 3, 2, 8, 64, 1000, 16, ragged=True),
        # the new token's projections of a decode step, from a fused QKV row
        _case("append step 8", "append", 8, 8, 4, 128, 20001, 64, s_new=1),
        # prompts of different lengths entering the cache
        _case("append prompts 4 x 8192", "append", 4, 8, 4, 128, 8192, 64, s_new=8192, ragged=True, paired=True),
        # a chat kept to 1024 tokens
        _case("evict 1 x 1500", "evict", 1, 8, 4, 128, 1500, 16, keep=1024),
        # the batch of the tiered workload cut to a quarter of its length
        _case("evict 8 x 32768", "evict", 8, 8, 4, 128, 32768, 64, keep=8192, paired=True),
        # a long float32 cache that drops a little
        _case("evict f32 2 x 65531", "evict", 2, 4, 2, 64, 65531, 128, "f32", keep=61440),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "weights", "append", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    kv, group, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    elt = 2 if dtype == "bf16" else 4
    batch = _log(rng, 1, 64)
    most = (1 << 30) // (2 * batch * kv * d * elt)  # slots a sequence: at most 1 GiB of K and V
    kw = {"ragged": rng.random() < 0.5, "paired": rng.random() < 0.5}
    if op == "append":
        s_new = 1 if rng.random() < 0.5 else _log(rng, 2, max(3, min(8192, most // 4)))
        n = min(most, s_new + _log(rng, 1, 16384))
        return _case(None, op, batch, kv, group, d, max(n, s_new), page, dtype, s_new=s_new, **kw)
    n = _log(rng, 1 if op != "evict" else 160, min(131072, max(200, most)))
    if op == "evict":
        kw["keep"] = min(n, max(SINKS + RECENT, _log(rng, 100, n)))
    return _case(None, op, batch, kv, group, d, n, page, dtype, **kw)


def _lens(case):
    """Slots in use of each sequence, the new tokens counted."""
    b, n = case["batch"], case["n"]
    if not case["ragged"] or b == 1:
        return [n] * b
    got = [max(1, n * ((7 * i + 3) % b + 1) // b) for i in range(b)]
    if b >= 4 and case["op"] != "append":
        got[1] = 0  # an idle row of a padded batch
    return got


def _news(case):
    """Tokens appended to each sequence."""
    return [min(case["s_new"], x) if case["ragged"] else case["s_new"] for x in _lens(case)]


def _last(case):
    """Position of each sequence's last token (a cache that was cut before is behind its position)."""
    return [2 * x + 5 for x in _lens(case)]


def work(case):
    kv, hq, d = case["kv"], case["kv"] * case["group"], case["d"]
    elt = 2 if case["dtype"] == "bf16" else 4
    lens, b = _lens(case), case["batch"]
    pages = 4 * sum(-(-x // case["page"]) for x in lens)
    if case["op"] in ("decode", "weights"):
        n = sum(lens)
        size = 2 * n * kv * d * elt + pages + 2 * b * hq * d * elt + 4 * b * hq + 4 * b
        if case["op"] == "weights":
            size += 8 * n * kv
        return {"bytes": size, "flops": 4 * n * hq * d}
    if case["op"] == "append":
        t = sum(_news(case))
        return {"bytes": t * (2 * (hq + 2 * kv) * d * elt + 8 * kv), "flops": 3 * t * (hq + kv) * d}
    size = 4 * b
    for x in lens:
        if x > case["keep"]:
            free = x - SINKS - RECENT
            moved = RECENT + max(0, x - case["keep"] - RECENT) * (case["keep"] - SINKS - RECENT) / max(1, free)
            size += 8 * x * kv + min(moved, case["keep"]) * kv * (4 * d * elt + 16)
    return {"bytes": size, "flops": 0}


# --------------------------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    b, kv, d, ps = case["batch"], case["kv"], case["d"], case["page"]
    hq = kv * case["group"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def randn(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    lens = torch.tensor(_lens(case), device=dev)
    max_pages = -(-case["n"] // ps)
    need = (lens + ps - 1) // ps
    n_pages = int(need.sum()) + 3
    # every sequence's pages lie anywhere in the pool; entries behind the last page name none
    order = torch.randperm(n_pages, generator=g, device=dev)
    at = (need.cumsum(0) - need)[:, None] + torch.arange(max_pages, device=dev)
    table = torch.where(torch.arange(max_pages, device=dev) < need[:, None], order[at.clamp(max=n_pages - 1)], -1)
    if case["paired"]:
        pool = randn(n_pages, 2, kv, ps, d)
        k, v = pool[:, 0], pool[:, 1]
    else:
        k, v = randn(n_pages, kv, ps, d), randn(n_pages, kv, ps, d)
    state = {"case": dict(case), "k": k, "v": v, "table": table.to(torch.int32), "n_slots": lens.to(torch.int32),
             "last": torch.tensor(_last(case), device=dev)}
    # per-slot records: the accumulated weight (heavy-tailed, some zeros) and the position of the token
    records = torch.empty((2, n_pages, kv, ps), device=dev)
    records[0] = torch.exp(2 * randn(n_pages, kv, ps, dtype=torch.float32))
    records[0] *= torch.rand((n_pages, kv, ps), generator=g, device=dev) > 0.1
    slot_pos = records[1].view(torch.int32)
    slot_pos.fill_(-1)
    # the later half of a sequence in order up to its last position, the half that earlier cuts went through mixed
    half = (lens // 2)[:, None, None]
    s = torch.arange(max_pages * ps, device=dev)
    shuffled = torch.where(s < half, torch.rand((b, kv, max_pages * ps), generator=g, device=dev), 2.0 + s)
    early = 2 * torch.argsort(shuffled, dim=-1)
    late = state["last"][:, None, None] - lens[:, None, None] + 1 + s
    pos = torch.where(s < half, early, late).to(torch.int32)
    bb, ss = torch.nonzero(s < lens[:, None], as_tuple=True)
    slot_pos[table[bb, ss // ps], :, ss % ps] = pos[bb, :, ss]
    state["records"], state["weight"], state["slot_pos"] = records, records[0], slot_pos
    if case["op"] in ("decode", "weights"):
        state["q"] = 2 * randn(b, hq, d)
        state["o"] = torch.zeros((b, hq, d), dtype=dt, device=dev)
        state["lse"] = torch.zeros((b, hq), device=dev)
    elif case["op"] == "append":
        s_new = case["s_new"]
        state["qkv"] = randn(b, s_new, (hq + 2 * kv) * d)  # token-major, Q, K and V in one row
        state["n_new"] = torch.tensor(_news(case), dtype=torch.int32, device=dev)
        state["q_out"] = torch.zeros((b, hq, s_new, d), dtype=dt, device=dev)
    else:
        state["records_before"] = records.clone()
    return state


# --------------------------------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------------------------------

def run(state):
    return run_own(state) if own else run_plain(state)


def run_own(state):
    import hierarchical_routed_sparse_hga_b200 as hga
    case, st = state["case"], state
    if "cache" not in st:  # the description of the cache and the workspace, kept as long as the cache
        cfg = hga.Config(case["batch"], case["kv"] * case["group"], case["kv"], case["d"], 1, 1,
                         hga.HGA_BF16 if case["dtype"] == "bf16" else hga.HGA_F32)
        cache = hga.PagedCache(cfg, st["k"], st["v"], st["table"], st["weight"], st["slot_pos"])
        if case["op"] in ("decode", "weights"):
            size = hga.hga_paged_decode_workspace_size(cfg, cache, case["op"] == "weights")
        else:
            size = hga.hga_paged_evict_workspace_size(cfg, cache)
        st["cfg"], st["cache"] = cfg, cache
        st["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device=st["k"].device)
    cfg, cache = st["cfg"], st["cache"]
    if case["op"] in ("decode", "weights"):
        accumulate = case["op"] == "weights"
        hga.hga_paged_decode(cfg, cache, st["q"], st["n_slots"], accumulate, st["o"], st["lse"], st["workspace"])
        return (st["o"], st["lse"], st["weight"]) if accumulate else (st["o"], st["lse"])
    if case["op"] == "append":
        row, hq, kv, d = st["qkv"].shape[2], case["kv"] * case["group"], case["kv"], case["d"]
        base = st["qkv"].data_ptr()
        elt = st["qkv"].element_size()
        hga.hga_paged_append(cfg, cache, base, base + hq * d * elt, base + (hq + kv) * d * elt, row, row,
                             case["s_new"], st["n_new"], st["n_slots"], st["last"], ROPE_BASE, st["q_out"])
        return st["q_out"], st["k"], st["v"], st["weight"], st["slot_pos"]
    # a pass begins with the records that the decode steps left, so that each pass cuts the same cache
    st["records"].copy_(st["records_before"])
    hga.hga_paged_evict(cfg, cache, st["n_slots"], st["last"], case["keep"], SINKS, RECENT, st["workspace"])
    return st["k"], st["v"], st["weight"], st["slot_pos"]


def run_plain(state):
    case = state["case"]
    if case["op"] == "append":
        return _append_plain(state)
    if case["op"] == "evict":
        return _evict_plain(state)
    return _decode_plain(state)


def _slots(state):
    """(slot numbers, which of them are in use [B, S])."""
    s = torch.arange(state["table"].shape[1] * state["case"]["page"], device=state["k"].device)
    return s, s < state["n_slots"][:, None]


def _rows(pool, table):
    """[B, heads, S, d] of a pool in 32 bits, by the table."""
    x = pool[table.clamp(min=0).long()]
    b, p, h, r, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, p * r, d).float()


def _decode_plain(state):
    case = state["case"]
    b, kv, g, d, ps = case["batch"], case["kv"], case["group"], case["d"], case["page"]
    s, used = _slots(state)
    mask = used[:, None, None, :]
    q = state["q"].float().view(b, kv, g, d)
    score = (q @ _rows(state["k"], state["table"]).transpose(-1, -2)) / math.sqrt(d)
    score = torch.where(mask, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(mask, torch.exp(score - top), 0.0)
    total = p.sum(-1, keepdim=True)
    p = torch.where(mask, p / total, 0.0)
    v = _rows(state["v"], state["table"])
    o = p @ torch.where(used[:, None, :, None], v, 0.0)
    lse = torch.where(used.any(-1)[:, None, None], (top + torch.log(total)).squeeze(-1), -math.inf)
    state["o"].copy_(o.reshape(b, kv * g, d))
    state["lse"].copy_(lse.reshape(b, kv * g))
    if case["op"] == "decode":
        return state["o"], state["lse"]
    bb, ss = torch.nonzero(used, as_tuple=True)
    page = state["table"][bb, ss // ps].long()
    state["weight"][page, :, ss % ps] += p.sum(2)[bb, :, ss]
    return state["o"], state["lse"], state["weight"]


def _append_plain(state):
    case = state["case"]
    b, kv, d, ps, s_new = case["batch"], case["kv"], case["d"], case["page"], case["s_new"]
    hq = kv * case["group"]
    dev = state["k"].device
    x = state["qkv"].view(b, s_new, hq + 2 * kv, d)
    i = torch.arange(s_new, device=dev)
    pos = state["last"][:, None] - state["n_new"][:, None] + 1 + i  # [B, S]
    theta = ROPE_BASE ** (-2.0 * torch.arange(d // 2, device=dev, dtype=torch.float64) / d)
    angle = pos[..., None].double() * theta
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    x1, x2 = x[:, :, :hq + kv, :d // 2].float(), x[:, :, :hq + kv, d // 2:].float()
    turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).to(x.dtype)
    bb, ii = torch.nonzero(i < state["n_new"][:, None], as_tuple=True)
    state["q_out"][bb, :, ii] = turned[bb, ii, :hq]
    slot = state["n_slots"].long()[bb] - state["n_new"].long()[bb] + ii
    page, row = state["table"][bb, slot // ps].long(), slot % ps
    state["k"][page, :, row] = turned[bb, ii, hq:]
    state["v"][page, :, row] = x[bb, ii, hq + kv:]
    state["weight"][page, :, row] = 0.0
    state["slot_pos"][page, :, row] = pos[bb, ii].to(torch.int32)[:, None].expand(-1, kv)
    return state["q_out"], state["k"], state["v"], state["weight"], state["slot_pos"]


def _evict_plain(state):
    case = state["case"]
    ps, keep = case["page"], case["keep"]
    state["records"].copy_(state["records_before"])
    s, used = _slots(state)
    # a record per slot, [B, heads, S]
    at = state["table"].clamp(min=0).long()
    weight = state["weight"][at].permute(0, 2, 1, 3).flatten(2)
    pos = state["slot_pos"][at].permute(0, 2, 1, 3).flatten(2)
    held = (pos < SINKS) | (pos > state["last"][:, None, None] - RECENT)
    key = torch.where(used[:, None], torch.where(held, math.inf, weight), -math.inf)
    rank = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.zeros(key.shape, dtype=torch.bool, device=key.device).scatter_(-1, rank, True)
    cut = (state["n_slots"] > keep)[:, None, None] & used[:, None]
    hb, hh, hs = torch.nonzero(cut & ~kept & (s < keep), as_tuple=True)
    mb, mh, ms = torch.nonzero(cut & kept & (s >= keep), as_tuple=True)
    to, frm = state["table"][hb, hs // ps].long(), state["table"][mb, ms // ps].long()
    for x in (state["k"], state["v"], state["weight"], state["slot_pos"]):
        x[to, hh, hs % ps] = x[frm, mh, ms % ps]
    return state["k"], state["v"], state["weight"], state["slot_pos"]


# --------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits, a sequence (and a head) at a time
# --------------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _append_exact(st)
    if case["op"] == "evict":
        return _evict_exact(st)
    return _decode_exact(st)


def _places(st, b):
    """(page, row) of each slot in use of sequence b."""
    s = torch.arange(int(st["n_slots"][b]), device=st["k"].device)
    return st["table"][b].long()[s // st["case"]["page"]], s % st["case"]["page"]


def _decode_exact(st):
    case = st["case"]
    kv, g, d = case["kv"], case["group"], case["d"]
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device=st["o"].device)
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device=st["o"].device)
    weight = st["weight"].double()
    for b in range(case["batch"]):
        page, row = _places(st, b)
        if page.numel() == 0:
            continue
        for h in range(kv):
            q = st["q"][b, h * g:(h + 1) * g].double()
            z = torch.einsum("gd,sd->gs", q, st["k"][page, h, row].double()) * d ** -0.5
            lse[b, h * g:(h + 1) * g] = torch.logsumexp(z, -1)
            p = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
            o[b, h * g:(h + 1) * g] = torch.einsum("gs,sd->gd", p, st["v"][page, h, row].double())
            weight[page, h, row] += p.sum(0)
    return (o, lse) if case["op"] == "decode" else (o, lse, weight)


def _append_exact(st):
    case = st["case"]
    kv, d, hq = case["kv"], case["d"], case["kv"] * case["group"]
    half = d // 2
    dev = st["k"].device
    q_out, k, v = st["q_out"].double(), st["k"].double(), st["v"].double()
    weight, slot_pos = st["weight"].double(), st["slot_pos"].clone()
    freq = torch.exp(-math.log(ROPE_BASE) * torch.arange(half, device=dev, dtype=torch.float64) / half)
    for b in range(case["batch"]):
        m, n, last = int(st["n_new"][b]), int(st["n_slots"][b]), int(st["last"][b])
        x = st["qkv"][b, :m].double().view(m, hq + 2 * kv, d)
        p = torch.arange(last - m + 1, last + 1, device=dev)
        # rotation of the pair (x_i, x_(i + d/2)) as a product of complex numbers
        turn = torch.polar(torch.ones((m, half), dtype=torch.float64, device=dev), p[:, None].double() * freq)
        z = torch.complex(x[..., :half], x[..., half:]) * turn[:, None]
        y = torch.cat([z.real, z.imag], -1)
        q_out[b, :, :m] = y[:, :hq].transpose(0, 1)
        page, row = _places(st, b)
        page, row = page[n - m:], row[n - m:]
        k[page, :, row] = y[:, hq:hq + kv]
        v[page, :, row] = x[:, hq + kv:]
        weight[page, :, row] = 0.0
        slot_pos[page, :, row] = p.to(torch.int32)[:, None].expand(-1, kv)
    return q_out, k, v, weight, slot_pos


def _evict_exact(st):
    case = st["case"]
    keep = case["keep"]
    k, v, weight, slot_pos = st["k"].double(), st["v"].double(), st["weight"].double(), st["slot_pos"].clone()
    for b in range(case["batch"]):
        n = int(st["n_slots"][b])
        if n <= keep:
            continue
        page, row = _places(st, b)
        for h in range(case["kv"]):
            w, p = st["weight"][page, h, row].double(), st["slot_pos"][page, h, row]
            held = (p < SINKS) | (p > st["last"][b] - RECENT)
            # held slots first, then by weight, then by slot
            by = torch.argsort(-w, stable=True)
            by = by[torch.argsort((~held[by]).to(torch.int8), stable=True)]
            kept = torch.sort(by[:keep]).values
            drop = torch.sort(by[keep:]).values
            frm, to = kept[kept >= keep], drop[drop < keep]
            for x in (k, v, weight, slot_pos):
                x[page[to], h, row[to]] = x[page[frm], h, row[frm]]
    return k, v, weight, slot_pos
