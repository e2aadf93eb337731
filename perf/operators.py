"""Measured cases of the KV-cache operators: the page bookkeeping of a serving
step (`ss_kv_append`, `ss_kv_commit`), the norms and rotary positions of
queries and keys with the store into the paged cache (`ss_rope_store`), and the
attention of a step's new tokens over the paged cache (`ss_attend`).

`own` chooses between the plain form of each operator in elementary torch
operations (False) and the calls of this library (True).  Both run on what
`prepare` makes.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "e4m3": 1}
# row status bits of the page bookkeeping
POOL, TABLE = 1 << 11, 1 << 12


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a small chat server's step: page bookkeeping for one new token of each request
        {"name": "append 16 x 1", "op": "append", "rows": 16, "new": 1, "longest": 4000, "page": 16, "spare": 64},
        # a full server after verification: what was accepted stays, the other pages go back
        {"name": "commit 512 x 8", "op": "commit", "rows": 512, "new": 8, "longest": 12000, "page": 16, "spare": 2048},
        # one decoding step of 8 requests
        {"name": "rope 8", "op": "rope", "tokens": 8, "hq": 32, "hkv": 8, "dim": 128, "rot": 128, "pairs": "half",
         "norm": True, "type": "bf16", "cache": "bf16", "layout": "hnd", "page": 16, "longest": 8000},
        # a verification step of about 250 requests, six tokens each; interleaved pairs on half of the head
        {"name": "rope 1531 interleaved", "op": "rope", "tokens": 1531, "hq": 64, "hkv": 8, "dim": 64, "rot": 32,
         "pairs": "interleaved", "norm": False, "type": "f16", "cache": "f16", "layout": "nhd", "page": 32, "longest": 30000},
        # pieces of prompts into a cache of 8-bit values
        {"name": "rope 6000 e4m3", "op": "rope", "tokens": 6000, "hq": 40, "hkv": 8, "dim": 128, "rot": 128, "pairs": "half",
         "norm": True, "type": "bf16", "cache": "e4m3", "layout": "hnd", "page": 64, "longest": 130000},
        # a whole batch of prompts, far positions
        {"name": "rope 16384", "op": "rope", "tokens": 16384, "hq": 32, "hkv": 8, "dim": 128, "rot": 128, "pairs": "half",
         "norm": True, "type": "bf16", "cache": "bf16", "layout": "hnd", "page": 16, "longest": 1000000},
        # one user, one token: latency
        {"name": "attend 1 x 1", "op": "attend", "rows": 1, "new": 1, "longest": 700, "hq": 32, "hkv": 8, "dim": 128,
         "type": "bf16", "cache": "bf16", "layout": "hnd", "page": 16, "window": 0, "sinks": 0},
        # ordinary decoding
        {"name": "attend 64 x 1", "op": "attend", "rows": 64, "new": 1, "longest": 6000, "hq": 32, "hkv": 8, "dim": 128,
         "type": "bf16", "cache": "bf16", "layout": "hnd", "page": 16, "window": 0, "sinks": 0},
        # verification: up to 7 drafts and the token before them, 8 query heads to a key head
        {"name": "attend 48 x 8", "op": "attend", "rows": 48, "new": 8, "longest": 16000, "hq": 64, "hkv": 8, "dim": 128,
         "type": "bf16", "cache": "bf16", "layout": "hnd", "page": 16, "window": 0, "sinks": 0},
        # long contexts in 8 bits, short drafts
        {"name": "attend 32 x 4 e4m3", "op": "attend", "rows": 32, "new": 4, "longest": 32000, "hq": 32, "hkv": 8, "dim": 128,
         "type": "bf16", "cache": "e4m3", "layout": "hnd", "page": 64, "window": 0, "sinks": 0},
        # a layer with a sliding window and a few first tokens that stay visible
        {"name": "attend 96 x 3 window", "op": "attend", "rows": 96, "new": 3, "longest": 20000, "hq": 28, "hkv": 4, "dim": 64,
         "type": "f16", "cache": "f16", "layout": "nhd", "page": 32, "window": 4000, "sinks": 4},
        # two very long contexts: the split over the cache's length
        {"name": "attend 2 x 5 long", "op": "attend", "rows": 2, "new": 5, "longest": 400000, "hq": 40, "hkv": 8, "dim": 128,
         "type": "bf16", "cache": "bf16", "layout": "hnd", "page": 16, "window": 0, "sinks": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    page = rng.choice([16, 32, 64, 128])
    op = rng.choice(["append", "commit", "rope", "rope", "attend", "attend", "attend", "attend"])
    if op in ("append", "commit"):
        rows = _log(rng, 1, 1000)
        return {"op": op, "rows": rows, "new": _log(rng, 1, max(1, min(300, 60000 // rows))), "longest": _log(rng, 1, 20000), "page": page,
                "spare": _log(rng, 1, 4000)}
    hq, hkv, dim = rng.choice([(32, 8, 128), (64, 8, 128), (40, 8, 128), (28, 4, 128), (16, 16, 128), (28, 4, 64), (71, 1, 64), (32, 4, 64),
                               (8, 1, 256), (16, 8, 256)])
    kind = rng.choice(["bf16", "f16"])
    cache = rng.choice([kind, kind, "e4m3"])
    layout = rng.choice(["hnd", "nhd"])
    if op == "rope":
        tokens = _log(rng, 1, 16384 * 6144 // ((hq + 2 * hkv) * dim))
        return {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim, "rot": rng.choice([dim, dim, dim // 2, dim // 4]),
                "pairs": rng.choice(["half", "interleaved"]), "norm": rng.random() < 0.6, "type": kind, "cache": cache, "layout": layout,
                "page": page, "longest": _log(rng, 100, 1000000)}
    rows = _log(rng, 1, 256)
    case = {"op": op, "rows": rows, "new": rng.choice([1, 1, 2, 3, 4, 5, 6, 7, 8, 11, 16]), "longest": _log(rng, 1, 200000), "hq": hq, "hkv": hkv,
            "dim": dim, "type": kind, "cache": cache, "layout": layout, "page": page, "window": 0, "sinks": 0}
    if rng.random() < 0.3:
        case.update(window=_log(rng, 16, 5000), sinks=rng.choice([0, 1, 4, 60]))
    # no more keys or scores than the largest listed cases, also in the plain form, whose rows are as long as the longest
    while rows * (case["longest"] + case["new"]) * max(hkv * dim / 1.3e9, hq * case["new"] / 0.4e9, hq * case["new"] * dim / 50e9) > 1:
        if case["longest"] > 1:
            case["longest"] = case["longest"] * 2 // 3
        else:
            case["rows"] = rows = rows // 2
    return case


def _lengths(case):
    """Cached tokens of each row, before its new ones: from one token to the longest, spread evenly over the square root."""
    n, longest = case["rows"], case["longest"]
    return [max(1, int(longest * ((i + 1) / n) ** 2)) - (1 if longest == 1 and i % 2 else 0) for i in range(n)]


def _news(case):
    """New tokens of each row: 1 .. new, the last rows the most."""
    return [1 + (i * 5 + case["new"] - 1) % case["new"] if i else case["new"] for i in range(case["rows"])]


def _attend_keys(case):
    """Keys that the rows' queries see, summed over the rows."""
    total = 0
    for held, new in zip(_lengths(case), _news(case)):
        seen = held + new
        if case["window"]:
            seen = min(seen, case["window"] + new - 1 + min(case["sinks"], seen))
        total += seen
    return total


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat, step = out.view(-1), 1 << 27
    for at in range(0, flat.numel(), step):  # in pieces: the 32-bit draws of a large cache need not all be held
        n = min(step, flat.numel() - at)
        flat[at:at + n] = (torch.randn(n, generator=g, device=DEV) * scale).to(dtype)
    return out


def _order(g, values):
    """The same values for every seed, in an order of the seed's own."""
    t = torch.tensor(values, dtype=torch.int64, device=DEV)
    return t[torch.randperm(len(values), generator=g, device=DEV)]


def _cumulative(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(n, 0)]).to(torch.int32)


def _cache(g, case, pages, fill):
    """Keys or values [pages, kv heads, page, dim] ("hnd") or [pages, page, kv heads, dim] ("nhd"), seen as [pages, page, kv heads, dim]."""
    hnd = case["layout"] == "hnd"
    shape = (pages, case["hkv"], case["page"], case["dim"]) if hnd else (pages, case["page"], case["hkv"], case["dim"])
    dtype = TYPES[case["cache"]]
    t = _normal(g, shape, dtype) if fill else torch.zeros(shape, dtype=dtype, device=DEV)
    return t.transpose(1, 2) if hnd else t


def prepare(case, seed):
    return {"append": _prepare_pages, "commit": _prepare_pages, "rope": _prepare_rope, "attend": _prepare_attend}[case["op"]](case, seed)


def _handle(case, rows, tokens, new, pages, blocks):
    """The plan and workspace that a program keeps."""
    from spec_verification_gb300 import kv
    plan = kv.Plan(max_rows=rows, max_tokens=tokens, max_new=new, q_heads=case.get("hq", 8), kv_heads=case.get("hkv", 8),
                   head_dim=case.get("dim", 128), page_size=case["page"], num_pages=pages, max_blocks=blocks,
                   dtype=case.get("type", "bf16"), cache_dtype=case.get("cache", "bf16"))
    return plan, torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)


def _prepare_pages(case, seed):
    g, page, rows = _gen(seed), case["page"], case["rows"]
    held, new = _order(g, _lengths(case)), _order(g, _news(case))
    blocks = -(-(case["longest"] + case["new"]) // page) + 1
    used = (held + page - 1) // page
    total = int(used.sum())
    pages = total + case["spare"]
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((rows, blocks), -1, dtype=torch.int32, device=DEV)
    column = torch.arange(blocks, device=DEV)[None]
    first = (torch.cumsum(used, 0) - used)[:, None]
    table = torch.where(column < used[:, None], ids[(first + column).clamp(max=pages - 1)], table)
    s = {"case": case, "table": table, "cu_new": _cumulative(new), "tokens": int(new.sum())}
    # the pool's state in one buffer: lengths, free count, free pages (the last ones are handed out first)
    pool = torch.zeros(rows + 1 + pages, dtype=torch.int32, device=DEV)
    pool[:rows] = held.to(torch.int32)
    pool[rows] = case["spare"]
    pool[rows + 1:rows + 1 + case["spare"]] = ids[total:]
    s["pool"] = pool
    s["kv_len"], s["free_count"], s["free_pages"] = pool[:rows], pool[rows:rows + 1], pool[rows + 1:]
    s["slots"] = torch.empty(s["tokens"], dtype=torch.int32, device=DEV)
    s["positions"] = torch.empty(s["tokens"], dtype=torch.int32, device=DEV)
    s["seq_len"] = torch.empty(rows, dtype=torch.int32, device=DEV)
    s["row_status"] = torch.empty(rows, dtype=torch.int32, device=DEV)
    if case["op"] == "commit":  # the state after an append, and what verification kept of each row
        s["table"], s["slots"], s["positions"], s["seq_len"], s["row_status"] = _append(s)
        s["accepted"] = (torch.rand(rows, generator=g, device=DEV) * new).to(torch.int32)
        s["finished"] = (torch.rand(rows, generator=g, device=DEV) < 0.02).to(torch.int32)
        s["before"] = pool.clone()
    if own:
        s["plan"], s["workspace"] = _handle(case, rows, s["tokens"], case["new"], pages, blocks)
    return s


def _frequencies(rot, base=500000.0):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)


def _prepare_rope(case, seed):
    g, t, hq, hkv, d, page = _gen(seed), case["tokens"], case["hq"], case["hkv"], case["dim"], case["page"]
    kind = TYPES[case["type"]]
    qkv = _normal(g, (t, (hq + 2 * hkv) * d), kind, 1.5)  # one projection's output: q, k and v are parts of its rows
    pages = -(-t * 5 // (4 * page)) + 1
    s = {"case": case, "qkv": qkv, "q": qkv[:, :hq * d].view(t, hq, d), "k": qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
         "v": qkv[:, (hq + hkv) * d:].view(t, hkv, d), "inv_freq": _frequencies(case["rot"]),
         "positions": torch.randint(0, case["longest"], (t,), generator=g, device=DEV).to(torch.int32),
         "slots": torch.randperm(pages * page, generator=g, device=DEV)[:t].to(torch.int32),
         "q_out": torch.empty(t, hq, d, dtype=kind, device=DEV), "k_cache": _cache(g, case, pages, False), "v_cache": _cache(g, case, pages, False)}
    s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(kind) if case["norm"] else None
    s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(kind) if case["norm"] else None
    low = case["cache"] == "e4m3"  # one factor to a key head: a value x is held as x / factor
    s["k_scale"] = 0.02 + 0.03 * torch.rand(hkv, generator=g, device=DEV) if low else None
    s["v_scale"] = 0.02 + 0.03 * torch.rand(hkv, generator=g, device=DEV) if low else None
    if own:
        s["plan"], s["workspace"] = _handle(case, 1, t, 1, pages, 1)
    return s


def _prepare_attend(case, seed):
    g, rows, page, hq, d = _gen(seed), case["rows"], case["page"], case["hq"], case["dim"]
    kind = TYPES[case["type"]]
    held, new = torch.tensor(_lengths(case), device=DEV), torch.tensor(_news(case), device=DEV)
    at = torch.randperm(rows, generator=g, device=DEV)
    held, new = held[at], new[at]
    length = held + new
    used = (length + page - 1) // page
    blocks, total = int(used.max()), int(used.sum())
    pages = total + 7
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    column = torch.arange(blocks, device=DEV)[None]
    first = (torch.cumsum(used, 0) - used)[:, None]
    table = torch.where(column < used[:, None], ids[(first + column).clamp(max=pages - 1)], -1).to(torch.int32)
    tokens = int(new.sum())
    s = {"case": case, "q": _normal(g, (tokens, hq, d), kind, 2.0), "k_cache": _cache(g, case, pages, True), "v_cache": _cache(g, case, pages, True),
         "table": table, "seq_len": length.to(torch.int32), "cu_new": _cumulative(new), "scale": d ** -0.5,
         "out": torch.empty(tokens, hq, d, dtype=kind, device=DEV), "row_status": torch.empty(rows, dtype=torch.int32, device=DEV)}
    low = case["cache"] == "e4m3"
    s["k_scale"] = 0.5 + torch.rand(case["hkv"], generator=g, device=DEV) if low else None
    s["v_scale"] = 0.5 + torch.rand(case["hkv"], generator=g, device=DEV) if low else None
    if own:
        s["plan"], s["workspace"] = _handle(case, rows, tokens, case["new"], pages, blocks)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        from spec_verification_gb300 import kv
        if op == "append":
            kv.ss_kv_append(s["plan"], s["table"], s["kv_len"], s["free_pages"], s["free_count"], s["cu_new"], slots=s["slots"],
                            positions=s["positions"], seq_len=s["seq_len"], row_status=s["row_status"])
            return s["table"], s["slots"], s["positions"], s["seq_len"], s["row_status"]
        if op == "commit":
            s["pool"].copy_(s["before"])
            kv.ss_kv_commit(s["plan"], s["table"], s["kv_len"], s["free_pages"], s["free_count"], s["seq_len"], counts=s["accepted"], plus=1,
                            finished=s["finished"])
            return s["kv_len"], s["free_count"], s["free_pages"]
        if op == "rope":
            kv.ss_rope_store(s["plan"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["inv_freq"], s["positions"], s["slots"],
                             q_out=s["q_out"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                             interleaved=s["case"]["pairs"] == "interleaved", k_scale=s["k_scale"], v_scale=s["v_scale"])
            return _rope_outputs(s)
        kv.ss_attend(s["plan"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_len"], s["cu_new"], out=s["out"],
                     row_status=s["row_status"], workspace=s["workspace"], scale=s["scale"], window=s["case"]["window"], sinks=s["case"]["sinks"],
                     k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"]
    if op == "append":
        return _append(s)
    if op == "commit":
        s["pool"].copy_(s["before"])
        return _commit(s)
    if op == "rope":
        return _rope(s)
    return _attend(s)


def _append(s):
    """Slots of the new tokens and the pages they need, rows in order, from the end of the free pages."""
    page, table, free = s["case"]["page"], s["table"], s["free_pages"]
    kv_len, cu = s["kv_len"].long(), s["cu_new"].long()
    new, blocks = cu[1:] - cu[:-1], table.shape[1]
    old, want = (kv_len + page - 1) // page, (kv_len + new + page - 1) // page
    fits = want <= blocks
    need = torch.where(fits, want - old, 0)
    upto = torch.cumsum(need, 0)
    enough = (need == 0) | (upto <= s["free_count"])
    served = fits & enough
    seq_len = torch.where(served, kv_len + new, kv_len)
    status = torch.where(fits, torch.where(enough, 0, POOL), TABLE)
    row = torch.repeat_interleave(torch.arange(table.shape[0], device=table.device), new, output_size=s["tokens"])
    position = kv_len[row] + torch.arange(s["tokens"], device=table.device) - cu[row]
    block = position // page
    at = (s["free_count"] - 1 - (upto - need - old)[row] - block).clamp(0, free.shape[0] - 1)
    held = table[row, block.clamp(max=blocks - 1)]
    ids = torch.where(served[row] & (block >= old[row]), free[at], held)
    slots = torch.where(served[row], ids * page + position % page, -1)
    table = table.index_put((row, block.clamp(max=blocks - 1)), ids)  # a page's tokens all write the same
    return table, slots.to(torch.int32), position.to(torch.int32), seq_len.to(torch.int32), status.to(torch.int32)


def _commit(s):
    """Rows keep accepted + 1 of their new tokens (finished rows nothing at all); pages that hold nothing kept go back, in order of row and block."""
    page, table, free, rows = s["case"]["page"], s["table"], s["free_pages"], s["case"]["rows"]
    kv_len, seq_len = s["kv_len"].long(), s["seq_len"].long()
    keep = torch.minimum((s["accepted"] + 1).clamp(min=0), seq_len - kv_len)
    done = s["finished"] != 0
    after = torch.where(done, 0, kv_len + keep)
    top = (seq_len + page - 1) // page
    base = s["free_count"].long() - (top - (kv_len + page - 1) // page).sum()
    first = (after + page - 1) // page
    back = top - first
    start = base + torch.cumsum(back, 0) - back
    column = torch.arange(table.shape[1], device=table.device)[None]
    at = torch.where((column >= first[:, None]) & (column < top[:, None]), start[:, None] + column - first[:, None], free.shape[0])
    wide = torch.cat([free, free[:1]])  # the last place takes what is not written
    wide.index_put_((at.reshape(-1),), table.reshape(-1))
    free.copy_(wide[:-1])
    s["free_count"].copy_(base + back.sum())
    s["kv_len"].copy_(after)
    return s["kv_len"], s["free_count"], free


def _rotated(x, weight, s):
    """Norm over the head where there is a weight, then the rotation; x [tokens, heads, dim] in 32 bits."""
    rot = s["case"]["rot"]
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    part = x[..., :rot]
    if s["case"]["pairs"] == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _stored(cache, x, scale, s):
    if scale is not None:
        x = (x / scale[:, None]).clamp(-448.0, 448.0)
    slots, page = s["slots"].long(), s["case"]["page"]
    x = x.to(cache.dtype)
    if scale is not None:  # by their bits: indexing does not know the 8-bit type
        cache, x = cache.view(torch.uint8), x.view(torch.uint8)
    cache[slots // page, slots % page] = x


def _rope_outputs(s):
    caches = s["k_cache"], s["v_cache"]
    if s["case"]["cache"] == "e4m3":
        caches = tuple(c.to(torch.bfloat16) for c in caches)
    return (s["q_out"],) + caches


def _rope(s):
    s["q_out"].copy_(_rotated(s["q"].float(), s["q_weight"], s))
    _stored(s["k_cache"], _rotated(s["k"].float(), s["k_weight"], s), s["k_scale"], s)
    _stored(s["v_cache"], s["v"].float(), s["v_scale"], s)
    return _rope_outputs(s)


def _gathered(cache, page, inside, scale):
    """Tokens of a cache as [rows, kv heads, tokens, dim] in 32 bits."""
    if scale is not None:
        x = cache.view(torch.uint8)[page, inside].view(cache.dtype).float() * scale[:, None]
    else:
        x = cache[page, inside].float()
    return x.transpose(1, 2)


def _attend(s):
    case = s["case"]
    rows, page, hq, hkv, d, most = case["rows"], case["page"], case["hq"], case["hkv"], case["dim"], case["new"]
    dev, window, sinks, group = s["q"].device, case["window"], case["sinks"], hq // hkv
    length, cu = s["seq_len"].long(), s["cu_new"].long()
    new = cu[1:] - cu[:-1]
    if window:  # the first tokens, then as many last ones as a window can reach
        head = min(sinks, case["longest"] + most)
        back = min(window + most - 1, case["longest"] + most)
        token = torch.cat([torch.arange(head, device=dev).expand(rows, -1), (length - back)[:, None] + torch.arange(back, device=dev)], 1)
        valid = (token >= 0) & (token < length[:, None])
        valid[:, head:] &= token[:, head:] >= head
    else:
        token = torch.arange(case["longest"] + most, device=dev).expand(rows, -1)
        valid = token < length[:, None]
    token = torch.where(valid, token, 0)
    ids = torch.gather(s["table"], 1, token // page).long()
    k = _gathered(s["k_cache"], ids, token % page, s["k_scale"])
    j = torch.arange(most, device=dev)
    take = (cu[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][take].float().view(rows, most, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(rows, hkv, most * group, d)
    score = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    position = (length - new)[:, None] + j  # of the queries
    seen = valid[:, None] & (token[:, None] <= position[..., None])
    if window:
        seen &= (token[:, None] > position[..., None] - window) | (token[:, None] < sinks)
    score = score.view(rows, hkv, most, group, -1).masked_fill_(~seen[:, None, :, None], -math.inf).view(rows, hkv, most * group, -1)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score, _gathered(s["v_cache"], ids, token % page, s["v_scale"])) / total.clamp(min=1e-37)
    out = out.view(rows, hkv, most, group, d).permute(0, 2, 1, 3, 4).reshape(rows * most, hq, d)
    row = torch.repeat_interleave(torch.arange(rows, device=dev), new, output_size=s["q"].shape[0])
    flat = row * most + torch.arange(s["q"].shape[0], device=dev) - cu[row]
    s["out"].copy_(out[flat])
    return s["out"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("append", "commit"):
        rows, tokens = case["rows"], sum(_news(case))
        turned = sum(-(-(h + n) // case["page"]) - -(-h // case["page"]) for h, n in zip(_lengths(case), _news(case)))
        if op == "append":  # lengths, offsets; slots, positions, lengths, status; a page id read for each token, new ones written
            return {"bytes": 4.0 * (rows * 4 + tokens * 3 + turned), "flops": 0.0}
        return {"bytes": 4.0 * (rows * 5 + 2 * turned + 2), "flops": 0.0}
    hq, hkv, d = case["hq"], case["hkv"], case["dim"]
    wide, held = SIZE[case["type"]], SIZE[case["cache"]]
    if op == "rope":
        t = case["tokens"]
        return {"bytes": t * ((2 * hq + 2 * hkv) * d * wide + 2 * hkv * d * held + 8.0), "flops": t * (hq + hkv) * d * 8.0}
    news = _news(case)
    seen = 0
    for h, n in zip(_lengths(case), news):
        for i in range(n):
            keys = h + i + 1
            seen += min(keys, case["window"] + min(case["sinks"], max(0, keys - case["window"]))) if case["window"] else keys
    return {"bytes": _attend_keys(case) * 2.0 * hkv * d * held + sum(news) * 2.0 * hq * d * wide, "flops": 4.0 * seen * hq * d}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    if case["op"] in ("append", "commit"):
        return None  # whole numbers: compared as they are
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    table, length, cu = s["table"].long(), s["seq_len"].tolist(), s["cu_new"].tolist()
    group, page = case["hq"] // case["hkv"], case["page"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    low = case["cache"] == "e4m3"
    for r in range(case["rows"]):
        n, total = cu[r + 1] - cu[r], length[r]
        first = total - n
        # keys that any of the row's queries sees
        t = torch.arange(total, device=DEV)
        if case["window"]:
            t = t[(t > first - case["window"]) | (t < case["sinks"])]
        where = (table[r, t // page], t % page)
        for h in range(case["hkv"]):
            k, v = s["k_cache"][:, :, h], s["v_cache"][:, :, h]
            if low:
                k = k.view(torch.uint8)[where].view(torch.float8_e4m3fn).double() * s["k_scale"][h].double()
                v = v.view(torch.uint8)[where].view(torch.float8_e4m3fn).double() * s["v_scale"][h].double()
            else:
                k, v = k[where].double(), v[where].double()
            q = s["q"][cu[r]:cu[r + 1], h * group:(h + 1) * group].double()  # n, group, d
            score = torch.einsum("ngd,td->ngt", q, k) * s["scale"]
            at = torch.arange(first, total, device=DEV)[:, None]
            visible = t[None] <= at
            if case["window"]:
                visible &= (at - t[None] < case["window"]) | (t[None] < case["sinks"])
            score[~visible[:, None].expand_as(score)] = -math.inf
            out[cu[r]:cu[r + 1], h * group:(h + 1) * group] = torch.einsum("ngt,td->ngd", torch.softmax(score, -1), v)
    return out


def _exact_rope(case, s):
    rot, page = case["rot"], case["page"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None, None] * s["inv_freq"][None, None])  # e^(i angle)

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
        y = x.clone()
        at = torch.arange(rot // 2, device=DEV)
        one, two = (at, at + rot // 2) if case["pairs"] == "half" else (2 * at, 2 * at + 1)
        z = torch.complex(x[..., one], x[..., two]) * turn
        y[..., one], y[..., two] = z.real, z.imag
        return y

    def held(cache, x, scale):
        full = torch.zeros(cache.shape, dtype=torch.float64, device=DEV)
        if scale is not None:
            x = (x / scale.double()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double()  # the held value is the rounded one
        slot = s["slots"].long()
        full[torch.div(slot, page, rounding_mode="floor"), slot.remainder(page)] = x
        return full

    return (turned(s["q"], s["q_weight"]), held(s["k_cache"], turned(s["k"], s["k_weight"]), s["k_scale"]),
            held(s["v_cache"], s["v"].double(), s["v_scale"]))
