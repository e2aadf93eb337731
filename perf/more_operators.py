"""Measured cases of the operators around an 8-bit cache with a factor for each
block of tokens and head, and of the attention over whole prompts: the store of
a step's keys and values (`ss_kv_store_blocks`), reading held tokens back
(`ss_kv_load_blocks`), the attention of a step's new tokens over such a cache
(`ss_attend_blocks`), and the causal attention of packed prompts over
themselves (`ss_attend_prompt`).

`own` chooses between the plain form of each operator in elementary torch
operations (False) and the calls of this library (True).  Both run on what
`prepare` makes.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
LOWEST, HIGHEST = -40, 40  # exponents of a block's factor


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decoding step of a small server: one token of each of 24 requests; the rest of its block may have to be scaled anew
        {"name": "store 24 x 1", "op": "store", "rows": 24, "new": 1, "longest": 1500, "hkv": 8, "dim": 128, "type": "bf16",
         "layout": "hnd", "page": 16, "block": 16},
        # a verification step of many requests with up to 7 drafts
        {"name": "store 300 x 8", "op": "store", "rows": 300, "new": 8, "longest": 700, "hkv": 4, "dim": 64, "type": "f16",
         "layout": "nhd", "page": 64, "block": 32},
        # a batch of prompts on its way into the cache
        {"name": "store 9 x 4100", "op": "store", "rows": 9, "new": 4100, "longest": 40, "hkv": 8, "dim": 128, "type": "bf16",
         "layout": "hnd", "page": 64, "block": 16},
        # a short shared beginning, read back for a request that continues it in 16 bits
        {"name": "load 500", "op": "load", "tokens": 500, "hkv": 8, "dim": 128, "type": "bf16", "layout": "hnd", "page": 16, "block": 16},
        # a long document that moves to a 16-bit cache
        {"name": "load 40000", "op": "load", "tokens": 40000, "hkv": 8, "dim": 128, "type": "bf16", "layout": "nhd", "page": 64, "block": 64},
        # one user, one token: latency
        {"name": "attend 1 x 1 blocks", "op": "attend", "rows": 1, "new": 1, "longest": 900, "hq": 32, "hkv": 8, "dim": 128,
         "type": "bf16", "layout": "hnd", "page": 16, "block": 16, "window": 0, "sinks": 0},
        # ordinary decoding over contexts of up to 12000 tokens
        {"name": "attend 80 x 1 blocks", "op": "attend", "rows": 80, "new": 1, "longest": 12000, "hq": 32, "hkv": 8, "dim": 128,
         "type": "bf16", "layout": "hnd", "page": 64, "block": 16, "window": 0, "sinks": 0},
        # verification with up to 4 drafts, 8 query heads to a key head
        {"name": "attend 40 x 5 blocks", "op": "attend", "rows": 40, "new": 5, "longest": 16000, "hq": 64, "hkv": 8, "dim": 128,
         "type": "f16", "layout": "hnd", "page": 32, "block": 32, "window": 0, "sinks": 0},
        # the first prompt of a chat
        {"name": "prompt 60", "op": "prompt", "rows": 1, "longest": 60, "hq": 32, "hkv": 8, "dim": 128, "type": "bf16", "window": 0, "sinks": 0},
        # prompts of many requests packed together, narrow heads
        {"name": "prompt 100 x 700", "op": "prompt", "rows": 100, "longest": 700, "hq": 28, "hkv": 4, "dim": 64, "type": "f16", "window": 0,
         "sinks": 0},
        # long prompts in a layer with a sliding window and first tokens that stay visible
        {"name": "prompt 5 x 9000 window", "op": "prompt", "rows": 5, "longest": 9000, "hq": 16, "hkv": 8, "dim": 256, "type": "bf16",
         "window": 1024, "sinks": 4},
        # a whole document
        {"name": "prompt 16000", "op": "prompt", "rows": 1, "longest": 16000, "hq": 32, "hkv": 8, "dim": 128, "type": "bf16", "window": 0,
         "sinks": 0},
    ]


HEADS = [(32, 8, 128), (64, 8, 128), (40, 8, 128), (28, 4, 128), (16, 16, 128), (28, 4, 64), (71, 1, 64), (32, 4, 64), (8, 1, 256), (16, 8, 256)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "store", "load", "attend", "attend", "attend", "prompt", "prompt", "prompt"])
    hq, hkv, dim = rng.choice(HEADS)
    case = {"op": op, "hkv": hkv, "dim": dim, "type": rng.choice(["bf16", "f16"])}
    if op != "prompt":
        page = rng.choice([16, 32, 64, 128])
        case.update(layout=rng.choice(["hnd", "nhd"]), page=page, block=rng.choice([b for b in (16, 32, 64, 128) if b <= page]))
    if op == "store":
        rows = _log(rng, 1, 500)
        most = 18000 * 1024 // (hkv * dim)  # tokens
        case.update(rows=rows, new=_log(rng, 1, max(1, min(8000, most // rows))), longest=_log(rng, 1, max(1, min(4000, 8 * most // rows))))
        return case
    if op == "load":
        case["tokens"] = _log(rng, 1, 40000 * 1024 // (hkv * dim))
        return case
    case["hq"] = hq
    if op == "attend":
        case.update(rows=_log(rng, 1, 256), new=rng.choice([1, 1, 2, 3, 4, 5, 6, 7, 8, 11, 16]), longest=_log(rng, 1, 100000), window=0, sinks=0)
    else:
        case.update(rows=_log(rng, 1, 200), longest=_log(rng, 1, 16000), window=0, sinks=0)
    if rng.random() < 0.3:
        case.update(window=_log(rng, 16, 5000), sinks=rng.choice([0, 1, 4, 60]))
    if op == "attend":
        # no more keys or scores than the largest listed cases, also in the plain form, whose rows are as long as the longest
        while case["rows"] * (case["longest"] + case["new"]) * max(hkv * dim / 1.0e9, hq * case["new"] / 0.2e9) > 1:
            if case["longest"] > 1:
                case["longest"] = case["longest"] * 2 // 3
            else:
                case["rows"] //= 2
    else:
        while case["rows"] > 1 and sum(_prompts(case)) * (hq + 2 * hkv) * dim > 16000 * 48 * 128:
            case["rows"] = case["rows"] * 2 // 3
        while sum(n * n for n in _prompts(case)) * hq * dim > 16000 ** 2 * 32 * 128:
            case["longest"] = case["longest"] * 2 // 3
    return case


def _lengths(case):
    """Cached tokens of each row, before its new ones: from one token to the longest, spread evenly over the square root."""
    n, longest = case["rows"], case["longest"]
    return [max(1, int(longest * ((i + 1) / n) ** 2)) - (1 if longest == 1 and i % 2 else 0) for i in range(n)]


def _news(case):
    """New tokens of each row: 1 .. new, the last rows the most."""
    return [1 + (i * 5 + case["new"] - 1) % case["new"] if i else case["new"] for i in range(case["rows"])]


def _stores(case):
    """(held, new) of each row of a store: prompts are new rows, beside a few that go on."""
    return [(0 if case["new"] > 64 and i % 3 else h, n) for i, (h, n) in enumerate(zip(_lengths(case), _news(case)))]


def _prompts(case):
    """Tokens of each prompt: from one to the longest, spread evenly over the square root."""
    n = case["rows"]
    return [max(1, int(case["longest"] * ((i + 1) / n) ** 2)) for i in range(n)]


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
        x = torch.randn(n, generator=g, device=DEV) * scale
        flat[at:at + n] = (x.clamp_(-448.0, 448.0) if dtype is E4M3 else x).to(dtype)
    return out


def _cumulative(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(n, 0)]).to(torch.int32)


def _cache(g, case, pages):
    """Held keys or values, seen as [pages, page, kv heads, dim], and their factors [pages, kv heads, blocks of a page]: values of about one."""
    hnd = case["layout"] == "hnd"
    shape = (pages, case["hkv"], case["page"], case["dim"]) if hnd else (pages, case["page"], case["hkv"], case["dim"])
    t = _normal(g, shape, E4M3, 100.0)
    exponent = torch.randint(-9, -4, (pages, case["hkv"], case["page"] // case["block"]), generator=g, device=DEV)
    return (t.transpose(1, 2) if hnd else t), torch.exp2(exponent.float())


def _table(g, length, page, spare=7):
    """Block table of rows of these lengths and the number of pages."""
    used = (length + page - 1) // page
    blocks, pages = max(1, int(used.max())), int(used.sum()) + spare
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    column = torch.arange(blocks, device=DEV)[None]
    first = (torch.cumsum(used, 0) - used)[:, None]
    return torch.where(column < used[:, None], ids[(first + column).clamp(max=pages - 1)], -1).to(torch.int32), pages


def _handle(case, rows, tokens, new, pages, blocks):
    """The plan and workspace that a program keeps."""
    from spec_verification_gb300 import kv
    plan = kv.Plan(max_rows=rows, max_tokens=tokens, max_new=new, q_heads=case.get("hq", case["hkv"]), kv_heads=case["hkv"],
                   head_dim=case["dim"], page_size=case.get("page", 16), num_pages=pages, max_blocks=blocks, dtype=case["type"],
                   cache_dtype="e4m3")
    return plan, torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)


def prepare(case, seed):
    return {"store": _prepare_store, "load": _prepare_load, "attend": _prepare_attend, "prompt": _prepare_prompt}[case["op"]](case, seed)


def _prepare_store(case, seed):
    g, page, block, hkv, d = _gen(seed), case["page"], case["block"], case["hkv"], case["dim"]
    both = torch.tensor(_stores(case), device=DEV)
    both = both[torch.randperm(case["rows"], generator=g, device=DEV)]
    held, new = both[:, 0], both[:, 1]
    length = held + new
    table, pages = _table(g, length, page)
    t = int(new.sum())
    # a projection's output: keys and values are parts of its rows; some tokens are larger than what their block holds
    kv = _normal(g, (t, 2 * hkv * d), TYPES[case["type"]])
    kv *= torch.exp2(torch.randint(-2, 3, (t, 1), generator=g, device=DEV).float()).to(kv.dtype)
    k_cache, k_scale = _cache(g, case, pages)
    v_cache, v_scale = _cache(g, case, pages)
    # slots of all tokens in the blocks that get new ones: what is read back
    first = held // block * block
    count = length - first
    row = torch.repeat_interleave(torch.arange(case["rows"], device=DEV), count)
    position = first[row] + torch.arange(int(count.sum()), device=DEV) - (torch.cumsum(count, 0) - count)[row]
    slots = table[row, position // page].long() * page + position % page
    n = slots.shape[0]
    s = {"case": case, "k": kv[:, :hkv * d].view(t, hkv, d), "v": kv[:, hkv * d:].view(t, hkv, d), "k_cache": k_cache, "v_cache": v_cache,
         "k_scale": k_scale, "v_scale": v_scale, "table": table, "kv_len": held.to(torch.int32), "seq_len": length.to(torch.int32),
         "cu_new": _cumulative(new), "slots": slots.to(torch.int32), "row_status": torch.zeros(case["rows"], dtype=torch.int32, device=DEV),
         "k_out": torch.empty(n, hkv, d, dtype=kv.dtype, device=DEV), "v_out": torch.empty(n, hkv, d, dtype=kv.dtype, device=DEV)}
    if own:
        s["plan"], s["workspace"] = _handle(case, case["rows"], n, case["new"], pages, table.shape[1])
    return s


def _prepare_load(case, seed):
    g, t, page, hkv, d = _gen(seed), case["tokens"], case["page"], case["hkv"], case["dim"]
    pages = -(-t * 5 // (4 * page)) + 1
    k_cache, k_scale = _cache(g, case, pages)
    v_cache, v_scale = _cache(g, case, pages)
    at = torch.arange(t, device=DEV)
    slots = torch.randperm(pages, generator=g, device=DEV)[at // page] * page + at % page
    s = {"case": case, "k_cache": k_cache, "v_cache": v_cache, "k_scale": k_scale, "v_scale": v_scale, "slots": slots.to(torch.int32),
         "k_out": torch.empty(t, hkv, d, dtype=TYPES[case["type"]], device=DEV), "v_out": torch.empty(t, hkv, d, dtype=TYPES[case["type"]], device=DEV)}
    if own:
        s["plan"], s["workspace"] = _handle(case, 1, t, 1, pages, 1)
    return s


def _prepare_attend(case, seed):
    g, rows, hq, d = _gen(seed), case["rows"], case["hq"], case["dim"]
    held, new = torch.tensor(_lengths(case), device=DEV), torch.tensor(_news(case), device=DEV)
    at = torch.randperm(rows, generator=g, device=DEV)
    held, new = held[at], new[at]
    length = held + new
    table, pages = _table(g, length, case["page"])
    tokens = int(new.sum())
    kind = TYPES[case["type"]]
    s = {"case": case, "q": _normal(g, (tokens, hq, d), kind, 2.0), "table": table, "seq_len": length.to(torch.int32), "cu_new": _cumulative(new),
         "scale": d ** -0.5, "out": torch.empty(tokens, hq, d, dtype=kind, device=DEV), "row_status": torch.zeros(rows, dtype=torch.int32, device=DEV)}
    s["k_cache"], s["k_scale"] = _cache(g, case, pages)
    s["v_cache"], s["v_scale"] = _cache(g, case, pages)
    if own:
        s["plan"], s["workspace"] = _handle(case, rows, tokens, case["new"], pages, table.shape[1])
    return s


def _prepare_prompt(case, seed):
    g, hq, hkv, d = _gen(seed), case["hq"], case["hkv"], case["dim"]
    lengths = _prompts(case)
    lengths = [lengths[i] for i in torch.randperm(case["rows"], generator=g, device=DEV).tolist()]
    t, kind = sum(lengths), TYPES[case["type"]]
    qkv = _normal(g, (t, (hq + 2 * hkv) * d), kind, 1.2)  # one projection's output: q, k and v are parts of its rows
    s = {"case": case, "q": qkv[:, :hq * d].view(t, hq, d), "k": qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
         "v": qkv[:, (hq + hkv) * d:].view(t, hkv, d), "cu_seq": _cumulative(torch.tensor(lengths, device=DEV)), "lengths": lengths,
         "scale": d ** -0.5, "out": torch.empty(t, hq, d, dtype=kind, device=DEV),
         "row_status": torch.zeros(case["rows"], dtype=torch.int32, device=DEV)}
    if own:
        s["plan"], s["workspace"] = _handle(case, case["rows"], t, 1, 1, 1)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op, case = s["case"]["op"], s["case"]
    if own:
        from spec_verification_gb300 import kv
        if op == "prompt":
            kv.ss_attend_prompt(s["plan"], s["q"], s["k"], s["v"], s["cu_seq"], out=s["out"], row_status=s["row_status"], workspace=s["workspace"],
                                scale=s["scale"], window=case["window"], sinks=case["sinks"])
            return s["out"]
        cache = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        if op == "attend":
            kv.ss_attend_blocks(s["plan"], s["q"], *cache, s["table"], s["seq_len"], s["cu_new"], out=s["out"], row_status=s["row_status"],
                                workspace=s["workspace"], scale=s["scale"], window=case["window"], sinks=case["sinks"])
            return s["out"]
        if op == "store":
            kv.ss_kv_store_blocks(s["plan"], s["k"], s["v"], *cache, s["table"], s["kv_len"], s["seq_len"], s["cu_new"],
                                  row_status=s["row_status"])
        kv.ss_kv_load_blocks(s["plan"], *cache, s["slots"], k_out=s["k_out"], v_out=s["v_out"])
    elif op == "prompt":
        return _prompt(s)
    elif op == "attend":
        return _attend(s)
    else:
        if op == "store":
            _store(s)
        for name in "kv":
            s[name + "_out"].copy_(_read(s[name + "_cache"], s[name + "_scale"], s["slots"].long(), case))
    return (s["k_out"], s["v_out"], s["k_scale"], s["v_scale"]) if op == "store" else (s["k_out"], s["v_out"])


def _read(cache, scale, slots, case):
    """Held values of tokens, [tokens, kv heads, dim] in 32 bits."""
    page, place = slots // case["page"], slots % case["page"]
    # by their bits: indexing does not know the 8-bit type
    return cache.view(torch.uint8)[page, place].view(E4M3).float() * scale[page, :, place // case["block"]][..., None]


def _store(s):
    """New tokens into the cache; blocks that they start or outgrow get another factor."""
    case = s["case"]
    page, block, hkv = case["page"], case["block"], case["hkv"]
    per = page // block
    held, cu, t = s["kv_len"].long(), s["cu_new"].long(), s["k"].shape[0]
    row = torch.repeat_interleave(torch.arange(case["rows"], device=DEV), cu[1:] - cu[:-1], output_size=t)
    position = held[row] + torch.arange(t, device=DEV) - cu[row]
    place = position % page
    id = s["table"][row, position // page].long() * per + place // block  # block among all of the cache
    # the block that each row goes on in: what it held before the call keeps its place
    last = held // block * block
    kept_page = s["table"].gather(1, (last // page)[:, None]).long()
    kept_place = (last % page)[:, None] + torch.arange(block, device=DEV)
    nth = last % page // block
    count = s["k_scale"].shape[0] * per
    touched = torch.zeros(count, dtype=torch.bool, device=DEV).index_fill_(0, id, True).view(-1, 1, per)
    begun = (torch.zeros(count, dtype=torch.int32, device=DEV).index_add_(0, id, (position % block == 0).int()) > 0).view(-1, 1, per)
    for name in "kv":
        x, raw, scale = s[name].float(), s[name + "_cache"].view(torch.uint8), s[name + "_scale"]
        top = torch.zeros(count, hkv, device=DEV).scatter_reduce_(0, id[:, None].expand(t, hkv), x.abs().amax(-1), "amax")
        part, exponent = torch.frexp(top)  # the least exponent e with top <= 448 2^e
        need = torch.exp2((exponent - 9 + (part > 0.875)).clamp(LOWEST, HIGHEST).float())
        need = torch.where(top > 0, need, 2.0 ** LOWEST).view(-1, per, hkv).transpose(1, 2)
        after = torch.where(begun, need, torch.maximum(scale, need))
        after = torch.where(touched, after, scale)
        ratio = scale[kept_page[:, 0], :, nth] / after[kept_page[:, 0], :, nth]  # rows, heads
        old = raw[kept_page, kept_place].view(E4M3).float() * ratio[:, None, :, None]
        raw[kept_page, kept_place] = old.to(E4M3).view(torch.uint8)  # of a block that is begun, its new tokens come over it
        factor = after.transpose(1, 2).reshape(-1, hkv)[id]
        raw[id // per, place] = (x / factor[..., None]).to(E4M3).view(torch.uint8)
        scale.copy_(after)


def _gathered(cache, scale, page, inside, case):
    """Tokens of a cache as [rows, kv heads, tokens, dim] in 32 bits."""
    x = cache.view(torch.uint8)[page, inside].view(E4M3).float() * scale[page, :, inside // case["block"]][..., None]
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
    k = _gathered(s["k_cache"], s["k_scale"], ids, token % page, case)
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
    out = torch.matmul(score, _gathered(s["v_cache"], s["v_scale"], ids, token % page, case)) / total.clamp(min=1e-37)
    out = out.view(rows, hkv, most, group, d).permute(0, 2, 1, 3, 4).reshape(rows * most, hq, d)
    row = torch.repeat_interleave(torch.arange(rows, device=dev), new, output_size=s["q"].shape[0])
    flat = row * most + torch.arange(s["q"].shape[0], device=dev) - cu[row]
    s["out"].copy_(out[flat])
    return s["out"]


def _prompt(s):
    """Prompt after prompt, as many queries at a time as 2^28 scores allow; each over the keys that any of them sees."""
    case = s["case"]
    hq, hkv, d, window, sinks = case["hq"], case["hkv"], case["dim"], case["window"], case["sinks"]
    group, at = hq // hkv, 0
    for n in s["lengths"]:
        q, k, v = (s[x][at:at + n].float().transpose(0, 1) for x in "qkv")  # heads, tokens, dim
        step = max(1, min(n, (1 << 28) // (hq * n)))
        for i in range(0, n, step):
            end = min(n, i + step)
            first = max(0, i - window + 1) if window else 0
            head = min(sinks, first) if window else 0
            token = torch.cat([torch.arange(head, device=DEV), torch.arange(first, end, device=DEV)])
            keys, values = (torch.cat([x[:, :head], x[:, first:end]], 1) if head else x[:, first:end] for x in (k, v))
            query = q[:, i:end].reshape(hkv, group * (end - i), d)
            score = torch.matmul(query, keys.transpose(1, 2)) * s["scale"]
            position = torch.arange(i, end, device=DEV)[:, None]
            seen = token <= position
            if window:
                seen &= (token > position - window) | (token < sinks)
            score = score.view(hkv, group, end - i, -1).masked_fill_(~seen, -math.inf).view(hkv, group * (end - i), -1)
            score = score.sub_(score.amax(-1, keepdim=True)).exp_()
            out = torch.matmul(score, values) / score.sum(-1, keepdim=True)
            s["out"][at + i:at + end] = out.view(hq, end - i, d).transpose(0, 1)
        at += n
    return s["out"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    hkv, d = case["hkv"], case["dim"]
    if case["op"] == "load":
        return {"bytes": case["tokens"] * 2.0 * hkv * (d * 3.0 + 4.0 / case["block"]) + 4.0 * case["tokens"], "flops": case["tokens"] * 2.0 * hkv * d}
    if case["op"] == "store":  # keys and values in, held, with what their blocks held before; read back; factors
        block = case["block"]
        new = sum(n for _, n in _stores(case))
        kept = sum(h % block for h, _ in _stores(case))
        blocks = sum(-(-(h + n) // block) - h // block for h, n in _stores(case))
        return {"bytes": 2.0 * hkv * d * (new * 3.0 + kept + (new + kept) * 3.0) + 16.0 * hkv * blocks + 4.0 * (new + kept),
                "flops": 4.0 * hkv * d * (new + kept)}
    hq, window, sinks = case["hq"], case["window"], case["sinks"]
    keys = pairs = queries = 0
    rows = [(0, n) for n in _prompts(case)] if case["op"] == "prompt" else zip(_lengths(case), _news(case))
    for h, n in rows:
        queries += n
        keys += min(h + n, window + n - 1 + min(sinks, h + n)) if window else h + n
        if not window:
            pairs += n * h + n * (n + 1) // 2
        else:
            full = window + sinks  # a query at position p sees min(p + 1, window) + min(sinks, max(0, p + 1 - window))
            short = max(0, min(n, full - h))  # queries that see everything before them
            pairs += short * h + short * (short + 1) // 2 + (n - short) * full
    held = 1.0 if case["op"] == "attend" else 2.0
    factors = keys * 2.0 * hkv * 4.0 / case["block"] if case["op"] == "attend" else 0.0
    return {"bytes": keys * 2.0 * hkv * d * held + factors + queries * 4.0 * hq * d, "flops": 4.0 * pairs * hq * d}


# ------------------------------------------------------------------ the definition, in 64 bits
def _decoded(bits):
    """e4m3 from its bits: sign, four bits of exponent, three of fraction."""
    bits = bits.long()
    exponent, fraction = (bits >> 3) & 15, bits & 7
    size = torch.where(exponent == 0, fraction.double() / 8 * 2.0 ** -6, (1 + fraction.double() / 8) * torch.exp2(exponent.double() - 7))
    return torch.where(bits >= 128, -size, size)


def _rounded(y):
    """To the nearest multiple of e4m3's step at y, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (y / step).round().mul(step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("load", "store"):
        if case["op"] == "store":
            return _exact_store(case, s)
        page, place = s["slots"].long() // case["page"], s["slots"].long() % case["page"]
        return tuple(_decoded(s[n + "_cache"].view(torch.uint8)[page, place]) * s[n + "_scale"].double()[page, :, place // case["block"]].unsqueeze(-1)
                     for n in "kv")
    group, q = case["hq"] // case["hkv"], s["q"]
    out = torch.empty(q.shape, dtype=torch.float64, device=DEV)
    cu = (s["cu_seq"] if case["op"] == "prompt" else s["cu_new"]).tolist()
    for r in range(case["rows"]):
        n = cu[r + 1] - cu[r]
        total = n if case["op"] == "prompt" else int(s["seq_len"][r])
        for h in range(case["hkv"]):
            if case["op"] == "prompt":
                k, v = s["k"][cu[r]:cu[r + 1], h].double(), s["v"][cu[r]:cu[r + 1], h].double()
            else:
                t = torch.arange(total, device=DEV)
                page, place = s["table"][r, t // case["page"]].long(), t % case["page"]
                k, v = (_decoded(s[x + "_cache"].view(torch.uint8)[:, :, h][page, place]) * s[x + "_scale"].double()[page, h, place // case["block"]][:, None]
                        for x in "kv")
            for i in range(0, n, 1024):  # queries i .. j at positions i + total - n ..
                j = min(n, i + 1024)
                p0 = total - n + i
                lo = max(0, p0 - case["window"] + 1) if case["window"] else 0
                t = torch.arange(total - n + j, device=DEV)
                t = t[(t >= lo) | (t < case["sinks"])]
                p = torch.arange(p0, total - n + j, device=DEV)[:, None]
                visible = t[None] <= p
                if case["window"]:
                    visible &= (p - t[None] < case["window"]) | (t[None] < case["sinks"])
                x = q[cu[r] + i:cu[r] + j, h * group:(h + 1) * group].double()
                score = torch.einsum("ngd,td->gnt", x, k[t]) * s["scale"]
                score.masked_fill_(~visible, -math.inf)
                out[cu[r] + i:cu[r] + j, h * group:(h + 1) * group] = torch.einsum("gnt,td->ngd", torch.softmax(score, -1), v[t])
    return out


def _exact_store(case, s):
    """Row by row: the blocks that its new tokens reach, what they held before, and their factors."""
    block, page = case["block"], case["page"]
    scales = {n: s[n + "_scale"].double() for n in "kv"}
    outs = {"k": [], "v": []}
    cu, held, table = s["cu_new"].tolist(), s["kv_len"].tolist(), s["table"].long()
    for r in range(case["rows"]):
        first = held[r] // block * block
        kept, n = held[r] - first, cu[r + 1] - cu[r]
        blocks = -(-(kept + n) // block)
        at = first + block * torch.arange(blocks, device=DEV)
        pages, nth = table[r, at // page], at % page // block
        for name in "kv":
            values = torch.zeros(blocks * block, case["hkv"], case["dim"], dtype=torch.float64, device=DEV)
            values[kept:kept + n] = s[name][cu[r]:cu[r + 1]].double()
            top = values.view(blocks, block, case["hkv"], case["dim"]).abs().amax((1, 3))
            exponent = torch.ceil(torch.log2(top / 448)).clamp(LOWEST, HIGHEST)  # -inf where all are zero
            exponent += (torch.exp2(exponent) * 448 < top).double() * (exponent < HIGHEST)
            exponent -= (torch.exp2(exponent - 1) * 448 >= top).double() * (exponent > LOWEST)
            factor = torch.exp2(exponent)
            before = scales[name][pages, :, nth]
            if kept:
                factor[0] = torch.maximum(factor[0], before[0])
            full = factor.repeat_interleave(block, 0)[..., None]
            result = _rounded(values / full) * full
            if kept:
                place = at[0] % page + torch.arange(kept, device=DEV)
                old = _decoded(s[name + "_cache"].view(torch.uint8)[pages[0], place])
                result[:kept] = _rounded(old * (before[0] / factor[0])[None, :, None]) * factor[0][None, :, None]
            scales[name][pages, :, nth] = factor
            outs[name].append(result[:kept + n])
    return torch.cat(outs["k"]), torch.cat(outs["v"]), scales["k"], scales["v"]
