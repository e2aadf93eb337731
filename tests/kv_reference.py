"""Plain forms of the KV-cache operators for the tests: loops over rows for the
page bookkeeping, 64-bit torch for the arithmetic."""
import math

import torch


def append(table, kv_len, free, count, cu, page, max_blocks, num_pages, max_tokens):
    """Lists in, lists out: (table, slots, positions, seq_len, status)."""
    table, used = [list(r) for r in table], 0
    slots, positions, seq, status = [], [], [], []
    for r, held in enumerate(kv_len):
        n = cu[r + 1] - cu[r]
        if cu[r] < 0 or n < 0 or cu[r + 1] > max_tokens or held < 0 or held > max_blocks * page:
            seq.append(held)
            status.append(1 << 4)
            for j in range(max(0, min(cu[r + 1], max_tokens) - max(cu[r], 0))):
                slots.append(-1)
                positions.append(j)
            continue
        old, want = -(-held // page), -(-(held + n) // page)
        st = 0
        if want > max_blocks:
            st = 1 << 12
        else:
            need = want - old
            if need and used + need > count:
                st = 1 << 11
            else:
                for b in range(old, want):
                    table[r][b] = free[count - 1 - used - (b - old)]
            used += need
        for j in range(n):
            pos = held + j
            positions.append(pos)
            if st & ~(1 << 13):
                slots.append(-1)
                continue
            p = table[r][pos // page]
            if not 0 <= p < num_pages:
                st |= 1 << 13
                slots.append(-1)
            else:
                slots.append(p * page + pos % page)
        seq.append(held if st & ~(1 << 13) else held + n)
        status.append(st)
    return table, slots, positions, seq, status


def commit(table, kv_len, free, count, seq, page, counts, plus, finished):
    """(kv_len, free, count)"""
    free, kv_len = list(free), list(kv_len)
    reserved = sum(-(-s // page) - -(-h // page) for s, h in zip(seq, kv_len))
    at = count - reserved
    for r, held in enumerate(kv_len):
        new = seq[r] - held
        keep = new if counts is None else max(0, min(counts[r] + plus, new))
        after = 0 if finished is not None and finished[r] else held + keep
        for b in range(-(-after // page), -(-seq[r] // page)):
            free[at] = table[r][b]
            at += 1
        kv_len[r] = after
    return kv_len, free, at


def rope(x, weight, positions, inv_freq, interleaved, eps=1e-6, scale=1.0):
    """x [tokens, heads, dim] -> 64-bit."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    if inv_freq is None:
        return x
    rot = 2 * len(inv_freq)
    angle = positions.double()[:, None, None] * inv_freq
    cos, sin = torch.cos(angle) * scale, torch.sin(angle) * scale
    out = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out


def attend(q, k, v, first, scale, window=0, sinks=0, hidden=None):
    """One row: q [n, hq, d], k and v [tokens, hkv, d] in 64 bits, `first` the position of its first query, hidden a set
    of tokens that nobody sees.  Returns out, lse and, for the bounds, sum w |v| / sum w, sum |v| / sum w (w = 1 at
    the largest score) and the largest sum |q k| scale."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    weighted, plain, size = torch.zeros_like(out), torch.zeros_like(out), torch.zeros_like(lse)
    for j in range(n):
        p = first + j
        see = [t for t in range(min(p + 1, k.shape[0])) if (not window or t > p - window or t < sinks) and
               (hidden is None or t not in hidden)]
        if p < 0 or not see:
            continue
        kk, vv = k[see].repeat_interleave(g, 1), v[see].repeat_interleave(g, 1)
        s = torch.einsum("hd,thd->ht", q[j], kk) * scale
        size[j] = torch.einsum("hd,thd->ht", q[j].abs(), kk.abs()).amax(1) * scale
        top = s.amax(1, keepdim=True)
        w = torch.exp(s - top)
        z = w.sum(1)
        out[j] = torch.einsum("ht,thd->hd", w, vv) / z[:, None]
        weighted[j] = torch.einsum("ht,thd->hd", w, vv.abs()) / z[:, None]
        plain[j] = vv.abs().sum(0) / z[:, None]
        lse[j] = top[:, 0] + torch.log(z)
    return out, lse, weighted, plain, size
