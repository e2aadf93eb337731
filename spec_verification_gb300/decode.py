"""A small speculative-decoding loop that uses the library's calls together.

`python -m spec_verification_gb300.decode` decodes a batch of random prompts
with a random-weight transformer: prompts go through ss_kv_append,
ss_rope_store and ss_attend like any other new tokens, drafts come from the
row's own text (the tokens that followed the last occurrence of its latest
token), ss_verify accepts a prefix of them and adds a token, and ss_kv_commit
keeps exactly what was accepted.  With an 8-bit cache whose blocks have factors
of their own, prompts are attended as they come from the projection
(ss_attend_prompt) while their keys and values are quantised into the cache
(ss_kv_store_blocks), which the steps then read (ss_attend_blocks).  Only the
matrix products, embeddings and activations are torch's.
"""
from __future__ import annotations

import argparse
import time

import numpy as np
import torch

from . import kv, native
from . import workloads as W


class Model:
    """Random weights of a decoder: per layer qkv and output projections, a gated feed-forward pair, norms."""

    def __init__(self, vocab=8000, layers=2, width=512, q_heads=8, kv_heads=2, head_dim=64, dtype="bf16", device="cuda:0", seed=0,
                 rope_base=10000.0):
        g = torch.Generator(device=device).manual_seed(seed)
        t = kv._TORCH[dtype]
        self.vocab, self.width, self.q_heads, self.kv_heads, self.head_dim = vocab, width, q_heads, kv_heads, head_dim
        self.dtype, self.device = dtype, torch.device(device)

        def w(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device=device) * scale / shape[-1] ** 0.5).to(t)

        heads = q_heads + 2 * kv_heads
        self.embed = w(vocab, width, scale=width ** 0.5)
        self.layers = [dict(qkv=w(heads * head_dim, width), out=w(width, q_heads * head_dim), up=w(4 * width, width), down=w(width, 2 * width),
                            q_norm=(1 + 0.1 * torch.randn(head_dim, generator=g, device=device)).to(t),
                            k_norm=(1 + 0.1 * torch.randn(head_dim, generator=g, device=device)).to(t)) for _ in range(layers)]
        self.inv_freq = torch.tensor(kv.rope_frequencies(head_dim, rope_base), device=device)

    @staticmethod
    def norm(x):
        y = x.float()
        return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def feed_forward(self, layer, x):
        a, b = (self.norm(x) @ layer["up"].T).chunk(2, -1)
        return x + (torch.nn.functional.silu(a.float()).to(x.dtype) * b) @ layer["down"].T


class Decoder:
    """A batch of requests: their pages and lengths on the device, one cache per layer, the plans and workspaces."""

    def __init__(self, model: Model, rows: int, max_tokens: int, max_drafts: int = 4, page_size: int = 16, num_pages: int | None = None,
                 cache_dtype: str | None = None, greedy: bool = True, seed: int = 0, block_tokens: int = 0):
        """block_tokens: of an e4m3 cache, tokens of a block with a factor of its own (0: none, every value is held as it is)."""
        self.model, self.rows, self.max_drafts = model, rows, max_drafts
        dev, i32 = model.device, torch.int32
        blocks = -(-(max_tokens + max_drafts + 1) // page_size)
        pages = num_pages or rows * blocks
        self.plan = kv.Plan(max_rows=rows, max_tokens=rows * max_tokens, max_new=max_drafts + 1, q_heads=model.q_heads,
                            kv_heads=model.kv_heads, head_dim=model.head_dim, page_size=page_size, num_pages=pages, max_blocks=blocks,
                            dtype=model.dtype, cache_dtype=cache_dtype, device=dev.index or 0)
        self.workspace = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device=dev)
        shape = (2, pages, model.kv_heads, page_size, model.head_dim)
        self.caches = [torch.zeros(shape, device=dev).to(self.plan.cache_type).transpose(2, 3) for _ in model.layers]
        self.factors = None
        if block_tokens:
            if self.plan.cache_dtype != "e4m3" or page_size % block_tokens:
                raise ValueError("blocks with factors belong to an e4m3 cache whose pages they divide")
            self.factors = [torch.zeros(2, pages, model.kv_heads, page_size // block_tokens, device=dev) for _ in model.layers]
            # rotated keys (and values) of a step in a row, on their way into the cache: 16-bit pages that follow one another
            self.most = rows * max_tokens
            self.rope_plan = kv.Plan(max_rows=1, max_tokens=self.most, q_heads=model.q_heads, kv_heads=model.kv_heads, head_dim=model.head_dim,
                                     page_size=16, num_pages=-(-self.most // 16), max_blocks=1, dtype=model.dtype, device=dev.index or 0)
            self.rotated = torch.empty((2,) + tuple(self.rope_plan.cache_shape), dtype=self.rope_plan.type, device=dev)
            self.in_order = torch.arange(self.most, dtype=i32, device=dev)
        self.block_table = torch.full((rows, blocks), -1, dtype=i32, device=dev)
        self.kv_len = torch.zeros(rows, dtype=i32, device=dev)
        self.begun = False  # does a row hold tokens?
        self.free_pages = torch.arange(pages, dtype=i32, device=dev)
        self.free_count = torch.tensor([pages], dtype=i32, device=dev)
        self.seq_len = torch.zeros(rows, dtype=i32, device=dev)
        self.status = torch.zeros(rows, dtype=i32, device=dev)
        # verification: at most max_drafts + 1 positions to a row
        positions = rows * (max_drafts + 1)
        self.verify = native.Plan(model.vocab, rows, positions, model.dtype if model.dtype == "bf16" else "f32", "f32", 0, dev.index or 0)
        self.verify_workspace = torch.zeros(self.verify.workspace_bytes, dtype=torch.uint8, device=dev)
        params = np.zeros(rows, native.ROW_DTYPE)
        params["flags"] = W.GREEDY if greedy else W.TOPP
        params["temperature"], params["top_p"], params["rep"] = 1.0, 0.9, 1.0
        self.params = torch.from_numpy(params.view(np.uint8).reshape(rows, -1).copy()).to(dev)
        self.seeds = torch.arange(rows, dtype=torch.int64, device=dev) * 7919 + seed
        self.tokens = torch.full((rows, max_drafts + 1), -1, dtype=i32, device=dev)
        self.accepted = torch.zeros(rows, dtype=i32, device=dev)
        self.verify_status = torch.zeros(rows, dtype=i32, device=dev)

    def _attention(self, i: int, q, k, v, cu, slots, positions, whole: bool):
        """Layer i's keys and values into the cache, and its attention of the new tokens."""
        m, (k_cache, v_cache) = self.model, self.caches[i]
        layer, n, d = m.layers[i], q.shape[0], m.head_dim
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        norms = dict(q_weight=layer["q_norm"], k_weight=layer["k_norm"])
        after = dict(out=out, row_status=self.status, workspace=self.workspace, scale=d ** -0.5)
        if self.factors is None:
            kv.ss_rope_store(self.plan, q, k, v, k_cache, v_cache, m.inv_freq, positions, slots, q_out=q, **norms)
            kv.ss_attend(self.plan, q, k_cache, v_cache, self.block_table, self.seq_len, cu, **after)
            return out
        kv.ss_rope_store(self.rope_plan, q, k, v, *self.rotated, m.inv_freq, positions, self.in_order[:n], q_out=q, **norms)
        k, v = (x.view(-1, m.kv_heads, d)[:n] for x in self.rotated)
        cache = (k_cache, v_cache, *self.factors[i])
        kv.ss_kv_store_blocks(self.plan, k, v, *cache, self.block_table, self.kv_len, self.seq_len, cu, row_status=self.status)
        if whole:
            kv.ss_attend_prompt(self.plan, q, k, v, cu, **after)
        else:
            kv.ss_attend_blocks(self.plan, q, *cache, self.block_table, self.seq_len, cu, **after)
        return out

    def forward(self, new: list, whole: bool = False) -> tuple:
        """Runs the rows' new tokens (a list of token lists) through the model: their hidden states, and cu_new.  whole: they are
        all that the rows have, so that nothing is to be read from the cache."""
        m, dev = self.model, self.model.device
        tokens = torch.tensor([t for row in new for t in row], dtype=torch.int64, device=dev)
        cu = torch.tensor(np.concatenate([[0], np.cumsum([len(r) for r in new])]), dtype=torch.int32, device=dev)
        n = tokens.shape[0]
        slots, positions = torch.empty(n, dtype=torch.int32, device=dev), torch.empty(n, dtype=torch.int32, device=dev)
        kv.ss_kv_append(self.plan, self.block_table, self.kv_len, self.free_pages, self.free_count, cu, slots=slots, positions=positions,
                        seq_len=self.seq_len, row_status=self.status)
        x = m.embed[tokens]
        hq, hkv, d = m.q_heads, m.kv_heads, m.head_dim
        for i, layer in enumerate(m.layers):
            qkv = m.norm(x) @ layer["qkv"].T
            q, k, v = (part.view(n, heads, d) for part, heads in zip(qkv.split([hq * d, hkv * d, hkv * d], 1), (hq, hkv, hkv)))
            out = self._attention(i, q, k, v, cu, slots, positions, whole)
            x = x + out.view(n, hq * d) @ layer["out"].T
            x = m.feed_forward(layer, x)
        return m.norm(x), cu

    @staticmethod
    def _check(status):
        bad = status.tolist()
        if any(bad):
            raise RuntimeError(f"row status {[hex(b) for b in bad]}")

    def prompt(self, prompts: list):
        """Caches all tokens of the prompts but the last of each, which the first step takes.  Where a prompt does not fit
        its table row or the free pages, nothing is kept of any."""
        self.forward([p[:-1] for p in prompts], whole=not self.begun)
        self._check(self.status)  # the next append writes it anew
        kv.ss_kv_commit(self.plan, self.block_table, self.kv_len, self.free_pages, self.free_count, self.seq_len)
        self.begun = True

    def step(self, last: list, drafts: list, finished=None) -> list:
        """One step: each row's last token and its drafts go in, the tokens it gains come out (accepted drafts and one more)."""
        hidden, cu = self.forward([[t] + d for t, d in zip(last, drafts)])
        self.begun = True
        logits = torch.nn.functional.pad(hidden @ self.model.embed.T, (0, -self.model.vocab % 8))  # rows on 16-byte boundaries
        if self.model.dtype != "bf16":
            logits = logits.float()
        dev = self.model.device
        cu_draft = cu - torch.arange(self.rows + 1, dtype=torch.int32, device=dev)
        flat = [t for d in drafts for t in d] or [0]
        draft_ids = torch.tensor(flat, dtype=torch.int32, device=dev)
        self.params.view(torch.int32)[:, 10] = self.kv_len  # the random numbers' position
        native.ss_verify(self.verify, logits, None, draft_ids, self.params, cu_draft, self.seeds, workspace=self.verify_workspace,
                         tokens=self.tokens, num_accepted=self.accepted, row_status=self.verify_status, B=self.rows)
        done = None if finished is None else torch.tensor(finished, dtype=torch.int32, device=dev)
        kv.ss_kv_commit(self.plan, self.block_table, self.kv_len, self.free_pages, self.free_count, self.seq_len, counts=self.accepted,
                        plus=1, finished=done)
        self._check(self.status | self.verify_status)
        return [row[:n + 1] for row, n in zip(self.tokens.tolist(), self.accepted.tolist())]


def look_up(text: list, most: int) -> list:
    """Drafts from a row's own text: what followed the last earlier occurrence of its latest token."""
    for i in range(len(text) - 2, -1, -1):
        if text[i] == text[-1]:
            return text[i + 1:i + 1 + most]
    return []


def generate(decoder: Decoder, prompts: list, steps: int, draft=look_up) -> tuple:
    """Texts after `steps` steps and how many tokens each row gained."""
    texts = [list(p) for p in prompts]
    decoder.prompt(prompts)
    for _ in range(steps):
        drafts = [draft(t, decoder.max_drafts) for t in texts]
        gained = decoder.step([t[-1] for t in texts], drafts)
        for t, g in zip(texts, gained):
            t.extend(g)
    return texts, [len(t) - len(p) for t, p in zip(texts, prompts)]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--cache", choices=["bf16", "e4m3"], default="bf16")
    ap.add_argument("--block-tokens", type=int, default=0, help="of an e4m3 cache: tokens of a block with a factor of its own")
    a = ap.parse_args()
    rng = np.random.default_rng(0)
    model = Model()
    prompts = [rng.integers(0, 50, rng.integers(2, a.prompt + 1)).tolist() for _ in range(a.rows)]
    decoder = Decoder(model, a.rows, a.prompt + a.steps * (a.drafts + 1), a.drafts, cache_dtype=a.cache, block_tokens=a.block_tokens)
    torch.cuda.synchronize()
    t = time.perf_counter()
    texts, gained = generate(decoder, prompts, a.steps)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.rows} rows, {a.steps} steps, {sum(gained)} tokens in {t:.3f} s; tokens per row and step {sum(gained) / a.rows / a.steps:.2f}; "
          f"pages free {decoder.free_count.item()} of {decoder.plan.num_pages}")


if __name__ == "__main__":
    main()
