"""Serve requests with different LoRA adapters from one pool: adapters and the 8-bit KV cache side by side.

    python examples/serve.py

A stack of attention layers with random weights takes requests as an iteration-level scheduler
hands them out: each iteration holds the prompts that joined and one new token of every request
that is running, each with its own adapter.  Per layer and iteration:

    q, k, v = x W + the adapters' deltas     slora_lora_apply_multi
    rotation; k and v to the cache's pages   slora_kv_append
    attention over the pages                 slora_kv_attend
    x += attention W_o + its delta           slora_lora_apply_multi

Adapter rows and KV blocks are pages of one pool.  KV blocks are taken as sequences grow, evicting
adapters that no running request holds where the free list is short, and go back when a request
ends.  One cache serves all layers: a block's scale belongs to its page, and each layer has pages
of its own in its block table.
"""
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import rank_delta_paged_gb300 as rdp  # noqa: E402

NO_PAGE = -1


class Request:
    def __init__(self, name: str, adapter: int, prompt: torch.Tensor, n_new: int):
        self.name, self.adapter, self.prompt, self.n_new = name, adapter, prompt, n_new
        self.length = 0                  # tokens in the cache
        self.blocks = []                 # per block: int32 [layers][n_heads][2]
        self.x = prompt                  # fp16 [n][hidden]: what the next iteration runs
        self.outputs = []


class Server:
    """n_layers attention layers over hidden channels in heads of head_dim, with max_adapters adapters."""

    def __init__(self, hidden=1024, head_dim=64, n_layers=2, num_pages=8192, max_adapters=8, ranks=(8, 16, 32),
                 max_positions=4096, fmt=rdp.SLORA_KV_E4M3, seed=0):
        self.hidden, self.head_dim, self.n_layers = hidden, head_dim, n_layers
        self.n_heads = hidden // head_dim
        rng = np.random.default_rng(seed)
        self.pool = rdp.slora_pool_create(0, hidden, num_pages, 4 * n_layers, max_adapters, seed)
        self.kv = rdp.slora_kv_create(self.pool, self.n_heads, head_dim, fmt)
        self.block = rdp.slora_kv_block_tokens(self.kv)
        for a in range(max_adapters):    # A^T and B rows fp16 [4 n_layers][rank][hidden], in the pinned host store
            rank = ranks[a % len(ranks)]
            at, b = (rng.normal(0, 0.02, (4 * n_layers, rank, hidden)).astype(np.float16).view(np.uint16)
                     for _ in range(2))
            rdp.slora_adapter_register(self.pool, a, rank, 2.0, at, b)
        w = rng.normal(0, hidden ** -0.5, (n_layers, 4, hidden, hidden)).astype(np.float16)
        self.w = torch.from_numpy(w).cuda()
        angle = np.arange(max_positions)[:, None] * 10000.0 ** (-np.arange(0, head_dim, 2) / head_dim)
        cos, sin = (torch.from_numpy(f(angle).astype(np.float32)).cuda() for f in (np.cos, np.sin))
        self.rope = rdp.KVRope(head_dim, False, max_positions, cos, sin)
        self.running = []

    def submit(self, r: Request) -> None:
        rdp.slora_adapters_acquire(self.pool, [r.adapter])     # loads it if need be, and holds it
        self.running.append(r)

    def finish(self, r: Request) -> None:
        for pages in r.blocks:
            rdp.slora_pages_free(self.pool, pages.size, pages)
        rdp.slora_adapters_release(self.pool, [r.adapter])
        self.running.remove(r)

    def _grow(self, r: Request, length: int) -> None:
        while len(r.blocks) * self.block < length:
            pages = np.empty((self.n_layers, self.n_heads, 2), np.int32)
            rdp.slora_pages_alloc_evict(self.pool, pages.size, pages)
            r.blocks.append(pages)

    def attend(self, layer: int, batch: rdp.KVBatch, q, k, v):
        """The layer's append and attention; q, k, v fp16 [T][hidden]."""
        out = torch.empty_like(q)
        h = self.hidden
        rdp.slora_kv_append(self.kv, batch, k, h, v, h, q, h, q, h, self.n_heads, self.rope)
        rdp.slora_kv_attend(self.kv, batch, q, h, self.n_heads, out, h, softmax_scale=self.head_dim ** -0.5)
        return out

    def step(self) -> int:
        """One iteration over the running requests; returns its tokens."""
        # prompts first: the deltas take them as segments, the single tokens behind them by their adapter
        order = sorted(self.running, key=lambda r: len(r.x) == 1)
        n = [len(r.x) for r in order]
        prompts = sum(m > 1 for m in n)
        indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        for r, m in zip(order, n):
            self._grow(r, r.length + m)
        max_blocks = max(len(r.blocks) for r in order)
        table = np.full((self.n_layers, len(order), max_blocks, self.n_heads, 2), NO_PAGE, np.int32)
        for s, r in enumerate(order):
            table[:, s, :len(r.blocks)] = np.stack(r.blocks, axis=1)
        lengths = np.array([r.length + m for r, m in zip(order, n)], np.int32)
        table, d_indptr, lengths, idx = (
            torch.from_numpy(a).cuda()
            for a in (table, indptr, lengths, np.repeat([r.adapter for r in order], n).astype(np.int32)))
        x, t = torch.cat([r.x for r in order]), int(indptr[-1])
        seg = d_indptr[:prompts + 1] if prompts else None
        for layer in range(self.n_layers):
            batch = rdp.KVBatch(t, len(order), max(n), max_blocks, d_indptr, lengths, table[layer])
            xn = torch.nn.functional.rms_norm(x, (self.hidden,))
            w = self.w[layer]
            qkv = [xn @ w[j] for j in range(3)]
            rdp.slora_lora_apply_multi(self.pool, [4 * layer + j for j in range(3)], [xn] * 3, qkv, t, idx, seg, prompts)
            a = self.attend(layer, batch, *qkv)
            o = a @ w[3]
            rdp.slora_lora_apply_multi(self.pool, [4 * layer + 3], [a], [o], t, idx, seg, prompts)
            x = x + o
        for s, (r, m) in enumerate(zip(order, n)):
            r.length += m
            r.x = x[indptr[s + 1] - 1:indptr[s + 1]]           # the next token's input: this one's output
            r.outputs.append(r.x)
            if len(r.outputs) == r.n_new:
                self.finish(r)
        return t

    def close(self) -> None:
        rdp.slora_kv_destroy(self.kv)
        rdp.slora_pool_destroy(self.pool)


def main() -> int:
    rdp.build.build()
    s = Server()
    rng = np.random.default_rng(1)
    waiting = [Request(f"r{i}", i % 8, torch.from_numpy(rng.normal(0, 1, (m, s.hidden)).astype(np.float16)).cuda(), k)
               for i, (m, k) in enumerate([(200, 40), (1, 12), (65, 30), (700, 20), (17, 25), (128, 9)])]
    it = 0
    while waiting or s.running:
        if waiting and it % 4 == 0:
            s.submit(waiting.pop(0))
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        done = [r.name for r in s.running]
        tokens = s.step()
        torch.cuda.synchronize()
        done = [n for n in done if n not in [r.name for r in s.running]]
        print(f"iteration {it}: {tokens} tokens, {len(s.running)} running, "
              f"{1e6 * (time.perf_counter() - t0):.0f} us, {rdp.slora_pool_num_free(s.pool)} pages free"
              + (f", done: {' '.join(done)}" if done else ""))
        it += 1
    status = rdp.slora_get_device_status(s.pool)
    s.close()
    return 1 if status else 0


if __name__ == "__main__":
    sys.exit(main())
