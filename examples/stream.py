"""Streams that outlive their cache: a window with sinks, branches and drafts over the 8-bit KV cache.

    python examples/stream.py

A stack of attention layers with random weights and normed queries and keys continues streams of
tokens up to the last position of the rotation's table.  Per layer and step:

    q, k, v = x W
    norms, rotation; k and v to the pages        slora_kv_append_norm
    attention over the window and the sinks      slora_kv_attend_sinks

Blocks that the window has left and that hold no sink go back to the pool, so a stream holds the
same number of pages however long it gets.  A stream forks by sharing its whole blocks
(slora_pages_share) and copying the one it writes next (slora_kv_copy).  Drafted tokens run as
one step, each after the ones before it, so the accepted ones are a prefix; the others are forgotten, and
the block's scales are fitted to what is left (slora_kv_compact).
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import rank_delta_paged_gb300 as rdp  # noqa: E402

NO_PAGE = -1


class Stream:
    def __init__(self, length=0, blocks=None):
        self.length = length             # tokens in the cache
        self.settled = length            # those of them that no accept() may take back: a fork has them too
        self.blocks = blocks or {}       # block -> int32 [layers][n_heads][2]


class Streams:
    def __init__(self, hidden=512, head_dim=64, n_layers=2, num_pages=2048, window=200, sinks=4, max_positions=1 << 14,
                 fmt=rdp.SLORA_KV_E4M3, seed=0):
        self.hidden, self.head_dim, self.n_layers, self.n_heads = hidden, head_dim, n_layers, hidden // head_dim
        self.window, self.sinks = window, sinks
        self.pool = rdp.slora_pool_create(0, hidden, num_pages, 1, 1, seed)
        self.kv = rdp.slora_kv_create(self.pool, self.n_heads, head_dim, fmt)
        self.block = rdp.slora_kv_block_tokens(self.kv)
        rng = np.random.default_rng(seed)
        f32 = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
        self.max_positions = max_positions
        self.w = f32(rng.normal(0, hidden ** -0.5, (n_layers, 4, hidden, hidden))).half()
        self.norms = [rdp.KVNorm(1e-6, False, f32(rng.normal(1, 0.1, head_dim)), 0, f32(rng.normal(1, 0.1, head_dim)), 0)
                      for _ in range(n_layers)]
        angle = np.arange(max_positions)[:, None] * 10000.0 ** (-np.arange(0, head_dim, 2) / head_dim)
        self.rope = rdp.KVRope(head_dim, False, max_positions, f32(np.cos(angle)), f32(np.sin(angle)))

    def table(self, streams):
        """int32 [layers][streams][blocks][n_heads][2] of the blocks that the streams hold."""
        width = max(max(s.blocks, default=0) for s in streams) + 1
        t = np.full((self.n_layers, len(streams), width, self.n_heads, 2), NO_PAGE, np.int32)
        for i, s in enumerate(streams):
            for b, pages in s.blocks.items():
                t[:, i, b] = pages
        return t

    def step(self, work):
        """Runs new tokens x fp16 [n][hidden] of each (stream, x); returns their outputs.  They are the streams' from then
        on, or drafts until accept()."""
        streams, xs = zip(*work)
        n = [len(x) for x in xs]
        if any(s.length + m > self.max_positions for s, m in zip(streams, n)):
            raise ValueError(f"a stream has {self.max_positions} positions")
        taken = []
        try:
            for s, m in zip(streams, n):
                for b in range(s.length // self.block, (s.length + m - 1) // self.block + 1):
                    if b not in s.blocks:
                        s.blocks[b] = self._take()
                        taken.append((s, b))
        except rdp.SloraError:                          # a full pool: the streams stay as they were
            for s, b in taken:
                self._give_back(s.blocks.pop(b))
            raise
        table = torch.from_numpy(self.table(streams)).cuda()
        indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        lengths = np.array([s.length + m for s, m in zip(streams, n)], np.int32)
        d_indptr, d_lengths = torch.from_numpy(indptr).cuda(), torch.from_numpy(lengths).cuda()
        x, t, h = torch.cat(xs), int(indptr[-1]), self.hidden
        for layer in range(self.n_layers):
            batch = rdp.KVBatch(t, len(streams), max(n), table.shape[2], d_indptr, d_lengths, table[layer])
            xn = torch.nn.functional.rms_norm(x, (h,))
            q, k, v = (xn @ self.w[layer, j] for j in range(3))
            out = torch.empty_like(q)
            rdp.slora_kv_append_norm(self.kv, batch, k, h, v, h, q, h, q, h, self.n_heads, self.norms[layer], self.rope)
            rdp.slora_kv_attend_sinks(self.kv, batch, q, h, self.n_heads, out, h, softmax_scale=self.head_dim ** -0.5,
                                      window=self.window, n_sinks=self.sinks)
            x = x + out @ self.w[layer, 3]
        for s, m in zip(streams, n):
            s.length += m
        return [x[indptr[i]:indptr[i + 1]] for i in range(len(streams))]

    def trim(self, s):
        """Gives back the blocks that no later token sees, once the last drafts are accepted."""
        for b in [b for b in s.blocks if b * self.block >= self.sinks and (b + 1) * self.block <= s.length - self.window + 1]:
            self._give_back(s.blocks.pop(b))

    def accept(self, s, drafts, kept):
        """Of the stream's last `drafts` tokens only those numbered kept[] (ascending) stay: a prefix, as every draft has
        attended to the ones before it and is rotated by its place.  (slora_kv_compact moves any choice up; for another
        one, drafts have to be run by a tree's mask and depths.)"""
        first, k = s.length - drafts, len(kept)
        if first < s.settled:
            raise ValueError("a fork holds pages of these drafts")
        L = self.n_layers
        ints = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
        if k:
            table = self.table([s])[:, 0]               # the layers as the sequences of one call
            rdp.slora_kv_compact(self.kv, rdp.KVKeep(L, L * k, k, table.shape[1], ints(np.arange(L + 1) * k),
                                                     ints(np.tile(first + np.asarray(kept), L)), ints(np.full(L, first)),
                                                     ints(np.full(L, s.length)), ints(table)))
        s.length = first + k
        for b in [b for b in s.blocks if b * self.block >= max(s.length, 1)]:
            self._give_back(s.blocks.pop(b))

    def fork(self, s):
        """A stream that goes on from here by itself."""
        child = Stream(s.length)
        whole, rest = divmod(s.length, self.block)
        try:
            for b, pages in s.blocks.items():
                if b == whole and rest:
                    child.blocks[b] = self._take()
                    src, dst = (torch.from_numpy(p.ravel().copy()).cuda() for p in (pages, child.blocks[b]))
                    rows = torch.full((pages.size,), rest, dtype=torch.int32, device="cuda")
                    rdp.slora_kv_copy(self.kv, pages.size, src, dst, rows)
                elif b < whole:
                    rdp.slora_pages_share(self.pool, pages.size, pages)
                    child.blocks[b] = pages
        except rdp.SloraError:
            self.drop(child)
            raise
        s.settled = s.length
        return child

    def _take(self):
        """The pages of a block."""
        pages = np.empty((self.n_layers, self.n_heads, 2), np.int32)
        rdp.slora_pages_alloc(self.pool, pages.size, pages)
        return pages

    def _give_back(self, pages):
        rdp.slora_pages_free(self.pool, pages.size, np.ascontiguousarray(pages))

    def drop(self, s):
        for pages in s.blocks.values():
            self._give_back(pages)
        s.blocks = {}

    def close(self):
        rdp.slora_kv_destroy(self.kv)
        rdp.slora_pool_destroy(self.pool)


def main() -> int:
    rdp.build.build()
    e = Streams()
    rng = np.random.default_rng(1)
    tokens = lambda n: torch.from_numpy(rng.normal(0, 1, (n, e.hidden)).astype(np.float16)).cuda()  # noqa: E731
    a, b = Stream(), Stream()
    e.step([(a, tokens(300)), (b, tokens(7))])
    c = e.fork(a)
    for i in range(1, 601):
        if i % 100 == 0:                 # a few drafts, of which some are accepted
            e.step([(a, tokens(8)), (b, tokens(1)), (c, tokens(1))])
            e.accept(a, 8, list(range(rng.integers(0, 9))))
        else:
            e.step([(s, tokens(1)) for s in (a, b, c)])
        for s in (a, b, c):
            e.trim(s)
        if i % 150 == 0:
            print(f"step {i}: lengths {a.length} {b.length} {c.length}, blocks {len(a.blocks)} {len(b.blocks)} {len(c.blocks)}, "
                  f"{rdp.slora_pool_num_free(e.pool)} pages free")
    for s in (a, b, c):
        e.drop(s)
    torch.cuda.synchronize()
    status, free = rdp.slora_get_device_status(e.pool), rdp.slora_pool_num_free(e.pool)
    e.close()
    return 0 if status == 0 and free == 2048 else 1


if __name__ == "__main__":
    sys.exit(main())
