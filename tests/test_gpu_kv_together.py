"""GPU check of the KV cache's operators in the order in which a serving loop runs them, on one stream without the host
in between: drafted tokens are appended with their norms and attend over a window and sinks, the accepted ones
move up, the sequences fork, and the next tokens attend over both branches.  Each attention against the
formula in fp64 over the cache as it stands; the same from a graph."""
import copy

import numpy as np
import pytest
import torch

import kv_reference as R
import rank_delta_paged_gb300 as rdp
from test_gpu_kv import Case, dev, half
from test_gpu_kv_norm import Call
from test_gpu_kv_sinks import give_back, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


class Loop:
    drafts, branch, window, sinks, scale = 6, [0, 2, 3], 60, 5, 0.05

    def __init__(self, lengths, fmt, d, seed):
        n, hkv = self.drafts, 2
        c = self.c = Case([(n, m + n) for m in lengths], hq=8, hkv=hkv, d=d, fmt=fmt, seed=seed, spare=4 * len(lengths) * hkv)
        give_back(c, self.window + n, self.sinks)           # the accepted tokens' windows reach as far
        self.call = Call(c, rot=d, centered=True)
        S = self.S = len(lengths)
        self.row = c.hq * d
        self.out1 = torch.zeros((c.T, self.row), dtype=torch.float16, device="cuda")
        first = np.array(lengths, np.int32)
        kept = np.concatenate([m + np.array(self.branch) for m in lengths]).astype(np.int32)
        self.new_len = torch.zeros(S, dtype=torch.int32, device="cuda")
        k = len(self.branch)
        self.keep = rdp.KVKeep(S, S * k, k, c.max_blocks, dev(np.arange(S + 1, dtype=np.int32) * k), dev(kept), dev(first), c.d_len,
                               c.d_table, new_len=self.new_len)
        # the fork of each sequence: a table of its own whose last block is a copy; rows of it are in use
        self.lens = first + k
        used = set(c.table[c.table >= 0].tolist())
        spare = np.array([p for p in range(len(c.pages)) if p not in used], np.int32)
        self.fork = c.table.copy()
        src, dst, rows = [], [], []
        for s, m in enumerate(self.lens):
            b = (m - 1) // c.bt
            new = spare[s * 2 * hkv:(s + 1) * 2 * hkv]
            src.append(c.table[s, b].ravel())
            dst.append(new)
            rows.append(np.full(2 * hkv, m - b * c.bt, np.int32))
            self.fork[s, b] = new.reshape(hkv, 2)
        self.src, self.dst, self.rows = (dev(np.concatenate(x).astype(np.int32)) for x in (src, dst, rows))
        # then a query per branch
        self.tables = np.concatenate([c.table, self.fork])
        self.q2 = np.random.default_rng(seed).normal(0, 1, (2 * S, c.hq, d)).astype(np.float16)
        self.dq2 = half(self.q2).view(2 * S, -1)
        self.out2 = torch.zeros_like(self.dq2)
        self.batch2 = rdp.KVBatch(2 * S, 2 * S, 1, c.max_blocks, dev(np.arange(2 * S + 1, dtype=np.int32)),
                                  torch.zeros(2 * S, dtype=torch.int32, device="cuda"), dev(self.tables))
        self.len2 = self.batch2._keep[1]
        self.between = torch.empty_like(c.s.pages), torch.empty_like(c.s.exponents)

    def run(self, st):
        c, kv = self.c, self.c.s.kv
        with torch.cuda.stream(st):
            self.call.run(st)
            rdp.slora_kv_attend_sinks(kv, self.call.batch, self.call.q_out, self.call.q_out.stride(0), c.hq, self.out1, self.row, None,
                                      self.scale, self.window, self.sinks, st)
            self.between[0].copy_(c.s.pages)
            self.between[1].copy_(c.s.exponents)
            rdp.slora_kv_compact(kv, self.keep, st)
            rdp.slora_kv_copy(kv, len(self.src), self.src, self.dst, self.rows, st)
            self.len2[:self.S].copy_(self.new_len)
            self.len2[self.S:].copy_(self.new_len)
            rdp.slora_kv_attend_sinks(kv, self.batch2, self.dq2, self.row, c.hq, self.out2, self.row, None, self.scale, self.window,
                                      self.sinks, st)

    def seen(self, pages, exps, seqs, table, q):
        """The reference over a state of the cache."""
        c = copy.copy(self.c)
        val = R.decode(np.ascontiguousarray(pages[:, :c.bt * c.d].reshape(-1, c.bt, c.d)), c.fmt)
        c.values = lambda: (val, exps)
        c.seqs, c.table, c.q, c.T = seqs, table, q, len(q)
        c.indptr = np.concatenate([[0], np.cumsum([n for n, _ in seqs])])
        return reference(c, self.window, self.sinks, self.scale)

    def check(self):
        c = self.c
        torch.cuda.synchronize()
        assert c.s.device_status() == 0
        assert self.new_len.tolist() == self.lens.tolist()
        q1 = self.call.q_out.cpu().view(torch.int16).numpy().view(np.float16)[:, :self.row].reshape(c.T, c.hq, c.d)
        ref, _, tol, _ = self.seen(self.between[0].cpu().numpy(), self.between[1].cpu().numpy(), c.seqs, c.table, q1)
        assert (np.abs(self.out1.float().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()
        pages, exps = c.s.pages.cpu().numpy(), c.s.exponents.cpu().numpy()
        ref, _, tol, _ = self.seen(pages, exps, [(1, int(m)) for m in self.lens] * 2, self.tables, self.q2)
        assert (np.abs(self.out2.float().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()
        assert np.array_equal(exps[self.src.cpu()], exps[self.dst.cpu()])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_drafts_are_appended_attend_move_up_and_fork(fmt, d):
    lengths = [200, 61, 3, 124, 700]
    a, b = (Loop(lengths, fmt, d, 400) for _ in range(2))
    st = torch.cuda.Stream()
    a.run(st)
    a.check()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        b.run(st)
    for _ in range(2):
        b.c.s.pages.copy_(dev(b.c.pages))
        b.c.s.exponents.copy_(dev(b.c.exps))
        torch.cuda.synchronize()
        g.replay()
        b.check()
        for x, y in ((a.out1, b.out1), (a.out2, b.out2), (a.c.s.pages, b.c.s.pages), (a.c.s.exponents, b.c.s.exponents)):
            assert torch.equal(x, y)
