"""GPU checks of the compaction of KV cache sequences against its definition in fp64, in place and into other pages:
block edges, lists for each head, scales far apart, entries that cannot be used, and attention afterwards.

Codes and exponents are powers of two times integers of a few bits, so fp64 gives them exactly: no tolerance.
"""
import ctypes

import numpy as np
import pytest
import torch

import kv_reference as R
import rank_delta_paged_gb300 as rdp
from test_gpu_kv import Case, dev

pytestmark = pytest.mark.gpu
BAD_PAGE, BAD_SEGMENT, BAD_LENGTH, BAD_POSITION = 3, 4, 6, 7


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


class Moves:
    """A Case's sequences (lengths; new tokens are not used) and the tokens that each keeps."""

    def __init__(self, lengths, first, n_kept, hkv=2, d=128, hidden=4096, fmt="e4m3", seed=0, in_place=True, per_head=False,
                 spread=3, pick=None, edit=None):
        rng = np.random.default_rng(seed)
        self.fmt, self.hkv, self.in_place = fmt, hkv, in_place
        self.S = len(lengths)
        # a Case takes the pages of every block; the destinations are pages of sequences of its own
        bt = hidden * 2 // d // 8 * 8
        self.first, self.len = np.array(first, np.int32), np.array(lengths, np.int32)
        self.n = np.array(n_kept, np.int32)
        b0, b1 = self.first // bt, -(-(self.first + self.n) // bt)
        fresh = [] if in_place else [int(max(0, y - x)) * bt if k else 0 for x, y, k in zip(b0, b1, self.n)]
        c = self.c = Case([(0, n) for n in list(lengths) + fresh], hq=hkv, hkv=hkv, d=d, hidden=hidden, fmt=fmt, seed=seed,
                          spread=spread)
        self.bt = bt
        if edit:
            edit(c)
            c.push()
        self.table = c.table[:self.S].copy()
        self.dst = None
        if not in_place:
            self.dst = np.full((self.S, max(1, int(b1.max())), hkv, 2), -1, np.int32)
            for s in range(self.S):
                if fresh[s]:
                    self.dst[s, b0[s]:b1[s]] = c.table[self.S + s, :b1[s] - b0[s]]
        self.indptr = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.heads = hkv if per_head else 1
        K = int(self.indptr[-1])
        self.kept = np.zeros((self.heads, K + 5), np.int32)
        for h in range(self.heads):
            for s in range(self.S):
                where = np.arange(self.first[s], self.len[s])
                x = pick(where, self.n[s]) if pick else np.sort(rng.permutation(where)[:self.n[s]])
                self.kept[h, self.indptr[s]:self.indptr[s + 1]] = x
        self.new_len = torch.full((self.S,), -5, dtype=torch.int32, device="cuda")
        self.per_head = per_head

    def lists(self, **kw):
        up = dict(kept_indptr=self.indptr, kept=self.kept, first=self.first, kv_len=self.len, block_table=self.table)
        up = {k: dev(kw.pop(k, v)) for k, v in up.items()}
        dst = kw.pop("dst", self.dst)
        a = dict(n_seqs=self.S, n_kept=int(self.indptr[-1]), max_kept=int(self.n.max()), max_blocks=self.table.shape[1], **up,
                 dst_blocks=0 if dst is None else dst.shape[1], dst_table=None if dst is None else dev(dst),
                 head_stride=self.kept.shape[1] if self.per_head else 0, new_len=self.new_len)
        a.update(kw)
        return rdp.KVKeep(**a)

    def run(self, stream=None, **kw):
        k = self.lists(**kw)
        torch.cuda.synchronize()
        rdp.slora_kv_compact(self.c.s.kv, k, stream)
        torch.cuda.synchronize()

    def definition(self, skip=()):
        """(values, exponents, rows that are written) as they have to be; `skip`: (sequence, block, head or None)."""
        c, bt = self.c, self.bt
        val, exps = c.values()
        new, ne = val.copy(), exps.copy()
        rows = np.zeros(val.shape[:2], bool)
        behind = np.zeros(val.shape[:2], bool)
        to_table = self.table if self.dst is None else self.dst
        for s in range(self.S):
            f, n = int(self.first[s]), int(self.n[s])
            for blk in range(f // bt, -(-(f + n) // bt) if n else f // bt):
                end = min(f + n, (blk + 1) * bt)
                for h in range(self.hkv):
                    if (s, blk, h) in skip or (s, blk, None) in skip or (s, None, None) in skip:
                        continue
                    kept = self.kept[h if self.per_head else 0, self.indptr[s]:self.indptr[s + 1]]
                    src = np.array([t if t < f else kept[t - f] for t in range(blk * bt, end)])
                    for w in (0, 1):
                        page = self.table[s, src // bt, h, w]
                        e0 = np.clip(exps[page].astype(int), -60, 60)
                        x = val[page, src % bt] * 2.0 ** e0[:, None]
                        mag = np.abs(x[np.isfinite(x)])
                        e = R.fit_exponent(mag.max() if mag.size else 0.0, self.fmt)
                        d = to_table[s, blk, h, w]
                        new[d, :len(src)] = R.nearest(x * 2.0 ** -float(e), self.fmt)
                        ne[d] = e
                        rows[d, :len(src)] = True
                        behind[d, len(src):] = True
        return new, ne, rows, behind

    def check(self, stream=None, skip=(), status=0, **kw):
        want, we, rows, behind = self.definition(skip)
        before = self.c.s.pages.cpu().numpy()
        was = self.new_len.cpu().numpy()
        self.run(stream, **kw)
        assert self.c.s.device_status() == status
        got, ge = self.c.values()
        assert np.array_equal(ge, we)
        assert np.array_equal(got[rows], want[rows], equal_nan=True)
        after = self.c.s.pages.cpu().numpy()
        n = self.bt * self.c.d
        same = ~np.repeat(rows | behind, self.c.d, axis=1)
        assert np.array_equal(after[:, :n][same], before[:, :n][same]) and np.array_equal(after[:, n:], before[:, n:])
        skipped = [s for s, b, _ in skip if b is None]
        lens = np.where(np.isin(np.arange(self.S), skipped), was, self.first + self.n)
        assert np.array_equal(self.new_len.cpu().numpy(), lens)
        return got, ge


LENGTHS = [1, 64, 65, 200, 129, 333, 70, 10, 0, 500, 128, 90]
FIRST = [0, 0, 64, 100, 0, 17, 70, 3, 0, 130, 64, 5]
KEPT = [1, 64, 1, 40, 64, 300, 0, 7, 0, 333, 64, 60]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,hidden", [(128, 4096), (128, 5120), (64, 4096), (64, 256), (128, 640), (64, 8192), (128, 8192), (64, 320)])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("per_head", [False, True])
def test_compact_at_block_edges(fmt, d, hidden, in_place, per_head):
    Moves(LENGTHS, FIRST, KEPT, d=d, hidden=hidden, fmt=fmt, seed=200, in_place=in_place, per_head=per_head).check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_scales_far_apart(fmt, in_place):
    """Rows of one block from pages whose scales differ by up to 2^40, and exponents outside what append writes."""
    Moves([900, 64, 300], [0, 3, 100], [200, 30, 150], fmt=fmt, seed=201, spread=20, in_place=in_place).check()

    def edit(c):
        c.exps[:] = c.rng.choice([-128, -100, -61, -60, -41, 11, 40, 60, 61, 127], len(c.exps))
    Moves([900, 64, 300], [0, 3, 100], [200, 30, 150], fmt=fmt, seed=202, in_place=in_place, edit=edit).check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_compact_zeros_and_nan(fmt):
    def edit(c):
        p = c.pages.view()
        p[c.table[0, 0].ravel()] = 0                        # a block of zeros gets the smallest exponent
        p[c.table[0, 1].ravel()] = 0x80 if fmt == "e4m3" else 0     # minus zeros
        if fmt == "e4m3":                                   # NaN of both signs among the rows, and rows of nothing else
            p[c.table[1, 0, 0, 0], 128 * 3 + 5], p[c.table[1, 0, 1, 1], 128 * 9 + 100] = 0x7F, 0xFF
            p[c.table[1, 1].ravel(), :128 * 64] = 0x7F
    for in_place in (False, True):
        Moves([128, 200, 100], [0, 0, 20], [100, 150, 60], fmt=fmt, seed=203, in_place=in_place, edit=edit).check()


def test_compact_of_what_needs_no_move():
    """Everything is kept: only the exponents are fitted anew."""
    keep_all = lambda where, n: where[:n]                   # noqa: E731
    Moves([200, 64], [0, 10], [200, 54], seed=204, pick=keep_all).check()


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_long_sequences(in_place):
    Moves([20011, 9000], [5, 0], [7001, 65], hkv=1, seed=205, in_place=in_place).check()
    last = lambda where, n: where[len(where) - n:]          # noqa: E731
    Moves([6000], [1], [5900], hkv=2, d=64, fmt="int8", seed=206, in_place=in_place, pick=last).check()


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_by_several_ctas_in_turn(in_place):
    """Few sequences and many blocks: in place their blocks are dealt out to 2, 4 and 8 CTAs, with rounds that are full,
    and with one to all but one of a round's blocks missing."""
    for d, hidden, fmt in ((64, 256, "e4m3"), (128, 640, "int8"), (64, 8192, "e4m3")):
        bt = hidden * 2 // d // 8 * 8
        for blocks in (2, 3, 5, 7, 8, 9, 15, 16, 17, 31):
            n = blocks * bt
            Moves([4 * n + 5, n + 40, 30], [7, 0, 3], [n - 9, n, 20], d=d, hidden=hidden, fmt=fmt, seed=217, in_place=in_place).check()
            Moves([n + 3], [0], [n + 2], d=d, hidden=hidden, fmt=fmt, seed=218, in_place=in_place, hkv=3, per_head=True).check()


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_many_sequences_and_heads(in_place):
    rng = np.random.default_rng(7)
    n = rng.integers(0, 40, 1500)
    first = (n * rng.random(1500)).astype(int)
    kept = ((n - first) * rng.random(1500)).astype(int)
    Moves(list(n), list(first), list(kept), hkv=1, d=64, hidden=512, seed=207, in_place=in_place).check()
    Moves([30, 9], [7, 0], [20, 3], hkv=300, d=64, hidden=512, seed=208, in_place=in_place, per_head=True).check()


def test_compact_keeps_the_page_of_the_first_block():
    """dst_table may keep the block of first[s] where it is."""
    m = Moves([300, 200], [100, 3], [120, 150], seed=209, in_place=False)
    for s in range(2):
        m.dst[s, m.first[s] // m.bt] = m.table[s, m.first[s] // m.bt]
    m.check()


def test_compact_shared_sources():
    """Two sequences that read the same pages go to pages of their own."""
    m = Moves([300, 300], [0, 0], [100, 120], seed=210, in_place=False)
    m.table[1] = m.table[0]
    m.check()


def test_compact_without_optional_arrays():
    m = Moves([300, 200], [0, 0], [100, 50], seed=211)
    want, we, rows, _ = m.definition()
    m.run(first=np.zeros(2, np.int32), new_len=None)
    a, ea = m.c.values()
    m.c.push()
    k = m.lists(new_len=None)
    k.first = None
    rdp.slora_kv_compact(m.c.s.kv, k)
    b, eb = m.c.values()
    assert np.array_equal(a, b, equal_nan=True) and np.array_equal(ea, eb) and np.array_equal(ea, we)
    assert np.array_equal(a[rows], want[rows], equal_nan=True)
    assert (m.new_len == -5).all() and m.c.s.device_status() == 0


def test_compact_into_the_same_table_is_in_place():
    """The block table as dst_table, of whatever width it says."""
    for n in ([300, 200], [9000]):
        a, b = (Moves(n, [0] * len(n), [100] * (len(n) - 1) + [n[-1] - 50], seed=219) for _ in range(2))
        a.check()
        k = b.lists()
        k.dst_table, k.dst_blocks = k.block_table, 1
        rdp.slora_kv_compact(b.c.s.kv, k)
        torch.cuda.synchronize()
        assert torch.equal(a.c.s.pages, b.c.s.pages) and torch.equal(a.c.s.exponents, b.c.s.exponents)
        assert b.c.s.device_status() == 0


def test_compact_does_not_depend_on_max_kept():
    for in_place in (False, True):
        m = Moves([300, 200], [10, 0], [100, 50], seed=212, in_place=in_place)
        m.check(max_kept=1 << 30)


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_skips_what_it_cannot_use(in_place):
    top = (1 << 31) - 1
    make = lambda: Moves([300, 200, 150], [10, 0, 20], [100, 70, 60], seed=213, in_place=in_place)   # noqa: E731
    m = make()
    # positions out of order, below their destination, past the end: that block is not written
    for i, bad in ((3, -1), (5, None), (69, 200), (69, top), (66, -top)):
        m = make()
        at = m.indptr[1] + i
        m.check(kept=_with(m.kept, (0, at), m.kept[0, at - 1] if bad is None else bad), skip=[(1, i // m.bt, None)], status=BAD_POSITION)
    # pages
    for s, blk, h, w in ((1, 1, 1, 0), (2, 0, 0, 1)):
        for bad in (-1, len(m.c.pages), top, -top - 1):
            m = make()
            to = m.table if in_place else m.dst
            t = _with(to, (s, blk, h, w), bad)
            if in_place:
                _check_one_side(m, [(s, b, h) for b in range(4) if b == blk or _reads(m, s, b, blk)], w, block_table=t)
            else:
                _check_one_side(m, [(s, blk, h)], w, dst=t)
    # sequences
    for field, values in (("kv_len", (-1, m.table.shape[1] * m.bt + 1, (1 << 30) + 1, 69)), ("first", (-1, 201, 131, top))):
        for bad in values:
            m = make()
            m.check(**{field: _with(m.len if field == "kv_len" else m.first, 1, bad)}, skip=[(1, None, None)], status=BAD_LENGTH)
    m = make()
    m.check(kept_indptr=np.array([0, 100, 100 + 131, 5], np.int32), skip=[(1, None, None), (2, None, None)], status=BAD_SEGMENT,
            max_kept=100)
    m = make()
    m.check(max_kept=99, skip=[(0, None, None)], status=BAD_SEGMENT)
    if not in_place:
        m = make()
        m.check(dst=m.dst[:, :1].copy(), skip=[(0, 1, None), (1, 1, None), (2, 1, None)], status=BAD_LENGTH)


def _with(a, at, value):
    a = a.copy()
    a[at] = value
    return a


def _reads(m, s, blk, source):
    """Whether destination block blk of sequence s takes a row from block `source`."""
    f, n = int(m.first[s]), int(m.n[s])
    kept = m.kept[0, m.indptr[s]:m.indptr[s + 1]]
    src = [t if t < f else kept[t - f] for t in range(blk * m.bt, min(f + n, (blk + 1) * m.bt))]
    return any(p // m.bt == source for p in src) and blk >= f // m.bt


def _check_one_side(m, skipped, w, **kw):
    """Bad pages of keys (w 0) or values (1): the other side of the block is written all the same."""
    want, we, rows, behind = m.definition()
    val, exps = m.c.values()
    to = m.table if m.dst is None else m.dst
    for s, blk, h in skipped:
        if blk < to.shape[1] and to[s, blk, h, w] >= 0:
            p = to[s, blk, h, w]
            want[p], we[p], rows[p], behind[p] = val[p], exps[p], True, False
    m.run(**kw)
    assert m.c.s.device_status() == BAD_PAGE
    got, ge = m.c.values()
    assert np.array_equal(ge, we) and np.array_equal(got[rows], want[rows], equal_nan=True)


def test_compact_in_a_graph_and_on_another_stream():
    m, e = (Moves([300, 200, 90], [10, 0, 20], [100, 70, 30], seed=214, in_place=False) for _ in range(2))
    k = m.lists()
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        rdp.slora_kv_compact(m.c.s.kv, k, st)
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        e.check(stream=st)
        assert torch.equal(m.c.s.pages, e.c.s.pages) and torch.equal(m.c.s.exponents, e.c.s.exponents)
        m.c.s.exponents += 1
        e.c.s.exponents += 1


@pytest.mark.parametrize("n", [90, 700, 3000])
def test_compact_in_place_in_a_graph(n):
    """By clusters of 1 to 8 CTAs; every pass moves what the last one left, so the passes are counted alike."""
    m, e = (Moves([n, n // 2], [5, 0], [n // 2, n // 3], seed=220, d=64, hidden=512) for _ in range(2))
    k = m.lists()
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        rdp.slora_kv_compact(m.c.s.kv, k, st)
    for _ in range(3):
        g.replay()
        e.check()
        torch.cuda.synchronize()
        assert torch.equal(m.c.s.pages, e.c.s.pages) and torch.equal(m.c.s.exponents, e.c.s.exponents)
    assert m.c.s.device_status() == 0


def test_accepted_drafts_move_up_and_are_attended():
    """A tree of drafts is appended, its accepted branch moves up behind the sequence, the next token attends: as if
    only the branch had been appended, where its block's scale is the same."""
    cached, drafts, branch = [70, 200], 12, [0, 3, 4, 9]
    a, b = (Case([(drafts if i == 0 else len(branch), n + (drafts if i == 0 else len(branch))) for n in cached], hq=4, hkv=2, seed=215)
            for i in range(2))
    rng = np.random.default_rng(0)
    k = rng.normal(0, 1, (2 * drafts, 256)).astype(np.float16)
    some = np.concatenate([np.array(branch), drafts + np.array(branch)])
    outs = []
    for c, rows in ((a, k), (b, k[some])):
        # the cached rows alike in both, with scales that the drafts do not change
        for s, n in enumerate(cached):
            for p in range(n):
                r = np.random.default_rng(1000 * s + p)
                codes = torch.from_numpy(r.normal(0, 60, (2, 2, 128)).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                codes[:, :, 0] = 0x7E                      # 448
                for h in range(2):
                    for w in range(2):
                        page = c.table[s, p // c.bt, h, w]
                        c.pages[page, p % c.bt * 128:(p % c.bt + 1) * 128] = codes[h, w]
                        c.exps[page] = -3
        c.push()
        x = torch.from_numpy(rows).cuda()
        rdp.slora_kv_append(c.s.kv, c.batch(), x, 256, x, 256)
        lens = c.kv_len
        if c is a:
            keep = np.concatenate([n + np.array(branch) for n in cached]).astype(np.int32)
            new_len = torch.zeros(2, dtype=torch.int32, device="cuda")
            rdp.slora_kv_compact(c.s.kv, rdp.KVKeep(2, 8, 4, c.max_blocks, dev(np.array([0, 4, 8], np.int32)), dev(keep),
                                                    dev(np.array(cached, np.int32)), c.d_len, c.d_table, new_len=new_len))
            lens = new_len.cpu().numpy()
            assert lens.tolist() == [n + 4 for n in cached]
        q = torch.from_numpy(np.random.default_rng(2).normal(0, 1, (2, 512)).astype(np.float16)).cuda()
        out = torch.zeros_like(q)
        batch = rdp.KVBatch(2, 2, 1, c.max_blocks, dev(np.arange(3, dtype=np.int32)), dev(lens), c.d_table)
        rdp.slora_kv_attend(c.s.kv, batch, q, 512, 4, out, 512, softmax_scale=0.05)
        torch.cuda.synchronize()
        assert c.s.device_status() == 0
        outs.append(out)
    assert torch.equal(*outs)


def test_compact_refusals():
    m = Moves([300, 200], [10, 0], [100, 50], seed=216, in_place=False)
    before, exps = m.c.s.pages.clone(), m.c.s.exponents.clone()

    def refused(kv=m.c.s.kv, keep=None, **fields):
        k = keep or m.lists()
        for f, x in fields.items():
            setattr(k, f, x)
        with pytest.raises(rdp.SloraError) as e:
            rdp.slora_kv_compact(kv, k)
        assert e.value.status == 1

    refused(kv=None)
    for bad in (dict(n_seqs=-1), dict(n_seqs=(1 << 20) + 1), dict(n_kept=-1), dict(n_kept=(1 << 30) + 1), dict(max_kept=-1),
                dict(max_kept=(1 << 30) + 1), dict(max_blocks=0), dict(dst_blocks=0), dict(kept_head_stride=149),
                dict(kept_head_stride=-1), dict(kept_indptr=None), dict(kept=None), dict(kv_len=None), dict(block_table=None)):
        refused(**bad)
    k = m.lists()
    for f in ("kept_indptr", "kept", "first", "kv_len", "block_table", "dst_table", "new_len"):
        refused(**{f: getattr(k, f) + 2})
    for f in ("kept_indptr", "first", "kv_len"):
        refused(keep=k, new_len=getattr(k, f))
        refused(keep=k, new_len=getattr(k, f) + 4)
    with pytest.raises(rdp.SloraError):
        rdp._call("slora_kv_compact", m.c.s.kv, None, None)
    for empty in (dict(n_seqs=0), dict(n_seqs=0, n_kept=0, max_kept=0, kept=None, kept_indptr=None, kv_len=None, block_table=None)):
        k = m.lists()
        for f, x in empty.items():
            setattr(k, f, x)
        rdp.slora_kv_compact(m.c.s.kv, k)
    torch.cuda.synchronize()
    assert torch.equal(before, m.c.s.pages) and torch.equal(exps, m.c.s.exponents) and (m.new_len == -5).all()
    assert m.c.s.device_status() == 0
    assert ctypes.sizeof(rdp.KVKeep) == 88
