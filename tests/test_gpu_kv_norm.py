"""GPU checks of the append with norms of queries and keys per head: codes, exponents and rotated queries against the
formula in fp64, every kernel against the others, and the call's refusals.

What fp32 may lose, in units u = 2^-24 of a row's own values: the squares of a row are summed in at most 8 roundings
(and are rounded themselves once, and twice more for the mean's subtraction), eps adds one, half of that passes the
root; the reciprocal root is good to 4 u; two products 2 u.  That is 10.5 u, or 13 u with the mean; the mean
itself is 8 u of the mean magnitude off, which reaches a channel times its weight over the deviation.
"""
import ctypes

import numpy as np
import pytest
import torch

import kv_reference as R
import rank_delta_paged_gb300 as rdp
from test_gpu_kv import Case, check_append, dev, half

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


def normed(x, w, eps, centered):
    """fp64 (norm of x [T][heads][d], how far fp32 may be off)."""
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        m = x.mean(-1, keepdims=True) if centered else 0.0
        off = 8 * U * np.abs(x).mean(-1, keepdims=True) if centered else 0.0
        r = 1 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
        y = (x - m) * r * w
        return y, np.abs(y) * (14 * U + (off * r) ** 2) + off * r * np.abs(w)


def turned(y, t, cos, sin, interleaved):
    """The rotation of y and of its tolerance t."""
    c, s = cos.astype(np.float64), sin.astype(np.float64)
    z = R.rotate(y, c, s, interleaved, np.float64)
    h = cos.shape[-1]
    ia, ib = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    c, s = np.abs(c)[:, None], np.abs(s)[:, None]
    a, b, ta, tb = np.abs(y[..., ia]), np.abs(y[..., ib]), t[..., ia], t[..., ib]
    t = t.copy()
    t[..., ia] = ta * c + tb * s + 2 * U * (a * c + b * s)
    t[..., ib] = tb * c + ta * s + 2 * U * (b * c + a * s)
    return z, t * 1.001


class Call:
    """Random tokens for a Case, and the norm and rotation that they get."""

    def __init__(self, c, rot=128, interleaved=False, centered=False, eps=1e-6, weights="shared", with_q=True, values=None,
                 positions=None, seed=0):
        rng = np.random.default_rng(seed + 100)
        self.c, self.rot, self.inter, self.centered, self.eps, self.with_q = c, rot, interleaved, centered, np.float32(eps), with_q
        T, hq, hkv, d = c.T, c.hq, c.hkv, c.d
        self.q, self.k, self.v = (rng.normal(0, 1, (T, h, d)) * np.exp(rng.normal(0, 2, (T, h, 1))) for h in (hq, hkv, hkv))
        self.q, self.k, self.v = (np.clip(x, -60000, 60000).astype(np.float16) for x in (self.q, self.k, self.v))
        if values:
            values(self.q, self.k, self.v)
        self.qw = self.kw = None
        self.each = 0
        if weights == "shared":
            self.qw, self.kw = (rng.normal(1, 0.3, (1, d)).astype(np.float32) for _ in range(2))
        if weights == "heads":       # of each head, and a gap between them
            self.qw, self.kw = (rng.normal(1, 0.3, (h, d + 4)).astype(np.float32) for h in (hq, hkv))
            self.each = d + 4
        self.row = (hq + 2 * hkv) * d + 8
        self.buf = half(np.concatenate([x.reshape(T, -1) for x in (self.q, self.k, self.v)] + [np.zeros((T, 8), np.float16)], 1))
        self.dq, self.dk, self.dv = self.buf, self.buf[:, hq * d:], self.buf[:, (hq + hkv) * d:]
        self.pos = np.concatenate([np.arange(n - m, n) for m, n in c.seqs]).astype(np.int32)
        if positions:
            self.pos = positions(self.pos)
        n_pos = int(self.pos.max()) + 5
        self.rope = None
        if rot:
            angle = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
            self.cos, self.sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
            self.rope = rdp.KVRope(rot, interleaved, n_pos, dev(self.cos), dev(self.sin), dev(self.pos) if positions else None)
        w = [None if x is None else dev(x) for x in (self.qw, self.kw)]
        self.norm = rdp.KVNorm(float(self.eps), centered, w[0], self.each, w[1], self.each)
        self.q_out = torch.full((max(T, 1), hq * d + 16), 7.0, dtype=torch.float16, device="cuda")
        self.batch = c.batch()

    def run(self, stream=None):
        c, qs = self.c, self.q_out.stride(0)
        q = (self.dq, self.row, self.q_out, qs, c.hq) if self.with_q else (None, 0, None, 0, 0)
        rdp.slora_kv_append_norm(c.s.kv, self.batch, self.dk, self.row, self.dv, self.row, *q, self.norm, self.rope, stream)

    def want(self, x, w):
        w = 1.0 if w is None else w[:, :self.c.d].astype(np.float64)
        y, t = normed(x, w, float(self.eps), self.centered)
        if self.rot:
            with np.errstate(invalid="ignore"):
                y, t = turned(y, t, self.cos[self.pos], self.sin[self.pos], self.inter)
        return y, t

    def check(self, stream=None):
        c, bt = self.c, self.c.bt
        before, exps = c.values()
        bytes_before = c.s.pages.cpu().numpy()
        torch.cuda.synchronize()
        self.run(stream)
        torch.cuda.synchronize()
        assert c.s.device_status() == 0
        got, ge = c.values()
        k, tk = self.want(self.k, self.kw)
        touched = np.zeros(len(got), bool)
        rows = np.zeros(got.shape[:2], bool)
        for s, (n, length) in enumerate(c.seqs):
            p0 = length - n
            for blk in range(p0 // bt, -(-length // bt) if n else p0 // bt):
                lo, hi = max(p0, blk * bt), min(length, (blk + 1) * bt)
                held, at = lo - blk * bt, slice(c.indptr[s] + lo - p0, c.indptr[s] + hi - p0)
                for h in range(c.hkv):
                    for w, (x, t) in enumerate(((k[at, h], tk[at, h]), (self.v[at, h].astype(np.float64), np.zeros((hi - lo, c.d))))):
                        page = c.table[s, blk, h, w]
                        touched[page] = True
                        rows[page, :held + hi - lo] = True
                        fine = np.isfinite(x)
                        mag, tm = np.abs(x[fine]), t[fine]
                        es = {R.fit_exponent(max(0.0, (mag + sign * tm).max()) if mag.size else 0.0, c.fmt) for sign in (-1, 0, 1)}
                        if held:
                            es = {max(e, int(exps[page])) for e in es}
                        e = int(ge[page])
                        assert e in es, (s, blk, h, w, e, es)
                        if held:
                            assert np.array_equal(got[page, :held], R.nearest(before[page, :held] * 2.0 ** (int(exps[page]) - e), c.fmt))
                        new = got[page, held:held + hi - lo]
                        u = 2.0 ** -e
                        nan = np.isnan(x)
                        assert (np.isnan(new[nan]).all() if c.fmt == "e4m3" else (new[nan] == 0).all())
                        z = np.where(fine, x * u, 0)
                        lim = np.clip(z, -R.LIMIT[c.fmt], R.LIMIT[c.fmt])
                        assert (np.abs(new - lim)[fine] <= (R.half_step(lim, c.fmt) + t * u)[fine] * (1 + 1e-9)).all()
        assert np.array_equal(ge[~touched], exps[~touched])
        after = c.s.pages.cpu().numpy()
        assert np.array_equal(after[:, bt * c.d:], bytes_before[:, bt * c.d:])
        rest = ~np.repeat(rows, c.d, axis=1)
        assert np.array_equal(after[:, :bt * c.d][rest], bytes_before[:, :bt * c.d][rest])
        out = self.q_out.cpu().view(torch.int16).numpy().view(np.float16)
        assert (out[:, c.hq * c.d:] == 7).all()
        if self.with_q:
            q, tq = self.want(self.q, self.qw)
            g = out[:c.T, :c.hq * c.d].reshape(q.shape).astype(np.float64)
            fine = np.isfinite(q)
            assert np.isnan(g[~fine]).all()
            q = np.where(fine, q, 0)
            step = np.maximum(2.0 ** -11 * 2.0 ** np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -14))), 2.0 ** -25)
            assert (np.abs(g - q)[fine] <= (step + tq)[fine] * (1 + 1e-9)).all()
        return got, ge, out


SEQS = [(1, 1), (1, 64), (1, 65), (1, 200), (3, 3), (5, 68), (64, 64), (65, 65), (70, 131), (1, 80), (130, 400), (0, 10), (2, 161)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,hidden", [(128, 4096), (128, 5120), (64, 4096), (64, 256), (128, 640), (64, 8192), (128, 8192)])
@pytest.mark.parametrize("centered", [False, True])
def test_norm_at_block_edges(fmt, d, hidden, centered):
    Call(Case(SEQS, hq=4, hkv=2, d=d, hidden=hidden, fmt=fmt, seed=70), rot=d, centered=centered).check()


@pytest.mark.parametrize("rot", [0, 16, 48, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weights", [None, "shared", "heads"])
def test_norm_rotations_and_weights(rot, interleaved, weights):
    seqs = [(1, 70), (3, 10), (40, 90)]
    Call(Case(seqs, hq=6, hkv=3, seed=71), rot=rot, interleaved=interleaved, weights=weights, eps=1e-5).check()
    Call(Case([(1, 70)] * 5, hq=6, hkv=3, seed=72), rot=rot, interleaved=interleaved, weights=weights, centered=True).check()
    if rot <= 64:
        Call(Case(seqs, hq=5, hkv=5, d=64, seed=73), rot=rot, interleaved=interleaved, weights=weights).check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (40, 40), (7, 1), (9, 3), (64, 32)])
@pytest.mark.parametrize("with_q", [False, True])
def test_norm_head_layouts(hq, hkv, with_q):
    Call(Case([(1, 33), (1, 100), (20, 70)], hq=hq, hkv=hkv, seed=74), weights="heads", with_q=with_q).check()
    Call(Case([(1, 33), (1, 100)], hq=hq, hkv=hkv, seed=75), weights="heads", with_q=with_q, rot=0).check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("centered", [False, True])
def test_norm_of_odd_rows(fmt, centered):
    """Zeros, equal channels, the smallest and the largest numbers, infinities and NaN."""
    def odd(q, k, v):
        for x in (q, k):
            x[0], x[1] = 0, 3
            x[2], x[3] = 6e-8, 65504
            x[4, :, 5], x[5, :, 9] = np.inf, np.nan
            x[6], x[7, :, ::2] = -65504, 0
            x[8, :, 1] = -np.inf
    for rot in (0, 128):
        Call(Case([(1, 70), (8, 8), (2, 71), (30, 30)], hq=4, hkv=2, fmt=fmt, seed=76), rot=rot, values=odd, centered=centered).check()
        Call(Case([(1, 70)] * 9, hq=4, hkv=2, fmt=fmt, seed=76), rot=rot, values=odd, centered=centered).check()


def test_norm_without_eps():
    Call(Case([(1, 70), (9, 30)], hq=4, hkv=2, seed=77), eps=0.0).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("centered", [False, True])
def test_norm_does_not_depend_on_the_kernel(d, centered):
    """The same tokens as single ones and within a prompt: queries bit for bit, and each token's key where the prompt
    has it alone in a block."""
    n = 40
    a, b = Case([(1, 1)] * n, hq=4, hkv=2, d=d, hidden=8 * d // 2, seed=78), Case([(n, n)], hq=4, hkv=2, d=d, hidden=8 * d // 2, seed=78)
    assert a.bt == 8
    pos = np.arange(n, dtype=np.int32)
    x, y = (Call(c, rot=d, centered=centered, weights="heads", positions=lambda p: pos) for c in (a, b))
    (va, ea, qa), (vb, eb, qb) = x.check(), y.check()
    assert np.array_equal(qa.view(np.uint16), qb.view(np.uint16))
    # a key's codes in its own block, and in the prompt's block, where its scale is the block's
    for t in range(n):
        for h in range(2):
            pa, pb = a.table[t, 0, h, 0], b.table[0, t // 8, h, 0]
            assert ea[pa] <= eb[pb]
            if ea[pa] == eb[pb]:
                assert np.array_equal(va[pa, 0], vb[pb, t % 8])


def step_by_step(x, w, eps, centered):
    """The norm in fp32, each step rounded once: the even and the odd channels of each 8 summed one after another, then
    the eights by twos; the reciprocal root is CUDA's."""
    def mean(y):
        y = y.reshape(*y.shape[:-1], -1, 4, 2)
        y = ((y[..., 0, :] + y[..., 1, :]) + y[..., 2, :]) + y[..., 3, :]
        y = y[..., 0] + y[..., 1]
        while y.shape[-1] > 1:
            y = y[..., 0::2] + y[..., 1::2]
        return y * np.float32(1.0 / x.shape[-1])
    x = x.astype(np.float32)
    if centered:
        x = x - mean(x)
    r = torch.rsqrt(dev(mean(x * x) + np.float32(eps))).cpu().numpy()
    return (x * r) * w


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("centered", [False, True])
@pytest.mark.parametrize("seqs", [[(1, 70)] * 300, [(300, 400)]], ids=["single", "prompt"])
def test_norm_rounds_every_step_by_itself(d, centered, seqs):
    """No product is contracted into a sum, in either kernel: the queries bit for bit."""
    c = Case(seqs, hq=8, hkv=2, d=d, seed=82)
    x = Call(c, rot=0, centered=centered, weights="heads", eps=1e-5)
    _, _, out = x.check()
    want = step_by_step(x.q, x.qw[:, :d], 1e-5, centered).astype(np.float16).reshape(c.T, -1)
    assert np.array_equal(out[:c.T, :8 * d].view(np.uint16), want.view(np.uint16))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [64, 67, 71])
def test_queries_in_runs_of_heads(d, hq):
    """Batches so large that a group of lanes takes 8 heads of a token (128 channels) or 4 (64), the last run short, with
    rows of skipped sequences between; with norms and without, and in place."""
    seqs = [(1000, 1003), (0, 9), (3, 7), (1, 40), (1150, 1150)]
    Call(Case(seqs, hq=hq, hkv=1, d=d, seed=84), rot=d, weights="heads", centered=True).check()
    check_append(Case(seqs, hq=hq, hkv=1, d=d, seed=85), rot=d)
    check_append(Case(seqs, hq=hq, hkv=1, d=d, seed=86), rot=d // 2, interleaved=hq == 67)
    c = Case(seqs, hq=hq, hkv=1, d=d, seed=87)
    x = Call(c, rot=d)
    x.run()
    want = x.q_out[:, :hq * d].clone()
    q = x.buf[:, :hq * d].contiguous()
    pad = torch.full((7, hq * d), 3.0, dtype=torch.float16, device="cuda")
    q = torch.cat([pad, q, pad])
    k = torch.zeros((len(q), d), dtype=torch.float16, device="cuda")
    b = rdp.KVBatch(len(q), len(seqs), 1150, c.max_blocks, dev(c.indptr + 7), c.d_len, c.d_table)
    rdp.slora_kv_append_norm(c.s.kv, b, k, d, k, d, q, hq * d, q, hq * d, hq, x.norm, x.rope)
    torch.cuda.synchronize()
    assert torch.equal(q[7:-7].view(torch.int16), want.view(torch.int16))
    assert (q[:7] == 3).all() and (q[-7:] == 3).all() and c.s.device_status() == 0


def test_norm_in_a_graph_on_another_stream_then_attention():
    """A graph of an append with norms and the attention over it, replayed with other tokens, against eager calls."""
    seqs = [(1, 70), (1, 200), (130, 300), (2, 65), (9, 70)]
    eager, c = (Case(seqs, hq=6, hkv=2, seed=79) for _ in range(2))
    x, y = Call(eager, centered=True), Call(c, centered=True)
    st = torch.cuda.Stream()
    row = c.hq * c.d
    outs = [torch.zeros((c.T, row), dtype=torch.float16, device="cuda") for _ in range(2)]

    def step(z, out, stream):
        z.run(stream)
        rdp.slora_kv_attend(z.c.s.kv, z.batch, z.q_out, z.q_out.stride(0), 6, out, row, softmax_scale=0.1, stream=stream)

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        step(y, outs[1], st)
    for i in range(3):
        new = torch.from_numpy(np.random.default_rng(i).normal(0, 1, tuple(x.buf.shape)).astype(np.float16)).cuda()
        x.buf.copy_(new)
        y.buf.copy_(new)
        torch.cuda.synchronize()
        step(x, outs[0], None)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x.q_out, y.q_out) and torch.equal(*outs)
        assert torch.equal(eager.s.pages, c.s.pages) and torch.equal(eager.s.exponents, c.s.exponents)
    assert c.s.device_status() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_norm_with_weights_past_the_exponents(fmt):
    """Keys beyond the largest scale become the largest code, and the block's other rows stay what they were."""
    for seqs in ([(1, 70)] * 3, [(5, 70)]):
        c = Case(seqs, hq=4, hkv=2, fmt=fmt, seed=83)
        x = Call(c, rot=0, weights="heads")
        x.norm = rdp.KVNorm(1e-6, False, None, 0, torch.full((128,), 1e30, device="cuda"), 0)
        before, exps = c.values()
        x.run()
        got, ge = c.values()
        assert c.s.device_status() == 0
        for s, (n, length) in enumerate(seqs):
            for h in range(2):
                p = c.table[s, 1, h, 0]
                held = length - n - c.bt
                assert ge[p] == 60
                new = got[p, held:held + n]
                k = x.k[c.indptr[s]:c.indptr[s] + n, h].astype(np.float64)
                r = 1 / np.sqrt((k ** 2).mean(-1, keepdims=True) + 1e-6)
                large = np.abs(k * r) > 1e-8                   # 1e22 and more, of 5e20
                assert np.array_equal(new[large], (R.LIMIT[fmt] * np.sign(k))[large])
                assert np.array_equal(got[p, :held], R.nearest(before[p, :held] * 2.0 ** (int(exps[p]) - 60), fmt))


def test_norm_in_place_and_rows_of_nobody():
    """q_out is q; rows outside every sequence are left as they were."""
    c = Case([(1, 33), (6, 20)], hq=4, hkv=2, seed=80)
    x = Call(c)
    _, _, want = x.check()
    rows, pad = c.hq * c.d, 3
    q = torch.full((c.T + 2 * pad, rows), 5.0, dtype=torch.float16, device="cuda")
    q[pad:pad + c.T] = x.buf[:, :rows]
    k = torch.ones((c.T + 2 * pad, 256), dtype=torch.float16, device="cuda")
    b = rdp.KVBatch(c.T + 2 * pad, 2, 6, c.max_blocks, dev(c.indptr + pad), c.d_len, c.d_table)
    rdp.slora_kv_append_norm(c.s.kv, b, k, 256, k, 256, q, rows, q, rows, 4, x.norm, x.rope)
    torch.cuda.synchronize()
    got = q.cpu().view(torch.int16).numpy().view(np.float16)
    assert np.array_equal(got[pad:pad + c.T].view(np.uint16), want[:, :rows].view(np.uint16))
    assert (got[:pad] == 5).all() and (got[pad + c.T:] == 5).all() and c.s.device_status() == 0


def test_norm_refusals():
    c = Case([(1, 10), (2, 20)], hq=4, hkv=2, seed=81)
    row = 4 * 128
    q, k = half(c.q).view(-1, row), torch.zeros((c.T, 256), dtype=torch.float16, device="cuda")
    out, w = torch.zeros_like(q), torch.ones((4, 132), device="cuda")
    tab = torch.zeros((32, 64), device="cuda")
    before, exps = c.s.pages.clone(), c.s.exponents.clone()

    def call(norm, rope=None, q=q, qo=out, b=None):
        rdp.slora_kv_append_norm(c.s.kv, b or c.batch(), k, 256, k, 256, q, row, qo, row, 4, norm, rope)

    good = rdp.KVNorm(1e-6)
    odd = rdp.KVNorm(1e-6)
    odd.centered = 2
    rope = rdp.KVRope(128, 0, 0, tab, tab)
    bad = [(dict(norm=n), None) for n in (
        None, odd, rdp.KVNorm(-1e-6), rdp.KVNorm(float("nan")), rdp.KVNorm(float("inf")), rdp.KVNorm(1e-6, False, w.data_ptr() + 4),
        rdp.KVNorm(1e-6, False, w, 64), rdp.KVNorm(1e-6, False, w, 130), rdp.KVNorm(1e-6, False, None, 0, w.data_ptr() + 8),
        rdp.KVNorm(1e-6, False, None, 0, w, -128))]
    bad += [(dict(norm=good, rope=rope), None), (dict(norm=good, qo=None), None), (dict(norm=good, q=None), None)]
    for kw, _ in bad:
        with pytest.raises(rdp.SloraError) as e:
            call(**kw)
        assert e.value.status == 1
    with pytest.raises(rdp.SloraError) as e:
        rdp.slora_kv_append_norm(None, c.batch(), k, 256, k, 256, norm=good)
    assert e.value.status == 1
    empty = torch.empty((0, row), dtype=torch.float16, device="cuda")
    call(good, q=empty, qo=empty, b=rdp.KVBatch(0, 0, 1, 1, None, None, None))
    torch.cuda.synchronize()
    assert torch.equal(before, c.s.pages) and torch.equal(exps, c.s.exponents) and (out == 0).all()
    assert c.s.device_status() == 0
    assert ctypes.sizeof(rdp.KVNorm) == 40
