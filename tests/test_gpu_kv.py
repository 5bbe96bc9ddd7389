"""GPU checks of the 8-bit KV cache: append and attention against their definitions in fp64
(tests/kv_reference.py), at block edges, ragged lengths, strides, windows, empty rows, stale
pages and every head layout class, and the calls' refusals."""
import ctypes

import numpy as np
import pytest
import torch

import kv_reference as R
import rank_delta_paged_gb300 as rdp
from rank_delta_paged_gb300.harness import KVSession

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def half(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.float16)


class Case:
    """A cache with scattered pages, random codes everywhere (NaN codes and other formats' bytes
    among the rows that no sequence has), and a batch over it."""

    def __init__(self, seqs, hq=8, hkv=2, d=128, hidden=4096, fmt="e4m3", seed=0, spare=3, stale=True, spread=3):
        self.rng = rng = np.random.default_rng(seed)
        self.seqs, self.hq, self.hkv, self.d, self.fmt = seqs, hq, hkv, d, fmt
        self.bt = bt = hidden * 2 // d // 8 * 8
        nb = [-(-n // bt) for _, n in seqs]
        self.max_blocks = max(nb + [1]) + 1
        num = max(1, 2 * hkv * sum(nb)) + spare
        self.s = KVSession(hidden, num, hkv, d, fmt)
        assert self.s.block == bt
        ids = rng.permutation(num).astype(np.int32)
        self.table = np.full((len(seqs), self.max_blocks, hkv, 2), -1, np.int32)
        at = 0
        for i, b in enumerate(nb):
            self.table[i, :b] = ids[at:at + b * hkv * 2].reshape(b, hkv, 2)
            at += b * hkv * 2
        self.indptr = np.concatenate([[0], np.cumsum([q for q, _ in seqs])]).astype(np.int32)
        self.kv_len = np.array([n for _, n in seqs], np.int32)
        self.T = int(self.indptr[-1])
        self.pages = rng.integers(0, 256, (num, hidden * 2), dtype=np.uint8)
        if not stale:
            self.pages[:] = 0
        self.exps = rng.integers(-8 - spread, -8 + spread + 1, num).astype(np.int8)
        # rows that sequences hold: finite codes
        for i, (_, n) in enumerate(seqs):
            for b in range(nb[i]):
                rows = min(bt, n - b * bt)
                for p in self.table[i, b].ravel():
                    c = rng.normal(0, 60, (rows, d))
                    if fmt == "e4m3":
                        c = torch.from_numpy(c.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                    else:
                        c = np.clip(np.rint(c), -127, 127).astype(np.int8).view(np.uint8)
                    self.pages[p, :rows * d] = c.ravel()
        self.push()
        self.q = rng.normal(0, 1, (max(self.T, 1), hq, d)).astype(np.float16)

    def push(self):
        self.s.pages.copy_(dev(self.pages))
        self.s.exponents.copy_(dev(self.exps))
        self.d_table, self.d_indptr, self.d_len = dev(self.table), dev(self.indptr), dev(self.kv_len)

    def batch(self, max_q=None):
        mq = max([q for q, _ in self.seqs] + [1]) if max_q is None else max_q
        return rdp.KVBatch(self.T, len(self.seqs), mq, self.max_blocks, self.d_indptr, self.d_len, self.d_table)

    def values(self):
        """Code values fp64 [num_pages][bt][d] as they stand on the device."""
        torch.cuda.synchronize()
        p = self.s.pages.cpu().numpy()[:, :self.bt * self.d].reshape(-1, self.bt, self.d)
        return R.decode(np.ascontiguousarray(p), self.fmt), self.s.exponents.cpu().numpy()

    def attend(self, causal=True, window=0, scale=None, pad=0, want_lse=True, max_q=None, stream=None):
        scale = 0.5 / np.sqrt(self.d) if scale is None else scale
        row = self.hq * self.d
        qb = torch.full((max(self.T, 1), row + pad), float("nan"), dtype=torch.float16, device="cuda")
        qb[:, :row] = half(self.q).view(-1, row)
        ob = torch.full((max(self.T, 1), row + 2 * pad), 7.0, dtype=torch.float16, device="cuda")
        lse = torch.full((max(self.T, 1), self.hq), 7.0, device="cuda") if want_lse else None
        torch.cuda.synchronize()
        rdp.slora_kv_attend(self.s.kv, self.batch(max_q), qb, row + pad, self.hq, ob, row + 2 * pad, lse, scale, causal,
                            window, stream)
        torch.cuda.synchronize()
        assert (ob[:, row:] == 7).all()
        out = ob[:, :row].float().cpu().numpy().reshape(-1, self.hq, self.d)
        return out, None if lse is None else lse.cpu().numpy()

    def check(self, **kw):
        out, lse = self.attend(**kw)
        assert self.s.device_status() == 0
        val, exps = self.values()
        scale = kw.get("scale") or 0.5 / np.sqrt(self.d)
        ref, rl, to, tl = R.attend(val, exps, self.table, self.indptr, self.kv_len, self.q, self.bt, scale,
                                   kw.get("causal", True), kw.get("window", 0))
        err = np.abs(out - ref)
        assert np.isfinite(out).all()
        assert (err <= to).all(), f"worst {np.max(err / to)} of the tolerance at {np.unravel_index(np.argmax(err / to), err.shape)}"
        if lse is not None:
            assert np.array_equal(np.isinf(lse), np.isinf(rl))
            ok = np.isfinite(rl)
            worst = np.max(np.abs(lse[ok] - rl[ok]) / tl[ok])
            assert worst <= 1, worst
        return out, lse


DECODE = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65), (1, 79), (1, 80), (1, 81), (1, 127),
          (1, 128), (1, 129), (1, 1000)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,hidden", [(128, 4096), (128, 5120), (64, 4096), (64, 256), (128, 2048), (128, 640)])
def test_attend_single_tokens_at_every_edge(fmt, d, hidden):
    Case(DECODE, hq=8, hkv=2, d=d, hidden=hidden, fmt=fmt, seed=1).check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (40, 40), (6, 2), (7, 1), (14, 2), (16, 1), (17, 1), (32, 2), (71, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_head_layouts(hq, hkv, d):
    Case([(1, 70), (1, 3), (1, 333)], hq=hq, hkv=hkv, d=d, seed=2).check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (8, 2), (12, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_several_tokens(fmt, hq, hkv, d):
    Case([(3, 3), (1, 40), (8, 71), (2, 130), (5, 64), (0, 50), (7, 500), (16, 16), (1, 1)], hq=hq, hkv=hkv, d=d, fmt=fmt,
         seed=3).check()


@pytest.mark.parametrize("fmt,d,hidden,hq,hkv", [("e4m3", 128, 4096, 8, 2), ("int8", 128, 5120, 3, 3), ("e4m3", 64, 4096, 4, 1),
                                                  ("int8", 64, 256, 4, 4), ("int8", 128, 640, 6, 2)])
def test_attend_prompts(fmt, d, hidden, hq, hkv):
    Case([(129, 129), (1, 77), (200, 333), (64, 64), (127, 128), (257, 300), (31, 500), (1, 1)], hq=hq, hkv=hkv, d=d,
         hidden=hidden, fmt=fmt, seed=4).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 15, 64, 65, 100, 5000])
def test_attend_window(d, window):
    c = Case([(1, 1), (1, 64), (1, 200), (5, 130), (1, 777), (40, 300), (150, 400)], hq=4, hkv=2, d=d, fmt="int8", seed=5)
    # blocks that the window has left behind are gone from the table
    for i, (n, length) in enumerate(c.seqs):
        first = max(0, length - n - window + 1) // c.bt
        c.table[i, :first] = -1
    c.push()
    c.check(window=window)


@pytest.mark.parametrize("n", [1, 3, 40, 150])
def test_attend_not_causal(n):
    Case([(n, 200), (n, 150), (1, 9)], hq=4, hkv=2, seed=6).check(causal=False)


def test_attend_rows_that_see_nothing():
    c = Case([(1, 0), (1, 5), (4, 2), (3, 0), (150, 140), (20, 0)], hq=4, hkv=2, seed=7)
    out, lse = c.check()
    for t in (0, 2, 3, 6, 7, 8, 9, 18):
        assert (out[t] == 0).all() and (lse[t] == -np.inf).all()


def test_attend_rows_out_of_the_window_and_strides_and_no_lse():
    c = Case([(1, 100), (33, 700), (2, 2)], hq=12, hkv=4, seed=8)
    a, _ = c.check(pad=40, window=7)
    b, none = c.attend(window=7, want_lse=False)
    assert none is None and np.array_equal(a, b)


@pytest.mark.parametrize("spread", [0, 12])
def test_attend_scales_far_apart(spread):
    """Value pages whose scales differ by up to 2^24, key pages likewise: the weights share one scale."""
    Case([(1, 900), (1, 64), (2, 500), (140, 600)], hq=4, hkv=1, d=128, seed=9, spread=spread).check()


def test_attend_large_scores():
    """Scores of hundreds: one key dominates, the running maximum climbs."""
    Case([(1, 500), (3, 333), (130, 400)], hq=4, hkv=2, seed=10).check(scale=4.0)


@pytest.mark.parametrize("scale", [3e4, -3e4, 1e30, -1e30, 0.0])
@pytest.mark.parametrize("n", [1, 140])
def test_attend_scores_beyond_fp32s_fractions(scale, n):
    """Scores so large that fp32 holds no fraction of them (and past its range at 1e30, and all equal at 0):
    the rows stay within the values they average, or are NaN where a score is infinite."""
    c = Case([(n, 400)], hq=4, hkv=2, seed=33, stale=False)
    out, lse = c.attend(scale=scale)
    assert c.s.device_status() == 0
    val, exps = c.values()
    for h in range(2):
        pages = c.table[0, :-(-400 // c.bt), h, 1]
        top = np.abs(val[pages] * 2.0 ** exps[pages][:, None, None]).max()
        got = out[:, 2 * h:2 * h + 2]
        if abs(scale) < 1e20:
            assert np.isfinite(got).all() and np.abs(got).max() <= top * 1.001
        else:
            assert (np.isnan(got) | (np.abs(got) <= top * 1.001)).all()
    if scale == 0:
        for t in range(n):
            assert np.allclose(lse[t], np.log(400 - n + 1 + t), atol=1e-5)


def test_attend_rising_scores():
    """Every tile's scores pass the ones before by more than the rescaling threshold."""
    c = Case([(1, 1000), (130, 1000)], hq=2, hkv=1, seed=11, stale=False)
    c.q[:] = 1.0
    for b in range(-(-1000 // c.bt)):
        for i in range(2):
            c.pages[c.table[i, b, 0, 0], :c.bt * c.d] = 0x38      # 1.0
            c.exps[c.table[i, b, 0, 0]] = b // 2 - 3
    c.push()
    c.check(scale=0.2)


def test_attend_long_and_few_rows_is_split_and_joined():
    Case([(1, 20011)], hq=4, hkv=1, seed=12).check()
    Case([(1, 9001), (1, 3), (2, 12345)], hq=3, hkv=3, d=64, hidden=2048, fmt="int8", seed=13).check()
    Case([(140, 9001), (1, 3), (200, 6000)], hq=2, hkv=1, d=128, seed=14).check()


def test_attend_many_sequences():
    rng = np.random.default_rng(0)
    Case([(int(rng.integers(0, 3)), int(rng.integers(3, 40))) for _ in range(2500)], hq=2, hkv=1, d=64, hidden=2048,
         seed=15).check()


def test_attend_repeats_bit_for_bit_and_on_another_stream():
    c = Case([(1, 4000), (3, 300), (200, 500)], hq=8, hkv=2, seed=16)
    a, la = c.attend()
    st = torch.cuda.Stream()
    for stream in (None, st, st, None):
        b, lb = c.attend(stream=stream)
        assert np.array_equal(a, b) and np.array_equal(la, lb)


def test_attend_does_not_depend_on_max_q_or_neighbours():
    c = Case([(1, 300), (20, 300)], hq=4, hkv=2, seed=17)
    c.check(max_q=1 << 20)
    c.check()


def test_attend_inf_and_nan_queries_stay_in_their_rows():
    c = Case([(1, 100), (2, 200), (140, 300)], hq=4, hkv=2, seed=18)
    clean, _ = c.attend()
    c.q[0, 0, 3], c.q[2, 1, 0], c.q[60, 2, 5] = np.nan, np.inf, np.nan
    got, _ = c.attend()
    for t, h in ((0, 0), (2, 1), (60, 2)):
        assert np.isnan(got[t, h]).all()
        got[t, h] = clean[t, h]
    assert np.array_equal(got, clean)


def test_attend_in_a_graph():
    c = Case([(1, 500), (4, 100)], hq=8, hkv=2, seed=19)
    want, _ = c.attend()
    row = c.hq * c.d
    q, out = half(c.q).view(-1, row), torch.zeros((c.T, row), dtype=torch.float16, device="cuda")
    b = c.batch()
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        rdp.slora_kv_attend(c.s.kv, b, q, row, c.hq, out, row, None, 0.5 / np.sqrt(c.d), True, 0, st)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.float().cpu().numpy().reshape(want.shape), want)


# ---- append -------------------------------------------------------------------------------
def run_append(c, rot=128, interleaved=False, positions=None, packed=True, with_q=True, values=None, stream=None):
    """Appends random tokens; returns what the library wrote and what the definition gives."""
    rng = c.rng
    T, hq, hkv, d = c.T, c.hq, c.hkv, c.d
    k = rng.normal(0, 1, (T, hkv, d)).astype(np.float16)
    v = (rng.normal(0, 1, (T, hkv, d)) * np.exp(rng.normal(0, 2, (T, 1, 1)))).astype(np.float16)
    if values is not None:
        k, v = values(k, v)
    q = c.q
    row = (hq + 2 * hkv) * d if packed else None
    if packed:
        buf = half(np.concatenate([q.reshape(T, -1), k.reshape(T, -1), v.reshape(T, -1)], axis=1))
        dq, dk, dv = buf, buf[:, hq * d:], buf[:, (hq + hkv) * d:]
        sq = sk = sv = row
    else:
        dq, dk, dv = half(q), half(k), half(v)
        sq, sk, sv = hq * d, hkv * d, hkv * d
    n_pos = int(max(c.kv_len.max(), 1)) + 10
    angle = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot) if rot else None
    rope = None
    pos = np.concatenate([np.arange(n - m, n) for m, n in c.seqs]).astype(np.int32)
    if rot:
        cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
        if positions is not None:
            pos = positions(pos)
        dpos = None if positions is None else dev(pos)
        rope = rdp.KVRope(rot, interleaved, n_pos, dev(cos), dev(sin), dpos)
    q_out = torch.full((T, hq * d), 7.0, dtype=torch.float16, device="cuda")
    before_val, before_exp = c.values()
    torch.cuda.synchronize()
    if with_q and rot:
        rdp.slora_kv_append(c.s.kv, c.batch(), dk, sk, dv, sv, dq, sq, q_out, hq * d, hq, rope, stream)
    else:
        rdp.slora_kv_append(c.s.kv, c.batch(), dk, sk, dv, sv, rope=rope, stream=stream)
    torch.cuda.synchronize()
    k32, q32 = k.astype(np.float32), q.astype(np.float32)
    if rot:
        co, si = cos[pos], sin[pos]
        k64 = R.rotate(k, co, si, interleaved, np.float64)
        k32, q32 = R.rotate(k, co, si, interleaved, np.float32), R.rotate(q, co, si, interleaved, np.float32)
    else:
        k64 = k.astype(np.float64)
    want_val, want_exp = before_val.copy(), before_exp.copy()
    R.append(want_val, want_exp, c.table, c.indptr, c.kv_len, k32, v, c.bt, c.fmt)
    got_val, got_exp = c.values()
    return dict(got=got_val, got_exp=got_exp, want=want_val, want_exp=want_exp, k64=k64, v=v, q32=q32, before=before_val,
                before_exp=before_exp, q_out=q_out.cpu().view(torch.int16).numpy().view(np.float16).reshape(T, hq, d))


def check_append(c, **kw):
    bytes_before = c.s.pages.cpu().numpy()
    r = run_append(c, **kw)
    assert c.s.device_status() == 0
    # codes and exponents are those of the fp32 definition, every byte that is no new or held row is untouched
    assert np.array_equal(r["got_exp"], r["want_exp"])
    assert np.array_equal(r["got"], r["want"], equal_nan=True)
    after = c.s.pages.cpu().numpy()
    assert np.array_equal(after[:, c.bt * c.d:], bytes_before[:, c.bt * c.d:])
    same = np.zeros(after.shape, bool)
    same[:, :c.bt * c.d] = (np.nan_to_num(r["want"], nan=1e9) == np.nan_to_num(r["before"], nan=1e9)).reshape(len(after), -1)
    keep = same & ~np.isnan(np.concatenate([r["want"].reshape(len(after), -1),
                                            np.zeros((len(after), after.shape[1] - c.bt * c.d))], 1))
    changed = keep & (after != bytes_before)
    assert np.isin(after[changed] & 0x7F, [0]).all()      # only the sign of a zero
    if kw.get("rot", 128) and kw.get("with_q", True):
        assert np.array_equal(r["q_out"].view(np.uint16), r["q32"].astype(np.float16).view(np.uint16))
    # and within half a code of the values in 64 bits
    for s, (n, length) in enumerate(c.seqs):
        for i in range(n):
            p = length - n + i
            for w, src in enumerate((r["k64"], r["v"].astype(np.float64))):
                page = c.table[s, p // c.bt, :, w]
                x = src[c.indptr[s] + i]
                u = 2.0 ** -r["got_exp"][page].astype(np.float64)[:, None]
                got = r["got"][page, p % c.bt]
                fine = np.isfinite(x) & (np.abs(x * u) <= R.LIMIT[c.fmt])
                tol = R.half_step(np.where(fine, x * u, 0), c.fmt) * (1 + 2.0 ** -10) + np.abs(np.where(fine, x * u, 0)) * 2.0 ** -20
                assert (np.abs(got - x * u)[fine] <= tol[fine]).all()
    return r


APPEND = [(1, 1), (1, 64), (1, 65), (1, 200), (3, 3), (4, 66), (5, 68), (64, 64), (65, 65), (70, 131), (1, 80), (1, 81), (130, 400),
          (0, 10), (2, 161)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,hidden", [(128, 4096), (128, 5120), (64, 4096), (64, 256), (128, 640), (64, 8192), (128, 8192)])
def test_append_at_block_edges(fmt, d, hidden):
    check_append(Case(APPEND, hq=4, hkv=2, d=d, hidden=hidden, fmt=fmt, seed=20), rot=d)


@pytest.mark.parametrize("rot", [0, 16, 32, 48, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rotations(rot, interleaved):
    check_append(Case([(1, 70), (3, 10), (40, 90)], hq=6, hkv=3, seed=21), rot=rot, interleaved=interleaved)
    if rot <= 64:
        check_append(Case([(1, 70), (3, 10), (40, 90)], hq=5, hkv=5, d=64, seed=22), rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (40, 40), (7, 1), (9, 3), (64, 32)])
def test_append_head_layouts_and_layouts_of_rows(hq, hkv):
    for packed in (True, False):
        check_append(Case([(1, 33), (1, 100), (20, 70)], hq=hq, hkv=hkv, seed=23), packed=packed)
    check_append(Case([(1, 33), (1, 100), (20, 70)], hq=hq, hkv=hkv, seed=24), with_q=False)


def test_append_many_sequences():
    """Blocks are found through long stretches of sequences that have none."""
    rng = np.random.default_rng(3)
    few = [(int(rng.choice([0, 1, 1, 1, 2, 9])), int(rng.integers(9, 60))) for _ in range(2200)]
    seqs = [(0, 5)] * 70 + few + [(200, 333)] + [(1, 7)] * 400 + [(0, 0)] * 40 + [(33, 90), (1, 1)]
    check_append(Case(seqs, hq=2, hkv=1, d=64, hidden=512, seed=33), rot=64)
    check_append(Case([(1, 9)] * 2100 + [(2, 9)], hq=2, hkv=1, d=64, hidden=512, seed=34), rot=64)


def test_append_more_pages_than_a_cta_lists():
    """A CTA's run is longer than the pages it looks up at a time, and a block has more pages than that."""
    check_append(Case([(330, 400), (1, 5), (310, 310)], hq=512, hkv=512, d=64, hidden=512, seed=35, stale=False), rot=64,
                 with_q=False)


def test_append_given_positions():
    check_append(Case([(1, 33), (5, 100), (20, 70)], hq=4, hkv=2, seed=25), positions=lambda p: p[::-1] + 3)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_token_by_token_grows_the_scale(fmt):
    """A block filled one token at a time, each larger than the last: exponents grow, held rows follow."""
    for step in range(1, 90):
        if step == 1:
            c = Case([(1, 90), (1, 90)], hq=2, hkv=2, fmt=fmt, seed=26)
            table = c.table
        c.seqs = [(1, step), (1, step)]
        c.kv_len[:] = step
        c.d_len = dev(c.kv_len)
        grow = np.float16(1.3 ** (step % 40 - 20))
        check_append(c, values=lambda k, v: (k * grow, v * grow))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_zeros_infinities_and_nan(fmt):
    def odd(k, v):
        k[:], v[0] = 0, 0
        v[1, 0, 5], v[2, 1, 7], v[3, 0, 9] = np.inf, -np.inf, np.nan
        v[8, 1, 0], v[9] = np.nan, 6e-8
        v[10], k[10] = 65504, -65504
        return k, v
    for rot in (0, 128):
        check_append(Case([(1, 70), (8, 8), (2, 71), (30, 30)], hq=4, hkv=2, fmt=fmt, seed=27), rot=rot, values=odd)


def test_append_then_attend():
    """The two together: attention over what append wrote, within the codes' rounding of exact attention."""
    c = Case([(1, 70), (20, 20), (3, 131), (150, 150)], hq=8, hkv=2, seed=28)
    r = check_append(c)
    c.q = r["q_out"]
    c.check()


# ---- refusals -------------------------------------------------------------------------------
def refused(status, fn, *args, **kw):
    with pytest.raises(rdp.SloraError) as e:
        fn(*args, **kw)
    assert e.value.status == status, str(e.value)


def test_create_refusals():
    pool = rdp.slora_pool_create(0, 256, 8, 1, 1)
    try:
        refused(1, rdp.slora_kv_create, None, 1, 64)
        refused(1, rdp.slora_kv_create, pool, 0, 64)
        refused(1, rdp.slora_kv_create, pool, 1025, 64)
        refused(1, rdp.slora_kv_create, pool, 1, 64, 2)
        refused(11, rdp.slora_kv_create, pool, 1, 96)
        refused(11, rdp.slora_kv_create, pool, 1, 128)      # a 512-byte page holds 4 rows
        kv = rdp.slora_kv_create(pool, 1, 64)
        assert rdp.slora_kv_block_tokens(kv) == 8
        assert rdp.slora_kv_exponents(kv) % 16 == 0
        rdp.slora_kv_destroy(kv)
        rdp.slora_kv_destroy(None)
    finally:
        rdp.slora_pool_destroy(pool)


def test_call_refusals():
    c = Case([(1, 10), (2, 20)], hq=4, hkv=2)
    row, kvrow = 4 * 128, 2 * 128
    q = half(c.q).view(-1, row)
    out, k = torch.zeros_like(q), torch.zeros((c.T, kvrow), dtype=torch.float16, device="cuda")
    tab = torch.zeros((32, 64), device="cuda")
    good = c.batch()

    def attend(b=good, q=q, qs=row, hq=4, out=out, os=row, lse=None, scale=1.0, causal=True, window=0, kv=c.s.kv):
        rdp.slora_kv_attend(kv, b, q, qs, hq, out, os, lse, scale, causal, window)

    def append(b=good, k=k, ks=kvrow, v=k, vs=kvrow, q=None, qs=0, qo=None, qos=0, hq=0, rope=None, kv=c.s.kv):
        rdp.slora_kv_append(kv, b, k, ks, v, vs, q, qs, qo, qos, hq, rope)

    def batch(**kw):
        b = c.batch()
        for f, x in kw.items():
            setattr(b, f, x)
        return b

    for fn in (attend, append):
        for bad in (dict(n_tokens=-1), dict(n_tokens=(1 << 20) + 1), dict(n_seqs=-1), dict(n_seqs=(1 << 20) + 1),
                    dict(max_q=0), dict(max_blocks=0), dict(tok_indptr=None), dict(kv_len=None), dict(block_table=None)):
            refused(1, fn, b=batch(**bad))
        refused(1, fn, kv=None)
        fn(b=batch(n_tokens=0))
        fn(b=batch(n_seqs=0))
    for bad in (dict(q=None), dict(out=None), dict(out=q), dict(q=q.data_ptr() + 8), dict(out=out.data_ptr() + 2), dict(qs=row - 8),
                dict(qs=row + 4), dict(os=row - 8), dict(os=row + 1), dict(hq=3), dict(hq=0), dict(window=-1),
                dict(window=4, causal=False), dict(causal=2), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(lse=out.data_ptr() + 2)):
        refused(1, attend, **bad)
    rope = lambda rot=64, inter=0, n=32, cos=tab, sin=tab: rdp.KVRope(rot, inter, n, cos, sin)   # noqa: E731
    for bad in (dict(k=None), dict(v=None), dict(k=k.data_ptr() + 8), dict(ks=kvrow - 8), dict(vs=kvrow + 2), dict(q=q),
                dict(q=q, qs=row, qo=out, qos=row, hq=4), dict(qo=out, rope=rope()), dict(q=q, rope=rope()),
                dict(rope=rope(rot=0)), dict(rope=rope(rot=8)), dict(rope=rope(rot=144)), dict(rope=rope(inter=2)),
                dict(rope=rope(n=0)), dict(rope=rope(cos=None)), dict(rope=rope(sin=tab.data_ptr() + 4)),
                dict(q=q, qs=row, qo=out, qos=row, hq=0, rope=rope()), dict(q=q, qs=row - 8, qo=out, qos=row, hq=4, rope=rope()),
                dict(q=q, qs=row, qo=out, qos=row - 8, hq=4, rope=rope())):
        refused(1, append, **bad)
    assert (out == 0).all() and c.s.device_status() == 0


def test_device_checks_skip_the_work_and_set_the_status():
    seqs = [(1, 100), (2, 70), (1, 30)]
    c = Case(seqs, hq=4, hkv=2, seed=30)
    want, _ = c.attend()

    def expect(code, rows_kept):
        got, _ = c.attend()
        assert c.s.device_status() == code
        assert np.array_equal(got[rows_kept], want[rows_kept])
        before = c.values()
        T = c.T
        k = torch.ones((T, 2 * 128), dtype=torch.float16, device="cuda")
        rdp.slora_kv_append(c.s.kv, c.batch(), k, 256, k, 256)
        assert c.s.device_status() == code
        c.push()
        return got

    for page in (-7, 1 << 30):                                   # a bad page id: that block is not seen
        keep = c.table[1, 0].copy()
        c.table[1, 0, 0, 0] = page
        c.push()
        got, _ = c.attend()
        assert c.s.device_status() == 3
        assert np.array_equal(got[[0, 3]], want[[0, 3]]) and np.array_equal(got[1:3, 2:], want[1:3, 2:])
        assert np.isfinite(got).all()
        c.table[1, 0] = keep
    c.kv_len[1] = c.max_blocks * c.bt + 1                        # beyond the block table
    c.push()
    assert (expect(6, [0, 3])[1:3] == 7).all()
    c.kv_len[1] = -1
    c.push()
    expect(6, [0, 3])
    c.kv_len[1] = 70
    keep = c.indptr.copy()
    c.indptr[:] = [0, 1, 5, 5]                                   # past the last row
    c.push()
    assert (expect(4, [0])[1:] == 7).all()
    c.indptr[:] = [0, 1, 0, 4]                                   # decreasing
    c.push()
    expect(4, [0])
    c.indptr[:] = keep
    c.push()
    got, _ = c.attend()
    assert np.array_equal(got, want) and c.s.device_status() == 0


def test_append_device_checks():
    c = Case([(1, 100), (2, 70)], hq=4, hkv=2, seed=31)
    k = torch.ones((3, 256), dtype=torch.float16, device="cuda")
    tab = torch.ones((50, 64), device="cuda")
    q, qo = half(c.q).view(-1, 512), torch.zeros((3, 512), dtype=torch.float16, device="cuda")
    # positions 99, 68, 69 of a table of 50: unrotated, reported
    rdp.slora_kv_append(c.s.kv, c.batch(), k, 256, k, 256, q, 512, qo, 512, 4, rdp.KVRope(128, 0, 50, tab, tab))
    assert c.s.device_status() == 7
    assert torch.equal(q, qo)
    val, exps = c.values()
    assert (val[c.table[0, 1, :, 0], 99 - c.bt] * 2.0 ** exps[c.table[0, 1, :, 0]][:, None] == 1.0).all()
    # fewer keys than new tokens: the sequence is not written
    c.kv_len[1] = 1
    c.push()
    before = c.s.pages.clone()
    rdp.slora_kv_append(c.s.kv, c.batch(), k, 256, k, 256)
    assert c.s.device_status() == 6
    same = (c.s.pages == before).all(dim=1).cpu().numpy()
    assert same[c.table[1, 0].ravel()].all() and not same[c.table[0, 1].ravel()].all()


def test_lengths_past_the_positions_are_refused():
    # a block table wide enough by its own account, of which nothing may be read
    c = Case([(2, 70), (1, 30)], hq=4, hkv=2, seed=32)
    want, _ = c.attend()
    c.kv_len[0] = (1 << 30) + 1
    c.d_len = dev(c.kv_len)
    wide = (1 << 24) + 1
    b = rdp.KVBatch(c.T, 1, 2, wide, c.d_indptr, c.d_len, c.d_table)
    out = torch.full((c.T, 512), 7.0, dtype=torch.float16, device="cuda")
    rdp.slora_kv_attend(c.s.kv, b, half(c.q).view(-1, 512), 512, 4, out, 512)
    assert c.s.device_status() == 6
    assert (out == 7).all()
    before = c.s.pages.clone()
    k = torch.ones((c.T, 256), dtype=torch.float16, device="cuda")
    rdp.slora_kv_append(c.s.kv, b, k, 256, k, 256)
    assert c.s.device_status() == 6
    assert torch.equal(before, c.s.pages)
    c.kv_len[0] = 70
    c.push()
    assert np.array_equal(c.attend()[0], want)
