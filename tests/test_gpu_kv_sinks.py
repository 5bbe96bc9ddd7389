"""GPU checks of attention with a window and sinks over the 8-bit KV cache against its definition in fp64: every
placing of the sinks before the window, block and tile edges, short and long sequences, pages given back in
between, entries that cannot be used, NaN, and the call's refusals.

The tolerances are those of tests/kv_reference.py: the sums are the same over fewer keys.
"""
import numpy as np
import pytest
import torch

import kv_reference as R
import rank_delta_paged_gb300 as rdp
from test_gpu_kv import Case, dev, half

pytestmark = pytest.mark.gpu
BAD_PAGE, TIMEOUT = 3, 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


def visible(n, length, window, sinks):
    """[n][length]: what each of the last n positions sees."""
    p, j = length - n + np.arange(n)[:, None], np.arange(length)[None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def give_back(c, window, sinks):
    """Blocks that no new token of a sequence sees are gone from the table."""
    for s, (n, length) in enumerate(c.seqs):
        if n == 0 or length == 0:
            c.table[s] = -1
            continue
        used = visible(n, length, window, sinks).any(0)
        for b in range(-(-length // c.bt)):
            if not used[b * c.bt:(b + 1) * c.bt].any():
                c.table[s, b] = -1
    c.d_table = dev(c.table)


def reference(c, window, sinks, scale, missing=()):
    """fp64 (out, lse, tolerance of out, tolerance of lse); `missing`: (sequence, block, head) that are not seen."""
    val, exps = c.values()
    T, hq, d, bt = c.T, c.hq, c.d, c.bt
    g = hq // c.hkv
    out, lse = np.zeros((T, hq, d)), np.full((T, hq), -np.inf)
    t_out, t_lse = np.zeros((T, hq, d)), np.zeros((T, hq))
    for s, (n, L) in enumerate(c.seqs):
        if n == 0 or L == 0:
            continue
        t0 = c.indptr[s]
        see0 = visible(n, L, window, sinks)
        keys = np.nonzero(see0.any(0))[0]
        for h in range(c.hkv):
            see = see0[:, keys] & ~np.isin(keys // bt, [b for (x, b, y) in missing if (x, y) == (s, h)])[None]
            page = c.table[s, keys // bt, h]
            ok = see.any(0)
            page = np.where(ok[:, None], page, 0)
            kk, vv = (np.where(ok[:, None], val[page[:, w], keys % bt] * 2.0 ** exps[page[:, w]].astype(float)[:, None], 0) for w in (0, 1))
            q = c.q[t0:t0 + n, h * g:(h + 1) * g].astype(np.float64)
            z = np.where(see[:, None], np.einsum("ngd,kd->ngk", q, kk) * scale, -np.inf)
            m = z.max(-1, initial=-np.inf)
            m0 = np.where(np.isinf(m), 0.0, m)
            p = np.exp(z - m0[..., None])
            l = p.sum(-1)
            w = p / np.where(l > 0, l, 1.0)[..., None]
            at = (slice(t0, t0 + n), slice(h * g, (h + 1) * g))
            out[at] = w @ vv
            with np.errstate(divide="ignore"):
                lse[at] = np.where(l > 0, m0 + np.log(l), -np.inf)
            ds = np.where(see[:, None], np.einsum("ngd,kd->ngk", np.abs(q), np.abs(kk)), 0).max(-1, initial=0) * abs(scale) * (d + 8) * 2.0 ** -24
            ds = ds + 2.0 ** -21 + len(keys) * 2.0 ** -24
            t_out[at] = (2.0 ** -11 * 1.01 + 2 * ds[..., None]) * (w @ np.abs(vv)) + 2.0 ** -11 * np.abs(out[at]) + 2.0 ** -24
            t_lse[at] = ds + 2.0 ** -21 * (1 + np.abs(np.where(l > 0, lse[at], 0)))
    return out, lse, t_out, t_lse


def attend(c, window, sinks, scale=None, pad=0, want_lse=True, max_q=None, stream=None):
    scale = 0.5 / np.sqrt(c.d) if scale is None else scale
    row = c.hq * c.d
    qb = torch.full((max(c.T, 1), row + pad), float("nan"), dtype=torch.float16, device="cuda")
    qb[:, :row] = half(c.q).view(-1, row)
    ob = torch.full((max(c.T, 1), row + 2 * pad), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((max(c.T, 1), c.hq), 7.0, device="cuda") if want_lse else None
    torch.cuda.synchronize()
    rdp.slora_kv_attend_sinks(c.s.kv, c.batch(max_q), qb, row + pad, c.hq, ob, row + 2 * pad, lse, scale, window, sinks, stream)
    torch.cuda.synchronize()
    assert (ob[:, row:] == 7).all()
    out = ob[:, :row].float().cpu().numpy().reshape(-1, c.hq, c.d)
    return out, None if lse is None else lse.cpu().numpy()


def check(c, window, sinks, scale=None, missing=(), status=0, **kw):
    out, lse = attend(c, window, sinks, scale, **kw)
    assert c.s.device_status() == status
    ref, rl, to, tl = reference(c, window, sinks, 0.5 / np.sqrt(c.d) if scale is None else scale, missing)
    err = np.abs(out - ref)
    assert np.isfinite(out).all()
    assert (err <= to).all(), f"worst {np.max(err / to)} of the tolerance at {np.unravel_index(np.argmax(err / to), err.shape)}"
    if lse is not None:
        assert np.array_equal(np.isinf(lse), np.isinf(rl))
        ok = np.isfinite(rl)
        assert np.max(np.abs(lse[ok] - rl[ok]) / tl[ok], initial=0) <= 1
    return out, lse


ONE = [(1, n) for n in (1, 2, 4, 5, 15, 16, 17, 63, 64, 65, 79, 80, 81, 127, 128, 129, 190, 255, 256, 257, 1000, 2077)]
FEW = [(3, 3), (1, 40), (8, 71), (2, 130), (5, 64), (0, 50), (7, 500), (16, 16), (1, 1), (4, 1999)]
MANY = [(129, 129), (1, 77), (200, 333), (64, 64), (127, 128), (257, 300), (31, 500), (1, 1), (300, 1500), (40, 1041)]


@pytest.mark.parametrize("seqs,hq", [(ONE, 8), (FEW, 4), (FEW, 12), (MANY, 4), (MANY, 12)])
@pytest.mark.parametrize("window", [1, 2, 15, 64, 65, 100, 700])
@pytest.mark.parametrize("sinks", [1, 4, 16, 17, 63, 64, 130])
def test_sinks_and_windows(seqs, hq, window, sinks):
    c = Case(seqs, hq=hq, hkv=2 if hq < 12 else 4, d=64 if sinks % 2 else 128, fmt="int8" if window % 2 else "e4m3", seed=300)
    give_back(c, window, sinks)
    check(c, window, sinks)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,hidden", [(128, 5120), (64, 4096), (64, 256), (128, 2048), (128, 640), (64, 8192), (64, 320)])
@pytest.mark.parametrize("sinks", [3, 24, 100])
def test_sinks_in_pages_of_every_size(fmt, d, hidden, sinks):
    for seqs, hq in ((ONE, 8), (FEW, 2), (MANY, 6)):
        c = Case(seqs, hq=hq, hkv=2, d=d, hidden=hidden, fmt=fmt, seed=301)
        give_back(c, 90, sinks)
        check(c, 90, sinks)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (40, 40), (7, 1), (16, 1), (17, 1), (71, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_sinks_head_layouts(hq, hkv, d):
    c = Case([(1, 70), (1, 3), (1, 333), (40, 333), (3, 500)], hq=hq, hkv=hkv, d=d, seed=302)
    give_back(c, 50, 9)
    check(c, 50, 9)


@pytest.mark.parametrize("sinks", [1, 64, 1 << 30])
def test_a_window_that_sees_everything(sinks):
    """Nothing lies between: the results of plain causal attention."""
    c = Case([(1, 300), (2, 77), (150, 400), (4, 2), (20, 0)], hq=4, hkv=2, seed=303)
    want, wl = c.attend()
    for window in (400, 5000, (1 << 31) - 1):
        out, lse = check(c, window, sinks)
        assert np.allclose(out, want, atol=2e-2) and np.allclose(lse, wl, atol=1e-4)


def test_no_sinks_is_the_window_alone():
    c = Case([(1, 300), (2, 77), (150, 400)], hq=4, hkv=2, seed=304)
    a, la = c.attend(window=60)
    b, lb = attend(c, 60, 0)
    assert np.array_equal(a, b) and np.array_equal(la, lb)


@pytest.mark.parametrize("sinks", [5, 1 << 30])
def test_rows_that_see_nothing(sinks):
    c = Case([(1, 0), (1, 5), (4, 2), (3, 0), (150, 140), (20, 0)], hq=4, hkv=2, seed=305)
    out, lse = check(c, 9, sinks)
    for t in (0, 2, 3, 6, 7, 8, 9, 18):
        assert (out[t] == 0).all() and (lse[t] == -np.inf).all()


def test_sinks_strides_and_no_lse():
    c = Case([(1, 100), (33, 700), (2, 2)], hq=12, hkv=4, seed=306)
    a, _ = check(c, 7, 3, pad=40)
    b, none = attend(c, 7, 3, want_lse=False)
    assert none is None and np.array_equal(a, b)


def test_sinks_scales_far_apart_and_large_scores():
    c = Case([(1, 900), (1, 64), (2, 500), (140, 600)], hq=4, hkv=1, seed=307, spread=12)
    check(c, 300, 20)
    check(Case([(1, 500), (3, 333), (130, 400)], hq=4, hkv=2, seed=308), 150, 40, scale=4.0)


def test_long_streams_are_split_and_joined():
    for seqs, kw, window, sinks in (([(1, 50011)], dict(hq=4, hkv=1), 20000, 4),
                                    ([(1, 9001), (1, 3), (2, 12345)], dict(hq=3, hkv=3, d=64, hidden=2048, fmt="int8"), 7777, 900),
                                    ([(140, 9001), (1, 3), (200, 16000)], dict(hq=2, hkv=1), 6000, 128)):
        c = Case(seqs, seed=309, **kw)
        give_back(c, window, sinks)
        a, la = check(c, window, sinks)
        st = torch.cuda.Stream()
        for stream in (None, st, st):
            b, lb = attend(c, window, sinks, stream=stream)
            assert np.array_equal(a, b) and np.array_equal(la, lb)


def test_positions_past_a_million():
    """A stream far along: only the sinks' block and the window's have pages."""
    c = Case([(1, 200), (3, 333)], hq=2, hkv=1, d=128, hidden=4096, seed=310)
    bt, window, sinks = c.bt, 70, 5
    far = [(1 << 22) + 13, (1 << 20) + 77]
    table = np.full((2, (far[0] + bt) // bt, 1, 2), -1, np.int32)
    for s, (n, L) in enumerate(c.seqs):
        shift = (far[s] - L) // bt * bt                    # whole blocks: the rows stand where they stood in theirs
        far[s] = L + shift
        table[s, 0] = c.table[s, 0]
        first = max(1, (L - n - window + 1) // bt)
        assert first > 0
        table[s, first + shift // bt:-(-far[s] // bt)] = c.table[s, first:-(-L // bt)]
    a, la = check(c, window, sinks)
    lens = dev(np.array(far, np.int32))
    b = rdp.KVBatch(c.T, 2, 3, table.shape[1], c.d_indptr, lens, dev(table))
    q, out = half(c.q).view(-1, 256), torch.zeros((c.T, 256), dtype=torch.float16, device="cuda")
    lse = torch.zeros((c.T, 2), device="cuda")
    rdp.slora_kv_attend_sinks(c.s.kv, b, q, 256, 2, out, 256, lse, 0.5 / np.sqrt(128), window, sinks)
    torch.cuda.synchronize()
    assert c.s.device_status() == 0
    assert np.array_equal(out.float().cpu().numpy().reshape(a.shape), a) and np.array_equal(lse.cpu().numpy(), la)


def test_many_sequences_with_sinks():
    rng = np.random.default_rng(0)
    seqs = [(int(rng.integers(0, 3)), int(rng.integers(3, 300))) for _ in range(2500)]
    c = Case(seqs, hq=2, hkv=1, d=64, hidden=2048, seed=311)
    give_back(c, 60, 4)
    check(c, 60, 4)
    seqs = [(int(rng.integers(30, 41)), int(rng.integers(41, 300))) for _ in range(900)] + [(1, 200)] * 400 + [(0, 0)] * 50
    c = Case(seqs, hq=2, hkv=1, d=64, hidden=2048, seed=312)
    give_back(c, 60, 4)
    check(c, 60, 4)


@pytest.mark.parametrize("seqs", [[(70, 400), (40, 400), (130, 333)], [(1, 400), (2, 300), (4, 333)], [(130, 333)] + [(1, 400)] * 200],
                         ids=["prompts", "stream", "mixed"])
@pytest.mark.parametrize("d,hidden", [(128, 4096), (64, 256)])
@pytest.mark.parametrize("block", ["first", "last"])
@pytest.mark.parametrize("which", [0, 1])
def test_bad_pages_are_not_seen(seqs, d, hidden, block, which):
    """Of the sinks or of the window; the others keep their results bit for bit."""
    c = Case(seqs, hq=8, hkv=2, d=d, hidden=hidden, seed=313)
    window, sinks = 100, 6
    give_back(c, window, sinks)
    want, wl = attend(c, window, sinks)
    for s, h in ((0, 0), (len(seqs) - 1, 1)):
        b = 0 if block == "first" else (seqs[s][1] - 1) // c.bt
        keep = c.table[s, b, h, which]
        for page in (-1, -(1 << 31), len(c.pages), (1 << 31) - 1):
            c.table[s, b, h, which] = page
            c.d_table = dev(c.table)
            out, lse = check(c, window, sinks, missing=[(s, b, h)], status=BAD_PAGE)
            mine = np.zeros(out.shape[:2], bool)
            mine[c.indptr[s]:c.indptr[s + 1], 4 * h:4 * h + 4] = True
            assert np.array_equal(out[~mine], want[~mine]) and np.array_equal(lse[~mine], wl[~mine])
        c.table[s, b, h, which] = keep
    c.d_table = dev(c.table)
    out, lse = attend(c, window, sinks)
    assert np.array_equal(out, want) and np.array_equal(lse, wl) and c.s.device_status() == 0


@pytest.mark.parametrize("seqs", [[(1, 400)], [(5, 400)], [(140, 500)]], ids=["one", "few", "prompt"])
def test_nan_values_reach_those_that_see_them(seqs):
    """Among the sinks, in the window of some rows, and in rows that nobody sees."""
    window, sinks = 60, 10
    (n, L), = seqs
    for at in (3, 9, 10, 15, L - n - window + 1, L - 30, L - 1, L - n - window):
        c = Case(seqs, hq=4, hkv=2, seed=314)
        clean, cl = check(c, window, sinks)
        ref, _, to, _ = reference(c, window, sinks, 0.5 / np.sqrt(c.d))
        page = c.table[0, at // c.bt, 1, 1]
        c.pages[page, at % c.bt * c.d + 77] = 0x7F
        c.push()
        got, gl = attend(c, window, sinks)
        see = visible(n, L, window, sinks)[:, at]
        assert np.array_equal(gl, cl)
        assert np.isnan(got[see][:, 2:, 77]).all()
        # (a prompt's rows that do not see it may have been summed again)
        assert (np.abs(got - ref)[~see] <= to[~see]).all()
        got[:, 2:, 77] = clean[:, 2:, 77]
        assert np.array_equal(got, clean)


def test_inf_and_nan_queries_stay_in_their_rows():
    c = Case([(1, 100), (2, 200), (140, 300)], hq=4, hkv=2, seed=315)
    clean, _ = attend(c, 40, 5)
    c.q[0, 0, 3], c.q[2, 1, 0], c.q[60, 2, 5] = np.nan, np.inf, np.nan
    got, _ = attend(c, 40, 5)
    for t, h in ((0, 0), (2, 1), (60, 2)):
        assert np.isnan(got[t, h]).all()
        got[t, h] = clean[t, h]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("seqs", [[(1, 9000), (4, 100)], [(140, 5000), (1, 90), (60, 60)]], ids=["stream", "prompts"])
def test_sinks_in_a_graph_between_other_attends(seqs):
    """One workspace for all: plain and sinks attention by turns, eager and replayed."""
    c = Case(seqs, hq=8, hkv=2, seed=316)
    window, sinks = 2500, 70
    plain, want = c.attend()[0], attend(c, window, sinks)[0]
    row = c.hq * c.d
    q, out, o2 = half(c.q).view(-1, row), torch.zeros((c.T, row), dtype=torch.float16, device="cuda"), torch.zeros((c.T, row), dtype=torch.float16, device="cuda")
    b = c.batch()
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        rdp.slora_kv_attend_sinks(c.s.kv, b, q, row, c.hq, out, row, None, 0.5 / np.sqrt(c.d), window, sinks, st)
        rdp.slora_kv_attend(c.s.kv, b, q, row, c.hq, o2, row, None, 0.5 / np.sqrt(c.d), True, 0, st)
    for _ in range(3):
        out.zero_()
        o2.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.float().cpu().numpy().reshape(want.shape), want)
        assert np.array_equal(o2.float().cpu().numpy().reshape(plain.shape), plain)
        assert np.array_equal(attend(c, window, sinks)[0], want) and np.array_equal(c.attend()[0], plain)


@pytest.mark.parametrize("seqs", [[(1, 60)] * 40, [(60, 200)] * 30], ids=["stream", "prompts"])
def test_a_cta_that_gives_up_ends_and_reports_it(seqs):
    c = Case(seqs, hq=8, hkv=2, seed=317)
    want, wl = attend(c, 50, 4)
    try:
        for cta in (0, 7):
            rdp.slora_debug_kv_give_up(cta)
            attend(c, 50, 4)
            assert c.s.device_status() == TIMEOUT
            rdp.slora_debug_kv_give_up(-1)
            out, lse = attend(c, 50, 4)
            assert np.array_equal(out, want) and np.array_equal(lse, wl) and c.s.device_status() == 0
    finally:
        rdp.slora_debug_kv_give_up(-1)


def test_sinks_refusals():
    c = Case([(1, 10), (2, 20)], hq=4, hkv=2, seed=318)
    row = 512
    q = half(c.q).view(-1, row)
    out = torch.zeros_like(q)

    def call(b=None, q=q, qs=row, hq=4, out=out, os=row, lse=None, scale=1.0, window=8, sinks=4, kv=c.s.kv):
        rdp.slora_kv_attend_sinks(kv, b or c.batch(), q, qs, hq, out, os, lse, scale, window, sinks)

    for bad in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(sinks=(1 << 30) + 1), dict(kv=None), dict(q=None), dict(out=None),
                dict(out=q), dict(q=q.data_ptr() + 8), dict(qs=row - 8), dict(os=row + 1), dict(hq=3), dict(hq=0), dict(scale=float("nan")),
                dict(lse=out.data_ptr() + 2)):
        with pytest.raises(rdp.SloraError) as e:
            call(**bad)
        assert e.value.status == 1
    empty = torch.empty((0, row), dtype=torch.float16, device="cuda")
    call(b=rdp.KVBatch(0, 0, 1, 1, None, None, None), q=empty, out=empty)
    torch.cuda.synchronize()
    assert (out == 0).all() and c.s.device_status() == 0
