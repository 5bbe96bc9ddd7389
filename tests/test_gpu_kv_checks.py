"""GPU checks of what the 8-bit KV cache does with entries that it must not use: page ids, lengths and
token offsets out of range reach a status word, never memory, and every other block, head and
sequence of the call keeps its result bit for bit."""
import numpy as np
import pytest
import torch

import kv_reference as R
import rank_delta_paged_gb300 as rdp
from test_gpu_kv import Case, dev, half

pytestmark = pytest.mark.gpu

BAD_PAGE, BAD_SEGMENT, TIMEOUT, BAD_LENGTH, BAD_POSITION = 3, 4, 5, 6, 7


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


def masked_attend(c, s, h, missing, scale):
    """fp64 causal attention of sequence s, KV head h, with the blocks `missing` not seen: (out, tolerance), the
    tolerance by the same account as kv_reference.attend."""
    val, exps = c.values()
    n, L = c.seqs[s]
    t0, g, bt = c.indptr[s], c.hq // c.hkv, c.bt
    nb = -(-L // bt)
    ok = np.repeat([b not in missing for b in range(nb)], bt)[:L]
    rows = []
    for w in (0, 1):
        rows.append(np.concatenate([np.zeros((bt, c.d)) if b in missing else
                                    val[c.table[s, b, h, w]] * 2.0 ** float(exps[c.table[s, b, h, w]])
                                    for b in range(nb)])[:L])
    see = (np.arange(L)[None] <= (L - n + np.arange(n))[:, None]) & ok[None]
    out, tol = np.zeros((n, g, c.d)), np.zeros((n, g, c.d))
    for j in range(g):
        q = c.q[t0:t0 + n, h * g + j].astype(np.float64)
        z = np.where(see, q @ rows[0].T * scale, -np.inf)
        m = z.max(1)
        p = np.exp(z - np.where(np.isinf(m), 0.0, m)[:, None])
        w = p / np.maximum(p.sum(1), 1e-300)[:, None]
        out[:, j] = w @ rows[1]
        ds = np.where(see, np.abs(q) @ np.abs(rows[0]).T, 0).max(1) * scale * (c.d + 8) * 2.0 ** -24 + 2.0 ** -21 + L * 2.0 ** -24
        tol[:, j] = (2.0 ** -11 * 1.01 + 2 * ds[:, None]) * (w @ np.abs(rows[1])) + 2.0 ** -11 * np.abs(out[:, j]) + 2.0 ** -24
    return out, tol


# new tokens of each sequence: of single tokens the streaming kernel's, else the prompt kernel's (its rows per KV
# head are new tokens x 4), in one call or beside each other
PROMPTS = [(70, 200), (40, 40), (130, 333)]
STREAM = [(1, 200), (2, 40), (4, 333)]
MIXED = [(130, 333)] + [(1, 90)] * 200


@pytest.mark.parametrize("seqs", [PROMPTS, STREAM, MIXED], ids=["prompts", "stream", "mixed"])
@pytest.mark.parametrize("d,hidden", [(128, 4096), (64, 256)])
@pytest.mark.parametrize("block", [0, 1])
@pytest.mark.parametrize("which", [0, 1])
def test_bad_pages_are_not_seen(seqs, d, hidden, block, which):
    """A page id below 0, the first past the pool and one far past it, of keys and of values, in the first block of
    a call's first tile and in a later one."""
    c = Case(seqs, hq=8, hkv=2, d=d, hidden=hidden, seed=40)
    scale = 0.5 / np.sqrt(d)
    want, wl = c.attend()
    num = len(c.pages)
    for s, h in ((0, 0), (len(seqs) - 1, 1)):
        if block >= -(-seqs[s][1] // c.bt):
            continue
        keep = c.table[s, block, h, which]
        good, tol = masked_attend(c, s, h, {block}, scale)
        for page in (-1, -(1 << 31), num, (1 << 31) - 1):
            c.table[s, block, h, which] = page
            c.d_table = dev(c.table)
            out, lse = c.attend()
            assert c.s.device_status() == BAD_PAGE
            mine = np.zeros(out.shape[:2], bool)
            mine[c.indptr[s]:c.indptr[s + 1], 4 * h:4 * h + 4] = True
            assert np.array_equal(out[~mine], want[~mine]) and np.array_equal(lse[~mine], wl[~mine])
            got = out[c.indptr[s]:c.indptr[s + 1], 4 * h:4 * h + 4]
            assert (np.abs(got - good) <= tol).all()
        c.table[s, block, h, which] = keep
    c.d_table = dev(c.table)
    out, lse = c.attend()
    assert np.array_equal(out, want) and np.array_equal(lse, wl) and c.s.device_status() == 0


@pytest.mark.parametrize("seqs", [PROMPTS, STREAM], ids=["prompts", "stream"])
def test_every_page_bad(seqs):
    c = Case(seqs, hq=8, hkv=2, seed=41)
    c.table[:] = -1
    c.d_table = dev(c.table)
    out, lse = c.attend()
    assert c.s.device_status() == BAD_PAGE
    assert (out == 0).all() and (lse == -np.inf).all()


def test_bad_lengths_and_offsets_of_prompts():
    """The prompt kernel skips the sequence and reports it; the others keep their results."""
    c = Case(PROMPTS, hq=8, hkv=2, seed=42)
    want, _ = c.attend()
    t0, t1 = c.indptr[1], c.indptr[2]
    rest = np.r_[0:t0, t1:c.T]
    for length in (-1, c.max_blocks * c.bt + 1, (1 << 30) + 1, -(1 << 31)):
        keep = c.kv_len[1]
        c.kv_len[1] = length
        c.d_len = dev(c.kv_len)
        out, _ = c.attend()
        assert c.s.device_status() == BAD_LENGTH
        assert np.array_equal(out[rest], want[rest]) and (out[t0:t1] == 7).all()
        c.kv_len[1] = keep
    c.d_len = dev(c.kv_len)
    for indptr, kept in (([0, 70, c.T + 1, c.T + 1], np.r_[0:70]), ([0, 70, 60, 60], np.r_[0:70]), ([-1, 70, 70, 70], np.r_[0:0])):
        c.d_indptr = dev(np.array(indptr, np.int32))
        out, _ = c.attend()
        assert c.s.device_status() == BAD_SEGMENT
        other = np.setdiff1d(np.arange(c.T), kept)
        assert np.array_equal(out[kept], want[kept]) and (out[other] == 7).all()
    c.d_indptr = dev(c.indptr)
    out, _ = c.attend(max_q=70)                     # a sequence with more new tokens than max_q
    assert c.s.device_status() == BAD_SEGMENT
    assert np.array_equal(out[:110], want[:110]) and (out[110:] == 7).all()


def append_ones(c, batch=None):
    k = torch.ones((c.T, c.hkv * c.d), dtype=torch.float16, device="cuda")
    rdp.slora_kv_append(c.s.kv, batch or c.batch(), k, c.hkv * c.d, k, c.hkv * c.d)
    status = c.s.device_status()
    return status, c.s.pages.cpu().numpy(), c.s.exponents.cpu().numpy()


@pytest.mark.parametrize("seqs", [[(1, 70), (1, 40), (1, 130)], [(9, 70), (30, 40), (130, 200)]], ids=["single", "several"])
def test_append_skips_bad_pages(seqs):
    """The page is not written, every other page is written as without the bad entry."""
    c = Case(seqs, hq=4, hkv=2, seed=43)
    _, want, we = append_ones(c)
    for s, h, which in ((0, 0, 0), (1, 1, 1), (2, 0, 1)):
        blk = (seqs[s][1] - 1) // c.bt
        page = c.table[s, blk, h, which]
        for bad in (-1, -(1 << 31), len(c.pages), (1 << 31) - 1):
            c.push()
            t = c.table.copy()
            t[s, blk, h, which] = bad
            c.d_table = dev(t)
            status, got, ge = append_ones(c)
            assert status == BAD_PAGE
            others = np.arange(len(got)) != page
            assert np.array_equal(got[others], want[others]) and np.array_equal(ge[others], we[others])
            assert np.array_equal(got[page], c.pages[page]) and ge[page] == c.exps[page]


@pytest.mark.parametrize("seqs", [[(1, 70), (1, 40), (1, 130)], [(9, 70), (30, 40), (130, 200)]], ids=["single", "several"])
def test_append_leaves_skipped_sequences_alone(seqs):
    """A sequence with an unusable length or offsets: none of its pages and exponents change."""
    c = Case(seqs, hq=4, hkv=2, seed=44)
    _, want, we = append_ones(c)
    mine = np.zeros(len(c.pages), bool)
    mine[c.table[1][c.table[1] >= 0]] = True
    for length in (-1, seqs[1][0] - 1, c.max_blocks * c.bt + 1, (1 << 30) + 1):
        c.push()
        lens = c.kv_len.copy()
        lens[1] = length
        c.d_len = dev(lens)
        status, got, ge = append_ones(c)
        assert status == BAD_LENGTH
        assert np.array_equal(got[mine], c.pages[mine]) and np.array_equal(ge[mine], c.exps[mine])
        assert np.array_equal(got[~mine], want[~mine]) and np.array_equal(ge[~mine], we[~mine])
    c.push()
    c.d_indptr = dev(np.array([0, seqs[0][0], c.T + 1, c.T + 1], np.int32))
    status, got, ge = append_ones(c)
    assert status == BAD_SEGMENT
    first = np.zeros(len(c.pages), bool)
    first[c.table[0][c.table[0] >= 0]] = True
    assert np.array_equal(got[first], want[first]) and np.array_equal(got[~first], c.pages[~first])
    assert np.array_equal(ge[~first], c.exps[~first])


@pytest.fixture
def give_up():
    yield rdp.slora_debug_kv_give_up
    rdp.slora_debug_kv_give_up(-1)


WHOLE = {"stream": ([(1, 60)] * 40, 8, 2), "stream16": ([(3, 60)] * 40, 8, 2), "prompts": ([(60, 60)] * 30, 8, 2)}


@pytest.mark.parametrize("kind", WHOLE)
@pytest.mark.parametrize("hidden,d", [(4096, 128), (256, 64)])
def test_a_cta_that_gives_up_ends_and_reports_it(give_up, kind, hidden, d):
    """Units of one tile, a CTA each: the one that gives up (with its first copies under way) leaves its rows, the
    others and the calls after it are as ever."""
    seqs, hq, hkv = WHOLE[kind]
    c = Case(seqs, hq=hq, hkv=hkv, d=d, hidden=hidden, seed=45)
    want, wl = c.attend()
    for cta in (0, 7, 33):
        give_up(cta)
        out, _ = c.attend()
        assert c.s.device_status() == TIMEOUT
        # a CTA's run holds one unit here: one sequence and KV head
        s, h = divmod(cta, hkv)
        mine = np.zeros(out.shape[:2], bool)
        mine[c.indptr[s]:c.indptr[s + 1], h * 4:h * 4 + 4] = True
        assert np.array_equal(out[~mine], want[~mine])
        give_up(-1)
        out, lse = c.attend()
        assert c.s.device_status() == 0
        assert np.array_equal(out, want) and np.array_equal(lse, wl)
    give_up(1 << 20)                                    # no such CTA
    out, _ = c.attend()
    assert np.array_equal(out, want) and c.s.device_status() == 0
    with pytest.raises(rdp.SloraError):
        give_up(-2)


SPLIT = {"stream": [(1, 100011), (1, 3), (1, 40001)], "stream16": [(3, 100011), (2, 60345)], "prompts": [(140, 9001), (1, 3), (200, 6000)]}


@pytest.mark.parametrize("kind", SPLIT)
@pytest.mark.parametrize("graph", [False, True])
def test_calls_after_a_cta_gave_up_join_their_parts_as_ever(give_up, kind, graph):
    """Units cut between many CTAs.  One that gives up never arrives at its unit's join; what it leaves there does not
    reach a later call, eager or replayed from a graph, with other queries or lengths and so another split."""
    c = Case(SPLIT[kind], hq=4, hkv=1, seed=46)
    row = c.hq * c.d
    longer = c.batch()                                    # what gives up: the full lengths
    c.kv_len = np.array([n if n < 1000 else n * 5 // 8 for n in c.kv_len], np.int32)
    c.d_len = dev(c.kv_len)
    qs, wants = [], []
    for _ in range(4):
        c.q = c.rng.normal(0, 1, c.q.shape).astype(np.float16)
        qs.append(half(c.q).view(-1, row))
        wants.append(c.attend())
    q, b = torch.zeros_like(qs[0]), c.batch()
    out, lse = torch.zeros((c.T, row), dtype=torch.float16, device="cuda"), torch.zeros((c.T, c.hq), device="cuda")
    st = torch.cuda.Stream()

    def calls(batch):
        """What runs one call: the call itself, or a graph of it."""
        run = lambda: rdp.slora_kv_attend(c.s.kv, batch, q, row, c.hq, out, row, lse, 0.5 / np.sqrt(c.d), True, 0, st)  # noqa: E731
        if not graph:
            return run
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            run()
        return g.replay

    good, n = calls(b), 0
    for cta in (0, 1, 50, 149, 303):
        for batch in (longer, b):
            give_up(cta)
            calls(batch)()
            torch.cuda.synchronize()
            give_up(-1)
            c.s.device_status()                           # TIMEOUT where a grid has this CTA
            for _ in range(4):
                n += 1
                q.copy_(qs[n % 4])
                out.fill_(7)
                torch.cuda.synchronize()
                good()
                torch.cuda.synchronize()
                assert np.array_equal(out.float().cpu().numpy().reshape(c.q.shape), wants[n % 4][0])
                assert np.array_equal(lse.cpu().numpy(), wants[n % 4][1])
            assert c.s.device_status() == 0


def test_a_batch_without_tokens_or_sequences_needs_no_rows():
    """An empty tensor has no address; the scalar arguments are still checked."""
    c = Case([(1, 10), (2, 20)], hq=4, hkv=2, seed=48)
    z = lambda *shape: torch.empty(shape, dtype=torch.float16, device="cuda")  # noqa: E731
    zi = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, tab = z(0, 512), z(0, 256), torch.zeros((32, 64), device="cuda")
    assert q.data_ptr() == 0
    before = c.s.pages.clone()
    for b in (rdp.KVBatch(0, 0, 1, 1, zi(0), zi(0), zi(0, 1, 2, 2)), rdp.KVBatch(0, 2, 3, c.max_blocks, c.d_indptr, c.d_len, c.d_table),
              rdp.KVBatch(3, 0, 1, 1, None, None, None)):
        for lse in (None, torch.empty((0, 4), device="cuda")):
            rdp.slora_kv_attend(c.s.kv, b, q, 512, 4, q, 512, lse)
        rdp.slora_kv_append(c.s.kv, b, k, 256, k, 256)
        for q_out in (q, z(4, 512)):
            for pos in (None, zi(0)):
                rdp.slora_kv_append(c.s.kv, b, k, 256, k, 256, q, 512, q_out, 512, 4, rdp.KVRope(128, 0, 32, tab, tab, pos))
        for bad in (dict(hq=3), dict(qs=504), dict(os=516), dict(window=-1)):
            a = dict(hq=4, qs=512, os=512, window=0)
            a.update(bad)
            with pytest.raises(rdp.SloraError) as e:
                rdp.slora_kv_attend(c.s.kv, b, q, a["qs"], a["hq"], q, a["os"], window=a["window"])
            assert e.value.status == 1
        with pytest.raises(rdp.SloraError) as e:
            rdp.slora_kv_append(c.s.kv, b, k, 248, k, 256)
        assert e.value.status == 1
    assert torch.equal(before, c.s.pages) and c.s.device_status() == 0


def rotate_with_padding(seqs, pad, in_place, given, bad=None, max_q=None):
    """Appends with `pad` spare rows before and behind the sequences' rows; returns the case, q, q_out, the rows that
    the sequences have, and the status."""
    c = Case(seqs, hq=6, hkv=2, seed=49)
    T = c.T + 2 * pad
    rng = np.random.default_rng(5)
    q = rng.normal(0, 1, (T, 6 * 128)).astype(np.float16)
    k = torch.from_numpy(rng.normal(0, 1, (T, 256)).astype(np.float16)).cuda()
    n_pos = int(c.kv_len.max()) + 1
    angle = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, 128, 2) / 128)
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    pos = np.full(T, -1, np.int32)
    rows = pad + np.arange(c.T)
    pos[rows] = np.concatenate([np.arange(n - m, n) for m, n in seqs])
    if bad is not None:                                  # a skipped sequence: its positions are nobody's
        mine = rows[c.indptr[bad]:c.indptr[bad + 1]]
        c.kv_len[bad] = c.max_blocks * c.bt + 1
        c.d_len = dev(c.kv_len)
        pos[mine] = 1 << 30
        rows = np.setdiff1d(rows, mine)
    dq = torch.from_numpy(q).cuda()
    out = dq if in_place else torch.full_like(dq, 7.0)
    kept = out.cpu().numpy().copy()
    b = rdp.KVBatch(T, len(seqs), max_q or max(m for m, _ in seqs), c.max_blocks, dev(c.indptr + pad), c.d_len, c.d_table)
    rope = rdp.KVRope(128, False, n_pos, dev(cos), dev(sin), dev(pos) if given else None)
    rdp.slora_kv_append(c.s.kv, b, k, 256, k, 256, dq, 768, out, 768, 6, rope)
    status = c.s.device_status()
    got = out.cpu().numpy()
    want = R.rotate(q.reshape(T, 6, 128)[rows], cos[pos[rows]], sin[pos[rows]], False, np.float32).astype(np.float16)
    assert np.array_equal(got[rows].reshape(want.shape).view(np.uint16), want.view(np.uint16))
    other = np.setdiff1d(np.arange(T), rows)
    assert np.array_equal(got[other].view(np.uint16), kept[other].view(np.uint16))
    return status


SINGLE, SEVERAL = [(1, 30), (0, 9), (1, 65), (1, 1)], [(5, 30), (0, 9), (1, 65), (70, 70), (0, 0)]


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seqs", [SINGLE, SEVERAL, SEVERAL * 90], ids=["single", "several", "many"])
def test_rows_outside_every_sequence_are_left_alone(seqs, in_place, given):
    """A padded batch: spare rows before and behind the sequences, whose positions are -1."""
    assert rotate_with_padding(seqs, 11, in_place, given) == 0
    assert rotate_with_padding(seqs, 0, in_place, given) == 0
    assert rotate_with_padding(seqs, 3, in_place, given, max_q=1 << 20) == 0


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("seqs", [SINGLE, SEVERAL], ids=["single", "several"])
def test_rows_of_a_skipped_sequence_are_left_alone(seqs, given):
    assert rotate_with_padding(seqs, 2, False, given, bad=0) == BAD_LENGTH
    assert rotate_with_padding(seqs, 2, True, given, bad=3) == BAD_LENGTH


def dominated(n, length, at, below, fmt, page_exponent, hkv, group):
    """A cache whose key at position `at` outweighs every other by 2^(below - 1) to 2^below and has the value 0, so that the
    outputs are made of the others alone; its value page's scale is 2^page_exponent of the others'."""
    c = Case([(n, length)], hq=hkv * group, hkv=hkv, fmt=fmt, seed=51)
    sixteen = {"e4m3": 0x58, "int8": 16}[fmt]
    small = np.array([0, 8, 12, 16])                       # 0 to 1 in units of 2^-4
    codes = np.array([0, 0x50, 0x54, 0x58] if fmt == "e4m3" else small, np.uint8)
    c.q[:] = 0
    c.q[:, :, 0], c.q[:, :, 1] = 1, below
    for b in range(-(-length // c.bt)):
        for h in range(hkv):
            kp, vp = c.table[0, b, h]
            k, v = (c.pages[p, :c.bt * c.d].reshape(c.bt, c.d) for p in (kp, vp))
            k[:] = 0
            k[:, 0] = codes[c.rng.integers(0, 4, c.bt)]
            c.exps[kp], c.exps[vp] = -4, 0
            if b == at // c.bt:
                k[at % c.bt, :2] = 0, sixteen
                c.exps[vp] = page_exponent
                v[:] = 0
                if at == 0:                                # one for each warp of the streaming kernel
                    k[16:64:16] = k[0]
            else:                                          # of one sign, so that errors add up
                v[:] = v & 0x7F if fmt == "e4m3" else np.abs(v.view(np.int8)).view(np.uint8)
                v[v == 0x7F] = 0x7E
    c.push()
    return c


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n,group", [(1, 1), (3, 4), (140, 2)])
@pytest.mark.parametrize("at", [0, 700, 1300])
@pytest.mark.parametrize("below,page_exponent", [(4, 0), (11.3, 0), (15.3, 0), (20.3, 0), (9.3, 11), (20.3, -9)])
def test_attend_keys_beside_one_that_outweighs_them(fmt, n, group, at, below, page_exponent):
    """The rest of the softmax keeps its bits: each key's weight is within fp16's rounding of its value, although it is
    2^-20 of the largest."""
    dominated(n, 1500, at, below, fmt, page_exponent, 2, group).check(scale=float(np.log(2)))


@pytest.mark.parametrize("n,group", [(1, 1), (3, 4), (140, 2)])
@pytest.mark.parametrize("power", range(8, 16))
def test_attend_scores_whose_steps_are_the_rescaling_s(n, group, power):
    """Scores of 2^(power + 15) and their neighbours in fp32, 2^(power - 8) apart, each block one step above the last:
    no weight passes fp16's range whatever the rounding of the sums that decide about it."""
    c = Case([(n, 900)], hq=2 * group, hkv=2, seed=52, stale=False)
    c.q[:] = 0
    c.q[:, :, 0], c.q[:, :, 1] = 2.0 ** 15, 2.0 ** -8
    steps = torch.arange(1, 17).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    for b in range(-(-900 // c.bt)):
        for h in range(2):
            kp, vp = c.table[0, b, h]
            k, v = (c.pages[p, :c.bt * c.d].reshape(c.bt, c.d) for p in (kp, vp))
            k[:] = 0
            k[:, 0], k[:, 1] = 0x38, steps[b]                      # 1, and the step
            v[:] = 0x7E                                            # 448
            c.exps[kp] = c.exps[vp] = 0
    c.push()
    out, lse = c.attend(scale=float(2.0 ** power * np.log(2)))
    assert c.s.device_status() == 0
    assert np.abs(out - 448).max() <= 0.5 and np.isfinite(lse).all()


@pytest.mark.parametrize("seqs", [[(1, 70), (0, 40), (1, 9), (0, 5)], [(0, 9), (9, 70), (0, 40), (130, 200), (1, 7), (0, 0)]],
                         ids=["single", "several"])
def test_sequences_without_new_tokens_may_hold_anything(seqs):
    """Spare places of a padded batch: their lengths and pages are not looked at."""
    c = Case(seqs, hq=8, hkv=2, seed=53)
    want, wl = c.attend()
    _, pages, exps = append_ones(c)
    spare = [s for s, (n, _) in enumerate(seqs) if n == 0]
    for length in (-1, -(1 << 31), (1 << 31) - 1, c.max_blocks * c.bt + 1):
        c.kv_len[spare] = length
        c.table[spare] = 1 << 30
        c.push()
        out, lse = c.attend()
        assert c.s.device_status() == 0
        assert np.array_equal(out, want) and np.array_equal(lse, wl)
        status, got, ge = append_ones(c)
        assert status == 0 and np.array_equal(got, pages) and np.array_equal(ge, exps)


NAN_CASES = {
    "drafts": ([(4, 70), (1, 33), (7, 150), (3, 3)], 8, 2, 128, 4096),
    "drafts, 64-wide": ([(4, 70), (1, 33), (7, 150), (3, 3)], 4, 4, 64, 256),
    "drafts, 16 rows": ([(4, 200), (5, 64)], 6, 2, 128, 5120),
    "drafts beyond the cache": ([(6, 4), (5, 200)], 4, 2, 128, 4096),
    "prompts": ([(130, 333), (70, 70), (1, 9), (300, 300)], 4, 2, 128, 4096),
    "prompts beyond the cache": ([(150, 90), (70, 70)], 4, 2, 128, 4096),
    "prompts, 64-wide": ([(130, 333), (70, 70)], 3, 1, 64, 640),
    "prompts beside tokens": ([(150, 200)] + [(1, 40)] * 200, 4, 2, 128, 4096),
    "split prompts": ([(280, 9001)], 2, 1, 128, 4096),
}


@pytest.mark.parametrize("kind", NAN_CASES)
@pytest.mark.parametrize("window", [0, 50])
def test_a_nan_value_reaches_the_tokens_that_see_it_only(kind, window):
    """NaN codes among the values, at new tokens, at the window's edge and deep in the cache: the outputs of the tokens
    that see one are NaN in its channel; all else, the log-sum-exp too, is as with 0 in its place."""
    seqs, hq, hkv, d, hidden = NAN_CASES[kind]
    c = Case(seqs, hq=hq, hkv=hkv, d=d, hidden=hidden, seed=54)
    g = hq // hkv
    spots = []
    for s, (n, length) in enumerate(seqs[:4]):
        for p in {length - 1, length - n, length - n + 1, length - 1 - n // 2, max(0, length - n - 49), length // 3, 0}:
            if 0 <= p < length:
                spots.append((s, p, int(c.rng.integers(hkv)), int(c.rng.integers(d)), int(c.rng.choice([0x7F, 0xFF]))))
    codes = c.pages.reshape(len(c.pages), -1)

    def put(nan):
        for s, p, h, ch, code in spots:
            codes[c.table[s, p // c.bt, h, 1], (p % c.bt) * d + ch] = code if nan else 0
        c.push()

    put(False)
    clean, cl = c.attend(window=window)
    put(True)
    out, lse = c.attend(window=window)
    assert c.s.device_status() == 0
    want = clean.copy()
    for s, p, h, ch, _ in spots:
        n, length = seqs[s]
        pos = length - n + np.arange(n)
        see = (p <= pos) & ((p > pos - window) if window else True)
        want[c.indptr[s] + np.nonzero(see)[0], h * g:(h + 1) * g, ch] = np.nan
    assert np.isnan(want).any() and not np.isnan(want).all()
    assert np.array_equal(np.isnan(out), np.isnan(want)) and np.array_equal(lse, cl)
    # the prompt kernel sums such a channel of a token that sees no NaN once more, by fp32 weights: within the
    # tolerance of the definition; every other channel bit for bit
    val, exps = c.values()
    ref, _, tol, _ = R.attend(np.nan_to_num(val), exps, c.table, c.indptr, c.kv_len, c.q, c.bt, 0.5 / np.sqrt(d), True, window)
    touched = np.zeros(out.shape, bool)
    for s, p, h, ch, _ in spots:
        touched[c.indptr[s]:c.indptr[s + 1], h * g:(h + 1) * g, ch] = True
    ok = ~np.isnan(want)
    assert np.array_equal(out[ok & ~touched], want[ok & ~touched])
    assert (np.abs(out - ref) <= tol)[ok].all()
    a, la = c.attend(causal=False)                        # every token sees every key
    for s, p, h, ch, _ in spots:
        n, length = seqs[s]
        assert np.isnan(a[c.indptr[s]:c.indptr[s + 1], h * g:(h + 1) * g, ch]).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("seqs", [[(1, 100), (3, 70)], [(70, 130), (40, 40)]], ids=["stream", "prompts"])
def test_exponents_beyond_sixty_are_read_as_sixty(seqs, fmt):
    """As the header says, by attend and, for the rows that a block holds, by append."""
    c = Case(seqs, hq=8, hkv=2, fmt=fmt, seed=55, stale=False)
    for sign in (1, -1):
        got = []
        for e in (60, 61, 100, 127):
            c.exps[:] = sign * e
            c.exps[::3] = sign * 60
            c.push()
            out, lse = c.attend(scale=2.0 ** (-58 * sign))
            assert np.isfinite(lse).all()
            got.append((out, lse) + append_ones(c))
        for g in got[1:]:
            assert np.array_equal(g[0], got[0][0], equal_nan=True) and np.array_equal(g[1], got[0][1])
            touched = np.unique(np.concatenate([c.table[s, (n - m) // c.bt:-(-n // c.bt)].ravel() for s, (m, n) in enumerate(seqs)]))
            assert g[2] == got[0][2] == 0 and np.array_equal(g[3], got[0][3]) and np.array_equal(g[4][touched], got[0][4][touched])


def test_misaligned_arrays_of_integers_are_refused():
    c = Case([(1, 10), (2, 20)], hq=4, hkv=2, seed=56)
    q, k = torch.zeros((c.T, 512), dtype=torch.float16, device="cuda"), torch.zeros((c.T, 256), dtype=torch.float16, device="cuda")
    out, tab = torch.zeros_like(q), torch.zeros((32, 64), device="cuda")

    def attend(b):
        rdp.slora_kv_attend(c.s.kv, b, q, 512, 4, out, 512)

    def append(b, pos=None):
        rdp.slora_kv_append(c.s.kv, b, k, 256, k, 256, rope=rdp.KVRope(128, False, 32, tab, tab, pos))

    def refused(fn, *args):
        with pytest.raises(rdp.SloraError) as e:
            fn(*args)
        assert e.value.status == 1

    for field in ("tok_indptr", "kv_len", "block_table"):
        for off in (1, 2, 3):
            b = c.batch()
            setattr(b, field, getattr(b, field) + off)
            refused(attend, b)
            refused(append, b)
    for off in (1, 2, 3):
        refused(append, c.batch(), torch.zeros(8, dtype=torch.int32, device="cuda").data_ptr() + off)
    assert (out == 0).all() and c.s.device_status() == 0


@pytest.mark.parametrize("seqs,hq,hkv,d", [([(280, 30001), (40, 40)], 2, 1, 128), ([(100, 5000), (90, 90), (200, 333)], 8, 2, 64)])
@pytest.mark.parametrize("window", [0, 300])
def test_whole_rows_of_nan_values(seqs, hq, hkv, d, window):
    """Tokens whose values are all NaN, as a bad one leaves them: new ones and cached ones, over long contexts."""
    c = Case(seqs, hq=hq, hkv=hkv, d=d, seed=57)
    rows = []
    for s, (n, length) in enumerate(seqs):
        rows += [(s, length - 3), (s, length - n // 2)]
        if window or s == len(seqs) - 1:
            rows += [(s, 5), (s, max(0, length - n - 290))]
    for value in (0, 0x7F):
        for s, p in rows:
            for h in range(hkv):
                at = p % c.bt * d
                c.pages[c.table[s, p // c.bt, h, 1], at:at + d] = value
        c.push()
        if value == 0:
            clean, cl = c.attend(window=window)
    out, lse = c.attend(window=window)
    assert c.s.device_status() == 0 and np.array_equal(lse, cl)
    val, exps = c.values()
    ref, _, tol, _ = R.attend(np.nan_to_num(val), exps, c.table, c.indptr, c.kv_len, c.q, c.bt, 0.5 / np.sqrt(d), True, window)
    hit = np.zeros(c.T, bool)
    for s, p in rows:
        n, length = seqs[s]
        pos = length - n + np.arange(n)
        hit[c.indptr[s]:c.indptr[s + 1]] |= (p <= pos) & ((p > pos - window) if window else True)
    assert np.isnan(out[hit]).all() and np.isfinite(out[~hit]).all() and (~hit).sum() > 30
    assert (np.abs(out - ref) <= tol)[~hit].all()
