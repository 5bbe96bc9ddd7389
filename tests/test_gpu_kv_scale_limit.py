"""GPU checks of the KV cache at its largest scale, 2^60: no INT8 code leaves -127 .. 127, and what is moved there reads as
it did."""
import numpy as np
import pytest
import torch

import kv_reference as R
import rank_delta_paged_gb300 as rdp
from test_gpu_kv import Case, half
from test_gpu_kv_compact import Moves

pytestmark = pytest.mark.gpu
TOP = 60


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,hidden", [(128, 4096), (64, 4096), (64, 8192)])
@pytest.mark.parametrize("seqs", [[(1, 70)] * 3, [(5, 75), (1, 9)], [(70, 70)], [(100, 200)]])
def test_normed_keys_next_to_the_largest_code(fmt, d, hidden, seqs):
    """Rows of ones and minus ones, whose norm they are themselves, times weights of 100 to 520 times 2^60: with eps 0 the
    mean square is 1, and the reciprocal root is good to 2^-22, which no weight here is near enough to a border between two
    codes to show."""
    c = Case(seqs, hq=2, hkv=2, d=d, hidden=hidden, fmt=fmt, seed=90)
    rng = np.random.default_rng(0)
    k = rng.choice([-1.0, 1.0], (c.T, 2, d)).astype(np.float16)
    units = np.linspace(100, 160, d) if fmt == "int8" else np.linspace(381, 519, d)
    units[:8] = [126.4, 126.6, 127.4, 127.51, 127.6, 128.25, 128.49, 128.6] if fmt == "int8" else [431, 433, 447, 449, 463, 465, 479, 481]
    units = units.astype(np.float32)
    step = 1 if fmt == "int8" else 32
    assert np.abs((units / step - 0.5) - np.rint(units / step - 0.5)).min() > 1e-3      # of a step between codes
    norm = rdp.KVNorm(0.0, False, None, 0, torch.from_numpy(units).cuda() * 2.0 ** TOP, 0)
    dk = half(k).view(c.T, -1)
    rdp.slora_kv_append_norm(c.s.kv, c.batch(), dk, 2 * d, dk, 2 * d, norm=norm)
    got, exps = c.values()
    assert c.s.device_status() == 0
    want = R.nearest(k.astype(np.float64) * units.astype(np.float64), fmt)
    for s, (n, length) in enumerate(c.seqs):
        for i in range(n):
            p = length - n + i
            for h in range(2):
                page = c.table[s, p // c.bt, h, 0]
                assert exps[page] == TOP
                assert np.array_equal(got[page, p % c.bt], want[c.indptr[s] + i, h])


@pytest.mark.parametrize("in_place", [False, True])
def test_compaction_at_the_largest_scale(in_place):
    """A code of -128, which only a caller can have written, at the largest exponent that is read: there is no scale above to
    move it to, so it reads as it did, and so do the rows beside it."""
    m = Moves([200, 70], [0, 3], [150, 60], fmt="int8", seed=91, in_place=in_place, edit=lowest_codes)
    before, exps = m.c.values()
    was = [[kept_values(m, before, exps, m.table, s, h, w, m.kept[0, m.indptr[s]:m.indptr[s + 1]]) for h in range(2) for w in range(2)]
           for s in range(2)]
    m.run()
    after, exps = m.c.values()
    assert m.c.s.device_status() == 0 and exps.max() <= TOP
    to = m.table if m.dst is None else m.dst
    now = [[kept_values(m, after, exps, to, s, h, w, m.first[s] + np.arange(m.n[s])) for h in range(2) for w in range(2)]
           for s in range(2)]
    for a, b in zip(was, now):
        for x, y in zip(a, b):
            assert np.array_equal(x, y)


def lowest_codes(c):
    """Every page at 2^60 with a -128 in its fifth row."""
    c.exps[:] = TOP
    c.pages[:, 4 * c.d + 7] = 0x80


def kept_values(m, val, exps, table, s, h, w, at):
    page = table[s, at // m.bt, h, w]
    return val[page, at % m.bt] * 2.0 ** np.clip(exps[page].astype(float), -60, 60)[:, None]
