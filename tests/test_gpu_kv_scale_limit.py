"""GPU checks of the KV cache at its largest scale, 2^60: no INT8 code leaves -127 .. 127, and what is moved there reads as
it did."""
import numpy as np
import pytest
import torch

import kv_reference as R
import rank_delta_paged_gb300 as rdp
from test_gpu_kv import Case, half

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
