"""GPU checks of what a compaction leaves alone: a page that cannot be used is skipped by itself, keys and values apart, and a
sequence that keeps nothing has nothing written."""
import numpy as np
import pytest
import torch

import rank_delta_paged_gb300 as rdp
from test_gpu_kv_compact import BAD_PAGE, Moves

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("w", [0, 1])
@pytest.mark.parametrize("source", [True, False])
def test_a_bad_page_is_skipped_by_itself(fmt, w, source):
    """Entries out of range among the sources or the destinations: the block's other page, the other blocks and new_len
    are written."""
    spread = lambda where, n: where[np.linspace(0, len(where) - 1, n).astype(int)]     # noqa: E731
    for bad in (-1, 1 << 30, -(1 << 31)):
        m = Moves([400, 300], [10, 0], [150, 140], fmt=fmt, seed=220, in_place=False, pick=spread)
        s, blk, h = 0, 1, 1
        want, we, rows, behind = m.definition()
        before, exps = m.c.values()
        table = (m.table if source else m.dst).copy()
        table[s, blk, h, w] = bad
        kept = m.kept[0, m.indptr[s]:m.indptr[s + 1]]
        skipped = []
        for b in range(m.first[s] // m.bt, -(-(m.first[s] + m.n[s]) // m.bt)):
            src = [t if t < m.first[s] else kept[t - m.first[s]] for t in range(b * m.bt, min(m.first[s] + m.n[s], (b + 1) * m.bt))]
            if (source and blk in {p // m.bt for p in src}) or (not source and b == blk):
                skipped.append(m.dst[s, b, h, w])
        assert 0 < len(skipped) < 3
        for p in skipped:
            want[p], we[p], rows[p], behind[p] = before[p], exps[p], True, False
        m.run(**{"block_table" if source else "dst": table})
        got, ge = m.c.values()
        assert m.c.s.device_status() == BAD_PAGE
        assert np.array_equal(ge, we) and np.array_equal(got[rows], want[rows], equal_nan=True)
        assert np.array_equal(got[~(rows | behind)], before[~(rows | behind)], equal_nan=True)
        assert m.new_len.tolist() == [160, 140]


@pytest.mark.parametrize("in_place", [False, True])
def test_a_sequence_that_keeps_nothing(in_place):
    """Its length becomes first, and the block of first stays where it is."""
    m = Moves([300, 200, 64], [70, 10, 64], [0, 50, 0], seed=221, in_place=in_place)
    before, exps = m.c.values()
    m.check()
    got, ge = m.c.values()
    for s in (0, 2):
        pages = m.table[s][m.table[s] >= 0]
        assert np.array_equal(got[pages], before[pages], equal_nan=True) and np.array_equal(ge[pages], exps[pages])
    assert m.new_len.tolist() == [70, 60, 64]
