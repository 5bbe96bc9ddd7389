"""GPU checks of the append's rotations of every part of a row: single tokens, a few and prompts against the definition bit
for bit, and norms that do not depend on which part turns."""
import numpy as np
import pytest
import torch

import rank_delta_paged_gb300 as rdp
from test_gpu_kv import Case, check_append, dev
from test_gpu_kv_norm import Call

pytestmark = pytest.mark.gpu
SINGLE = [(1, 70), (1, 1), (1, 64), (1, 200), (1, 33)]
SEVERAL = [(1, 70), (3, 10), (40, 90), (0, 5), (2, 65), (130, 400)]
PARTS = [(d, rot) for d in (64, 128) for rot in range(16, d + 1, 16)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


@pytest.mark.parametrize("d,rot", PARTS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_every_part_of_a_row(d, rot, interleaved, fmt):
    for seqs in (SINGLE, SEVERAL):
        check_append(Case(seqs, hq=6, hkv=3, d=d, fmt=fmt, seed=110), rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("d,rot", [(64, 48), (128, 80), (128, 96), (128, 112), (128, 48)])
def test_pages_of_more_rows(d, rot):
    """Two rows of a page per lane."""
    check_append(Case(SEVERAL, hq=2, hkv=1, d=d, hidden=8192, fmt="int8", seed=111), rot=rot)


@pytest.mark.parametrize("d,rot", PARTS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("centered", [False, True])
def test_norms_do_not_depend_on_the_part_that_turns(d, rot, interleaved, centered):
    """Turned by angles of 0, rows are as without a rotation: the norm's sums run in the same order."""
    for seqs in (SINGLE, SEVERAL):
        some = []
        for r in (0, rot):
            c = Case(seqs, hq=6, hkv=3, d=d, seed=112)
            x = Call(c, rot=r, interleaved=interleaved, centered=centered, weights="heads")
            if r:
                x.rope = rdp.KVRope(r, interleaved, 400, dev(np.ones((400, r // 2), np.float32)), dev(np.zeros((400, r // 2), np.float32)))
            x.run()
            val, exps = c.values()
            assert c.s.device_status() == 0
            some.append((val, exps, x.q_out.cpu().float().numpy()))
        for a, b in zip(*some):
            assert np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("d,rot", [(64, 48), (128, 16), (128, 96), (128, 112)])
@pytest.mark.parametrize("weights", [None, "shared", "heads"])
def test_norms_and_rotations_of_a_part(d, rot, weights):
    for seqs in (SINGLE, SEVERAL):
        Call(Case(seqs, hq=6, hkv=3, d=d, seed=113), rot=rot, weights=weights, centered=weights is None).check()
