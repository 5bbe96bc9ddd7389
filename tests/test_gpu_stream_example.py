"""The streaming example: it runs, its pages come back, a stream's pages stay bounded, and a fork and an untouched copy
of it continue alike."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import rank_delta_paged_gb300 as rdp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "stream.py")
    spec = importlib.util.spec_from_file_location("stream_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs(example):
    assert example.main() == 0


def tokens(e, n, seed):
    return torch.from_numpy(np.random.default_rng(seed).normal(0, 1, (n, e.hidden)).astype(np.float16)).cuda()


def test_a_stream_holds_a_bounded_number_of_pages(example):
    e = example.Streams(window=40, sinks=3, num_pages=512)
    try:
        s = example.Stream()
        held = set()
        for i in range(300):
            e.step([(s, tokens(e, 1, i))])
            e.trim(s)
            if i > 100:
                held.add(len(s.blocks))
        # the sinks' block, and those that 40 tokens touch
        assert max(held) <= 2 + -(-40 // e.block) and s.length == 300
        e.drop(s)
        assert rdp.slora_pool_num_free(e.pool) == 512 and rdp.slora_get_device_status(e.pool) == 0
    finally:
        e.close()


def test_a_fork_continues_as_its_parent_would(example):
    e = example.Streams(window=60, sinks=5)
    try:
        for length in (30, e.block, 3 * e.block, 101):
            s = example.Stream()
            e.step([(s, tokens(e, length, length))])
            e.trim(s)
            f = e.fork(s)
            assert f.blocks.keys() == {b for b in s.blocks if b * e.block < length}
            outs = [[e.step([(x, tokens(e, m, 7 + m))])[0] for m in (1, 5, 40)] for x in (s, f)]
            assert all(torch.equal(a, b) for a, b in zip(*outs))
            # other tokens in one do not reach the other
            e.step([(s, tokens(e, 3, 1))])
            a = e.step([(f, tokens(e, 1, 2))])[0]
            g = example.Stream()
            e.step([(g, tokens(e, length, length))])
            e.trim(g)
            for m in (1, 5, 40):
                e.step([(g, tokens(e, m, 7 + m))])
            assert torch.equal(a, e.step([(g, tokens(e, 1, 2))])[0])
            for x in (s, f, g):
                e.drop(x)
        assert rdp.slora_get_device_status(e.pool) == 0
    finally:
        e.close()


def test_rejected_drafts_leave_no_pages(example):
    e = example.Streams(window=60, sinks=5)
    try:
        s = example.Stream()
        e.step([(s, tokens(e, 60, 0))])
        free = rdp.slora_pool_num_free(e.pool)
        for kept in ([], [0], [1, 3], list(range(9))):
            before = s.length
            e.step([(s, tokens(e, 9, 5))])
            e.accept(s, 9, kept)
            assert s.length == before + len(kept)
            assert set(s.blocks) == set(range((s.length - 1) // e.block + 1))
        assert rdp.slora_pool_num_free(e.pool) <= free and rdp.slora_get_device_status(e.pool) == 0
        e.drop(s)
    finally:
        e.close()
