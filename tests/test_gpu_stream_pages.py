"""The streaming example's pages to the last one: drafts, forks and a full pool leave no page held by nobody and none held
twice; positions end with the rotation's table; a fork settles drafts, and drafts are accepted as a prefix."""
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
    spec = importlib.util.spec_from_file_location("stream_pages_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def tokens(e, n, seed):
    return torch.from_numpy(np.random.default_rng(seed).normal(0, 1, (n, e.hidden)).astype(np.float16)).cuda()


def free(e):
    return rdp.slora_pool_num_free(e.pool)


def per_block(e):
    return e.n_layers * e.n_heads * 2


def test_drafts_hold_the_pages_of_their_blocks(example):
    e = example.Streams(window=60, sinks=5, num_pages=512)
    try:
        s = example.Stream()
        e.step([(s, tokens(e, e.block - 4, 0))])
        for kept in ([], [0], [0, 1], [1, 3], list(range(9)), []):
            e.step([(s, tokens(e, 9, 5))])
            e.accept(s, 9, kept)
            assert set(s.blocks) == set(range((s.length - 1) // e.block + 1))
            assert free(e) == 512 - len(s.blocks) * per_block(e)
        e.drop(s)
        assert free(e) == 512 and rdp.slora_get_device_status(e.pool) == 0
    finally:
        e.close()


def test_forks_share_and_return_their_pages(example):
    e = example.Streams(window=1000, sinks=5, num_pages=1024)
    try:
        for length in (30, e.block, 3 * e.block, 2 * e.block + 37):
            s = example.Stream()
            e.step([(s, tokens(e, length, length))])
            held = len(s.blocks)
            forks = [e.fork(s)]
            forks.append(e.fork(forks[0]))
            # whole blocks are shared, the last one is copied for each
            copies = 2 if length % e.block else 0
            assert free(e) == 1024 - (held + copies) * per_block(e)
            e.drop(s)
            assert free(e) == 1024 - (length // e.block + copies) * per_block(e)
            outs = [e.step([(f, tokens(e, 2, 3))])[0] for f in forks]
            assert torch.equal(*outs)
            for f in forks:
                e.drop(f)
            assert free(e) == 1024
        assert rdp.slora_get_device_status(e.pool) == 0
    finally:
        e.close()


def test_a_full_pool_leaves_the_streams_as_they_were(example):
    """Pages for two blocks and a half: what cannot be taken raises, and every page held is the stream's own."""
    e = example.Streams(num_pages=1)
    n = per_block(e)
    e.close()
    e = example.Streams(window=1000, num_pages=2 * n + n // 2)
    try:
        s, t = example.Stream(), example.Stream()
        e.step([(s, tokens(e, e.block + 1, 0))])
        pages = {b: p.copy() for b, p in s.blocks.items()}
        for _ in range(2):                               # (again: a retry finds no block that is not there)
            with pytest.raises(rdp.SloraError) as err:
                e.step([(t, tokens(e, 3, 1))])
            assert err.value.status == 2 and t.length == 0 and t.blocks == {} and free(e) == n // 2
            with pytest.raises(rdp.SloraError):
                e.fork(s)                                # a whole block to share, and one to copy
            assert free(e) == n // 2 and s.settled == 0
            with pytest.raises(rdp.SloraError):
                e.step([(s, tokens(e, e.block, 2))])
            assert s.length == e.block + 1 and all(np.array_equal(pages[b], s.blocks[b]) for b in s.blocks) and len(s.blocks) == 2
        e.drop(s)
        assert free(e) == 2 * n + n // 2                 # and no fork holds any
        s = example.Stream()
        e.step([(s, tokens(e, e.block + 1, 0))])         # all of it can be had again
        e.drop(s)
        assert rdp.slora_get_device_status(e.pool) == 0
    finally:
        e.close()


def test_positions_end_with_the_rotation(example):
    e = example.Streams(window=40, sinks=3, num_pages=512, max_positions=70)
    try:
        s = example.Stream()
        e.step([(s, tokens(e, 60, 0))])
        held = free(e)
        with pytest.raises(ValueError):
            e.step([(s, tokens(e, 11, 1))])
        assert s.length == 60 and free(e) == held
        e.step([(s, tokens(e, 10, 1))])
        with pytest.raises(ValueError):
            e.step([(s, tokens(e, 1, 1))])
        assert s.length == 70 and rdp.slora_get_device_status(e.pool) == 0
        e.drop(s)
    finally:
        e.close()


def test_a_fork_settles_what_was_drafted(example):
    """Blocks that a fork shares are not rewritten."""
    e = example.Streams(window=1000, num_pages=512)
    try:
        s = example.Stream()
        e.step([(s, tokens(e, e.block - 4, 0))])
        e.step([(s, tokens(e, 9, 1))])
        f = e.fork(s)
        for x in (s, f):
            with pytest.raises(ValueError):
                e.accept(x, 9, [0])
            assert x.length == e.block + 5
        e.step([(s, tokens(e, 3, 2))])
        e.accept(s, 3, [0])
        assert s.length == e.block + 6
        for x in (s, f):
            e.drop(x)
        assert free(e) == 512
    finally:
        e.close()


def test_the_run_accepts_prefixes(example, monkeypatch):
    """A draft's keys have attended to every draft before it, so with causal drafts only a prefix may stay."""
    some = []
    accept = example.Streams.accept
    monkeypatch.setattr(example.Streams, "accept", lambda e, s, drafts, kept: (some.append(list(kept)), accept(e, s, drafts, kept)))
    assert example.main() == 0
    assert some and all(k == list(range(len(k))) for k in some)
