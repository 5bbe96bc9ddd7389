"""GPU checks of copies of KV cache pages: bytes and exponents, partial pages, entries that cannot be used, and forked
sequences that share a prefix."""
import numpy as np
import pytest
import torch

import rank_delta_paged_gb300 as rdp
from rank_delta_paged_gb300.harness import KVSession
from test_gpu_kv import Case, dev

pytestmark = pytest.mark.gpu
BAD_PAGE, BAD_LENGTH = 3, 6


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


def pool(num, hidden, d, seed=0, fmt="e4m3"):
    s = KVSession(hidden, num, 2, d, fmt)
    rng = np.random.default_rng(seed)
    pages = rng.integers(0, 256, (num, hidden * 2), dtype=np.uint8)
    exps = rng.integers(-128, 128, num).astype(np.int8)
    s.pages.copy_(dev(pages))
    s.exponents.copy_(dev(exps))
    torch.cuda.synchronize()
    return s, pages, exps, rng


def expect(s, pages, exps, src, dst, rows, d):
    for i, j, r in zip(src, dst, rows):
        pages[j, :r * d] = pages[i, :r * d]
        if r:
            exps[j] = exps[i]
    torch.cuda.synchronize()
    assert np.array_equal(s.pages.cpu().numpy(), pages) and np.array_equal(s.exponents.cpu().numpy(), exps)


@pytest.mark.parametrize("d,hidden", [(128, 4096), (128, 5120), (64, 4096), (64, 256), (128, 640), (64, 8192), (128, 8192), (64, 320)])
@pytest.mark.parametrize("n", [1, 2, 31, 500, 5000])
def test_copy(d, hidden, n):
    s, pages, exps, rng = pool(2 * n + 1, hidden, d)
    order = rng.permutation(2 * n + 1).astype(np.int32)
    src, dst = order[:n], order[n:2 * n]
    src[n // 2:] = src[rng.integers(0, max(1, n // 2), n - n // 2)]          # sources of several
    rows = rng.integers(0, s.block + 1, n).astype(np.int32)
    rdp.slora_kv_copy(s.kv, n, dev(src), dev(dst), dev(rows))
    expect(s, pages, exps, src, dst, rows, d)
    dst = dst[::-1].copy()
    rdp.slora_kv_copy(s.kv, n, dev(src), dev(dst))
    expect(s, pages, exps, src, dst, np.full(n, s.block), d)
    assert s.device_status() == 0


def test_copy_onto_itself_and_nothing():
    s, pages, exps, _ = pool(8, 4096, 128)
    rdp.slora_kv_copy(s.kv, 3, dev(np.array([1, 2, 3], np.int32)), dev(np.array([1, 7, 3], np.int32)))
    expect(s, pages, exps, [2], [7], [s.block], 128)
    rdp.slora_kv_copy(s.kv, 0, None, None)
    rdp.slora_kv_copy(s.kv, 2, dev(np.array([1, 2], np.int32)), dev(np.array([3, 4], np.int32)), dev(np.zeros(2, np.int32)))
    expect(s, pages, exps, [], [], [], 128)
    assert s.device_status() == 0


def test_copy_skips_what_it_cannot_use():
    s, pages, exps, _ = pool(40, 4096, 64)
    top = (1 << 31) - 1
    for bad in (-1, 40, top, -top - 1):
        for at in range(2):
            src, dst = np.array([3, 4, 5], np.int32), np.array([20, 21, 22], np.int32)
            (src, dst)[at][1] = bad
            rdp.slora_kv_copy(s.kv, 3, dev(src), dev(dst))
            assert s.device_status() == BAD_PAGE
            expect(s, pages, exps, [3, 5], [20, 22], [s.block] * 2, 64)
    for bad in (-1, s.block + 1, top, -top - 1):
        rdp.slora_kv_copy(s.kv, 3, dev(np.array([6, 7, 8], np.int32)), dev(np.array([30, 31, 32], np.int32)),
                          dev(np.array([2, bad, 5], np.int32)))
        assert s.device_status() == BAD_LENGTH
        expect(s, pages, exps, [6, 8], [30, 32], [2, 5], 64)


def test_copy_far_into_a_large_pool():
    """Offsets past 32 bits."""
    num = 300000
    s = KVSession(8192, num, 1, 128)
    rng = np.random.default_rng(1)
    src, dst = np.array([num - 1, 5, 280000, 263000], np.int32), np.array([7, num - 2, 270000, 262144], np.int32)
    data = rng.integers(0, 256, (4, 16384), dtype=np.uint8)
    s.pages[torch.from_numpy(src).long().cuda()] = dev(data)
    s.pages[torch.from_numpy(dst).long().cuda()] = 0
    s.exponents[torch.from_numpy(src).long().cuda()] = dev(np.array([1, -2, 3, -4], np.int8))
    torch.cuda.synchronize()
    rdp.slora_kv_copy(s.kv, 4, dev(src), dev(dst))
    torch.cuda.synchronize()
    assert np.array_equal(s.pages[torch.from_numpy(dst).long().cuda()].cpu().numpy(), data)
    assert s.exponents[torch.from_numpy(dst).long().cuda()].tolist() == [1, -2, 3, -4]
    assert s.device_status() == 0


def test_copies_in_a_graph_and_on_another_stream():
    s, pages, exps, rng = pool(200, 4096, 128)
    src, dst, rows = dev(np.arange(60, dtype=np.int32)), dev(np.arange(100, 160, dtype=np.int32)), dev(np.full(60, 9, np.int32))
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        rdp.slora_kv_copy(s.kv, 60, src, dst, rows, st)
    for i in range(3):
        rows.fill_(9 + i)
        src.copy_(src.flip(0))
        torch.cuda.synchronize()
        g.replay()
        expect(s, pages, exps, src.tolist(), range(100, 160), [9 + i] * 60, 128)
    with torch.cuda.stream(st):
        rdp.slora_kv_copy(s.kv, 60, src, dst, None, st)
    expect(s, pages, exps, src.tolist(), range(100, 160), [s.block] * 60, 128)


def test_copy_refusals():
    s, pages, exps, _ = pool(8, 4096, 128)
    a = dev(np.arange(8, dtype=np.int32))
    for args in ((None, 1, a, a), (s.kv, -1, a, a), (s.kv, 1 << 31, a, a), (s.kv, 1, None, a), (s.kv, 1, a, None),
                 (s.kv, 1, a.data_ptr() + 2, a), (s.kv, 1, a, a.data_ptr() + 1), (s.kv, 1, a, a, a.data_ptr() + 3)):
        with pytest.raises(rdp.SloraError) as e:
            rdp.slora_kv_copy(*args)
        assert e.value.status == 1
    expect(s, pages, exps, [], [], [], 128)
    assert s.device_status() == 0


def test_forked_sequences_share_their_prefix():
    """Two sequences fork in two: whole blocks are shared, the last one is copied; both branches append and attend as
    two sequences that were never one."""
    c = Case([(1, 200), (1, 129)], hq=4, hkv=2, seed=90)
    p = c.s.pool
    lengths = [199, 128]                                   # what is cached before the new tokens; 128 fills its block
    blocks = [-(-n // c.bt) for n in lengths]
    mine = [c.table[s, :blocks[s]].copy() for s in range(2)]
    used = np.concatenate([c.table[s, :4].ravel() for s in range(2)])
    used = used[used >= 0]
    rdp.slora_pages_free(p, len(c.pages) - len(used), np.setdiff1d(np.arange(len(c.pages)), used).astype(np.int32))
    rest = [c.table[s, b] for s in range(2) for b in range(blocks[s], 4) if c.table[s, b, 0, 0] >= 0]
    for t in rest:
        rdp.slora_pages_free(p, t.size, t.ravel().copy())
    free = rdp.slora_pool_num_free(p)
    src, dst, rows = [], [], []
    fork = []
    for s in range(2):
        whole = lengths[s] // c.bt
        t = mine[s].copy()
        rdp.slora_pages_share(p, t[:whole].size, t[:whole].ravel().copy())
        if whole < blocks[s]:
            new = np.empty(t[whole].shape, np.int32)
            rdp.slora_pages_alloc(p, new.size, new)
            src.append(t[whole].ravel().copy())
            dst.append(new.ravel())
            rows.append(np.full(new.size, lengths[s] % c.bt, np.int32))
            t[whole] = new
        fork.append(t)
    src, dst, rows = (np.concatenate(x).astype(np.int32) for x in (src, dst, rows))
    before = c.s.pages.cpu().numpy()
    rdp.slora_kv_copy(c.s.kv, len(src), dev(src), dev(dst), dev(rows))
    torch.cuda.synchronize()
    after = c.s.pages.cpu().numpy()
    for i, j, r in zip(src, dst, rows):
        assert np.array_equal(after[j, :r * c.d], before[i, :r * c.d])
    # the branches' rows read alike through either table, in calls of the same shape
    q = torch.from_numpy(c.rng.normal(0, 1, (2, 512)).astype(np.float16)).cuda()
    ones, lens = dev(np.arange(3, dtype=np.int32)), dev(np.array(lengths, np.int32))
    outs = []
    for tables in (mine, fork):
        table = np.full((2, 4, 2, 2), -1, np.int32)
        for s in range(2):
            table[s, :blocks[s]] = tables[s]
        b = rdp.KVBatch(2, 2, 1, 4, ones, lens, dev(table))
        outs.append(torch.zeros_like(q))
        rdp.slora_kv_attend(c.s.kv, b, q, 512, 4, outs[-1], 512, softmax_scale=0.05)
    torch.cuda.synchronize()
    assert torch.equal(*outs) and c.s.device_status() == 0
    for t in mine + fork:
        rdp.slora_pages_free(p, t.size, t.ravel().copy())
    assert rdp.slora_pool_num_free(p) == free + sum(t.size for t in mine)
