"""GPU checks of the 8-bit KV cache over long lists of sequences for the prompt kernel, appends in a graph, the largest
pages, and several caches over one pool."""
import numpy as np
import pytest
import torch

import kv_reference as R
import rank_delta_paged_gb300 as rdp
from rank_delta_paged_gb300.harness import _DeviceBytes
from test_gpu_kv import Case, check_append, dev, half

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


def some(rng, n, lo, hi, ctx):
    return [(q, q + int(rng.integers(0, ctx))) for q in map(int, rng.integers(lo, hi + 1, n))]


LISTS = {
    # every sequence a prompt: groups of 32, and several chunks of them
    "prompts": lambda r: some(r, 1500, 30, 40, 30),
    "few more than a group": lambda r: some(r, 33, 50, 60, 10),
    # prompts far apart among the other kernel's sequences and empty ones, the first and the last among them
    "prompts far apart": lambda r: ([(150, 300)] + [(0, 5)] * 100 + some(r, 700, 1, 2, 20) + [(40, 300), (90, 90)] + [(0, 0)] * 300 +
                                    some(r, 800, 1, 1, 9) + [(33, 70)] + [(0, 3)] * 31 + [(300, 333)] + some(r, 400, 1, 2, 9) + [(64, 64)]),
    "prompts at the end": lambda r: [(0, 7)] * 2100 + some(r, 60, 1, 1, 9) + [(70, 200), (35, 36)],
    "one prompt before everything": lambda r: [(129, 700)] + some(r, 2200, 1, 1, 30),
}


@pytest.mark.parametrize("kind", LISTS)
@pytest.mark.parametrize("hq,hkv,d,hidden", [(2, 1, 64, 2048), (2, 2, 128, 2048)])
def test_attend_finds_prompts_in_long_lists(kind, hq, hkv, d, hidden):
    rng = np.random.default_rng(60)
    Case(LISTS[kind](rng), hq=hq, hkv=hkv, d=d, hidden=hidden, seed=61).check()


def test_attend_long_lists_not_causal_and_in_a_window():
    rng = np.random.default_rng(62)
    c = Case(LISTS["prompts far apart"](rng), hq=2, hkv=1, d=64, hidden=2048, seed=63)
    c.check(causal=False)
    c.check(window=40)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_the_largest_pages(fmt, d):
    """Pages of 16384 bytes: blocks of 128 and 256 tokens."""
    seqs = [(1, 1), (1, 128), (1, 257), (5, 300), (2, 130), (0, 9), (140, 500), (33, 256)]
    Case(seqs, hq=8, hkv=2, d=d, hidden=8192, fmt=fmt, seed=64).check()
    Case(seqs[:6], hq=4, hkv=4, d=d, hidden=8192, fmt=fmt, seed=65).check(window=70)
    check_append(Case(seqs, hq=4, hkv=2, d=d, hidden=8192, fmt=fmt, seed=66), rot=d, positions=lambda p: p + 2)


@pytest.mark.parametrize("seqs", [[(1, 70), (1, 200), (0, 3), (1, 64)], [(9, 70), (1, 200), (130, 300), (2, 65)]], ids=["single", "several"])
@pytest.mark.parametrize("given", [False, True])
def test_append_in_a_graph(seqs, given):
    """The append's kernels, chained by programmatic launch, replayed with other tokens each time, then attention over
    what they wrote, in the same graph."""
    eager, c = (Case(seqs, hq=6, hkv=2, seed=67) for _ in range(2))
    batches = {id(x): x.batch() for x in (eager, c)}       # hold the arrays that the graph reads
    n_pos = int(c.kv_len.max())
    angle = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, 128, 2) / 128)
    cos, sin = dev(np.cos(angle).astype(np.float32)), dev(np.sin(angle).astype(np.float32))
    pos = dev(np.concatenate([np.arange(n - m, n) for m, n in seqs]).astype(np.int32)) if given else None
    rope = rdp.KVRope(128, False, n_pos, cos, sin, pos)
    qkv = torch.zeros((c.T, 10 * 128), dtype=torch.float16, device="cuda")
    st = torch.cuda.Stream()

    def step(x, q_out, out, stream):
        q, k, v = qkv, qkv[:, 768:], qkv[:, 1024:]
        b = batches[id(x)]
        rdp.slora_kv_append(x.s.kv, b, k, 1280, v, 1280, q, 1280, q_out, 768, 6, rope, stream)
        rdp.slora_kv_attend(x.s.kv, b, q_out, 768, 6, out, 768, None, 0.1, True, 0, stream)

    bufs = [[torch.zeros((c.T, 768), dtype=torch.float16, device="cuda") for _ in range(2)] for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        step(c, *bufs[0], st)
    for i in range(5):
        x = c.rng.normal(0, 1.5 ** i, (c.T, 1280)).astype(np.float16)      # larger each time: held rows are rescaled
        qkv.copy_(half(x))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        step(eager, *bufs[1], None)
        torch.cuda.synchronize()
        assert torch.equal(c.s.pages, eager.s.pages) and torch.equal(c.s.exponents, eager.s.exponents)
        assert torch.equal(bufs[0][0], bufs[1][0]) and torch.equal(bufs[0][1], bufs[1][1])
    assert c.s.device_status() == 0


def test_two_caches_over_one_pool():
    """Another cache's heads, format and exponents on pages of the same pool, the two in turn on one stream."""
    c = Case([(1, 3000), (3, 400), (150, 300)], hq=8, hkv=2, seed=68, spare=12)
    want, wl = c.attend()
    pages0, exps0 = c.s.pages.cpu().numpy(), c.s.exponents.cpu().numpy()
    kv2 = rdp.slora_kv_create(c.s.pool, 1, 64, rdp.SLORA_KV_INT8)
    try:
        bt = rdp.slora_kv_block_tokens(kv2)
        num = len(c.pages)
        free = np.setdiff1d(np.arange(num), c.table[c.table >= 0])[:12].astype(np.int32)
        table = np.full((2, 3, 1, 2), -1, np.int32)
        table[0, :3, 0], table[1, :2, 0] = free[:6].reshape(3, 2), free[6:10].reshape(2, 2)
        lens, indptr = np.array([2 * bt + 7, bt + 1], np.int32), np.array([0, 2 * bt + 7, 3 * bt + 8], np.int32)
        T = int(indptr[-1])
        b = rdp.KVBatch(T, 2, int(lens.max()), 3, dev(indptr), dev(lens), dev(table))
        rng = np.random.default_rng(69)
        q, k, v = (rng.normal(0, 1, (T, h * 64)).astype(np.float16) for h in (3, 1, 1))
        dq, dk, dv = half(q), half(k), half(v)
        out, lse = torch.empty((T, 192), dtype=torch.float16, device="cuda"), torch.empty((T, 3), device="cuda")
        rdp.slora_kv_append(kv2, b, dk, 64, dv, 64)
        for _ in range(2):
            rdp.slora_kv_attend(kv2, b, dq, 192, 3, out, 192, lse, 0.125)
            got, gl = c.attend()
            assert np.array_equal(got, want) and np.array_equal(gl, wl)
        exps = torch.as_tensor(_DeviceBytes(rdp.slora_kv_exponents(kv2), (num,), "|i1", c.s), device="cuda").cpu().numpy()
        after = c.s.pages.cpu().numpy()
        mine = np.zeros(num, bool)
        mine[free[:10]] = True
        assert np.array_equal(after[~mine], pages0[~mine]) and np.array_equal(c.s.exponents.cpu().numpy(), exps0)
        values = R.decode(np.ascontiguousarray(after[:, :bt * 64].reshape(num, bt, 64)), "int8")
        ref, rl, to, tl = R.attend(values, exps, table, indptr, lens, q.reshape(T, 3, 64), bt, 0.125)
        assert (np.abs(out.float().cpu().numpy().reshape(T, 3, 64) - ref) <= to).all()
        assert (np.abs(lse.cpu().numpy() - rl) <= tl).all()
        for s in range(2):                     # within half a step of what was appended
            for p in range(lens[s]):
                page, x = table[s, p // bt, 0, 1], v[indptr[s] + p].astype(np.float64)
                assert np.abs(values[page, p % bt] * 2.0 ** float(exps[page]) - x).max() <= 0.5000001 * 2.0 ** float(exps[page])
        assert c.s.device_status() == 0
    finally:
        rdp.slora_kv_destroy(kv2)
    got, _ = c.attend()
    assert np.array_equal(got, want)
