"""GPU check of the order between the KV attention and the adapters' deltas that follow it on a stream: the attention's
output is the x of a planned apply with prefill segments, whose kernels may start before those ahead of
them have ended and read x only once it is written."""
import numpy as np
import pytest
import torch

import rank_delta_paged_gb300 as rdp
from rank_delta_paged_gb300 import workloads as W
from rank_delta_paged_gb300.harness import PoolSession
from test_gpu_kv import Case, dev, half

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rdp.build.build()
    rdp.lib()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("seqs_of", ["prompts and single tokens", "one sequence of each row"])
def test_attention_then_planned_deltas(seqs_of, graph):
    w = W.mixed_iteration(n_layers=2, pool_bytes=2 << 30, n_prefill=4, n_decode=200)
    lens = np.diff(w.seg_indptr)
    if seqs_of.startswith("prompts"):
        seqs = [(int(m), int(m) + 37) for m in lens] + [(1, 50)] * (w.T - int(lens.sum()))
    else:                                                  # the streaming kernel alone
        seqs = [(1, 20)] * w.T
    c = Case(seqs, hq=32, hkv=1, d=128, hidden=4096, seed=50, stale=False)
    assert c.T == w.T and w.hidden == 4096
    with PoolSession(w) as s:
        s.load(w.used_adapters())
        idx, seg = dev(w.token_adapter_idx), dev(w.seg_indptr)
        plan = rdp.slora_plan_create(s.pool, 2, w.T, idx, seg, len(lens))
        b = c.batch()
        rng = np.random.default_rng(6)
        q = torch.empty((c.T, 4096), dtype=torch.float16, device="cuda")
        x, y = torch.zeros_like(q), [torch.zeros_like(q) for _ in range(2)]
        st = torch.cuda.Stream()

        def attend():
            rdp.slora_kv_attend(c.s.kv, b, q, 4096, 32, x, 4096, None, 0.1, True, 0, st)

        def layer():
            attend()
            rdp.slora_plan_apply(plan, [0, 1], [x, x], y, st)
            attend()
            rdp.slora_plan_apply(plan, [2, 3], [x, x], y, st)

        run = layer
        try:
            # the first use of a plan is not to be captured: its kernels differ from the later ones'
            rdp.slora_plan_apply(plan, [0, 1], [x, x], y, st)
            torch.cuda.synchronize()
            if graph:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=st):
                    layer()
                run = g.replay
            for i in range(6):
                q.copy_(half(rng.normal(0, 1, (c.T, 4096)).astype(np.float16)))
                x.fill_(float("nan"))
                for t in y:
                    t.zero_()
                torch.cuda.synchronize()
                attend()
                torch.cuda.synchronize()
                for p in ([0, 1], [2, 3]):
                    rdp.slora_plan_apply(plan, p, [x, x], y, st)
                    torch.cuda.synchronize()
                want = [t.clone() for t in y]
                assert all(bool(torch.isfinite(t).all()) for t in want)
                x.fill_(float("nan"))
                for t in y:
                    t.zero_()
                torch.cuda.synchronize()
                run()
                torch.cuda.synchronize()
                assert all(torch.equal(a, t) for a, t in zip(want, y)), i
            assert s.device_status() == 0 and c.s.device_status() == 0
        finally:
            rdp.slora_plan_destroy(plan)
