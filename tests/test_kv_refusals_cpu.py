"""CPU checks of the KV cache calls' refusals that need no cache: null handles and structures return a status and a
message, and launch nothing."""
import shutil

import pytest

import rank_delta_paged_gb300 as rdp
from rank_delta_paged_gb300 import build as B

pytestmark = pytest.mark.skipif(shutil.which(B.NVCC) is None, reason="nvcc not available")


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def test_null_caches_are_refused():
    b = rdp.KVBatch(1, 1, 1, 1, None, None, None)
    keep = rdp.KVKeep(1, 0, 0, 1, None, None, None, None, None)
    for fn, args in ((rdp.slora_kv_append_norm, (None, b, None, 64, None, 64, None, 0, None, 0, 0, rdp.KVNorm(1e-6))),
                     (rdp.slora_kv_append_norm, (None, b, None, 64, None, 64)),
                     (rdp.slora_kv_attend_sinks, (None, b, None, 64, 1, None, 64, None, 1.0, 8, 4)),
                     (rdp.slora_kv_attend_sinks, (None, b, None, 64, 1, None, 64, None, 1.0, 0, 4)),
                     (rdp.slora_kv_copy, (None, 0, None, None)),
                     (rdp.slora_kv_compact, (None, keep)),
                     (rdp.slora_pages_share, (None, 0, None))):
        with pytest.raises(rdp.SloraError) as e:
            fn(*args)
        assert e.value.status == 1 and len(rdp.slora_last_error()) > len("SLORA_ERR_INVALID_ARG: ")


def test_version_names_the_operators():
    assert rdp.slora_version() >= 400
