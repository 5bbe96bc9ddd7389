"""CPU checks of page sharing: holders are counted, a page returns with its last one."""
import shutil

import numpy as np
import pytest

import rank_delta_paged_gb300 as rdp
from rank_delta_paged_gb300 import build as B

pytestmark = pytest.mark.skipif(shutil.which(B.NVCC) is None, reason="nvcc not available")


@pytest.fixture
def pages():
    B.build()
    a = rdp.slora_pagealloc_create(10, 3)
    out = np.empty(6, np.int32)
    rdp.slora_pagealloc_alloc(a, 6, out)
    yield a, out
    rdp.slora_pagealloc_destroy(a)


def refused(fn, *args):
    with pytest.raises(rdp.SloraError) as e:
        fn(*args)
    assert e.value.status == 1


def test_a_page_returns_with_its_last_holder(pages):
    a, p = pages
    rdp.slora_pagealloc_share(a, 3, p[[0, 1, 0]])          # page 0 has three holders, page 1 two
    rdp.slora_pagealloc_free(a, 3, p[:3].copy())
    assert rdp.slora_pagealloc_num_free(a) == 5            # page 2
    rdp.slora_pagealloc_free(a, 2, p[:2].copy())
    assert rdp.slora_pagealloc_num_free(a) == 6            # page 1
    refused(rdp.slora_pagealloc_free, a, 2, p[[1, 0]])     # page 1 is gone, and page 0 keeps its holder
    assert rdp.slora_pagealloc_num_free(a) == 6
    rdp.slora_pagealloc_free(a, 1, p[:1].copy())
    assert rdp.slora_pagealloc_num_free(a) == 7
    refused(rdp.slora_pagealloc_free, a, 1, p[:1].copy())


def test_a_free_that_is_refused_keeps_every_holder(pages):
    a, p = pages
    rdp.slora_pagealloc_share(a, 1, p[:1].copy())
    refused(rdp.slora_pagealloc_free, a, 2, p[[0, 0]])     # twice in one call
    rdp.slora_pagealloc_free(a, 1, p[:1].copy())
    assert rdp.slora_pagealloc_num_free(a) == 4
    rdp.slora_pagealloc_free(a, 1, p[:1].copy())
    assert rdp.slora_pagealloc_num_free(a) == 5


def test_share_refusals_change_nothing(pages):
    a, p = pages
    free = np.setdiff1d(np.arange(10), p).astype(np.int32)
    for bad in (free[0], -1, 10, np.int32(1 << 30)):
        refused(rdp.slora_pagealloc_share, a, 2, np.array([p[0], bad], np.int32))
    refused(rdp.slora_pagealloc_share, a, -1, p)
    refused(rdp.slora_pagealloc_share, a, 1, None)
    refused(rdp.slora_pagealloc_share, None, 1, p)
    refused(rdp.slora_pages_share, None, 1, p)
    rdp.slora_pagealloc_share(a, 0, None)
    rdp.slora_pagealloc_free(a, 6, p)                      # one holder each
    assert rdp.slora_pagealloc_num_free(a) == 10


def test_a_page_that_came_back_starts_with_one_holder(pages):
    a, p = pages
    rdp.slora_pagealloc_share(a, 6, p)
    rdp.slora_pagealloc_free(a, 6, p)
    rdp.slora_pagealloc_free(a, 6, p)
    assert rdp.slora_pagealloc_num_free(a) == 10
    again = np.empty(10, np.int32)
    rdp.slora_pagealloc_alloc(a, 10, again)
    rdp.slora_pagealloc_free(a, 10, again)
    assert rdp.slora_pagealloc_num_free(a) == 10
