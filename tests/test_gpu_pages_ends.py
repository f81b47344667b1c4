"""GPU: pages found and given back where a call is at an end of what it takes; compared exactly with the
definition, as in the other tests of pages."""
import numpy as np
import pytest
import torch

from tests.test_gpu_pages import Pool, dev

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("mxfp4_routed_expert_topk_gb300")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()


@pytest.mark.parametrize("length", [-2 ** 31, -5, -1, 0, 1, 40, 64, 65, 2 ** 31 - 1])
@pytest.mark.parametrize("keep", [-1, -2 ** 31])
def test_a_negative_keep_is_reported_whatever_the_length(keep, length):
    c = Pool(3, 4, 30, 16)
    c.reserve([40, 33, 1])
    moe.moe_kv_release(dev([keep, 16, 1]), dev([length, 33, 1]), c.d_table, c.d_refs, 16, ws=c.ws)
    assert moe.moe_check_status(c.ws) == moe.MOE_ERR_BAD_PAGE
    c.refs[c.table[1, 1:3]] = 0                              # (the others' pages go back all the same)
    c.table[1, 1:3] = -1
    c.same()


@pytest.mark.parametrize("length", [-2 ** 31, -1, 0, 39, 40])
def test_a_keep_from_the_length_on_gives_nothing_back(length):
    c = Pool(2, 4, 30, 16)
    c.reserve([40, 33])
    for keep in (max(length, 0), 64, 65, 2 ** 31 - 1):
        moe.moe_kv_release(dev([keep, 33]), dev([length, 33]), c.d_table, c.d_refs, 16, ws=c.ws)
        assert moe.moe_check_status(c.ws) == moe.MOE_OK
        c.same()
    moe.moe_kv_release(dev([2 ** 31 - 1, 33]), dev([2 ** 31 - 1, 33]), c.d_table, c.d_refs, 16, ws=c.ws)
    assert moe.moe_check_status(c.ws) == moe.MOE_OK
    c.same()
