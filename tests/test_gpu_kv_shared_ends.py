"""GPU: attention with shared prefixes where a call is at an end of what it takes: groups that do not take
the sequences, parts of a row's sum that are far apart."""
import pytest
import torch

from tests.test_gpu_kv_shared import Shared

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("mxfp4_routed_expert_topk_gb300")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()


@pytest.fixture(autouse=True, params=[False, True], ids=["once", "twice"])
def _ways(request):
    Shared.twice = request.param
    yield
    Shared.twice = False


def test_groups_past_the_last_sequence_are_reported():
    c = Shared([2, 2], [128, 64], [1, 2, 1, 1], [9, 0, 5, 1], 2, 7, 128, 32, seed=8)
    good, _ = c.check()
    ws = moe.workspace(c.workspace())

    def call(groups, prefix):
        out = moe.moe_kv_attention_shared(c.cache, 0, c.q, c.dev(c.cu), c.dev(c.lens), c.dev(c.table), c.dev(groups),
                                          c.dev(prefix), max_rows=2, max_group_rows=3, ws=ws)
        return out, moe.moe_check_status(ws)

    big = 2 ** 31 - 1
    for more in ([5], [big], [4, 5], [4, 4, 6], [6, 5], [3], [4, 3], [-1], [-2 ** 31]):
        assert call([0, 2, 4] + more, [128, 64] + [0] * len(more))[1] == moe.MOE_ERR_BAD_PAGE, more
    for groups in ([0, 2, 5], [0, 2, big], [-1, 0, 2, 4], [-2 ** 31, 0, 2, 4], [0, 2, 3]):
        assert call(groups, [128, 64, 0][:len(groups) - 1])[1] == moe.MOE_ERR_BAD_PAGE, groups
    for groups, prefix in (([0, 2, 4], [128, 64]), ([0, 0, 2, 2, 4, 4], [7, 128, 99, 64, 64])):
        out, status = call(groups, prefix)
        assert status == moe.MOE_OK and torch.equal(out, good), groups
