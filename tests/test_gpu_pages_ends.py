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


def spread(total, seqs, r):
    """`total` pages over `seqs` sequences, an eighth of them idle."""
    p = np.where(r.random(seqs) < 0.125, 0.0, r.random(seqs))
    return r.multinomial(total, p / p.sum())


@pytest.mark.parametrize("lead", [0, 1, 3])
@pytest.mark.parametrize("border", ["idle", "inside"])
@pytest.mark.parametrize("total", [32767, 32768, 32769, 65536, 65537, 70000])
def test_more_pages_than_are_handed_out_at_a_time(total, border, lead):
    """32768 pages are handed out at a time: what was taken then is not free any more, and the next ones go on inside
    a sequence, or behind one after which some stand idle.  The counts lie at any address."""
    r = np.random.default_rng(total + lead)
    if border == "inside" or total <= 32768:
        pages = spread(total, 900, r)
    else:
        pages = np.concatenate([spread(32768, 500, r), [0, 0, 0], spread(total - 32768, 400, r)])
    n_pages = total + total // 2 + 11
    c = Pool(len(pages), int(pages.max()) + 2, n_pages, 16, held=np.sort(r.permutation(n_pages)[:total // 2]))
    wide = torch.full((n_pages + 9,), 5, dtype=torch.int32, device="cuda")
    wide[lead:lead + n_pages] = c.d_refs
    c.d_refs = wide[lead:lead + n_pages]
    more = r.integers(1, 17, len(pages))
    c.reserve(np.where(pages > 0, 16 * (pages - 1) + more, 0))
    c.reserve(np.where(r.random(len(pages)) < 0.01, 3, 0))
    c.release(np.zeros(len(pages), dtype=np.int64))
    assert c.refs.sum() == total // 2
    assert (wide[:lead] == 5).all() and (wide[lead + n_pages:] == 5).all()


def test_one_page_more_than_there_are_past_a_round():
    c = Pool(2, 40000, 66000, 16, held=range(0, 66000, 660))
    free = 66000 - 100
    c.reserve([16 * 33000, 16 * (free - 33000) + 1], status=moe.MOE_ERR_NO_PAGE)
    c.reserve([16 * 33000, 16 * (free - 33000)])
    c.reserve([1, 0], status=moe.MOE_ERR_NO_PAGE)
    c.release([0, 0])
