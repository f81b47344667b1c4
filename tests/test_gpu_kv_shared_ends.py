"""GPU: attention with shared prefixes where a call is at an end of what it takes: groups that do not take
the sequences, parts of a row's sum that are far apart."""
import copy
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_kv import e4m3_values
from tests.test_gpu_kv_ranges import GROUPS, reference
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


def far_apart(c, octaves, low, prefix_scale, own_scale):
    """All keys equal but for their sign, so that the scores of the prefixes (low = 0) or of the own tokens (1)
    lie `octaves` below the others; values as they were, on pages of the given scales.  Returns the scale."""
    c.q.fill_(1.0)
    val = e4m3_values()
    for g, p in enumerate(c.prefix):
        w = p // c.P
        lead = c.table[c.groups[g]].copy()
        for b in range(c.groups[g], c.groups[g + 1]):
            ids = np.concatenate([lead[:w], c.table[b, w:-(-c.lens[b] // c.P)]])
            for part, ours in ((0, ids[:w]), (1, ids[w:])):
                keys = c.codes_np[ours, 0]
                c.codes_np[ours, 0] = np.where(keys & 0x7F == 0x7F, keys, 0xB8 if part == low else 0x38)  # -1, 1
                c.scales_np[ours, 0] = 1.0
                c.scales_np[ours, 1] = own_scale if part else prefix_scale
            full = val[c.codes_np[ids]] * c.scales_np[ids].astype(np.float64)[..., None, None]
            c.kv[b] = tuple(full.transpose(1, 0, 3, 2, 4).reshape(2, -1, c.H, c.D)[:, :c.lens[b]])
    c.upload()
    return octaves * np.log(2.0) / (2 * c.D)


FAR = [
    ([3], [256], [1, 1, 1], [30, 1, 200], 2, 4, 128, 64),             # the few-rows form
    ([2, 1], [64, 32], [1, 2, 1], [0, 7, 5], 2, 3, 64, 16),
    ([3], [384], [5, 2, 5], [40, 3, 300], 2, 7, 128, 64),             # the rows form, with copies and without
    ([2], [256], [20, 17], [9, 150], 1, 8, 64, 32),
    ([2], [6016], [1, 1], [3000, 5000], 1, 7, 128, 64),               # units that several workers join
    ([2], [6016], [9, 9], [3000, 5000], 1, 4, 128, 64),
]


@pytest.mark.parametrize("octaves,big,small", [(1, 70, -70), (60, 20, -30), (125, 60, -60), (130, 60, -60), (144, 60, -80), (200, 100, -90),
                                               (222, 110, -90)])
@pytest.mark.parametrize("low", [0, 1])
@pytest.mark.parametrize("shape", FAR, ids=[str(i) for i in range(len(FAR))])
def test_a_part_far_below_may_have_the_larger_values(shape, low, octaves, big, small):
    """A part whose sum is 2^-octaves of the other's counts where its values are 2^(big - small) times as large."""
    c = Shared(*shape, seed=octaves)
    scales = (2.0 ** big, 2.0 ** small) if low == 0 else (2.0 ** small, 2.0 ** big)
    scale = far_apart(c, octaves, low, *scales)
    c.check(scale=scale)


def check_ranges(c, scale=None):
    """Against 64 bits with the tolerance for scales that lie far apart; prefixes end with a tile."""
    scale = c.D ** -0.5 if scale is None else scale
    assert all(p % 128 == 0 for p in c.prefix)
    out, lse = c.run(scale=scale)
    ref = copy.copy(c)
    ref.table = c.table.copy()
    for g, p in enumerate(c.prefix):
        lead = next(b for b in range(c.groups[g], c.groups[g + 1]) if c.n[b])
        ref.table[c.groups[g]:c.groups[g + 1], :p // c.P] = c.table[lead, :p // c.P]
    want, rl, tol, ltol = reference(ref, scale)
    over = np.abs(out.double().cpu().numpy() - want) - tol
    assert over.max() <= 0, f"output off by {over.max():.3e} beyond its tolerance"
    assert (np.abs(lse.double().cpu().numpy() - rl) <= ltol).all()


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 32)])
@pytest.mark.parametrize("exponents", [(0, -16), (4, -20), (60, 0, -60), (-80, 2), (-126,), (90,)])
def test_value_scales_far_apart(group, dim, page, exponents):
    """Peaked weights over pages whose value scales differ, in the prefixes and behind them."""
    c = Shared([2, 1], [256, 128], [5, 2, 3], [54, 7, 140], 2, group, dim, page, seed=group, qscale=9.0)
    r = np.random.default_rng(group)
    pages = np.unique(c.table[c.table >= 0])
    c.scales_np[pages, 1] = 2.0 ** r.choice(exponents, (len(pages), c.H))
    c.upload()
    check_ranges(c)


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("part", ["prefix", "own", "all"])
def test_pages_of_zero_values(group, part):
    """Values of nothing but zeros (their scale is 2^-126) in one part of a row's tokens, or in both."""
    c = Shared([3], [256], [1, 4, 5], [60, 3, 140], 1, group, 128, 16, seed=group, qscale=4.0)
    lead = c.table[0, :16].copy()
    own = np.unique(c.table[:, 16:][c.table[:, 16:] >= 0])
    zero = {"prefix": lead, "own": own, "all": np.concatenate([lead, own])}[part]
    c.codes_np[zero, 1] = np.where(c.codes_np[zero, 1] & 0x7F == 0x7F, c.codes_np[zero, 1], 0)
    c.scales_np[zero, 1] = 2.0 ** -126
    c.upload()
    check_ranges(c)


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("scale", [math.inf, math.nan, -math.inf])
def test_scales_that_are_no_numbers_reach_those_that_see_them(group, scale):
    """A page of the prefix: all rows of its group, in that head.  A page of one sequence: its rows from there on."""
    c = Shared([2, 1], [128, 64], [5, 2, 3], [30, 7, 9], 2, group, 128, 16, seed=5)
    clean, lse = c.run()
    keep = c.scales_np.copy()
    c.scales_np[c.table[0, 2], 1, 0] = scale
    c.upload()
    out, lse2 = c.run()
    assert torch.isnan(out[:7, :group]).all()
    assert torch.equal(out[7:], clean[7:]) and torch.equal(out[:, group:], clean[:, group:]) and torch.equal(lse2[7:], lse[7:])
    c.scales_np = keep
    assert (128 + 30 + 2) % 16 == 0                          # the third row of sequence 0 begins a page
    c.scales_np[c.table[0, 160 // 16], 1, 1] = scale
    c.upload()
    out, lse2 = c.run()
    assert torch.isnan(out[2:5, group:]).all()
    assert torch.equal(out[:2], clean[:2]) and torch.equal(out[5:], clean[5:]) and torch.equal(out[:, :group], clean[:, :group])
