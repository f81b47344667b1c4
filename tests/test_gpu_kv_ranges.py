"""GPU: the cache attention where pages' value scales, queries and lengths lie far apart,
against 64 bits.

A softmax weight enters the product with its page's value scale, as w = p vs in two E4M3
parts under a power of two that puts the largest w a row sees in its 128-token tile at 256
(a scale below 2^-90 counts as 2^-90 for that).  E4M3's step is 2^-9 at its finest, so a
weight keeps 8 significant bits (2^-9 of itself) or is off by one such step at most, which
is 2^-17 of the tile's largest w: each token's codes times that are the tolerance below,
beside the terms of the queries and of the bf16 output.  Scores are fp32 in units of log2,
with log2 vs added: below 2^8, so each of their three roundings is 2^-17 at most, and the
weights are off by 2^-15."""
import math

import numpy as np
import pytest
import torch

from tests._util import bf16_half_ulp
from tests.test_gpu_kv import Case, _append_case, e4m3_values, ref_append

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("mxfp4_routed_expert_topk_gb300")

# rows of a tile (5 of each sequence): 15, 35, 60, 100 and 180, which is every form
GROUPS = [3, 7, 12, 20, 36]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()


def reference(c, scale):
    """(out, lse, tolerance of out, tolerance of lse) of a Case, from its codes and scales as they are."""
    val = e4m3_values()
    q = c.q.double().cpu().numpy()
    R, Hq, D = q.shape
    out, lse = np.zeros((R, Hq, D)), np.full((R, Hq), -np.inf)
    tol, ltol = np.zeros((R, Hq, D)), np.zeros((R, Hq))
    for b, T in enumerate(c.lens):
        n, pages = c.n[b], c.table[b, :-(-T // c.P)]
        codes = val[c.codes_np[pages]].transpose(1, 0, 3, 2, 4).reshape(2, -1, c.H, D)[:, :T]
        sc = c.scales_np[pages].astype(np.float64).transpose(1, 0, 2).repeat(c.P, 1)[:, :T]
        for i in range(n):
            see, r = min(T, max(0, T - n + i + 1)), c.cu[b] + i
            for hq in range(Hq if see else 0):
                h, qr = hq // c.G, q[r, hq]
                K, V, vs = codes[0, :see, h] * sc[0, :see, h, None], codes[1, :see, h], sc[1, :see, h]
                s = scale * (K @ qr)
                p = np.exp(s - s.max())
                l = p.sum()
                w = p * vs
                out[r, hq] = w @ V / l
                lse[r, hq] = s.max() + math.log(l)
                ds = scale * (2.0 ** -17 * np.abs(qr).max() * np.abs(K).sum(1).max()
                              + 2.0 ** -18 * (np.abs(K) @ np.abs(qr)).max())
                A = w @ np.abs(V) / l
                floor = np.zeros(D)
                for t in range(0, see, 128):
                    top = (p[t:t + 128] * np.maximum(vs[t:t + 128], 2.0 ** -90)).max()
                    floor += 2.0 ** -17 * top * np.abs(V[t:t + 128]).sum(0)
                tol[r, hq] = bf16_half_ulp(out[r, hq]) * 1.001 + (2.0 ** -9 + 2 * ds + 2.0 ** -15) * A + floor / l
                ltol[r, hq] = ds + 2.0 ** -15 + 2.0 ** -20 * (abs(lse[r, hq]) + np.abs(s).max())
    return out, lse, tol, ltol


def check(c, scale=None):
    scale = c.D ** -0.5 if scale is None else scale
    got, lse = c.run(scale=scale)
    ref, rl, tol, ltol = reference(c, scale)
    over = np.abs(got.double().cpu().numpy() - ref) - tol
    assert over.max() <= 0, f"output off by {over.max():.3e} beyond its tolerance"
    assert (np.abs(lse.double().cpu().numpy() - rl) <= ltol).all()


# ------------------------------------------------------------ value scales


@pytest.mark.parametrize("old", [30, 1006])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("scale", [math.inf, math.nan, 2.0 ** 20, 2.0 ** 60, 2.0 ** -60])
def test_scales_of_unseen_pages_do_not_reach(old, group, side, scale):
    """A draft's page inside a tile that earlier rows share: whatever its scales are, rows
    before it, the other head and the other sequence keep their results bit for bit."""
    n = 5
    c = Case([n, 2], [old, 9], 2, group, 128, 16, seed=5)
    clean, lse = c.run()
    first = old + 2                                       # token of row 2
    assert first % 16 == 0 and first % 128 != 0
    c.scales_np[c.table[0, first // 16], side, 0] = scale
    c.upload()
    out, lse2 = c.run()
    for a, b in ((out, clean), (lse2, lse)):
        assert torch.equal(a[:2], b[:2]) and torch.equal(a[n:], b[n:]) and torch.equal(a[:n, group:], b[:n, group:])
    if side == 1:
        seen = out[2:n, :group]
        if math.isfinite(scale):
            check(c)
        else:
            assert torch.isnan(seen).all()


def spread_values(c, exponents, rng):
    """Value scales 2^e of every page and head, e drawn from `exponents`."""
    pages = c.table[c.table >= 0]
    c.scales_np[pages, 1] = 2.0 ** rng.choice(exponents, (len(pages), c.H))
    c.upload()


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 32)])
@pytest.mark.parametrize("exponents", [(0, -12), (0, -16), (4, -20), (20, 0, -20), (60, 0, -60), (-80, 2)])
def test_value_scales_far_apart(group, dim, page, exponents):
    """Peaked weights over pages whose scales differ by 2^12 to 2^120: many rows have nearly all
    their weight on a small one, and large ones beside it in the tile."""
    c = Case([5, 2], [310, 40], 2, group, dim, page, seed=group, qscale=9.0)
    spread_values(c, exponents, np.random.default_rng(group))
    check(c)


@pytest.mark.parametrize("group", [3, 7, 20])
@pytest.mark.parametrize("ratio", [8, 12, 18, 24, 40])
def test_all_weight_on_the_small_scale(group, ratio):
    """Two pages of a tile: scores of one stand 60 (in log2) above the other's, whose scale is larger."""
    c = Case([2], [30], 1, group, 128, 16, seed=ratio)
    q = np.zeros(tuple(c.q.shape))
    q[..., 0] = 16.0
    c.q = torch.from_numpy(q).to(torch.bfloat16).cuda()
    small, large = c.table[0, 0], c.table[0, 1]
    c.scales_np[[small, large], 0] = 2.0 ** -5
    c.codes_np[small, 0, ..., 0] = 0x78                   # 256 / 32 * 16 / sqrt(128) = 11.3
    c.codes_np[large, 0, ..., 0] = 0xF8                   # -256
    c.scales_np[small, 1], c.scales_np[large, 1] = 2.0 ** -ratio, 1.0
    c.upload()
    check(c)


@pytest.mark.parametrize("group", GROUPS)
def test_pages_of_zero_values(group):
    """Pages of nothing but zeros have the scale 2^-126; their tokens still count in the sums,
    beside other pages and alone."""
    for which in (slice(0, None, 2), slice(0, 6), slice(0, None)):
        c = Case([5], [200], 1, group, 128, 16, seed=group, qscale=4.0)
        zero = c.table[0][c.table[0] >= 0][which]
        c.codes_np[zero, 1] = 0
        c.scales_np[zero, 1] = 2.0 ** -126
        c.upload()
        check(c)


@pytest.mark.parametrize("group", [3, 7, 20])
@pytest.mark.parametrize("e", [-126, -100, -90, -60, 60, 90])
def test_value_scales_alike_at_the_ends(group, e):
    c = Case([5], [300], 2, group, 64, 16, seed=group)
    spread_values(c, (e,), np.random.default_rng(0))
    check(c)


# ----------------------------------------------------------------- queries


@pytest.mark.parametrize("group", [16, 32, 64, 128])
def test_small_query_values(group):
    """Every significand at 2^-7 to 2^-18 of the row's largest value, read from lse: one token, whose
    key has one value at the small one's place, so that lse is the score.  The parts are multiples
    of 2^-16 of the largest (E4M3's step 2^-9 at 2^7), which lse tells apart.  Exact from 2^-9 on;
    to 2^-17 of the largest below."""
    x = np.concatenate([np.arange(128, 256) / 128 * 2.0 ** e for e in range(-18, -6)])
    x[::2] *= -1
    seqs = len(x) // group
    c = Case([1] * seqs, [0] * seqs, 1, group, 64, 16)
    page = c.table[:, 0]
    c.codes_np[page, 0, 0, 0] = 0
    c.codes_np[page, 0, 0, 0, 9] = 0x38                   # 1
    c.scales_np[page] = 1.0
    c.upload()
    q = np.zeros((seqs, group, 64))
    q[..., 3], q[..., 9] = 1.0, x.reshape(seqs, group)
    c.q = torch.from_numpy(q).to(torch.bfloat16).cuda()
    _, lse = c.run(scale=256.0)
    got = np.round(lse.double().cpu().numpy().reshape(-1) / 256 * 2.0 ** 16) * 2.0 ** -16
    assert (np.abs(got - x) <= np.where(np.abs(x) >= 2.0 ** -9, 0, 2.0 ** -17)).all()


# ------------------------------------------------------------- workspaces


@pytest.mark.parametrize("heads,group", [(2, 1), (1, 7), (2, 8), (1, 16), (1, 20), (1, 136)])
def test_workspace_serves_fewer_rows(heads, group):
    """A workspace made for max_rows rows serves every smaller number, across 128 rows a tile and more."""
    cache = moe.KvCache(2, 1, heads, 64, 16)
    sizes = [moe.moe_kv_attention_workspace_size(cache, m, heads * group) for m in range(40)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("group,most", [(7, 19), (8, 17), (16, 9)])
def test_fewer_rows_in_a_workspace_for_more(group, most):
    c = Case([most, 1], [100, 300], 1, group, 64, 16, seed=group)
    ws = moe.workspace(moe.moe_kv_attention_workspace_size(c.cache, most, group))
    for m in range(1, most + 1):
        cu, lens = [0, m, m + 1], [100 + m, 301]
        args = (c.cache, 0, c.q[:m + 1], c.dev(cu), c.dev(lens), c.dev(c.table))
        want = moe.moe_kv_attention(*args, max_rows=m)
        got = moe.moe_kv_attention(*args, max_rows=m, ws=ws)
        assert torch.equal(got, want) and moe.moe_check_status(ws) == moe.MOE_OK


# ---------------------------------------------------------- division of work


@pytest.mark.parametrize("group", [4, 20, 70])
def test_long_sequence_beside_short_ones(group):
    """The parts that a long sequence is cut into, each of them joined after all others, are as many
    beside short sequences as alone; they are counted by what the call leaves in the workspace."""
    parts = []
    for short in (0, 10, 63):
        n = [1] * (1 + short)
        c = Case(n, [100000] + [4] * short, 1, group, 64, 128, seed=3)
        ws = moe.workspace(moe.moe_kv_attention_workspace_size(c.cache, 1, group))
        ws[256:] = 0xFF
        moe.moe_kv_attention(c.cache, 0, c.q, c.dev(c.cu), c.dev(c.lens), c.dev(c.table), max_rows=1, ws=ws)
        assert moe.moe_check_status(ws) == moe.MOE_OK
        words = (ws[256:].view(torch.int32) != -1).sum().item()
        assert words % (group * 66) == 0                  # whole parts: a row's 64 values, reference and sum
        parts.append(words // (group * 66))
    assert parts[0] > 1 and max(parts) <= 1.25 * parts[0], parts


@pytest.mark.parametrize("group", [4, 7, 12, 24])
@pytest.mark.parametrize("dim", [64, 128])
def test_tables_of_one_tile(group, dim):
    """Tables that have room for 128 tokens take the rows in one copy where longer ones take several."""
    c = Case([5, 1, 3], [107, 0, 40], 2, group, dim, 16, seed=group)
    assert c.table.shape[1] * 16 == 128
    check(c)
    few, lse = c.run()
    c.table = np.concatenate([c.table, np.full((3, 4), -1, dtype=np.int32)], 1)
    check(c)
    more, lse2 = c.run()
    assert torch.allclose(few.float(), more.float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    assert torch.allclose(lse, lse2, rtol=0, atol=2.0 ** -12)


# ----------------------------------------------------------------- appends


def test_append_with_idle_sequences():
    """A sequence without rows is left alone wherever it is said to start."""
    cache, codes, scales, table, k, v = _append_case([3, 0, 2, 0], [10, 4, 30, 7], 2, 128, 16, seed=2)
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    cu = [0, 3, 3, 5, 5]
    ws = moe.workspace(moe.moe_kv_append_workspace_size())
    for idle in (-1, -2 ** 31, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        moe.moe_kv_append(cache, 1, k, v, dev(cu), dev([10, idle, 30, idle]), dev(table), ws=ws)
        assert moe.moe_check_status(ws) == moe.MOE_OK
    ref_append(codes, scales, k.double().cpu().numpy(), v.double().cpu().numpy(), cu, [10, 0, 30, 0], table, 16)
    assert np.array_equal(cache.codes(1).double().cpu().numpy(), codes)
    assert np.array_equal(cache.scales(1).double().cpu().numpy(), scales)


def test_append_at_the_longest_lengths():
    """A table with room for more than 2^31 tokens: up to 2^30 of them rows are written."""
    rng = np.random.default_rng(1)
    cache = moe.KvCache(2, 1, 1, 64, 128)
    cache.buffer.fill_(0x31)
    table = torch.full((1, (1 << 24) + 1), 1, dtype=torch.int32, device="cuda")
    k, v = (torch.from_numpy(rng.standard_normal((2, 1, 64))).to(torch.bfloat16).cuda() for _ in range(2))
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    ws = moe.workspace(moe.moe_kv_append_workspace_size())
    before = cache.buffer.clone()
    for start in (2 ** 30, 2 ** 31 - 2, 2 ** 31 - 1):
        moe.moe_kv_append(cache, 0, k, v, cu, torch.tensor([start], dtype=torch.int32, device="cuda"), table, ws=ws)
        assert moe.moe_check_status(ws) == moe.MOE_ERR_BAD_PAGE and torch.equal(cache.buffer, before)
        moe.moe_clear_status(ws)
    for start, written in ((2 ** 30 - 130, 2), (2 ** 30 - 1, 1)):
        cache.buffer.copy_(before)
        cache.scales(0).fill_(1.0)
        moe.moe_kv_append(cache, 0, k, v, cu, torch.tensor([start], dtype=torch.int32, device="cuda"), table, ws=ws)
        assert moe.moe_check_status(ws) == (moe.MOE_OK if written == 2 else moe.MOE_ERR_BAD_PAGE)
        moe.moe_clear_status(ws)
        slot = start % 128
        for side, x in enumerate((k, v)):
            want = x[:written].float().to(torch.float8_e4m3fn)
            assert torch.equal(cache.codes(0)[1, side, 0, slot:slot + written].float(), want[:, 0].float())
            assert cache.scales(0)[1, side, 0] == 1.0


def test_append_into_no_table():
    """Rows that have no table to land in are reported; sequences without rows need none."""
    cache, _, _, _, k, v = _append_case([3], [0], 2, 64, 16, seed=2)
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    none = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    ws = moe.workspace(moe.moe_kv_append_workspace_size())
    before = cache.buffer.clone()
    moe.moe_kv_append(cache, 1, k, v, dev([1, 1, 1]), dev([0, 5]), none, ws=ws)
    assert moe.moe_check_status(ws) == moe.MOE_OK
    moe.moe_kv_append(cache, 1, k, v, dev([0, 2, 3]), dev([0, 0]), none, ws=ws)
    assert moe.moe_check_status(ws) == moe.MOE_ERR_BAD_PAGE and torch.equal(cache.buffer, before)
