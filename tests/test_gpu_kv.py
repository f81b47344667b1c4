"""GPU: the paged 8-bit key/value cache and the attention over it, against plain
implementations in 64 bits.

Appending is compared exactly: scales and codes follow from the definition (largest
finite magnitude, smallest power of two, round to nearest even).  The attention's
tolerance is derived from its stated number formats, element by element:

  - the output is bf16: half a bf16 step at |o|;
  - each softmax weight enters the product with 8 significant bits: 2^-9 of
    A = sum_t p_t |v_t|; weights below 2^-9 of 1/256 of the largest in their 128-token
    tile round to a multiple of that: 2^-18 of (largest weight) x (largest |v|) per token;
  - the query's two parts leave at most 2^-17 of the row's largest value, fp32 sums of
    head_dim products at most 2^-18 of the sum of their magnitudes; a score error of ds
    changes the weights by 2 ds at most;
  - fp32 exponentials, sums and scalings: 2^-16 of A.
"""
import math

import numpy as np
import pytest
import torch

from tests._util import bf16_half_ulp
from tests.test_gpu_guard_bands import Guarded

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("mxfp4_routed_expert_topk_gb300")
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()


# ------------------------------------------------------------- references


def e4m3_values():
    """The 256 code values, from the bit fields (0x7F and 0xFF are NaN)."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = math.nan if (c & 0x7F) == 0x7F else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -x if s else x
    return v


def round_e4m3(x):
    """Nearest E4M3 value (ties to even), saturating; NaN kept.  64 bits."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -20))), -6) - 3)
    return np.copysign(np.minimum(np.round(a / step) * step, 448.0), x)


def ref_append(codes, scales, k, v, cu, start, table, P):
    """In place, on float64 arrays codes [pages][2][H][P][D] and scales [pages][2][H]."""
    for b in range(len(start)):
        n, s0 = cu[b + 1] - cu[b], start[b]
        if n == 0:
            continue
        for col in range(s0 // P, (s0 + n - 1) // P + 1):
            lo, hi = max(s0, col * P), min(s0 + n, (col + 1) * P)
            page, keep = table[b][col], lo - col * P
            for side, src in enumerate((k, v)):
                x = src[cu[b] + lo - s0:cu[b] + hi - s0].astype(np.float64)  # [t][H][D]
                fin = np.where(np.isfinite(x), np.abs(x), 0.0)
                for h in range(x.shape[1]):
                    e = -126
                    amax = fin[:, h].max()
                    while amax > 448.0 * 2.0 ** e:
                        e += 1
                    now = 2.0 ** e
                    if keep:
                        old = scales[page, side, h]
                        now = max(now, old)
                        codes[page, side, h, :keep] = round_e4m3(codes[page, side, h, :keep] * (old / now))
                    codes[page, side, h, keep:hi - col * P] = round_e4m3(x[:, h] / now)
                    scales[page, side, h] = now


def ref_attention(kv, q, cu, lens, scale, P_tile=128):
    """kv: per sequence (K [T][H][D], V [T][H][D]) float64; q [R][Hq][D] float64.
    Returns (out, lse, tolerance of out, tolerance of lse)."""
    R, Hq, D = q.shape
    out, lse = np.zeros((R, Hq, D)), np.full((R, Hq), -np.inf)
    tol, ltol = np.zeros((R, Hq, D)), np.zeros((R, Hq))
    for b, (K, V) in enumerate(kv):
        n, T = cu[b + 1] - cu[b], lens[b]
        G = Hq // K.shape[1] if T else 1
        for i in range(n):
            see = min(T, max(0, T - n + i + 1))
            r = cu[b] + i
            if see == 0:
                continue
            for hq in range(Hq):
                Kh, Vh, qr = K[:see, hq // G], V[:see, hq // G], q[r, hq]
                s = scale * (Kh @ qr)
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                out[r, hq] = p @ Vh / l
                lse[r, hq] = m + math.log(l)
                ds = scale * (2.0 ** -17 * np.abs(qr).max() * np.abs(Kh).sum(1).max()
                              + 2.0 ** -18 * (np.abs(Kh) @ np.abs(qr)).max())
                A = p @ np.abs(Vh) / l
                flush = 0.0
                for t in range(0, see, P_tile):
                    flush += len(p[t:t + P_tile]) * p[t:t + P_tile].max() * np.abs(Vh[t:t + P_tile]).max()
                tol[r, hq] = bf16_half_ulp(np.abs(out[r, hq])) * 1.001 + (2.0 ** -9 + 2 * ds + 2.0 ** -16) * A \
                    + 2.0 ** -18 * flush / l * 2
                ltol[r, hq] = ds + 2.0 ** -20 * (1 + abs(lse[r, hq]) + np.abs(s).max())
    return out, lse, tol, ltol


# ----------------------------------------------------------------- set-up


class Case:
    """Sequences with `old` tokens of random cache content and `n` query rows; pages lie in
    a random order; everything no sequence holds is NaN (codes 0x7F / 0xFF, NaN scales)."""

    def __init__(self, n, old, heads, group, dim, page, layers=1, layer=0, seed=0, spread=3, qscale=1.5):
        rng = np.random.default_rng(seed)
        self.n, self.H, self.G, self.D, self.P, self.layer = n, heads, group, dim, page, layer
        self.lens = [max(0, o + m) for o, m in zip(old, n)]
        used = [-(-t // page) for t in self.lens]
        pages = sum(used) + 2
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        order = rng.permutation(pages)
        width = max(used + [1]) + 1
        self.table = np.full((len(n), width), -1, dtype=np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        self.cache = moe.KvCache(pages, layers, heads, dim, page)
        self.cache.buffer.copy_(torch.from_numpy(rng.choice([0x7F, 0xFF], pages * self.cache.page_bytes).astype(np.uint8)))
        val = e4m3_values()
        codes = rng.choice([0x7F, 0xFF], (pages, 2, heads, page, dim)).astype(np.uint8)
        scales = np.full((pages, 2, heads), np.nan, dtype=np.float32)
        self.kv = []
        for b, T in enumerate(self.lens):
            for c in range(used[b]):
                m = min(page, T - c * page)
                x = round_e4m3(rng.standard_normal((2, heads, m, dim)) * 60)
                codes[self.table[b, c], :, :, :m] = self.encode(x)
                scales[self.table[b, c]] = 2.0 ** rng.integers(-7, -7 + spread, (2, heads))
            if T:
                ids = self.table[b, :used[b]]
                full = val[codes[ids]] * scales[ids].astype(np.float64)[..., None, None]
                full = full.transpose(1, 0, 3, 2, 4).reshape(2, -1, heads, dim)[:, :T]
                self.kv.append((full[0], full[1]))
            else:
                self.kv.append((np.zeros((0, heads, dim)), np.zeros((0, heads, dim))))
        self.codes_np, self.scales_np = codes, scales
        self.upload()
        R = int(self.cu[-1])
        self.q = torch.from_numpy(rng.standard_normal((R, heads * group, dim)) * qscale).to(torch.bfloat16).cuda()

    @staticmethod
    def encode(x):
        return torch.from_numpy(x).to(FP8).view(torch.uint8).numpy()

    def upload(self):
        self.cache.codes(self.layer).view(torch.uint8).copy_(torch.from_numpy(self.codes_np))
        self.cache.scales(self.layer).copy_(torch.from_numpy(self.scales_np))

    def dev(self, a):
        return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()

    def run(self, **kw):
        R, Hq = self.q.shape[:2]
        lse = torch.full((R, Hq), 7.0, device="cuda")
        ws = moe.workspace(moe.moe_kv_attention_workspace_size(self.cache, max(self.n), Hq))
        out = moe.moe_kv_attention(self.cache, self.layer, kw.pop("q", self.q), self.dev(self.cu), self.dev(self.lens),
                                   self.dev(self.table), max_rows=max(self.n), lse=lse, ws=ws, **kw)
        assert moe.moe_check_status(ws) == moe.MOE_OK
        return out, lse

    def check(self, scale=None, **kw):
        scale = self.D ** -0.5 if scale is None else scale
        out, lse = self.run(scale=scale, **kw)
        ref, rl, tol, ltol = ref_attention(self.kv, self.q.double().cpu().numpy(), self.cu, self.lens, scale)
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(gl), np.isneginf(rl))
        live = ~np.isneginf(rl)
        assert np.isfinite(got).all()
        worst = (np.abs(got - ref) - tol).max() if got.size else 0.0
        assert worst <= 0, f"output off by {worst:.3e} beyond its tolerance"
        assert (np.abs(gl[live] - rl[live]) <= ltol[live]).all()
        return out, lse


# -------------------------------------------------------------- attention

SHAPES = [
    # n, old, heads, group, dim, page
    ([1], [0], 1, 1, 128, 16),
    ([1], [0], 2, 7, 64, 64),
    ([1], [127], 2, 8, 128, 128),
    ([1], [128], 1, 16, 64, 32),
    ([1, 1, 1], [5, 300, 1000], 8, 7, 128, 64),
    ([1] * 40, list(range(0, 400, 10)), 2, 4, 128, 16),
    ([5, 5], [123, 124], 2, 7, 128, 32),            # the drafts straddle a tile's end
    ([2, 9, 17], [700, 63, 0], 4, 7, 128, 64),
    ([17, 17], [250, 1], 1, 8, 128, 128),            # 136 rows: two row tiles
    ([9, 1, 4], [40, 511, 0], 3, 5, 64, 16),
    ([3, 0, 2], [9, 77, 500], 2, 3, 64, 16),         # a sequence without rows
    ([1], [4000], 2, 7, 128, 64),                    # one sequence over many CTAs
    ([40], [100], 1, 7, 128, 16),                    # 280 rows: a short prompt over a cached prefix
    ([300], [0], 2, 2, 64, 32),                      # a whole prompt, causal
    ([2], [1500], 1, 64, 128, 64),                   # one key/value head for 64 query heads
    ([33], [7], 1, 1, 128, 32),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_attention_against_64_bits(shape):
    Case(*shape, seed=len(shape[0]) + shape[4]).check()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("group", [1, 3, 10, 20])
def test_attention_pages_and_groups(dim, page, group):
    """Every page size and head width with 16 to 128-row tiles (4 rows of 1..20 heads)."""
    Case([4, 1, 3], [page - 2, 3 * page, 257], 2, group, dim, page, layers=3, layer=1, seed=page + group).check()


@pytest.mark.parametrize("rows,dim,group", [(1, 128, 3), (2, 64, 8), (5, 128, 7)])
def test_attention_many_short_sequences(rows, dim, group):
    """Thousands of units of one to three tiles: every part of the device walks through several."""
    r = np.random.default_rng(rows)
    n = [int(x) for x in r.integers(0, rows + 1, 700)]
    Case(n, [int(x) for x in r.integers(0, 300, 700)], 4, group, dim, 32, seed=dim).check()


def test_attention_rows_that_see_nothing():
    """Fewer tokens than rows: the first rows stand before token 0; no tokens at all."""
    c = Case([5, 3, 2], [-3, -3, -1], 2, 7, 128, 16)
    assert c.lens == [2, 0, 1]
    out, lse = c.check()
    assert (out[:3] == 0).all() and torch.isneginf(lse[:3]).all()
    assert (out[5:8] == 0).all() and (out[8:9] == 0).all() and (out[9] != 0).any()


@pytest.mark.parametrize("old,group", [(20, 7), (126, 7), (1000, 3)])
@pytest.mark.parametrize("what", ["nan_v", "nan_k", "nan_both", "inf_scale"])
def test_attention_masked_tokens_do_not_reach(old, group, what):
    """NaN keys, values and scales of drafts that a row does not see leave it untouched;
    rows that see them show it."""
    n = 5
    c = Case([n, 2], [old, 9], 2, group, 128, 16, seed=5)
    clean, _ = c.check()
    bad = old + 2  # token of row 2: rows 0 and 1 do not see it
    page, slot = c.table[0, bad // 16], bad % 16
    if what in ("nan_k", "nan_both"):
        c.codes_np[page, 0, 0, slot, 3] = 0x7F
    if what in ("nan_v", "nan_both"):
        c.codes_np[page, 1, 0, slot, 5] = 0xFF
    if what == "inf_scale":
        if slot > 0:
            pytest.skip("the page's scale belongs to visible tokens too")
        c.scales_np[page, 1, 0] = np.inf
    c.upload()
    out, _ = c.run()
    G = c.G
    assert torch.equal(out[:2], clean[:2]) and torch.equal(out[n:], clean[n:])
    assert torch.equal(out[:n, G:], clean[:n, G:])          # the other head
    seen = out[2:n, :G].float()
    if what == "nan_v":
        assert torch.isnan(seen[..., 5]).all() and not torch.isnan(seen[..., 6:]).any()
    else:
        assert torch.isnan(seen).any()


@pytest.mark.parametrize("n,old", [(1, 0), (1, 300), (9, 0), (9, 300)])
def test_attention_shows_nan_that_a_row_sees(n, old):
    """A NaN key is in every row that sees it, even where it is all the row sees."""
    c = Case([n], [old], 1, 7, 128, 16, seed=old + n)
    at = old                                              # the first row's own token
    c.codes_np[c.table[0, at // 16], 0, 0, at % 16, 7] = 0x7F
    c.upload()
    out, lse = c.run()
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("n", [1, 9])
def test_attention_wait_that_runs_out_is_reported(n):
    """With a wait limit far below a kernel's start, every role gives up, drains what it has in
    flight and reports; the same workspace then serves the next call."""
    c = Case([n] * 40, [400 * i for i in range(40)], 2, 7, 128, 64, seed=n)
    ws = moe.workspace(moe.moe_kv_attention_workspace_size(c.cache, n, 14))
    call = lambda: moe.moe_kv_attention(c.cache, 0, c.q, c.dev(c.cu), c.dev(c.lens), c.dev(c.table),  # noqa: E731
                                        max_rows=n, ws=ws)
    want = call()
    assert moe.moe_check_status(ws) == moe.MOE_OK
    moe.moe_debug_set_wait_limit(200)  # ns
    try:
        call()
        got = moe.moe_check_status(ws)
    finally:
        moe.moe_debug_set_wait_limit(0)
    assert got == moe.MOE_ERR_TIMEOUT
    moe.moe_clear_status(ws)
    assert torch.equal(call().view(torch.int16), want.view(torch.int16))
    assert moe.moe_check_status(ws) == moe.MOE_OK


def test_attention_wide_range_of_weights():
    """One token far above the rest, and a long tail of tiny weights that together matter."""
    c = Case([1], [3000], 1, 4, 128, 64, seed=11)
    q = np.zeros((1, 4, 128))
    q[..., 0] = 16.0
    c.q = torch.from_numpy(q).to(torch.bfloat16).cuda()
    c.codes_np[c.table[0, 0], 0, 0, 0, 0] = 0x7E   # 448
    c.scales_np[:, 0] = np.where(np.isnan(c.scales_np[:, 0]), np.nan, 2.0 ** -6)
    val = e4m3_values()
    used = c.table[0][c.table[0] >= 0]
    full = val[c.codes_np[used]] * c.scales_np[used].astype(np.float64)[..., None, None]
    full = full.transpose(1, 0, 3, 2, 4).reshape(2, -1, 1, 128)[:, :c.lens[0]]
    c.kv = [(full[0], full[1])]
    c.upload()
    c.check()


def test_attention_scale_and_extremes():
    for scale, qscale in ((1e-3, 1.0), (3.0, 4.0), (0.25, 1e-20), (0.1, 0.0)):
        Case([3], [200], 2, 2, 64, 32, seed=3, qscale=qscale).check(scale=scale)


def test_attention_strides_and_streams():
    """q as a slice of one projection's output, out with a wider row, another stream."""
    c = Case([5, 2], [300, 10], 2, 7, 128, 32, seed=7)
    want, _ = c.check()
    R, Hq, D = c.q.shape
    wide = torch.randn(R, Hq + 4, D, device="cuda").to(torch.bfloat16)
    wide[:, :Hq] = c.q
    out = torch.full((R, Hq + 2, D), 5.0, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = moe.moe_kv_attention(c.cache, 0, wide[:, :Hq], c.dev(c.cu), c.dev(c.lens), c.dev(c.table), max_rows=5,
                               out=out[:, :Hq], stream=st)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and (out[:, Hq:] == 5.0).all()
    side = moe.moe_kv_attention(c.cache, 0, c.q, c.dev(c.cu), c.dev(c.lens), c.dev(c.table), max_rows=9, stream=st)
    st.synchronize()
    assert side.shape == want.shape


def test_attention_is_deterministic_and_captures():
    c = Case([1, 1, 1], [6000, 2500, 37], 4, 7, 128, 64, seed=9)
    a, la = c.run()
    for _ in range(5):
        b, lb = c.run()
        assert torch.equal(a, b) and torch.equal(la, lb)
    args = (c.dev(c.cu), c.dev(c.lens), c.dev(c.table))
    ws = moe.workspace(moe.moe_kv_attention_workspace_size(c.cache, 1, 28))
    out = torch.empty_like(c.q)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for _ in range(3):
            moe.moe_kv_attention(c.cache, 0, c.q, *args, max_rows=1, out=out, ws=ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a)
    # the lengths are read on the device: the same graph serves other lengths
    args[1].copy_(c.dev([50, 2501, 0]))
    g.replay()
    torch.cuda.synchronize()
    c.lens = [50, 2501, 0]
    c.kv = [(k[:t], v[:t]) for (k, v), t in zip(c.kv, c.lens)]
    ref, _, tol, _ = ref_attention(c.kv, c.q.double().cpu().numpy(), c.cu, c.lens, 128 ** -0.5)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()


def test_attention_page_offsets_beyond_32_bits():
    """A cache of more than 4 GiB whose sequence lies in its last pages."""
    n_pages = 45000
    cache = moe.KvCache(n_pages, 1, 8, 128, 64)
    assert cache.page_bytes * n_pages > 5 << 30
    c = Case([2], [200], 8, 2, 128, 64, seed=13)
    used = int((c.table[0] >= 0).sum())
    table = np.full_like(c.table, -1)
    for j in range(used):
        table[0, j] = n_pages - 1 - j
        cache.codes(0)[n_pages - 1 - j].view(torch.uint8).copy_(torch.from_numpy(c.codes_np[c.table[0, j]]))
        cache.scales(0)[n_pages - 1 - j].copy_(torch.from_numpy(c.scales_np[c.table[0, j]]))
    c.cache, c.table = cache, table
    c.check()


def test_attention_reports_bad_pages_and_lengths():
    c = Case([2, 2], [100, 100], 2, 7, 128, 32)
    good, _ = c.run()
    ws = moe.workspace(moe.moe_kv_attention_workspace_size(c.cache, 4, 14))

    def call(table=None, lens=None, cu=None, max_rows=2):
        out = torch.full_like(c.q, 9.0)
        moe.moe_kv_attention(c.cache, 0, c.q, c.dev(c.cu if cu is None else cu), c.dev(c.lens if lens is None else lens),
                             c.dev(c.table if table is None else table), max_rows=max_rows, out=out, ws=ws)
        return out, moe.moe_check_status(ws)

    for page in (-1, c.cache.n_pages, 2 ** 31 - 1, -2 ** 31):
        t = c.table.copy()
        t[0, 1] = page
        out, st = call(table=t)
        assert st == moe.MOE_ERR_BAD_PAGE
        assert torch.equal(out[2:], good[2:])                # the other sequence is right
    out, st = call(lens=[102, 2 ** 31 - 1])
    assert st == moe.MOE_ERR_BAD_PAGE and torch.equal(out[:2], good[:2])
    out, st = call(lens=[102, -5])
    assert st == moe.MOE_OK and torch.equal(out[:2], good[:2]) and (out[2:] == 0).all()
    for cu in ([0, 3, 2], [0, 2, 5], [-1, 2, 4], [0, 2, 2 ** 31 - 1]):
        _, st = call(cu=cu, max_rows=4)
        assert st == moe.MOE_ERR_BAD_PAGE
    out, st = call(max_rows=1)
    assert st == moe.MOE_ERR_BAD_PAGE
    out, st = call()
    assert st == moe.MOE_OK and torch.equal(out, good)       # the workspace is usable again


def test_writes_stay_inside():
    g = Guarded()
    c = Case([1, 5, 2], [700, 0, 63], 2, 7, 128, 16, seed=21)
    R, Hq, D = c.q.shape
    buf = g.tensor((c.cache.n_pages * c.cache.page_bytes,), torch.uint8)
    buf.copy_(c.cache.buffer)
    cache = moe.KvCache(c.cache.n_pages, 1, 2, 128, 16, buffer=buf)
    out = g.tensor((R, Hq, D), torch.bfloat16, zero=False)
    lse = g.tensor((R, Hq), torch.float32, zero=False)
    ws = g.workspace(moe.moe_kv_attention_workspace_size(cache, 5, Hq))
    want, _ = c.check()
    for _ in range(2):
        moe.moe_kv_attention(cache, 0, c.q, c.dev(c.cu), c.dev(c.lens), c.dev(c.table), max_rows=5, out=out, lse=lse, ws=ws)
        assert moe.moe_check_status(ws) == moe.MOE_OK
        assert torch.equal(out, want)
    g.check("moe_kv_attention")
    before = buf.clone()
    kv = torch.randn(R, 2, D, device="cuda").to(torch.bfloat16)
    ws = g.workspace(moe.moe_kv_append_workspace_size())
    start = [t - m for t, m in zip(c.lens, c.n)]
    moe.moe_kv_append(cache, 0, kv, kv, c.dev(c.cu), c.dev(start), c.dev(c.table), ws=ws)
    assert moe.moe_check_status(ws) == moe.MOE_OK
    g.check("moe_kv_append")
    same = (buf == before).view(c.cache.n_pages, -1)
    untouched = sorted(set(range(c.cache.n_pages)) - {int(c.table[b, t // 16]) for b in range(3)
                                                       for t in range(start[b], c.lens[b])})
    assert bool(same[untouched].all())


# ----------------------------------------------------------------- append


def _append_case(n, start, heads, dim, page, seed, special=False, layers=2, layer=1):
    rng = np.random.default_rng(seed)
    used = [-(-(s + m) // page) for s, m in zip(start, n)]
    pages = sum(used) + 2
    order = rng.permutation(pages)
    table = np.full((len(n), max(used + [1])), -1, dtype=np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    cache = moe.KvCache(pages, layers, heads, dim, page)
    cache.buffer.fill_(0x31)
    codes = round_e4m3(rng.standard_normal((pages, 2, heads, page, dim)) * 50)
    scales = 2.0 ** rng.integers(-9, -2, (pages, 2, heads)).astype(np.float64)
    cache.codes(layer).view(torch.uint8).copy_(torch.from_numpy(Case.encode(codes)))
    cache.scales(layer).copy_(torch.from_numpy(scales))
    R = sum(n)
    x = [rng.standard_normal((R, heads, dim)) * 2.0 ** rng.integers(-4, 6, (R, heads, 1)) for _ in range(2)]
    if special and R:
        x[0][0, 0, :4] = [np.inf, -np.inf, np.nan, 3e38]
        x[1][R // 2] = 0.0
        x[1][-1, -1] = 1e-39
    k, v = (torch.from_numpy(a).to(torch.bfloat16).cuda() for a in x)
    return cache, codes, scales, table, k, v


@pytest.mark.parametrize("n,start,heads,dim,page", [
    ([1], [0], 1, 64, 16), ([1], [15], 2, 128, 16), ([1], [16], 2, 128, 16), ([1, 1, 1], [3, 31, 64], 8, 128, 32),
    ([5, 17, 2], [14, 120, 0], 2, 128, 16), ([9, 0, 1], [60, 7, 127], 3, 64, 64), ([300, 129], [0, 77], 2, 128, 128),
    ([1] * 200, list(range(200)), 1, 64, 64), ([1000], [1], 1, 128, 64)])
@pytest.mark.parametrize("special", [False, True])
def test_append_exactly(n, start, heads, dim, page, special):
    cache, codes, scales, table, k, v = _append_case(n, start, heads, dim, page, seed=sum(n) + page, special=special)
    other = cache.codes(0).view(torch.uint8).clone()
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    ws = moe.workspace(moe.moe_kv_append_workspace_size())
    moe.moe_kv_append(cache, 1, k, v, dev(cu), dev(start), dev(table), ws=ws)
    assert moe.moe_check_status(ws) == moe.MOE_OK
    ref_append(codes, scales, k.double().cpu().numpy(), v.double().cpu().numpy(), cu, start, table, page)
    assert np.array_equal(cache.scales(1).double().cpu().numpy(), scales)
    got = cache.codes(1).double().cpu().numpy()
    assert np.array_equal(got, codes, equal_nan=True)
    assert torch.equal(cache.codes(0).view(torch.uint8), other)   # the other layer is untouched
    # again, from the same start: nothing changes
    moe.moe_kv_append(cache, 1, k, v, dev(cu), dev(start), dev(table), ws=ws)
    assert np.array_equal(cache.codes(1).double().cpu().numpy(), codes, equal_nan=True)


def test_append_token_by_token_then_truncate():
    """Growing scales, then fewer tokens (rejected drafts) overwritten by others."""
    heads, dim, page = 2, 64, 16
    cache, codes, scales, table, k, v = _append_case([40], [0], heads, dim, page, seed=3)
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    kn, vn = k.double().cpu().numpy(), v.double().cpu().numpy()
    steps = [(t, 1, t) for t in range(20)] + [(17, 9, 20), (19, 3, 29), (22, 8, 32)]
    for start, m, at in steps:
        moe.moe_kv_append(cache, 1, k[at:at + m], v[at:at + m], dev([0, m]), dev([start]), dev(table))
        ref_append(codes, scales, kn[at:at + m], vn[at:at + m], [0, m], [start], table, page)
    assert np.array_equal(cache.scales(1).double().cpu().numpy(), scales)
    assert np.array_equal(cache.codes(1).double().cpu().numpy(), codes)


def test_append_keeps_a_scale_that_is_no_power_of_two():
    cache, codes, scales, table, k, v = _append_case([2], [5], 1, 64, 16, seed=4)
    s = np.float32(3.3)
    scales[table[0, 0]] = s
    cache.scales(1)[int(table[0, 0])] = float(s)
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    k, v = k * 0.01, v * 0.01
    moe.moe_kv_append(cache, 1, k, v, dev([0, 2]), dev([5]), dev(table))
    page = int(table[0, 0])
    for side, x in enumerate((k, v)):
        want = round_e4m3((x.float() / float(s)).double().cpu().numpy())  # the fp32 quotient, rounded
        got = cache.codes(1)[page, side, :, 5:7].double().cpu().numpy().transpose(1, 0, 2)
        assert np.array_equal(got, want)
        assert np.array_equal(cache.codes(1)[page, side, :, :5].double().cpu().numpy(), codes[page, side, :, :5])
    assert np.array_equal(cache.scales(1).double().cpu().numpy(), scales)


def test_append_strided_rows_and_bad_places():
    cache, codes, scales, table, k, v = _append_case([4, 4], [10, 30], 2, 128, 16, seed=8)
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    fused = torch.cat([torch.zeros_like(k), k, v], dim=1)          # [rows][6][128]
    cu, start = dev([0, 4, 8]), dev([10, 30])
    ws = moe.workspace(moe.moe_kv_append_workspace_size())
    before = cache.buffer.clone()

    def status(**kw):
        a = dict(cu=cu, start=start, table=dev(table))
        a.update(kw)
        moe.moe_kv_append(cache, 1, fused[:, 2:4], fused[:, 4:], a["cu"], a["start"], a["table"], ws=ws)
        return moe.moe_check_status(ws)

    t = table.copy()
    t[0, 0], t[1, 1:] = -7, cache.n_pages
    assert status(table=dev(t)) == moe.MOE_ERR_BAD_PAGE
    only = [p for p in range(cache.n_pages) if p not in (t[1, 1:3].tolist() + [int(table[0, 0])])]
    assert status(start=dev([-1, 2 ** 31 - 1])) == moe.MOE_ERR_BAD_PAGE
    assert status(cu=dev([0, 9, 8])) == moe.MOE_ERR_BAD_PAGE
    assert status(cu=dev([-3, -2, -1])) == moe.MOE_ERR_BAD_PAGE
    cache.buffer.copy_(before)
    assert len(only) > 0 and status() == moe.MOE_OK
    ref_append(codes, scales, k.double().cpu().numpy(), v.double().cpu().numpy(), [0, 4, 8], [10, 30], table, 16)
    assert np.array_equal(cache.codes(1).double().cpu().numpy(), codes)
    assert np.array_equal(cache.scales(1).double().cpu().numpy(), scales)


def test_append_then_attend():
    """The two together, token by token, against attention over the unquantised rows."""
    rng = np.random.default_rng(17)
    heads, group, dim, page, T = 2, 7, 128, 16, 70
    cache = moe.KvCache(8, 1, heads, dim, page)
    cache.buffer.fill_(0x7F)
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    table = dev([[5, 2, 7, 0, 1]])
    k, v = (torch.from_numpy(rng.standard_normal((T, heads, dim))).to(torch.bfloat16).cuda() for _ in range(2))
    t = 0
    for m in (1, 1, 5, 17, 1, 9, 36):
        moe.moe_kv_append(cache, 0, k[t:t + m], v[t:t + m], dev([0, m]), dev([t]), table)
        t += m
    q = torch.from_numpy(rng.standard_normal((3, heads * group, dim))).to(torch.bfloat16).cuda()
    out = moe.moe_kv_attention(cache, 0, q, dev([0, 3]), dev([t]), table, max_rows=3).double().cpu().numpy()
    kv = [(k.double().cpu().numpy(), v.double().cpu().numpy())]
    ref, _, tol, _ = ref_attention(kv, q.double().cpu().numpy(), [0, 3], [T], dim ** -0.5)
    # E4M3 keeps 4 significant bits: 2^-4 of each value, so a few percent of the output
    assert np.linalg.norm(out - ref) / np.linalg.norm(ref) < 2.0 ** -4


def test_empty_calls():
    cache = moe.KvCache(2, 1, 2, 64, 16)
    e = lambda *s, **k: torch.empty(s, device="cuda", **k)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    kv = e(0, 2, 64, dtype=torch.bfloat16)
    moe.moe_kv_append(cache, 0, kv, kv, i(1), i(0), i(0, 4))
    moe.moe_kv_append(cache, 0, kv, kv, i(4), i(3), i(3, 4))
    q = e(0, 4, 64, dtype=torch.bfloat16)
    assert moe.moe_kv_attention(cache, 0, q, i(4), i(3), i(3, 4), max_rows=0).shape == (0, 4, 64)
    assert moe.moe_kv_attention(cache, 0, q, i(1), i(0), i(0, 4), max_rows=0).shape == (0, 4, 64)
    # rows whose sequence has no tokens and no table
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    assert (moe.moe_kv_attention(cache, 0, q, cu, i(1), i(1, 0), max_rows=2) == 0).all()
    torch.cuda.synchronize()
