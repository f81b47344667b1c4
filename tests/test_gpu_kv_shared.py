"""GPU: attention of sequences that share prefixes, against plain attention of each sequence over all of
its own tokens in 64 bits.

The tolerance is that of the cache attention (bf16 output, 8-bit weights and queries, fp32 sums; derived
in the tests of that), where tiles of 128 tokens begin at token 0 and, anew, at the end of the prefix.
Adding the two parts takes an exponential, a product and a sum in fp32 for each: 2^-20 of the weights'
sum, which its 2^-16 for fp32 sums and scalings hold, too."""
import numpy as np
import pytest
import torch

from tests._util import bf16_half_ulp
from tests.test_gpu_guard_bands import Guarded
from tests.test_gpu_kv import Case, e4m3_values

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("mxfp4_routed_expert_topk_gb300")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()


class Shared(Case):
    """Sequences in groups: members[g] of them share the first prefix[g] tokens.  The other members' own
    entries for the shared pages name no page.  Tables with room for many tokens make the call run twice
    (prefixes, then own tokens), others once."""

    twice = False

    def __init__(self, members, prefix, n, own, heads, group, dim, page, **kw):
        old, at = [], 0
        for m, p in zip(members, prefix):
            old += [p + o for o in own[at:at + m]]
            at += m
        super().__init__(n, old, heads, group, dim, page, **kw)
        self.groups = [0]
        self.prefix = list(prefix)
        self.whole = []
        for m, p in zip(members, prefix):
            b0 = self.groups[-1]
            w = p // page
            lead = next((b for b in range(b0, b0 + m) if n[b]), b0)  # whose row of the table names the pages
            for b in range(b0, b0 + m):
                if b == lead:
                    continue
                self.table[b, :w] = -1
                if self.kv[b][0].shape[0]:
                    self.kv[b] = tuple(np.concatenate([self.kv[lead][i][:w * page], self.kv[b][i][w * page:]]) for i in (0, 1))
            self.groups.append(b0 + m)
            self.whole += [w * page] * m
        if self.twice:
            tiles = 33 * torch.cuda.get_device_properties(0).multi_processor_count // (len(n) * heads) + 1
            room = np.full((len(n), -(-128 * tiles // page)), -1, dtype=np.int32)
            room[:, :self.table.shape[1]] = self.table[:, :room.shape[1]]
            self.table = room if room.shape[1] > self.table.shape[1] else self.table
        self.max_rows = max(n)
        self.max_group_rows = max(1, max(sum(n[a:b]) for a, b in zip(self.groups, self.groups[1:])))

    def workspace(self):
        R, Hq = self.q.shape[:2]
        return moe.moe_kv_attention_shared_workspace_size(self.cache, R, self.max_rows, self.max_group_rows, Hq)

    def run(self, ws=None, **kw):
        R, Hq = self.q.shape[:2]
        lse = torch.full((R, Hq), 7.0, device="cuda")
        ws = moe.workspace(self.workspace()) if ws is None else ws
        out = moe.moe_kv_attention_shared(self.cache, self.layer, kw.pop("q", self.q), self.dev(self.cu), self.dev(self.lens),
                                          self.dev(self.table), self.dev(self.groups), self.dev(self.prefix),
                                          max_rows=self.max_rows, max_group_rows=self.max_group_rows, lse=lse, ws=ws, **kw)
        assert moe.moe_check_status(ws) == moe.MOE_OK
        return out, lse

    def check(self, scale=None, **kw):
        scale = self.D ** -0.5 if scale is None else scale
        out, lse = self.run(scale=scale, **kw)
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        q = self.q.double().cpu().numpy()
        for b, (K, V) in enumerate(self.kv):
            T, n, w = self.lens[b], self.n[b], self.whole[b]
            for i in range(n):
                r, see = self.cu[b] + i, T - n + i + 1
                Kv, Vv = K[:see], V[:see]                      # [t][H][D]
                qr = q[r].reshape(self.H, self.G, self.D)
                s = scale * np.einsum("hgd,thd->hgt", qr, Kv)
                m = s.max(-1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(-1)
                o = np.einsum("hgt,thd->hgd", p, Vv) / l[..., None]
                A = np.einsum("hgt,thd->hgd", p, np.abs(Vv)) / l[..., None]
                ds = scale * (2.0 ** -17 * np.abs(qr).max(-1) * np.abs(Kv).sum(-1).max(0)[:, None]
                              + 2.0 ** -18 * np.einsum("hgd,thd->hgt", np.abs(qr), np.abs(Kv)).max(-1))
                flush = 0.0
                cuts = sorted(set(range(0, w, 128)) | set(range(w, see, 128)) | {see})
                for t0, t1 in zip(cuts, cuts[1:]):
                    flush = flush + (t1 - t0) * p[..., t0:t1].max(-1) * np.abs(Vv[t0:t1]).max((0, 2))[:, None]
                tol = bf16_half_ulp(np.abs(o)) * 1.001 + (2.0 ** -9 + 2 * ds + 2.0 ** -16)[..., None] * A \
                    + (2.0 ** -18 * flush / l * 2)[..., None]
                worst = (np.abs(got[r].reshape(o.shape) - o) - tol).max()
                assert worst <= 0, f"row {i} of sequence {b} off by {worst:.3e} beyond its tolerance"
                want = m[..., 0] + np.log(l)
                assert (np.abs(gl[r].reshape(want.shape) - want) <= ds + 2.0 ** -20 * (1 + np.abs(want) + np.abs(s).max(-1))).all()
        return out, lse


@pytest.fixture(autouse=True, params=[False, True], ids=["once", "twice"])
def _ways(request):
    Shared.twice = request.param
    yield
    Shared.twice = False


SHAPES = [
    # members, prefix, n, tokens of its own before the new rows, heads, group, dim, page
    ([1], [0], [1], [0], 1, 1, 128, 16),
    ([1], [16], [1], [0], 1, 1, 128, 16),
    ([2], [16], [1, 1], [0, 0], 2, 7, 64, 16),
    ([4], [500], [1] * 4, [3, 60, 0, 11], 8, 7, 128, 64),            # the prefix ends inside a page
    ([3], [15], [1, 2, 1], [5, 0, 300], 2, 4, 128, 16),              # ... of which it fills none
    ([20], [1000], [1] * 20, list(range(0, 400, 20)), 2, 7, 128, 32),
    ([5], [384], [5, 3, 1, 5, 2], [0, 130, 17, 1, 60], 4, 7, 128, 64),
    ([3], [777], [17, 9, 17], [250, 1, 0], 1, 8, 128, 128),
    ([1, 4, 1, 3], [100, 300, 0, 64], [1, 1, 2, 1, 1, 3, 1, 1, 1], [5, 0, 9, 44, 3, 70, 0, 1, 2], 2, 5, 64, 16),
    ([1, 1, 1], [0, 0, 0], [1, 3, 1], [200, 0, 5], 2, 3, 64, 32),    # nothing is shared
    ([4, 3], [256, 128], [1, 0, 2, 0, 0, 1, 0], [3, 0, 4, 9, 1, 0, 2], 2, 7, 128, 16),   # sequences without rows
    ([6, 2], [64, 32], [0, 0, 0, 1, 0, 2, 0, 1], [3, 0, 4, 9, 1, 0, 2, 5], 2, 3, 64, 16),  # the first ones have ended
    ([0, 3, 0, 0, 2, 0], [64, 128, 0, 9, 40, 5], [1, 1, 1, 1, 1], [5, 6, 7, 8, 9], 1, 7, 128, 16),  # empty groups
    ([70], [256], [1] * 70, [2] * 70, 1, 2, 128, 64),
    ([2], [6000], [1, 1], [10, 200], 2, 7, 128, 64),                 # a long prefix over many CTAs
    ([2], [130], [40, 33], [1, 0], 1, 7, 128, 16),
    ([6], [2000], [2] * 6, [1] * 6, 1, 64, 64, 64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_against_64_bits(shape):
    Shared(*shape, seed=len(shape[2]) + shape[4]).check()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("group", [1, 3, 8])
@pytest.mark.parametrize("rows", [1, 3, 7])
def test_pages_groups_and_rows(dim, page, group, rows):
    """Every page size and head width with prefix tiles of 16 to 128 rows and more."""
    n = [rows, 1, rows, rows, 1, rows]
    Shared([4, 2], [3 * page + 5, 200], n, [0, page, 2, 140, 9, 1], 2, group, dim, page, layers=3, layer=1,
           seed=page + group + rows).check()


def test_many_groups():
    """Hundreds of groups of one to four sequences, most with a prefix of their own."""
    r = np.random.default_rng(5)
    members = [int(x) for x in r.integers(1, 5, 150)]
    prefix = [int(x) for x in r.choice([0, 16, 33, 130, 400], 150)]
    S = sum(members)
    Shared(members, prefix, [int(x) for x in r.integers(0, 3, S)], [int(x) for x in r.integers(0, 40, S)], 2, 3, 64, 16,
           seed=7).check()


def test_equals_the_attention_of_each_sequence():
    """The same call without sharing, over tables that name the shared pages for everyone."""
    c = Shared([6, 2], [700, 128], [1, 2, 1, 1, 3, 1, 1, 1], [9, 0, 5, 100, 2, 3, 4, 5], 4, 7, 128, 64, seed=2)
    out, lse = c.check()
    table = c.table.copy()
    for g, p in enumerate(c.prefix):
        table[c.groups[g]:c.groups[g + 1], :p // 64] = c.table[c.groups[g], :p // 64]
    ref = moe.moe_kv_attention(c.cache, 0, c.q, c.dev(c.cu), c.dev(c.lens), c.dev(table), max_rows=3)
    # each is within half a bf16 step and the weights' 2^-9 of the same value
    assert ((out.float() - ref.float()).abs() <= 2.0 ** -7 * ref.float().abs() + 2.0 ** -7 * ref.float().abs().max()).all()


@pytest.mark.parametrize("what", ["k", "v"])
def test_nan_reaches_only_those_that_see_it(what):
    c = Shared([4], [130], [1, 2, 1, 3], [20, 3, 40, 5], 2, 7, 128, 16, seed=3)
    clean, _ = c.check()
    side, G = 0 if what == "k" else 1, c.G
    at = c.lens[1] - 1                                          # the second row of sequence 1 alone
    c.codes_np[c.table[1, at // 16], side, 0, at % 16, 5] = 0x7F
    c.upload()
    out, lse = c.run()
    assert torch.equal(out[:2], clean[:2]) and torch.equal(out[3:], clean[3:]) and torch.equal(out[2, G:], clean[2, G:])
    assert torch.isnan(out[2, :G, 5]).all()
    c.codes_np[c.table[0, 2], side, 1, 3, 5] = 0xFF              # everybody
    c.upload()
    out, lse = c.run()
    assert torch.isnan(out[:, G:, 5]).all() and torch.equal(out[:2, :G], clean[:2, :G])


def test_prefix_far_above_or_below_the_rest():
    """One part of the sum all but vanishes beside the other, either way."""
    for big in (0, 1):
        c = Shared([3], [256], [1, 1, 2], [30, 1, 200], 2, 4, 128, 64, seed=9)
        for b in range(3):
            own = c.table[b, 4:][c.table[b, 4:] >= 0]
            ids = c.table[0, :4] if big else own
            c.scales_np[ids, 0] = 2.0 ** -1
        c.upload()
        for b in range(3):
            K = c.kv[b][0]
            part = slice(0, 256) if big else slice(256, None)
            pages = c.table[0, :4] if big else c.table[b, 4:][c.table[b, 4:] >= 0]
            full = e4m3_values()[c.codes_np[pages, 0]] * c.scales_np[pages, 0].astype(np.float64)[..., None, None]
            full = full.transpose(0, 2, 1, 3).reshape(-1, c.H, c.D)
            K[part] = full[:len(K[part])]
        c.check()


def test_strides_streams_and_untouched_rows():
    c = Shared([3], [300], [2, 1, 4], [3, 60, 11], 2, 7, 128, 32, seed=4)
    want, _ = c.check()
    R, Hq, D = c.q.shape
    wide = torch.full((R + 5, Hq + 4, D), 3.0, device="cuda").to(torch.bfloat16)
    wide[2:R + 2, :Hq] = c.q
    out = torch.full((R + 5, Hq + 2, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((R + 5, Hq), 6.0, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = moe.moe_kv_attention_shared(c.cache, 0, wide[:, :Hq], c.dev(c.cu + 2), c.dev(c.lens), c.dev(c.table), c.dev(c.groups),
                                      c.dev(c.prefix), max_rows=c.max_rows, max_group_rows=c.max_group_rows,
                                      out=out[:, :Hq], lse=lse, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(got[2:R + 2], want) and (out[:, Hq:] == 5).all()
    assert (out[:2] == 5).all() and (out[R + 2:] == 5).all() and (lse[:2] == 6).all() and (lse[R + 2:] == 6).all()
    c.max_rows, c.max_group_rows = 9, 40  # room for more rows than there are: other tiles
    c.check()


def test_deterministic_and_captured():
    c = Shared([5, 1], [4000, 50], [1, 1, 2, 1, 1, 1], [30, 1, 200, 9, 700, 3], 4, 7, 128, 64, seed=6)
    a, la = c.check()
    ws = moe.workspace(c.workspace())
    for _ in range(4):
        b, lb = c.run(ws=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)
    cu, lens, table, groups, prefix = (c.dev(t) for t in (c.cu, c.lens, c.table, c.groups, c.prefix))
    out = torch.empty_like(c.q)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for _ in range(2):
            moe.moe_kv_attention_shared(c.cache, 0, c.q, cu, lens, table, groups, prefix, max_rows=2, max_group_rows=6,
                                        out=out, ws=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a)
    # lengths are read on the device: a shorter prefix (the rest of it is then the first sequence's alone)
    full = c.table.copy()
    full[:5, :4000 // 64] = c.table[0, :4000 // 64]
    table.copy_(c.dev(full))
    prefix.copy_(c.dev([130, 0]))
    g.replay()
    torch.cuda.synchronize()
    err = (out.float() - a.float()).abs()
    assert (err <= 2.0 ** -7 * a.float().abs() + 2.0 ** -7 * a.float().abs().max()).all()


def test_reports_what_it_cannot_do():
    c = Shared([2, 2], [128, 64], [1, 2, 1, 1], [9, 0, 5, 1], 2, 7, 128, 32, seed=8)
    good, _ = c.check()
    ws = moe.workspace(c.workspace())

    def call(cu=None, lens=None, groups=None, prefix=None, table=None, max_rows=2, max_group_rows=3):
        out = torch.full_like(c.q, 9.0)
        pick = lambda a, b: c.dev(b if a is None else a)  # noqa: E731
        moe.moe_kv_attention_shared(c.cache, 0, c.q, pick(cu, c.cu), pick(lens, c.lens), pick(table, c.table),
                                    pick(groups, c.groups), pick(prefix, c.prefix), max_rows=max_rows,
                                    max_group_rows=max_group_rows, out=out, ws=ws)
        st = moe.moe_check_status(ws)
        moe.moe_clear_status(ws)
        return out, st

    big = 2 ** 31 - 1
    bad = [dict(groups=[0, 2, 3]), dict(groups=[1, 2, 4]), dict(groups=[0, 5, 4]), dict(groups=[0, -1, 4]), dict(groups=[0, 2, big]),
           dict(groups=[3, 2, 4]), dict(groups=[0, 3, 2, 4], prefix=[128, 0, 64]), dict(cu=[0, 1, 3, 4, 6]), dict(cu=[0, 3, 1, 4, 5]), dict(cu=[-1, 1, 3, 4, 5]),
           dict(prefix=[160, 64]), dict(prefix=[big, 64]), dict(lens=[100, 130, 70, 66]), dict(lens=[138, 130, big, 66]),
           dict(max_rows=1), dict(max_group_rows=2)]
    for page in (-1, c.cache.n_pages, big, -2 ** 31):
        t = c.table.copy()
        t[0, 1] = page
        bad.append(dict(table=t))
    for kw in bad:
        out, st = call(**kw)
        assert st == moe.MOE_ERR_BAD_PAGE, kw
    out, st = call(prefix=[-5, 64], table=np.where(c.table < 0, c.table[:1], c.table))
    assert st == moe.MOE_OK
    out, st = call()
    assert st == moe.MOE_OK and torch.equal(out, good)


@pytest.mark.parametrize("n", [1, 9])
def test_wait_that_runs_out_is_reported(n):
    c = Shared([20, 20], [2000, 500], [n] * 40, [10 * i for i in range(40)], 2, 7, 128, 64, seed=n)
    ws = moe.workspace(c.workspace())
    want, _ = c.run(ws=ws)
    moe.moe_debug_set_wait_limit(200)  # ns
    try:
        moe.moe_kv_attention_shared(c.cache, 0, c.q, c.dev(c.cu), c.dev(c.lens), c.dev(c.table), c.dev(c.groups),
                                    c.dev(c.prefix), max_rows=c.max_rows, max_group_rows=c.max_group_rows, ws=ws)
        got = moe.moe_check_status(ws)
    finally:
        moe.moe_debug_set_wait_limit(0)
    assert got == moe.MOE_ERR_TIMEOUT
    moe.moe_clear_status(ws)
    assert torch.equal(c.run(ws=ws)[0].view(torch.int16), want.view(torch.int16))


def test_offsets_beyond_32_bits():
    n_pages = 45000
    cache = moe.KvCache(n_pages, 1, 8, 128, 64)
    assert cache.page_bytes * n_pages > 5 << 30
    c = Shared([3], [200], [1, 2, 1], [30, 100, 0], 8, 2, 128, 64, seed=13)
    table, at = np.full_like(c.table, -1), n_pages
    for b in range(3):
        for j in range(c.table.shape[1]):
            if c.table[b, j] >= 0:
                at -= 1
                table[b, j] = at
                cache.codes(0)[at].view(torch.uint8).copy_(torch.from_numpy(c.codes_np[c.table[b, j]]))
                cache.scales(0)[at].copy_(torch.from_numpy(c.scales_np[c.table[b, j]]))
    c.cache, c.table = cache, table
    c.check()


def test_writes_stay_inside():
    g = Guarded()
    c = Shared([3, 1], [700, 0], [1, 5, 2, 1], [0, 63, 5, 1], 2, 7, 128, 16, seed=21)
    want, _ = c.check()
    R, Hq, D = c.q.shape
    out, lse = g.tensor((R, Hq, D), torch.bfloat16, zero=False), g.tensor((R, Hq), torch.float32, zero=False)
    ws = g.workspace(c.workspace())
    for _ in range(2):
        moe.moe_kv_attention_shared(c.cache, 0, c.q, c.dev(c.cu), c.dev(c.lens), c.dev(c.table), c.dev(c.groups), c.dev(c.prefix),
                                    max_rows=5, max_group_rows=8, out=out, lse=lse, ws=ws)
        assert moe.moe_check_status(ws) == moe.MOE_OK and torch.equal(out, want)
    g.check("moe_kv_attention_shared")


def test_nothing_to_do():
    c = Shared([1], [16], [1], [0], 1, 1, 128, 16)
    none = torch.zeros((0, 1, 128), dtype=torch.bfloat16, device="cuda")
    out = moe.moe_kv_attention_shared(c.cache, 0, none, c.dev([0]), c.dev([]), c.dev(np.zeros((0, 2))), c.dev([0]), c.dev([]),
                                      max_rows=1, max_group_rows=1)
    assert out.shape == none.shape
