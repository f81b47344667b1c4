"""GPU: sampling against the definition in whole numbers.  Every comparison is exact: weights follow
from fp32 operations that are rounded one by one, sums are whole numbers, and a probability is one
fp32 division (and one rounding to bf16)."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_guard_bands import Guarded

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("mxfp4_routed_expert_topk_gb300")

F = np.float32
C = [F(float.fromhex(h)) for h in ("0x1.62e42ap-1", "0x1.ebf9bcp-3", "0x1.c6b752p-5", "0x1.3cea88p-7", "0x1.5bba14p-10")]
MAX = np.finfo(np.float32).max


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()


def bits24(v, none):
    return none if math.isnan(v) else int(min(max(v, 0.0), 1.0) * 2 ** 24)


def ref_row(x, T, k=0, p=1.0, m=0.0, u=0.0):
    """(next token, probabilities in fp32) of one row, x float32."""
    V = len(x)
    probs = np.zeros(V, dtype=F)
    order = np.argsort(np.where(np.isnan(x), np.inf, -x), kind="stable")
    order = order[(~np.isnan(x) & (x > -np.inf))[order]]
    if len(order) == 0:
        return -1, probs
    T = F(T)
    if not T > 0:
        probs[order[0]] = 1
        return int(order[0]), probs
    s = x[order]
    with np.errstate(all="ignore"):
        c = min(F(float.fromhex("0x1.715476p+0")) / T, MAX)
        y = np.where(s == s[0], F(0), (s - s[0]) * c)
        n = np.rint(y)
        f = y - n
        e = np.full_like(f, C[4])
        for a in (C[3], C[2], C[1], C[0], F(1)):
            e = e * f + a
        live = y > -39
        W = np.zeros(len(y), dtype=np.int64)
        W[live] = np.floor(np.ldexp(e[live].astype(np.float64), n[live].astype(np.int64) + 38)).astype(np.int64)
    if k > 0:
        W[k:] = 0
    before = np.cumsum(W) - W
    S, t = int(W.sum()), max(1, bits24(p, 1 << 24))
    keep = before < -(-S * t // 2 ** 24)
    keep &= W >= bits24(m, 0) << 14
    W[~keep] = 0
    S = int(W.sum())
    probs[order] = W.astype(F) / F(S)
    left = np.zeros(V, dtype=np.int64)
    left[order] = W
    aim = S * min(0 if math.isnan(u) else int(max(u, 0.0) * 2 ** 24) if u < 1 else 2 ** 24 - 1, 2 ** 24 - 1) >> 24
    return int(np.searchsorted(np.cumsum(left), aim, side="right")), probs


def dev(v, dtype=torch.float32):
    return None if v is None else torch.tensor(v, dtype=dtype, device="cuda")


def check(x, T, k=None, p=None, m=None, u=None, **kw):
    """x: a CUDA tensor; the settings: lists."""
    R = len(x)
    u = [0.5] * R if u is None else u
    got = moe.moe_sample(x, dev(T), dev(u), top_k=dev(k, torch.int32), top_p=dev(p), min_p=dev(m), **kw).tolist()
    probs = moe.moe_sample_probs(x, dev(T), top_k=dev(k, torch.int32), top_p=dev(p), min_p=dev(m))
    f32 = lambda v, r, none: none if v is None else float(F(v[r]))  # noqa: E731
    for r in range(R):
        want, q = ref_row(x[r].float().cpu().numpy(), f32(T, r, 0), 0 if k is None else k[r], f32(p, r, 1.0), f32(m, r, 0.0),
                          f32(u, r, 0.0))
        assert got[r] == want, (r, got[r], want)
        q = torch.from_numpy(q).to(x.dtype)
        assert torch.equal(probs[r].cpu(), q), (r, (probs[r].cpu() != q).nonzero()[:4])
    return got, probs


def logits(R, V, dtype, seed, sigma=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((R, V), generator=g, device="cuda") * sigma
    x[::2, V // 2] += 9
    return x.to(dtype)


def settings(R, V, seed):
    r = np.random.default_rng(seed)
    pick = lambda v: [v[i] for i in r.integers(0, len(v), R)]  # noqa: E731
    return dict(T=pick([0.0, 0.3, 0.7, 1.0, 1.0, 1.3, 4.0]), k=pick([0, 1, 2, 5, 50, 300, 1500, V - 1, V, V + 5, -3]),
                p=pick([0.0, 0.1, 0.5, 0.9, 0.95, 0.999, 1.0, 2.0, -1.0, math.nan]),
                m=pick([0.0, 0.0, 0.0, 0.01, 0.2, 1.0, math.nan, -2.0]), u=[float(v) for v in r.random(R, dtype=np.float32)])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 31, 257, 1000, 2049, 5000, 32001])
def test_every_mix_of_settings(dtype, V):
    R = 40
    check(logits(R, V, dtype, V), **settings(R, V, V))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R", [1, 3, 19, 20, 76, 153, 320])
def test_row_counts(dtype, R):
    """One cluster of any size per row."""
    check(logits(R, 3000, dtype, R), **settings(R, 3000, R))


@pytest.mark.parametrize("cut", ["k", "p", "m", "none"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_cut_at_a_time(dtype, cut):
    R, V = 24, 70001
    s = settings(R, V, 5)
    s["T"] = [0.9] * R
    check(logits(R, V, dtype, 3), **{n: v for n, v in s.items() if n in ("T", "u", cut)})


@pytest.mark.parametrize("V", [1500, 70000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties(dtype, V):
    """Equal logits: the lower index stands first, however many there are."""
    x = torch.zeros((8, V), device="cuda")
    x[1] = 3.0
    x[2, ::3] = 1.0
    x[3] = torch.arange(V, device="cuda") % 5
    x[4] = -(torch.arange(V, device="cuda") // 700).float()
    x[5, 1::2] = -0.0
    x[6] = torch.finfo(dtype).min
    x[7] = -1e-3 * (torch.arange(V, device="cuda") % 2)
    x = x.to(dtype)
    for k, p in ((0, 0.5), (1, 1.0), (V // 2 + 1, 1.0), (V // 2 + 1, 0.3), (V - 1, 0.9999), (1200, 0.97), (0, 1.0)):
        for u in (0.0, 0.4, 0.9999999):
            check(x, [1.0] * 8, k=[k] * 8, p=[p] * 8, u=[u] * 8)


def test_masked_and_odd_values():
    V, inf, nan = 600, math.inf, math.nan
    x = torch.randn((12, V), device="cuda") * 3
    x[0] = -inf
    x[1] = nan
    x[2] = -inf
    x[2, 77] = -5.0
    x[3, ::2] = nan
    x[4, 5] = inf
    x[5, 5] = x[5, 400] = inf
    x[6] = inf
    x[7, 100:] = -3.4028234e38
    x[8] = -3.4028234e38
    x[9, 3:] = -inf
    x[10, 9] = 3.4028234e38
    x[11] = torch.where(torch.arange(V, device="cuda") % 3 == 0, nan, -inf)
    for T in (0.0, -1.0, nan, 1e-45, 1e-38, 1e-3, 1.0, 1e3, 3e38, inf):
        for cuts in (dict(), dict(k=[3] * 12), dict(p=[0.7] * 12), dict(k=[500] * 12, p=[0.99] * 12, m=[0.001] * 12)):
            check(x, [T] * 12, u=[0.83] * 12, **cuts)
    check(x.to(torch.bfloat16), [1.0] * 12, k=[500] * 12, p=[0.99] * 12)


def test_uniforms():
    us = [0.0, 1e-9, 0.25, 0.5, 0.99999994, 1.0, 5.0, -1.0, math.nan, math.inf, -math.inf]
    x = logits(1, 4000, torch.float32, 1).expand(len(us), -1).contiguous()
    a, _ = check(x, [1.0] * len(us), u=us)
    b, _ = check(x, [1.0] * len(us), k=[40] * len(us), p=[0.9] * len(us), u=us)
    assert a[0] == a[7] == a[8] == a[10] and a[4] == a[5] == a[6] == a[9] and b[0] == b[7]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lead", [0, 1, 3])
def test_strides_and_addresses(dtype, lead):
    R, V = 9, 1237
    wide = torch.full((R, V + 50), 100.0, dtype=dtype, device="cuda")  # (what is not of a row would win)
    x = wide[:, lead:lead + V]
    x.copy_(logits(R, V, dtype, 8))
    s = settings(R, V, 8)
    got, probs = check(x, **s)
    out = torch.full((R, V + 37), 7.0, dtype=dtype, device="cuda")
    cuts = dict(top_k=dev(s["k"], torch.int32), top_p=dev(s["p"]), min_p=dev(s["m"]))
    moe.moe_sample_probs(x, dev(s["T"]), probs=out[:, lead:lead + V], **cuts)
    assert torch.equal(out[:, lead:lead + V], probs) and (out[:, :lead] == 7).all() and (out[:, lead + V:] == 7).all()
    moe.moe_sample_probs(x, dev(s["T"]), probs=x, **cuts)     # over the logits themselves
    assert torch.equal(x, probs) and (wide[:, lead + V:] == 100).all() and (wide[:, :lead] == 100).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(1, 1 << 20), (40, 131071), (160, 65537)])
def test_large_vocabularies(dtype, R, V):
    """All in place too: many rows at once, each over its own logits."""
    x = logits(R, V, dtype, V)
    s = settings(R, V, R)
    if R == 1:
        s.update(T=[1.2], k=[300000], p=[0.9999], m=[0.0])
    _, probs = check(x, **s)
    moe.moe_sample_probs(x, dev(s["T"]), top_k=dev(s["k"], torch.int32), top_p=dev(s["p"]), min_p=dev(s["m"]), probs=x)
    assert torch.equal(x, probs)


def test_no_rows_and_refusals():
    x = torch.zeros((0, 10), device="cuda")
    assert moe.moe_sample(x, dev([]), dev([])).shape == (0,)
    assert moe.moe_sample_probs(x, dev([])).shape == (0, 10)
    x = torch.zeros((2, 10), device="cuda")
    with pytest.raises(ValueError):
        moe.moe_sample(x, dev([1.0]), dev([0.5, 0.5]))
    with pytest.raises(ValueError):
        moe.moe_sample(x, dev([1.0, 1.0]), dev([0.5]))
    with pytest.raises(ValueError):
        moe.moe_sample(x.half(), dev([1.0, 1.0]), dev([0.5, 0.5]))
    with pytest.raises(ValueError):
        moe.moe_sample(x.t(), dev([1.0] * 10), dev([0.5] * 10))
    with pytest.raises(ValueError):
        moe.moe_sample_probs(x, dev([1.0, 1.0]), probs=x.to(torch.bfloat16))
    with pytest.raises(ValueError):
        moe.moe_sample_probs(x, dev([1.0, 1.0]), top_k=dev([1.0, 1.0]))


def test_captured_streams_and_repeats():
    """A captured call follows its inputs; two calls at once on two streams share nothing."""
    R, V = 33, 20000
    x, s = logits(R, V, torch.float32, 4), settings(R, V, 4)
    args = dict(top_k=dev(s["k"], torch.int32), top_p=dev(s["p"]), min_p=dev(s["m"]))
    T, u = dev(s["T"]), dev(s["u"])
    want, probs = check(x, **s)
    nxt, out, ws = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty_like(x), moe.workspace(256)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        moe.moe_sample(x, T, u, next_token=nxt, ws=ws, **args)
        moe.moe_sample_probs(x, T, probs=out, ws=ws, **args)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert nxt.tolist() == want and torch.equal(out, probs)
    x.copy_(logits(R, V, torch.float32, 6))
    g.replay()
    torch.cuda.synchronize()
    assert nxt.tolist() == check(x, **s)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [moe.moe_sample(x, T, u, stream=streams[i % 2], **args) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(t, nxt) for t in got)


def test_distributions_go_into_verification():
    """Drafts that equal the only token left are accepted; a cut token is not."""
    V = 5000
    x = logits(4, V, torch.float32, 2)
    q = moe.moe_sample_probs(x, dev([1.0] * 4), top_k=dev([1] * 4, torch.int32))
    best = q.argmax(-1).to(torch.int32)
    cu = dev([0, 4], torch.int32)
    u = dev([0.999] * 4)
    tok = torch.cat([dev([7], torch.int32), best[:3]])
    took, nxt = moe.moe_verify_sampled(q, None, tok, cu, u, u[:1])
    assert took.item() == 3 and nxt.item() == best[3].item()
    tok[2] = (best[1] + 1) % V
    took, nxt = moe.moe_verify_sampled(q, None, tok, cu, u, u[:1])
    assert took.item() == 1 and nxt.item() == best[1].item()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_writes_stay_inside(dtype):
    g = Guarded()
    R, V = 5, 777
    s = settings(R, V, 2)
    x = g.tensor((R, V), dtype, zero=False)
    x.copy_(logits(R, V, dtype, 2))
    out, nxt = g.tensor((R, V), dtype, zero=False), g.tensor((R,), torch.int32, zero=False)
    ws = g.workspace(moe.moe_sample_workspace_size(R, V))
    want, probs = check(x, **s, next_token=nxt, ws=ws)
    moe.moe_sample_probs(x, dev(s["T"]), top_k=dev(s["k"], torch.int32), top_p=dev(s["p"]), min_p=dev(s["m"]), probs=out, ws=ws)
    assert nxt.tolist() == want and torch.equal(out, probs) and moe.moe_check_status(ws) == moe.MOE_OK
    g.check("moe_sample")
