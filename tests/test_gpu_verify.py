"""GPU: verification of drafted tokens against the definition in Python's whole numbers.
Every comparison is exact: the results are whole numbers that no order of sums changes."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_guard_bands import Guarded

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("mxfp4_routed_expert_topk_gb300")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()


def whole(x, bits, top):
    x = float(x)
    if math.isnan(x) or x <= 0:
        return 0
    if math.isinf(x):
        return top
    return min(int(x * 2.0 ** bits), top)   # exact: 24 significant bits


def wholes(row):
    return [whole(x, 38, 1 << 38) for x in row.tolist()]


def ref_sampled(p, q, tok, cu, u, us, vocab):
    took, nxt = [], []
    for b in range(len(cu) - 1):
        if cu[b] == cu[b + 1]:
            took.append(0)
            nxt.append(-1)
            continue
        r, W = cu[b], None
        while W is None:
            P = wholes(p[r])
            if r + 1 == cu[b + 1]:
                W = P
                break
            d, m = tok[r + 1], whole(u[r], 24, (1 << 24) - 1)
            inside = 0 <= d < vocab
            Q = wholes(q[r]) if q is not None else [1 << 38 if i == d else 0 for i in range(vocab)]
            if inside and m * Q[d] < P[d] << 24:
                r += 1
                continue
            W = [max(x - y, 0) for x, y in zip(P, Q)]
            if sum(W) == 0:
                W = P
        S = sum(W)
        aim, at, token = (S * whole(us[b], 24, (1 << 24) - 1)) >> 24, 0, -1
        if S:
            for i, w in enumerate(W):
                at += w
                if at > aim:
                    token = i
                    break
        took.append(r - cu[b])
        nxt.append(token)
    return took, nxt


def ref_greedy(x, tok, cu):
    took, nxt = [], []
    for b in range(len(cu) - 1):
        best, r = -1, cu[b]
        while r < cu[b + 1]:
            row = x[r].double().cpu().numpy()
            live = ~np.isnan(row)
            best = -1 if not live.any() else int(np.flatnonzero(live & (row == row[live].max()))[0])
            if r + 1 == cu[b + 1] or best < 0 or tok[r + 1] != best:
                break
            r += 1
        took.append(r - cu[b] if cu[b] < cu[b + 1] else 0)
        nxt.append(best)
    return took, nxt


def dev(a, dt=torch.int32):
    return torch.tensor(a, dtype=dt, device="cuda")


def check_sampled(p, q, tok, cu, u, us, rows_of=lambda t: t):
    vocab = p.shape[1]
    ws = moe.workspace(moe.moe_verify_workspace_size(len(cu) - 1, p.shape[0]))
    got = moe.moe_verify_sampled(rows_of(p), None if q is None else rows_of(q), dev(tok), dev(cu), dev(u, torch.float32),
                                 dev(us, torch.float32), ws=ws)
    assert moe.moe_check_status(ws) == moe.MOE_OK
    u32, us32 = np.float32(u), np.float32(us)
    want = ref_sampled(p, q, tok, cu, u32, us32, vocab)
    assert [g.tolist() for g in got] == [list(w) for w in want]
    again = moe.moe_verify_sampled(rows_of(p), None if q is None else rows_of(q), dev(tok), dev(cu),
                                   dev(u, torch.float32), dev(us, torch.float32), ws=ws)
    assert [g.tolist() for g in again] == [list(w) for w in want]
    return want


def draw_case(rng, n, vocab, dtype, close=0.3, sharp=2.0):
    R = sum(n)
    x = rng.standard_normal((R, vocab)) * sharp
    y = x + close * rng.standard_normal((R, vocab))
    soft = lambda z: torch.softmax(torch.from_numpy(z), -1).to(dtype).cuda()  # noqa: E731
    p, q = soft(x), soft(y)
    tok = [0] * R
    for r in range(R - 1):
        w = q[r].double().cpu().numpy()
        tok[r + 1] = int(rng.choice(vocab, p=w / w.sum()))
    cu = np.concatenate([[0], np.cumsum(n)]).tolist()
    return p, q, tok, cu, rng.random(R).tolist(), rng.random(len(n)).tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,vocab", [([1], 1), ([2, 3], 2), ([5], 7), ([1, 17, 4, 0, 9], 100), ([6] * 20, 333),
                                     ([3, 3], 1025), ([5, 2], 4099), ([4], 32001), ([33, 40], 65)])
@pytest.mark.parametrize("lookup", [False, True])
def test_sampled(dtype, n, vocab, lookup):
    rng = np.random.default_rng(vocab + len(n))
    p, q, tok, cu, u, us = draw_case(rng, n, vocab, dtype)
    if lookup:
        tok[1:] = [int(t) for t in p.float().argmax(-1)[:-1]]
    check_sampled(p, None if lookup else q, tok, cu, u, us)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sampled_large_vocabulary(dtype):
    rng = np.random.default_rng(3)
    p, q, tok, cu, u, us = draw_case(rng, [3, 2], 163_841, dtype, sharp=4.0)
    check_sampled(p, q, tok, cu, u, us)
    check_sampled(p, None, tok, cu, u, [0.0, 0.99999994])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,pad", [(1000, 1), (1001, 2), (77, 3), (4096, 8)])
def test_sampled_rows_at_any_stride(dtype, vocab, pad):
    rng = np.random.default_rng(vocab)
    p, q, tok, cu, u, us = draw_case(rng, [4, 1, 3], vocab, dtype)

    def padded(t):
        w = torch.full((t.shape[0], vocab + pad), float("nan"), dtype=dtype, device="cuda")
        w[:, :vocab] = t
        return w[:, :vocab]

    check_sampled(p, q, tok, cu, u, us, rows_of=padded)


def test_sampled_edges():
    nan, inf = float("nan"), float("inf")
    V = 6
    rows = [
        # p, q, draft, u: what each row checks
        ([0.5, 0.5, 0, 0, 0, 0], [0.5, 0.5, 0, 0, 0, 0], 0, 0.99999994),   # equal: accepted at any u
        ([0.2, 0.8, 0, 0, 0, 0], [0.4, 0.6, 0, 0, 0, 0], 0, 0.5),          # u exactly p/q is a rejection
        ([0.2, 0.8, 0, 0, 0, 0], [0.4, 0.6, 0, 0, 0, 0], 0, 0.49999997),   # just below is not
        ([0, 1, 0, 0, 0, 0], [1, 0, 0, 0, 0, 0], 0, 0.0),                  # p = 0: rejected even at u = 0
        ([0.1, 0.9, 0, 0, 0, 0], [0, 1, 0, 0, 0, 0], 0, 0.9),              # q = 0 < p: accepted
        ([0, 0, 0, 0, 0, 0], [0, 0, 0, 0, 0, 0], 2, 0.0),                  # nothing anywhere: no token
        ([nan, 0.5, 0.5, 0, 0, 0], [nan, 0.5, 0.4, 0, 0, 0], 0, 0.1),      # NaN counts as 0
        ([inf, 0.5, 0.5, 0, 0, 0], [0.5, 0.5, 0.4, 0, 0, 0], 0, 0.1),      # infinity as 1
        ([-1.0, 0.5, 0.5, 0, 0, 0], [0.5, 0.5, 0.4, 0, 0, 0], 0, 0.1),     # negative as 0
        ([0.3, 0.3, 0.4, 0, 0, 0], [0.4, 0.4, 0.4, 1, 0, 0], 0, 0.9),      # rejected, nothing left: all of p
        ([1e-12, 0, 0, 0, 0, 1], [0, 0, 0, 0, 0, 1], 5, 1.5),              # u above 1 counts as just below
        ([0.5, 0.5, 0, 0, 0, 0], [0.5, 0.5, 0, 0, 0, 0], 0, nan),          # u NaN counts as 0
        ([0.5, 0.5, 0, 0, 0, 0], [0.5, 0.5, 0, 0, 0, 0], 6, 0.0),          # a draft outside the vocabulary
        ([0.5, 0.5, 0, 0, 0, 0], [0.5, 0.5, 0, 0, 0, 0], -1, 0.0),
    ]
    for us in (0.0, 0.3, 0.999, 0.99999994, 1.0, -1.0, nan):
        for use_q in (True, False):
            p, q, tok, u, cu = [], [], [], [], [0]
            for a, b, d, x in rows:   # each as a sequence of its own: the row, then a last row
                p += [a, [0.25, 0, 0.25, 0, 0.25, 0.25]]
                q += [b, [nan] * V]
                tok += [0, d]
                u += [x, nan]
                cu.append(cu[-1] + 2)
            check_sampled(dev(p, torch.float32), dev(q, torch.float32) if use_q else None, tok, cu, u, [us] * len(rows))


def test_sampled_keeps_the_target_distribution():
    """First tokens over many uniforms follow p, whatever the draft's q was."""
    V, N = 5, 1 << 14
    p = np.array([0.1, 0.4, 0.05, 0.25, 0.2])
    q = np.array([0.3, 0.1, 0.3, 0.25, 0.05])
    rng = np.random.default_rng(0)
    d = rng.choice(V, size=N, p=q)
    tok = np.stack([np.zeros(N), d], 1).astype(np.int32).reshape(-1)
    P = torch.tensor(np.tile(p, (2 * N, 1)), dtype=torch.float32, device="cuda")
    Q = torch.tensor(np.tile(q, (2 * N, 1)), dtype=torch.float32, device="cuda")
    took, nxt = moe.moe_verify_sampled(P, Q, dev(tok), dev(np.arange(0, 2 * N + 1, 2)),
                                       dev(rng.random(2 * N), torch.float32), dev(rng.random(N), torch.float32))
    first = np.where(took.cpu().numpy() > 0, d, nxt.cpu().numpy())
    got = np.bincount(first, minlength=V) / N
    assert np.abs(got - p).max() < 5 * 0.5 / math.sqrt(N)   # five standard deviations


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,vocab,pad", [([1], 1, 0), ([3, 0, 5], 7, 1), ([17, 1, 9], 1000, 0), ([5] * 30, 257, 3),
                                         ([2, 6], 32003, 1), ([4], 131_072, 0), ([40], 515, 5)])
def test_greedy(dtype, n, vocab, pad):
    rng = np.random.default_rng(vocab)
    R = sum(n)
    full = torch.full((R, vocab + pad), float("inf"), dtype=dtype, device="cuda")
    full[:, :vocab] = torch.from_numpy(rng.standard_normal((R, vocab)) * 3).to(dtype)
    x = full[:, :vocab]
    cu = np.concatenate([[0], np.cumsum(n)]).tolist()
    best = [int((r == r.max()).nonzero()[0, 0]) for r in x]
    for good in (1.0, 0.8, 0.0):
        tok = [0] + [b if rng.random() < good else int(rng.integers(vocab)) for b in best[:-1]]
        ws = moe.workspace(moe.moe_verify_workspace_size(len(n), R))
        for _ in range(2):
            got = moe.moe_verify_greedy(x, dev(tok), dev(cu), ws=ws)
            assert moe.moe_check_status(ws) == moe.MOE_OK
            assert [g.tolist() for g in got] == [list(w) for w in ref_greedy(x, tok, cu)]


def test_greedy_edges():
    nan, inf = float("nan"), float("inf")
    rows = [[nan, 1, 2, 2], [nan] * 4, [-inf] * 4, [nan, -inf, -inf, nan], [-0.0, 0.0, -0.0, -1], [0.0, -0.0, 0, 0],
            [inf, 1, inf, 2], [-1e-40, -2e-40, -1e-40, -3], [1e-40, 2e-40, 2e-40, 0]]
    for dtype in (torch.float32, torch.bfloat16):
        x = dev(rows, dtype)
        for tok1 in (0, 1, 2, -1):
            y = x.repeat_interleave(2, 0)
            tok, cu = [0, tok1] * len(rows), list(range(0, 2 * len(rows) + 1, 2))
            got = moe.moe_verify_greedy(y, dev(tok), dev(cu))
            assert [g.tolist() for g in got] == [list(w) for w in ref_greedy(y, tok, cu)]


def test_bad_rows_are_reported():
    p = torch.full((4, 8), 0.125, device="cuda")
    for cu in ([0, 5, 4], [-1, 2, 4], [2, 1, 4], [0, 2, 2 ** 31 - 1]):
        ws = moe.workspace(moe.moe_verify_workspace_size(2, 4))
        u = torch.zeros(4, device="cuda")
        for _ in range(2):
            took, nxt = moe.moe_verify_sampled(p, p, dev([1] * 4), dev(cu), u, u[:2], ws=ws)
            assert moe.moe_check_status(ws) == moe.MOE_ERR_BAD_PAGE
            bad = [b for b in range(2) if not 0 <= cu[b] <= cu[b + 1] <= 4]
            assert all(took[b] == 0 and nxt[b] == -1 for b in bad)
            took, nxt = moe.moe_verify_greedy(p, dev([1] * 4), dev(cu), ws=ws)
            assert moe.moe_check_status(ws) == moe.MOE_ERR_BAD_PAGE
            assert all(took[b] == 0 and nxt[b] == -1 for b in bad)


def test_empty_sequences_and_streams_and_graphs():
    z = torch.empty((0, 5), device="cuda")
    for f in (lambda: moe.moe_verify_sampled(z, None, dev([]), dev([0, 0, 0]), z[:, 0], dev([0.5, 0.5], torch.float32)),
              lambda: moe.moe_verify_greedy(z, dev([]), dev([0, 0, 0]))):
        took, nxt = f()
        assert took.tolist() == [0, 0] and nxt.tolist() == [-1, -1]
    assert moe.moe_verify_greedy(z, dev([]), dev([0]))[0].numel() == 0
    rng = np.random.default_rng(5)
    p, q, tok, cu, u, us = draw_case(rng, [5, 3], 5000, torch.float32)
    want = check_sampled(p, q, tok, cu, u, us)
    args = (p, q, dev(tok), dev(cu), dev(u, torch.float32), dev(us, torch.float32))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = moe.moe_verify_sampled(*args, stream=st)
    st.synchronize()
    assert [g.tolist() for g in got] == [list(w) for w in want]
    ws = moe.workspace(moe.moe_verify_workspace_size(2, 8))
    a, b = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    c, d = torch.empty_like(a), torch.empty_like(a)
    moe.moe_verify_sampled(*args, accepted=a, next_token=b, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_verify_sampled(*args, accepted=a, next_token=b, ws=ws)
        moe.moe_verify_greedy(p, args[2], args[3], accepted=c, next_token=d, ws=ws)
    greedy = ref_greedy(p, tok, cu)
    for _ in range(3):
        for t in (a, b, c, d):
            t.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        assert [a.tolist(), b.tolist()] == [list(w) for w in want]
        assert [c.tolist(), d.tolist()] == [list(w) for w in greedy]


def test_writes_stay_inside():
    g = Guarded()
    rng = np.random.default_rng(6)
    p, q, tok, cu, u, us = draw_case(rng, [5, 3, 1], 3001, torch.bfloat16)
    took, nxt = g.tensor((3,), torch.int32), g.tensor((3,), torch.int32)
    ws = g.workspace(moe.moe_verify_workspace_size(3, 9))
    moe.moe_verify_sampled(p, q, dev(tok), dev(cu), dev(u, torch.float32), dev(us, torch.float32), accepted=took,
                           next_token=nxt, ws=ws)
    g.check("moe_verify_sampled")
    moe.moe_verify_greedy(p, dev(tok), dev(cu), accepted=took, next_token=nxt, ws=ws)
    g.check("moe_verify_greedy")
