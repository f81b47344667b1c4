"""GPU: sampling from vocabularies of which many tokens are masked, or hold infinities or NaN, at sizes that a
small list does not hold, with every cut; compared exactly, as in the other tests of sampling."""
import math

import pytest
import torch

from tests.test_gpu_sample import check, dev

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("mxfp4_routed_expert_topk_gb300")

INF, NAN, LOW = math.inf, math.nan, -3.3895314e38  # (the lowest bf16)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()


def rows_of(V, dtype, seed=0):
    """Rows that differ in what is left of them."""
    g = torch.Generator(device="cuda").manual_seed(V + seed)
    x = torch.randn((22, V), generator=g, device="cuda") * 3
    order = torch.randperm(V, generator=g, device="cuda")
    at = torch.arange(V, device="cuda")

    def only(r, where):
        y = torch.full((V,), -INF, device="cuda")
        y[where] = x[r, where]
        x[r] = y

    x[0] = -INF
    x[1] = NAN
    only(2, order[:1])
    only(3, at[-5:])
    only(4, order[:300])
    only(5, order[:1024])
    only(6, order[:1025])
    only(7, order[:V // 2])
    only(8, at[:V // 2])                       # whole CTAs without a token
    only(9, at[V // 2:])
    only(10, at[-1:])
    x[11, ::2] = NAN
    x[12, order[0]] = INF
    x[13, order[:3]] = INF
    x[14, order[:2048 + V // 64]] = INF        # more than the list holds
    x[15] = INF
    x[16] = LOW
    x[17, order[100:]] = LOW                   # a mask of the lowest value
    x[18] = torch.where(at % 3 == 0, NAN, -INF)
    x[19, order[:7]] = 3.0e38
    x[20, order[:2]], x[20, order[2:V // 3]], x[20, order[V // 3:V // 2]] = INF, NAN, LOW
    only(21, order[:40])
    x[21, order[:40]] = 1.0                    # as many equal ones as are left
    return x.to(dtype)


def in_place(x, T, probs, k=None, p=None, m=None, **_):
    moe.moe_sample_probs(x, dev(T), top_k=dev(k, torch.int32), top_p=dev(p), min_p=dev(m), probs=x)
    assert torch.equal(x, probs)


CUTS = [dict(), dict(k=5), dict(k=50, p=0.9), dict(k=1024), dict(k=1025), dict(k=1500, p=0.99, m=0.001), dict(k=-1, p=0.3),
        dict(p=0.999), dict(p=0.5, m=0.01), dict(m=0.2), dict(k=3000, p=0.5)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2049, 2056, 5003, 70000, 131071])
def test_rows_with_little_left(V, dtype):
    x = rows_of(V, dtype)
    R = len(x)
    for i, cut in enumerate(CUTS + [dict(k=V - 1)]):
        s = {n: [v] * R for n, v in cut.items()}
        T, u = [1.0] * R, [(0.07 + 0.31 * (i + r)) % 1.0 for r in range(R)]
        _, probs = check(x, T, u=u, **s)
        in_place(x.clone(), T, probs, **s)


@pytest.mark.parametrize("T", [0.0, -1.0, NAN, 1e-45, 1e-3, 0.2, 1e3, 3e38, INF])
@pytest.mark.parametrize("V", [2049, 20000])
def test_temperatures(V, T):
    x = rows_of(V, torch.float32, seed=1)
    R = len(x)
    for cut in (dict(), dict(k=40), dict(k=1100, p=0.9), dict(p=0.7), dict(p=0.95, m=0.001)):
        check(x, [T] * R, u=[0.83] * R, **{n: [v] * R for n, v in cut.items()})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,times", [(2049, 30), (2305, 1), (4099, 12), (9001, 5)])
def test_many_rows_without_a_bound(V, times, dtype):
    """A top-k that no list holds, next to others, with clusters of every size: the first token of the order, the
    counts and the sums of a row's CTAs are exchanged one right after the other."""
    x = torch.cat([rows_of(V, dtype, seed=i) for i in range(times)])
    R = len(x)
    k = [(1025, 1500, V - 1, 2000, 60)[r % 5] for r in range(R)]
    p = [(1.0, 0.9, 0.5, 0.99)[r % 4] for r in range(R)]
    u = [((r * 37) % 101) / 101 for r in range(R)]
    got, probs = check(x, [0.9] * R, k=k, p=p, u=u)
    in_place(x.clone(), [0.9] * R, probs, k=k, p=p)
    args = dict(top_k=dev(k, torch.int32), top_p=dev(p))
    for _ in range(20):
        assert moe.moe_sample(x, dev([0.9] * R), dev(u), **args).tolist() == got
        assert torch.equal(moe.moe_sample_probs(x, dev([0.9] * R), **args), probs)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,lead", [(2051, 1), (5003, 3), (40007, 0), (40007, 7)])
def test_over_the_logits_at_any_address(V, lead, dtype):
    """Rows that begin and end inside a vector, written over while other CTAs of the row still read theirs, each
    call into the values that the one before has left."""
    rows = rows_of(V, dtype, seed=lead)
    R = len(rows)
    wide = torch.full((R, V + 9), 100.0, dtype=dtype, device="cuda")  # (what is not of a row would win)
    x = wide[:, lead:lead + V]
    for cut in (dict(), dict(k=30), dict(k=1100), dict(p=0.9), dict(k=1100, p=0.8, m=0.001)):
        x.copy_(rows)
        s = {n: [v] * R for n, v in cut.items()}
        for T in (1.0, 0.0):
            _, probs = check(x.clone(), [T] * R, **s)
            in_place(x, [T] * R, probs, **s)
        assert (wide[:, :lead] == 100).all() and (wide[:, lead + V:] == 100).all()


def test_more_rows_than_are_put_in_order():
    """Above 4096 rows the clusters take them one after the other; above 100000, of a few tokens."""
    R, V = 4500, 2100
    x = rows_of(V, torch.bfloat16)[torch.arange(R, device="cuda") % 22]
    k, p = [(0, 3, 1100, 0)[r % 4] for r in range(R)], [(0.9, 1.0, 0.5)[r % 3] for r in range(R)]
    u = [r / R for r in range(R)]
    args = dict(top_k=dev(k, torch.int32), top_p=dev(p))
    got, probs = moe.moe_sample(x, dev([1.0] * R), dev(u), **args), moe.moe_sample_probs(x, dev([1.0] * R), **args)
    for part in (range(0, 60), range(4090, 4130), range(4460, 4500)):
        a, b = part[0], part[-1] + 1
        few, q = check(x[a:b], [1.0] * len(part), k=k[a:b], p=p[a:b], u=u[a:b])
        assert got[a:b].tolist() == few and torch.equal(probs[a:b], q)
    x = torch.randn((120000, 3), device="cuda")
    got = moe.moe_sample(x, dev([0.0] * 120000), dev([0.5] * 120000))
    assert torch.equal(got.long(), x.argmax(-1))
