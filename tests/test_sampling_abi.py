"""CPU checks of the entry points for shared prefixes, pages from lengths and sampling: sizes, refusals,
devices (none of these calls reaches the GPU)."""
import ctypes
import types

import pytest
import torch

import mxfp4_routed_expert_topk_gb300 as moe
from mxfp4_routed_expert_topk_gb300 import _lib as binding
from tests.test_binding_devices import CACHE, F32, I32, U8, Machine, Tensor, heads

vp = ctypes.c_void_p
FAKE = vp(1 << 20)       # never dereferenced: validation fails first
ODD = vp((1 << 20) + 8)
BAD = moe.MOE_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


@pytest.fixture()
def kv(L):
    h = vp()
    assert L.moe_kv_create(ctypes.byref(h), FAKE, 1 << 40, 64, 2, 8, 128, 64) == moe.MOE_OK
    yield h
    L.moe_kv_destroy(h)


def test_status_text(L):
    assert moe.status_string(moe.MOE_ERR_NO_PAGE) not in ("", "unknown status")


def test_shared_attention_refusals(L, kv):
    def call(h=kv, layer=0, q=FAKE, ldq=7168, rows=4, heads_q=56, cu=FAKE, lens=FAKE, table=FAKE, width=8, seqs=2, cg=FAKE,
             pre=FAKE, groups=1, max_rows=2, mgr=4, scale=0.1, out=FAKE, ldo=7168, lse=None, ws=FAKE, n=256):
        return L.moe_kv_attention_shared(h, layer, q, ldq, rows, heads_q, cu, lens, table, width, seqs, cg, pre, groups,
                                         max_rows, mgr, scale, out, ldo, lse, ws, n, None)

    for bad in (dict(h=None), dict(layer=2), dict(layer=-1), dict(rows=-1), dict(seqs=-1), dict(width=-1), dict(heads_q=0),
                dict(heads_q=57), dict(max_rows=-1), dict(mgr=-1), dict(groups=-1), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(ws=None)):
        assert call(**bad) == BAD, bad
    assert call(heads_q=32776) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(max_rows=(1 << 20) + 1) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(mgr=(1 << 20) + 1) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    n = ctypes.c_size_t()
    size = L.moe_kv_attention_shared_workspace_size
    assert size(kv, 4, 1, 1, 56, None) == BAD and size(None, 4, 1, 1, 56, ctypes.byref(n)) == BAD
    assert size(kv, 4, 1, 1, 55, ctypes.byref(n)) == BAD and size(kv, -1, 1, 1, 56, ctypes.byref(n)) == BAD


def test_pages_refusals(L):
    assert moe.moe_kv_pages_workspace_size(64, 1000) >= 256

    def reserve(new=FAKE, start=FAKE, seqs=2, table=FAKE, width=8, refs=FAKE, pages=100, page=64, rows=4, cu=FAKE, lens=FAKE,
                ws=FAKE, n=256):
        return L.moe_kv_reserve(new, start, seqs, table, width, refs, pages, page, rows, cu, lens, None, None, None, ws, n, None)

    def release(keep=FAKE, lens=FAKE, seqs=2, table=FAKE, width=8, refs=FAKE, pages=100, page=64, ws=FAKE, n=256):
        return L.moe_kv_release(keep, lens, seqs, table, width, refs, pages, page, ws, n, None)

    for f in (reserve, release):
        for bad in (dict(seqs=-1), dict(table=None), dict(width=-1), dict(refs=None), dict(pages=-1), dict(lens=None),
                    dict(ws=None), dict(ws=ODD)):
            assert f(**bad) == BAD, bad
        for bad in (dict(seqs=16385), dict(pages=(1 << 24) + 1), dict(page=48), dict(page=0)):
            assert f(**bad) == moe.MOE_ERR_UNSUPPORTED_SHAPE, bad
        assert f(n=255) == moe.MOE_ERR_WORKSPACE
    for bad in (dict(new=None), dict(start=None), dict(cu=None), dict(rows=-1)):
        assert reserve(**bad) == BAD, bad
    assert reserve(rows=(1 << 30) + 1) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    assert release(keep=None) == BAD
    assert release(seqs=0, keep=None, lens=None, table=None) == moe.MOE_OK


def test_sampling_refusals(L):
    def sample(x=FAKE, ld=100, dt=0, rows=8, vocab=100, t=FAKE, u=FAKE, nxt=FAKE, ws=FAKE, n=256):
        return L.moe_sample(x, ld, dt, rows, vocab, t, None, None, None, u, nxt, ws, n, None)

    def probs(x=FAKE, ld=100, dt=0, rows=8, vocab=100, t=FAKE, out=FAKE, ldp=100, ws=FAKE, n=256):
        return L.moe_sample_probs(x, ld, dt, rows, vocab, t, None, None, None, out, ldp, ws, n, None)

    for f in (sample, probs):
        for bad in (dict(x=None), dict(x=vp((1 << 20) + 2)), dict(ld=99), dict(dt=2), dict(dt=-1), dict(rows=-1), dict(vocab=0),
                    dict(t=None), dict(ws=None), dict(ws=ODD)):
            assert f(**bad) == BAD, bad
        assert f(vocab=(1 << 20) + 1, ld=1 << 21) == moe.MOE_ERR_UNSUPPORTED_SHAPE
        assert f(rows=(1 << 20) + 1) == moe.MOE_ERR_UNSUPPORTED_SHAPE
        assert f(n=255) == moe.MOE_ERR_WORKSPACE
        assert f(rows=0, x=None, t=None) == moe.MOE_OK
    assert sample(u=None) == BAD and sample(nxt=None) == BAD
    assert probs(out=FAKE, x=FAKE, ldp=101) == BAD      # over the logits with other rows
    assert probs(out=None) == BAD and probs(ldp=99) == BAD and probs(out=vp((1 << 20) + 2)) == BAD


# ------------------------------------------------------- several devices


@pytest.fixture()
def machine(monkeypatch):
    m = Machine()
    names = ("moe_kv_attention_shared", "moe_kv_reserve", "moe_kv_release", "moe_sample", "moe_sample_probs",
             "moe_kv_attention_shared_workspace_size")
    monkeypatch.setattr(binding, "lib", lambda: types.SimpleNamespace(**{n: m.entry(n) for n in names}))
    monkeypatch.setattr(binding, "_current_device", lambda: m.current, raising=False)
    monkeypatch.setattr(binding, "_raw_stream_of", lambda d: 1000 + d)
    monkeypatch.setattr(torch.cuda, "device", m.device)
    return m


def i32(*shape):
    return Tensor(shape, I32)


def f32(*shape):
    return Tensor(shape, F32)


ENTRIES = {
    "moe_kv_attention_shared": (dict(cache=CACHE, layer=0, max_rows=5, max_group_rows=5), lambda: dict(
        q=heads(4), cu_rows=i32(3), kv_len=i32(2), page_table=i32(2, 4), cu_groups=i32(2), prefix_len=i32(1), out=heads(4),
        lse=f32(5, 4), ws=Tensor((256,), U8))),
    "moe_kv_reserve": (dict(page_tokens=16, rows=5), lambda: dict(
        new_rows=i32(2), start=i32(2), page_table=i32(2, 4), refs=i32(9), cu_rows=i32(3), kv_len=i32(2), row_seq=i32(5),
        row_pos=i32(5), row_slot=Tensor((5,), torch.int64), ws=Tensor((256,), U8))),
    "moe_kv_release": (dict(page_tokens=16), lambda: dict(keep=i32(2), kv_len=i32(2), page_table=i32(2, 4), refs=i32(9),
                                                          ws=Tensor((256,), U8))),
    "moe_sample": ({}, lambda: dict(logits=f32(5, 9), temperature=f32(5), u=f32(5), top_k=i32(5), top_p=f32(5), min_p=f32(5),
                                    next_token=i32(5), ws=Tensor((256,), U8))),
    "moe_sample_probs": ({}, lambda: dict(logits=f32(5, 9), temperature=f32(5), top_k=i32(5), top_p=f32(5), min_p=f32(5),
                                          probs=f32(5, 9), ws=Tensor((256,), U8))),
}


@pytest.mark.parametrize("name", ENTRIES)
def test_calls_run_on_the_tensors_device(machine, name):
    first, tensors = ENTRIES[name]
    for current in (0, 1):
        machine.current = current
        getattr(binding, name)(**first, **tensors())
        assert machine.calls.pop() == (name, 1, 1001) and machine.current == current
        getattr(binding, name)(**first, **tensors(), stream=types.SimpleNamespace(cuda_stream=77, device_index=1))
        assert machine.calls.pop() == (name, 1, 77)
    with pytest.raises(ValueError):
        getattr(binding, name)(**first, **tensors(), stream=types.SimpleNamespace(cuda_stream=77, device_index=0))
    assert machine.calls == []


@pytest.mark.parametrize("name", ENTRIES)
@pytest.mark.parametrize("other", [0, -1])
def test_tensors_of_other_devices_are_refused(machine, name, other):
    first, make = ENTRIES[name]
    for odd in make():
        tensors = make()
        tensors[odd].at, tensors[odd].is_cuda = other, other >= 0
        with pytest.raises(ValueError):
            getattr(binding, name)(**first, **tensors)
        assert machine.calls == []
