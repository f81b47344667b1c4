"""CPU checks of the serving operators' entry points: sizes, refusals, error texts (none
of these calls reaches the GPU)."""
import ctypes

import pytest
import torch

import mxfp4_routed_expert_topk_gb300 as moe

vp = ctypes.c_void_p
FAKE = vp(1 << 20)       # never dereferenced: validation fails first
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


@pytest.fixture()
def kv(L):
    h = vp()
    assert L.moe_kv_create(ctypes.byref(h), FAKE, BIG, 64, 2, 8, 128, 64) == moe.MOE_OK
    yield h
    L.moe_kv_destroy(h)


def test_page_bytes(L):
    # 2 * 8 heads * 64 tokens * 128 codes, 64 bytes of scales, padded to 128 bytes; two layers
    assert moe.moe_kv_page_bytes(1, 8, 128, 64) == 131072 + 128
    assert moe.moe_kv_page_bytes(2, 8, 128, 64) == 2 * (131072 + 128)
    assert moe.moe_kv_page_bytes(1, 1, 64, 16) == 2048 + 128
    assert moe.moe_kv_page_bytes(3, 17, 128, 32) == 3 * (17 * 8192 + 256)
    for bad in ((0, 8, 128, 64), (1, 0, 128, 64), (1, 8, 96, 64), (1, 8, 256, 64), (1, 8, 128, 8), (1, 8, 128, 48),
                (1, 1025, 128, 64), (4097, 8, 128, 64), (-1, 8, 128, 64)):
        assert moe.moe_kv_page_bytes(*bad) == 0


def test_create_refusals(L):
    h = vp()
    rec = moe.moe_kv_page_bytes(1, 8, 128, 64)
    c = L.moe_kv_create
    assert c(None, FAKE, BIG, 4, 1, 8, 128, 64) == moe.MOE_ERR_INVALID_ARG
    assert c(ctypes.byref(h), None, BIG, 4, 1, 8, 128, 64) == moe.MOE_ERR_INVALID_ARG
    assert c(ctypes.byref(h), vp((1 << 20) + 64), BIG, 4, 1, 8, 128, 64) == moe.MOE_ERR_INVALID_ARG   # alignment
    assert c(ctypes.byref(h), FAKE, 4 * rec - 1, 4, 1, 8, 128, 64) == moe.MOE_ERR_INVALID_ARG          # room
    assert c(ctypes.byref(h), FAKE, BIG, 0, 1, 8, 128, 64) == moe.MOE_ERR_INVALID_ARG
    assert c(ctypes.byref(h), FAKE, BIG, 4, 1, 8, 80, 64) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    assert c(ctypes.byref(h), FAKE, 1 << 62, (1 << 24) + 1, 1, 8, 128, 64) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    assert h.value is None
    assert c(ctypes.byref(h), FAKE, 4 * rec, 4, 1, 8, 128, 64) == moe.MOE_OK
    L.moe_kv_destroy(h)
    L.moe_kv_destroy(None)


def test_append_refusals(L, kv):
    def call(h=kv, layer=0, k=FAKE, ldk=1024, v=FAKE, ldv=1024, rows=4, cu=FAKE, start=FAKE, table=FAKE, width=8, seqs=2,
             ws=FAKE, n=256):
        return L.moe_kv_append(h, layer, k, ldk, v, ldv, rows, cu, start, table, width, seqs, ws, n, None)

    odd = vp((1 << 20) + 8)
    for bad in (dict(h=None), dict(layer=-1), dict(layer=2), dict(k=None), dict(v=None), dict(ldk=1016), dict(ldv=1028),
                dict(k=odd), dict(v=odd), dict(rows=-1), dict(seqs=-1), dict(width=-1), dict(cu=None), dict(start=None),
                dict(table=None), dict(ws=None), dict(ws=odd)):
        assert call(**bad) == moe.MOE_ERR_INVALID_ARG, bad
    assert call(n=255) == moe.MOE_ERR_WORKSPACE
    # nothing to write: accepted without touching the arrays
    assert call(rows=0, k=None, v=None) == moe.MOE_OK and call(seqs=0, cu=None, start=None, table=None) == moe.MOE_OK


def test_attention_refusals(L, kv):
    def call(h=kv, layer=0, q=FAKE, ldq=7168, rows=4, heads_q=56, cu=FAKE, lens=FAKE, table=FAKE, width=8, seqs=2,
             max_rows=2, scale=0.1, out=FAKE, ldo=7168, lse=None, ws=FAKE, n=256):
        return L.moe_kv_attention(h, layer, q, ldq, rows, heads_q, cu, lens, table, width, seqs, max_rows, scale, out, ldo,
                                  lse, ws, n, None)

    for bad in (dict(h=None), dict(layer=2), dict(layer=-1), dict(rows=-1), dict(seqs=-1), dict(width=-1), dict(heads_q=0),
                dict(heads_q=57), dict(max_rows=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(ws=None)):
        assert call(**bad) == moe.MOE_ERR_INVALID_ARG, bad
    assert call(heads_q=32776) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(max_rows=(1 << 20) + 1) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    n = ctypes.c_size_t()
    assert L.moe_kv_attention_workspace_size(kv, 1, 56, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_attention_workspace_size(None, 1, 56, ctypes.byref(n)) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_attention_workspace_size(kv, 1, 55, ctypes.byref(n)) == moe.MOE_ERR_INVALID_ARG


def test_verify_refusals(L):
    size = moe.moe_verify_workspace_size(2, 8)

    def sampled(p=FAKE, ldp=100, q=FAKE, ldq=100, dt=0, rows=8, vocab=100, tok=FAKE, cu=FAKE, seqs=2, u=FAKE, us=FAKE,
                a=FAKE, x=FAKE, ws=FAKE, n=size):
        return L.moe_verify_sampled(p, ldp, q, ldq, dt, rows, vocab, tok, cu, seqs, u, us, a, x, ws, n, None)

    def greedy(p=FAKE, ldp=100, dt=0, rows=8, vocab=100, tok=FAKE, cu=FAKE, seqs=2, a=FAKE, x=FAKE, ws=FAKE, n=size):
        return L.moe_verify_greedy(p, ldp, dt, rows, vocab, tok, cu, seqs, a, x, ws, n, None)

    for bad in (dict(p=None), dict(ldp=99), dict(dt=2), dict(rows=-1), dict(vocab=0), dict(tok=None), dict(cu=None),
                dict(seqs=-1), dict(a=None), dict(x=None), dict(ws=None), dict(p=vp((1 << 20) + 2)),
                dict(ws=vp((1 << 20) + 16))):
        assert sampled(**bad) == moe.MOE_ERR_INVALID_ARG, bad
        assert greedy(**bad) == moe.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(u=None), dict(us=None), dict(ldq=99), dict(q=vp((1 << 20) + 2))):
        assert sampled(**bad) == moe.MOE_ERR_INVALID_ARG, bad
    for f in (sampled, greedy):
        assert f(vocab=(1 << 20) + 1, ldp=1 << 21) == moe.MOE_ERR_UNSUPPORTED_SHAPE
        assert f(n=size - 1) == moe.MOE_ERR_WORKSPACE
    with pytest.raises(moe.MoeError):
        moe.moe_verify_workspace_size(-1, 1)
    assert moe.status_string(moe.MOE_ERR_BAD_PAGE) not in ("", "unknown status")


def test_binding_refuses_wrong_tensors(L):
    t = torch.zeros(4, 8, 128, dtype=torch.bfloat16)      # host tensors
    with pytest.raises(ValueError):
        moe.KvCache(2, 1, 8, 128, 64, buffer=torch.zeros(10, dtype=torch.uint8))
    with pytest.raises(moe.MoeError):
        moe.KvCache(2, 1, 8, 100, 64)
    with pytest.raises(ValueError):
        moe.moe_verify_greedy(t[0], torch.zeros(8, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
