"""GPU: calls that are the first of their process.  A kernel whose static and dynamic shared memory are more
than 48 KB together needs its limit raised, also where the dynamic part alone is less; what an earlier, larger
call has raised would hide that, so each of these runs in a process of its own."""
import pathlib
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("mxfp4_routed_expert_topk_gb300")

ROOT = pathlib.Path(__file__).resolve().parent.parent
HEAD = """
import torch
import mxfp4_routed_expert_topk_gb300 as moe
i32 = dict(dtype=torch.int32, device="cuda")
"""


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()


def in_a_process(code):
    r = subprocess.run([sys.executable, "-c", HEAD + code + "print('served')\n"], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["served"], r.stdout + r.stderr


def test_reserving_for_any_number_of_sequences():
    """12 bytes a sequence, next to 19 KB: more than 48 KB from 2504 sequences on."""
    in_a_process("""
for seqs in (1, 2503, 2504, 2505, 3000, 4094, 4095, 4096, 9000):
    table, refs = torch.full((seqs, 2), -1, **i32), torch.zeros(seqs + 5, **i32)
    one, ws = torch.ones(seqs, **i32), moe.workspace(moe.moe_kv_pages_workspace_size(seqs, seqs + 5))
    cu, total, seq, pos, slot = moe.moe_kv_reserve(one, 0 * one, table, refs, 16, seqs, ws=ws)
    assert moe.moe_check_status(ws) == moe.MOE_OK, seqs
    at = torch.arange(seqs + 1, **i32)
    assert torch.equal(cu, at) and torch.equal(table[:, 0], at[:-1]) and (table[:, 1] == -1).all(), seqs
    assert torch.equal(seq, at[:-1]) and torch.equal(slot, 16 * at[:-1].long()) and (total == 1).all() and (pos == 0).all(), seqs
    assert int(refs.sum()) == seqs and (refs[:seqs] == 1).all(), seqs
""")


@pytest.mark.parametrize("M,H", [(6, 4096), (5, 4896), (7, 3504), (1, 24576), (1, 24512)])
def test_routing_rows_of_48_kb(M, H):
    """The rows' 2 M H bytes are 48 KB or a little less, and stand next to some that are static."""
    in_a_process(f"""
g = torch.Generator(device="cuda").manual_seed({M + H})
x = torch.randn(({M}, {H}), generator=g, device="cuda").to(torch.bfloat16)
w = torch.randn((64, {H}), generator=g, device="cuda").to(torch.bfloat16)
idx, _ = moe.moe_route_topk(x, w, 4)
want = (x.double() @ w.double().T).topk(4, sorted=True).indices
assert torch.equal(idx.long(), want), (idx, want)
""")


CAPTURED = {
    "reserve": """
n = 3000
table, refs, one = torch.full((n, 2), -1, **i32), torch.zeros(n + 5, **i32), torch.ones(n, **i32)
zero, ws = 0 * one, moe.workspace(256)
cu, lens = torch.zeros(n + 1, **i32), torch.zeros(n, **i32)
maps = dict(row_seq=torch.zeros(n, **i32), row_pos=torch.zeros(n, **i32), row_slot=torch.zeros(n, dtype=torch.int64, device="cuda"))
call = lambda: moe.moe_kv_reserve(one, zero, table, refs, 16, n, cu_rows=cu, kv_len=lens, ws=ws, **maps)
done = lambda: torch.equal(cu, torch.arange(n + 1, **i32)) and int(refs.sum()) == n
""",
    "sample": """
x = torch.randn((3, 70000), device="cuda")
x[:, 777] = 60.0
t, u, out, ws = torch.ones(3, device="cuda"), torch.full((3,), 0.5, device="cuda"), torch.zeros(3, **i32), moe.workspace(256)
call = lambda: moe.moe_sample(x, t, u, next_token=out, ws=ws)
done = lambda: out.tolist() == [777] * 3
""",
    "route": """
x, w = torch.ones((6, 4096), device="cuda").bfloat16(), torch.zeros((64, 4096), device="cuda").bfloat16()
w[[5, 9]] = torch.tensor([[2.0], [1.0]], device="cuda").bfloat16()
idx, wt = torch.zeros((6, 2), **i32), torch.zeros((6, 2), device="cuda")
ws = moe.workspace(moe.moe_workspace_size(moe.MOE_OP_ROUTE, 64, 4096, 32, 6, 2))
call = lambda: moe.moe_route_topk(x, w, 2, idx=idx, w=wt, ws=ws)
done = lambda: idx.tolist() == [[5, 9]] * 6
""",
    "attention": """
c = moe.KvCache(4, 1, 1, 128, 16)
c.buffer.zero_()
c.codes(0).view(torch.uint8).fill_(0x38)
c.scales(0).fill_(1.0)
at, lens, table = torch.tensor([0, 1], **i32), torch.tensor([40], **i32), torch.tensor([[2, 0, 3]], **i32)
q, out = torch.ones((1, 2, 128), device="cuda").bfloat16(), torch.zeros((1, 2, 128), device="cuda").bfloat16()
pre = torch.tensor([32], **i32)
ws = moe.workspace(moe.moe_kv_attention_shared_workspace_size(c, 1, 1, 1, 2))
call = lambda: moe.moe_kv_attention_shared(c, 0, q, at, lens, table, at, pre, 1, 1, out=out, ws=ws)
done = lambda: bool((out == 1).all())
""",
}


@pytest.mark.parametrize("what", CAPTURED)
def test_first_call_inside_a_capture(what):
    """What a kernel needs before its first launch is set up while a stream is captured, too."""
    in_a_process(CAPTURED[what] + """
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call()
assert not done()
g.replay()
torch.cuda.synchronize()
assert done() and moe.moe_check_status(ws) == moe.MOE_OK
""")
