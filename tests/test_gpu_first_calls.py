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
