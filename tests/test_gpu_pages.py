"""GPU: pages found and given back on the device, against the definition.  All results are whole
numbers and are compared exactly."""
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


def dev(v):
    return torch.from_numpy(np.array(v, dtype=np.int32)).cuda()


class Pool:
    """Page tables and counts, kept on the device and in the reference."""

    def __init__(self, seqs, width, n_pages, page, seed=0, held=()):
        self.P, self.n_pages = page, n_pages
        self.refs = np.zeros(n_pages, dtype=np.int32)
        self.refs[list(held)] = 1
        self.table = np.full((seqs, width), -1, dtype=np.int32)
        self.len = np.zeros(seqs, dtype=np.int64)
        self.d_refs, self.d_table = dev(self.refs), dev(self.table)
        self.ws = moe.workspace(moe.moe_kv_pages_workspace_size(seqs, n_pages))

    def same(self):
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs)
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)

    def reserve(self, n, rows=None, status=None, **kw):
        status = moe.MOE_OK if status is None else status
        n = np.asarray(n)
        rows = int(np.maximum(n, 0).sum()) if rows is None else rows
        maps = dict(row_seq=torch.full((rows,), -7, dtype=torch.int32, device="cuda"),
                    row_pos=torch.full((rows,), -7, dtype=torch.int32, device="cuda"),
                    row_slot=torch.full((rows,), -7, dtype=torch.int64, device="cuda"))
        start = kw.pop("start", dev(self.len))
        got = moe.moe_kv_reserve(dev(n), start, self.d_table, self.d_refs, self.P, rows, ws=self.ws, **maps, **kw)
        assert moe.moe_check_status(self.ws) == status
        moe.moe_clear_status(self.ws)
        cu, total, seq, pos, slot = (t.cpu().numpy() for t in got)
        wcu, wseq, wpos, wslot, at = [0], [], [], [], 0
        if status != moe.MOE_OK:
            n = np.zeros(len(n), dtype=np.int64)
        for b, m in enumerate(n):
            o = int(self.len[b])
            for col in range(-(-o // self.P), -(-(o + m) // self.P)) if m else ():
                while self.refs[at] != 0:
                    at += 1
                self.refs[at], self.table[b, col] = 1, at
            wseq += [b] * m
            wpos += list(range(o, o + m))
            wslot += [int(self.table[b, t // self.P]) * self.P + t % self.P for t in range(o, o + m)]
            wcu.append(wcu[-1] + m)
        self.len = self.len + n
        pad = [-7] * (rows - len(wseq))
        assert cu.tolist() == wcu and total.tolist() == self.len.tolist()
        assert seq.tolist() == wseq + pad and pos.tolist() == wpos + pad and slot.tolist() == wslot + pad
        self.same()

    def release(self, keep, status=None):
        status = moe.MOE_OK if status is None else status
        keep = np.asarray(keep)
        moe.moe_kv_release(dev(keep), dev(self.len), self.d_table, self.d_refs, self.P, ws=self.ws)
        assert moe.moe_check_status(self.ws) == status
        moe.moe_clear_status(self.ws)
        for b, m in enumerate(keep):
            if m < 0:
                continue
            for col in range(-(-int(m) // self.P), -(-int(self.len[b]) // self.P)):
                p = self.table[b, col]
                self.table[b, col] = -1
                if 0 <= p < self.n_pages and self.refs[p] > 0:
                    self.refs[p] -= 1
        self.len = np.where(keep < 0, self.len, np.minimum(self.len, keep))
        self.same()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("seqs", [1, 2, 33, 1024, 1025, 2500])
def test_steps_of_a_scheduler(seqs, page):
    """Prompts, decoded rows, rejected drafts and finished sequences, in turn."""
    r = np.random.default_rng(seqs + page)
    hi = max(3, 40000 // seqs)
    c = Pool(seqs, 6 * hi // page + 4, seqs * (5 * hi // page + 5) + 37, page, held=[0, 3, 4, 5, 130, 131])
    c.reserve(r.integers(0, hi, seqs))
    for _ in range(3):
        c.reserve(r.integers(0, 2, seqs))
        c.reserve(r.integers(0, 18, seqs))
        c.release(np.maximum(c.len - r.integers(0, 12, seqs), 0))
        done = r.random(seqs) < 0.3
        c.release(np.where(done, 0, c.len))
        c.reserve(np.where(done, r.integers(0, hi, seqs), 0))
    c.release(np.zeros(seqs, dtype=np.int64))
    assert c.refs.sum() == 6


@pytest.mark.parametrize("n_pages", [1, 2, 127, 128, 129, 1023, 1025, 8193, 131072, 300001])
def test_pool_sizes(n_pages):
    """The last free page of the pool, and one more than there are."""
    held = np.random.default_rng(n_pages).permutation(n_pages)[:n_pages // 2]
    free = n_pages - len(held)
    c = Pool(3, free + 1, n_pages, 16, held=held)
    c.reserve([16 * (free // 2), 0, 16 * (free - free // 2) + 1], status=moe.MOE_ERR_NO_PAGE)
    c.reserve([16 * (free // 2), 0, 16 * (free - free // 2) - 3])
    c.reserve([0, 1, 0], status=moe.MOE_ERR_NO_PAGE)
    c.reserve([0, 0, 3])
    c.release([0, 0, 0])


def test_a_call_that_cannot_be_served_changes_nothing():
    c = Pool(3, 4, 100, 16)
    c.reserve([20, 5, 0])
    bad = moe.MOE_ERR_BAD_PAGE
    c.reserve([1, -1, 0], status=bad)
    c.reserve([1, -2 ** 31, 0], status=bad)
    c.reserve([1, 60, 0], status=bad)                       # past the table's room
    c.reserve([1, 2 ** 31 - 1, 0], rows=64, status=bad)
    c.reserve([3, 3, 3], rows=8, status=bad)                # room of the maps
    c.reserve([3, 3, 3], rows=12)
    shared = c.table[0, 1]
    c.refs[shared] += 1                                     # its last page is somebody else's, too
    c.d_refs.copy_(dev(c.refs))
    c.reserve([1, 1, 1], status=bad)
    c.reserve([0, 1, 1])
    c.refs[shared] = 0                                      # or nobody's
    c.d_refs.copy_(dev(c.refs))
    c.reserve([1, 0, 0], status=bad)
    c.refs[shared] = 1
    c.d_refs.copy_(dev(c.refs))
    for page in (-1, 100, 2 ** 31 - 1):
        c.table[0, 1] = page
        c.d_table.copy_(dev(c.table))
        c.reserve([1, 0, 0], status=bad)
    c.table[0, 1] = shared
    c.d_table.copy_(dev(c.table))
    c.reserve([1, 0, 0])


def test_idle_sequences_may_stand_anywhere():
    c = Pool(4, 3, 50, 16)
    c.len = np.array([-5, 0, 10 ** 9, -2 ** 31])
    c.reserve([0, 17, 0, 0])


def test_lengths_in_place_and_missing_maps():
    c = Pool(3, 9, 64, 16)
    c.reserve([33, 1, 0])
    lens = dev(c.len)
    c.reserve([15, 20, 0], start=lens, kv_len=lens)
    assert lens.tolist() == [48, 21, 0]
    n, L = dev([1, 1, 1]), moe.lib()
    cu = torch.empty(4, dtype=torch.int32, device="cuda")
    args = (n.data_ptr(), lens.data_ptr(), 3, c.d_table.data_ptr(), 9, c.d_refs.data_ptr(), 64, 16, 3, cu.data_ptr(),
            lens.data_ptr(), None, None, None, c.ws.data_ptr(), 256, torch.cuda.current_stream().cuda_stream)
    assert L.moe_kv_reserve(*args) == moe.MOE_OK
    assert lens.tolist() == [49, 22, 1] and cu.tolist() == [0, 1, 2, 3]


def test_no_sequences():
    cu, *_ = moe.moe_kv_reserve(dev([]), dev([]), dev(np.zeros((0, 4))), dev([0, 0]), 16, 0)
    assert cu.tolist() == [0]
    moe.moe_kv_release(dev([]), dev([]), dev(np.zeros((0, 4))), dev([0, 0]), 16)


def test_counts_at_any_address():
    for lead in range(4):
        c = Pool(5, 60, 901, 16, held=range(0, 901, 7))
        wide = torch.full((910,), 5, dtype=torch.int32, device="cuda")
        wide[lead:lead + 901] = c.d_refs
        c.d_refs = wide[lead:lead + 901]
        c.reserve([100, 0, 900, 17, 1])
        c.release([20, 0, 0, 17, 1])
        assert (wide[:lead] == 5).all() and (wide[lead + 901:] == 5).all()


def test_shared_pages_go_with_their_last_holder():
    c = Pool(4, 8, 40, 16)
    c.reserve([70, 0, 0, 0])
    for b in (1, 2):
        c.table[b, :4] = c.table[0, :4]
        c.refs[c.table[0, :4]] += 1
        c.len[b] = 64
    c.d_table.copy_(dev(c.table))
    c.d_refs.copy_(dev(c.refs))
    c.reserve([5, 9, 20, 3])
    c.release([0, 64, 30, 3])
    assert (c.refs[[0, 1]] == 2).all()
    c.release([0, 0, 0, 3])
    assert c.refs.sum() == 1
    c.reserve([128, 0, 0, 0])


def test_release_reports_what_it_cannot_give_back():
    c = Pool(3, 4, 30, 16)
    c.reserve([40, 33, 1])
    c.release([-1, 33, 1], status=moe.MOE_ERR_BAD_PAGE)
    good = c.len.copy()
    c.len[0] = 65                                            # past the table: left alone
    moe.moe_kv_release(dev([0, 33, 1]), dev(c.len), c.d_table, c.d_refs, 16, ws=c.ws)
    assert moe.moe_check_status(c.ws) == moe.MOE_ERR_BAD_PAGE
    moe.moe_clear_status(c.ws)
    c.same()
    c.len = good
    for page in (-1, 30, 2 ** 31 - 1):
        c.table[0, 1] = page
        c.d_table.copy_(dev(c.table))
        c.release([16, 33, 1], status=moe.MOE_ERR_BAD_PAGE)
        c.table[0, 1:3] = [20, 21]
        c.refs[[20, 21]] = 1
        c.len[0] = 40
        c.d_table.copy_(dev(c.table))
        c.d_refs.copy_(dev(c.refs))
    c.refs[20] = 0                                           # held by nobody
    c.d_refs.copy_(dev(c.refs))
    c.release([0, 0, 0], status=moe.MOE_ERR_BAD_PAGE)
    assert c.refs.nonzero()[0].tolist() == [1]               # (whose entry was overwritten above)


def test_a_step_in_a_graph_follows_its_lengths():
    """Reserve, append's arguments, release: captured once, replayed with other lengths."""
    P, seqs, rows = 16, 7, 64
    c = Pool(seqs, 40, 200, P)
    n, lens, keep = dev([0] * seqs), dev([0] * seqs), dev([0] * seqs)
    total = torch.empty_like(lens)
    outs = dict(cu_rows=torch.empty(seqs + 1, dtype=torch.int32, device="cuda"), kv_len=total,
                row_seq=torch.empty(rows, dtype=torch.int32, device="cuda"),
                row_pos=torch.empty(rows, dtype=torch.int32, device="cuda"),
                row_slot=torch.empty(rows, dtype=torch.int64, device="cuda"))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        moe.moe_kv_reserve(n, lens, c.d_table, c.d_refs, P, rows, ws=c.ws, **outs)
        torch.minimum(total, keep, out=lens)
        moe.moe_kv_release(lens, total, c.d_table, c.d_refs, P, ws=c.ws)
    r = np.random.default_rng(3)
    for _ in range(20):
        m = r.integers(0, 9, seqs)
        k = np.where(r.random(seqs) < 0.1, 0, c.len + m - r.integers(0, 5, seqs))
        k = np.maximum(k, 0)
        n.copy_(dev(m))
        keep.copy_(dev(k))
        g.replay()
        torch.cuda.synchronize()
        assert moe.moe_check_status(c.ws) == moe.MOE_OK
        at = 0
        for b in range(seqs):
            for col in range(-(-int(c.len[b]) // P), -(-int(c.len[b] + m[b]) // P)):
                while c.refs[at]:
                    at += 1
                c.refs[at], c.table[b, col] = 1, at
        c.len = c.len + m
        for b in range(seqs):
            for col in range(-(-int(k[b]) // P), -(-int(c.len[b]) // P)):
                c.refs[c.table[b, col]] -= 1
                c.table[b, col] = -1
        c.len = np.minimum(c.len, k)
        assert lens.tolist() == c.len.tolist() and outs["cu_rows"].tolist() == [0] + np.cumsum(m).tolist()
        c.same()


def test_writes_stay_inside():
    g = Guarded()
    seqs, width, n_pages, rows = 6, 9, 301, 200
    table, refs = g.tensor((seqs, width), torch.int32), g.tensor((n_pages,), torch.int32)
    table.fill_(-1)
    outs = dict(cu_rows=g.tensor((seqs + 1,), torch.int32), kv_len=g.tensor((seqs,), torch.int32),
                row_seq=g.tensor((rows,), torch.int32), row_pos=g.tensor((rows,), torch.int32),
                row_slot=g.tensor((rows,), torch.int64))
    ws = g.workspace(moe.moe_kv_pages_workspace_size(seqs, n_pages))
    start = dev([0] * seqs)
    moe.moe_kv_reserve(dev([144, 0, 7, 17, 16, 16]), start, table, refs, 16, rows, ws=ws, **outs)
    assert moe.moe_check_status(ws) == moe.MOE_OK and int(refs.sum()) == 9 + 1 + 2 + 1 + 1
    moe.moe_kv_reserve(dev([145, 0, 7, 17, 16, 16]), start, table, refs, 16, rows, ws=ws, **outs)
    assert moe.moe_check_status(ws) == moe.MOE_ERR_BAD_PAGE
    moe.moe_kv_release(dev([0] * seqs), dev([144, 0, 7, 17, 16, 16]), table, refs, 16, ws=ws)
    assert int(refs.sum()) == 0 and (table == -1).all()
    g.check("moe_kv_reserve")


def test_refusals():
    t, r, n = dev(np.full((2, 4), -1)), dev([0] * 10), dev([1, 1])
    with pytest.raises(moe.MoeError):
        moe.moe_kv_reserve(n, n, t, r, 48, 2)
    with pytest.raises(ValueError):
        moe.moe_kv_reserve(dev([1]), n, t, r, 16, 2)
    with pytest.raises(ValueError):
        moe.moe_kv_reserve(n, n, t, r.long(), 16, 2)
    with pytest.raises(ValueError):
        moe.moe_kv_reserve(n, n, t, r, 16, 2, row_slot=dev([0, 0]))
    with pytest.raises(ValueError):
        moe.moe_kv_release(n, dev([1]), t, r, 16)


def test_as_many_sequences_as_there_may_be():
    r = np.random.default_rng(5)
    c = Pool(16384, 12, 16384 * 6 + 11, 16, held=[0, 7, 9])
    c.reserve(r.integers(0, 40, 16384))
    c.reserve(r.integers(0, 3, 16384))
    c.release(np.maximum(c.len - 9, 0))
    c.reserve(r.integers(0, 60, 16384))


def test_as_many_pages_as_there_may_be():
    """2^24 pages, of which few are free: the last ones and some in between."""
    n_pages = 1 << 24
    free = torch.tensor([5, 4095, 4096, 9000001] + list(range(n_pages - 300, n_pages)), device="cuda")
    refs = torch.ones(n_pages, dtype=torch.int32, device="cuda")
    refs[free] = 0
    table = torch.full((4, 100), -1, dtype=torch.int32, device="cuda")
    ws = moe.workspace(moe.moe_kv_pages_workspace_size(4, n_pages))
    n = [128 * 100, 1, 128 * 99 + 1, 128 * 100]
    cu, total, seq, pos, slot = moe.moe_kv_reserve(dev(n), dev([0] * 4), table, refs, 128, sum(n), ws=ws)
    assert moe.moe_check_status(ws) == moe.MOE_OK
    want = free[:301].tolist()
    got = table.tolist()
    assert got[0] + got[1][:1] + got[2] + got[3] == want and got[1][1:] == [-1] * 99
    assert refs.sum().item() == n_pages - len(free) + 301 and (refs[free[:301]] == 1).all()
    at = 0
    for b, m in enumerate(n):
        pages = torch.tensor(got[b], device="cuda").long()
        t = torch.arange(m, device="cuda")
        assert torch.equal(slot[at:at + m], pages[t // 128] * 128 + t % 128)
        assert (seq[at:at + m] == b).all() and torch.equal(pos[at:at + m].long(), t)
        at += m
    moe.moe_kv_release(dev([0] * 4), total, table, refs, 128, ws=ws)
    assert moe.moe_check_status(ws) == moe.MOE_OK
    assert refs.sum().item() == n_pages - len(free) and (table == -1).all()
