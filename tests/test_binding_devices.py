"""CPU: the serving operators' binding on a machine with several devices, with stand-ins for
tensors, streams and the library.  Every pointer a call hands over must lie on one device, and
that device must be the current one while the call runs (the default stream's handle is 0 on
each, and the number of SMs is the current device's)."""
import contextlib
import types

import pytest
import torch

from mxfp4_routed_expert_topk_gb300 import _lib as binding


class Tensor:
    is_cuda = True

    def __init__(self, shape, dtype, device=1):
        self.shape, self.dtype, self.at, self.is_cuda = torch.Size(shape), dtype, device, device >= 0

    def get_device(self):
        return self.at

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    @property
    def device(self):
        return torch.device("cuda", self.at)


class Machine:
    """Current device, the calls made, and the device and stream that each was made with."""

    def __init__(self):
        self.current, self.calls = 0, []

    @contextlib.contextmanager
    def device(self, n):
        before, self.current = self.current, n
        yield
        self.current = before

    def entry(self, name):
        def call(*args):
            self.calls.append((name, self.current, args[-1]))
            return 0
        return call


@pytest.fixture()
def machine(monkeypatch):
    m = Machine()
    names = ("moe_kv_append", "moe_kv_attention", "moe_verify_sampled", "moe_verify_greedy",
             "moe_kv_attention_workspace_size")
    monkeypatch.setattr(binding, "lib", lambda: types.SimpleNamespace(**{n: m.entry(n) for n in names}))
    monkeypatch.setattr(binding, "_current_device", lambda: m.current, raising=False)
    monkeypatch.setattr(binding, "_raw_stream_of", lambda d: 1000 + d)
    monkeypatch.setattr(torch.cuda, "device", m.device)
    return m


CACHE = types.SimpleNamespace(handle=0, heads=2, head_dim=64, page_tokens=16, device=1,
                              buffer=Tensor((4096,), torch.uint8))
I32, F32, BF16, U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8


def heads(n):
    return Tensor((5, n, 64), BF16)


ENTRIES = {
    "moe_kv_append": lambda: dict(k=heads(2), v=heads(2), cu_rows=Tensor((3,), I32), start=Tensor((2,), I32),
                                  page_table=Tensor((2, 4), I32), ws=Tensor((256,), U8)),
    "moe_kv_attention": lambda: dict(q=heads(4), cu_rows=Tensor((3,), I32), kv_len=Tensor((2,), I32),
                                     page_table=Tensor((2, 4), I32), out=heads(4), lse=Tensor((5, 4), F32),
                                     ws=Tensor((256,), U8)),
    "moe_verify_sampled": lambda: dict(p=Tensor((5, 9), F32), q=Tensor((5, 9), F32), tokens=Tensor((5,), I32),
                                       cu_rows=Tensor((3,), I32), u_accept=Tensor((5,), F32), u_sample=Tensor((2,), F32),
                                       accepted=Tensor((2,), I32), next_token=Tensor((2,), I32), ws=Tensor((256,), U8)),
    "moe_verify_greedy": lambda: dict(logits=Tensor((5, 9), F32), tokens=Tensor((5,), I32), cu_rows=Tensor((3,), I32),
                                      accepted=Tensor((2,), I32), next_token=Tensor((2,), I32), ws=Tensor((256,), U8)),
}


def call(name, tensors, stream=None):
    first = dict(cache=CACHE, layer=0) if name.startswith("moe_kv") else {}
    if name == "moe_kv_attention":
        first["max_rows"] = 5
    getattr(binding, name)(**first, **tensors, stream=stream)


@pytest.mark.parametrize("name", ENTRIES)
def test_calls_run_on_the_tensors_device(machine, name):
    for current in (0, 1):
        machine.current = current
        call(name, ENTRIES[name]())
        assert machine.calls.pop() == (name, 1, 1001) and machine.current == current
        call(name, ENTRIES[name](), types.SimpleNamespace(cuda_stream=77, device_index=1))
        assert machine.calls.pop() == (name, 1, 77)


@pytest.mark.parametrize("name", ENTRIES)
@pytest.mark.parametrize("other", [0, -1])
def test_tensors_of_other_devices_are_refused(machine, name, other):
    """-1: a host tensor."""
    for odd in ENTRIES[name]():
        tensors = ENTRIES[name]()
        tensors[odd].at, tensors[odd].is_cuda = other, other >= 0
        with pytest.raises(ValueError):
            call(name, tensors)
        assert machine.calls == []


@pytest.mark.parametrize("name", ENTRIES)
def test_streams_of_other_devices_are_refused(machine, name):
    with pytest.raises(ValueError):
        call(name, ENTRIES[name](), types.SimpleNamespace(cuda_stream=77, device_index=0))
    assert machine.calls == []


def test_workspace_size_is_the_caches_devices(machine):
    binding.moe_kv_attention_workspace_size(CACHE, 5, 4)
    assert machine.calls[0][1] == 1
