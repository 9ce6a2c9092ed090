"""The binding of the operators between the projections, on the host: what it hands to the library and
where, with stand-ins for tensors, devices and the library."""
import pytest
import torch

import weight_only_quantized_tma_gb300 as wq
from weight_only_quantized_tma_gb300 import _attn, _lib


class Stub(torch.Tensor):
    """A tensor on a device that this machine need not have: shape, type and strides, no data."""

    @staticmethod
    def __new__(cls, shape, dtype, device="cuda:1"):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    def data_ptr(self):
        return 0x10000

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} on a stand-in")


class Machine:
    """A library that notes its calls and the device that is current in them."""

    def __init__(self, monkeypatch, need=1000):
        self.device, self.calls, self.zeroed, self.status_bits = 0, [], [], 0
        machine = self

        class on:
            def __init__(self, device):
                self.to = torch.device(device).index if not isinstance(device, int) else device

            def __enter__(self):
                self.back, machine.device = machine.device, self.to

            def __exit__(self, *a):
                machine.device = self.back

        class library:
            def __getattr__(self, name):
                def call(*args):
                    machine.calls.append((name, machine.device, args))
                    if name == "wq_attn_kv4_workspace_bytes":
                        args[-1]._obj.value = need
                    if name == "wq_kv4_page_bytes":
                        args[-1]._obj.value = 1
                    if name == "wq_device_status":
                        args[-1]._obj.value = machine.status_bits
                        return 9 if machine.status_bits & 63 else 10 if machine.status_bits else 0
                    if name == "wq_clear_device_status":
                        machine.status_bits = 0
                    return 0
                return call

        def zeros(n, dtype=None, device=None):
            self.zeroed.append((n, torch.device(device).index))
            return Stub((n,), dtype, device)

        fake = library()
        monkeypatch.setattr(_attn, "lib", lambda: fake)
        monkeypatch.setattr(_lib, "lib", lambda: fake)
        monkeypatch.setattr(_attn, "_fns", {})
        monkeypatch.setattr(_attn, "_ws_need", {})
        monkeypatch.setattr(_attn, "_ws_cache", {})
        monkeypatch.setattr(_lib, "_ws_cache", {})
        monkeypatch.setattr(_attn, "_stream", lambda device: 40 + device.index)
        monkeypatch.setattr(_attn, "_current", lambda: self.device, raising=False)
        monkeypatch.setattr(_attn, "_several", None, raising=False)
        monkeypatch.setattr(torch.cuda, "device_count", lambda: 4)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.device)
        monkeypatch.setattr(torch.cuda, "device", on)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.device == self.capturing)
        monkeypatch.setattr(torch, "zeros", zeros)
        self.capturing = None


@pytest.fixture
def machine(monkeypatch):
    return Machine(monkeypatch)


H = torch.float16


def _arguments(device):
    q, k = Stub((4, 2, 64), H, device), Stub((4, 1, 64), H, device)
    pages = Stub((3, 1, 16 * (64 + 8 * 2)), torch.uint8, device)
    i64 = Stub((4,), torch.int64, device)
    table, lens = Stub((4, 2), torch.int32, device), Stub((4,), torch.int32, device)
    cs = Stub((8, 64), torch.float32, device)
    return {
        "wq_qk_norm_rope": lambda: wq.wq_qk_norm_rope(q, k, i64, cs, q_out=q, k_out=k),
        "wq_kv4_write": lambda: wq.wq_kv4_write(k, k, i64, pages, 32, 16),
        "wq_kv4_read": lambda: wq.wq_kv4_read(pages, i64, 64, 32, 16, H, k=k, v=k),
        "wq_attn_kv4": lambda: wq.wq_attn_kv4(q, pages, table, lens, 32, 16, out=q),
    }


@pytest.mark.parametrize("name", ["wq_qk_norm_rope", "wq_kv4_write", "wq_kv4_read", "wq_attn_kv4"])
@pytest.mark.parametrize("own", [0, 1, 3])
def test_the_library_runs_on_the_tensors_device(machine, name, own):
    """Whichever device is current: it takes SM count, status word and launch from the current one."""
    _arguments(f"cuda:{own}")[name]()
    assert machine.calls[-1][0] == name and machine.calls[-1][2][-1] == 40 + own
    assert [d for _, d, _ in machine.calls] == [own] * len(machine.calls)
    assert machine.device == 0 and all(d == own for _, d in machine.zeroed)


def test_capture_is_asked_of_the_tensors_device(machine):
    machine.capturing = 1
    _arguments("cuda:1")["wq_attn_kv4"]()
    assert not _attn._ws_cache      # the graph's own workspace
    _arguments("cuda:0")["wq_attn_kv4"]()
    assert list(_attn._ws_cache) == [(0, 40)]


@pytest.mark.parametrize("clear", [False, True])
@pytest.mark.parametrize("bits,timeout", [(0, False), (1 << 6, False), (1 << 1, True), (1 << 6 | 1 << 3, True)])
def test_a_timeout_clears_the_arrival_counters(machine, monkeypatch, bits, timeout, clear):
    """A kernel that gave up may leave counters that are not zero: later calls must not count from there.
    Workspaces of other devices stay as they are, and so do all of them after an index out of range."""
    zeroed = []
    monkeypatch.setattr(_lib, "_ws_caches", [_lib._ws_cache, _attn._ws_cache], raising=False)
    monkeypatch.setattr(_lib, "_zero_counters", lambda buf: zeroed.append(id(buf)), raising=False)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda: zeroed.append("wait"))
    for own in (0, 1):
        _arguments(f"cuda:{own}")["wq_attn_kv4"]()
        _lib._ws_cache[(own, 7)] = torch.zeros(1 << 20, dtype=torch.uint8, device=f"cuda:{own}")
    machine.status_bits = bits
    if clear:
        wq.wq_clear_device_status()
        assert machine.status_bits == 0
    else:
        assert wq.wq_device_status() == bits
    mine = [id(_lib._ws_cache[(0, 7)]), id(_attn._ws_cache[(0, 40)])]
    assert zeroed == (["wait", *mine, "wait"] if timeout else [])


def test_every_cache_of_workspaces_is_known():
    assert any(c is _attn._ws_cache for c in _lib._ws_caches) and any(c is _lib._ws_cache for c in _lib._ws_caches)


BIG = 1 << 32     # what an int32 drops


@pytest.mark.parametrize("name", ["group", "page_size", "head_dim", "kv_heads"])
def test_sizes_that_would_wrap_are_refused(machine, name):
    sizes = dict(kv_heads=1, head_dim=64, group=32, page_size=16)
    sizes[name] += BIG
    with pytest.raises(ValueError):
        wq.wq_kv4_page_bytes(**sizes)
    # pages of the size that Python's own arithmetic asks for: with a group beyond the head, smaller than
    # the library's pages of group 32
    block = sizes["page_size"] * (sizes["head_dim"] + 8 * (sizes["head_dim"] // sizes["group"]))
    pages = Stub((3, sizes["kv_heads"], block), torch.uint8)
    k = Stub((4, sizes["kv_heads"], sizes["head_dim"]), H)
    with pytest.raises(ValueError):
        wq.wq_kv4_read(pages, Stub((4,), torch.int64), sizes["head_dim"], sizes["group"], sizes["page_size"], H, k=k, v=k)
    assert not machine.calls


def test_counts_beyond_every_sequence_do_not_wrap(machine):
    q, pages = Stub((4, 2, 64), H), Stub((3, 1, 16 * 80), torch.uint8)
    table, lens, cu = Stub((4, 2), torch.int32), Stub((4,), torch.int32), Stub((5,), torch.int32)
    for given, max_q, window in ((5, 5, 5), (BIG + 5, (1 << 31) - 1, (1 << 31) - 1), (-BIG, 0, -1), (-(1 << 64) + 5, 0, -1)):
        wq.wq_attn_kv4(q, pages, table, lens, 32, 16, cu_q=cu, max_q=given, window=given, out=q)
        name, _, args = machine.calls[-1]
        assert name == "wq_attn_kv4" and (args[6], args[14]) == (max_q, window)


def test_workspace_bytes(machine):
    pages = Stub((3, 1, 16 * 80), torch.uint8)
    assert wq.wq_attn_kv4_workspace_bytes(pages, 2, 64, 32, 16, H, max_q=BIG) == 1000
    name, device, args = machine.calls[-1]
    assert name == "wq_attn_kv4_workspace_bytes" and device == 1 and args[1:3] == (2, (1 << 31) - 1)
    for bad in (dict(q_heads=2 + BIG), dict(group=64), dict(page_size=32), dict(head_dim=128), dict(dtype=torch.float32)):
        with pytest.raises(ValueError):
            wq.wq_attn_kv4_workspace_bytes(**{**dict(pages=pages, q_heads=2, head_dim=64, group=32, page_size=16, dtype=H),
                                              **bad})
