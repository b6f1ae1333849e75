"""Host checks of the binding's own workspaces (workspace="auto"), with
torch's allocator, streams and capture state, and the library's entry point,
replaced by stand-ins on the CPU: no GPU needed."""
from __future__ import annotations

import contextlib
import ctypes
import threading
import time

import pytest
import torch

import block_scaled_precision_mm_amd as mx

A = 0x10000             # an operand's address, never dereferenced
COUNTERS = 65536        # bytes of a workspace that have to be zero before a call
# K splits over workgroups, with a larger workspace for the second
SMALL, LARGE = (128, 4096, 14336), (512, 4096, 14336)


class Gpu:
    """What the binding sees of torch.cuda: a current stream, streams that are
    being captured, and the tensors it made, each with the stream that was
    current and whether that one was being captured."""

    def __init__(self, monkeypatch):
        self.current, self.capturing, self.made, self.calls = 7, set(), [], []
        real_zeros, real_empty = torch.zeros, torch.empty

        def make(real):
            def f(*a, device=None, **kw):
                t = real(*a, **kw)
                if real is real_empty:
                    t.fill_(0xAB)
                self.made.append((t, self.current, self.current in self.capturing))
                return t
            return f

        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s
            yield
            self.current = before

        monkeypatch.setattr(torch, "zeros", make(real_zeros))
        monkeypatch.setattr(torch, "empty", make(real_empty))
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, **kw: ptr)
        monkeypatch.setattr(mx, "_is_capturing", lambda: self.current in self.capturing, raising=False)
        monkeypatch.setattr(mx, "_current_device", lambda: 0)
        monkeypatch.setattr(mx, "_raw_stream", lambda device: self.current)
        monkeypatch.setattr(mx, "_WORKSPACES", {})
        monkeypatch.setattr(mx._lib, "mx_scaled_mm_fp4", self.launch)

    def launch(self, *args):
        ptr, size, stream = args[-3:]
        counters = (ctypes.c_uint8 * COUNTERS).from_address(ptr)
        assert not any(counters), "counters that are not zero"
        if stream in self.capturing:        # recorded, and not run before the next call
            counters[0] = 1
        self.calls.append((ptr, size))
        return 0

    def call(self, shape, stream=None):
        mx.mx_scaled_mm_fp4(A, A, A, A, A, *shape, out_dtype=0, stream=stream)
        return self.calls[-1]

    def owner(self, ptr):
        return next(i for i in range(len(self.made) - 1, -1, -1)
                    if self.made[i][0].data_ptr() <= ptr < self.made[i][0].data_ptr() + self.made[i][0].numel())


@pytest.fixture
def gpu(monkeypatch):
    return Gpu(monkeypatch)


def test_eager_calls_of_a_stream_share_one(gpu):
    a, b = gpu.call(SMALL), gpu.call(SMALL)
    assert a == b and a[1] >= mx.mx_scaled_mm_workspace_bytes(True, *SMALL)
    c = gpu.call(LARGE)
    assert c[1] >= mx.mx_scaled_mm_workspace_bytes(True, *LARGE) > a[1]
    assert gpu.call(SMALL) == c
    assert gpu.call(SMALL, stream=8)[0] != c[0]
    assert gpu.made[gpu.owner(gpu.calls[-1][0])][1] == 8        # made on the stream that uses it


def test_a_captured_call_has_one_of_its_own(gpu):
    # not the stream's, which a later, larger call replaces while the graph keeps its address
    warm = gpu.call(SMALL)
    gpu.capturing.add(7)
    captured = gpu.call(SMALL)
    assert captured[0] != warm[0]
    i = gpu.owner(captured[0])
    assert gpu.made[i][1:] == (7, True)     # of the captured graph's memory
    gpu.capturing.clear()
    assert gpu.call(SMALL) == warm          # and the stream's is not the graph's
    gpu.call(LARGE)
    assert all(t is not gpu.made[i][0] for t in mx._WORKSPACES.values())


def test_every_captured_call_clears_its_counters_itself(gpu):
    # two graphs captured on one stream may be replayed in any order
    gpu.capturing.add(7)
    gpu.call(SMALL)
    gpu.call(SMALL)
    gpu.call(LARGE)
    gpu.capturing.clear()
    gpu.call(SMALL)


def test_the_stream_of_the_call_counts_and_not_the_current_one(gpu):
    gpu.capturing.add(9)
    a = gpu.call(SMALL, stream=9)
    assert gpu.made[gpu.owner(a[0])][1:] == (9, True)
    assert gpu.made[gpu.owner(gpu.call(SMALL)[0])][1:] == (7, False)
    assert gpu.current == 7


@pytest.mark.parametrize("entry", ["mx_scaled_mm_fp4", "mx_scaled_mm_config"])
def test_calls_of_several_threads_do_not_share_one_at_a_time(gpu, monkeypatch, entry):
    # a call may launch twice, its second kernel reading what the first left in the workspace: no other call
    # of the stream's workspace may come between them, nor replace it before the launch
    inside, most, lock = {}, {}, threading.Lock()

    def launch(*args):
        stream = args[-1]
        with lock:
            inside[stream] = inside.get(stream, 0) + 1
            most[stream] = max(most.get(stream, 0), inside[stream])
        held = [t for t in mx._WORKSPACES.values() if t.data_ptr() == args[-3]]
        assert len(held) == 1, "not the workspace that the stream holds"
        time.sleep(0.002)
        with lock:
            inside[stream] -= 1
        return 0

    variant = mx.mx_default_config(True, *SMALL)[0]
    monkeypatch.setattr(mx._lib, entry, launch)
    failed = []

    def work(i):
        try:
            for n in range(8):
                if entry == "mx_scaled_mm_fp4":
                    mx.mx_scaled_mm_fp4(A, A, A, A, A, *(LARGE if (i + n) % 3 == 0 else SMALL), out_dtype=0, stream=7)
                else:
                    mx.mx_scaled_mm_config(True, A, A, A, A, A, *SMALL, variant, splits=2 + (i + n) % 3, out_dtype=0, stream=7)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed and most == {7: 1}


def test_a_refused_call_leaves_the_workspace_free(gpu, monkeypatch):
    monkeypatch.setattr(mx._lib, "mx_scaled_mm_fp4", lambda *args: -2)
    for _ in range(2):
        with pytest.raises(mx.MxGemmError):
            gpu.call(SMALL)
    monkeypatch.setattr(mx._lib, "mx_scaled_mm_fp4", gpu.launch)
    t = threading.Thread(target=gpu.call, args=(SMALL,), daemon=True)
    t.start()
    t.join(10)
    assert not t.is_alive() and len(gpu.calls) == 1
