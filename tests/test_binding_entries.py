"""The compiled binding's table of entry points: a call stays with the one it
began with (CPU only, on entry points that record)."""
import ctypes
import threading

import pytest
import torch

from tiled_attention_bwd_gb300 import build as fa_build
from tiled_attention_bwd_gb300 import fa


class Entries:
    """Entry points that count their calls; `inside`, if set, runs within the
    attention's workspace query or within the attention itself."""

    def __init__(self, lib):
        self.calls, self.in_size, self.in_call = 0, None, None
        for name in fa._NATIVE:
            real = getattr(lib, name)
            kind = ctypes.CFUNCTYPE(real.restype, *real.argtypes)
            f = self.size if name.endswith("_size") else self.call
            setattr(self, name, kind(lambda *a, f=f: f()))

    def size(self):
        if self.in_size:
            self.in_size()
        return 512

    def call(self):
        self.calls += 1
        if self.in_call:
            self.in_call()
        return 0


@pytest.fixture
def two():
    fa_build.build()
    lib = fa.load_library()
    native = fa._native()
    yield native, Entries(lib), Entries(lib)
    fa._connect(native, lib)


def attn():
    z = torch.zeros
    fa.fa_cache4_attn(z((1, 1, 1, 64), dtype=torch.bfloat16),
                      z((1, 1, 1, 18 * 64), dtype=torch.uint8),
                      z((1, 1), dtype=torch.int32), z(1, dtype=torch.int32), 0.1)


def test_a_call_keeps_its_entry_points(two):
    native, a, b = two
    fa._connect(native, a, host=True)
    a.in_size = lambda: fa._connect(native, b, host=True)
    attn()
    assert (a.calls, b.calls) == (1, 0)
    attn()
    assert (a.calls, b.calls) == (1, 1)


def test_another_thread_connects_while_a_call_runs(two):
    """The call has let go of the interpreter's lock and comes back to
    tensors that the new table would not take."""
    native, a, b = two
    fa._connect(native, a, host=True)

    def reconnect():
        t = threading.Thread(target=fa._connect, args=(native, b))
        t.start()
        t.join()

    a.in_call = reconnect
    attn()
    assert (a.calls, b.calls) == (1, 0)
    with pytest.raises(ValueError):        # b takes CUDA tensors only
        attn()
