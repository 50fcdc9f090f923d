"""Kernels that are launched while the work before them in the stream still
runs (CPU only: their sources).

Such a kernel's inputs may still be written when it starts, so it reads
global memory only behind wait_for_stream(), and by loads that the compiler
keeps behind it.  A load through the read-only path (__ldg, a const
__restrict__ pointer, ld.global.nc) promises that nobody writes the data
during the kernel's whole life, and may be moved ahead of the wait.
"""
import os
import re

import pytest

from tiled_attention_bwd_gb300 import build as fa_build


def source(name):
    text = open(os.path.join(fa_build.CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


OVERLAPPED = [f for f in fa_build.SOURCES
              if re.search(r"wait_for_stream\(\)", source(f))]


def test_the_kernels_are_found():
    assert {"fa_rope.cu", "fa_cache4.cu", "fa_cache4_attn.cu"} <= set(OVERLAPPED)


@pytest.mark.parametrize("name", OVERLAPPED + ["fa_serve.h", "fa_cache4.cuh"])
def test_no_read_only_loads(name):
    assert not re.search(r"__ldg\b|__restrict__|\.nc\b|ld_nc|__ldcs|__ldca",
                         source(name))


@pytest.mark.parametrize("name", OVERLAPPED)
def test_every_kernel_waits(name):
    """Each __global__ function calls wait_for_stream() once in its body."""
    text = source(name)
    starts = [m.start() for m in re.finditer(r"__global__", text)]
    assert starts
    for a, b in zip(starts, starts[1:] + [len(text)]):
        assert text[a:b].count("wait_for_stream()") == 1
