"""How the work of the attention over the 8-bit cache is dealt (CPU only): the
kernels' header with their own item costs, items and limits to the live rows, and
what the loads' lanes compute ahead of the last key."""
import ctypes
import random
import subprocess

import pytest

from tiled_attention_bwd_gb300 import build as fa_build

AHEAD = r"""
#include "fa_cache4_work.h"
extern "C" unsigned token(int lo, int unit, int group) { return fa::c4::group_token(lo, unit, group); }
"""
SANITIZED = ["-fsanitize=undefined", "-static-libubsan", "-fno-sanitize-recover=undefined"]


def compiled(d, name, text):
    src, lib = d / (name + ".cpp"), d / (name + ".so")
    src.write_text(text)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", *SANITIZED,
                    "-I", fa_build.CSRC, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def test_groups_ahead_of_the_last_key(tmp_path):
    """Up to the longest table that a call may have, and 31 units on."""
    token = compiled(tmp_path, "ahead", AHEAD).token
    token.restype = ctypes.c_uint
    rng = random.Random(1)
    for end in (1, 4000, 2 ** 31 - 258, 2 ** 31 - 1):
        for _ in range(200):
            lo = rng.choice([0, rng.randrange(end)]) // 32 * 32
            units = -(-(end - lo) // 128)
            first = rng.choice([0, units - 1, max(0, units - 4)])
            for ahead in range(32):
                for group in (0, 3, 7):
                    assert token(lo, first + ahead, group) == lo + (first + ahead) * 128 + group * 16
