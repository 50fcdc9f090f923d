"""How the cache attention's work is dealt to blocks (CPU only): the kernel's
own header, compiled as plain C++ and gone through for whole calls.

Every key that a live row sees is worked once, by the one segment whose unit
holds it; nothing else is worked; and the join reads exactly the partial
results that were written.
"""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from tiled_attention_bwd_gb300 import build as fa_build

HARNESS = r"""
#include "fa_cache4_work.h"
using namespace fa;
extern "C" int deal(int B, int Hkv, int T, int window, int heads, int rows, int max_len,
                    const int* lens, const int* q_lens, int grid, int threads, int* seg,
                    int seg_room, int* join) {
  const c4::Call c = {B, Hkv, T, window, heads, rows, (heads * T - 1) / rows + 1, max_len,
                      FastDiv::of(heads)};
  auto read = [&](int b) { return c4::request_of(c, lens[b], q_lens ? q_lens[b] : T); };
  const int pairs = B * c.row_blocks, per = (pairs - 1) / threads + 1;
  long long total = 0;
  for (int t = 0; t < threads; ++t) {
    const int p0 = pairs < t * per ? pairs : t * per, p1 = pairs < p0 + per ? pairs : p0 + per;
    total += c4::cost_of(c, read, p0, p1);
  }
  const c4::Shares s(total * Hkv, grid);
  int n = 0;
  for (int k = 0; k < grid; ++k) {
    join[5 * k] = -1;
    if (k >= s.blocks) continue;
    const long long u0 = s.first(k);
    c4::Cursor at;
    int into = -1;
    long long before = 0;
    for (int t = 0; t < threads; ++t) {
      const int p0 = pairs < t * per ? pairs : t * per, p1 = pairs < p0 + per ? pairs : p0 + per;
      const long long upto = before + c4::cost_of(c, read, p0, p1);
      if (u0 >= before * Hkv && u0 < upto * Hkv) {
        if (into >= 0) return -1;
        into = at.seek(c, read, p0, u0 - before * Hkv, (int)(s.first(k + 1) - u0));
      }
      before = upto;
    }
    if (into < 0) return -2;
    if (at.end == at.unit) continue;
    int last, part;
    if (c4::join_of(s, at, k, u0, into, &last, &part)) {
      const int j[5] = {at.b, at.rb, at.hk, last, part};
      for (int i = 0; i < 5; ++i) join[5 * k + i] = j[i];
    }
    int i = 0;
    do {
      if (n == seg_room) return -3;
      const int v[10] = {k, i++, at.b, at.rb, at.hk, at.unit, at.end, at.k.units, at.k.lo, at.k.hi};
      for (int x = 0; x < 10; ++x) seg[10 * n + x] = v[x];
      ++n;
    } while (at.next(c, read));
  }
  return n;
}
extern "C" unsigned fast_div(unsigned by, unsigned x) { return FastDiv::of(by).div(x); }
"""


@pytest.fixture(scope="module")
def work(tmp_path_factory):
    d = tmp_path_factory.mktemp("work")
    src, lib = d / "work.cpp", d / "work.so"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-fsanitize=undefined",
                    "-static-libubsan", "-fno-sanitize-recover=undefined",
                    "-I", fa_build.CSRC, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def deal(work, Hkv, T, window, heads, rows, lens, q_lens, grid, max_len=1 << 20):
    B = len(lens)
    arr = lambda x: None if x is None else (ctypes.c_int * len(x))(*x)  # noqa: E731
    room = 2 * grid + B * Hkv * ((heads * T - 1) // rows + 1) + 8
    seg, join = (ctypes.c_int * (10 * room))(), (ctypes.c_int * (5 * grid))()
    n = work.deal(B, Hkv, T, window, heads, rows, max_len, arr(lens), arr(q_lens),
                  grid, 128, seg, room, join)
    assert n >= 0, n
    return (np.array(seg[:10 * n]).reshape(n, 10).tolist(),
            np.array(join).reshape(grid, 5).tolist())


def needed(T, window, heads, rows, length, ql):
    """By row block with a live row: the keys that its live rows see, from a
    multiple of 32 on, as (lo, hi); hi = lo = 0 where they see none."""
    out = []
    for r0 in range(0, ql * heads, rows):
        pos = [length - ql + r // heads for r in range(r0, min(ql * heads, r0 + rows))]
        lo = [0 if window < 0 else max(0, p - window) for p in pos if p >= 0]
        hi = [p + 1 for p in pos if p >= 0]
        out.append((min(lo) // 32 * 32, max(hi)) if hi else (0, 0))
    return out


def check(work, Hkv, T, window, heads, rows, lens, q_lens, grid, max_len=1 << 20):
    segs, joins = deal(work, Hkv, T, window, heads, rows, lens, q_lens, grid, max_len)
    want = {}
    for b, n in enumerate(lens):
        n = min(max(n, 0), max_len)
        ql = T if q_lens is None else min(max(q_lens[b], 0), T)
        for rb, keys in enumerate(needed(T, window, heads, rows, n, ql)):
            for hk in range(Hkv):
                want[b, rb, hk] = keys
    seen, parts = {}, {}
    for k, i, b, rb, hk, unit, end, units, lo, hi in segs:
        assert (lo, hi) == want[b, rb, hk] or lo >= hi == want[b, rb, hk][1] == 0
        assert units == max(1, -(-(hi - lo) // 128)) and 0 <= unit < end <= units
        seen.setdefault((b, rb, hk), []).extend(range(unit, end))
        if (unit, end) != (0, units):
            slot = 2 * k + (1 if i else 0)
            assert slot not in parts
            parts[slot] = (b, rb, hk)
    assert set(seen) == set(want)
    for (b, rb, hk), u in seen.items():
        lo, hi = want[b, rb, hk]
        assert u == list(range(max(1, -(-(hi - lo) // 128))))
    read = {}
    for k, (b, rb, hk, last, first) in enumerate(joins):
        if b < 0:
            continue
        for slot in [first] + [2 * c for c in range(k, last + 1)]:
            assert parts.pop(slot) == (b, rb, hk)
        assert (b, rb, hk) not in read
        read[b, rb, hk] = k
    assert not parts
    return sum(len(u) for u in seen.values())


def test_division(work):
    rng = random.Random(0)
    work.fast_div.restype = ctypes.c_uint
    for by in [1, 2, 3, 5, 7, 8, 31, 1 << 20, (1 << 31) - 1] + [rng.randint(1, 1 << 31) for _ in range(300)]:
        for x in [0, 1, by - 1, by, min(by * 7, (1 << 31) - 1), (1 << 31) - 1] + [
                rng.randrange(1 << 31) for _ in range(20)]:
            if x < 1 << 31:
                assert work.fast_div(by, x) == x // by, (by, x)


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(work, seed):
    rng = random.Random(seed)
    for _ in range(25):
        B = rng.choice([1, 2, 3, 7, 40, 200])
        heads, T = rng.choice([1, 2, 3, 5, 8, 16]), rng.choice([1, 1, 2, 3, 5, 33, 130])
        if B > 7 and T > 5:
            T = 3
        top = rng.choice([1, 40, 700, 5000])
        lens = [rng.randint(-1, top) for _ in range(B)]
        q_lens = rng.choice([None, [rng.randint(-1, T + 1) for _ in range(B)],
                             [T if i == 0 else min(1, T) for i in range(B)]])
        check(work, rng.choice([1, 2, 8]), T, rng.choice([-1, -1, 0, 1, 31, 200, 4999]), heads,
              rng.choice([8, 16, 24, 32, 40]), lens, q_lens, rng.choice([1, 2, 40, 304, 456]),
              rng.choice([1 << 20, 640]))


def test_nothing_to_do(work):
    assert check(work, 2, 4, -1, 3, 8, [5, 9], [0, -1], 304) == 0


def test_rows_without_a_new_token_cost_nothing(work):
    """One request with a chunk of 512 tokens beside 63 with one token each:
    those are worked as in a call for one token."""
    lens = [4096 + 7 * i for i in range(64)]
    one = check(work, 8, 1, -1, 8, 32, lens[1:], None, 304)
    chunk = check(work, 8, 512, -1, 8, 32, lens[:1], None, 304)
    assert check(work, 8, 512, -1, 8, 32, lens, [512] + [1] * 63, 304) == one + chunk


def test_a_chunk_is_worked_up_to_its_diagonal(work):
    """A prompt of 2048 tokens without history: the row blocks' units are those
    of a triangle, not of a square."""
    units = check(work, 1, 2048, -1, 8, 32, [2048], None, 304)
    assert units == sum(-(-4 * (i + 1) // 128) for i in range(512))
    # With a window, a band's.
    units = check(work, 1, 2048, 256, 8, 32, [2048], None, 304)
    assert units <= 512 * 4


def test_counts_past_32_bits(work):
    """400 requests of nearly 2^31 keys: more than 2^32 units."""
    n = (1 << 31) - 64
    segs, _ = deal(work, 1, 1, -1, 1, 8, [n] * 400, None, 304, n)
    units = [0] * 400
    for _, _, b, _, _, unit, end, _, _, _ in segs:
        assert unit == units[b]
        units[b] = end
    assert units == [1 << 24] * 400
