"""How the work of the attention over the 8-bit cache is dealt (CPU only): the
kernels' header with their own item costs, items and limits to the live rows, and
what the loads' lanes compute ahead of the last key."""
import ctypes
import random
import subprocess

import pytest

import test_cache4_work as base
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


# Goes through a call as the kernels do: `threads` threads sum up shares of the
# pairs, a block seeks its first segment and walks on.
DEAL = r"""
#include "fa_cache4_work.h"
using namespace fa;
extern "C" int deal(int B, int Hkv, int T, int window, int heads, int rows, int max_len,
                    const int* lens, const int* q_lens, int grid, int threads, int* seg,
                    int seg_room, int* join, int cost, int least, int most) {
  const int live = heads * T < most ? heads * T : most;
  c4::Call c = {B, Hkv, T, window, heads, rows, (live - 1) / rows + 1, max_len,
                FastDiv::of(heads)};
  c.least_rows = least, c.most_rows = most, c.item_cost = cost;
  auto read = [&](int b) { return c4::request_of(c, lens[b], q_lens ? q_lens[b] : T); };
  const int pairs = B * c.row_blocks, per = (pairs - 1) / threads + 1;
  auto first_pair = [&](int t) { return pairs < t * per ? pairs : t * per; };
  long long total = 0;
  for (int t = 0; t < threads; ++t) total += c4::cost_of(c, read, first_pair(t), first_pair(t + 1));
  const c4::Shares shares(total * Hkv, grid);
  int n = 0;
  for (int block = 0; block < grid; ++block) {
    join[5 * block] = -1;
    if (block >= shares.blocks) continue;
    const long long u0 = shares.first(block);
    c4::Cursor at;
    int into = -1;
    long long before = 0;
    for (int t = 0; t < threads; ++t) {
      const long long upto = before + c4::cost_of(c, read, first_pair(t), first_pair(t + 1));
      if (u0 >= before * Hkv && u0 < upto * Hkv) {
        if (into >= 0) return -1;
        into = at.seek(c, read, first_pair(t), u0 - before * Hkv,
                       (int)(shares.first(block + 1) - u0));
      }
      before = upto;
    }
    if (into < 0) return -2;
    if (at.end == at.unit) continue;
    int last, part;
    if (c4::join_of(shares, at, block, u0, into, &last, &part)) {
      const int j[5] = {at.b, at.rb, at.hk, last, part};
      for (int i = 0; i < 5; ++i) join[5 * block + i] = j[i];
    }
    int i = 0;
    do {
      if (n == seg_room) return -3;
      const int v[10] = {block, i++, at.b, at.rb, at.hk, at.unit, at.end, at.k.units, at.k.lo, at.k.hi};
      for (int x = 0; x < 10; ++x) seg[10 * n + x] = v[x];
      ++n;
    } while (at.next(c, read));
  }
  return n;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("work8"), "deal", DEAL)


class Kernel:
    """Stands in for the 4-bit harness: the same call with this kernel's cost and
    limits, and with all requests' new tokens (the checked ones are its own)."""

    def __init__(self, lib, cost, threads, least, most, q_lens):
        self.lib, self.cost, self.threads = lib, cost, threads
        self.least, self.most = least, most
        self.q_lens = None if q_lens is None else (ctypes.c_int * len(q_lens))(*q_lens)

    def deal(self, B, Hkv, T, window, heads, rows, max_len, lens, q_lens, grid, threads, seg,
             room, join):
        return self.lib.deal(B, Hkv, T, window, heads, rows, max_len, lens, self.q_lens, grid,
                             self.threads, seg, room, join, self.cost, self.least, self.most)


# Item cost, threads that sum, rows of an item, blocks.
NARROW = (1, 128, [8, 16, 24, 32, 40], [1, 40, 304, 456])
TURNS = (4, 512, [128], [1, 148, 152, 160])
WIDE = (4, 512, [256], [1, 148, 152, 160])


def go_through(lib, rng, kind, least, most):
    cost, threads, items, grids = kind
    B = rng.choice([1, 2, 3, 7, 40, 200])
    heads, T = rng.choice([1, 2, 3, 8, 16, 64]), rng.choice([1, 2, 5, 33, 130, 300])
    if B > 7:
        T = min(T, 5)
    if kind is TURNS:
        T = min(T, 128 // heads)
    top = rng.choice([1, 3, 40, 700, 5000])  # (1 and 3: shares below an item's cost)
    lens = [rng.randint(-1, top) for _ in range(B)]
    q_lens = rng.choice([None, [rng.randint(-1, T + 1) for _ in range(B)],
                         [T if i == 0 else 1 for i in range(B)]])
    new = [T if q_lens is None else min(max(q_lens[b], 0), T) for b in range(B)]
    mine = [n if least <= n * heads <= most else 0 for n in new]
    base.check(Kernel(lib, cost, threads, least, most, q_lens), rng.choice([1, 2, 8]), T,
               rng.choice([-1, -1, 0, 1, 31, 200, 4999]), heads, rng.choice(items), lens, mine,
               rng.choice(grids), rng.choice([1 << 20, 640]))


@pytest.mark.parametrize("kind", [NARROW, TURNS, WIDE], ids=["narrow", "turns", "wide"])
@pytest.mark.parametrize("seed", range(10))
def test_every_key_once_and_every_part_joined(lib, kind, seed):
    rng = random.Random(seed)
    for _ in range(25):
        least, most = 0, (1 << 31) - 1
        if rng.random() < 0.5:             # the other kernel has the other requests
            limit = rng.choice([8, 16, 48, 64])
            least, most = (0, limit) if kind is NARROW else (limit + 1, most)
        go_through(lib, rng, kind, least, most)


@pytest.mark.parametrize("kind", [NARROW, TURNS, WIDE], ids=["narrow", "turns", "wide"])
def test_shares_of_nothing_but_an_item_s_cost(lib, kind):
    """More blocks than units: a share may end before its item's first unit."""
    cost, threads, items, grids = kind
    for B in range(1, 60):
        for length in (1, 128, 129, 300):
            base.check(Kernel(lib, cost, threads, 0, (1 << 31) - 1, None), 1, 1, -1, 1, items[-1],
                       [length] * B, None, grids[-1])
