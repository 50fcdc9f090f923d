// fa_cache4_work.h -- how the cache attention's work is cut and dealt to
// blocks.  Plain C++ for both sides, so that it can be gone through on the CPU.
//
// The query rows of one request and key/value head are its T tokens times the
// G = H / Hkv heads that share it.  They are numbered by token first (row
// t G + h), so that a request's live rows, those of its q_lens new tokens, come
// first, and the rows of a row block are of neighbouring tokens.  A row block
// of R rows with one key/value head is an item.  It needs the keys that its
// live rows see and no others: those up to its last token's position and, with
// a window, from its first token's window on.  They are cut into units; an
// item counts as kC4ItemCost units more, for what it costs to begin and end
// one.  All items' units, in the order request, row block, head, are dealt to
// the blocks in equal consecutive shares.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define FA_BOTH __host__ __device__ __forceinline__
#else
#define FA_BOTH inline
#endif

namespace fa {

constexpr int kC4Unit = 128;    // keys of a unit
constexpr int kC4Align = 32;    // an item's first key is a multiple of it
constexpr int kC4ItemCost = 3;  // in units

// Division of 0 <= x < 2^31 by a number fixed at launch: three instructions
// instead of about twenty (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994).
struct FastDiv {
  uint32_t by, mul, shift;
  static FastDiv of(uint32_t by) {
    FastDiv f = {by, 0, 0};
    while (f.shift < 31 && (1u << f.shift) < by) ++f.shift;
    f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - by)) / by + 1);
    return f;
  }
  FA_BOTH uint32_t div(uint32_t x) const {
#ifdef __CUDA_ARCH__
    return (__umulhi(mul, x) + x) >> shift;
#else
    return (uint32_t)((((uint64_t)mul * x) >> 32) + x) >> shift;
#endif
  }
};

namespace c4 {

FA_BOTH int lesser(int a, int b) { return a < b ? a : b; }

// What a call deals with.
struct Call {
  int B, Hkv, T, window;  // window < 0: none
  int heads;              // G
  int rows;               // R
  int row_blocks;         // of T tokens: a request's most
  int max_len;            // tokens of a block table
  FastDiv by_heads;
  // (Most calls have one row block; a division costs 0.1 us of a short one.)
  FA_BOTH int request_of_pair(int at) const { return row_blocks == 1 ? at : at / row_blocks; }
};

struct Request {
  int len, ql;     // cached tokens, new tokens
  int row_blocks;  // with a live row
};
// From the values in memory, brought into range.
FA_BOTH Request request_of(const Call& c, int len, int n) {
  Request r;
  r.len = len < 0 ? 0 : lesser(len, c.max_len);
  r.ql = n < 0 ? 0 : lesser(n, c.T);
  r.row_blocks = r.ql == 0 ? 0 : (r.ql * c.heads - 1) / c.rows + 1;
  return r;
}

// The keys of a row block's items.
struct Keys {
  int lo, hi;  // lo: a multiple of kC4Align; behind the last token's
  int first;   // position of the first token, negative before the cache
  int units;
  FA_BOTH int cost() const { return units + kC4ItemCost; }
};
FA_BOTH Keys keys_of(const Call& c, const Request& r, int row_block) {
  const int row = row_block * c.rows, live = r.ql * c.heads - row;
  const int pos0 = r.len - r.ql;
  Keys k;
  k.first = pos0 + (int)c.by_heads.div(row);
  k.hi = pos0 + (int)c.by_heads.div(row + lesser(live, c.rows) - 1) + 1;
  if (k.hi < 0) k.hi = 0;
  // (With a window, first - window is above -2^31: the host checks that.)
  k.lo = c.window < 0 || k.first < c.window ? 0 : (k.first - c.window) & ~(kC4Align - 1);
  // Without keys one unit is left, which writes the empty rows.
  k.units = k.hi > k.lo ? (k.hi - k.lo - 1) / kC4Unit + 1 : 1;
  return k;
}

// Equal shares: `units` of cost dealt to blocks 0 .. blocks-1 in order, the
// first `more` blocks one more than the others' `least`.
struct Shares {
  long long least;
  int more, blocks;
  FA_BOTH Shares(long long units, int grid) {
    // No more blocks than units: every one that works has at least one.
    blocks = units < grid ? (int)units : grid;
    if (blocks == 0) {
      least = more = 0;
    } else if ((units >> 32) == 0) {
      least = (uint32_t)units / (uint32_t)blocks;
      more = (int)((uint32_t)units - (uint32_t)least * (uint32_t)blocks);
    } else {
      least = units / blocks;
      more = (int)(units - least * blocks);
    }
  }
  FA_BOTH long long first(int c) const { return least * c + lesser(c, more); }
  FA_BOTH int block_of(long long u) const {
    const long long big = (least + 1) * more;
    if ((u >> 31) == 0)
      return u < big ? (int)u / (int)(least + 1) : more + (int)(u - big) / (int)least;
    return (int)(u < big ? u / (least + 1) : more + (u - big) / least);
  }
};

// Pairs of request and row block, `at` = request * row_blocks + row block:
// what those from `at` up to `end` cost per head.  `read(b)` is request b.
template <typename Read>
FA_BOTH long long cost_of(const Call& c, Read read, int at, int end) {
  long long sum = 0;
  int b = c.request_of_pair(at), rb = at - b * c.row_blocks;
  for (; at < end; ++b, rb = 0) {
    const Request r = read(b);
    const int stop = lesser(r.row_blocks, rb + (end - at));
    at += c.row_blocks - rb;
    for (; rb < stop; ++rb) sum += keys_of(c, r, rb).cost();
  }
  return sum;
}

// A block's place in the list of items: the segment of the present item that
// is its own, units [unit, end).
struct Cursor {
  int b, rb, hk;  // the item's request, row block and key/value head
  int unit, end;
  int left;       // of the share, behind this segment
  Request r;
  Keys k;

  // The segment of the present item that begins `at` into its cost.
  FA_BOTH void segment(int at) {
    const int here = lesser(k.cost() - at, left), to = at + here;
    left -= here;
    unit = at < kC4ItemCost ? 0 : at - kC4ItemCost;
    end = to < kC4ItemCost ? 0 : to - kC4ItemCost;
  }
  // Goes to the item that holds place `u` of the pairs from `at` on, and its
  // segment of at most `share`; returns how far into the item's cost it is.
  template <typename Read>
  FA_BOTH int seek(const Call& c, Read read, int at, long long u, int share) {
    b = c.request_of_pair(at);
    rb = at - b * c.row_blocks;
    for (r = read(b);;) {
      if (rb < r.row_blocks) {
        k = keys_of(c, r, rb);
        const long long all = (long long)k.cost() * c.Hkv;
        if (u < all) break;
        u -= all;
        ++rb;
      } else {
        rb = 0;
        r = read(++b);
      }
    }
    hk = (u >> 31) == 0 ? (int)u / k.cost() : (int)(u / k.cost());
    const int into = (int)(u - (long long)hk * k.cost());
    left = share;
    segment(into);
    return into;
  }
  // The next item's; false if the share has none.
  template <typename Read>
  FA_BOTH bool next(const Call& c, Read read) {
    if (left == 0) return false;
    if (++hk == c.Hkv) {
      hk = 0;
      if (++rb == r.row_blocks) {
        rb = 0;
        do {
          if (++b >= c.B) return false;
          r = read(b);
        } while (r.row_blocks == 0);
      }
      k = keys_of(c, r, rb);
    }
    segment(0);
    return end > 0;  // (a share may end before an item's first unit)
  }
};

// What the join does for the item of a block's first segment, which begins
// at place u0, `into` its cost, where the item began in the block before: its
// last block, and the first of its partial results (block c's first segment
// leaves its own at 2 c, its last one at 2 c + 1).  False if there is nothing
// to join on behalf of this block.
FA_BOTH bool join_of(const Shares& s, const Cursor& at, int block, long long u0, int into,
                     int* last, int* first_part) {
  if (at.unit == 0) return false;
  const long long i0 = u0 - into, before = s.first(block - 1);
  if (before > i0 + kC4ItemCost) return false;
  *last = s.block_of(i0 + at.k.cost() - 1);
  *first_part = 2 * (block - 1) + (before < i0 ? 1 : 0);
  return true;
}

}  // namespace c4
}  // namespace fa
