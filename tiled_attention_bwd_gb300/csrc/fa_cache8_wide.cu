// fa_cache8_wide.cu -- the attention over the 8-bit cache for requests with
// many query rows (chunks of a prompt, many drafts): codes are made f16 once
// for up to 256 rows, and the products run on tcgen05.
//
// The division of work is that of fa_cache4_work.h with 256 rows to an item:
// two tiles of 128 rows (a token's heads next to one another), units of 128
// keys.  One block per SM, sixteen warps:
//   warps 0-7    softmax, tile 0 and tile 1; thread = row.  They also bring
//                the rows of Q, scaled by a power of two to f16 as in
//                fa_cache_attn.cuh, and write the results.
//   warps 8-11   make f16 tiles of K and V (128-byte swizzle) of a unit's
//                groups, 32 of its keys each
//   warp 12      deals out the segments and copies the groups of the next
//                units into shared memory
//   warp 13      issues S_t = Q_t K^T and O_t += P_t V, P_t f16 in TMEM
// While one tile's softmax runs, the tensor core works for the other.  In calls
// of up to 128 rows a request both tiles are of the same rows and take the units
// in turn, each with a maximum, sum and O of its own, which a segment's end joins
// (16 requests of 4096 to 8192 tokens x 8 heads, 128 rows: 102 us with one tile
// empty, so 84; 64 rows, which then went through the first kernel twice, 108 and
// 75).
//
// Products.  Codes are f16 values, so K and V enter exactly.  A group's power
// of two for K multiplies its 16 columns of S; the row's maximum is taken of
// s + e_v, and P = 2^(s + e_v - m + 8) in f16: as in fa_cache8_attn.cu, whose
// accuracy this kernel shares.
//
// What bounds it is each tile's chain S -> P -> P V -> next S, with two tiles in
// turn.  Of the 3500 cycles that a unit takes, a tile's softmax takes 1850 (the
// maximum 500, the exponentials 930, the stores of P 310); the products are 2048
// of the tensor pipe's (45 to 48% busy); the issuing warp waits for weights 15% of
// the time and for tiles 10%.  Issue slots are 46% busy, shared memory's banks 31%.
// 2 x 512 tokens (the second with 256) over 5000 and 16384, 64 heads over 8,
// d = 128: 222 us a call, 1.19 PFLOP/s; 2048 tokens over 32768: 1.24 PFLOP/s.  A
// launch begins cold: 20000 to 30000 cycles pass until the first unit's weights
// are there, most of them instruction fetches.  The roles share an instruction
// cache that their loops fill: the making warps' loops are not unrolled (292 us
// otherwise, so 270), the masks are bits, the issuing warp runs uniformly (below:
// 257, so 228).  One S for both tiles, with P apart so that Q K^T need not wait
// for P V, was slower (271): both softmaxes then run at once and share the same
// issue slots.  With one row block to a unit the making warps and the tiles' chains
// share the time (2900 cycles a unit); eight making warps, with the softmax's
// columns in two parts for their registers, gained nothing (64 rows 106 us, 100
// with four).
//
// NaN.  A hidden key is masked by selection.  A hidden value would reach a row
// as 0 * NaN: in units that some row does not see all of, NaN codes of V are
// taken as zero, and rows that do see them note their dims (in the workspace;
// rare) and write NaN at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fa_cache4_work.h"
#include "fa_cache8.cuh"
#include "fa_common.cuh"
#include "fa_serve.h"

namespace fa {
namespace {

constexpr int kThreads = 512;
constexpr int kMakeWarp = 8, kLoadWarp = 12, kMmaWarp = 13;
// Registers: launched at 128 a thread; the four warpgroups' shares add up to
// 512 * 128.
constexpr int kSoftmaxRegs = 200, kMakeRegs = 64, kCtrlRegs = 48;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kMakeRegs + 128 * kCtrlRegs <= kThreads * 128);
// TMEM columns, of the 512 that the block takes: S of each tile, O of each.
constexpr uint32_t kTmemS = 0, kTmemO = 256;
constexpr float kNoMax = -1e30f;  // m of a row that has seen no key
constexpr float kUp = 8.0f;       // P carries 2^kUp
constexpr float kSlack = 7.0f;    // growth of m that is left standing (f16 ends at 2^16)
constexpr int kUnitGroups = kC4Unit / kGroup;
constexpr int kItemCost = 4;  // what beginning and ending an item costs, in units
constexpr int kSegs = 4, kInfos = 4;

// Where-codes of the waits.
constexpr uint32_t kWLoadSeg = 0x531, kWLoadRaw = 0x532, kWMakeSeg = 0x533, kWMakeRaw = 0x534,
                   kWMakeTile = 0x535, kWMmaSeg = 0x536, kWMmaQ = 0x537, kWMmaTile = 0x538,
                   kWMmaP = 0x539, kWSmSeg = 0x53a, kWSmInfo = 0x53b, kWSmS = 0x53c,
                   kWSmO = 0x53d, kWSmMeet = 0x53e;

// A segment: some units of an item.
struct Seg {
  int b, hk, row0, live;   // live: rows of the item, from row0 on
  int pos0;                // position of the request's first new token
  int tok0, units;         // units < 0: no more segments
  int key_end;             // behind the last key that the item needs
  int plain_lo, plain_hi;  // tokens within are seen by every live row
  int whole, part;         // part: place of the partial results
};
// What the softmax needs of a group: factor of the keys and exponent of the
// values (read together), the exponent again and 2^-that.
struct alignas(16) Info {
  float2 key, value;
};

// kAlternate: items of 128 rows; the two tiles are of the same rows and take the
// units in turn.
template <int D, bool kAlternate>
struct Wide {
  static constexpr int kRows = kAlternate ? 128 : 256;
  static constexpr int kQTiles = kAlternate ? 1 : 2;
  static constexpr int kTileBytes = 128 * D * 2;
  // Of the ring of K and V tiles.  (A unit's notes, of which kInfos are kept, are
  // written behind the values of the unit before, whose place the values three or
  // four units back, or the keys two back, had: the softmax is done with the unit
  // kInfos back.)
  static constexpr int kStages = D == 128 ? (kAlternate ? 4 : 3) : 6;
  static constexpr int kRawStages = D == 128 ? 2 : 4;  // units on their way
  static constexpr int kRawBytes = kUnitGroups * group8_bytes(D);
  static constexpr int kRingOff = kQTiles * kTileBytes;  // (behind the Q tiles)
  static constexpr int kRawOff = kRingOff + kStages * kTileBytes;
  static constexpr int kCtrlOff = kRawOff + kRawStages * kRawBytes;
  struct Ctrl {
    uint64_t raw_full[kRawStages], raw_empty[kRawStages];
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t q_full[2], s_full[2], p_full[2], o_done[2], meet, mma_done;
    uint64_t seg_full[kSegs], seg_empty[kSegs], info_full[kInfos];
    Info info[kInfos][kUnitGroups];
    uint8_t nan[kInfos][kUnitGroups];  // 1: some value is NaN (in edge units)
    int edge[kInfos];                // 0: every live row sees all of the unit; else
                                     // 256 + (bit g: group g is there)
    int raw_there[kRawStages];
    Seg seg[kSegs];
    c4::Cursor at;  // of the loading warp
    int into;
    uint32_t abort, tmem;
  };
  static constexpr int kSmem = kCtrlOff + (int)sizeof(Ctrl) + 1024;  // + alignment
};
static_assert(Wide<128, false>::kSmem <= 232448 && Wide<64, false>::kSmem <= 232448);
static_assert(Wide<128, true>::kSmem <= 232448 && Wide<64, true>::kSmem <= 232448);

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return idesc_bf16(M, N, false, b_mn) & ~((1u << 7) | (1u << 10));  // A and B: f16
}
// The issuing warp runs its loop with all lanes and only the instructions
// themselves are predicated: addresses and descriptors then are uniform values,
// which tcgen05.mma takes from uniform registers.  (In a branch of one lane each
// has to be moved there.)  TMEM
// addresses are constants, all columns being this block's.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_ss_if(uint32_t who, uint32_t d, uint64_t a, uint64_t b,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
      "r"(idesc), "r"(accumulate), "r"(who)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t who, uint32_t d, uint32_t a, uint64_t b,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b),
      "r"(idesc), "r"(accumulate), "r"(who)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t who, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_addr(bar)), "r"(who)
      : "memory");
}
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t who, uint32_t s, uint64_t q, uint64_t k) {
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const uint32_t off = (i >> 2) * kSubTileBytes + (i & 3) * 32;
    mma_ss_if(who, s, sdesc_adv(q, off), sdesc_adv(k, off), idesc_f16(128, 128, false), i > 0);
  }
}
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t who, uint32_t o, uint32_t p, uint64_t v, bool accumulate) {
#pragma unroll
  for (int i = 0; i < kC4Unit / 16; ++i)
    mma_ts_if(who, o, p + i * 8, sdesc_adv(v, i * 2048), idesc_f16(128, D, true), accumulate || i > 0);
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint4 make8(uint32_t a, uint32_t b) {
  uint4 r;
  e4m3_to_f16(a, r.x, r.y);
  e4m3_to_f16(b, r.z, r.w);
  return r;
}
// 16 bytes, dims `dim` .. + 7 of row `row` of a tile.
__device__ __forceinline__ uint4* chunk_of(uint8_t* tile, int row, int dim) {
  return reinterpret_cast<uint4*>(tile + (dim >> 6) * kSubTileBytes + row * 128 +
                                  ((((dim >> 3) & 7) ^ (row & 7)) << 4));
}

// One group's keys into 16 rows of a K tile, `tile` being where the first stands
// (a multiple of eight rows: a lane's places are the same in each).  kAhead: with
// all loads before the first use.
template <int D, bool kAhead>
__device__ __forceinline__ void make_keys(uint8_t* tile, const uint8_t* grp, bool there, int lane) {
  const int g = lane >> 2, t = lane & 3;
  // Odd rows write their halves in the other order: eight lanes then write
  // eight different chunks.
  const bool odd = g & 1;
  uint8_t* const first = reinterpret_cast<uint8_t*>(chunk_of(tile, g, 8 * t + (odd ? 32 : 0)));
  uint8_t* const second = reinterpret_cast<uint8_t*>(chunk_of(tile, g, 8 * t + (odd ? 0 : 32)));
  uint4 ahead[2][D / 64];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      if (kAhead)
        ahead[h][c] = there ? *reinterpret_cast<const uint4*>(grp + k8_piece(D, h, c, lane)) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (kAhead) u = ahead[h][c];
      else if (there) u = *reinterpret_cast<const uint4*>(grp + k8_piece(D, h, c, lane));
      const int off = 8 * h * 128 + c * kSubTileBytes;
      *reinterpret_cast<uint4*>(first + off) = make8(odd ? u.z : u.x, odd ? u.w : u.y);
      *reinterpret_cast<uint4*>(second + off) = make8(odd ? u.x : u.z, odd ? u.y : u.w);
    }
}
// One group's values; in an edge unit NaN as zero.
template <int D>
__device__ __forceinline__ void make_values(uint8_t* tile, const uint8_t* grp, bool there,
                                            bool edge, int lane) {
  const int g = lane >> 2, t = lane & 3;
  uint8_t* to[2];  // of the lane's two tokens
#pragma unroll
  for (int e = 0; e < 2; ++e) to[e] = reinterpret_cast<uint8_t*>(chunk_of(tile, 2 * t + e, 8 * g));
  uint4 u[D / 64][2];
#pragma unroll
  for (int j = 0; j < D / 64; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      u[j][h] = there ? *reinterpret_cast<const uint4*>(grp + v8_piece(D, j, h, lane)) : make_uint4(0, 0, 0, 0);
  if (__builtin_expect(edge, 0)) {
    uint32_t* w = reinterpret_cast<uint32_t*>(u);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) w[i] &= ~__vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
  }
#pragma unroll
  for (int j = 0; j < D / 64; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t sel = e ? 0x7531 : 0x6420;  // one token's codes of a pair
        *reinterpret_cast<uint4*>(to[e] + 8 * h * 128 + j * kSubTileBytes) =
            make8(__byte_perm(u[j][h].x, u[j][h].y, sel), __byte_perm(u[j][h].z, u[j][h].w, sel));
      }
}
// Whether a group has a NaN value (the same on every lane).
template <int D>
__device__ __forceinline__ bool has_nan(const uint8_t* grp, int lane) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint4 u = *reinterpret_cast<const uint4*>(grp + 16 * D + (i * 32 + lane) * 16);
    for (uint32_t w : {u.x, u.y, u.z, u.w}) any |= __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
  }
  return __any_sync(0xffffffffu, any != 0);
}

// A wait of a whole warp.  kHook: with the failure-path test hook, which stops
// a warp at its site whether the barrier is complete or not (the first look at
// one may sleep until it is).
template <bool kHook>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const WaitCtl& wc,
                                          uint32_t where) {
  if (kHook && c_expire_site == where) {
    if ((threadIdx.x & 31) == 0) raise_abort(wc, where);
    __syncwarp();
    return false;
  }
  return __all_sync(0xffffffffu, wait_bar<true>(bar, parity, wc, where));
}

template <int kRows>
__device__ __forceinline__ c4::Call wide_call(const CacheAttnArgs& a) {
  c4::Call c = {a.B, a.Hkv, a.T, a.window, a.heads, kRows, a.row_blocks, a.M << a.shift, a.by_heads};
  c.least_rows = a.least_rows;
  c.most_rows = a.most_rows;
  c.item_cost = kItemCost;
  return c;
}
__device__ __forceinline__ size_t row_at(const CacheAttnArgs& a, int b, int hk, int row) {
  const int t = (int)a.by_heads.div(row), h = row - t * a.heads;
  return (((size_t)b * a.Hkv + hk) * a.heads + h) * a.T + t;
}
// A request's group that holds token `tok`, or null.
__device__ __forceinline__ const uint8_t* group_at(const CacheAttnArgs& a, int b, int hk, int tok,
                                                   int bytes) {
  const int page = a.block_table[(size_t)b * a.M + (tok >> a.shift)], gpp = a.shift - 4;
  if (page < 0 || page >= a.pages) return nullptr;
  return a.cache + ((((size_t)page * a.Hkv + hk) << gpp) + ((tok >> 4) & ((1 << gpp) - 1))) * bytes;
}

// Four words of a thread's row, at a column of TMEM.
__device__ __forceinline__ void tmem_st4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void tmem_ld4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

template <int D, bool kAlternate, bool kHook>
__global__ void __launch_bounds__(kThreads, 1) cache8_wide_kernel(CacheAttnArgs a) {
  using L = Wide<D, kAlternate>;
  using Ctrl = typename L::Ctrl;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  Ctrl* c = reinterpret_cast<Ctrl*>(smem + L::kCtrlOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < L::kRawStages; ++i) mbar_init(&c->raw_full[i], 1), mbar_init(&c->raw_empty[i], 4);
    for (int i = 0; i < L::kStages; ++i) mbar_init(&c->kv_full[i], 4), mbar_init(&c->kv_empty[i], 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&c->q_full[t], kAlternate ? 8 : 4), mbar_init(&c->s_full[t], 1);
      mbar_init(&c->p_full[t], 4), mbar_init(&c->o_done[t], 1);
    }
    mbar_init(&c->meet, 8), mbar_init(&c->mma_done, 1);
    // A segment is let go of by the making warps, the MMA thread and the
    // softmax warps.
    for (int i = 0; i < kSegs; ++i) mbar_init(&c->seg_full[i], 1), mbar_init(&c->seg_empty[i], 4 + 1 + 8);
    for (int i = 0; i < kInfos; ++i) mbar_init(&c->info_full[i], 4);
    c->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&c->tmem, 512);
    tmem_relinquish();
  }
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this block's share of the units
  const c4::Call call = wide_call<L::kRows>(a);
  auto read = [&](int b) {
    return c4::request_of(call, a.seq_lens[b], a.q_lens ? a.q_lens[b] : a.T);
  };
  long long* scan = reinterpret_cast<long long*>(smem);  // (before the tiles are in use)
  const int pairs = a.B * a.row_blocks, per = (pairs - 1) / kThreads + 1;
  const int p0 = (int)min((long long)pairs, (long long)tid * per), p1 = p0 + min(pairs - p0, per);
  const long long mine = c4::cost_of(call, read, p0, p1);
  long long upto = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, upto, m);
    if (lane >= m) upto += u;
  }
  if (lane == 31) scan[warp] = upto;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) upto += scan[w];
    total += scan[w];
  }
  const long long before = upto - mine;
  const c4::Shares shares(total * a.Hkv, gridDim.x);
  bool work = (int)blockIdx.x < shares.blocks;  // of the block
  const long long u0 = work ? shares.first(blockIdx.x) : 0;
  if (work && u0 >= before * a.Hkv && u0 < upto * a.Hkv)
    c->into = c->at.seek(call, read, p0, u0 - before * a.Hkv, (int)(shares.first(blockIdx.x + 1) - u0));
  __syncthreads();  // (the tiles are free, too)
  if (work && c->at.end == c->at.unit) work = false;  // a share of nothing but an item's cost
  if (tid == 0) {
    int4 j = make_int4(-1, 0, 0, 0);
    int last, first_part;
    if (work && c4::join_of(shares, c->at, blockIdx.x, u0, c->into, &last, &first_part))
      j = make_int4(c->at.b, c->at.hk * a.row_blocks + c->at.rb, last, first_part);
    a.joins[blockIdx.x] = j;
  }
  const WaitCtl wc = {a.st, &c->abort, a.timeout_ns};
  __syncthreads();  // every thread has seen the cursor

  if (warp >= kLoadWarp) {
    reg_dealloc<kCtrlRegs>();
    if (warp == kLoadWarp && work) {
      // ------------------------------------------------- segments and copies
      bool ok = true;
      int stage = 0, used = 0;  // used: stages that copies went into
      uint32_t phase = 0;
      for (int s = 0; ok; ++s) {
        Seg& seg = c->seg[s % kSegs];
        ok = wait_warp<kHook>(&c->seg_empty[s % kSegs], ((s / kSegs) & 1) ^ 1, wc, kWLoadSeg);
        if (!ok) break;
        if (lane == 0) {  // (the cursor stays in shared memory: registers are scarce)
          if (s > 0 && !c->at.next(call, read)) {
            seg.units = -1;
          } else {
            const c4::Cursor& at = c->at;
            seg.b = at.b, seg.hk = at.hk, seg.row0 = at.rb * L::kRows;
            seg.live = min(L::kRows, at.r.ql * a.heads - seg.row0);
            seg.pos0 = at.r.len - at.r.ql;
            seg.tok0 = at.k.lo + at.unit * kC4Unit;
            seg.units = at.end - at.unit;
            seg.key_end = at.k.hi;
            seg.plain_hi = at.k.first + 1;
            seg.plain_lo = a.window < 0 ? 0 : at.k.hi - 1 - a.window;
            seg.whole = at.unit == 0 && at.end == at.k.units;
            seg.part = 2 * blockIdx.x + (s == 0 ? 0 : 1);
          }
          mbar_arrive(&c->seg_full[s % kSegs]);
        }
        __syncwarp();
        const int units = seg.units;
        if (units < 0) break;
        // Each lane looks up one group of the next four units.
        for (int base = 0; base < units && ok; base += 4) {
          const int u = base + lane / kUnitGroups;
          const unsigned tok = c4::group_token(seg.tok0, u, lane % kUnitGroups);
          const uint8_t* src = nullptr;
          if (u < units && tok < (unsigned)seg.key_end) src = group_at(a, seg.b, seg.hk, tok, group8_bytes(D));
          const uint32_t have = __ballot_sync(0xffffffffu, src != nullptr);
          const int n = min(4, units - base);
#pragma unroll 1
          for (int q = 0; q < n; ++q) {
            ok = wait_warp<kHook>(&c->raw_empty[stage], phase ^ 1, wc, kWLoadRaw);
            if (!ok) break;
            const int mask = (have >> (q * kUnitGroups)) & 0xff;
            if (lane == 0) {
              c->raw_there[stage] = mask;
              if (mask) mbar_arrive_expect_tx(&c->raw_full[stage], __popc(mask) * group8_bytes(D));
              else mbar_arrive(&c->raw_full[stage]);
            }
            __syncwarp();
            if (lane / kUnitGroups == q && src)
              bulk_load(smem + L::kRawOff + stage * L::kRawBytes + lane % kUnitGroups * group8_bytes(D), src,
                        group8_bytes(D), &c->raw_full[stage]);
            used |= 1 << stage;
            if (++stage == L::kRawStages) stage = 0, phase ^= 1;
          }
        }
      }
      // The copies land before the block leaves, whether it stops or not.
      // (A stage's last phase is this one before the ring's present stage, the
      // one before from there on.)
#pragma unroll 1
      for (int i = 0; i < L::kRawStages; ++i)
        if ((used >> i) & 1) drain_bar<true>(&c->raw_full[i], i < stage ? phase : phase ^ 1, a.timeout_ns);
      __syncwarp();
    } else if (warp == kMmaWarp && work) {
      // --------------------------------------------------------- MMA issuer
      // Q and K: rows of 128 bytes along the dims; V: 64-dim columns of keys.
      const uint64_t q_desc = sdesc_sw128(smem_addr(smem), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_addr(smem + L::kRingOff), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_addr(smem + L::kRingOff), kSubTileBytes, 1024);
      const uint32_t who = elect_one();
      int stage = 0, u_seg = 0;  // u_seg: units of the segments before
      uint32_t phase = 0, q_par = 0, p_par = 0;  // bit t: of tile t
      bool ok = true;
      // A unit's K (half 0) or V tile, in the ring's order.
      auto tile_at = [&](int u, int half, int& st) {
        const uint32_t at = 2u * u + half;
        st = at % L::kStages;
        const bool r = wait_warp<kHook>(&c->kv_full[st], (at / L::kStages) & 1, wc, kWMmaTile);
        tc_fence_after();
        return r;
      };
      auto next_tile = [&](int& st) {
        st = stage;
        const bool r = wait_warp<kHook>(&c->kv_full[stage], phase, wc, kWMmaTile);
        if (++stage == L::kStages) stage = 0, phase ^= 1;
        tc_fence_after();
        return r;
      };
      for (int s = 0; ok; ++s) {
        ok = wait_warp<kHook>(&c->seg_full[s % kSegs], (s / kSegs) & 1, wc, kWMmaSeg);
        if (!ok) break;
        const int units = __shfl_sync(0xffffffffu, c->seg[s % kSegs].units, 0);
        const int tiles = __shfl_sync(0xffffffffu, c->seg[s % kSegs].live > 128 ? 2 : 1, 0);
        warp_arrive(&c->seg_empty[s % kSegs]);
        if (units < 0) break;
        if constexpr (kAlternate) {
          // Of unit j's tile: P V of its last unit, then Q K^T of unit j, which
          // overwrites that P.
#pragma unroll 1
          for (int j = 0; j < units + 2 && ok; ++j) {
            const int t = j & 1;
            int st = 0;
            if (j >= 2) {
              ok = tile_at(u_seg + j - 2, 1, st) &&
                   wait_warp<kHook>(&c->p_full[t], (p_par >> t) & 1, wc, kWMmaP);
              if (!ok) break;
              p_par ^= 1u << t;
              tc_fence_after();
              issue_pv<D>(who, kTmemO + t * D, kTmemS + t * 128, sdesc_adv(v_desc, st * L::kTileBytes), j > 3);
              commit_if(who, &c->kv_empty[st]);
            }
            if (j < units) {
              if (j == 0) {
                ok = wait_warp<kHook>(&c->q_full[0], q_par & 1, wc, kWMmaQ);
                q_par ^= 1u;
              }
              ok = ok && tile_at(u_seg + j, 0, st);
              if (!ok) break;
              issue_qk<D>(who, kTmemS + t * 128, q_desc, sdesc_adv(k_desc, st * L::kTileBytes));
              commit_if(who, &c->s_full[t]);
              commit_if(who, &c->kv_empty[st]);
            }
          }
          if (ok) commit_if(who, &c->o_done[0]);
          u_seg += units;
        } else {
          // A tile's P V of unit j - 1, then its Q K^T of unit j, which overwrites
          // that P.
          for (int j = 0; j <= units && ok; ++j) {
            int kst = 0, vst = 0;
            if (j > 0) ok = next_tile(vst);
#pragma unroll 1
            for (int t = 0; t < tiles && ok; ++t) {
              if (j == 0) {
                ok = wait_warp<kHook>(&c->q_full[t], (q_par >> t) & 1, wc, kWMmaQ);
                q_par ^= 1u << t;
              } else {
                ok = wait_warp<kHook>(&c->p_full[t], (p_par >> t) & 1, wc, kWMmaP);
                p_par ^= 1u << t;
                tc_fence_after();
                issue_pv<D>(who, kTmemO + t * D, kTmemS + t * 128, sdesc_adv(v_desc, vst * L::kTileBytes), j > 1);
                if (t == tiles - 1) commit_if(who, &c->kv_empty[vst]);
                if (j == units) commit_if(who, &c->o_done[t]);
              }
              if (j < units) {
                if (t == 0) ok = ok && next_tile(kst);
                tc_fence_after();
                issue_qk<D>(who, kTmemS + t * 128, sdesc_adv(q_desc, t * L::kTileBytes),
                            sdesc_adv(k_desc, kst * L::kTileBytes));
                commit_if(who, &c->s_full[t]);
                if (t == tiles - 1) commit_if(who, &c->kv_empty[kst]);
              }
            }
          }
        }
      }
      // Every MMA issued above must finish before TMEM is released.
      commit_if(who, &c->mma_done);
      drain_bar<true>(&c->mma_done, 0, a.timeout_ns);
      __syncwarp();
    }
  } else if (warp >= kMakeWarp) {
    reg_dealloc<kMakeRegs>();
    // ------------------------------------------------------- f16 of the codes
    const int w = warp - kMakeWarp;
    int stage = 0, raw = 0, u = 0;
    uint32_t phase = 0, raw_phase = 0;
    bool ok = work;
    auto tile_free = [&]() {
      return wait_warp<kHook>(&c->kv_empty[stage], phase ^ 1, wc, kWMakeTile);
    };
    auto tile_done = [&]() {
      fence_proxy_async_smem();
      warp_arrive(&c->kv_full[stage]);
      if (++stage == L::kStages) stage = 0, phase ^= 1;
    };
    for (int s = 0; ok; ++s) {
      ok = wait_warp<kHook>(&c->seg_full[s % kSegs], (s / kSegs) & 1, wc, kWMakeSeg);
      if (!ok) break;
      const int units = c->seg[s % kSegs].units, tok0 = c->seg[s % kSegs].tok0;
      const int lo = c->seg[s % kSegs].plain_lo, hi = c->seg[s % kSegs].plain_hi;
      warp_arrive(&c->seg_empty[s % kSegs]);
      if (units < 0) break;
      for (int j = 0; j < units; ++j, ++u) {
        ok = wait_warp<kHook>(&c->raw_full[raw], raw_phase, wc, kWMakeRaw) && tile_free();
        if (!ok) break;
        const int there = c->raw_there[raw], tok = tok0 + j * kC4Unit;
        const bool edge = there != 0xff || tok < lo || tok + kC4Unit > hi;
        const uint8_t* base = smem + L::kRawOff + raw * L::kRawBytes;
        uint8_t* tile = smem + L::kRingOff + stage * L::kTileBytes;
        auto note = [&](int g) {
          const uint32_t two = *reinterpret_cast<const uint16_t*>(base + g * group8_bytes(D) + 32 * D);
          const int ve = exp8(two >> 8);
          c->info[u % kInfos][g] = {make_float2(pow2(exp8(two & 0xff)), (float)ve),
                                    make_float2((float)ve, pow2(-ve))};
          c->nan[u % kInfos][g] = 0;
        };
        // (Keys as fast as they can be made are a tenth faster where the units'
        // tiles take turns, the making being what is waited for there, and 3%
        // slower where it is not: 2048 tokens over 32768 1767 us, so 1715.)
        if (kAlternate && lane < 2) note(2 * w + lane);
        // (Loops, not unrolled: the roles' code shares the instruction cache.)
#pragma unroll 1
        for (int g = 2 * w; g < 2 * w + 2; ++g) {
          make_keys<D, kAlternate>(tile + g * kGroup * 128, base + g * group8_bytes(D), (there >> g) & 1, lane);
          if (!kAlternate && lane == 0) note(g);
        }
        if (__builtin_expect(edge, 0)) {
          __syncwarp();
#pragma unroll 1
          for (int g = 2 * w; g < 2 * w + 2; ++g)
            if (((there >> g) & 1) && has_nan<D>(base + g * group8_bytes(D), lane) && lane == 0)
              c->nan[u % kInfos][g] = 1;
        }
        if (w == 0 && lane == 0) c->edge[u % kInfos] = edge ? 256 + there : 0;
        warp_arrive(&c->info_full[u % kInfos]);
        tile_done();
        ok = tile_free();
        if (!ok) break;
        tile = smem + L::kRingOff + stage * L::kTileBytes;
#pragma unroll 1
        for (int g = 2 * w; g < 2 * w + 2; ++g)
          make_values<D>(tile + g * kGroup * 128, base + g * group8_bytes(D), (there >> g) & 1, edge, lane);
        tile_done();
        warp_arrive(&c->raw_empty[raw]);
        if (++raw == L::kRawStages) raw = 0, raw_phase ^= 1;
      }
    }
  } else {
    reg_alloc<kSoftmaxRegs>();
    // ------------------------------------------------- softmax (thread = row)
    const int t = warp >> 2, quarter = warp & 3;
    const uint32_t tl = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tl + kTmemS + t * 128, tO = tl + kTmemO + t * D;
    const int in_tile = quarter * 32 + lane, tile_row = (kAlternate ? 0 : t * 128) + in_tile;
    uint32_t s_cnt = 0, o_cnt = 0;
    int u_seg = 0;  // units of the segments before
    bool ok = work;
    for (int s = 0; ok; ++s) {
      ok = wait_warp<kHook>(&c->seg_full[s % kSegs], (s / kSegs) & 1, wc, kWSmSeg);
      if (!ok) break;
      const Seg& seg = c->seg[s % kSegs];  // (kept until the segment's end)
      const int units = seg.units;
      if (units < 0) break;
      if (!kAlternate && seg.live <= t * 128) {
        u_seg += units;
        warp_arrive(&c->seg_empty[s % kSegs]);
        continue;
      }
      const bool valid = tile_row < seg.live;
      const int row = seg.row0 + (valid ? tile_row : 0);
      const int pos = seg.pos0 + (int)a.by_heads.div(row);

      // ---- the row of Q, scaled by a power of two: largest in [2^8, 2^9)
      float cr;
      {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + row_at(a, seg.b, seg.hk, row) * D);
        uint4 q[D / 8];
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          q[i] = valid ? src[i] : make_uint4(0, 0, 0, 0);
          big = __vmaxu2(__vmaxu2(big, q[i].x & 0x7fff7fffu), q[i].y & 0x7fff7fffu);
          big = __vmaxu2(__vmaxu2(big, q[i].z & 0x7fff7fffu), q[i].w & 0x7fff7fffu);
        }
        big = max(big & 0xffffu, big >> 16);
        int e = big >> 7;
        e = e < 16 ? 16 : (e > 250 ? 250 : e);
        const float down = __uint_as_float((uint32_t)(262 - e) << 23);
        cr = __uint_as_float((uint32_t)(e - 8) << 23) * a.scale_log2;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
          uint32_t f[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) f[x] = f16x2(bf16_lo(w[x]) * down, bf16_hi(w[x]) * down);
          uint8_t* tile = smem + (kAlternate ? 0 : t * L::kTileBytes);
          if (!kAlternate || i / (D / 16) == t)  // (or half of the tile's)
            *chunk_of(tile, in_tile, 8 * i) = make_uint4(f[0], f[1], f[2], f[3]);
        }
        fence_proxy_async_smem();
        warp_arrive(&c->q_full[kAlternate ? 0 : t]);
      }

      float m = kNoMax, l = 0.f;
      bool had_nan = false;
      const int j0 = kAlternate ? t : 0;
      for (int j = j0; j < units; j += kAlternate ? 2 : 1) {
        const int u = u_seg + j;
        // (Behind a segment that the second tile had no part in, its first wait may
        // pass early, a barrier's phase being one bit.  The second may not, and S
        // comes from a tile of keys that all making warps wrote behind their notes.)
        ok = wait_warp<kHook>(&c->info_full[u % kInfos], (u / kInfos) & 1, wc, kWSmInfo) &&
             wait_warp<kHook>(&c->s_full[t], s_cnt & 1, wc, kWSmS);
        ++s_cnt;
        if (!ok) break;
        tc_fence_after();
        const Info* info = c->info[u % kInfos];
        uint32_t x[128];
        tmem_ld32(tS, x);
        tmem_ld32(tS + 32, x + 32);
        tmem_ld32(tS + 64, x + 64);
        tmem_ld32(tS + 96, x + 96);
        tmem_wait_ld();
        reg_fence32(x);
        reg_fence32(x + 32);
        reg_fence32(x + 64);
        reg_fence32(x + 96);
        const int edge = c->edge[u % kInfos];
        if (__builtin_expect(edge != 0, 0)) {
          const int tok = seg.tok0 + j * kC4Unit;
          const int hi = pos - tok, lo = a.window < 0 ? 0 : max(pos - a.window - tok, 0);
#pragma unroll
          for (int w = 0; w < 4; ++w) {  // 32 keys, those that the row sees as bits
            const int n = min(max(hi + 1 - 32 * w, 0), 32), z = min(max(lo - 32 * w, 0), 32);
            uint32_t see = (uint32_t)((1ull << n) - 1) & ~(uint32_t)((1ull << z) - 1);
            if (!((edge >> (2 * w)) & 1)) see &= 0xffff0000u;
            if (!((edge >> (2 * w + 1)) & 1)) see &= 0xffffu;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1)) x[32 * w + e] = __float_as_uint(-INFINITY);
          }
          // Dims of NaN values that the row sees, into the workspace.
          const uint8_t* nan = c->nan[u % kInfos];
          if (*reinterpret_cast<const unsigned long long*>(nan)) {
            uint32_t* note = a.nan_rows + ((size_t)blockIdx.x * kC8WideThreads + t * 128 + in_tile) * 4;
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 32) {
              uint32_t dims = had_nan ? note[d0 / 32] : 0;
#pragma unroll 1
              for (int e = lo; e <= min(hi, 127); ++e) {
                const uint8_t* grp = nullptr;
                if (nan[e / kGroup])
                  grp = group_at(a, seg.b, seg.hk, tok + e, group8_bytes(D));
                if (!grp) continue;
#pragma unroll 1
                for (int d = 0; d < 32; ++d)
                  if ((grp[v8_at(D, e % kGroup, d0 + d)] & 0x7f) == 0x7f) dims |= 1u << d;
              }
              note[d0 / 32] = dims;
            }
            had_nan = true;
          }
          __syncwarp();
        }
        // Largest s + e_v, in powers of two.
        float top = -INFINITY, w[kUnitGroups];
#pragma unroll
        for (int g = 0; g < kUnitGroups; ++g) {
          const float2 f = info[g].key;
          // (Not zero: a masked score, minus infinity, is multiplied with it.)
          w[g] = fmaxf(cr * f.x, 1.2e-38f);
          float mg = fmaxf(__uint_as_float(x[16 * g]), __uint_as_float(x[16 * g + 1]));
#pragma unroll
          for (int e = 16 * g + 2; e < 16 * g + 16; e += 2)
            mg = max3(mg, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          top = fmaxf(top, fmaf(mg, w[g], f.y));
        }
        const bool bump = top > m + kUp + kSlack;
        float alpha = 1.f;
        if (bump) {
          alpha = ex2(m - (top - kUp));
          m = top - kUp;
          l *= alpha;
        }
#pragma unroll
        for (int g = 0; g < kUnitGroups; ++g) {
          const float2 f = info[g].value;
          const uint64_t w2 = bcast2(w[g]), c2 = bcast2(f.x - m);
          float la[2] = {0.f, 0.f}, lb[2] = {0.f, 0.f};
#pragma unroll
          for (int e = 16 * g; e < 16 * g + 16; e += 2) {
            float y0, y1;
            fma2_bcast(y0, y1, __uint_as_float(x[e]), __uint_as_float(x[e + 1]), w2, c2);
            const float p0 = ex2(y0), p1 = ex2(y1);
            add2_acc(la[(e >> 1) & 1], lb[(e >> 1) & 1], p0, p1);
            x[e / 2] = f16x2(p0, p1);
          }
          l = fmaf((la[0] + lb[0]) + (la[1] + lb[1]), f.y, l);
        }
        tmem_st32(tS, x);
        tmem_st32(tS + 32, x + 32);
        if (j > j0 && __any_sync(0xffffffffu, bump)) {
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t o[32];
            tmem_ld32(tO + ch * 32, o);
            tmem_wait_ld();
            reg_fence32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tO + ch * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&c->p_full[t]);
      }
      if (!ok) break;
      u_seg += units;
      ok = wait_warp<kHook>(&c->o_done[kAlternate ? 0 : t], o_cnt & 1, wc, kWSmO);
      if (!ok) break;
      tc_fence_after();

      // ---- the results
      // A row's two sums, where its units went to both tiles: the tiles' threads
      // tell each other theirs, and either brings half of the dims.  (In columns
      // of S, whose next product waits for both.)
      float f[2] = {1.f, 1.f};  // of the tiles' O
      bool nan_at[2] = {had_nan, false};
      if constexpr (kAlternate) {
        tmem_st4(tS, __float_as_uint(m), __float_as_uint(l), had_nan, 0);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&c->meet);
        ok = wait_warp<kHook>(&c->meet, o_cnt & 1, wc, kWSmMeet);
        if (!ok) break;
        tc_fence_after();
        uint32_t other[4];
        tmem_ld4(tl + kTmemS + (t ^ 1) * 128, other);
        tmem_wait_ld();
        asm volatile("" : "+r"(other[0]), "+r"(other[1]), "+r"(other[2]), "+r"(other[3]));
        const float m2 = __uint_as_float(other[0]), top = fmaxf(m, m2);
        const float mine = ex2(m - top), its = ex2(m2 - top);
        l = mine * l + its * __uint_as_float(other[1]);
        m = top;
        f[t] = mine, f[t ^ 1] = its;
        nan_at[t] = had_nan, nan_at[t ^ 1] = other[2] != 0;
      }
      ++o_cnt;
      const bool whole = seg.whole;
      const float mul = !whole ? 1.f : (l > 0.f || l != l ? 1.f / l : 0.f);
      const size_t out = row_at(a, seg.b, seg.hk, row);
      const size_t part = (size_t)seg.part * L::kRows + tile_row;
      const uint32_t* note = a.nan_rows + ((size_t)blockIdx.x * kC8WideThreads + in_tile) * 4;
      const int dim0 = kAlternate ? t * (D / 2) : 0;
#pragma unroll 1
      for (int ch = 0; ch < (kAlternate ? D / 64 : D / 32); ++ch) {
        const int dim = dim0 + ch * 32;
        uint32_t o[32], dims = 0;
        tmem_ld32(tl + kTmemO + (kAlternate ? 0 : t * D) + dim, o);
        tmem_wait_ld();
        reg_fence32(o);
        if constexpr (kAlternate) {
          uint32_t o1[32];
          if (units > 1) {  // (else the second tile has nothing)
            tmem_ld32(tl + kTmemO + D + dim, o1);
            tmem_wait_ld();
            reg_fence32(o1);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float v = __uint_as_float(o[e]) * f[0];
            if (units > 1) v = fmaf(__uint_as_float(o1[e]), f[1], v);
            o[e] = __float_as_uint(v);
          }
          for (int i = 0; i < 2; ++i)
            if (nan_at[i]) dims |= note[i * 512 + dim / 32];
        } else if (had_nan) {
          dims = note[t * 512 + dim / 32];
        }
#pragma unroll
        for (int e = 0; e < 32; ++e)
          o[e] = (dims >> e) & 1 ? 0x7fffffffu : __float_as_uint(__uint_as_float(o[e]) * mul);
        if (valid && whole) {
          uint4* dst = reinterpret_cast<uint4*>(a.o + out * D + dim);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t pk[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              pk[k] = pack_bf16(__uint_as_float(o[8 * i + 2 * k]), __uint_as_float(o[8 * i + 2 * k + 1]));
            dst[i] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        } else if (valid) {
          float* dst = a.part + part * D + dim;
#pragma unroll
          for (int i = 0; i < 4; ++i) st_global_v8(dst + 8 * i, o + 8 * i);
        }
        __syncwarp();
      }
      if (valid && (!kAlternate || t == 0)) {
        if (whole) a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        else a.part_ml[part] = make_float2(m, l);
      }
      tc_fence_before();
      warp_arrive(&c->seg_empty[s % kSegs]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(c->tmem, 512);
  }
}

// Joins the partial results of an item that lies in several blocks' shares, in
// block order.  A warp takes kRows rows, D / 32 dims a lane, and has the loads
// of kParts parts on their way at once.  (One row and four parts at a time: 22
// us for 152 joins of 256 rows.)
template <int D, int kItem, int kRows, int kParts>
__device__ __forceinline__ void join_rows(const CacheAttnArgs& a, const int4& j, int block, int in0) {
  constexpr int kDims = D / 32;
  using Vec = std::conditional_t<D == 128, float4, float2>;
  const int lane = threadIdx.x & 31, hk = j.y / a.row_blocks;
  const int row0 = (j.y - hk * a.row_blocks) * kItem + in0;
  const int live = min(a.q_lens ? a.q_lens[j.x] : a.T, a.T) * a.heads;
  const int parts = j.z - block + 2;
  auto at = [&](int k, int r) {
    return (size_t)(k == 0 ? j.w : 2 * (block + k - 1)) * kItem + in0 + r;
  };
  float acc[kRows][kDims], sum[kRows], mx[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    mx[r] = kNoMax, sum[r] = 0.f;
#pragma unroll
    for (int d = 0; d < kDims; ++d) acc[r][d] = 0.f;
  }
#pragma unroll 1
  for (int k0 = 0; k0 < parts; k0 += kParts) {
    float2 ml[kRows][kParts];
    Vec v[kRows][kParts];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        const bool there = k0 + k < parts && row0 + r < live;
        ml[r][k] = there ? a.part_ml[at(k0 + k, r)] : make_float2(kNoMax, 0.f);
        v[r][k] = there ? reinterpret_cast<const Vec*>(a.part + at(k0 + k, r) * D)[lane] : Vec{};
      }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float top = mx[r];
#pragma unroll
      for (int k = 0; k < kParts; ++k) top = fmaxf(top, ml[r][k].x);
      const float f0 = ex2(mx[r] - top);
      mx[r] = top;
      sum[r] *= f0;
#pragma unroll
      for (int d = 0; d < kDims; ++d) acc[r][d] *= f0;
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        const float f = ex2(ml[r][k].x - top);
        sum[r] += f * ml[r][k].y;
        const float* o = reinterpret_cast<const float*>(&v[r][k]);
#pragma unroll
        for (int d = 0; d < kDims; ++d) acc[r][d] += f * o[d];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (row0 + r >= live) break;
    const float inv = sum[r] > 0.f || sum[r] != sum[r] ? 1.f / sum[r] : 0.f;
    const size_t out = row_at(a, j.x, hk, row0 + r);
    __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(a.o + out * D) + lane * (kDims / 2);
#pragma unroll
    for (int d = 0; d < kDims; d += 2)
      dst[d / 2] = __floats2bfloat162_rn(acc[r][d] * inv, acc[r][d + 1] * inv);
    if (lane == 0) a.lse[out] = sum[r] == 0.f ? -INFINITY : (mx[r] + log2f(sum[r])) * kLn2;
  }
}

constexpr int kJoinWarps = 8;
constexpr int join_rows_each(int item) { return item > 128 ? 2 : 1; }
template <int D, int kItem>
__global__ void __launch_bounds__(kJoinWarps * 32) cache8_wide_join_kernel(CacheAttnArgs a) {
  wait_for_stream();
  const int4 j = a.joins[blockIdx.x];
  if (j.x < 0) return;
  constexpr int kJoinRows = join_rows_each(kItem);
  const int in0 = (blockIdx.y * kJoinWarps + (threadIdx.x >> 5)) * kJoinRows;
  if (j.z - (int)blockIdx.x + 2 <= 4) {
    join_rows<D, kItem, kJoinRows, 4>(a, j, blockIdx.x, in0);
  } else {  // a long history of few rows
#pragma unroll 1
    for (int r = 0; r < kJoinRows; ++r) join_rows<D, kItem, 1, 16>(a, j, blockIdx.x, in0 + r);
  }
}

template <int D, bool kAlternate, bool kHook = false>
cudaError_t run(const CacheAttnArgs& a, int sm_count, cudaStream_t stream) {
  // The hook has its own instantiation, for d = 128.
  if constexpr (D == 128 && !kHook) {
    if (a.hook) return run<D, kAlternate, true>(a, sm_count, stream);
  }
  using L = Wide<D, kAlternate>;
  static std::atomic<unsigned long long> done{0};
  auto* kernel = cache8_wide_kernel<D, kAlternate, kHook>;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), L::kSmem, done);
  if (e != cudaSuccess) return e;
  const int blocks = sm_count < kC8WideBlocks ? sm_count : kC8WideBlocks;
  e = launch_overlapped(kernel, dim3(blocks), dim3(kThreads), L::kSmem, stream, a);
  if (e != cudaSuccess) return e;
  const int rows = std::min(a.rows, L::kRows), of_a_block = kJoinWarps * join_rows_each(L::kRows);
  return launch_overlapped(cache8_wide_join_kernel<D, L::kRows>, dim3(blocks, (rows - 1) / of_a_block + 1),
                           dim3(32 * kJoinWarps), 0, stream, a);
}

}  // namespace

int cache8_wide_rows(int rows) { return rows <= 128 ? 128 : 256; }

cudaError_t launch_cache8_wide(const CacheAttnArgs& a, int d, int sm_count, cudaStream_t stream) {
  if (a.item_rows == 128)
    return d == 128 ? run<128, true>(a, sm_count, stream) : run<64, true>(a, sm_count, stream);
  return d == 128 ? run<128, false>(a, sm_count, stream) : run<64, false>(a, sm_count, stream);
}

cudaError_t set_expire_site_cache8_wide(uint32_t site) {
  return cudaMemcpyToSymbol(c_expire_site, &site, sizeof(site));
}

}  // namespace fa
