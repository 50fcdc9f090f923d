// fa_cache4_attn.cu -- attention of new tokens over the paged 4-bit cache.
//
//   o_r = sum_j softmax_j(scale q_r . k_j) v_j,   k_j, v_j = code * scale * g
//
// with one pass over the keys: running maximum m and sum l per row, the
// values' sums rescaled when m grows.
//
// Work.  The query rows of one request and key/value head (H / Hkv heads x
// its new tokens, by token first) are taken 8 to 40 at a time; such a row block
// is an item, the keys that it sees are cut into units of 128, and all items'
// units together are dealt to the blocks in equal consecutive shares, whatever
// the lengths (fa_cache4_work.h).  A block's four warps take two 16-token
// groups of a unit each, with sums of their own, and join them when the item
// (or the share) ends; an item that lies in several blocks' shares is joined
// by a second kernel.  (Rows by head first, every item with all of its
// request's keys, took 13.6 ms where one of 64 requests has 512 new tokens and
// the others one each, of 64 heads over 8; so it takes 0.35 ms.)
//
// Feeding.  Each warp copies its own groups (18 d bytes, K and V together)
// into a ring in shared memory by bulk copies, several ahead; nothing in the
// main loop waits for another warp.
//
// Products.  The scores are computed as S^T = K Q^T and the output as
// O^T = V^T P^T by mma m16n8k16 in f16 with fp32 sums: keys and dims fill
// the 16-high side and the few query rows the 8-wide side, so that eight
// rows (one decode token of a group of up to 8 heads) waste nothing.  A code
// times its scale has at most six significant bits: K and V enter exactly.
// Q's rows are scaled by a power of two, the largest to [2^8, 2^9): bf16's 8
// bits fit f16's 11, and elements down to 2^-25 of their row's largest enter
// exactly; below, f16's spacing is off by at most 2^-33 of the largest.  P is
// rounded to f16 (half a step: 2^-11), after a factor 2^8: weights below 2^-22
// of the row's largest lose low bits, those below about 2^-32 vanish.
//
// What bounds it is making f16 of 4-bit codes: a 16-token group of one head
// costs 269 warp instructions (64 conversions, 64 products with scales, 24 to
// put two tokens' value codes side by side, which the layout asks for, 16
// matrix products, the softmax and the loop), and twelve warps per SM find
// issue slots for 58% of the time.
// Measured (d = 128, 8 query heads to a key/value head): 64 requests of 100 to
// 8192 tokens x 8 heads 61 us, 5.0 TB/s of codes and scales; 3 requests of
// 100000 to 131072 tokens x 8 heads 72 us, 5.5 TB/s; with all pages in L2
// 2 us less.  Tiles: two groups per step (one: 98 us at the batch, two: 79),
// blocks per SM three (four, at 128 registers: 72 us, three: 70), kC4ItemCost
// three units (one: 79 us, three: 72, five: 74).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fa_cache4.cuh"
#include "fa_cache4_work.h"
#include "fa_common.cuh"
#include "fa_serve.h"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kGroups = 2;                        // of a warp in a unit
static_assert(kC4Unit == kWarps * kGroups * kGroup && kC4Align == kGroups * kGroup);
constexpr float kNoMax = -1e30f;                  // m of a row that has seen no key
constexpr float kUp = 8.0f;                       // P carries 2^kUp
constexpr float kSlack = 6.0f;                    // growth of m that is left standing
constexpr uint32_t kWCopy = 0x511;                // where-code of the waits for copies

__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t* r) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Two E4M3 bytes (low 16 bits) as f16.
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The same by a half of a pair: as __half2 the compiler takes the half in the
// multiplication itself.
__device__ __forceinline__ uint32_t mul2(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The call as the division of work sees it, for items of kRows rows, and its
// requests (read by plain loads: the kernel before may have written them).
template <int kRows>
__device__ __forceinline__ c4::Call call_of(const Cache4AttnArgs& a) {
  return {a.B, a.Hkv, a.T, a.window, a.heads, kRows, a.row_blocks, a.M << a.shift, a.by_heads};
}
// Row `row` of a request and key/value head in q, o and lse.
__device__ __forceinline__ size_t row_at(const Cache4AttnArgs& a, int b, int hk, int row) {
  const int t = (int)a.by_heads.div(row), h = row - t * a.heads;
  return (((size_t)b * a.Hkv + hk) * a.heads + h) * a.T + t;
}

template <int D, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr bool kQInRegs = NT <= 2;  // else Q's fragments are in shared memory
  static constexpr int kTiles = D / 16;                    // 16-dim tiles of O^T
  static constexpr int kSlot = kGroups * group_bytes(D);
  static constexpr int kStages = 2;
  // Groups of a step: both, but where the registers are full with sums.
  static constexpr int kTogether = D == 128 && NT > 3 ? 1 : kGroups;
  static constexpr int kBlocksPerSm = NT == 1 || (NT == 2 && D == 64) ? 3 : 2;
  static constexpr int kRing = kWarps * kStages * kSlot;
  static constexpr int kPitch = D + 4;  // floats of a row in the join buffer
  static constexpr int kJoin = kWarps * 8 * kPitch * 4;  // eight rows of every warp
  static constexpr int kQPitch = 2 * D + 16;             // bytes of a raw row of Q
  static constexpr int kQRaw = kRows * kQPitch;
  static constexpr int kQBuffers = kQInRegs ? 2 : 1;
  static constexpr int kQFrag = kQInRegs ? 0 : NT * (D / 32) * 512;
  static constexpr int kSmem = kRing + kJoin + kQBuffers * kQRaw + kQFrag;
};

// Where the partial results of a block's first (2 c) and last (2 c + 1)
// segment lie in the workspace.
struct Partial {
  float* o;    // [D]
  float2* ml;  // m, l
};
template <int D, int NT>
__device__ __forceinline__ Partial partial_of(const Cache4AttnArgs& a, int slot, int row) {
  const size_t at = (size_t)slot * Shape<D, NT>::kRows + row;
  return Partial{a.part + at * D, a.part_ml + at};
}

// The running state of a segment's rows in one warp.
template <int D, int NT>
struct Rows {
  // Q: row 8 nt + g, dims t D/4 + 0 .. D/4 - 1, scaled to f16, here or in
  // shared memory (4 registers' worth per lane, [nt][D / 32][lane]).
  uint32_t qf[Shape<D, NT>::kQInRegs ? NT : 1][D / 8];
  const uint4* qs;
  // Score to power of two, of rows 8 nt + 2t and + 1, likewise.
  float rs[Shape<D, NT>::kQInRegs ? NT : 1][2];
  const float2* rss;
  __device__ __forceinline__ float2 scale(int nt) const {
    if constexpr (Shape<D, NT>::kQInRegs) return make_float2(rs[nt][0], rs[nt][1]);
    else return rss[4 * nt];
  }
  // m: the row's maximum less kUp, in powers of two; weights are 2^(s - m).
  float m[NT][2], l[NT][2];
  float o[Shape<D, NT>::kTiles][NT][4];
};

// One group's scores, S^T = K Q^T: tokens g and g + 8, rows 2t and 2t + 1.
template <int D, int NT>
__device__ __forceinline__ void scores(const uint8_t* grp, int g, int t, const Rows<D, NT>& r,
                                       float (&s)[NT][4]) {
  uint32_t kc[2][D / 32];
  __half2 ks[2][D / 64];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t* kp = grp + k_code_at(D, g + 8 * h, t * (D / 8));
    const uint8_t* sp = grp + k_scale_at(D, g + 8 * h, t * (D / 64));
    if constexpr (D == 128) {
      const uint4 u = *reinterpret_cast<const uint4*>(kp);
      kc[h][0] = u.x, kc[h][1] = u.y, kc[h][2] = u.z, kc[h][3] = u.w;
      const uint32_t two = e4m3_to_f16(*reinterpret_cast<const uint16_t*>(sp));
      const __half2 th = *reinterpret_cast<const __half2*>(&two);
      ks[h][0] = __low2half2(th);
      ks[h][1] = __high2half2(th);
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(kp);
      kc[h][0] = u.x, kc[h][1] = u.y;
      const uint32_t two = e4m3_to_f16(*sp);
      ks[h][0] = __low2half2(*reinterpret_cast<const __half2*>(&two));
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    uint32_t x[4], y[4];
    e2m1_to_f16(kc[0][w], x);
    e2m1_to_f16(kc[1][w], y);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], ks[0][w / 2]), y[i] = mul2(y[i], ks[1][w / 2]);
    const uint32_t f0[4] = {x[0], y[0], x[1], y[1]}, f1[4] = {x[2], y[2], x[3], y[3]};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint4 q;
      if constexpr (Shape<D, NT>::kQInRegs)
        q = make_uint4(r.qf[nt][4 * w], r.qf[nt][4 * w + 1], r.qf[nt][4 * w + 2], r.qf[nt][4 * w + 3]);
      else
        q = r.qs[(nt * (D / 32) + w) * 32];
      mma(s[nt], f0, q.x, q.y);
      mma(s[nt], f1, q.z, q.w);
    }
  }
}

// One group's part of O^T += V^T P^T.  vs: the scales of the lane's tokens
// 2t, 2t + 1 (low half of the group) and 2t + 8, 2t + 9.
template <int D, int NT>
__device__ __forceinline__ void values(const uint8_t* grp, int g, int t, const uint32_t (&vs)[2],
                                       const uint32_t (&pb)[NT][2],
                                       float (&o)[Shape<D, NT>::kTiles][NT][4]) {
  constexpr int kWords = D / 64;  // words of one token's eighth of the dims
  uint32_t vc[2][2][kWords];      // [half of the group][token parity][word]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t* vp = grp + v_code_at(D, 8 * h + 2 * t, g);
    if constexpr (D == 128) {
      const uint4 u = *reinterpret_cast<const uint4*>(vp);
      vc[h][0][0] = u.x, vc[h][0][1] = u.y, vc[h][1][0] = u.z, vc[h][1][1] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(vp);
      vc[h][0][0] = u.x, vc[h][1][0] = u.y;
    }
  }
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    // Bytes of the two tokens' codes of one dim: even dims, odd dims.
    uint32_t ev[2][4], od[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      constexpr uint32_t kLow = 0x0f0f0f0fu;
      const uint32_t x = vc[h][0][w], y = vc[h][1][w];
      e2m1_to_f16((x & kLow) | ((y << 4) & ~kLow), ev[h]);
      e2m1_to_f16(((x >> 4) & kLow) | (y & ~kLow), od[h]);
#pragma unroll
      for (int i = 0; i < 4; ++i) ev[h][i] = mul2(ev[h][i], vs[h]), od[h][i] = mul2(od[h][i], vs[h]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t f[4] = {ev[0][i], od[0][i], ev[1][i], od[1][i]};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma(o[4 * w + i][nt], f, pb[nt][0], pb[nt][1]);
    }
  }
}

// What bounds the keys that a segment's rows see: its place, in shared memory
// (it is needed for masks only, where registers are scarce).
struct Bounds {
  const Cache4AttnArgs& a;
  const c4::Cursor& at;
  int rows;  // of an item
  // Position of a row of the segment.
  __device__ __forceinline__ int pos(int row) const {
    return at.r.len - at.r.ql + (int)a.by_heads.div(at.rb * rows + row);
  }
  // A live row sees the keys low(pos) to pos, all of them in the cache.  Rows
  // behind the live ones have Q = 0 and are not written.
  __device__ __forceinline__ int low(int pos) const { return a.window < 0 ? 0 : pos - a.window; }
};

// kU groups' scores, minus infinity where a row does not see a token.
// kPlain: every row sees every token; else bit u of `there` says whether
// group u was copied.
template <int D, int NT, int kU, bool kPlain>
__device__ __forceinline__ void masked_scores(const Rows<D, NT>& r, const uint8_t* grps, int tok,
                                              int there, const Bounds& bd, int g, int t,
                                              float (&s)[kU][NT][4]) {
#pragma unroll
  for (int u = 0; u < kU; ++u) scores<D, NT>(grps + u * group_bytes(D), g, t, r, s[u]);
  if constexpr (!kPlain) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int pos = bd.pos(8 * nt + 2 * t + i);
        const int hi = pos + 1, lo = bd.low(pos);
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int j = tok + u * kGroup + g + 8 * h;
            if (j >= hi || j < lo || !((there >> u) & 1)) s[u][nt][i + 2 * h] = -INFINITY;
          }
      }
  }
}

// kU groups' products.
template <int D, int NT, int kU, bool kPlain>
__device__ __forceinline__ void use_groups(Rows<D, NT>& r, const uint8_t* grps, int tok, int there,
                                           const Bounds& bd, int g, int t) {
  float s[kU][NT][4], top = -INFINITY;
  masked_scores<D, NT, kU, kPlain>(r, grps, tok, there, bd, g, t, s);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float2 rs = r.scale(nt);
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = fmaxf(top, fmaf(s[u][nt][i], i & 1 ? rs.y : rs.x, -r.m[nt][i & 1]));
  }
  if (__any_sync(0xffffffffu, top > kUp + kSlack)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < kU; ++u) mx = fmaxf(mx, fmaxf(s[u][nt][i], s[u][nt][i + 2]));
        mx *= i ? r.scale(nt).y : r.scale(nt).x;  // (positive: minus infinity stays)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        mx = fmaxf(mx - kUp, r.m[nt][i]);
        const float f = ex2(r.m[nt][i] - mx);
        r.m[nt][i] = mx;
        r.l[nt][i] *= f;
#pragma unroll
        for (int dt = 0; dt < Shape<D, NT>::kTiles; ++dt) r.o[dt][nt][i] *= f, r.o[dt][nt][i + 2] *= f;
      }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    uint32_t pb[NT][2], vs[2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float p[4];
      const float2 rs = r.scale(nt);
#pragma unroll
      for (int i = 0; i < 4; ++i)  // (made again: fewer registers than kept from above)
        p[i] = ex2(fmaf(s[u][nt][i], i & 1 ? rs.y : rs.x, -r.m[nt][i & 1]));
      r.l[nt][0] += p[0] + p[2];
      r.l[nt][1] += p[1] + p[3];
      pb[nt][0] = transpose8x8(f16x2(p[0], p[1]));
      pb[nt][1] = transpose8x8(f16x2(p[2], p[3]));
    }
    const uint8_t* grp = grps + u * group_bytes(D);
    uint32_t nans = 0;  // by token of the group: a scale of the lane's dims is NaN
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t two = *reinterpret_cast<const uint16_t*>(
          grp + v_scale_at(D, 8 * h + 2 * t, D == 128 ? g : g >> 1));
      if constexpr (!kPlain) {
        if (!((there >> u) & 1)) two = 0;
        const uint32_t nan = __vcmpeq4(two & 0x7f7fu, 0x7f7f7f7fu);
        nans |= ((nan & 1) | (nan >> 7 & 2)) << (8 * h + 2 * t);
        two &= ~nan;
      }
      vs[h] = e4m3_to_f16(two);
    }
    values<D, NT>(grp, g, t, vs, pb, r.o);
    // A NaN goes to the rows that see its token, and not, by a weight of zero,
    // to the others (a token that no row sees may hold anything).
    if (!kPlain && __any_sync(0xffffffffu, nans != 0)) {
      nans |= __shfl_xor_sync(0xffffffffu, nans, 1);
      nans |= __shfl_xor_sync(0xffffffffu, nans, 2);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int pos = bd.pos(8 * nt + 2 * t + i), at = tok + u * kGroup;
          const int hi = min(max(pos + 1 - at, 0), kGroup);
          const int lo = min(max(bd.low(pos) - at, 0), kGroup);
          if (nans & ((1u << hi) - 1) & ~((1u << lo) - 1)) {
#pragma unroll
            for (int dt = 0; dt < Shape<D, NT>::kTiles; ++dt)
              r.o[dt][nt][i] = r.o[dt][nt][i + 2] = __uint_as_float(0x7fffffffu);
          }
        }
    }
  }
}

// One slot of the ring.
template <int D, int NT, bool kPlain>
__device__ __forceinline__ void use_slot(Rows<D, NT>& r, const uint8_t* grps, int tok, int there,
                                         const Bounds& bd, int g, int t) {
  constexpr int kU = Shape<D, NT>::kTogether;
#pragma unroll 1
  for (int u = 0; u < kGroups; u += kU)
    use_groups<D, NT, kU, kPlain>(r, grps + u * group_bytes(D), tok + u * kGroup, there >> u, bd, g, t);
}

// kHook: the instantiation with the failure-path test hook.
template <int D, int NT, bool kHook>
__global__ void __launch_bounds__(kWarps * 32, Shape<D, NT>::kBlocksPerSm)
    cache4_attn_kernel(Cache4AttnArgs a) {
  using S = Shape<D, NT>;
  constexpr int kTiles = S::kTiles;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kWarps][S::kStages];
  __shared__ int copied[kWarps][S::kStages];  // bit u: group u of the slot
  __shared__ uint32_t cta_abort;
  __shared__ c4::Cursor sh_load[kWarps], sh_use[kWarps], sh_first;
  __shared__ int sh_into;
  __shared__ long long sh_scan[kWarps];
  __shared__ float2 sh_ml[kWarps][8];
  __shared__ __align__(8) float sh_rs[S::kRows];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * S::kStages * S::kSlot;
  float* join = reinterpret_cast<float*>(smem + S::kRing);
  uint8_t* q_raw = smem + S::kRing + S::kJoin;
  uint4* q_frag = reinterpret_cast<uint4*>(q_raw + S::kQBuffers * S::kQRaw);
  const WaitCtl ctl = {a.st, &cta_abort, a.timeout_ns};
  if (lane < S::kStages) mbar_init(&full[warp][lane], 1);
  if (tid == 0) cta_abort = 0;
  fence_mbar_init();
  wait_for_stream();
  launch_dependents();

  // ---- this block's share of the units
  const c4::Call call = call_of<S::kRows>(a);
  auto read = [&](int b) {
    return c4::request_of(call, a.seq_lens[b], a.q_lens ? a.q_lens[b] : a.T);
  };
  const int pairs = a.B * a.row_blocks, per = (pairs - 1) / (kWarps * 32) + 1;
  const int p0 = (int)min((long long)pairs, (long long)tid * per), p1 = p0 + min(pairs - p0, per);
  const long long mine = c4::cost_of(call, read, p0, p1);
  long long upto = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, upto, m);
    if (lane >= m) upto += u;
  }
  if (lane == 31) sh_scan[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += sh_scan[w];
    total += sh_scan[w];
  }
  const long long before = upto - mine;
  const c4::Shares shares(total * a.Hkv, gridDim.x);
  if ((int)blockIdx.x >= shares.blocks) {
    if (tid == 0) a.joins[blockIdx.x].x = -1;
    return;
  }
  const long long u0 = shares.first(blockIdx.x);
  if (u0 >= before * a.Hkv && u0 < upto * a.Hkv)
    sh_into = sh_first.seek(call, read, p0, u0 - before * a.Hkv,
                            (int)(shares.first(blockIdx.x + 1) - u0));
  __syncthreads();
  const c4::Cursor use = sh_first;
  if (use.end == use.unit) {  // a share of nothing but an item's cost
    if (tid == 0) a.joins[blockIdx.x].x = -1;
    return;
  }

  // ---- the warp's own ring, one slot per unit.  Each lane works out where
  // one of the next 32 units' groups lie and issues those copies when its
  // turn comes.
  // (The loads' and the products' places are kept in shared memory, by warp:
  // they are needed once per 32 units and once per segment.)
  if (lane == 0) sh_load[warp] = sh_use[warp] = use;
  __syncwarp();
  bool more = true;         // there are units left to load
  int put = 0, put_slot = 0;  // units passed by the loads, and their slot
  int turn = 0, turns = 0;    // place in the lanes' units
  const uint8_t* src[kGroups];
  auto look_ahead = [&](const c4::Cursor& load) {
    turn = 0;
    turns = min(32, load.end - load.unit);
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      const int tok = load.k.lo + (load.unit + lane) * kC4Unit + (warp * kGroups + u) * kGroup;
      src[u] = nullptr;
      if (lane < turns && tok < load.k.hi) {
        const int page = a.block_table[(size_t)load.b * a.M + (tok >> a.shift)];
        const int gpp_shift = a.shift - 4;
        if (page >= 0 && page < a.pages)
          src[u] = a.cache + ((((size_t)page * a.Hkv + load.hk) << gpp_shift) +
                              ((tok >> 4) & ((1 << gpp_shift) - 1))) * group_bytes(D);
      }
    }
  };
  auto feed = [&]() {
    if (lane == turn) {
      uint64_t* bar = &full[warp][put_slot];
      uint8_t* dst = ring + put_slot * S::kSlot;
      const int n = (src[0] ? 1 : 0) + (src[1] ? 1 : 0);
      copied[warp][put_slot] = (src[0] ? 1 : 0) | (src[1] ? 2 : 0);
      if (n) mbar_arrive_expect_tx(bar, n * group_bytes(D));
      else mbar_arrive(bar);
      if (n == 2 && src[1] == src[0] + group_bytes(D)) {
        bulk_load(dst, src[0], S::kSlot, bar);
      } else {
        if (src[0]) bulk_load(dst, src[0], group_bytes(D), bar);
        if (src[1]) bulk_load(dst + group_bytes(D), src[1], group_bytes(D), bar);
      }
    }
    ++put;
    if (++put_slot == S::kStages) put_slot = 0;
    if (++turn == turns) {
      c4::Cursor load = sh_load[warp];
      load.unit += turns;
      if (load.unit == load.end) more = load.next(call, read);
      if (more) look_ahead(load);
      __syncwarp();  // every lane has read the old place
      if (lane == 0) sh_load[warp] = load;
      __syncwarp();
    }
  };
  look_ahead(use);
  for (int i = 0; i < S::kStages && more; ++i) feed();

  // ---- Q: the next segment's raw rows are on their way while one is worked on
  auto fetch_q = [&](const c4::Cursor& c, int buffer) {
    constexpr int kChunks = 2 * D / 16;
    uint8_t* dst = q_raw + buffer * S::kQRaw;
    const int row0 = c.rb * S::kRows, rows = min(S::kRows, c.r.ql * a.heads - row0);
    for (int i = tid; i < rows * kChunks; i += kWarps * 32)
      copy16_async(dst + i / kChunks * S::kQPitch + i % kChunks * 16,
                   a.q + row_at(a, c.b, c.hk, row0 + i / kChunks) * D + i % kChunks * 8);
  };
  fetch_q(use, 0);

  // What the joining kernel does for this block's first item, if that began
  // in the block before: the request, item, last block, and first partial.
  // (Here, the loads being on their way; by the last warp's first thread, the
  // first group's warp being the one that is waited for.)
  if (tid == (kWarps - 1) * 32) {
    int4 j = make_int4(-1, 0, 0, 0);
    int last, first_part;
    if (c4::join_of(shares, use, blockIdx.x, u0, sh_into, &last, &first_part))
      j = make_int4(use.b, use.hk * a.row_blocks + use.rb, last, first_part);
    a.joins[blockIdx.x] = j;
  }

  int got = 0, got_slot = 0;
  uint32_t parity = 0;
  bool dead = false;
  for (int seg = 0;; ++seg) {
    // ---- one segment
    // The item's live rows, if they are fewer than all.
    auto live_rows = [&] { return sh_use[warp].r.ql * a.heads - sh_use[warp].rb * S::kRows; };
    const int live_q = live_rows();
    const Bounds bd = {a, sh_use[warp], S::kRows};
    copies_done();
    __syncthreads();  // Q is there, and the other buffer's readers are done
    auto fetch_next = [&]() {
      c4::Cursor then = sh_use[warp];
      if (then.next(call, read)) fetch_q(then, (seg + 1) % S::kQBuffers);
    };
    if constexpr (S::kQBuffers == 2) fetch_next();

    Rows<D, NT> r;
    const uint8_t* raw = q_raw + seg % S::kQBuffers * S::kQRaw;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (!S::kQInRegs && nt % kWarps != warp) continue;
      uint32_t qf[D / 8], big = 0;
      const uint4* q = reinterpret_cast<const uint4*>(raw + (8 * nt + g) * S::kQPitch + t * (D / 2));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 u = 8 * nt + g < live_q ? q[i] : make_uint4(0, 0, 0, 0);
        qf[4 * i] = u.x, qf[4 * i + 1] = u.y, qf[4 * i + 2] = u.z, qf[4 * i + 3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) big = __vmaxu2(big, qf[i] & 0x7fff7fffu);
      big = max(big & 0xffffu, big >> 16);
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // Exponent field of the row's largest; the row is scaled to [2^8, 2^9).
      int e = big >> 7;
      e = e < 16 ? 16 : (e > 250 ? 250 : e);
      const float down = __uint_as_float((uint32_t)(262 - e) << 23);
      // (Not zero: a masked score, minus infinity, is multiplied with it.)
      const float back = fmaxf(__uint_as_float((uint32_t)(e - 8) << 23) * a.scale_log2, 1.2e-38f);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        qf[i] = f16x2(__uint_as_float(qf[i] << 16) * down, __uint_as_float(qf[i] & 0xffff0000u) * down);
      if constexpr (S::kQInRegs) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) r.qf[nt][i] = qf[i];
        r.rs[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);
        r.rs[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          q_frag[(nt * (D / 32) + i) * 32 + lane] =
              make_uint4(qf[4 * i], qf[4 * i + 1], qf[4 * i + 2], qf[4 * i + 3]);
        if (t == 0) sh_rs[8 * nt + g] = back;
      }
    }
    if constexpr (!S::kQInRegs) {
      __syncthreads();
      fetch_next();  // the one buffer is free
      r.qs = q_frag + lane;
      r.rss = reinterpret_cast<const float2*>(sh_rs) + t;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      r.m[nt][0] = r.m[nt][1] = kNoMax;
      r.l[nt][0] = r.l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
        r.o[i][nt][0] = r.o[i][nt][1] = r.o[i][nt][2] = r.o[i][nt][3] = 0.f;
    }
    // Tokens within [plain_lo, plain_hi) are seen by every live row.
    const int plain_hi = sh_use[warp].k.first + 1, plain_lo = bd.low(sh_use[warp].k.hi - 1);

    int tok = sh_use[warp].k.lo + sh_use[warp].unit * kC4Unit + warp * kGroups * kGroup;
    for (int left = dead ? 0 : sh_use[warp].end - sh_use[warp].unit; left > 0; --left, tok += kC4Unit) {
      // (The hook stops a block's first warp whether its copy has landed or
      // not: a warp's first look at a barrier may sleep until it has.)
      const bool expire = kHook && warp == 0 && c_expire_site == kWCopy;
      if (expire && lane == 0) raise_abort(ctl, kWCopy);
      if (expire || !wait_bar_warp(&full[warp][got_slot], parity, ctl, kWCopy)) {
        dead = true;
        break;
      }
      const uint8_t* slot = ring + got_slot * S::kSlot;
      const int there = copied[warp][got_slot];
      if (there == 3 && tok >= plain_lo && tok + kGroups * kGroup <= plain_hi)
        use_slot<D, NT, true>(r, slot, tok, there, bd, g, t);
      else if (there)
        use_slot<D, NT, false>(r, slot, tok, there, bd, g, t);
      __syncwarp();  // every lane has read the slot
      ++got;
      if (++got_slot == S::kStages) got_slot = 0, parity ^= 1;
      if (more) feed();
    }

    // ---- join the warps, eight rows at a time: a warp writes two
    c4::Cursor at = sh_use[warp];
    const bool whole = at.unit == 0 && at.end == at.k.units;
    const int live = live_rows();
    const int part_slot = 2 * blockIdx.x + (seg == 0 ? 0 : 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // (The buffer's last readers are done: the segment began with a barrier.)
      if (nt > 0) __syncthreads();
      // Lane (g, t) holds dims g D/8 + 0 .. D/8 - 1 of rows 2t, 2t + 1.
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = r.l[nt][i];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        const int row = 2 * t + i;
        if (8 * nt + row >= live) continue;
        if (g == 0) sh_ml[warp][row] = make_float2(r.m[nt][i], l);
        float* dst = join + (warp * 8 + row) * S::kPitch + g * (D / 8);
#pragma unroll
        for (int dt = 0; dt < kTiles; dt += 2)
          *reinterpret_cast<float4*>(dst + 2 * dt) = make_float4(
              r.o[dt][nt][i], r.o[dt][nt][i + 2], r.o[dt + 1][nt][i], r.o[dt + 1][nt][i + 2]);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int in = warp + k * kWarps, row = 8 * nt + in;
        if (row >= live) continue;
        const size_t out = row_at(a, at.b, at.hk, at.rb * S::kRows + row);
        float mx = kNoMax, f[kWarps], sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sh_ml[w][in].x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          f[w] = ex2(sh_ml[w][in].x - mx);
          sum += f[w] * sh_ml[w][in].y;
        }
        const float inv = sum > 0.f || sum != sum ? a.v_scale / sum : 0.f;
        const Partial part = partial_of<D, NT>(a, part_slot, row);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {  // two dims a lane
          float2 acc = make_float2(0.f, 0.f);
          const int dim = 64 * i + 2 * lane;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 v =
                *reinterpret_cast<const float2*>(join + (w * 8 + in) * S::kPitch + dim);
            acc.x += f[w] * v.x, acc.y += f[w] * v.y;
          }
          if (whole)
            *reinterpret_cast<__nv_bfloat162*>(a.o + out * D + dim) =
                __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
          else
            *reinterpret_cast<float2*>(part.o + dim) = acc;
        }
        if (lane == 0) {
          if (whole) a.lse[out] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
          else *part.ml = make_float2(mx, sum);
        }
      }
    }
    const bool again = at.next(call, read);
    __syncwarp();  // every lane has read the old place
    if (lane == 0) sh_use[warp] = at;
    __syncwarp();
    if (!again) break;
  }
  // A stopping block lets its copies land before it leaves.
  for (; got < put; ++got) {
    drain_bar(&full[warp][got_slot], parity, a.timeout_ns);
    if (++got_slot == S::kStages) got_slot = 0, parity ^= 1;
  }
}

// Joins the partial results of an item that lies in several blocks' shares,
// in block order; a lane takes D / 32 dims.  Few parts (an item across one
// border or two, as in a batch): a warp per row.  More (a long history): a
// block per row, the parts dealt to its warps.
template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32) cache4_join_kernel(Cache4AttnArgs a) {
  using S = Shape<D, NT>;
  constexpr int kDims = D / 32;
  __shared__ float sh_o[kWarps][D], sh_m[kWarps], sh_l[kWarps];
  wait_for_stream();
  const int4 j = a.joins[blockIdx.x];
  if (j.x < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = j.z - (int)blockIdx.x + 2;
  const bool few = parts <= 4;
  const int row = few ? blockIdx.y * kWarps + warp : blockIdx.y;
  const int b = j.x, hk = j.y / a.row_blocks;
  const int r = (j.y - hk * a.row_blocks) * S::kRows + row;
  // (Uniform in the block where the block shares a row.)
  if (row >= S::kRows || r >= min(a.q_lens ? a.q_lens[b] : a.T, a.T) * a.heads) return;
  auto part = [&](int k) {
    return partial_of<D, NT>(a, k == 0 ? j.w : 2 * ((int)blockIdx.x + k - 1), row);
  };
  const int first = few ? 0 : warp, step = few ? 1 : kWarps;
  float mx = kNoMax;
  for (int k = few ? lane : threadIdx.x; k < parts; k += few ? 32 : kWarps * 32)
    mx = fmaxf(mx, part(k).ml->x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
  if (!few) {
    if (lane == 0) sh_m[warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sh_m[w]);
  }
  float acc[kDims], sum = 0.f;
#pragma unroll
  for (int i = 0; i < kDims; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int k = first; k < parts; k += step) {
    const Partial p = part(k);
    const float2 ml = *p.ml;
    const float f = ex2(ml.x - mx);
    sum += f * ml.y;
    if constexpr (D == 128) {
      const float4 v = reinterpret_cast<const float4*>(p.o)[lane];
      acc[0] += f * v.x, acc[1] += f * v.y, acc[2] += f * v.z, acc[3] += f * v.w;
    } else {
      const float2 v = reinterpret_cast<const float2*>(p.o)[lane];
      acc[0] += f * v.x, acc[1] += f * v.y;
    }
  }
  if (!few) {
#pragma unroll
    for (int i = 0; i < kDims; ++i) sh_o[warp][lane * kDims + i] = acc[i];
    if (lane == 0) sh_l[warp] = sum;
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < kWarps; ++w) {
      sum += sh_l[w];
#pragma unroll
      for (int i = 0; i < kDims; ++i) acc[i] += sh_o[w][lane * kDims + i];
    }
  }
  const float inv = sum > 0.f || sum != sum ? a.v_scale / sum : 0.f;
  const size_t q_row = row_at(a, b, hk, r);
  __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(a.o + q_row * D) + lane * (kDims / 2);
#pragma unroll
  for (int i = 0; i < kDims; i += 2)
    out[i / 2] = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
  if (lane == 0) a.lse[q_row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

template <int D, int NT, bool kHook = false>
cudaError_t run(const Cache4AttnArgs& a, int sm_count, cudaStream_t stream) {
  using S = Shape<D, NT>;
  // The hook has its own instantiation, for d = 128 and items of 8 rows only.
  if constexpr (D == 128 && NT == 1 && !kHook) {
    if (a.hook) return run<D, NT, true>(a, sm_count, stream);
  }
  auto* kernel = cache4_attn_kernel<D, NT, kHook>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), S::kSmem, done);
  if (e != cudaSuccess) return e;
  int blocks = sm_count * S::kBlocksPerSm;
  if (blocks > kC4MaxBlocks) blocks = kC4MaxBlocks;
  e = launch_overlapped(kernel, dim3(blocks), dim3(kWarps * 32), S::kSmem, stream, a);
  if (e != cudaSuccess) return e;
  const int rows = a.rows < S::kRows ? a.rows : S::kRows;
  return launch_overlapped(cache4_join_kernel<D, NT>, dim3(blocks, rows), dim3(kWarps * 32), 0,
                           stream, a);
}

}  // namespace

// Rows of an item: what makes the least of the passes over the keys, each of
// a cost by its width.  Measured, 16 requests of 8192 tokens x 8 heads (us):
//   d = 128, 16 rows: 62 as 8 + 8, 50 as 16;  24: 84 as 8s, 60 at once;
//            32: 84 as 16s, 74 at once;  40: 118 as 16s, 103 as 24s, 129 as
//            32s (at once it spills: not built);  64: 144 as 24s, 130 as 32s;
//            512 (x 4096 tokens): 258 as 24s, 245 as 32s
//   d = 64,  32 rows: 53 as 16s, 49 at once;  40: 70 as 24s, 58 at once;
//            64: 94 as 16s, 82 as 32s;  512: 158 as 32s, 153 as 40s
int cache4_attn_rows(int rows, int d) {
  const int cost[2][5] = {{22, 26, 36, 43, 52}, {32, 41, 52, 65, 0}};
  int best = 8;
  long long least = 0;
  for (int nt = 1; nt <= (d == 128 ? 4 : 5); ++nt) {
    const long long c = (rows + 8LL * nt - 1) / (8 * nt) * cost[d == 128][nt - 1];
    if (nt == 1 || c < least) least = c, best = 8 * nt;
  }
  return best;
}

cudaError_t launch_cache4_attn(const Cache4AttnArgs& a, int d, int sm_count, cudaStream_t stream) {
  const int nt = cache4_attn_rows(a.rows, d) / 8;
  if (d == 128)
    return nt == 1   ? run<128, 1>(a, sm_count, stream)
           : nt == 2 ? run<128, 2>(a, sm_count, stream)
           : nt == 3 ? run<128, 3>(a, sm_count, stream)
                     : run<128, 4>(a, sm_count, stream);
  return nt == 1   ? run<64, 1>(a, sm_count, stream)
         : nt == 2 ? run<64, 2>(a, sm_count, stream)
         : nt == 3 ? run<64, 3>(a, sm_count, stream)
         : nt == 4 ? run<64, 4>(a, sm_count, stream)
                   : run<64, 5>(a, sm_count, stream);
}

cudaError_t set_expire_site_cache4(uint32_t site) {
  return cudaMemcpyToSymbol(c_expire_site, &site, sizeof(site));
}

}  // namespace fa
