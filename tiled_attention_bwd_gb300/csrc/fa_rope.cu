// fa_rope.cu -- norms of the query and key heads with the rotation of their
// positions, from a projection's output [B,N,H+2Hkv,d] to the attention's
// q [B,H,N,d] and k, v [B,Hkv,N,d], and the gradient of that.
//
//   y = x * r * w,  r = (mean(x^2) + eps)^(-1/2)     (skipped without weights)
//   z = R(p) y      rotation by the table's cosine and sine of position p
//
// and, with dy = R(p)^T dz and xh = x r,
//
//   dw = sum over rows of dy * xh
//   dx = r * (dy w - xh * mean(dy w xh)).
//
// A head's row of d bf16 values lies in d/16 lanes of 16 values each, so a
// warp takes 32 / (d/16) heads of one token at a time ("pack"): 4 at d = 128,
// 8 at d = 64.  The two 8-value chunks of a lane are chosen such that both
// members of every rotated pair are in one lane; the norm's sums are the only
// exchange between lanes.  Everything is computed in fp32 and rounded to
// bf16 once, at the store.
//
// Bound by bytes, once the instructions are few enough: packed fp32
// arithmetic, no division in the loop, loads that cost no registers.  On a
// GB300 (copy bandwidth 6.79 TB/s), in a stream of calls: forward, 4 x 4096
// tokens of 64 + 16 heads of 128, 107 us or 6.3 TB/s; backward, 4 x 1024
// tokens of 32 + 64 heads, 48 us or 5.7 TB/s, and 7 x 3001 tokens of 24 + 16
// heads of 64, half of each rotated, 54 us or 5.6 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "fa_serve.h"

namespace fa {
namespace {

constexpr int kWarps = 8;  // per block

struct Raw {  // a lane's 16 bf16 values
  uint4 c[2];
};

// Two fp32 values in one 64-bit register: Blackwell's packed fp32
// instructions do both at once.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 un2(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(F2 v) {
  const float2 f = un2(v);
  return f.x + f.y;
}

__device__ __forceinline__ void unpack(const Raw& r, F2 (&x)[8]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t w[4] = {r.c[c].x, r.c[c].y, r.c[c].z, r.c[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[4 * c + i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
}

__device__ __forceinline__ uint32_t pack2(F2 v) {
  const float2 f = un2(v);
  const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ Raw pack(const F2 (&x)[8]) {
  Raw r;
#pragma unroll
  for (int c = 0; c < 2; ++c)
    r.c[c] = make_uint4(pack2(x[4 * c]), pack2(x[4 * c + 1]), pack2(x[4 * c + 2]),
                        pack2(x[4 * c + 3]));
  return r;
}

// Where a lane's chunks lie in its head's row.  Neighbouring lanes take
// neighbouring chunks, so that a warp's access covers whole sectors.
struct Lane {
  int j;            // lane within the head
  int sub;          // head within the pack
  int c0, c1;       // element offsets of the two chunks
  bool turn0, turn1;  // rotated (paired with one another, unless interleaved)
};

template <int D, bool kInter>
__device__ __forceinline__ Lane lane_of(int rot) {
  constexpr int kLanes = D / 16;
  const int l = threadIdx.x & 31;
  Lane a;
  a.j = l % kLanes;
  a.sub = l / kLanes;
  if (kInter) {
    a.c0 = 8 * a.j;
    a.c1 = 8 * (a.j + kLanes);
    a.turn0 = a.c0 < rot;
    a.turn1 = a.c1 < rot;
  } else {
    const int pairs = rot / 16;  // lanes with a rotated pair of chunks
    a.turn0 = a.turn1 = a.j < pairs;
    a.c0 = 8 * (a.turn0 ? a.j : a.j + pairs);
    a.c1 = 8 * (a.turn0 ? a.j + pairs : a.j + kLanes);
  }
  return a;
}

// `at`: the lane's first chunk of a row; the second is c1 - c0 elements on.
__device__ __forceinline__ void store_row(__nv_bfloat16* at, const Lane& a, const Raw& r) {
  *reinterpret_cast<uint4*>(at) = r.c[0];
  *reinterpret_cast<uint4*>(at + (a.c1 - a.c0)) = r.c[1];
}

// ---- A warp's ring of rows on their way from memory, in shared memory: the
// loads in flight then cost no registers.  A lane copies its own two chunks
// of each of kRows rows and reads them back itself; the rotation's row of
// the table, 64 bytes per lane of a head, is copied once for all the warp's
// heads.
template <int D, int kRows>
struct Ring {
  static constexpr int kLanes = D / 16;
  static constexpr int kTurn = kLanes * 64;
  static constexpr int kStage = kRows * 1024 + kTurn;
  uint8_t* base;  // this warp's
  static __device__ __forceinline__ void copy16(uint8_t* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
  }
  __device__ __forceinline__ void fetch_row(int stage, int which, const __nv_bfloat16* src,
                                            const Lane& l) const {
    uint8_t* at = base + stage * kStage + which * 1024 + (threadIdx.x & 31) * 16;
    copy16(at, src);
    copy16(at + 512, src + (l.c1 - l.c0));
  }
  __device__ __forceinline__ Raw row(int stage, int which) const {
    const uint8_t* at = base + stage * kStage + which * 1024 + (threadIdx.x & 31) * 16;
    Raw r;
    r.c[0] = *reinterpret_cast<const uint4*>(at);
    r.c[1] = *reinterpret_cast<const uint4*>(at + 512);
    return r;
  }
  // The table's rows hold rot/2 cosines, then rot/2 sines.  Positions are
  // clamped to the table.  Piece q of lane j: 4 cosines (q = 0, 1) or sines
  // (2, 3), of the pair's first or second four angles, or (interleaved) of
  // its first or second chunk's.
  template <bool kInter>
  __device__ __forceinline__ void fetch_turn(int stage, const RopeArgs& a, const Lane& l,
                                             int pos) const {
    if (l.sub >= 4 || !(l.sub & 1 ? l.turn1 : l.turn0)) return;
    pos = pos < 0 ? 0 : (pos >= a.table_rows ? a.table_rows - 1 : pos);
    const int first = kInter ? 4 * (l.j + (l.sub & 1) * kLanes) : 8 * l.j + 4 * (l.sub & 1);
    const float* src = a.table + (size_t)pos * a.rot + first + (l.sub >> 1) * (a.rot / 2);
    // (Through L1: the block's other warps are at the same token.)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(
                         base + stage * kStage + kRows * 1024 + (l.sub * kLanes + l.j) * 16))),
                 "l"(src)
                 : "memory");
  }
  __device__ __forceinline__ void turn_of(int stage, const Lane& l, F2 (&cs)[4],
                                          F2 (&sn)[4]) const {
    const uint8_t* at = base + stage * kStage + kRows * 1024 + l.j * 16;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(at + q * kLanes * 16);
      F2* d = (q < 2 ? cs : sn) + (q & 1) * 2;
      d[0] = u.x, d[1] = u.y;
    }
  }
  static __device__ __forceinline__ void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  template <int kLeft>
  static __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
  }
};

// Rotates the lane's 8 pairs by the angle (kBack: by minus the angle).
template <bool kInter, bool kBack>
__device__ __forceinline__ void turn(F2 (&y)[8], const F2 (&cs)[4], const F2 (&sn)[4],
                                     const Lane& l) {
  if (!kInter && !l.turn0) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kInter && !(i < 2 ? l.turn0 : l.turn1)) continue;
    if constexpr (kInter) {  // pairs 2i and 2i + 1 are y[2i] and y[2i + 1]
      const float2 c = un2(cs[i]), s = un2(sn[i]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 v = un2(y[2 * i + h]);
        const float cc = h ? c.y : c.x, ss = (h ? s.y : s.x) * (kBack ? -1.f : 1.f);
        y[2 * i + h] = fma2(f2(v.x, v.y), f2(cc, cc), mul2(f2(v.y, v.x), f2(-ss, ss)));
      }
    } else {  // pairs 2i and 2i + 1 are (y[i], y[i + 4]), both halves
      const float2 s = un2(sn[i]);
      const F2 minus = f2(-s.x, -s.y), u = y[i], v = y[i + 4];
      y[i] = fma2(v, kBack ? sn[i] : minus, mul2(u, cs[i]));
      y[i + 4] = fma2(u, kBack ? minus : sn[i], mul2(v, cs[i]));
    }
  }
}

template <int D>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int m = D / 32; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// The lane's 16 norm weights, of either type (once per warp).
__device__ __forceinline__ void load_weight(const void* w, int is_bf16, const Lane& l,
                                            F2 (&out)[8]) {
  float f[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int i = (e < 8 ? l.c0 : l.c1 - 8) + e;
    f[e] = is_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i])
                   : static_cast<const float*>(w)[i];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = f2(f[2 * e], f[2 * e + 1]);
}

__device__ __forceinline__ int position_of(const RopeArgs& a, int token, int n) {
  return a.positions ? a.positions[token] : n;
}

// A warp's work: one pack of heads (query heads' packs first, then key heads',
// then value heads'; a pack never mixes kinds) of the tokens `first`, `first`
// + step, ... .  With the pack fixed, its weights (and in the backward their
// gradient's sums) stay in registers and the next token's place follows from
// the last without a division.  Warps next to one another take one token's
// packs, i.e. neighbouring memory.
struct Task {
  int kind;    // 0 query, 1 key, 2 value
  int head;    // of this lane, within its kind
  int heads;   // of the kind
  int column;  // of this lane's head in a token of qkv
  bool live;   // this lane has a head
};
template <int D>
__device__ __forceinline__ Task task_of(const RopeArgs& a, int pack, const Lane& l) {
  constexpr int kPack = 512 / D;
  const int nq = (a.H + kPack - 1) / kPack, nk = (a.Hkv + kPack - 1) / kPack;
  Task k;
  k.kind = pack < nq ? 0 : (pack < nq + nk ? 1 : 2);
  k.head = (pack - (k.kind == 0 ? 0 : (k.kind == 1 ? nq : nq + nk))) * kPack + l.sub;
  k.heads = k.kind == 0 ? a.H : a.Hkv;
  k.column = (k.kind == 0 ? 0 : (k.kind == 1 ? a.H : a.H + a.Hkv)) + k.head;
  k.live = k.head < k.heads;
  return k;
}

// A token of the batch, stepped without division; true where the step moves
// on by one more batch entry than step_b.
struct Place {
  int token, n;
  __device__ __forceinline__ bool advance(const RopeDeal& s, int N) {
    token += s.step;
    n += s.step_n;
    if (n < N) return false;
    n -= N;
    return true;
  }
};
// The lane's first chunk of a head's row at a Place, stepped along with it.
template <typename T>
struct Walk {
  T* at;
  long long step, wrap;  // elements; wrap is added where advance() says so
  // Strides of entries and tokens, in elements.
  __device__ __forceinline__ Walk(const RopeDeal& s, int N, T* base, long long sb, long long sn,
                                  int b, int n)
      : at(base + b * sb + n * sn), step(s.step_b * sb + s.step_n * sn), wrap(sb - N * sn) {}
  __device__ __forceinline__ void advance(bool w) { at += w ? step + wrap : step; }
};

// Stages of the rings: 3 to 6 of them measure the same within 2%.  Three blocks
// of the forward per SM (80 registers): 111 us at 4 x 4096 tokens, two 125.
constexpr int kFwdStages = 3, kBwdStages = 4;
template <int D>
constexpr int fwd_smem() { return kWarps * kFwdStages * Ring<D, 1>::kStage; }
template <int D>
constexpr int bwd_smem() { return kWarps * kBwdStages * Ring<D, 2>::kStage; }

// Forward: bound by bytes, each read and written once.
template <int D, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kWarps * 32, 3) rope_fwd_kernel(RopeArgs a) {
  using R = Ring<D, 1>;
  extern __shared__ __align__(16) uint8_t smem[];
  const Lane l = lane_of<D, kInter>(a.rot);
  const int warp = threadIdx.x >> 5, id = blockIdx.x * kWarps + warp;
  const Task k = task_of<D>(a, id % a.all.packs, l);
  Place here = {id / a.all.packs, 0};
  // (There may be more warps than whole tokens need.)
  if (here.token >= a.all.step || here.token >= a.tokens) return;
  const int b = here.token / a.N;
  here.n = here.token - b * a.N;
  const R ring = {smem + warp * kFwdStages * R::kStage};
  wait_for_stream();
  const bool turns = k.kind < 2;
  F2 w[8];
  if (kNorm && turns) load_weight(k.kind == 0 ? a.q_weight : a.k_weight, a.weight_bf16, l, w);
  Walk<const __nv_bfloat16> in(a.all, a.N, a.qkv + (size_t)k.column * D + l.c0, a.stride_b,
                               a.stride_n, b, here.n);
  __nv_bfloat16* to = k.kind == 0 ? a.q : (k.kind == 1 ? a.k : a.v);
  Walk<__nv_bfloat16> out(a.all, a.N, to + (size_t)k.head * a.N * D + l.c0,
                          (long long)k.heads * a.N * D, D, b, here.n);

  Place ahead = here;  // next to be fetched, with its position
  bool any = true;     // there is one
  int pos = turns ? position_of(a, ahead.token, ahead.n) : 0;
  auto fetch = [&](int stage) {
    if (any) {
      if (k.live) ring.fetch_row(stage, 0, in.at, l);
      if (turns) ring.template fetch_turn<kInter>(stage, a, l, pos);
      any = a.tokens - ahead.token > a.all.step;
      in.advance(ahead.advance(a.all, a.N));
      if (any && turns) pos = position_of(a, ahead.token, ahead.n);
    }
    R::commit();
  };
#pragma unroll
  for (int s = 0; s < kFwdStages - 1; ++s) fetch(s);
  for (int stage = 0;; stage = stage == kFwdStages - 1 ? 0 : stage + 1) {
    R::template wait<kFwdStages - 2>();
    __syncwarp();  // the table's pieces of other lanes; and all have read the last stage
    Raw raw = ring.row(stage, 0);
    F2 x[8], cs[4], sn[4];
    if (turns) ring.turn_of(stage, l, cs, sn);
    fetch(stage == 0 ? kFwdStages - 1 : stage - 1);
    if (turns) {
      unpack(raw, x);
      if (kNorm) {
        F2 ss = mul2(x[0], x[0]);
#pragma unroll
        for (int e = 1; e < 8; ++e) ss = fma2(x[e], x[e], ss);
        const float r = rsqrtf(sum_lanes<D>(sum2(ss)) * (1.0f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = mul2(mul2(x[e], f2(r, r)), w[e]);
      }
      turn<kInter, false>(x, cs, sn, l);
      raw = pack(x);
    }
    if (k.live) store_row(out.at, l, raw);
    if (a.tokens - here.token <= a.all.step) break;
    out.advance(here.advance(a.all, a.N));
  }
}

// Backward.  The warps first take the query and key packs together, then the
// value packs, which are only moved: all warps do the same work (51 us at
// 4 x 1024 tokens; 57 us with warps of value packs beside the others).  A lane sums
// its 16 dims of its weight's gradient over all its rows; heads of a warp,
// warps of a block (by kind) and blocks follow in that order, the last in
// rope_dw_kernel: the result does not depend on which block runs first.
template <int D, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kWarps * 32, 2) rope_bwd_kernel(RopeArgs a) {
  using R = Ring<D, 2>;
  constexpr int kPack = 512 / D;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float sums[kWarps][D];
  __shared__ int kinds[kWarps];
  const Lane l = lane_of<D, kInter>(a.rot);
  const int warp = threadIdx.x >> 5, id = blockIdx.x * kWarps + warp;
  const R ring = {smem + warp * kBwdStages * R::kStage};
  wait_for_stream();
  F2 dw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = 0;

  // One of the two deals; kGrad: query and key heads.
  auto take = [&](auto grad, const RopeDeal& s, int first_pack) {
    constexpr bool kGrad = decltype(grad)::value, kX = kGrad && kNorm;
    if (s.packs == 0) return;
    const Task k = task_of<D>(a, first_pack + id % s.packs, l);
    Place here = {id / s.packs, 0};
    // (There may be more warps than whole tokens need.)
    if (here.token >= s.step || here.token >= a.tokens) return;
    const int b = here.token / a.N;
    here.n = here.token - b * a.N;
    F2 w[8];
    if (kX) load_weight(k.kind == 0 ? a.q_weight : a.k_weight, a.weight_bf16, l, w);
    Walk<const __nv_bfloat16> in(s, a.N, a.qkv + (size_t)k.column * D + l.c0, a.stride_b,
                                 a.stride_n, b, here.n);
    const __nv_bfloat16* from = k.kind == 0 ? a.dq : (k.kind == 1 ? a.dk : a.dv);
    Walk<const __nv_bfloat16> dz(s, a.N, from + (size_t)k.head * a.N * D + l.c0,
                                 (long long)k.heads * a.N * D, D, b, here.n);
    Walk<__nv_bfloat16> out(s, a.N, a.dqkv + (size_t)k.column * D + l.c0, a.dstride_b, a.dstride_n,
                            b, here.n);
    Place ahead = here;  // next to be fetched, with its position
    bool any = true;     // there is one
    int pos = kGrad ? position_of(a, ahead.token, ahead.n) : 0;
    auto fetch = [&](int stage) {
      if (any) {
        if (k.live) {
          ring.fetch_row(stage, 0, dz.at, l);
          if (kX) ring.fetch_row(stage, 1, in.at, l);
        }
        if (kGrad) ring.template fetch_turn<kInter>(stage, a, l, pos);
        any = a.tokens - ahead.token > s.step;
        const bool wrap = ahead.advance(s, a.N);
        dz.advance(wrap);
        if (kX) in.advance(wrap);
        if (kGrad && any) pos = position_of(a, ahead.token, ahead.n);
      }
      R::commit();
    };
#pragma unroll
    for (int st = 0; st < kBwdStages - 1; ++st) fetch(st);
    for (int stage = 0;; stage = stage == kBwdStages - 1 ? 0 : stage + 1) {
      R::template wait<kBwdStages - 2>();
      __syncwarp();  // the table's pieces of other lanes; and all have read the last stage
      Raw gx = ring.row(stage, 0), rx = {};
      if (kX) rx = ring.row(stage, 1);
      F2 g[8], cs[4], sn[4];
      if (kGrad) ring.turn_of(stage, l, cs, sn);
      fetch(stage == 0 ? kBwdStages - 1 : stage - 1);
      if constexpr (kGrad) {
        unpack(gx, g);
        turn<kInter, true>(g, cs, sn, l);
        if constexpr (kNorm) {
          F2 x[8];
          unpack(rx, x);
          F2 ss = mul2(x[0], x[0]), dot = 0;
#pragma unroll
          for (int e = 1; e < 8; ++e) ss = fma2(x[e], x[e], ss);
          const float r = rsqrtf(sum_lanes<D>(sum2(ss)) * (1.0f / D) + a.eps);
          const F2 r2 = f2(r, r);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = mul2(x[e], r2);  // xh
            dw[e] = fma2(g[e], x[e], dw[e]);
            g[e] = mul2(g[e], w[e]);
            dot = fma2(g[e], x[e], dot);
          }
          const float mean = -sum_lanes<D>(sum2(dot)) * (1.0f / D);
          const F2 m2 = f2(mean, mean);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = mul2(r2, fma2(x[e], m2, g[e]));
        }
        gx = pack(g);
      }
      if (k.live) store_row(out.at, l, gx);
      if (a.tokens - here.token <= s.step) break;
      out.advance(here.advance(s, a.N));
    }
    if (kX && !k.live)  // no head: whatever the ring held
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[e] = 0;
    R::template wait<0>();
    __syncwarp();  // the ring is free for the next deal
  };
  take(std::true_type{}, a.grad, 0);
  take(std::false_type{}, a.value, a.grad.packs);
  if constexpr (kNorm) {
    const int kind = id % max(a.grad.packs, 1) < (a.H + kPack - 1) / kPack ? 0 : 1;
    // Heads of a pack, then the block's warps of each kind.
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 pair = un2(dw[e / 2]);
      float v = e & 1 ? pair.y : pair.x;
#pragma unroll
      for (int m = D / 16; m < 32; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
      if (l.sub == 0) sums[warp][(e < 8 ? l.c0 : l.c1 - 8) + e] = v;
    }
    if ((threadIdx.x & 31) == 0) kinds[warp] = kind;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v)
        if (kinds[v] == i / D) s += sums[v][i % D];
      a.partial[(size_t)blockIdx.x * 2 * D + i] = s;
    }
  }
}

// Weight gradients from the blocks' sums: 32 columns of the 2 D (queries',
// then keys') per block, 32 rows at a time.
template <int D>
__global__ void __launch_bounds__(1024) rope_dw_kernel(RopeArgs a) {
  __shared__ float sums[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  wait_for_stream();
  float s = 0.f;
#pragma unroll 8
  for (int i = threadIdx.y; i < a.blocks; i += 32) s += a.partial[(size_t)i * 2 * D + col];
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = sums[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  const int c = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0) (c < D ? a.dq_weight : a.dk_weight)[c % D] = s;
}

// Tokens that `blocks` take at a time when their warps share `packs` packs.
RopeDeal deal(const RopeArgs& a, int blocks, int packs) {
  RopeDeal s = {};
  s.packs = packs;
  if (packs == 0 || a.N == 0) return s;
  s.step = blocks * kWarps / packs;
  s.step_b = s.step / a.N;
  s.step_n = s.step % a.N;
  return s;
}
// `resident` blocks per SM, fewer if there is less than one of `packs` packs
// of a token for each warp, and at least a warp for every pack of one token.
int blocks_for(const RopeArgs& a, int packs, int sm_count, int resident) {
  long long blocks = ((long long)a.tokens * packs + kWarps - 1) / kWarps;
  if (blocks > (long long)resident * sm_count) blocks = (long long)resident * sm_count;
  if (blocks > kRopeMaxBlocks) blocks = kRopeMaxBlocks;
  const int least = (packs + kWarps - 1) / kWarps;
  return blocks < least ? least : (int)blocks;
}
template <int D>
int packs_of(int heads) { return (heads + 512 / D - 1) / (512 / D); }

template <int D, bool kInter, bool kNorm>
cudaError_t fwd(RopeArgs a, int sm_count, cudaStream_t stream) {
  const int packs = packs_of<D>(a.H) + 2 * packs_of<D>(a.Hkv);
  const int blocks = blocks_for(a, packs, sm_count, 3);
  a.all = deal(a, blocks, packs);
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(rope_fwd_kernel<D, kInter, kNorm>), fwd_smem<D>(), done);
  if (e != cudaSuccess) return e;
  return launch_overlapped(rope_fwd_kernel<D, kInter, kNorm>, dim3(blocks), dim3(kWarps * 32),
                           fwd_smem<D>(), stream, a);
}

template <int D, bool kInter, bool kNorm>
cudaError_t bwd(RopeArgs a, int sm_count, cudaStream_t stream) {
  const int packs = packs_of<D>(a.H) + packs_of<D>(a.Hkv);
  const int blocks = blocks_for(a, packs, sm_count, 2);
  a.grad = deal(a, blocks, packs);
  a.value = deal(a, blocks, packs_of<D>(a.Hkv));
  a.blocks = blocks;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(rope_bwd_kernel<D, kInter, kNorm>), bwd_smem<D>(), done);
  if (e != cudaSuccess) return e;
  if (blocks > 0)
    e = launch_overlapped(rope_bwd_kernel<D, kInter, kNorm>, dim3(blocks), dim3(kWarps * 32),
                          bwd_smem<D>(), stream, a);
  if (e != cudaSuccess || !kNorm) return e;
  return launch_overlapped(rope_dw_kernel<D>, dim3(2 * D / 32), dim3(32, 32), 0, stream, a);
}

template <bool kBwd>
cudaError_t pick(const RopeArgs& a, int d, bool inter, bool norm, int sm_count,
                 cudaStream_t s) {
#define FA_ROPE(DD, II, NN) \
  return kBwd ? bwd<DD, II, NN>(a, sm_count, s) : fwd<DD, II, NN>(a, sm_count, s)
  if (d == 128) {
    if (inter) { if (norm) FA_ROPE(128, true, true); else FA_ROPE(128, true, false); }
    else       { if (norm) FA_ROPE(128, false, true); else FA_ROPE(128, false, false); }
  }
  if (inter) { if (norm) FA_ROPE(64, true, true); else FA_ROPE(64, true, false); }
  if (norm) FA_ROPE(64, false, true); else FA_ROPE(64, false, false);
#undef FA_ROPE
}

}  // namespace

cudaError_t launch_rope_fwd(const RopeArgs& a, int d, bool interleaved, bool norm, int sm_count,
                            cudaStream_t stream) {
  return pick<false>(a, d, interleaved, norm, sm_count, stream);
}
cudaError_t launch_rope_bwd(const RopeArgs& a, int d, bool interleaved, bool norm, int sm_count,
                            cudaStream_t stream) {
  return pick<true>(a, d, interleaved, norm, sm_count, stream);
}

}  // namespace fa
