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
// members of every rotated pair are in one lane: chunks j and j + rot/16 for
// pairs (i, i + rot/2), chunks 2j and 2j + 1 for pairs (2i, 2i + 1).  The
// norm's sums are the only exchange between lanes.  Everything is computed
// in fp32 and rounded to bf16 once, at the store.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_launch.h"

namespace fa {
namespace {

constexpr int kWarps = 8;  // per block

struct Raw {  // a lane's 16 bf16 values
  uint4 c[2];
};

__device__ __forceinline__ void unpack(const Raw& r, float* f) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t w[4] = {r.c[c].x, r.c[c].y, r.c[c].z, r.c[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[8 * c + 2 * i] = __uint_as_float(w[i] << 16);
      f[8 * c + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}

__device__ __forceinline__ Raw pack(const float* f) {
  Raw r;
#pragma unroll
  for (int c = 0; c < 2; ++c)
    r.c[c] = make_uint4(pack2(f[8 * c], f[8 * c + 1]), pack2(f[8 * c + 2], f[8 * c + 3]),
                        pack2(f[8 * c + 4], f[8 * c + 5]), pack2(f[8 * c + 6], f[8 * c + 7]));
  return r;
}

// Where a lane's chunks lie in its head's row.
struct Lane {
  int j;        // lane within the head
  int sub;      // head within the pack
  int c0, c1;   // element offsets of the two chunks
  bool turned;  // both chunks are rotated (else neither is)
};

template <int D, bool kInter>
__device__ __forceinline__ Lane lane_of(int rot) {
  constexpr int kLanes = D / 16;
  const int l = threadIdx.x & 31;
  Lane a;
  a.j = l % kLanes;
  a.sub = l / kLanes;
  a.turned = a.j < rot / 16;
  const bool split = !kInter && a.turned;
  a.c0 = 8 * (split ? a.j : 2 * a.j);
  a.c1 = 8 * (split ? a.j + rot / 16 : 2 * a.j + 1);
  return a;
}

__device__ __forceinline__ Raw load_row(const __nv_bfloat16* row, const Lane& a) {
  // Plain loads: the backward's output may be its input.
  Raw r;
  r.c[0] = *reinterpret_cast<const uint4*>(row + a.c0);
  r.c[1] = *reinterpret_cast<const uint4*>(row + a.c1);
  return r;
}
__device__ __forceinline__ void store_row(__nv_bfloat16* row, const Lane& a, const Raw& r) {
  *reinterpret_cast<uint4*>(row + a.c0) = r.c[0];
  *reinterpret_cast<uint4*>(row + a.c1) = r.c[1];
}

// The lane's 8 cosines and sines of position `pos` (the table's rows hold
// rot/2 cosines, then rot/2 sines).  Positions are clamped to the table.
__device__ __forceinline__ void load_turn(const RopeArgs& a, const Lane& l, int pos, float* cs,
                                          float* sn) {
  if (!l.turned) return;
  pos = pos < 0 ? 0 : (pos >= a.table_rows ? a.table_rows - 1 : pos);
  const float* row = a.table + (size_t)pos * a.rot + 8 * l.j;
  const float4* c = reinterpret_cast<const float4*>(row);
  const float4* s = reinterpret_cast<const float4*>(row + a.rot / 2);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 u = __ldg(c + h), v = __ldg(s + h);
    cs[4 * h] = u.x, cs[4 * h + 1] = u.y, cs[4 * h + 2] = u.z, cs[4 * h + 3] = u.w;
    sn[4 * h] = v.x, sn[4 * h + 1] = v.y, sn[4 * h + 2] = v.z, sn[4 * h + 3] = v.w;
  }
}

// Rotates the lane's 8 pairs by the angle (kBack: by minus the angle).
template <bool kInter, bool kBack>
__device__ __forceinline__ void turn(float* y, const float* cs, const float* sn) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int p = kInter ? 2 * i : i, q = kInter ? 2 * i + 1 : i + 8;
    const float u = y[p], v = y[q], s = kBack ? -sn[i] : sn[i];
    y[p] = u * cs[i] - v * s;
    y[q] = v * cs[i] + u * s;
  }
}

template <int D>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int m = D / 32; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// A norm weight of either type.
__device__ __forceinline__ float weight_at(const void* w, int is_bf16, int i) {
  return is_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i])
                 : static_cast<const float*>(w)[i];
}

__device__ __forceinline__ void load_weight(const float* w, const Lane& l, float* out) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float4* p = reinterpret_cast<const float4*>(w + (c ? l.c1 : l.c0));
    const float4 u = p[0], v = p[1];
    out[8 * c] = u.x, out[8 * c + 1] = u.y, out[8 * c + 2] = u.z, out[8 * c + 3] = u.w;
    out[8 * c + 4] = v.x, out[8 * c + 5] = v.y, out[8 * c + 6] = v.z, out[8 * c + 7] = v.w;
  }
}

__device__ __forceinline__ int position_of(const RopeArgs& a, int token, int n) {
  return a.positions ? __ldg(a.positions + token) : n;
}

// Packs of one token: the query heads', then the key heads', then the value
// heads'; a pack never mixes kinds.
struct PackOf {
  int kind;   // 0 query, 1 key, 2 value
  int head;   // of this lane, within its kind
  int heads;  // of the kind
};
template <int D>
__device__ __forceinline__ PackOf pack_of(const RopeArgs& a, int p, const Lane& l) {
  constexpr int kPack = 512 / D;
  const int nq = (a.H + kPack - 1) / kPack, nk = (a.Hkv + kPack - 1) / kPack;
  PackOf r;
  r.kind = p < nq ? 0 : (p < nq + nk ? 1 : 2);
  r.head = (p - (r.kind == 0 ? 0 : (r.kind == 1 ? nq : nq + nk))) * kPack + l.sub;
  r.heads = r.kind == 0 ? a.H : a.Hkv;
  return r;
}
__device__ __forceinline__ int column_of(const RopeArgs& a, const PackOf& p) {
  return (p.kind == 0 ? 0 : (p.kind == 1 ? a.H : a.H + a.Hkv)) + p.head;
}

// One block: `tokens_per_block` tokens and the packs [first, first + count)
// of each, one (token, pack) per warp at a time.
template <int D, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kWarps * 32) rope_fwd_kernel(RopeArgs a) {
  __shared__ __align__(16) float w_sh[2][D];
  if (kNorm) {
    for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32)
      w_sh[i / D][i % D] = weight_at(i < D ? a.q_weight : a.k_weight, a.weight_bf16, i % D);
    __syncthreads();
  }
  const Lane l = lane_of<D, kInter>(a.rot);
  const int first = blockIdx.y * a.packs_per_block;
  const int count = min(a.packs_per_block, a.packs - first);
  const int t0 = blockIdx.x * a.tokens_per_block;
  const int here = min(a.tokens_per_block, a.tokens - t0) * count;
  for (int i = threadIdx.x >> 5; i < here; i += kWarps) {
    const int token = t0 + i / count;
    const PackOf p = pack_of<D>(a, first + i % count, l);
    const bool live = p.head < p.heads;
    const int b = token / a.N, n = token - b * a.N;
    Raw raw = {};
    if (live)
      raw = load_row(a.qkv + b * a.stride_b + n * a.stride_n + (size_t)column_of(a, p) * D, l);
    if (p.kind < 2) {
      float x[16], cs[8], sn[8];
      load_turn(a, l, position_of(a, token, n), cs, sn);
      unpack(raw, x);
      if (kNorm) {
        float ss = 0.f, w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
        const float r = rsqrtf(sum_lanes<D>(ss) * (1.0f / D) + a.eps);
        load_weight(w_sh[p.kind], l, w);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = x[e] * r * w[e];
      }
      if (l.turned) turn<kInter, false>(x, cs, sn);
      raw = pack(x);
    }
    if (live) {
      __nv_bfloat16* out = p.kind == 0 ? a.q : (p.kind == 1 ? a.k : a.v);
      store_row(out + (((size_t)b * p.heads + p.head) * a.N + n) * D, l, raw);
    }
  }
}

// Backward.  Blocks take one kind of head each (block ranges [0, split[0])
// queries, [split[0], split[1]) keys, the rest values), so that a lane keeps
// one set of 16 partial sums of its weight's gradient over all its rows.
// Block sums leave in fp32 and rope_dw_kernel adds them in block order: the
// result does not depend on which block runs first.
template <int D, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kWarps * 32) rope_bwd_kernel(RopeArgs a) {
  constexpr int kPack = 512 / D;
  __shared__ __align__(16) float w_sh[D];
  __shared__ float sums[kWarps][D];
  const int kind = (int)blockIdx.x < a.split[0] ? 0 : ((int)blockIdx.x < a.split[1] ? 1 : 2);
  const int block0 = kind == 0 ? 0 : a.split[kind - 1];
  const int blocks = (kind == 2 ? (int)gridDim.x : a.split[kind]) - block0;
  if (kNorm && kind < 2) {
    for (int i = threadIdx.x; i < D; i += kWarps * 32)
      w_sh[i] = weight_at(kind == 0 ? a.q_weight : a.k_weight, a.weight_bf16, i);
    __syncthreads();
  }
  const Lane l = lane_of<D, kInter>(a.rot);
  const int heads = kind == 0 ? a.H : a.Hkv;
  const int column0 = kind == 0 ? 0 : (kind == 1 ? a.H : a.H + a.Hkv);
  const unsigned packs = (heads + kPack - 1) / kPack;
  const __nv_bfloat16* dz = kind == 0 ? a.dq : (kind == 1 ? a.dk : a.dv);
  float w[16], dw[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) dw[e] = 0.f;
  if (kNorm && kind < 2) load_weight(w_sh, l, w);

  const unsigned total = (unsigned)a.tokens * packs;
  const unsigned step = blocks * kWarps;
  for (unsigned i = (blockIdx.x - block0) * kWarps + (threadIdx.x >> 5); i < total; i += step) {
    const int token = i / packs;
    const int head = (i - token * packs) * kPack + l.sub;
    const bool live = head < heads;
    const int b = token / a.N, n = token - b * a.N;
    Raw gx = {}, rx = {};
    if (live) {
      gx = load_row(dz + (((size_t)b * heads + head) * a.N + n) * D, l);
      if (kNorm && kind < 2)
        rx = load_row(a.qkv + b * a.stride_b + n * a.stride_n + (size_t)(column0 + head) * D, l);
    }
    if (kind < 2) {
      float g[16], cs[8], sn[8];
      load_turn(a, l, position_of(a, token, n), cs, sn);
      unpack(gx, g);
      if (l.turned) turn<kInter, true>(g, cs, sn);
      if (kNorm) {
        float x[16];
        unpack(rx, x);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
        const float r = rsqrtf(sum_lanes<D>(ss) * (1.0f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          x[e] *= r;  // xh
          dw[e] = fmaf(g[e], x[e], dw[e]);
          g[e] *= w[e];
          dot = fmaf(g[e], x[e], dot);
        }
        const float mean = sum_lanes<D>(dot) * (1.0f / D);
#pragma unroll
        for (int e = 0; e < 16; ++e) g[e] = r * fmaf(-x[e], mean, g[e]);
      }
      gx = pack(g);
    }
    if (live)
      store_row(a.dqkv + b * a.dstride_b + n * a.dstride_n + (size_t)(column0 + head) * D, l, gx);
  }
  if constexpr (kNorm) {
    if (kind == 2) return;  // the block has one kind: all leave
    // Heads of a pack, then warps of the block.
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
      for (int m = D / 16; m < 32; m <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], m);
    }
    if (l.sub == 0) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        sums[threadIdx.x >> 5][(e < 8 ? l.c0 : l.c1 - 8) + e] = dw[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kWarps * 32) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) s += sums[v][i];
      a.partial[(size_t)blockIdx.x * D + i] = s;
    }
  }
}

// Weight gradients from the block sums: one warp of 32 rows x 32 columns per
// block; kind 0 (queries) and 1 (keys) in blockIdx.y.
template <int D>
__global__ void __launch_bounds__(1024) rope_dw_kernel(RopeArgs a) {
  __shared__ float sums[32][33];
  const int kind = blockIdx.y;
  const int b0 = kind == 0 ? 0 : a.split[0], b1 = a.split[kind];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  for (int i = b0 + threadIdx.y; i < b1; i += 32) s += a.partial[(size_t)i * D + col];
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = sums[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  if (threadIdx.x == 0) (kind == 0 ? a.dq_weight : a.dk_weight)[blockIdx.x * 32 + threadIdx.y] = s;
}

template <int D, bool kInter, bool kNorm>
cudaError_t fwd(RopeArgs a, int sm_count, cudaStream_t stream) {
  constexpr int kPack = 512 / D;
  a.packs = (a.H + kPack - 1) / kPack + 2 * ((a.Hkv + kPack - 1) / kPack);
  // Few tokens: one pack per warp, spread over blocks.  Otherwise whole
  // tokens, about four packs per warp.
  const long long all = (long long)a.tokens * a.packs;
  if (all < (long long)sm_count * kWarps * 16) {
    a.tokens_per_block = 1;
    a.packs_per_block = kWarps;
  } else {
    a.packs_per_block = a.packs;
    a.tokens_per_block = (4 * kWarps + a.packs - 1) / a.packs;
  }
  const dim3 grid((a.tokens + a.tokens_per_block - 1) / a.tokens_per_block,
                  (a.packs + a.packs_per_block - 1) / a.packs_per_block);
  rope_fwd_kernel<D, kInter, kNorm><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, bool kInter, bool kNorm>
cudaError_t bwd(RopeArgs a, int sm_count, cudaStream_t stream) {
  constexpr int kPack = 512 / D;
  const long long pq = (a.H + kPack - 1) / kPack, pk = (a.Hkv + kPack - 1) / kPack;
  // Blocks in proportion to the packs of each kind, at least one each.
  const long long all = a.tokens * (pq + 2 * pk);
  long long grid = (all + kWarps - 1) / kWarps;
  if (grid > 4LL * sm_count) grid = 4LL * sm_count;
  if (grid > kRopeMaxBlocks) grid = kRopeMaxBlocks;
  if (grid < 3) grid = 3;
  long long k = grid * pk / (pq + 2 * pk);
  if (k < 1) k = 1;
  a.split[0] = (int)(grid - 2 * k);
  a.split[1] = (int)(grid - k);
  rope_bwd_kernel<D, kInter, kNorm><<<(int)grid, kWarps * 32, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !kNorm) return e;
  rope_dw_kernel<D><<<dim3(D / 32, 2), dim3(32, 32), 0, stream>>>(a);
  return cudaGetLastError();
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
