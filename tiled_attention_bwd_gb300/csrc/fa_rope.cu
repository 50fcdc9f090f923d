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

// The lane's 16 norm weights, of either type (once per warp).
__device__ __forceinline__ void load_weight(const void* w, int is_bf16, const Lane& l, float* out) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int i = (e < 8 ? l.c0 : l.c1 - 8) + e;
    out[e] = is_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i])
                     : static_cast<const float*>(w)[i];
  }
}

__device__ __forceinline__ int position_of(const RopeArgs& a, int token, int n) {
  return a.positions ? __ldg(a.positions + token) : n;
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

// A place in the batch, stepped without division.
struct Place {
  int token, b, n;
  __device__ __forceinline__ Place(const RopeArgs& a, int token_) : token(token_) {
    b = token / a.N;
    n = token - b * a.N;
  }
  __device__ __forceinline__ void advance(const RopeArgs& a) {
    token += a.step;
    b += a.step_b;
    n += a.step_n;
    if (n >= a.N) n -= a.N, ++b;
  }
};

// Forward: bound by bytes, each read and written once.  The next token's row
// and position are loaded before the present one is computed.
template <int D, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kWarps * 32) rope_fwd_kernel(RopeArgs a) {
  const Lane l = lane_of<D, kInter>(a.rot);
  const int id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const Task k = task_of<D>(a, id % a.packs, l);
  if (id / a.packs >= a.step) return;  // more warps than whole tokens need
  float w[16];
  if (kNorm && k.kind < 2) load_weight(k.kind == 0 ? a.q_weight : a.k_weight, a.weight_bf16, l, w);
  __nv_bfloat16* out = k.kind == 0 ? a.q : (k.kind == 1 ? a.k : a.v);
  auto row_at = [&](const Place& p) {
    Raw r = {};
    if (k.live)
      r = load_row(a.qkv + p.b * a.stride_b + p.n * a.stride_n + (size_t)k.column * D, l);
    return r;
  };
  Place here(a, id / a.packs);
  if (here.token >= a.tokens) return;
  Raw raw = row_at(here);
  int pos = position_of(a, here.token, here.n);
  while (true) {
    Place next = here;
    const bool more = a.tokens - here.token > a.step;
    next.advance(a);
    float x[16], cs[8], sn[8];
    if (k.kind < 2) load_turn(a, l, pos, cs, sn);
    Raw ahead = {};
    if (more) {
      ahead = row_at(next);
      pos = position_of(a, next.token, next.n);
    }
    if (k.kind < 2) {
      unpack(raw, x);
      if (kNorm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
        const float r = rsqrtf(sum_lanes<D>(ss) * (1.0f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = x[e] * r * w[e];
      }
      if (l.turned) turn<kInter, false>(x, cs, sn);
      raw = pack(x);
    }
    if (k.live)
      store_row(out + (((size_t)here.b * k.heads + k.head) * a.N + here.n) * D, l, raw);
    if (!more) break;
    here = next;
    raw = ahead;
  }
}

// Backward.  A lane sums its 16 dims of its weight's gradient over all its
// rows; heads of a warp, warps of a block (by kind) and blocks follow in
// that order, the last in rope_dw_kernel: the result does not depend on
// which block runs first.
template <int D, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kWarps * 32, 2) rope_bwd_kernel(RopeArgs a) {
  __shared__ float sums[kWarps][D];
  __shared__ int kinds[kWarps];
  const Lane l = lane_of<D, kInter>(a.rot);
  const int id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const Task k = task_of<D>(a, id % a.packs, l);
  const __nv_bfloat16* dz = k.kind == 0 ? a.dq : (k.kind == 1 ? a.dk : a.dv);
  const bool norm = kNorm && k.kind < 2;
  float w[16], dw[16];
  if (norm) load_weight(k.kind == 0 ? a.q_weight : a.k_weight, a.weight_bf16, l, w);
#pragma unroll
  for (int e = 0; e < 16; ++e) dw[e] = 0.f;
  auto dz_at = [&](const Place& p) {
    Raw r = {};
    if (k.live) r = load_row(dz + (((size_t)p.b * k.heads + k.head) * a.N + p.n) * D, l);
    return r;
  };
  auto row_at = [&](const Place& p) {
    Raw r = {};
    if (norm && k.live)
      r = load_row(a.qkv + p.b * a.stride_b + p.n * a.stride_n + (size_t)k.column * D, l);
    return r;
  };
  Place here(a, id / a.packs);
  // (Without tokens, a.N may be zero and `here` is not used.)
  bool more = id / a.packs < a.step && here.token < a.tokens;
  Raw gx = {}, rx = {};
  int pos = 0;
  if (more) {
    gx = dz_at(here), rx = row_at(here);
    pos = position_of(a, here.token, here.n);
  }
  while (more) {
    Place next = here;
    more = a.tokens - here.token > a.step;
    next.advance(a);
    float g[16], cs[8], sn[8];
    if (k.kind < 2) load_turn(a, l, pos, cs, sn);
    Raw ahead_g = {}, ahead_x = {};
    if (more) {
      ahead_g = dz_at(next), ahead_x = row_at(next);
      pos = position_of(a, next.token, next.n);
    }
    if (k.kind < 2) {
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
    if (k.live)
      store_row(a.dqkv + here.b * a.dstride_b + here.n * a.dstride_n + (size_t)k.column * D, l, gx);
    here = next;
    gx = ahead_g, rx = ahead_x;
  }
  if constexpr (kNorm) {
    // Heads of a pack, then the block's warps of each kind.
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
    if ((threadIdx.x & 31) == 0) kinds[threadIdx.x >> 5] = k.kind;
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
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

// Deals packs and tokens to warps: blocks for `resident` per SM, fewer if
// there is less than one (token, pack) for each warp.
template <int D>
int deal(RopeArgs& a, int sm_count, int resident) {
  constexpr int kPack = 512 / D;
  a.packs = (a.H + kPack - 1) / kPack + 2 * ((a.Hkv + kPack - 1) / kPack);
  const long long all = (long long)a.tokens * a.packs;
  long long blocks = (all + kWarps - 1) / kWarps;
  if (blocks > (long long)resident * sm_count) blocks = (long long)resident * sm_count;
  if (blocks > kRopeMaxBlocks) blocks = kRopeMaxBlocks;
  // At least one warp for every pack of a token.
  const long long least = (a.packs + kWarps - 1) / kWarps;
  if (blocks < least) blocks = least;
  a.step = (int)(blocks * kWarps / (a.packs > 0 ? a.packs : 1));
  a.step_b = a.N > 0 ? a.step / a.N : 0;
  a.step_n = a.N > 0 ? a.step % a.N : 0;
  a.blocks = (int)blocks;
  return a.blocks;
}

template <int D, bool kInter, bool kNorm>
cudaError_t fwd(RopeArgs a, int sm_count, cudaStream_t stream) {
  const int blocks = deal<D>(a, sm_count, 4);
  rope_fwd_kernel<D, kInter, kNorm><<<blocks, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, bool kInter, bool kNorm>
cudaError_t bwd(RopeArgs a, int sm_count, cudaStream_t stream) {
  const int blocks = deal<D>(a, sm_count, 2);
  if (blocks > 0) rope_bwd_kernel<D, kInter, kNorm><<<blocks, kWarps * 32, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !kNorm) return e;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_dw_kernel<D>, a);
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
