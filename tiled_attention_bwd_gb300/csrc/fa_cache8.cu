// fa_cache8.cu -- the paged 8-bit cache: new keys and values into their
// slots, and tokens back out of it.
//
// A group of 16 tokens of one head shares an exponent e (K and V apart):
//   code = E4M3(x / 2^e), nearest even, saturating;  value = code * 2^e.
// The smallest e that holds the largest finite magnitude, amax <= 448 2^e, is
// taken; in a group that holds earlier tokens, the larger of that and the
// present one, and the earlier codes are rounded to the grown scale.  Division
// by 2^e is exact, so every code is that of the exact quotient.
//
// Both directions are bound by memory: rows of bf16 and pieces of a group go
// straight between registers and memory, 16 bytes a lane and whole sectors a
// warp, in the order of the lanes that the attention reads them in.  Measured
// (d = 128, 8 heads): append of 8 x 4000 tokens with the values that are held
// 39.9 us, 6.2 TB/s, without them 25.4 us, 5.8 TB/s; read of 12 x 6000 tokens 53.5
// us, 6.5 TB/s; one token of 128 requests 3.2 us, the latency of loads that depend
// on one another: slots, then exponents and rows, then codes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fa_cache8.cuh"
#include "fa_serve.h"

namespace fa {
namespace {

constexpr int kWarps = 8;  // per block

// Codes, at the bytes 0 and 1, of two values (times a factor).
__device__ __forceinline__ uint32_t to_e4m3(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t to_e4m3(uint32_t f16_pair) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f16x2 t, %1;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(r) : "r"(f16_pair));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Eight bf16 values over 2^e as codes (w2: words 0 and 1).
__device__ __forceinline__ uint2 quantise(const uint4& u, float inv) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = to_e4m3(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv);
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// Two codes' values (an f16 pair times 2^e) as bf16.
__device__ __forceinline__ uint32_t value2(uint32_t f16_pair, float s) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f16_pair));
  const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * s, f.y * s);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Eight codes' values as bf16.
__device__ __forceinline__ uint4 values8(const uint2& c, float s) {
  uint32_t a, b, e, f;
  e4m3_to_f16(c.x, a, b);
  e4m3_to_f16(c.y, e, f);
  return make_uint4(value2(a, s), value2(b, s), value2(e, s), value2(f, s));
}
// Four codes rounded to a scale that is larger by 1 / factor (an f16 pair).  A
// code has four significant bits: the product is exact, or so small that its
// code is zero either way.
__device__ __forceinline__ uint32_t rescale(uint32_t w, uint32_t factor) {
  uint32_t lo, hi;
  e4m3_to_f16(w, lo, hi);
  return to_e4m3(mul2(lo, factor)) | to_e4m3(mul2(hi, factor)) << 16;
}
__device__ __forceinline__ uint4 rescale(const uint4& u, uint32_t factor) {
  return make_uint4(rescale(u.x, factor), rescale(u.y, factor), rescale(u.z, factor),
                    rescale(u.w, factor));
}
// 2^-by as an f16 pair (codes shifted further than 24 vanish anyway).
__device__ __forceinline__ uint32_t factor_of(int by) {
  by = min(by, 24);
  const uint32_t h = by < 15 ? (uint32_t)(15 - by) << 10 : 1u << (24 - by);
  return h | h << 16;
}

// Largest magnitude of a warp's bf16 pairs by its bits, of the finite ones where
// others are among them.
template <int N>
__device__ __forceinline__ uint32_t largest(const uint4 (&x)[N]) {
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    for (uint32_t w : {x[i].x, x[i].y, x[i].z, x[i].w}) big = __vmaxu2(big, w & 0x7fff7fffu);
  big = __reduce_max_sync(0xffffffffu, max(big & 0xffffu, big >> 16));
  if (big >= 0x7f80u) {
    big = 0;
    for (int i = 0; i < N; ++i)
      for (uint32_t w : {x[i].x, x[i].y, x[i].z, x[i].w}) {
        const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
        if (lo < 0x7f80u) big = max(big, lo);
        if (hi < 0x7f80u) big = max(big, hi);
      }
    big = __reduce_max_sync(0xffffffffu, big);
  }
  return big;
}
// Smallest exponent e with amax <= 448 2^e, 448 being 1.75 2^8; amax by its
// bf16 bits.
__device__ __forceinline__ int exponent_for(uint32_t amax) {
  const int e = (int)(amax >> 7) - 127 - 8 + ((amax & 0x7f) > 0x60 ? 1 : 0);
  return min(max(e, -kExp8), kExp8);
}

// A group's exponent: `big` is the largest magnitude among the new tokens, `old` the exponent's byte, `fresh` whether the group begins.
struct Exponent {
  int e;
  bool grown;     // the other tokens' codes are of a smaller one,
  uint32_t down;  // by this factor (an f16 pair)
  float unit, inv;  // 2^e, 2^-e
  __device__ __forceinline__ Exponent(uint32_t big, uint32_t old, bool fresh) {
    e = exponent_for(big);
    const int was = exp8(old);
    if (!fresh) e = max(e, was);
    grown = !fresh && e > was;
    down = factor_of(e - was);
    unit = pow2(e), inv = pow2(-e);
  }
};

// ----------------------------------------------------------------- append
// Which tokens of the call come to the places of a group.
struct Places {
  signed char at[16];  // relative to the warp's first token; -1: none
};

// One group's keys: a lane has the tokens g and g + 8.
template <int D>
__device__ __forceinline__ void append_keys(const Append8Args& a, const Places& p, uint8_t* grp,
                                            size_t row0, bool fresh, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t head = grp[32 * D];
  uint4 x[2 * (D / 32)];  // [h][j]
  int n[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    n[h] = p.at[8 * h + g];
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
      x[h * (D / 32) + j] = n[h] >= 0 ? *reinterpret_cast<const uint4*>(a.k + (row0 + n[h]) * D + 32 * j + 8 * t)
                          : make_uint4(0, 0, 0, 0);
  }
  const Exponent e(largest(x), head, fresh);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint4* at = reinterpret_cast<uint4*>(grp + k8_piece(D, h, c, lane));
      if (n[h] >= 0) {
        const uint4* row = x + h * (D / 32) + 2 * c;
        const uint2 u = quantise(row[0], e.inv), v = quantise(row[1], e.inv);
        *at = make_uint4(u.x, u.y, v.x, v.y);
        if (a.k_out) {
          __nv_bfloat16* out = a.k_out + (row0 + n[h]) * D + 64 * c + 8 * t;
          *reinterpret_cast<uint4*>(out) = values8(u, e.unit);
          *reinterpret_cast<uint4*>(out + 32) = values8(v, e.unit);
        }
      } else if (e.grown) {
        *at = rescale(*at, e.down);
      }
    }
  __syncwarp();  // every lane has the old exponent
  if (lane == 0) grp[32 * D] = (uint8_t)e.e;
}

// Its values: a lane has the tokens 2t, 2t + 1, 2t + 8 and 2t + 9.
template <int D>
__device__ __forceinline__ void append_values(const Append8Args& a, const Places& p, uint8_t* grp,
                                              size_t row0, bool fresh, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t head = grp[32 * D + 1];
  uint4 x[4 * (D / 64)];  // [h][s][j]
  int n[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      n[h][s] = p.at[8 * h + 2 * t + s];
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
        x[(2 * h + s) * (D / 64) + j] = n[h][s] >= 0 ? *reinterpret_cast<const uint4*>(a.v + (row0 + n[h][s]) * D + 64 * j + 8 * g)
                                  : make_uint4(0, 0, 0, 0);
    }
  const Exponent e(largest(x), head, fresh);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool has0 = n[h][0] >= 0, has1 = n[h][1] >= 0;
    if (!has0 && !has1 && !e.grown) continue;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      uint4* at = reinterpret_cast<uint4*>(grp + v8_piece(D, j, h, lane));
      const uint2 u = quantise(x[2 * h * (D / 64) + j], e.inv);
      const uint2 v = quantise(x[(2 * h + 1) * (D / 64) + j], e.inv);
      // The two tokens' codes side by side.
      uint4 c = make_uint4(__byte_perm(u.x, v.x, 0x5140), __byte_perm(u.x, v.x, 0x7362),
                           __byte_perm(u.y, v.y, 0x5140), __byte_perm(u.y, v.y, 0x7362));
      if (!(has0 && has1)) {
        uint4 old = *at;
        if (e.grown) old = rescale(old, e.down);
        const uint32_t m = (has0 ? 0x00ff00ffu : 0) | (has1 ? 0xff00ff00u : 0);
        c = make_uint4((c.x & m) | (old.x & ~m), (c.y & m) | (old.y & ~m), (c.z & m) | (old.z & ~m),
                       (c.w & m) | (old.w & ~m));
      }
      *at = c;
      if (a.v_out) {
        __nv_bfloat16* out = a.v_out + row0 * D + 64 * j + 8 * g;
        if (has0) *reinterpret_cast<uint4*>(out + (ptrdiff_t)n[h][0] * D) = values8(u, e.unit);
        if (has1) *reinterpret_cast<uint4*>(out + (ptrdiff_t)n[h][1] * D) = values8(v, e.unit);
      }
    }
  }
  __syncwarp();  // every lane has the old exponent
  if (lane == 0) grp[32 * D + 1] = (uint8_t)e.e;
}

// A warp takes 16 neighbouring tokens of one batch entry and head, their keys
// or their values (both: 51 us at 8 x 4000 tokens, at half the occupancy, so 43;
// with maxima by packed comparisons 40), and, one after the other, the groups whose first token (in
// the call's order) is among them, with all their tokens up to 15 places on: a
// group is written by one warp, which knows all that the call brings to it.
template <int D>
__global__ void __launch_bounds__(kWarps * 32, 4) append8_kernel(Append8Args a) {
  __shared__ Places places[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_for_stream();
  const unsigned id = blockIdx.x * kWarps + warp;
  if (id >= (unsigned)a.warps) return;
  const unsigned bh = a.by_chunks.div(id);
  const int n0 = (int)(id - bh * a.chunks) * 16;
  const unsigned b = a.by_Hkv.div(bh), hk = bh - b * a.Hkv;
  // Slots of the tokens n0 - 16 + lane and n0 + 16 + lane.
  const int* slots = a.slots + (size_t)b * a.N;
  auto slot_of = [&](int n) {
    if (n < 0 || n >= a.N) return -1;
    const int s = slots[n];
    return s >= 0 && s < a.slots_end ? s : -1;
  };
  const int sa = slot_of(n0 - 16 + lane);
  const int sb = lane < 15 ? slot_of(n0 + 16 + lane) : -1;
  const uint32_t same = __match_any_sync(0xffffffffu, sa >> 4);
  const uint32_t earlier = same & ((1u << lane) - 1) & ~((1u << (lane - 15 > 0 ? lane - 15 : 0)) - 1);
  uint32_t leaders = __ballot_sync(0xffffffffu, lane >= 16 && sa >= 0 && earlier == 0);
  for (; leaders; leaders &= leaders - 1) {
    const int first = __ffs(leaders) - 1, id16 = __shfl_sync(0xffffffffu, sa, first) >> 4;
    Places& p = places[warp];
    if (lane < 16) p.at[lane] = -1;
    __syncwarp();
    if (lane >= first && sa >= 0 && sa >> 4 == id16) p.at[sa & 15] = lane - 16;
    __syncwarp();
    if (lane <= first - 17 && sb >= 0 && sb >> 4 == id16) p.at[sb & 15] = 16 + lane;
    __syncwarp();
    // The group's first token begins it; what it held before is not there.
    const bool fresh = p.at[0] >= 0;
    const int gpp = a.shift - 4, page = id16 >> gpp;
    uint8_t* grp = a.cache + ((((size_t)page * a.Hkv + hk) << gpp) + (id16 & ((1 << gpp) - 1))) *
                                 group8_bytes(D);
    const size_t row0 = (size_t)bh * a.N + n0;
    if (blockIdx.y == 0) append_keys<D>(a, p, grp, row0, fresh, lane);
    else append_values<D>(a, p, grp, row0, fresh, lane);
    __syncwarp();  // the places are read
  }
}

// ------------------------------------------------------------------- read
// A warp takes the tokens that an entry wants of one group and head.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) read8_kernel(Read8Args a) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  wait_for_stream();
  const unsigned id = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= (unsigned)a.warps) return;
  const unsigned bh = a.by_chunks.div(id), chunk = id - bh * a.chunks;
  const unsigned b = a.by_Hkv.div(bh), hk = bh - b * a.Hkv;
  // Tokens [lo, hi) of the request, token lo + n in row n.
  const int cap = a.M << a.shift;
  const int len = min(max(a.seq_lens[b], 0), cap);
  const int lo = a.starts ? min(max(a.starts[b], 0), cap) : 0;
  const int hi = (int)min((long long)len, (long long)lo + a.N);
  const long long at = ((lo >> 4) + (long long)chunk) * kGroup;
  if (at >= hi) return;
  const int tok = (int)at;  // the group's first
  const int page = a.block_table[(size_t)b * a.M + (tok >> a.shift)];
  if (page < 0 || page >= a.pages) return;
  const int gpp = a.shift - 4;
  const uint8_t* grp = a.cache + ((((size_t)page * a.Hkv + hk) << gpp) + ((tok >> 4) & ((1 << gpp) - 1))) *
                                     group8_bytes(D);
  uint4 k[2][D / 64], v[2][D / 64];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      k[h][c] = *reinterpret_cast<const uint4*>(grp + k8_piece(D, h, c, lane));
      v[h][c] = *reinterpret_cast<const uint4*>(grp + v8_piece(D, c, h, lane));
    }
  const uint32_t head = *reinterpret_cast<const uint16_t*>(grp + 32 * D);
  const float ks = pow2(exp8(head & 0xff)), vs = pow2(exp8(head >> 8));
  const long long row0 = (long long)bh * a.N + tok - lo;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int kt = tok + 8 * h + g;
    if (kt >= lo && kt < hi) {
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        __nv_bfloat16* out = a.k_out + (row0 + 8 * h + g) * D + 64 * c + 8 * t;
        *reinterpret_cast<uint4*>(out) = values8(make_uint2(k[h][c].x, k[h][c].y), ks);
        *reinterpret_cast<uint4*>(out + 32) = values8(make_uint2(k[h][c].z, k[h][c].w), ks);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int vt = tok + 8 * h + 2 * t + e;
      if (vt < lo || vt >= hi) continue;
      const uint32_t sel = e ? 0x7531 : 0x6420;  // one token's codes of a pair
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint4 u = v[h][c];
        *reinterpret_cast<uint4*>(a.v_out + (row0 + 8 * h + 2 * t + e) * D + 64 * c + 8 * g) =
            values8(make_uint2(__byte_perm(u.x, u.y, sel), __byte_perm(u.z, u.w, sel)), vs);
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache8_append(const Append8Args& a, int d, cudaStream_t stream) {
  return launch_overlapped(d == 128 ? append8_kernel<128> : append8_kernel<64>,
                           dim3((a.warps + kWarps - 1) / kWarps, 2), dim3(kWarps * 32), 0, stream, a);
}
cudaError_t launch_cache8_read(const Read8Args& a, int d, cudaStream_t stream) {
  return launch_overlapped(d == 128 ? read8_kernel<128> : read8_kernel<64>,
                           dim3((a.warps + kWarps - 1) / kWarps), dim3(kWarps * 32), 0, stream, a);
}

}  // namespace fa
