// fa_cache4.cu -- the write side of the paged 4-bit cache: block tables and
// slot maps from request lengths, and the quantisation of new keys and
// values into their slots.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "fa_cache4.cuh"
#include "fa_launch.h"

namespace fa {
namespace {

// ------------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int pages_of(int tokens, int shift) {
  return (int)(((unsigned)tokens + (1u << shift) - 1) >> shift);
}

// Inclusive sums of one int per thread over the block; `total` the last.
__device__ __forceinline__ int block_scan(int v, int* sh, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += u;
  }
  __syncthreads();  // sh may still be read from the last call
  if (lane == 31) sh[warp] = v;
  __syncthreads();
  int s = sh[lane];
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, m);
    if (lane >= m) s += u;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, warp == 0 ? 0 : warp - 1);
  return v + (warp == 0 ? 0 : before);
}

// A request's state at the start of the call, with every value from memory
// brought into range first.
struct Req {
  int len, after, have, keep, grow;
};
__device__ __forceinline__ Req request(const PlanArgs& a, int r) {
  Req q = {0, 0, 0, 0, 0};
  if (r >= a.R) return q;
  const long long cap = (long long)a.M << a.shift;
  const int n = a.new_tokens[r];
  int len = a.lens[r];
  q.len = len < 0 ? 0 : (len > cap ? (int)cap : len);
  const long long less = (long long)q.len + (n < 0 ? n : 0);
  q.after = less < 0 ? 0 : (int)less;
  q.have = pages_of(q.len, a.shift);
  q.keep = pages_of(q.after, a.shift);
  q.grow = (n > 0 && n <= a.T && q.after + (long long)n <= cap) ? n : 0;
  return q;
}

// Copies between a request's table entries and the stack of free pages, one
// request per lane with the warp together on one request's pages:
// kPush: free_list[at + count - 1 - i] = table[first + i], else
//        table[first + i] = free_list[at - i].
template <bool kPush>
__device__ __forceinline__ void move_pages(const PlanArgs& a, int r, int first, int count, int at) {
  const int lane = threadIdx.x & 31;
  unsigned todo = __ballot_sync(0xffffffffu, count > 0);
  while (todo) {
    const int src = __ffs(todo) - 1;
    todo &= todo - 1;
    const int rr = __shfl_sync(0xffffffffu, r, src), f = __shfl_sync(0xffffffffu, first, src);
    const int c = __shfl_sync(0xffffffffu, count, src), p = __shfl_sync(0xffffffffu, at, src);
    int* row = a.block_table + (size_t)rr * a.M + f;
    for (int i = lane; i < c; i += 32) {
      const int s = kPush ? p + c - 1 - i : p - i;
      if (s < 0 || s >= a.P) continue;
      if (kPush) a.free_list[s] = row[i];
      else row[i] = a.free_list[s];
    }
  }
}

__device__ __forceinline__ void write_slot(const PlanArgs& a, int r, int t, int granted, int len) {
  int slot = -1, pos = 0;
  if (t < granted) {
    pos = len - granted + t;
    slot = a.block_table[(size_t)r * a.M + (pos >> a.shift)] * (1 << a.shift) +
           (pos & ((1 << a.shift) - 1));
  }
  const size_t at = (size_t)r * a.T + t;
  a.slots[at] = slot;
  a.positions[at] = pos;
}

// One block does the bookkeeping: sums over the requests, in order.  It is
// bound by latency (a few rounds of dependent loads), not by bytes.  Shrinks
// push their pages so that the last request's last page lies deepest; grows
// pop in request order: taking back exactly what a call granted restores
// the stack.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
  __shared__ int sh[32];
  int count = a.free_count[0];
  count = count < 0 ? 0 : (count > a.P ? a.P : count);
  const int chunks = (a.R + kPlanThreads - 1) / kPlanThreads;
  int total_back = 0;
  if (chunks > 1) {
    for (int c = 0; c < chunks; ++c) {
      const Req q = request(a, c * kPlanThreads + threadIdx.x);
      int t;
      block_scan(q.have - q.keep, sh, &t);
      total_back += t;
    }
  }
  int upto = 0;
  for (int c = 0; c < chunks; ++c) {
    const int r = c * kPlanThreads + threadIdx.x;
    const Req q = request(a, r);
    const int back = q.have - q.keep;
    int t;
    const int incl = block_scan(back, sh, &t);
    if (chunks == 1) total_back = t;
    move_pages<true>(a, r, q.keep, back, count + total_back - upto - incl);
    upto += t;
  }
  count = min(count + total_back, a.P);
  __syncthreads();  // the pushed pages are read below
  int need_before = 0, taken = 0;
  for (int c = 0; c < chunks; ++c) {
    const int r = c * kPlanThreads + threadIdx.x;
    const Req q = request(a, r);
    const int need = q.grow > 0 ? pages_of(q.after + q.grow, a.shift) - q.keep : 0;
    int t;
    const int incl = need_before + block_scan(need, sh, &t);
    need_before += t;
    const bool ok = q.grow > 0 && (need == 0 || incl <= count);
    const int granted = ok ? q.grow : 0;
    move_pages<false>(a, r, q.keep, ok ? need : 0, count - 1 - (incl - need));
    if (ok && need > 0 && incl > taken) taken = incl;
    if (r < a.R) {
      a.lens[r] = q.after + granted;
      a.granted[r] = granted;
    }
  }
  // Granted needs are a prefix of the requests that need pages: the largest
  // sum is what they took together.
  __syncthreads();
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, m));
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = taken;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) taken = max(taken, sh[w]);
    a.free_count[0] = count - taken;
  }
  if (a.fused) {
    for (int i = threadIdx.x; i < a.R * a.T; i += kPlanThreads) {
      const int r = i / a.T;
      write_slot(a, r, i - r * a.T, a.granted[r], a.lens[r]);
    }
  }
}

__global__ void __launch_bounds__(256) slots_kernel(PlanArgs a) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  for (int r = blockIdx.y; r < a.R; r += gridDim.y)
    if (t < a.T) write_slot(a, r, t, a.granted[r], a.lens[r]);
}

// ----------------------------------------------------------------- append
// One thread quantises 16 dims of one token and head of K or V.
//   scale = e4m3(amax / (6 g)), code = e2m1(x / (scale g)), nearest even.
// g is a power of two and the scale has four significant bits, x eight, so
// scale g is exact and no quotient x / (scale g) that is not itself half way
// between two codes lies within 2^-12 of such a point.  The quotient is
// therefore taken as a product with the reciprocal and one residual
// correction (Markstein's), whose error is far below that, and the codes
// are those of the exact quotient.
template <int D>
__global__ void __launch_bounds__(256) append_kernel(AppendArgs a) {
  constexpr int kBlk = D / 16;
  const unsigned row = blockIdx.x * (256 / kBlk) + threadIdx.x / kBlk;
  if (row >= (unsigned)a.rows) return;
  const int blk = threadIdx.x % kBlk;
  const unsigned bh = row / (unsigned)a.N, n = row - bh * a.N;
  const unsigned b = bh / (unsigned)a.Hkv, h = bh - b * a.Hkv;
  const int slot = __ldg(a.slots + (size_t)b * a.N + n);
  if (slot < 0 || slot >= (int)(a.pages << a.shift)) return;
  const bool is_v = blockIdx.y != 0;
  const size_t at = (size_t)row * D + blk * 16;
  const uint4* src = reinterpret_cast<const uint4*>((is_v ? a.v : a.k) + at);
  const uint4 u0 = src[0], u1 = src[1];  // plain loads: the values' output may be the input
  const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  // Largest magnitude by its bits: NaNs are above infinity.
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) big = __vmaxu2(big, w[i] & 0x7fff7fffu);
  big = max(big & 0xffffu, big >> 16);
  const float g = is_v ? a.v_scale : a.k_scale;
  const float amax = __uint_as_float(big << 16);
  uint32_t s8;
  if (big > 0x7f80u) s8 = 0x7f;  // a NaN: the block reads as NaN
  else s8 = __nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.0f * g), __NV_SATFINITE, __NV_E4M3);
  const __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s8, __NV_E4M3);
  const float s = __half2float(__half(hr)) * g;
  // Zero scale (all values round to nothing) and NaN: zero codes.
  const bool none = s8 == 0 || s8 == 0x7f;
  const float inv = none ? 0.f : __frcp_rn(s), lim = 4096.0f * g;
  uint32_t code[2] = {0, 0};
  uint32_t val[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float q[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // Beyond `lim` the scale is at its largest and the code saturates.
      const float x = __uint_as_float(e ? w[i] & 0xffff0000u : w[i] << 16);
      const float ax = fminf(fabsf(x), lim), y = ax * inv;
      q[e] = none ? 0.f : copysignf(fmaf(fmaf(-y, s, ax), inv, y), x);
    }
    uint32_t byte;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}"
        : "=r"(byte) : "f"(q[0]), "f"(q[1]));
    code[i >> 2] |= byte << (8 * (i & 3));
    uint32_t two;
    asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
        : "=r"(two) : "r"(byte));
    const __half2 hv = *reinterpret_cast<const __half2*>(&two);
    const float2 f = __half22float2(hv);
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * s, f.y * s);  // s NaN: NaN
    val[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  const int page = slot >> a.shift, in = slot & ((1 << a.shift) - 1), tok = in & 15;
  uint8_t* grp = a.cache + ((((size_t)page * a.Hkv + h) << (a.shift - 4)) + (in >> 4)) * group_bytes(D);
  if (!is_v) {
    *reinterpret_cast<uint2*>(grp + k_code_at(D, tok, blk * 8)) = make_uint2(code[0], code[1]);
    grp[k_scale_at(D, tok, blk)] = (uint8_t)s8;
  } else {
    if (D == 128) {
      *reinterpret_cast<uint2*>(grp + v_code_at(D, tok, blk)) = make_uint2(code[0], code[1]);
    } else {
      *reinterpret_cast<uint32_t*>(grp + v_code_at(D, tok, 2 * blk)) = code[0];
      *reinterpret_cast<uint32_t*>(grp + v_code_at(D, tok, 2 * blk + 1)) = code[1];
    }
    grp[v_scale_at(D, tok, blk)] = (uint8_t)s8;
  }
  __nv_bfloat16* out = is_v ? a.v_out : a.k_out;
  if (out) {
    uint4* dst = reinterpret_cast<uint4*>(out + at);
    dst[0] = make_uint4(val[0], val[1], val[2], val[3]);
    dst[1] = make_uint4(val[4], val[5], val[6], val[7]);
  }
}

}  // namespace

cudaError_t launch_cache4_plan(PlanArgs a, cudaStream_t stream) {
  // Up to 8192 slots (eight a thread) the block writes them itself; more
  // are spread over a second launch.
  a.fused = (long long)a.R * a.T <= 8 * kPlanThreads;
  plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.fused) return e;
  const int y = a.R < 32768 ? a.R : 32768;
  slots_kernel<<<dim3((a.T + 255) / 256, y), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache4_append(const AppendArgs& a, int d, cudaStream_t stream) {
  const int per = 256 / (d / 16);
  const dim3 grid((a.rows + per - 1) / per, 2);
  if (d == 128) append_kernel<128><<<grid, 256, 0, stream>>>(a);
  else append_kernel<64><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
