// fa_cache4.cu -- the write side of the paged 4-bit cache: block tables and
// slot maps from request lengths, and the quantisation of new keys and
// values into their slots.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "fa_cache4.cuh"
#include "fa_serve.h"

namespace fa {
namespace {

// ------------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int pages_of(int tokens, int shift) {
  return (int)(((unsigned)tokens + (1u << shift) - 1) >> shift);
}

// Two counts of pages, summed together.
struct Pages {
  int back, need;
};
// Inclusive sums over the block; `total` the last.
__device__ __forceinline__ Pages block_scan(Pages v, Pages* sh, Pages* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int b = __shfl_up_sync(0xffffffffu, v.back, m), n = __shfl_up_sync(0xffffffffu, v.need, m);
    if (lane >= m) v.back += b, v.need += n;
  }
  __syncthreads();  // sh may still be read from the last call
  if (lane == 31) sh[warp] = v;
  __syncthreads();
  Pages s = lane < warps ? sh[lane] : Pages{0, 0};
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int b = __shfl_up_sync(0xffffffffu, s.back, m), n = __shfl_up_sync(0xffffffffu, s.need, m);
    if (lane >= m) s.back += b, s.need += n;
  }
  total->back = __shfl_sync(0xffffffffu, s.back, 31);
  total->need = __shfl_sync(0xffffffffu, s.need, 31);
  const int b = __shfl_sync(0xffffffffu, s.back, max(warp - 1, 0));
  const int n = __shfl_sync(0xffffffffu, s.need, max(warp - 1, 0));
  if (warp > 0) v.back += b, v.need += n;
  return v;
}

// A request's state at the start of the call, with every value from memory
// brought into range first.
struct Req {
  int after, keep, grow;  // tokens and pages left by a shrink; tokens wanted
  Pages pages;            // given back, wanted
};
__device__ __forceinline__ Req request(const PlanArgs& a, int r) {
  Req q = {0, 0, 0, {0, 0}};
  if (r >= a.R) return q;
  const long long cap = (long long)a.M << a.shift;
  const int n = a.new_tokens[r];
  int len = a.lens[r];
  len = len < 0 ? 0 : (len > cap ? (int)cap : len);
  const long long less = (long long)len + (n < 0 ? n : 0);
  q.after = less < 0 ? 0 : (int)less;
  q.keep = pages_of(q.after, a.shift);
  q.grow = (n > 0 && n <= a.T && q.after + (long long)n <= cap) ? n : 0;
  q.pages.back = pages_of(len, a.shift) - q.keep;
  q.pages.need = q.grow > 0 ? pages_of(q.after + q.grow, a.shift) - q.keep : 0;
  return q;
}

// Per-request results of a chunk, for the work that its threads share.
struct Chunk {
  int upto[kPlanThreads];   // pages wanted (or given back) up to and including it
  int after[kPlanThreads];  // tokens before the new ones
  int keep[kPlanThreads];   // pages before the new ones
  int grow[kPlanThreads];   // tokens granted
  int at[kPlanThreads];     // place in the stack of its first page
};

// The request of the chunk's i-th page: the first with upto > i.
__device__ __forceinline__ int owner_of(const Chunk& c, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c.upto[mid] > i) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// All blocks of the grid, which is one cluster.
__device__ __forceinline__ void grid_sync() {
  if (gridDim.x == 1) __syncthreads();
  else
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" :::
                     "memory");
}

// One cluster does a call.  Every block goes through the requests' sums, a
// block's width of requests at a time; the copies of page ids and the slots
// are dealt over all the cluster's threads, whichever request they belong to.
// Shrinks push their pages so that the last request's last page lies deepest;
// grows pop in request order: taking back exactly what a call granted
// restores the stack.  Bound by latency: a few rounds of dependent loads and
// barriers.  (One block, with a request's pages moved by its own warp, took
// 89 us for 48 prompts of 4096 tokens, 12288 pages; a cluster of 16 takes 7.)
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
  __shared__ Pages sh[32];
  __shared__ int sh_taken[32];
  __shared__ Chunk ch;
  const int tid = threadIdx.x, width = blockDim.x, rank = blockIdx.x;
  const int first = rank * width + tid, step = gridDim.x * width;
  wait_for_stream();
  int count = a.free_count[0];
  count = count < 0 ? 0 : (count > a.P ? a.P : count);
  const int chunks = (a.R + width - 1) / width;

  // ---- pages given back
  int total_back = 0;
  if (chunks > 1) {
    for (int c = 0; c < chunks; ++c) {
      Pages t;
      block_scan(request(a, c * width + tid).pages, sh, &t);
      total_back += t.back;
    }
  }
  int before = 0;
  Req q;
  Pages t, incl;
  for (int c = 0; c < chunks; ++c) {
    const int r0 = c * width, n = min(width, a.R - r0);
    q = request(a, r0 + tid);
    incl = block_scan(q.pages, sh, &t);
    if (chunks == 1) total_back = t.back;
    if (t.back > 0) {
      ch.upto[tid] = incl.back;
      ch.keep[tid] = q.keep;
      __syncthreads();
      for (int i = first; i < t.back; i += step) {
        const int o = owner_of(ch, n, i);
        // The i-th page from the front is the last but i from the back.
        const int page = ch.keep[o] + i - (o > 0 ? ch.upto[o - 1] : 0);
        const int s = count + total_back - before - 1 - i;
        if (s < a.P) a.free_list[s] = a.block_table[(size_t)(r0 + o) * a.M + page];
      }
      before += t.back;
      __syncthreads();
    }
  }
  count = min(count + total_back, a.P);
  grid_sync();  // the pushed pages are read below

  // ---- pages taken, and the new tokens' slots
  int wanted = 0, taken = 0;
  for (int c = 0; c < chunks; ++c) {
    const int r0 = c * width, n = min(width, a.R - r0);
    if (chunks > 1) {
      q = request(a, r0 + tid);
      incl = block_scan(q.pages, sh, &t);
    }
    const int need = q.pages.need;
    const bool ok = q.grow > 0 && (need == 0 || wanted + incl.need <= count);
    // Granted needs are a prefix of the requests that need pages.
    if (ok && need > 0) taken = wanted + incl.need;
    ch.upto[tid] = incl.need;
    ch.after[tid] = q.after;
    ch.keep[tid] = q.keep;
    ch.grow[tid] = ok ? q.grow : 0;
    ch.at[tid] = count - 1 - (wanted + incl.need - need);
    if (rank == 0 && tid < n) a.granted[r0 + tid] = ch.grow[tid];
    wanted += t.need;
    __syncthreads();
    for (int i = first; i < t.need; i += step) {
      const int o = owner_of(ch, n, i), j = i - (o > 0 ? ch.upto[o - 1] : 0);
      if (ch.grow[o] > 0)
        a.block_table[(size_t)(r0 + o) * a.M + ch.keep[o] + j] = a.free_list[ch.at[o] - j];
    }
    // Slots, for rows of four and more four neighbours at a time, which may
    // lie across the end of a row.
    const unsigned all = (unsigned)n * a.T, w = a.T >= 4 ? 4 : 1;
    // Page p of request o; pages taken now come from the stack, as the table
    // may not have them yet.
    auto page_of = [&](int o, int p) {
      const int j = p - ch.keep[o];
      return j >= 0 ? a.free_list[ch.at[o] - j] : a.block_table[(size_t)(r0 + o) * a.M + p];
    };
    auto slot_of = [&](int page, int pos) {
      return (unsigned)page < (unsigned)a.P ? (page << a.shift) + (pos & ((1 << a.shift) - 1)) : -1;
    };
    for (unsigned i = w * first; i < all; i += w * step) {
      int o = a.by_T.div(i), tok = i - o * a.T;
      int slot[4] = {-1, -1, -1, -1}, pos[4] = {0, 0, 0, 0};
      if (tok <= a.T - (int)w) {  // of one request, on two pages at most
        const int left = min(ch.grow[o] - tok, (int)w), at = ch.after[o] + tok;
        if (left > 0) {
          const int p0 = at >> a.shift, p1 = (at + left - 1) >> a.shift;
          const int page0 = page_of(o, p0), page1 = p1 == p0 ? page0 : page_of(o, p1);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < left) {
              pos[k] = at + k;
              slot[k] = slot_of(pos[k] >> a.shift == p0 ? page0 : page1, pos[k]);
            }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (o < n && tok < ch.grow[o]) {
            pos[k] = ch.after[o] + tok;
            slot[k] = slot_of(page_of(o, pos[k] >> a.shift), pos[k]);
          }
          if (++tok == a.T) tok = 0, ++o;
        }
      }
      const size_t at = (size_t)r0 * a.T + i;
      if (w == 4 && a.wide && i + 4 <= all) {
        *reinterpret_cast<int4*>(a.slots + at) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        *reinterpret_cast<int4*>(a.positions + at) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < w && i + k < all) a.slots[at + k] = slot[k], a.positions[at + k] = pos[k];
      }
    }
    __syncthreads();
  }

  // ---- lengths and the count, once every block has read them
  if (gridDim.x > 1) grid_sync();
  if (rank != 0) return;
  for (int r = tid; r < a.R; r += width) a.lens[r] = request(a, r).after + a.granted[r];
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, m));
  if ((tid & 31) == 0) sh_taken[tid >> 5] = taken;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < width / 32; ++w) taken = max(taken, sh_taken[w]);
    a.free_count[0] = count - taken;
  }
}

// ----------------------------------------------------------------- append
// One thread quantises 16 dims of one token and head of K or V.
//   scale = e4m3(amax / (6 g)), code = e2m1(x / (scale g)), nearest even.
// g is a power of two, scale g has four significant bits and x eight, so
// scale g is exact and a quotient x / (scale g) is either exactly half way
// between two codes or at least 2^-8 of itself away from there.  It is taken
// as the product with the rounded reciprocal (within 2^-23), then rounded to
// f16 (within 2^-11, which returns the half-way points exactly), then to the
// code: the codes are those of the exact quotient.  (49 us at 8 x 4000 tokens
// of 8 heads of 128 with a residual correction per quotient instead of the
// two roundings; 36 us so in a stream of calls: 6.3 TB/s, and seven tenths of
// the issue slots.)
template <int D>
__global__ void __launch_bounds__(256) append_kernel(AppendArgs a) {
  constexpr int kBlk = D / 16;
  const unsigned row = blockIdx.x * (256 / kBlk) + threadIdx.x / kBlk;
  if (row >= (unsigned)a.rows) return;
  const int blk = threadIdx.x % kBlk;
  wait_for_stream();
  const unsigned bh = a.by_N.div(row), n = row - bh * a.N;
  const unsigned b = a.by_Hkv.div(bh), h = bh - b * a.Hkv;
  const int slot = a.slots[(size_t)b * a.N + n];
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
  const float inv = __frcp_rn(s);
  uint32_t code[2] = {0, 0};
  uint32_t val[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t q, byte, two;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;"
        : "=r"(q) : "f"(__uint_as_float(w[i] << 16) * inv), "f"(__uint_as_float(w[i] & 0xffff0000u) * inv));
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f16x2 t, %1;\n\tcvt.u32.u8 %0, t;\n\t}"
        : "=r"(byte) : "r"(q));
    // Zero scale (all values round to nothing) and NaN: zero codes.
    if (s8 == 0 || s8 == 0x7f) byte = 0;
    code[i >> 2] |= byte << (8 * (i & 3));
    asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
        : "=r"(two) : "r"(byte));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
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

// Blocks of the plan's large cluster on the current device: 16 where such a
// cluster fits one of its GPCs (found out once per device), else the 8 that
// always do.
static unsigned plan_cluster() {
  static std::atomic<unsigned> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 8;
  std::atomic<unsigned>& blocks = known[dev & 63];
  if (blocks.load() == 0) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 16;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int fit = 0;
    const bool ok =
        cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
            cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&fit, plan_kernel, &cfg) == cudaSuccess && fit > 0;
    if (!ok) (void)cudaGetLastError();
    blocks.store(ok ? 16 : 8);
  }
  return blocks.load();
}

cudaError_t launch_cache4_plan(PlanArgs a, cudaStream_t stream) {
  a.wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) &
            15) == 0;
  // One block for up to 8192 slots, as wide as there are requests or slots
  // (barriers of few warps are shorter), else a cluster: the slots are bound
  // by how many SMs write them (48 prompts of 4096: 9.5 us by 8, 7.3 by 16).
  const long long work = (long long)a.R * a.T, width = work > a.R ? work : a.R;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = work <= 8 * kPlanThreads ? 1 : plan_cluster();
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(attr[0].val.clusterDim.x);
  cfg.blockDim = dim3(width <= 128 ? 128 : (width <= 256 ? 256 : (width <= 512 ? 512 : kPlanThreads)));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, plan_kernel, a);
}

cudaError_t launch_cache4_append(const AppendArgs& a, int d, cudaStream_t stream) {
  const int per = 256 / (d / 16);
  const dim3 grid((a.rows + per - 1) / per, 2);
  return launch_overlapped(d == 128 ? append_kernel<128> : append_kernel<64>, grid, dim3(256), 0,
                           stream, a);
}

}  // namespace fa
