// fa_cache8_attn.cu -- the attention over the paged 8-bit cache
// (fa_cache_attn.cuh has the work's division and the main loop):
// k_j, v_j = E4M3 code * 2^e, e one exponent per group of 16 tokens, for K and V.
//
// Codes are f16 values: K and V enter the products exactly, without their
// factors.  K's factor multiplies the group's scores.  V's would leave f16's
// range in P; so a row's maximum is taken of s + e_v, in powers of two, the
// weights are 2^(s + e_v - m), which is what the product with the codes needs,
// and the sum l adds them over 2^e_v.  A weight's rounding is then relative to
// the largest possible contribution to the row's output.
//
// What bounds it is memory: a group of one head is 4112 bytes (d = 128) for
// about 150 warp instructions, 64 of them conversions; the cache's layout gives
// them whole registers in the fragments' order, without a permutation.
// Measured (d = 128, 8 query heads to a key/value head): 64 requests of 100 to
// 8192 tokens x 8 heads 89 us, 6.1 TB/s of codes; 3 requests of 100000 to 131072
// tokens x 8 heads 109 us, 6.5 TB/s; issue slots 30% busy, DRAM 77 and 83% of
// its nominal rate.  With more rows the warps' instructions and registers bound it:
// 32 rows take 76 us where 8 take 51, over the same 40 us of bytes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fa_cache8.cuh"
#include "fa_cache_attn.cuh"

namespace fa {
namespace {

struct Cache8 {
  static constexpr uint32_t kWhere = 0x521;
  static constexpr int kItemCost = 1;  // (three: 111.4 us at 3 x 131072 tokens, one: 108.8)
  static constexpr __host__ __device__ int group_bytes(int d) { return group8_bytes(d); }
  static constexpr __host__ __device__ int blocks_per_sm(int d, int nt) {
    return d == 64 && nt <= 2 ? 3 : 2;
  }
  // Lane t takes dims 32 i + 8 t + 0 .. 7 of K; lane g dims 64 j + 8 g + 0 .. 7
  // of V, two of them in a tile.
  static __device__ __forceinline__ int q_piece(int, int t, int i) { return 64 * i + 16 * t; }
  static __device__ __forceinline__ int o_dim(int, int g, int dt) {
    return 64 * (dt / 4) + 8 * g + 2 * (dt % 4);
  }
  struct Scales {
    float k, inv_v, log_v;
    // (Not zero: a masked score, minus infinity, is multiplied with it.)
    __device__ __forceinline__ float score(float x) const { return fmaxf(x * k, 1.2e-38f); }
    __device__ __forceinline__ float less(float m) const { return m - log_v; }
    __device__ __forceinline__ float more(float m) const { return m + log_v; }
    __device__ __forceinline__ void sum(float& l, float p) const { l = fmaf(p, inv_v, l); }
  };
  static __device__ __forceinline__ Scales scales(const uint8_t* grp, int d) {
    const uint32_t two = *reinterpret_cast<const uint16_t*>(grp + 32 * d);
    const int ke = exp8(two & 0xff), ve = exp8(two >> 8);
    return {pow2(ke), pow2(-ve), (float)ve};
  }

  // One group's scores, S^T = K Q^T: tokens g and g + 8, rows 2t and 2t + 1.
  template <int D, int NT, typename R>
  static __device__ __forceinline__ void scores(const uint8_t* grp, int g, int t, const R& r,
                                                float (&s)[NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint32_t w[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 u = *reinterpret_cast<const uint4*>(grp + k8_piece(D, h, c, 4 * g + t));
        w[h][0] = u.x, w[h][1] = u.y, w[h][2] = u.z, w[h][3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // 32 dims
        uint32_t f[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          e4m3_to_f16(w[0][2 * i + x], f[x][0], f[x][2]);
          e4m3_to_f16(w[1][2 * i + x], f[x][1], f[x][3]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int j = 2 * c + i;
          uint4 q;
          if constexpr (Shape<Cache8, D, NT>::kQInRegs)
            q = make_uint4(r.qf[nt][4 * j], r.qf[nt][4 * j + 1], r.qf[nt][4 * j + 2], r.qf[nt][4 * j + 3]);
          else
            q = r.qs[(nt * (D / 32) + j) * 32];
          mma(s[nt], f[0], q.x, q.y);
          mma(s[nt], f[1], q.z, q.w);
        }
      }
    }
  }

  // One group's part of O^T += V^T P^T.
  template <int D, int NT, bool kPlain>
  static __device__ __forceinline__ void values(const uint8_t* grp, int g, int t,
                                                const uint32_t (&pb)[NT][2], float (&o)[D / 16][NT][4],
                                                int there, int tok, const Bounds& bd) {
    uint32_t nans = 0;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      uint32_t w[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 u = *reinterpret_cast<const uint4*>(grp + v8_piece(D, j, h, 4 * g + t));
        w[h][0] = u.x, w[h][1] = u.y, w[h][2] = u.z, w[h][3] = u.w;
        if constexpr (!kPlain) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (!there) w[h][x] = 0;
            const uint32_t nan = __vcmpeq4(w[h][x] & 0x7f7f7f7fu, 0x7f7f7f7fu);
            nans |= nan;
            w[h][x] &= ~nan;
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t f[4];
        e4m3_to_f16(w[0][x], f[0], f[1]);
        e4m3_to_f16(w[1][x], f[2], f[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma(o[4 * j + x][nt], f, pb[nt][0], pb[nt][1]);
      }
    }
    // A NaN goes to the rows that see its token, and not, by a weight of zero,
    // to the others (a token that no row sees may hold anything).
    if (!kPlain && __any_sync(0xffffffffu, nans != 0)) {
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t at = 0;  // by token: the value of this dim is NaN
#pragma unroll 1
          for (int x = 0; x < kGroup; ++x)
            if ((grp[v8_at(D, x, o_dim(D, g, dt) + c)] & 0x7f) == 0x7f) at |= 1u << x;
          if (!there) at = 0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (at & bd.seen(8 * nt + 2 * t + i, tok)) o[dt][nt][i + 2 * c] = __uint_as_float(0x7fffffffu);
        }
    }
  }
};

template <int D, int NT, bool kHook>
__global__ void __launch_bounds__(kWarps * 32, Cache8::blocks_per_sm(D, NT))
    cache8_attn_kernel(CacheAttnArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Block<Cache8, D, NT> block;
  block.begin();
  wait_for_stream();
  cache_attn<Cache8, D, NT, kHook>(a, block, smem);
}

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32) cache8_join_kernel(CacheAttnArgs a) {
  wait_for_stream();
  cache_join<Cache8, D, NT>(a);
}

template <int D, int NT, bool kHook = false>
cudaError_t run(const CacheAttnArgs& a, int sm_count, cudaStream_t stream) {
  // The hook has its own instantiation, for d = 128 and items of 8 rows only.
  if constexpr (D == 128 && NT == 1 && !kHook) {
    if (a.hook) return run<D, NT, true>(a, sm_count, stream);
  }
  static std::atomic<unsigned long long> done{0};
  return run_cache_attn<Cache8, D, NT>(cache8_attn_kernel<D, NT, kHook>, cache8_join_kernel<D, NT>,
                                       a, sm_count, done, stream);
}

}  // namespace

// Rows of an item: what makes the least of the passes over the keys, each of a
// cost by its width (us measured at 16 requests of 8192 tokens x 8 heads; 40
// rows at once at d = 128 spill: not built).
int cache8_attn_rows(int rows, int d) {
  const int cost[2][5] = {{31, 36, 43, 50, 59}, {51, 54, 59, 76, 0}};
  int best = 8;
  long long least = 0;
  for (int nt = 1; nt <= (d == 128 ? 4 : 5); ++nt) {
    const long long c = (rows + 8LL * nt - 1) / (8 * nt) * cost[d == 128][nt - 1];
    if (nt == 1 || c < least) least = c, best = 8 * nt;
  }
  return best;
}

// Measured against the kernel for many rows (us: this one / the other without
// lengths of the new tokens / with them, where an empty launch of this one stands
// before it; 16 requests of 4096 to 8192 tokens x 8 heads, 64 of 500 to 1000 x 2,
// 2 of 30000 to 60000 x 1):
//   d = 128, 48 rows: 82/74/81, 28/25/30, 30/34/40; 64: 108/75/83, 35/27/32, 36/35/40
//   d = 64,  64 rows: 69/65/71, 27/23/28, 28/25/30; 80: 82/66/73, 33/24/29, 32/25/30
int cache8_narrow_rows(int d) { return d == 128 ? 48 : 64; }

// In a call with many rows the first kernel's items are of one token's rows, and it
// takes the requests of up to two such items, two passes over the keys.  Measured
// beside one chunk of 512 (63 requests of 4096 tokens x 8 heads, d = 128; us, one
// pass / two / the second kernel, whatever the rows up to 48): 8 query heads to a
// key/value head 193 / 265 / 333, 4 heads 155 / 227 / 300, 1 head 130 / 203 / 280;
// a pass is 73, so a third would gain nothing (d = 64, 8 heads: 128 / 166 / 268).
// Larger items for them, with one pass for 24 or 32 rows, are not built.  In calls
// of up to 128 rows the second kernel's items are of 128 rows and cost less: there
// the limit is at most that of a call without many.  Where two items are less than a
// token's heads the first kernel gets nothing.
int cache8_few_rows(int rows, int heads, int d) {
  const int two = 2 * cache8_attn_rows(heads, d);
  return cache8_wide_rows(rows) < 256 && two > cache8_narrow_rows(d) ? cache8_narrow_rows(d) : two;
}

cudaError_t launch_cache8_attn(const CacheAttnArgs& a, int d, int sm_count, cudaStream_t stream) {
  const int nt = a.item_rows / 8;
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

cudaError_t set_expire_site_cache8(uint32_t site) {
  return cudaMemcpyToSymbol(c_expire_site, &site, sizeof(site));
}

}  // namespace fa
