// fa_cache4_attn.cu -- the attention over the paged 4-bit cache
// (fa_cache_attn.cuh has the work's division and the main loop):
// k_j, v_j = code * scale * g, with a scale for every 16 dims of a token.
//
// A code times its scale has at most six significant bits: K and V enter the
// products exactly.
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
#include "fa_cache_attn.cuh"

namespace fa {
namespace {

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

struct Cache4 {
  static constexpr uint32_t kWhere = 0x511;
  static constexpr int kItemCost = kC4ItemCost;
  static constexpr __host__ __device__ int group_bytes(int d) { return fa::group_bytes(d); }
  static constexpr __host__ __device__ int blocks_per_sm(int d, int nt) {
    return nt == 1 || (nt == 2 && d == 64) ? 3 : 2;
  }
  // Lane t takes dims t D/4 + 0 .. D/4 - 1 of K; lane g the eighth g of V's.
  static __device__ __forceinline__ int q_piece(int d, int t, int i) { return t * (d / 2) + 16 * i; }
  static __device__ __forceinline__ int o_dim(int d, int g, int dt) { return g * (d / 8) + 2 * dt; }
  // (A group shares no factor: its scales are in the operands.)
  struct Scales {
    __device__ __forceinline__ float score(float x) const { return x; }
    __device__ __forceinline__ float less(float m) const { return m; }
    __device__ __forceinline__ float more(float m) const { return m; }
    __device__ __forceinline__ void sum(float& l, float p) const { l += p; }
  };
  static __device__ __forceinline__ Scales scales(const uint8_t*, int) { return {}; }

  // One group's scores, S^T = K Q^T: tokens g and g + 8, rows 2t and 2t + 1.
  template <int D, int NT, typename R>
  static __device__ __forceinline__ void scores(const uint8_t* grp, int g, int t, const R& r,
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
        if constexpr (Shape<Cache4, D, NT>::kQInRegs)
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
  static __device__ __forceinline__ void products(const uint8_t* grp, int g, int t, const uint32_t (&vs)[2],
                                                  const uint32_t (&pb)[NT][2],
                                                  float (&o)[D / 16][NT][4]) {
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

  // The same with the scales' NaNs looked after.
  template <int D, int NT, bool kPlain>
  static __device__ __forceinline__ void values(const uint8_t* grp, int g, int t,
                                                const uint32_t (&pb)[NT][2], float (&o)[D / 16][NT][4],
                                                int there, int tok, const Bounds& bd) {
    uint32_t vs[2], nans = 0;  // by token of the group: a scale of the lane's dims is NaN
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t two = *reinterpret_cast<const uint16_t*>(
          grp + v_scale_at(D, 8 * h + 2 * t, D == 128 ? g : g >> 1));
      if constexpr (!kPlain) {
        if (!there) two = 0;
        const uint32_t nan = __vcmpeq4(two & 0x7f7fu, 0x7f7f7f7fu);
        nans |= ((nan & 1) | (nan >> 7 & 2)) << (8 * h + 2 * t);
        two &= ~nan;
      }
      vs[h] = e4m3_to_f16(two);
    }
    products<D, NT>(grp, g, t, vs, pb, o);
    // A NaN goes to the rows that see its token, and not, by a weight of zero,
    // to the others (a token that no row sees may hold anything).
    if (!kPlain && __any_sync(0xffffffffu, nans != 0)) {
      nans |= __shfl_xor_sync(0xffffffffu, nans, 1);
      nans |= __shfl_xor_sync(0xffffffffu, nans, 2);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t see = bd.seen(8 * nt + 2 * t + i, tok);
          if (nans & see) {
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt)
              o[dt][nt][i] = o[dt][nt][i + 2] = __uint_as_float(0x7fffffffu);
          }
        }
    }
  }
};

template <int D, int NT, bool kHook>
__global__ void __launch_bounds__(kWarps * 32, Cache4::blocks_per_sm(D, NT))
    cache4_attn_kernel(CacheAttnArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Block<Cache4, D, NT> block;
  block.begin();
  wait_for_stream();
  cache_attn<Cache4, D, NT, kHook>(a, block, smem);
}

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32) cache4_join_kernel(CacheAttnArgs a) {
  wait_for_stream();
  cache_join<Cache4, D, NT>(a);
}

template <int D, int NT, bool kHook = false>
cudaError_t run(const CacheAttnArgs& a, int sm_count, cudaStream_t stream) {
  // The hook has its own instantiation, for d = 128 and items of 8 rows only.
  if constexpr (D == 128 && NT == 1 && !kHook) {
    if (a.hook) return run<D, NT, true>(a, sm_count, stream);
  }
  static std::atomic<unsigned long long> done{0};
  return run_cache_attn<Cache4, D, NT>(cache4_attn_kernel<D, NT, kHook>, cache4_join_kernel<D, NT>,
                                       a, sm_count, done, stream);
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

cudaError_t launch_cache4_attn(const CacheAttnArgs& a, int d, int sm_count, cudaStream_t stream) {
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

cudaError_t set_expire_site_cache4(uint32_t site) {
  return cudaMemcpyToSymbol(c_expire_site, &site, sizeof(site));
}

}  // namespace fa
