// fa_cache8.cuh -- layout of the 8-bit cache shared by the kernels that write
// it, read it back and attend over it.
//
// A page holds page_size tokens (a power of two, 16 to 256) of every
// key/value head; per head it is page_size / 16 groups of 16 tokens, and a
// group is 32 d + 16 bytes:
//   [0, 16d)    K codes [2][d/64][8][4][2][8]
//   [16d, 32d)  V codes [d/64][2][8][4][8][2]
//   32d, 32d+1  K's and V's exponent, signed bytes; the rest is not used
// with the K axes (token / 8, dim / 64, token % 8, dim % 32 / 8, dim % 64 / 32,
// dim % 8) and the V axes (dim / 64, token / 8, dim % 64 / 8, token % 8 / 2,
// dim % 8, token % 2).  A value is its E4M3 code times 2^exponent.
//
// The order is that of the attention's matrix fragments, 16 bytes a lane: lane
// 4 g + t of a warp finds in its pieces the keys of tokens g and g + 8, dims
// 8 t + 0 .. 7 of every 32, and the values of dims 8 g + 0 .. 7 of every 64,
// tokens 2t, 2t + 1, 2t + 8, 2t + 9, those of two neighbouring tokens side by
// side, because P V contracts over tokens.  A warp's loads of 16 bytes then
// cover 512 bytes in a row, and the rows of bf16 that the lanes hold outside
// are whole sectors.
//
// Exponents are powers of two and not any scale: E4M3 has the same relative
// step everywhere above 2^-6, so a finer scale gains nothing there, and a
// block whose scale grows keeps its codes exactly but for those that fall
// below 2^-6 of the new scale.
#pragma once
#include <cstdint>

#include "fa_cache4_work.h"

namespace fa {

constexpr int kExp8 = 60;  // exponents lie within -kExp8 .. kExp8
__host__ __device__ constexpr int group8_bytes(int d) { return 32 * d + 16; }

#ifdef __CUDACC__
// Lane's pieces of 16 bytes: keys of token lane / 4 + 8 h, dims 64 c and on;
// values of dims 64 j and on, tokens 8 h and on.
__device__ __forceinline__ int k8_piece(int d, int h, int c, int lane) {
  return ((h * (d / 64) + c) * 32 + lane) * 16;
}
__device__ __forceinline__ int v8_piece(int d, int j, int h, int lane) {
  return 16 * d + ((j * 2 + h) * 32 + lane) * 16;
}
// One value's code.
__device__ __forceinline__ int v8_at(int d, int tok, int dim) {
  return v8_piece(d, dim >> 6, tok >> 3, ((dim >> 3) & 7) * 4 + ((tok & 7) >> 1)) + (dim & 7) * 2 +
         (tok & 1);
}

// The exponents of a group, whatever its bytes.
__device__ __forceinline__ int exp8(uint32_t byte) {
  return min(max((int)(signed char)byte, -kExp8), kExp8);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Four E4M3 bytes as two pairs of f16 (exact).
__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
#endif

}  // namespace fa
