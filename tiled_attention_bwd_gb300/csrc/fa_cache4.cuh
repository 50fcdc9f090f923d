// fa_cache4.cuh -- layout of the 4-bit cache shared by the kernels that
// write it and the attention that reads it.
//
// A page holds page_size tokens (a power of two, 16 to 256) of every
// key/value head; per head it is page_size / 16 groups of 16 tokens, and a
// group is 18 d bytes:
//   [0, 8d)    K codes   [16 tokens][d/2]: two E2M1 codes a byte, even dim low
//   [8d, 9d)   K scales  [16 tokens][d/16]: E4M3, one per 16 dims
//   [9d, 17d)  V codes   [2][8][4][2][d/16]
//   [17d, 18d) V scales  [2][d/16][4][2]
// with the V axes (token / 8, the dims in eighths, token % 8 / 2, token % 2).
// A value is code * scale * g, g the call's power of two for K or V.
//
// K rows are plain because Q K^T contracts over dims: a matrix fragment's
// pairs are neighbouring dims, i.e. whole bytes.  P V contracts over tokens:
// the V order puts what one lane of a fragment needs (tokens 2t, 2t + 1 of
// one eighth of the dims) into d/8 consecutive bytes.
#pragma once
#include <cstdint>

namespace fa {

constexpr int kGroup = 16;  // tokens of a group
__host__ __device__ constexpr int group_bytes(int d) { return 18 * d; }

__device__ __forceinline__ int k_code_at(int d, int tok, int byte) { return tok * (d / 2) + byte; }
__device__ __forceinline__ int k_scale_at(int d, int tok, int blk) {
  return 8 * d + tok * (d / 16) + blk;
}
// First of the d/16 code bytes of eighth `oct`.
__device__ __forceinline__ int v_code_at(int d, int tok, int oct) {
  return 9 * d + ((((tok >> 3) * 8 + oct) * 4 + ((tok & 7) >> 1)) * 2 + (tok & 1)) * (d / 16);
}
__device__ __forceinline__ int v_scale_at(int d, int tok, int blk) {
  return 17 * d + (((tok >> 3) * (d / 16) + blk) * 4 + ((tok & 7) >> 1)) * 2 + (tok & 1);
}

}  // namespace fa
