// fa_launch.h -- internal interface between the host layer (fa_api.cu) and
// the kernel translation units (fa_fwd.cu, fa_bwd.cu).  Not part of the ABI.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "fa.h"

namespace fa {

struct DevState;

struct FwdArgs {
  __nv_bfloat16* o;     // [BH, N, d]
  int o_wide;           // 1: o is 32-byte aligned (rows leave in 32-byte stores)
  float* lse;           // [BH, N]
  int BH;               // batch x query heads
  int N;
  int H;                // query heads per batch entry
  int Hkv;              // key/value heads per batch entry (divides H)
  int window;           // band half-width in keys, < 0: none
  int group;            // heads per scheduling group
  float scale_log2;     // scale * log2(e): scores enter exp2 directly
  // Per-sequence lengths ([B] int32, device) or null: batch entry b attends
  // over its first seq_lens[b] rows only.
  const int* seq_lens;
  // With lengths: 1 when the kernel builds its balanced item table in shared
  // memory (set by the launcher when the table fits), else 0.
  int sched;
  // FP8 path only: per-16-row-block scales of the E4M3 Q and K,
  // [BH or BHkv][n_sblk] with n_sblk = N rounded up to 128, over 16.
  const float* q_scale;
  const float* k_scale;
  int n_sblk;
  // 1: blocks claim items from this call's work counter (a slot of a
  // zero-initialised ring, with its count of finished blocks; the last
  // block resets both); 0: items are dealt in alternating rounds.  Calls
  // with a window always use 0.
  int dynamic;
  // 1: each work item is one Q tile instead of a pair (set when a problem
  // has fewer pairs than SMs; never with per-sequence lengths).
  int single;
  unsigned int* work_next;
  unsigned int* work_done;
  int hook;           // 1: run the failure-path test hook instantiation
  DevState* st;
  uint64_t timeout_ns;
};

struct BwdArgs {
  const __nv_bfloat16* o;     // [BH, N, d]
  const __nv_bfloat16* dout;  // [BH, N, d]
  const float* lse;           // [BH, N]
  float* dq_acc;              // [BH, N, d]  fp32 workspace
  float* ddot;                // [BH, N_pad] D_i = dO_i . O_i  (0 past N)
  float* lse2;                // [BH, N_pad] -LSE_i * log2(e)  (-inf past N)
  __nv_bfloat16* dq;          // [BH, N, d]
  __nv_bfloat16* dk;          // [BHkv, N, d]
  __nv_bfloat16* dv;          // [BHkv, N, d]
  float* dk_acc;              // [BHkv, N, d] fp32, used when nsplit > 1
  float* dv_acc;              // [BHkv, N, d] fp32, used when nsplit > 1
  int BH;                     // batch x query heads
  int BHkv;                   // batch x key/value heads
  int H;                      // query heads per batch entry
  int Hkv;                    // key/value heads per batch entry (divides H)
  int window;                 // band half-width in keys, < 0: none
  const int* seq_lens;        // [B] int32 per-sequence lengths, or null
  int hpb;                    // query heads per block (divides H / Hkv)
  int nsplit;                 // blocks per (key/value head, key tile)
  int N;
  int N_pad;                  // N rounded up to a multiple of 128
  int group;                  // key/value heads per scheduling group
  float scale;
  float scale_log2;
  unsigned int* work_next;    // main kernel's work counter (workspace)
  int hook;                   // 1: run the failure-path test hook instantiation
  DevState* st;
  uint64_t timeout_ns;
};

// Norm of query and key heads with the rotation of positions, and backward.
constexpr int kRopeMaxHeads = 8192;   // of H and of Hkv
constexpr int kRopeMaxBlocks = 1024;  // a token of 3 kRopeMaxHeads heads needs 768
struct RopeDeal {
  int packs;                 // packs of heads of a token
  int step, step_b, step_n;  // tokens taken at a time = step_b entries + step_n
};
struct RopeArgs {
  const __nv_bfloat16* qkv;  // [B, N, H + 2 Hkv, d], strides below
  const float* table;        // [table_rows, rot]: rot/2 cosines, rot/2 sines
  const int* positions;      // [B, N] or null (row n of an entry: n)
  const void* q_weight;      // [d], bf16 or fp32
  const void* k_weight;
  int weight_bf16;
  __nv_bfloat16 *q, *k, *v;        // forward: out, [B, H or Hkv, N, d]
  const __nv_bfloat16 *dq, *dk, *dv;  // backward: in
  __nv_bfloat16* dqkv;             // backward: out
  float *dq_weight, *dk_weight;    // [d]
  float* partial;                  // [kRopeMaxBlocks, 2 d] (backward, with norm)
  long long stride_b, stride_n;    // of qkv, in elements
  long long dstride_b, dstride_n;  // of dqkv
  int N, H, Hkv, rot, table_rows;
  int tokens;                      // B * N
  float eps;
  // Set by the launcher: how warps take the packs of a token, all together
  // (forward) or query and key heads first, then value heads (backward).
  RopeDeal all, grad, value;
  int blocks;
};
cudaError_t launch_rope_fwd(const RopeArgs& a, int d, bool interleaved,
                            bool norm, int sm_count, cudaStream_t stream);
cudaError_t launch_rope_bwd(const RopeArgs& a, int d, bool interleaved,
                            bool norm, int sm_count, cudaStream_t stream);

// Block tables and slot maps of the paged cache.
struct PlanArgs {
  const int* new_tokens;  // [R]
  int* lens;              // [R]
  int* block_table;       // [R, M]
  int* free_list;         // [P]
  int* free_count;        // [1]
  int* slots;             // [R, T]
  int* positions;         // [R, T]
  int* granted;           // [R]
  int R, M, P, T;
  int shift;              // log2 of the page size
  int wide;               // set by the launcher: slots, positions 16-byte aligned
};
cudaError_t launch_cache4_plan(PlanArgs a, cudaStream_t stream);

// Division of 0 <= x < 2^31 by a number fixed at launch: three instructions
// instead of about twenty (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994).
struct FastDiv {
  uint32_t by, mul, shift;
  static FastDiv of(uint32_t by) {
    FastDiv f = {by, 0, 0};
    while (f.shift < 31 && (1u << f.shift) < by) ++f.shift;
    f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - by)) / by + 1);
    return f;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t x) const {
    return (__umulhi(mul, x) + x) >> shift;
  }
#endif
};

// New keys and values into their slots of the 4-bit cache.
struct AppendArgs {
  const __nv_bfloat16 *k, *v;    // [B, Hkv, N, d]
  __nv_bfloat16 *k_out, *v_out;  // rounded values, or null
  uint8_t* cache;
  const int* slots;              // [B, N]
  int rows;                      // B * Hkv * N
  int N, Hkv, pages, shift;
  FastDiv by_N, by_Hkv;
  float k_scale, v_scale;
};
cudaError_t launch_cache4_append(const AppendArgs& a, int d, cudaStream_t stream);

// Attention over the 4-bit cache.
constexpr int kC4MaxBlocks = 640;
struct Cache4AttnArgs {
  const __nv_bfloat16* q;   // [B, H, T, d]
  const uint8_t* cache;
  const int* block_table;   // [B, M]
  const int* seq_lens;      // [B]
  const int* q_lens;        // [B] or null
  __nv_bfloat16* o;         // [B, H, T, d]
  float* lse;               // [B, H, T]
  // Workspace: what the join does per block, and partial results.
  int4* joins;              // [kC4MaxBlocks]
  float* part;              // [2 kC4MaxBlocks][item rows][d]
  float2* part_ml;          // [2 kC4MaxBlocks][item rows]
  int B, Hkv, T, M, pages;
  int rows;                 // H / Hkv * T: rows of one key/value head
  int row_blocks;
  int shift;                // log2 of the page size
  int window;               // < 0: none
  float scale_log2;         // scale * k_scale * log2(e)
  float v_scale;
  DevState* st;
  uint64_t timeout_ns;
};
// Query rows of one work item: a multiple of 8 up to 40.
int cache4_attn_rows(int rows, int d);
cudaError_t launch_cache4_attn(const Cache4AttnArgs& a, int d, int sm_count,
                               cudaStream_t stream);

// Launches a kernel whose launch overlaps the end of the work before it in
// the stream.  The kernel waits for that work on the device, by
// wait_for_stream(), before its first access to global memory.
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, dim3 block,
                              size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}
#ifdef __CUDACC__
// Every thread that touches global memory calls it first, and at least one
// thread of a grid always does: a grid that ended without waiting would let
// the one after it start before the one before it is done.
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
#endif

// Lets a kernel use `bytes` of dynamic shared memory on the current device;
// the attribute is set once per kernel (its own `done`) and device.
cudaError_t allow_smem(const void* kernel, int bytes,
                       std::atomic<unsigned long long>& done);

// Status record, SM count and wait limit of the current device.
struct DeviceInfo {
  DevState* st;
  int sm_count;
  uint64_t timeout_ns;
};
fa_status device_info(DeviceInfo* out);

// Each returns the launch error (cudaSuccess on success).  `to` maps O
// ([BH, N, d] bf16, boxes of 32 rows x 64 columns, 128-byte swizzle) for the
// kernels that store O by TMA.
cudaError_t launch_fwd(const CUtensorMap& tq, const CUtensorMap& tk,
                       const CUtensorMap& tv, const CUtensorMap& to,
                       const FwdArgs& a, int BH, int d, bool causal,
                       int grid_blocks, cudaStream_t stream);
// FP8 forward: tq, tk are E4M3 tensor maps (one byte per element, rows of
// 128 bytes: at d = 64 the upper half of each row is zero), tv the bf16 V
// map; d = 64 or 128.
cudaError_t launch_fwd_fp8(const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& tv, const CUtensorMap& to,
                           const FwdArgs& a, int BH, int d, bool causal,
                           int grid_blocks, cudaStream_t stream);
// E4M3 codes and per-16-row-block scales of a bf16 [BH, N, d] tensor
// (d = 64 or 128); scales has BH * n_sblk entries, 1 for blocks past N.
// Code rows are `pitch` bytes apart (>= d), bytes d .. pitch - 1 zero.
cudaError_t launch_quant_e4m3(const __nv_bfloat16* x, uint8_t* codes,
                              float* scales, int BH, int N, int d, int n_sblk,
                              int pitch, int grid_blocks, cudaStream_t stream);
cudaError_t launch_bwd_pre(const BwdArgs& a, int d, int grid_blocks,
                           cudaStream_t stream);
// Persistent: min(work items, grid_blocks) blocks, one per SM.
cudaError_t launch_bwd_main(const CUtensorMap& tq, const CUtensorMap& tk,
                            const CUtensorMap& tv, const CUtensorMap& tdo,
                            const CUtensorMap& tdq, const CUtensorMap& tdk,
                            const CUtensorMap& tdv, const BwdArgs& a, int d,
                            bool causal, int grid_blocks, cudaStream_t stream);
cudaError_t launch_bwd_post(const BwdArgs& a, int d, int grid_blocks,
                            cudaStream_t stream);
cudaError_t launch_expire_wait(DevState* st, uint64_t timeout_ns,
                               cudaStream_t stream);
// The failure-path test hook of the forward / backward kernels (the site
// whose waits expire at once, 0 for none), for the current device.
// Synchronous; call only while no kernel of the library runs.
cudaError_t set_expire_site_fwd(uint32_t site);
cudaError_t set_expire_site_bwd(uint32_t site);

}  // namespace fa
