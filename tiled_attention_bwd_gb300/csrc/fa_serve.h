// fa_serve.h -- internal interface between the host layer (fa_serve_api.cu)
// and the kernels of the norm with rotation and of the caches (fa_rope.cu,
// fa_cache4.cu, fa_cache4_attn.cu, fa_cache8*.cu).  Not part of the ABI.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "fa.h"
#include "fa_cache4_work.h"

namespace fa {

struct DevState;

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
  const int* positions;      // [B, N] or null (row n of an entry: n); with
                             // axes [n_axes, B, N]
  int n_axes;                // 0: positions have no axes
  uint32_t axes[4];          // axis of each pair, two bits each
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
  FastDiv by_T;
  int shift;              // log2 of the page size
  int wide;               // set by the launcher: slots, positions 16-byte aligned
};
cudaError_t launch_cache4_plan(PlanArgs a, cudaStream_t stream);

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

// New keys and values into their slots of the 8-bit cache.
struct Append8Args {
  const __nv_bfloat16 *k, *v;    // [B, Hkv, N, d]
  __nv_bfloat16 *k_out, *v_out;  // rounded values, or null
  uint8_t* cache;
  const int* slots;              // [B, N]
  int warps;                     // B * Hkv * chunks
  int N, Hkv, chunks, slots_end, shift;
  FastDiv by_chunks, by_Hkv;
};
cudaError_t launch_cache8_append(const Append8Args& a, int d, cudaStream_t stream);

// Tokens of the 8-bit cache back into rows.
struct Read8Args {
  const uint8_t* cache;
  const int* block_table;        // [B, M]
  const int* seq_lens;           // [B]
  const int* starts;             // [B] or null (0)
  __nv_bfloat16 *k_out, *v_out;  // [B, Hkv, N, d]
  int warps;                     // B * Hkv * chunks
  int N, Hkv, M, pages, chunks, shift;
  FastDiv by_chunks, by_Hkv;
};
cudaError_t launch_cache8_read(const Read8Args& a, int d, cudaStream_t stream);

// Attention over a cache, in either format.
constexpr int kC4MaxBlocks = 640;
constexpr int kC8WideThreads = 256;  // of the wide kernel's softmax
struct CacheAttnArgs {
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
  uint32_t* nan_rows;       // [kC8WideBlocks][kC8WideThreads][4] (wide kernel)
  int B, Hkv, T, M, pages;
  int heads;                // H / Hkv, of one key/value head
  FastDiv by_heads;
  int rows;                 // heads * T: a request's most
  int item_rows;            // of an item
  int row_blocks;
  int least_rows, most_rows;  // live rows of the requests that the kernel takes
  int shift;                // log2 of the page size
  int window;               // < 0: none
  float scale_log2;         // scale * k_scale * log2(e)
  float v_scale;
  DevState* st;
  uint64_t timeout_ns;
  int hook;                 // 1: run the failure-path test hook instantiation
};
// Query rows of one work item for requests of `rows`: a multiple of 8 up to 40.
int cache4_attn_rows(int rows, int d);
cudaError_t launch_cache4_attn(const CacheAttnArgs& a, int d, int sm_count,
                               cudaStream_t stream);
int cache8_attn_rows(int rows, int d);
cudaError_t launch_cache8_attn(const CacheAttnArgs& a, int d, int sm_count,
                               cudaStream_t stream);
// The same for requests with many rows.  Calls of up to cache8_narrow_rows a
// request are for the first kernel alone; in others (of `rows` a request) it takes
// those with up to cache8_few_rows, which is less than `rows`.
int cache8_narrow_rows(int d);
int cache8_few_rows(int rows, int heads, int d);
int cache8_wide_rows(int rows);  // of an item, for requests of `rows`
constexpr int kC8WideBlocks = 160;
cudaError_t launch_cache8_wide(const CacheAttnArgs& a, int d, int sm_count,
                               cudaStream_t stream);
// The site whose waits expire (0: none), on the current device.  Synchronous;
// call only while no kernel of the library runs.
cudaError_t set_expire_site_cache4(uint32_t site);
cudaError_t set_expire_site_cache8(uint32_t site);
cudaError_t set_expire_site_cache8_wide(uint32_t site);

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
//
// What the work before wrote (lengths, tables, slots, positions, weights) is
// read by plain loads only.  A read-only load (__ldg, a const __restrict__
// pointer) says that the data does not change while the kernel lives, which
// is not so before the wait, and the clobber here does not hold it back.
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
#endif

// Lets a kernel use `bytes` of dynamic shared memory on the current device;
// the attribute is set once per kernel (its own `done`) and device.
cudaError_t allow_smem(const void* kernel, int bytes,
                       std::atomic<unsigned long long>& done);

// Status record, SM count and wait limit of the current device, and whether
// the failure-path test hook has a site.
struct DeviceInfo {
  DevState* st;
  int sm_count;
  uint64_t timeout_ns;
  int hook;
};
fa_status device_info(DeviceInfo* out);

}  // namespace fa
