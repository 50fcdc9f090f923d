// fa_serve_api.cu -- host side of the entry points around the attention
// kernels: norm and rotation of queries and keys, and the paged caches in 4 and 8
// bits.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "fa.h"
#include "fa_cache4.cuh"
#include "fa_cache8.cuh"
#include "fa_serve.h"

namespace {

bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
fa_status head_dim(int d) {
  if (d <= 0) return FA_ERR_INVALID_ARG;
  return d == 64 || d == 128 ? FA_OK : FA_ERR_UNSUPPORTED;
}
// A piece of memory that a call reads or writes, and whether two share a byte.
struct Span {
  const void* p;
  long long bytes;
  bool meets(const Span& o) const {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
    const uintptr_t apart = a <= b ? b - a : a - b;
    return bytes > 0 && o.bytes > 0 && apart < (uintptr_t)(a <= b ? bytes : o.bytes);
  }
};
// Rows of `width` bytes, one at p + b sb + n sn for each b < B, n < N (strides
// in bytes, of any sign).
using Wide = __int128;
struct Rows {
  const void* p;
  Wide sb, sn;
  long long B, N, width;
  // Whether a row begins at an offset between lo and hi, both left out.
  // (Walks the shorter axis and solves for the other.)
  bool begins_within(Wide lo, Wide hi) const {
    const Wide last_b = (B - 1) * sb, last_n = (N - 1) * sn;
    if ((last_b < 0 ? last_b : 0) + (last_n < 0 ? last_n : 0) >= hi ||
        (last_b > 0 ? last_b : 0) + (last_n > 0 ? last_n : 0) <= lo)
      return false;
    if (B > N) return Rows{p, sn, sb, N, B, width}.begins_within(lo, hi);
    const Wide step = sn < 0 ? -sn : sn;
    for (long long b = 0; b < B; ++b) {
      const Wide first = b * sb + (sn < 0 ? (N - 1) * sn : 0);  // then by `step` upwards
      const Wide n = first > lo ? 0 : (step > 0 ? (lo - first) / step + 1 : N);
      if (n < N && first + n * step < hi) return true;
    }
    return false;
  }
  // Two of these rows share a byte.
  bool meet() const {
    if (B > 1 && N > 1) {
      const Wide b = sb < 0 ? -sb : sb, n = sn < 0 ? -sn : sn;
      if (n >= width && b >= (N - 1) * n + width) return false;  // entries apart
      if (b >= width && n >= (B - 1) * b + width) return false;  // tokens apart
    }
    if (N > 1 && sn < width && -sn < width) return true;
    if (B <= 1) return false;
    // Row (b, n) less row (0, n'), b > 0: sb, 2 sb, ... and -(N-1) sn, ... on.
    const Wide from = sb - (N - 1) * sn;
    return Rows{p, sb, sn, B - 1, 2 * N - 1, width}.begins_within(-width - from, width - from);
  }
  bool meet(const Span& o) const {
    if (o.bytes <= 0 || width <= 0) return false;
    const Wide at = (Wide)reinterpret_cast<uintptr_t>(o.p) - (Wide)reinterpret_cast<uintptr_t>(p);
    return begins_within(at - width, at + o.bytes);
  }
};
// Two tensors of such rows share a byte; `may_be` lets the second be the
// first itself.  (Of different strides, each is taken as all of its extent.)
bool meet(const Rows& a, const Rows& b, bool may_be) {
  auto extent = [](const Rows& r, Wide* lo, Wide* hi) {
    *lo = (Wide)reinterpret_cast<uintptr_t>(r.p);
    *hi = *lo + r.width;
    for (Wide x : {(r.B - 1) * r.sb, (r.N - 1) * r.sn}) (x < 0 ? *lo : *hi) += x;
  };
  Wide al, ah, bl, bh;
  extent(a, &al, &ah), extent(b, &bl, &bh);
  if (al >= bh || bl >= ah) return false;
  if ((a.B > 1 && a.sb != b.sb) || (a.N > 1 && a.sn != b.sn)) return true;
  if (may_be && a.p == b.p) return false;
  // Differences of two rows' offsets: from this one up, by sb and sn.
  const Wide from = -((a.B - 1) * a.sb + (a.N - 1) * a.sn);
  const Wide at = (Wide)reinterpret_cast<uintptr_t>(b.p) - (Wide)reinterpret_cast<uintptr_t>(a.p);
  return Rows{a.p, a.sb, a.sn, 2 * a.B - 1, 2 * a.N - 1, a.width}.begins_within(
      at - a.width - from, at + a.width - from);
}
// Memory of a tensor, none where it is not given.
Span span(const void* p, long long bytes) { return {p, p ? bytes : 0}; }
// Whether an output meets an input, or another output.
bool meet(const Span* outs, const Span* outs_end, const Span* ins, const Span* ins_end) {
  for (const Span* o = outs; o != outs_end; ++o) {
    for (const Span* i = ins; i != ins_end; ++i)
      if (o->meets(*i)) return true;
    for (const Span* x = outs; x != o; ++x)
      if (o->meets(*x)) return true;
  }
  return false;
}
bool meet(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  return meet(outs.begin(), outs.end(), ins.begin(), ins.end());
}
fa_status launched(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// ------------------------------------------------------ norm and rotation
fa_status check_rope(int B, int N, int H, int Hkv, int d, int rot, int table_rows, int weight_bf16,
                     float eps, int interleaved, const void* qw, const void* kw,
                     const void* table, const void* qkv, const int* positions,
                     long long stride_b, long long stride_n) {
  if (B < 0 || N < 0 || H < 0 || Hkv < 0) return FA_ERR_INVALID_ARG;
  fa_status s = head_dim(d);
  if (s != FA_OK) return s;
  if (rot <= 0 || rot > d || rot % 16 != 0 || table_rows <= 0) return FA_ERR_INVALID_ARG;
  if (weight_bf16 != 0 && weight_bf16 != 1) return FA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
  if ((qw == nullptr) != (kw == nullptr)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || !(eps >= 0.0f)) return FA_ERR_INVALID_ARG;
  if (H > fa::kRopeMaxHeads || Hkv > fa::kRopeMaxHeads) return FA_ERR_UNSUPPORTED;
  // Rows of one head and packs of heads are counted in 31 bits.
  if ((long long)B * N > INT_MAX || (long long)B * N * (H + 2LL * Hkv) > INT_MAX)
    return FA_ERR_UNSUPPORTED;
  if (B == 0 || N == 0 || H + Hkv == 0) return FA_OK;
  if (!qkv || !table || !aligned(qkv, 16) || !aligned(table, 16) || !aligned(positions, 4))
    return FA_ERR_INVALID_ARG;
  // Weights are read one by one, in their own type.
  if (!aligned(qw, weight_bf16 ? 2 : 4) || !aligned(kw, weight_bf16 ? 2 : 4))
    return FA_ERR_INVALID_ARG;
  if (stride_b % 8 != 0 || stride_n % 8 != 0) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// The axes of positions: none, or n of them with the axis of every pair.
struct Axes {
  int n = 0;
  const uint8_t* of_pair = nullptr;
  // Positions' memory.
  long long bytes(int B, int N) const { return 4LL * B * N * (n > 0 ? n : 1); }
};
constexpr int kMaxAxes = 4;  // two bits a pair
// (Behind check_rope: rot is in range.)
fa_status check_axes(const Axes& x, int rot, const int* positions, bool empty) {
  if (x.n < 1) return FA_ERR_INVALID_ARG;
  if (x.n > kMaxAxes) return FA_ERR_UNSUPPORTED;
  if (!x.of_pair || (!empty && !positions)) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < rot / 2; ++i)
    if (x.of_pair[i] >= x.n) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// The tokens of a [B,N,H+2Hkv,d] tensor.
Rows tokens(const void* p, long long stride_b, long long stride_n, int B, int N, int H, int Hkv,
            int d) {
  return {p, 2 * (Wide)stride_b, 2 * (Wide)stride_n, B, N, 2 * (H + 2LL * Hkv) * d};
}

fa::RopeArgs rope_args(const void* qkv, long long sb, long long sn, const float* table,
                       int table_rows, int rot, const int* positions, const void* qw,
                       const void* kw, int weight_bf16, float eps, int B, int N, int H, int Hkv,
                       const Axes& axes) {
  fa::RopeArgs a = {};
  a.n_axes = axes.n;
  for (int i = 0; axes.n > 0 && i < rot / 2; ++i)
    a.axes[i / 16] |= (uint32_t)axes.of_pair[i] << (2 * (i % 16));
  a.qkv = static_cast<const __nv_bfloat16*>(qkv);
  a.table = table;
  a.positions = positions;
  a.q_weight = qw;
  a.k_weight = kw;
  a.weight_bf16 = weight_bf16;
  a.stride_b = sb;
  a.stride_n = sn;
  a.N = N;
  a.H = H;
  a.Hkv = Hkv;
  a.rot = rot;
  a.table_rows = table_rows;
  a.tokens = B * N;
  a.eps = eps;
  return a;
}

// ------------------------------------------------------------------ cache
// log2 of a page size, or -1.
int page_shift(int page) {
  for (int s = 4; s <= 8; ++s)
    if (page == 1 << s) return s;
  return -1;
}
// A finite power of two within 2^-60 .. 2^60.
bool cache_scale(float g) {
  int e = 0;
  return std::isfinite(g) && g > 0.0f && std::frexp(g, &e) == 0.5f && e > -60 && e <= 61;
}
fa_status check_cache(int pages, int Hkv, int page, int d, int* shift) {
  fa_status s = head_dim(d);
  if (s != FA_OK) return s;
  if (pages < 0 || Hkv < 0 || page <= 0) return FA_ERR_INVALID_ARG;
  if ((*shift = page_shift(page)) < 0) return FA_ERR_UNSUPPORTED;
  if (((long long)pages << *shift) > INT_MAX) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// A format's bytes of a group, and its attention's rows of an item and launch;
// for calls of more than narrow_rows rows a request, where the first kernel takes
// requests of up to few_rows, the second kernel's.
using AttnLaunch = cudaError_t (*)(const fa::CacheAttnArgs& a, int d, int sm_count,
                                   cudaStream_t stream);
struct Format {
  int (*group)(int d);
  int (*rows)(int rows, int d);
  AttnLaunch attn;
  int (*narrow_rows)(int d) = nullptr;
  int (*few_rows)(int rows, int heads, int d) = nullptr;
  int (*wide_rows)(int rows) = nullptr;
  int wide_blocks = 0;
  AttnLaunch wide = nullptr;
};
constexpr Format kCache4 = {fa::group_bytes, fa::cache4_attn_rows, fa::launch_cache4_attn};
constexpr Format kCache8 = {fa::group8_bytes,       fa::cache8_attn_rows, fa::launch_cache8_attn,
                            fa::cache8_narrow_rows, fa::cache8_few_rows,  fa::cache8_wide_rows,
                            fa::kC8WideBlocks,      fa::launch_cache8_wide};

long long cache_bytes(const Format& f, int pages, int Hkv, int page, int d) {
  return (long long)pages * Hkv * (page / fa::kGroup) * f.group(d);
}
size_t page_bytes(const Format& f, int Hkv, int page_size, int d) {
  int shift = 0;
  if (Hkv <= 0 || check_cache(0, Hkv, page_size, d, &shift) != FA_OK) return 0;
  return (size_t)cache_bytes(f, 1, Hkv, page_size, d);
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// Norm and rotation, with or without axes of positions.
fa_status norm_rope(const void* qkv, long long stride_b, long long stride_n, const float* rope,
                    int rope_rows, int rot, const int* positions, const Axes* axes,
                    const void* q_weight, const void* k_weight, int weight_bf16, float eps,
                    int interleaved, void* q, void* k, void* v, int B, int N, int H, int Hkv,
                    int d, void* stream) {
  fa_status s = check_rope(B, N, H, Hkv, d, rot, rope_rows, weight_bf16, eps, interleaved, q_weight,
                           k_weight, rope, qkv, positions, stride_b, stride_n);
  if (s != FA_OK) return s;
  const bool empty = B == 0 || N == 0 || H + Hkv == 0;
  if (axes && (s = check_axes(*axes, rot, positions, empty)) != FA_OK) return s;
  if (empty) return FA_OK;
  if ((H > 0 && !q) || (Hkv > 0 && (!k || !v)) || !aligned(q, 16) || !aligned(k, 16) ||
      !aligned(v, 16))
    return FA_ERR_INVALID_ARG;
  const long long head = 2LL * B * N * d, weight = (weight_bf16 ? 2LL : 4LL) * d;
  const Span qs = span(q, H * head), ks = span(k, Hkv * head), vs = span(v, Hkv * head);
  if (meet({qs, ks, vs}, {span(rope, 4LL * rope_rows * rot), span(positions, (axes ? *axes : Axes()).bytes(B, N)),
                          span(q_weight, weight), span(k_weight, weight)}))
    return FA_ERR_INVALID_ARG;
  const Rows in = tokens(qkv, stride_b, stride_n, B, N, H, Hkv, d);
  if (in.meet(qs) || in.meet(ks) || in.meet(vs)) return FA_ERR_INVALID_ARG;
  fa::DeviceInfo dev;
  if ((s = fa::device_info(&dev)) != FA_OK) return s;
  fa::RopeArgs a = rope_args(qkv, stride_b, stride_n, rope, rope_rows, rot, positions, q_weight,
                             k_weight, weight_bf16, eps, B, N, H, Hkv,
                             axes ? *axes : Axes());
  a.q = static_cast<__nv_bfloat16*>(q);
  a.k = static_cast<__nv_bfloat16*>(k);
  a.v = static_cast<__nv_bfloat16*>(v);
  return launched(fa::launch_rope_fwd(a, d, interleaved != 0, q_weight != nullptr, dev.sm_count,
                                      static_cast<cudaStream_t>(stream)));
}

size_t rope_bwd_workspace(int d) {
  return d == 64 || d == 128 ? (size_t)fa::kRopeMaxBlocks * 2 * d * sizeof(float) : 0;
}

fa_status norm_rope_bwd(const void* qkv, long long stride_b, long long stride_n, const float* rope,
                        int rope_rows, int rot, const int* positions, const Axes* axes,
                        const void* q_weight, const void* k_weight, int weight_bf16, float eps,
                        int interleaved, const void* dq, const void* dk, const void* dv,
                        void* dqkv, long long dstride_b, long long dstride_n, float* dq_weight,
                        float* dk_weight, void* workspace, size_t workspace_bytes, int B, int N,
                        int H, int Hkv, int d, void* stream) {
  fa_status s = check_rope(B, N, H, Hkv, d, rot, rope_rows, weight_bf16, eps, interleaved, q_weight,
                           k_weight, rope, qkv, positions, stride_b, stride_n);
  if (s != FA_OK) return s;
  const bool norm = q_weight != nullptr;
  const bool empty = B == 0 || N == 0 || H + Hkv == 0;
  if (axes && (s = check_axes(*axes, rot, positions, empty)) != FA_OK) return s;
  if (norm) {
    if (!dq_weight || !dk_weight || !aligned(dq_weight, 4) || !aligned(dk_weight, 4))
      return FA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < rope_bwd_workspace(d))
      return FA_ERR_WORKSPACE;
  }
  if (!empty) {
    if ((H > 0 && !dq) || (Hkv > 0 && (!dk || !dv)) || !dqkv || !aligned(dq, 16) ||
        !aligned(dk, 16) || !aligned(dv, 16) || !aligned(dqkv, 16))
      return FA_ERR_INVALID_ARG;
    if (dstride_b % 8 != 0 || dstride_n % 8 != 0) return FA_ERR_INVALID_ARG;
  } else if (!norm) {
    return FA_OK;
  }
  const long long head = 2LL * B * N * d, weight = (weight_bf16 ? 2LL : 4LL) * d;
  const Span ins[] = {span(dq, H * head),
                      span(dk, Hkv * head),
                      span(dv, Hkv * head),
                      span(empty ? nullptr : rope, 4LL * rope_rows * rot),
                      span(empty ? nullptr : positions, (axes ? *axes : Axes()).bytes(B, N)),
                      span(q_weight, weight),
                      span(k_weight, weight)};
  const Span sums[] = {span(norm ? dq_weight : nullptr, 4LL * d),
                       span(norm ? dk_weight : nullptr, 4LL * d),
                       span(norm ? workspace : nullptr, rope_bwd_workspace(d))};
  if (meet(sums, sums + 3, ins, ins + 7)) return FA_ERR_INVALID_ARG;
  if (!empty) {
    const Rows x = tokens(qkv, stride_b, stride_n, B, N, H, Hkv, d);
    const Rows out = tokens(dqkv, dstride_b, dstride_n, B, N, H, Hkv, d);
    // (Without weights qkv is not read.)
    if (out.meet() || (norm && meet(out, x, true))) return FA_ERR_INVALID_ARG;
    for (const Span& i : ins)
      if (out.meet(i)) return FA_ERR_INVALID_ARG;
    for (const Span& i : sums)
      if (out.meet(i) || x.meet(i)) return FA_ERR_INVALID_ARG;
  }
  fa::DeviceInfo dev;
  if ((s = fa::device_info(&dev)) != FA_OK) return s;
  // Without tokens the weights' gradients are zero: the kernels write that.
  fa::RopeArgs a = rope_args(qkv, stride_b, stride_n, rope, rope_rows, rot, positions, q_weight,
                             k_weight, weight_bf16, eps, B, N, H, Hkv,
                             axes ? *axes : Axes());
  a.dq = static_cast<const __nv_bfloat16*>(dq);
  a.dk = static_cast<const __nv_bfloat16*>(dk);
  a.dv = static_cast<const __nv_bfloat16*>(dv);
  a.dqkv = static_cast<__nv_bfloat16*>(dqkv);
  a.dstride_b = dstride_b;
  a.dstride_n = dstride_n;
  a.dq_weight = dq_weight;
  a.dk_weight = dk_weight;
  a.partial = static_cast<float*>(workspace);
  return launched(fa::launch_rope_bwd(a, d, interleaved != 0, norm, dev.sm_count,
                                      static_cast<cudaStream_t>(stream)));
}

// Attention over a cache in either format.
// The workspace of a kernel with items of `rows` rows, `blocks` blocks at
// most, from `ws` on; returns its end.
uintptr_t lay_out(fa::CacheAttnArgs& a, uintptr_t ws, int blocks, int rows, int d, bool notes) {
  a.joins = reinterpret_cast<int4*>(ws);
  ws += align_up(blocks * sizeof(int4));
  a.part = reinterpret_cast<float*>(ws);
  ws += align_up((size_t)blocks * 2 * rows * d * sizeof(float));
  a.part_ml = reinterpret_cast<float2*>(ws);
  ws += align_up((size_t)blocks * 2 * rows * sizeof(float2));
  a.nan_rows = reinterpret_cast<uint32_t*>(ws);
  if (notes) ws += (size_t)blocks * fa::kC8WideThreads * 4 * sizeof(uint32_t);
  a.row_blocks = (int)((a.rows + (long long)rows - 1) / rows);
  return ws;
}
// The kernels of a call of requests with up to `rows` rows, with their places
// in the workspace; returns its end.  In a call with many rows the first kernel
// gets the requests with few of them (by rows, whatever tokens these are): its items
// are of one token's heads.
uintptr_t lay_out(const Format& f, int rows, int heads, int d, uintptr_t ws,
                  fa::CacheAttnArgs& narrow, fa::CacheAttnArgs& wide, bool* is_wide) {
  *is_wide = f.wide && rows > f.narrow_rows(d);
  narrow.item_rows = f.rows(*is_wide ? heads : rows, d);
  narrow.least_rows = 0;
  narrow.most_rows = *is_wide ? f.few_rows(rows, heads, d) : INT_MAX;
  narrow.rows = *is_wide ? std::min(rows, narrow.most_rows) : rows;
  ws = lay_out(narrow, ws, fa::kC4MaxBlocks, narrow.item_rows, d, false);
  if (!*is_wide) return ws;
  wide.rows = rows;
  wide.least_rows = narrow.most_rows + 1;
  wide.most_rows = INT_MAX;
  wide.item_rows = f.wide_rows(rows);
  return lay_out(wide, ws, f.wide_blocks, wide.item_rows, d, true);
}

size_t attn_workspace_size(const Format& f, int B, int H, int Hkv, int T, int d) {
  if (head_dim(d) != FA_OK || B <= 0 || H <= 0 || T <= 0 || Hkv <= 0 || H % Hkv != 0) return 0;
  if ((long long)B * H * T > INT_MAX) return 0;
  fa::CacheAttnArgs narrow = {}, wide = {};
  bool is_wide;
  return lay_out(f, H / Hkv * T, H / Hkv, d, 0, narrow, wide, &is_wide);
}

fa_status cache_attn(const Format& f, const void* q, const void* cache, const int* block_table,
                     const int* seq_lens, const int* q_lens, void* o, float* lse, void* workspace,
                     size_t workspace_bytes, int B, int H, int Hkv, int T, int d, int max_blocks,
                     int pages, int page_size, int window, float scale, float k_scale,
                     float v_scale, void* stream) {
  int shift = 0;
  fa_status s = check_cache(pages, Hkv, page_size, d, &shift);
  if (s != FA_OK) return s;
  if (B < 0 || H < 0 || T < 0 || max_blocks < 0) return FA_ERR_INVALID_ARG;
  if (H > 0 && (Hkv == 0 || Hkv > H || H % Hkv != 0)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return FA_ERR_INVALID_ARG;
  if (!cache_scale(k_scale) || !cache_scale(v_scale)) return FA_ERR_INVALID_ARG;
  const float scale_log2 = scale * k_scale * 1.4426950408889634f;
  if (!std::isfinite(scale_log2)) return FA_ERR_INVALID_ARG;
  // Positions, which begin at -T, less a window stay within an int (and so does the
  // end of the unit that the last key is in, for the kernels that compare with it).
  if (((long long)max_blocks << shift) + T > INT_MAX - (f.wide ? 256 : 0) ||
      (long long)B * H > INT_MAX ||
      (long long)B * H * T > INT_MAX || (long long)B * max_blocks > INT_MAX)
    return FA_ERR_UNSUPPORTED;
  // All requests' units of 128 keys together, and a block's share of the
  // work, are counted in 31 bits.
  if ((double)B * ((double)max_blocks * page_size / 128 + 4) > INT_MAX) return FA_ERR_UNSUPPORTED;
  if ((double)B * max_blocks * page_size * H * T > 0x1p45) return FA_ERR_UNSUPPORTED;
  if (B == 0 || H == 0 || T == 0) return FA_OK;
  if (!q || !seq_lens || !o || !lse || (pages > 0 && !cache) || (max_blocks > 0 && !block_table))
    return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(q_lens, 4))
    return FA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < attn_workspace_size(f, B, H, Hkv, T, d))
    return FA_ERR_WORKSPACE;
  const long long q_rows = (long long)B * H * T;
  if (meet({span(o, 2 * q_rows * d), span(lse, 4 * q_rows),
            span(workspace, attn_workspace_size(f, B, H, Hkv, T, d))},
           {span(q, 2 * q_rows * d), span(cache, cache_bytes(f, pages, Hkv, page_size, d)),
            span(block_table, 4LL * B * max_blocks), span(seq_lens, 4LL * B),
            span(q_lens, 4LL * B)}))
    return FA_ERR_INVALID_ARG;
  fa::DeviceInfo dev;
  if ((s = fa::device_info(&dev)) != FA_OK) return s;
  fa::CacheAttnArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.cache = static_cast<const uint8_t*>(cache);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.q_lens = q_lens;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.B = B;
  a.Hkv = Hkv;
  a.T = T;
  a.M = max_blocks;
  a.pages = pages;
  a.heads = H / Hkv;
  a.by_heads = fa::FastDiv::of(a.heads);
  a.shift = shift;
  // A window of the whole table hides nothing.
  a.window = window < 0 || (long long)window >= ((long long)max_blocks << shift) ? -1 : window;
  a.scale_log2 = scale_log2;
  a.v_scale = v_scale;
  a.st = dev.st;
  a.timeout_ns = dev.timeout_ns;
  a.hook = dev.hook;
  fa::CacheAttnArgs wide = a;
  bool is_wide;
  lay_out(f, a.heads * T, a.heads, d, reinterpret_cast<uintptr_t>(workspace), a, wide,
          &is_wide);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // (Without lengths every request has as many rows, too many for the first.)
  cudaError_t e = cudaSuccess;
  if (!is_wide || q_lens) e = f.attn(a, d, dev.sm_count, st);
  if (is_wide && e == cudaSuccess) e = f.wide(wide, d, dev.sm_count, st);
  return launched(e);
}

}  // namespace

namespace fa {
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);  // (device_info has refused 64 and up)
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}
}  // namespace fa

extern "C" {

fa_status fa_qk_norm_rope(const void* qkv, long long stride_b, long long stride_n,
                          const float* rope, int rope_rows, int rot, const int* positions,
                          const void* q_weight, const void* k_weight, int weight_bf16, float eps,
                          int interleaved, void* q, void* k, void* v, int B, int N, int H, int Hkv,
                          int d, void* stream) {
  return norm_rope(qkv, stride_b, stride_n, rope, rope_rows, rot, positions, nullptr, q_weight,
                   k_weight, weight_bf16, eps, interleaved, q, k, v, B, N, H, Hkv, d, stream);
}

fa_status fa_qk_norm_rope_axes(const void* qkv, long long stride_b, long long stride_n,
                               const float* rope, int rope_rows, int rot, const int* positions,
                               int n_axes, const uint8_t* axes, const void* q_weight,
                               const void* k_weight, int weight_bf16, float eps, int interleaved,
                               void* q, void* k, void* v, int B, int N, int H, int Hkv, int d,
                               void* stream) {
  const Axes x = {n_axes, axes};
  return norm_rope(qkv, stride_b, stride_n, rope, rope_rows, rot, positions, &x, q_weight, k_weight,
                   weight_bf16, eps, interleaved, q, k, v, B, N, H, Hkv, d, stream);
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d) { return rope_bwd_workspace(d); }

fa_status fa_qk_norm_rope_bwd(const void* qkv, long long stride_b, long long stride_n,
                              const float* rope, int rope_rows, int rot, const int* positions,
                              const void* q_weight, const void* k_weight, int weight_bf16,
                              float eps, int interleaved, const void* dq, const void* dk,
                              const void* dv, void* dqkv, long long dstride_b, long long dstride_n,
                              float* dq_weight, float* dk_weight, void* workspace,
                              size_t workspace_bytes, int B, int N, int H, int Hkv, int d,
                              void* stream) {
  return norm_rope_bwd(qkv, stride_b, stride_n, rope, rope_rows, rot, positions, nullptr, q_weight,
                       k_weight, weight_bf16, eps, interleaved, dq, dk, dv, dqkv, dstride_b,
                       dstride_n, dq_weight, dk_weight, workspace, workspace_bytes, B, N, H, Hkv, d,
                       stream);
}

fa_status fa_qk_norm_rope_axes_bwd(const void* qkv, long long stride_b, long long stride_n,
                                   const float* rope, int rope_rows, int rot, const int* positions,
                                   int n_axes, const uint8_t* axes, const void* q_weight,
                                   const void* k_weight, int weight_bf16, float eps,
                                   int interleaved, const void* dq, const void* dk, const void* dv,
                                   void* dqkv, long long dstride_b, long long dstride_n,
                                   float* dq_weight, float* dk_weight, void* workspace,
                                   size_t workspace_bytes, int B, int N, int H, int Hkv, int d,
                                   void* stream) {
  const Axes x = {n_axes, axes};
  return norm_rope_bwd(qkv, stride_b, stride_n, rope, rope_rows, rot, positions, &x, q_weight,
                       k_weight, weight_bf16, eps, interleaved, dq, dk, dv, dqkv, dstride_b,
                       dstride_n, dq_weight, dk_weight, workspace, workspace_bytes, B, N, H, Hkv, d,
                       stream);
}

size_t fa_cache4_page_bytes(int Hkv, int page_size, int d) {
  return page_bytes(kCache4, Hkv, page_size, d);
}

fa_status fa_cache4_plan(const int* new_tokens, int* lens, int* block_table, int* free_list,
                         int* free_count, int* slots, int* positions, int* granted, int R,
                         int max_blocks, int pages, int page_size, int T, void* stream) {
  if (R < 0 || max_blocks < 0 || pages < 0 || T < 0 || page_size <= 0) return FA_ERR_INVALID_ARG;
  const int shift = page_shift(page_size);
  if (shift < 0) return FA_ERR_UNSUPPORTED;
  if (((long long)pages << shift) > INT_MAX || ((long long)max_blocks << shift) > INT_MAX ||
      (long long)R * max_blocks > INT_MAX || (long long)R * T > INT_MAX)
    return FA_ERR_UNSUPPORTED;
  if (R == 0) return FA_OK;
  if (!new_tokens || !lens || !free_count || !granted || (max_blocks > 0 && !block_table) ||
      (pages > 0 && !free_list) || (T > 0 && (!slots || !positions)))
    return FA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)new_tokens, (const void*)lens, (const void*)block_table,
                        (const void*)free_list, (const void*)free_count, (const void*)slots,
                        (const void*)positions, (const void*)granted})
    if (!aligned(p, 4)) return FA_ERR_INVALID_ARG;
  const Span spans[] = {{new_tokens, 4LL * R},      {lens, 4LL * R},
                        {free_count, 4},            {granted, 4LL * R},
                        {block_table, 4LL * R * max_blocks}, {free_list, 4LL * pages},
                        {slots, 4LL * R * T},       {positions, 4LL * R * T}};
  for (const Span& x : spans)
    for (const Span* y = spans; y != &x; ++y)
      if (x.meets(*y)) return FA_ERR_INVALID_ARG;
  fa::PlanArgs a = {};
  a.new_tokens = new_tokens;
  a.lens = lens;
  a.block_table = block_table;
  a.free_list = free_list;
  a.free_count = free_count;
  a.slots = slots;
  a.positions = positions;
  a.granted = granted;
  a.R = R;
  a.M = max_blocks;
  a.P = pages;
  a.T = T;
  a.by_T = fa::FastDiv::of(T > 0 ? T : 1);
  a.shift = shift;
  return launched(fa::launch_cache4_plan(a, static_cast<cudaStream_t>(stream)));
}

fa_status fa_cache4_append(const void* k, const void* v, void* cache, const int* slots,
                           float k_scale, float v_scale, void* k_out, void* v_out, int B, int Hkv,
                           int N, int d, int pages, int page_size, void* stream) {
  int shift = 0;
  fa_status s = check_cache(pages, Hkv, page_size, d, &shift);
  if (s != FA_OK) return s;
  if (B < 0 || N < 0) return FA_ERR_INVALID_ARG;
  if (!cache_scale(k_scale) || !cache_scale(v_scale)) return FA_ERR_INVALID_ARG;
  if ((k_out == nullptr) != (v_out == nullptr)) return FA_ERR_INVALID_ARG;
  if ((long long)B * Hkv > INT_MAX || (long long)B * Hkv * N > INT_MAX) return FA_ERR_UNSUPPORTED;
  if (B == 0 || Hkv == 0 || N == 0 || pages == 0) return FA_OK;
  if (!k || !v || !cache || !slots) return FA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16) || !aligned(slots, 4) ||
      !aligned(k_out, 16) || !aligned(v_out, 16))
    return FA_ERR_INVALID_ARG;
  const long long bytes = 2LL * B * Hkv * N * d;
  const Span ko = span(k_out, bytes), vo = span(v_out, bytes);
  if (meet({span(cache, cache_bytes(kCache4, pages, Hkv, page_size, d)), ko, vo},
           {span(slots, 4LL * B * N), span(k_out == k ? nullptr : k, bytes),
            span(v_out == v ? nullptr : v, bytes)}))
    return FA_ERR_INVALID_ARG;
  // (Values that replace their own keys or values still meet nothing else.)
  if (ko.meets(span(v, bytes)) || vo.meets(span(k, bytes))) return FA_ERR_INVALID_ARG;
  fa::AppendArgs a = {};
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  a.cache = static_cast<uint8_t*>(cache);
  a.slots = slots;
  a.rows = B * Hkv * N;
  a.N = N;
  a.Hkv = Hkv;
  a.by_N = fa::FastDiv::of(N);
  a.by_Hkv = fa::FastDiv::of(Hkv);
  a.pages = pages;
  a.shift = shift;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return launched(fa::launch_cache4_append(a, d, static_cast<cudaStream_t>(stream)));
}

size_t fa_cache4_attn_workspace_size(int B, int H, int Hkv, int T, int d) {
  return attn_workspace_size(kCache4, B, H, Hkv, T, d);
}

fa_status fa_cache4_attn(const void* q, const void* cache, const int* block_table,
                         const int* seq_lens, const int* q_lens, void* o, float* lse,
                         void* workspace, size_t workspace_bytes, int B, int H, int Hkv, int T,
                         int d, int max_blocks, int pages, int page_size, int window, float scale,
                         float k_scale, float v_scale, void* stream) {
  return cache_attn(kCache4, q, cache, block_table, seq_lens, q_lens, o, lse, workspace,
                    workspace_bytes, B, H, Hkv, T, d, max_blocks, pages, page_size, window, scale,
                    k_scale, v_scale, stream);
}

size_t fa_cache8_page_bytes(int Hkv, int page_size, int d) {
  return page_bytes(kCache8, Hkv, page_size, d);
}

fa_status fa_cache8_append(const void* k, const void* v, void* cache, const int* slots, void* k_out,
                           void* v_out, int B, int Hkv, int N, int d, int pages, int page_size,
                           void* stream) {
  int shift = 0;
  fa_status s = check_cache(pages, Hkv, page_size, d, &shift);
  if (s != FA_OK) return s;
  if (B < 0 || N < 0) return FA_ERR_INVALID_ARG;
  if ((k_out == nullptr) != (v_out == nullptr)) return FA_ERR_INVALID_ARG;
  // (A warp's work ends up to 31 tokens behind the last one.)
  if ((long long)B * Hkv > INT_MAX || (long long)B * Hkv * N > INT_MAX || N > INT_MAX - 64)
    return FA_ERR_UNSUPPORTED;
  if (B == 0 || Hkv == 0 || N == 0 || pages == 0) return FA_OK;
  if (!k || !v || !cache || !slots) return FA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16) || !aligned(slots, 4) ||
      !aligned(k_out, 16) || !aligned(v_out, 16))
    return FA_ERR_INVALID_ARG;
  const long long bytes = 2LL * B * Hkv * N * d;
  const Span ko = span(k_out, bytes), vo = span(v_out, bytes);
  if (meet({span(cache, cache_bytes(kCache8, pages, Hkv, page_size, d)), ko, vo},
           {span(slots, 4LL * B * N), span(k_out == k ? nullptr : k, bytes),
            span(v_out == v ? nullptr : v, bytes)}))
    return FA_ERR_INVALID_ARG;
  // (The cache meets no input; values that replace their own keys or values
  // still meet nothing else.)
  if (ko.meets(span(v, bytes)) || vo.meets(span(k, bytes))) return FA_ERR_INVALID_ARG;
  fa::Append8Args a = {};
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  a.cache = static_cast<uint8_t*>(cache);
  a.slots = slots;
  a.N = N;
  a.Hkv = Hkv;
  a.chunks = (N - 1) / 16 + 1;
  a.warps = B * Hkv * a.chunks;
  a.by_chunks = fa::FastDiv::of(a.chunks);
  a.by_Hkv = fa::FastDiv::of(Hkv);
  a.slots_end = pages << shift;
  a.shift = shift;
  return launched(fa::launch_cache8_append(a, d, static_cast<cudaStream_t>(stream)));
}

fa_status fa_cache8_read(const void* cache, const int* block_table, const int* seq_lens,
                         const int* starts, void* k_out, void* v_out, int B, int Hkv, int N, int d,
                         int max_blocks, int pages, int page_size, void* stream) {
  int shift = 0;
  fa_status s = check_cache(pages, Hkv, page_size, d, &shift);
  if (s != FA_OK) return s;
  if (B < 0 || N < 0 || max_blocks < 0) return FA_ERR_INVALID_ARG;
  // Positions and a row block's end are counted in 31 bits.
  if ((long long)B * Hkv > INT_MAX || (long long)B * Hkv * ((N + 15LL) / 16 + 1) > INT_MAX ||
      N > INT_MAX - 64 || (((long long)max_blocks << shift) + 64) > INT_MAX ||
      (long long)B * max_blocks > INT_MAX)
    return FA_ERR_UNSUPPORTED;
  if (B == 0 || Hkv == 0 || N == 0 || max_blocks == 0 || pages == 0) return FA_OK;
  if (!cache || !block_table || !seq_lens || !k_out || !v_out) return FA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(starts, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return FA_ERR_INVALID_ARG;
  const long long bytes = 2LL * B * Hkv * N * d;
  if (meet({span(k_out, bytes), span(v_out, bytes)},
           {span(cache, cache_bytes(kCache8, pages, Hkv, page_size, d)),
            span(block_table, 4LL * B * max_blocks), span(seq_lens, 4LL * B), span(starts, 4LL * B)}))
    return FA_ERR_INVALID_ARG;
  fa::Read8Args a = {};
  a.cache = static_cast<const uint8_t*>(cache);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.starts = starts;
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  a.N = N;
  a.Hkv = Hkv;
  a.M = max_blocks;
  a.pages = pages;
  a.chunks = (N - 1) / 16 + 2;  // groups that N tokens may lie in
  a.warps = B * Hkv * a.chunks;
  a.by_chunks = fa::FastDiv::of(a.chunks);
  a.by_Hkv = fa::FastDiv::of(Hkv);
  a.shift = shift;
  return launched(fa::launch_cache8_read(a, d, static_cast<cudaStream_t>(stream)));
}

size_t fa_cache8_attn_workspace_size(int B, int H, int Hkv, int T, int d) {
  return attn_workspace_size(kCache8, B, H, Hkv, T, d);
}

fa_status fa_cache8_attn(const void* q, const void* cache, const int* block_table,
                         const int* seq_lens, const int* q_lens, void* o, float* lse,
                         void* workspace, size_t workspace_bytes, int B, int H, int Hkv, int T,
                         int d, int max_blocks, int pages, int page_size, int window, float scale,
                         void* stream) {
  return cache_attn(kCache8, q, cache, block_table, seq_lens, q_lens, o, lse, workspace,
                    workspace_bytes, B, H, Hkv, T, d, max_blocks, pages, page_size, window, scale,
                    1.0f, 1.0f, stream);
}

}  // extern "C"
