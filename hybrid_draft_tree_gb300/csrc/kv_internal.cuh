// Declarations shared by the paged-cache translation units (kv.cu, kv_append.cu, kv_attend.cu).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "graft_internal.cuh"

namespace graft {

struct KvLayout {
  int32_t q_heads, kv_heads, dim, rot, interleaved, page_size, page_shift, num_pages;
  int64_t page_stride, head_stride, token_stride;  // elements
};

// Quotients of numbers below 2^31 by a divisor that the host knows: with s = ceil(log2 d) and
// mul = floor(2^32 (2^s - d) / d) + 1, n / d = (n + floor(n mul / 2^32)) / 2^s.
struct Divisor {
  uint32_t mul = 0, shift = 0, d = 1;
  Divisor() = default;
  explicit Divisor(uint32_t n) : d(n) {
    while ((1ull << shift) < n) ++shift;
    mul = (uint32_t)((((1ull << shift) - n) << 32) / n + 1);
  }
  __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift); }
};

struct AppendArgs {
  KvLayout c;
  int32_t batch, slots;
  int32_t vec;  // 1 = 16-byte loads and stores everywhere, and whole 16-byte pieces rotate together
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const int32_t *depth, *rows;
  const float* rope;
  int32_t rope_len, prefix_len;
  const int32_t* page_table;
  int32_t table_stride;
  const int32_t* ctx_len;
  void *q_out, *k_cache, *v_cache;
  Divisor by_slots, by_turn, by_value;  // slots; 16-byte pieces of a rotating head (each with its partner), of a head
  uint32_t* err;
};

// How a call's work is laid out (plan_kv_attend): packed items' rows of all requests against the prefix, then each
// request's rows against its own context (and, when none are packed, the prefix).
struct AttendPlan {
  int32_t packed, cut;       // cut: CTAs take equal pieces of the line of items; else an item each
  int32_t ctas, items_a;     // items_a: packed items
  int32_t tiles_b;           // row tiles of a request and head
  int32_t nt_a, nt_b;        // row tiles of an item
  int32_t tile;              // rows of a tile: the most whole groups in 128
  int32_t fixed_a, fixed_b, step_a, step_b;  // cost of an item before its first block, and of a block
  int64_t rows;              // query rows times query heads
};

struct AttendArgs {
  KvLayout c;
  int32_t batch, slots, group;  // group = query heads per kv head
  const void *q, *k_cache, *v_cache;
  int64_t q_stride, out_stride;
  const int32_t* prefix_pages;
  int32_t prefix_len;
  const int32_t* page_table;
  int32_t table_stride;
  const int32_t* ctx_len;
  int32_t max_ctx;
  const uint64_t* tree_mask;
  float scale;
  void* out;
  float* lse;
  int32_t q_map, out_vec;  // 1 = queries come by tensor map; the output's rows start on 16-byte boundaries
  Divisor by_group, by_heads;  // group, kv_heads
  AttendPlan plan;
  float *part_o, *part_lse;  // partial results (rows of dim) and their log-sum-exp in log2
  int64_t* line;             // [batch] starts of the requests' items; a CTA's share; [ctas] items that a CTA begins and does not end
  uint32_t wait_polls;       // 0 = the default
  uint32_t* err;
};

// 16-bit element types of the cache: packed pairs to and from fp32.
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 get(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t put(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 round(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 get(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t put(float lo, float hi) {
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  static __device__ __forceinline__ float one(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half round(float x) { return __float2half_rn(x); }
};

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t s);
cudaError_t prepare_kv_attend();
int64_t kv_attend_part_rows(int64_t rows, int num_sms);
AttendPlan plan_kv_attend(int batch, int slots, int group, int kv_heads, int dim, int prefix_len, int max_ctx,
                          int num_sms);
cudaError_t launch_kv_attend(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, int dtype, cudaStream_t s);

}  // namespace graft
