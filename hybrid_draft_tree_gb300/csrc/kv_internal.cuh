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
  int32_t eight;                                   // 1 = the caches hold e4m3 numbers
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
  const int32_t* position;  // [axes][tokens], or NULL
  int64_t tokens;           // batch * slots
  int32_t axes;
  uint8_t pair_axis[64];    // axis whose position turns a pair
  uint64_t piece_axis;      // 4 bits for each 16-byte piece: the axis of its pairs (8 of halves, 4 of neighbours), or kMixed
  const float *k_scale, *v_scale;  // of 8-bit caches
  uint32_t* err;
};

constexpr int kMixed = 15;

struct ReadArgs {
  KvLayout c;
  int32_t batch, slots, vec;  // vec: 16-byte stores of the rows
  const void *k_cache, *v_cache;
  const int32_t *page_table, *first, *count;
  int32_t table_stride;
  const float *k_scale, *v_scale;
  void *k_out, *v_out;
  int64_t k_stride, v_stride;
  Divisor by_slots, by_head;  // slots; 16-byte pieces of a head
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
  // An 8-bit cache and at most 16 rows a request and head: tiles of 8 rows (1 or 2; else 0) on the CTAs from `split` on;
  // those before take the packed items, `chunk_a` of their line each.
  int32_t few, split;
  int64_t chunk_a;
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
  const float *k_scale, *v_scale;  // of 8-bit caches
  float softcap;             // 0 = none
  int32_t window;            // 0 = none
  const float* slope;        // [q_heads], or NULL
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

// A head's scale of an 8-bit cache; one that is no number above zero counts as 1.
__device__ __forceinline__ float checked_scale(float s, uint32_t* err) {
  if (s > 0.f && s < INFINITY) return s;
  atomicOr(err, GRAFT_ERR_RULE);
  return 1.f;
}
__device__ __forceinline__ float kv_scale(const float* scale, int head, uint32_t* err) {
  return scale ? checked_scale(scale[head], err) : 1.f;
}

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_kv_read(const ReadArgs& a, int dtype, cudaStream_t s);
int kv_attend_form(const float* slope, float softcap, int window);  // which of the forms below a call takes, 0 the plain one
cudaError_t prepare_kv_attend(int form, int dtype, int dim, bool eight);
int64_t kv_attend_part_rows(int64_t rows, int num_sms);
AttendPlan plan_kv_attend(int batch, int slots, int group, int kv_heads, int dim, int prefix_len, int max_ctx,
                          int window, bool eight, bool capped, int num_sms);
cudaError_t launch_kv_attend(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, int dtype, cudaStream_t s);
// Its forms, a translation unit each: what becomes of scores (kPlain to kAny) over a cache in the model's type and over an
// 8-bit one.
struct AttendForm {
  cudaError_t (*prepare)(int dtype, int dim);
  cudaError_t (*launch)(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                        int dtype, cudaStream_t s);
};
extern const AttendForm kAttendPlain, kAttendWindowed, kAttendCapped, kAttendBiased, kAttendAny;
extern const AttendForm kAttendEightPlain, kAttendEightWindowed, kAttendEightCapped, kAttendEightBiased, kAttendEightAny;

}  // namespace graft
