// Keys and values out of the paged cache: rows in the model's type, of 8-bit
// caches the numbers that the codes stand for (code times the head's scale, one
// rounding).
#include "kv_internal.cuh"

namespace graft {
namespace {

constexpr int kThreads = 128;

// Two e4m3 numbers as fp32: exact, they are f16 numbers.
__device__ __forceinline__ float2 numbers(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A CTA a token; a thread takes 16 bytes of the cache at a time.
template <typename T, bool EIGHT>
__global__ void __launch_bounds__(kThreads) k_kv_read(const __grid_constant__ ReadArgs a) {
  grid_dependents_launch();
  grid_dependency_wait();
  constexpr int kPer = EIGHT ? 16 : 8;  // elements of a piece
  const int64_t n = blockIdx.x;
  const int b = a.by_slots.div((int)n), i = (int)n - b * a.slots;
  const int count = a.count[b], first = a.first[b];
  uint32_t bad = count < 0 || count > a.slots || first < 0 ? GRAFT_ERR_RANGE : 0;
  int64_t src = -1;
  if (i < count && first >= 0) {
    const int64_t at = (int64_t)first + i, p = at >> a.c.page_shift;
    const int32_t page = p < a.table_stride ? a.page_table[(int64_t)b * a.table_stride + p] : -1;
    if (page >= 0 && page < a.c.num_pages) src = page * a.c.page_stride + (at & (a.c.page_size - 1)) * a.c.token_stride;
    else bad = GRAFT_ERR_RANGE;
  }
  if (bad && threadIdx.x == 0) atomicOr(a.err, bad);
  if (src < 0) return;
  const int pieces = a.c.kv_heads * (a.c.dim / kPer);
  for (int w = threadIdx.x; w < 2 * pieces; w += kThreads) {
    const bool v = w >= pieces;
    const int x = v ? w - pieces : w, head = a.by_head.div(x), u = x - head * (int)a.by_head.d;
    const int64_t from = src + head * a.c.head_stride + u * kPer;
    T* to = (v ? static_cast<T*>(a.v_out) + n * a.v_stride : static_cast<T*>(a.k_out) + n * a.k_stride) + head * a.c.dim + u * kPer;
    const uint4 got = *reinterpret_cast<const uint4*>(static_cast<const char*>(v ? a.v_cache : a.k_cache) + from * (EIGHT ? 1 : 2));
    const uint32_t in[4] = {got.x, got.y, got.z, got.w};
    uint32_t out[EIGHT ? 8 : 4];
    if (EIGHT) {
      const float s = kv_scale(v ? a.v_scale : a.k_scale, head, a.err);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 lo = numbers((uint16_t)in[j]), hi = numbers((uint16_t)(in[j] >> 16));
        out[2 * j] = Pair<T>::put(lo.x * s, lo.y * s);
        out[2 * j + 1] = Pair<T>::put(hi.x * s, hi.y * s);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) out[j] = in[j];
    }
    if (a.vec) {
#pragma unroll
      for (int j = 0; j < kPer / 2; j += 4) *reinterpret_cast<uint4*>(to + 2 * j) = make_uint4(out[j], out[j + 1], out[j + 2], out[j + 3]);
    } else {
      uint16_t* h = reinterpret_cast<uint16_t*>(to);
#pragma unroll
      for (int j = 0; j < kPer / 2; ++j) {
        h[2 * j] = (uint16_t)out[j];
        h[2 * j + 1] = (uint16_t)(out[j] >> 16);
      }
    }
  }
}

template <typename T>
cudaError_t launch(const ReadArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.batch * a.slots));
  return launch_dependent(a.c.eight ? k_kv_read<T, true> : k_kv_read<T, false>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_kv_read(const ReadArgs& a, int dtype, cudaStream_t s) {
  return dtype == GRAFT_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace graft
