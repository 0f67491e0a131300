// Keys and values out of the paged cache: rows in the model's type, of 8-bit
// caches the numbers that the codes stand for (code times the head's scale, in
// fp32, then rounded to the type).  Bound by memory: 1 x 32768, 8 heads of 128, 33.4 us, 6.0 TB/s, 89%
// of the copy rate.
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

// A CTA takes N tokens in a row, a thread the same 16 bytes of each: their loads are under way together (1 x 32768 of 8
// bits: 33.4 us with two tokens, 41 with one, 37 with four, 46 with eight; 64 x 61: 6.3 us with one or two).
template <typename T, bool EIGHT, int N>
__global__ void __launch_bounds__(kThreads) k_kv_read(const __grid_constant__ ReadArgs a) {
  grid_dependents_launch();
  grid_dependency_wait();
  constexpr int kPer = EIGHT ? 16 : 8;  // elements of a piece
  const int64_t n0 = (int64_t)blockIdx.x * N, tokens = (int64_t)a.batch * a.slots;
  int64_t src[N];
  uint32_t bad = 0;
#pragma unroll
  for (int x = 0; x < N; ++x) {
    src[x] = -1;
    if (n0 + x >= tokens) continue;
    const int b = a.by_slots.div((int)(n0 + x)), i = (int)(n0 + x) - b * a.slots;
    const int count = a.count[b], first = a.first[b];
    if (count < 0 || count > a.slots || first < 0) bad = GRAFT_ERR_RANGE;
    if (i >= count || first < 0) continue;
    const int64_t at = (int64_t)first + i, p = at >> a.c.page_shift;
    const int32_t page = p < a.table_stride ? a.page_table[(int64_t)b * a.table_stride + p] : -1;
    if (page >= 0 && page < a.c.num_pages) src[x] = page * a.c.page_stride + (at & (a.c.page_size - 1)) * a.c.token_stride;
    else bad = GRAFT_ERR_RANGE;
  }
  if (bad && threadIdx.x == 0) atomicOr(a.err, bad);
  const int pieces = a.c.kv_heads * (a.c.dim / kPer);
  for (int w = threadIdx.x; w < 2 * pieces; w += kThreads) {
    const bool v = w >= pieces;
    const int y = v ? w - pieces : w, head = a.by_head.div(y), u = y - head * (int)a.by_head.d;
    const char* from = static_cast<const char*>(v ? a.v_cache : a.k_cache) + (head * a.c.head_stride + u * kPer) * (EIGHT ? 1 : 2);
    T* to = (v ? static_cast<T*>(a.v_out) + n0 * a.v_stride : static_cast<T*>(a.k_out) + n0 * a.k_stride) + head * a.c.dim + u * kPer;
    const int64_t step = v ? a.v_stride : a.k_stride;
    uint4 got[N];
#pragma unroll
    for (int x = 0; x < N; ++x)
      if (src[x] >= 0) got[x] = __ldcs(reinterpret_cast<const uint4*>(from + src[x] * (EIGHT ? 1 : 2)));
    const float s = EIGHT ? kv_scale(v ? a.v_scale : a.k_scale, head, a.err) : 1.f;
#pragma unroll
    for (int x = 0; x < N; ++x, to += step) {
      if (src[x] < 0) continue;
      const uint32_t in[4] = {got[x].x, got[x].y, got[x].z, got[x].w};
      uint32_t out[EIGHT ? 8 : 4];
      if (EIGHT) {
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
}

template <typename T, bool EIGHT>
cudaError_t launch(const ReadArgs& a, cudaStream_t s) {
  const int64_t tokens = (int64_t)a.batch * a.slots;
  return launch_dependent(k_kv_read<T, EIGHT, 2>, dim3((unsigned)((tokens + 1) / 2)), dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_kv_read(const ReadArgs& a, int dtype, cudaStream_t s) {
  if (a.c.eight) return dtype == GRAFT_BF16 ? launch<__nv_bfloat16, true>(a, s) : launch<__half, true>(a, s);
  return dtype == GRAFT_BF16 ? launch<__nv_bfloat16, false>(a, s) : launch<__half, false>(a, s);
}

}  // namespace graft
