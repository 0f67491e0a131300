// Attention over 8-bit caches, and with capped, windowed or distance-biased
// scores: the plainest form, a CTA a row and query head, a warp a key.
//
// The online softmax keeps, per warp, the maximum m, l = sum 2^(s-m) and
// o = sum 2^(s-m) v over the keys it has seen; the warps' results are joined at
// the end.
#include "kv_internal.cuh"

namespace graft {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float number(uint8_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) k_kv_attend_plain(const __grid_constant__ AttendArgs a) {
  constexpr int kPer = D / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  grid_dependents_launch();
  grid_dependency_wait();
  const int token = blockIdx.x, head = blockIdx.y, kv_head = head / a.group, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = token / a.slots, slot = token - b * a.slots;
  const uint64_t all = a.slots == 64 ? ~0ull : (1ull << a.slots) - 1;
  const uint64_t mask = (a.tree_mask ? a.tree_mask[token] : ~0ull >> (63 - slot)) & all;
  const int ctx = min(max(a.ctx_len[b], 0), a.max_ctx);
  uint32_t bad = ctx != a.ctx_len[b] ? GRAFT_ERR_RANGE : 0;
  const float ks = a.c.eight ? kv_scale(a.k_scale, kv_head, a.err) : 1.f, vs = a.c.eight ? kv_scale(a.v_scale, kv_head, a.err) : 1.f;
  float slope = a.slope ? a.slope[head] : 0.f;
  if (!isfinite(slope)) { slope = 0.f; bad |= GRAFT_ERR_RULE; }
  const int64_t keys = (int64_t)a.prefix_len + ctx + a.slots, place = (int64_t)a.prefix_len + ctx + __popcll(mask) - 1;
  float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = Pair<T>::one(static_cast<const T*>(a.q)[token * a.q_stride + head * D + lane + 32 * i]);
    o[i] = 0.f;
  }
  for (int64_t x = warp; x < keys && mask; x += kWarps) {
    const int64_t at = x - a.prefix_len;
    const int node = (int)(at - ctx);
    int64_t key_place = x;
    if (node >= 0) {
      if (!(mask >> node & 1)) continue;
      key_place = (int64_t)a.prefix_len + ctx + __popcll(mask & ((1ull << node) - 1));
    }
    const int64_t distance = place - key_place;
    if (a.window > 0 && distance >= a.window) continue;
    const int64_t p = (at < 0 ? x : at) >> a.c.page_shift, in = (at < 0 ? x : at) & (a.c.page_size - 1);
    const int32_t page = at < 0 ? a.prefix_pages[p] : a.page_table[(int64_t)b * a.table_stride + p];
    const bool held = page >= 0 && page < a.c.num_pages;  // else zeros
    if (!held) bad |= GRAFT_ERR_RANGE;
    const int64_t from = held ? page * a.c.page_stride + kv_head * a.c.head_stride + in * a.c.token_stride + lane : 0;
    float s = 0.f, v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      float k = 0.f;
      v[i] = 0.f;
      if (held && a.c.eight) {
        k = number(static_cast<const uint8_t*>(a.k_cache)[from + 32 * i]);
        v[i] = number(static_cast<const uint8_t*>(a.v_cache)[from + 32 * i]);
      } else if (held) {
        k = Pair<T>::one(static_cast<const T*>(a.k_cache)[from + 32 * i]);
        v[i] = Pair<T>::one(static_cast<const T*>(a.v_cache)[from + 32 * i]);
      }
      s += q[i] * k;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    s *= a.scale * ks;
    if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
    s = (s - slope * (float)distance) * kLog2e;
    const float top = fmaxf(m, s), f = m == -INFINITY ? 0.f : exp2f(m - top), w = exp2f(s - top);
    m = top;
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + w * v[i];
  }
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
  for (int i = 0; i < kPer; ++i) s_o[warp][lane + 32 * i] = o[i];
  if (bad && lane == 0) atomicOr(a.err, bad);
  __syncthreads();
  if (warp != 0) return;
  float top = s_m[0], sum = 0.f;
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  float f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - top);
    sum += s_l[w] * f[w];
  }
  const float inv = sum == 0.f ? 0.f : vs / sum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (s_m[w] != -INFINITY) x += s_o[w][lane + 32 * i] * f[w];
    static_cast<T*>(a.out)[token * a.out_stride + head * D + lane + 32 * i] = Pair<T>::round(x * inv);
  }
  if (lane == 0 && a.lse) a.lse[(int64_t)token * a.c.q_heads + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

template <typename T>
cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.slots), (unsigned)a.c.q_heads);
  return launch_dependent(a.c.dim == 128 ? k_kv_attend_plain<T, 128> : k_kv_attend_plain<T, 64>, grid, dim3(kWarps * 32), 0, s, a);
}

}  // namespace

cudaError_t launch_kv_attend_ext(const AttendArgs& a, int dtype, cudaStream_t s) {
  return dtype == GRAFT_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace graft
