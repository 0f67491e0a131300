// Attention of a step's slots over the paged cache (a shared prefix, each
// request's own context, the tree under its ancestor masks).
#include "kv_internal.cuh"

namespace graft {
namespace {

constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

// One CTA a query row and head: a thread scores one key of each 128, then one
// element of the output sums the 128 weighted values; running maximum and sum.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_kv_attend(AttendArgs a) {
  __shared__ float qs[128], ps[kThreads], red[4];
  __shared__ int64_t off[kThreads];
  const int row = blockIdx.x / a.c.q_heads, head = blockIdx.x % a.c.q_heads;
  const int b = row / a.slots, i = row % a.slots, t = threadIdx.x, dim = a.c.dim;
  int ctx = a.ctx_len[b];
  if (ctx < 0 || ctx > a.max_ctx) {
    if (t == 0) atomicOr(a.err, GRAFT_ERR_RANGE);
    ctx = ctx < 0 ? 0 : a.max_ctx;
  }
  const uint64_t mask = a.tree_mask ? a.tree_mask[row] : (i == 63 ? ~0ull : (1ull << (i + 1)) - 1);
  if (t < dim) qs[t] = Pair<T>::one(static_cast<const T*>(a.q)[row * a.q_stride + head * dim + t]);
  const int64_t keys = mask ? (int64_t)a.prefix_len + ctx + a.slots : 0;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int64_t k0 = 0; k0 < keys; k0 += kThreads) {
    __syncthreads();
    const int64_t k = k0 + t;
    float s = -INFINITY;
    off[t] = -1;
    if (k < keys) {
      const int64_t at = k < a.prefix_len ? k : k - a.prefix_len;
      const bool seen = k < a.prefix_len || at < ctx || ((mask >> (at - ctx)) & 1);
      if (seen) {
        const int32_t page = k < a.prefix_len ? a.prefix_pages[at >> a.c.page_shift]
                                              : a.page_table[(int64_t)b * a.table_stride + (at >> a.c.page_shift)];
        s = 0.f;
        if (page < 0 || page >= a.c.num_pages) {
          atomicOr(a.err, GRAFT_ERR_RANGE);
        } else {
          off[t] = page * a.c.page_stride + (at & (a.c.page_size - 1)) * a.c.token_stride +
                   head / a.group * a.c.head_stride;
          const T* kp = static_cast<const T*>(a.k_cache) + off[t];
          for (int d = 0; d < dim; ++d) s += qs[d] * Pair<T>::one(kp[d]);
        }
        s *= a.scale;
      }
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
    if ((t & 31) == 0) red[t >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float base = mx == -INFINITY ? 0.f : mx;
    ps[t] = exp2f((s - base) * kLog2e);
    __syncthreads();
    const float f = exp2f((m - base) * kLog2e);
    l *= f;
    acc *= f;
    m = mx;
    for (int j = 0; j < kThreads; ++j) {
      l += ps[j];
      if (off[j] >= 0 && t < dim) acc += ps[j] * Pair<T>::one(static_cast<const T*>(a.v_cache)[off[j] + t]);
    }
  }
  const bool none = m == -INFINITY && l == 0.f;
  if (t < dim) static_cast<T*>(a.out)[row * a.out_stride + head * dim + t] = Pair<T>::round(none ? 0.f : acc / l);
  if (t == 0 && a.lse) a.lse[(int64_t)row * a.c.q_heads + head] = none ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_kv_attend(const AttendArgs& a, int dtype, cudaStream_t s) {
  const unsigned grid = (unsigned)((int64_t)a.batch * a.slots * a.c.q_heads);
  if (dtype == GRAFT_BF16) k_kv_attend<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  else k_kv_attend<__half><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace graft
