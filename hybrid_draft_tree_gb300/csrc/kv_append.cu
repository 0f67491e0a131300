// Appending keys and values to the paged cache, with the position rotation
// applied on the way (and to the step's queries).
//
// A token at position p turns each pair (a, b) of a rotating head's elements by
// the pair's angle: (a c - b s, b c + a s), with c and s read from the row of p
// in the caller's table, so any scaling of the angles is the caller's.
#include "kv_internal.cuh"

namespace graft {
namespace {

constexpr int kThreads = 256;

struct Token {
  int64_t k_src, q_row;  // source row of the key and value (-1: none), row of the query (-1: a pad)
  int64_t dst;           // element offset of the place's first head in the caches
  int32_t k_pos, q_pos;
};

// Where token (b, i) comes from and goes to; bad data sets the error bit and drops the write.
__device__ __forceinline__ Token locate(const AppendArgs& a, int b, int i) {
  Token t{-1, -1, 0, 0, 0};
  const int64_t first = (int64_t)b * a.slots;
  const int64_t ctx = a.ctx_len[b];
  const int64_t base = a.prefix_len + ctx;
  const int64_t limit = a.c.rot > 0 ? a.rope_len : INT64_MAX;
  uint32_t bad = ctx < 0 ? GRAFT_ERR_RANGE : 0;
  if (!bad && a.q) {
    const int32_t d = a.depth ? a.depth[first + i] : i;
    if (d >= 0) {
      if (base + d < limit) { t.q_row = first + i; t.q_pos = (int32_t)(base + d); }
      else bad = GRAFT_ERR_RANGE;
    }
  }
  const int32_t r = a.rows ? a.rows[first + i] : i;
  if (ctx >= 0 && r >= a.slots) bad = GRAFT_ERR_RANGE;
  else if (ctx >= 0 && r >= 0) {
    const int32_t d = a.depth ? a.depth[first + r] : r;
    if (d >= 0) {
      const int64_t at = ctx + i, p = at >> a.c.page_shift;
      const int32_t page = p < a.table_stride ? a.page_table[(int64_t)b * a.table_stride + p] : -1;
      if (page >= 0 && page < a.c.num_pages && base + d < limit) {
        t.k_src = first + r;
        t.k_pos = (int32_t)(base + d);
        t.dst = page * a.c.page_stride + (at & (a.c.page_size - 1)) * a.c.token_stride;
      } else {
        bad = GRAFT_ERR_RANGE;
      }
    }
  }
  if (bad && threadIdx.x == 0) atomicOr(a.err, bad);
  return t;
}

// One head in 16-byte pieces: piece u < rot / 16 of the halves form turns with
// its partner rot / 16 pieces on (two loads, two stores); of the interleaved
// form each piece turns within itself; the rest is copied.
template <typename T>
__device__ __forceinline__ void head_piece(const AppendArgs& a, const T* src, T* dst, const float* cs, int u) {
  const int half = a.c.rot >> 1;
  if (!a.c.interleaved) {
    const int pairs = half >> 3;
    if (u >= pairs) {
      const int at = (u + pairs) << 3;
      *reinterpret_cast<uint4*>(dst + at) = *reinterpret_cast<const uint4*>(src + at);
      return;
    }
    const uint4 x = *reinterpret_cast<const uint4*>(src + 8 * u);
    const uint4 y = *reinterpret_cast<const uint4*>(src + half + 8 * u);
    const float4 c0 = *reinterpret_cast<const float4*>(cs + 8 * u), c1 = *reinterpret_cast<const float4*>(cs + 8 * u + 4);
    const float4 s0 = *reinterpret_cast<const float4*>(cs + half + 8 * u);
    const float4 s1 = *reinterpret_cast<const float4*>(cs + half + 8 * u + 4);
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
    const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    uint32_t ow[4], pw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = Pair<T>::get(xw[j]), q = Pair<T>::get(yw[j]);
      ow[j] = Pair<T>::put(p.x * c[2 * j] - q.x * s[2 * j], p.y * c[2 * j + 1] - q.y * s[2 * j + 1]);
      pw[j] = Pair<T>::put(q.x * c[2 * j] + p.x * s[2 * j], q.y * c[2 * j + 1] + p.y * s[2 * j + 1]);
    }
    *reinterpret_cast<uint4*>(dst + 8 * u) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
    *reinterpret_cast<uint4*>(dst + half + 8 * u) = make_uint4(pw[0], pw[1], pw[2], pw[3]);
    return;
  }
  uint4 x = *reinterpret_cast<const uint4*>(src + 8 * u);
  if (8 * u < a.c.rot) {
    const float4 c0 = *reinterpret_cast<const float4*>(cs + 4 * u);
    const float4 s0 = *reinterpret_cast<const float4*>(cs + half + 4 * u);
    const float c[4] = {c0.x, c0.y, c0.z, c0.w}, s[4] = {s0.x, s0.y, s0.z, s0.w};
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = Pair<T>::get(w[j]);
      w[j] = Pair<T>::put(p.x * c[j] - p.y * s[j], p.y * c[j] + p.x * s[j]);
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
  }
  *reinterpret_cast<uint4*>(dst + 8 * u) = x;
}

// Any alignment and any rot_dim: one element, or one rotating pair (u < rot / 2).
template <typename T>
__device__ __forceinline__ void head_element(const AppendArgs& a, const T* src, T* dst, const float* cs, int u) {
  const int half = a.c.rot >> 1;
  if (u >= half) {
    dst[u + half] = src[u + half];
    return;
  }
  const int i = a.c.interleaved ? 2 * u : u, j = a.c.interleaved ? 2 * u + 1 : u + half;
  const float x = Pair<T>::one(src[i]), y = Pair<T>::one(src[j]), c = cs[u], s = cs[half + u];
  dst[i] = Pair<T>::round(x * c - y * s);
  dst[j] = Pair<T>::round(y * c + x * s);
}

// One CTA a token.  A lane takes one piece of one head: the heads of q, then
// those of k, then those of v.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_kv_append(AppendArgs a) {
  const int64_t n = blockIdx.x;
  const int b = (int)(n / a.slots), i = (int)(n - (int64_t)b * a.slots);
  const Token t = locate(a, b, i);
  const int dim = a.c.dim;
  // pieces of a rotating head and of a value head
  const int ru = VEC ? (a.c.interleaved ? dim >> 3 : (dim >> 3) - (a.c.rot >> 4)) : dim - (a.c.rot >> 1);
  const int vu = VEC ? dim >> 3 : dim;
  const int nq = t.q_row >= 0 ? a.c.q_heads * ru : 0;
  const int nk = t.k_src >= 0 ? a.c.kv_heads * ru : 0;
  const int nv = t.k_src >= 0 ? a.c.kv_heads * vu : 0;
  for (int w = threadIdx.x; w < nq + nk + nv; w += kThreads) {
    const T* src;
    T* dst;
    if (w < nq + nk) {
      const bool is_q = w < nq;
      const int x = is_q ? w : w - nq, head = x / ru, u = x - head * ru;
      src = is_q ? static_cast<const T*>(a.q) + t.q_row * a.q_stride + head * dim
                 : static_cast<const T*>(a.k) + t.k_src * a.k_stride + head * dim;
      dst = is_q ? static_cast<T*>(a.q_out) + t.q_row * a.q_out_stride + head * dim
                 : static_cast<T*>(a.k_cache) + t.dst + head * a.c.head_stride;
      const float* cs = a.rope + (int64_t)(is_q ? t.q_pos : t.k_pos) * a.c.rot;
      if (VEC) head_piece<T>(a, src, dst, cs, u);
      else head_element<T>(a, src, dst, cs, u);
    } else {
      const int x = w - nq - nk, head = x / vu, u = x - head * vu;
      src = static_cast<const T*>(a.v) + t.k_src * a.v_stride + head * dim;
      dst = static_cast<T*>(a.v_cache) + t.dst + head * a.c.head_stride;
      if (VEC) *reinterpret_cast<uint4*>(dst + 8 * u) = *reinterpret_cast<const uint4*>(src + 8 * u);
      else dst[u] = src[u];
    }
  }
}

template <typename T>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)((int64_t)a.batch * a.slots);
  if (a.vec) k_kv_append<T, true><<<grid, kThreads, 0, s>>>(a);
  else k_kv_append<T, false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t s) {
  return dtype == GRAFT_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace graft
