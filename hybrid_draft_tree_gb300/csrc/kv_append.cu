// Appending keys and values to the paged cache, with the position rotation
// applied on the way (and to the step's queries).
//
// A token at position p turns each pair (a, b) of a rotating head's elements by
// the pair's angle: (a c - b s, b c + a s), with c and s read from the row of p
// in the caller's table, so any scaling of the angles is the caller's.
//
// A CTA a token, 128 threads, two 16-byte pieces (and their partners) a thread in
// flight; the source rows are on their way before the page table has answered.
// Bound by memory when there are many tokens (1 x 32768, 32/8 heads of 128: 127
// us, 6.4 TB/s, 95% of the copy rate; every element is read and written once), by
// the latency of launch, page table and row when there are few (16 x 61: 6.5 us,
// 3.7 TB/s; one token: 3.0 us).  256 threads or three pieces a thread were no
// faster.
#include "kv_internal.cuh"

namespace graft {
namespace {

constexpr int kThreads = 128;

// Where token (b, i) comes from and goes to.  Its source rows are known before its place: their loads do not wait for
// the page table.  Bad data sets the error bit and drops the write.
struct Token {
  int64_t dst;           // element offset of the place's first head in the caches
  int32_t k_pos, q_pos;  // positions, -1: no key and value to write, no query
};

__device__ __forceinline__ Token locate(const AppendArgs& a, int b, int i, int r) {
  Token t{0, -1, -1};
  const int64_t first = (int64_t)b * a.slots;
  const int64_t ctx = a.ctx_len[b];
  const int64_t base = a.prefix_len + ctx;
  const int64_t limit = a.c.rot > 0 ? a.rope_len : INT32_MAX;
  uint32_t bad = ctx < 0 || r >= a.slots ? GRAFT_ERR_RANGE : 0;
  if (ctx >= 0 && a.q) {
    const int32_t d = a.depth ? a.depth[first + i] : i;
    if (d >= 0 && base + d >= limit) bad = GRAFT_ERR_RANGE;
    else if (d >= 0) t.q_pos = (int32_t)(base + d);
  }
  if (ctx >= 0 && r >= 0 && r < a.slots) {
    const int32_t d = a.depth ? a.depth[first + r] : r;
    if (d >= 0) {
      const int64_t at = ctx + i, p = at >> a.c.page_shift;
      const int32_t page = p < a.table_stride ? a.page_table[(int64_t)b * a.table_stride + p] : -1;
      if (page >= 0 && page < a.c.num_pages && base + d < limit) {
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

// 16-byte pieces of a head.  Halves form: piece u < rot / 16 turns with its partner rot / 16 pieces on; interleaved form:
// a piece turns within itself; the rest is copied.  x: the piece, y: its partner.
template <typename T>
__device__ __forceinline__ void turn_halves(const float* cs, int half, int u, uint4& x, uint4& y) {
  const float4 c0 = *reinterpret_cast<const float4*>(cs + 8 * u), c1 = *reinterpret_cast<const float4*>(cs + 8 * u + 4);
  const float4 s0 = *reinterpret_cast<const float4*>(cs + half + 8 * u);
  const float4 s1 = *reinterpret_cast<const float4*>(cs + half + 8 * u + 4);
  uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
  const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = Pair<T>::get(xw[j]), q = Pair<T>::get(yw[j]);
    xw[j] = Pair<T>::put(p.x * c[2 * j] - q.x * s[2 * j], p.y * c[2 * j + 1] - q.y * s[2 * j + 1]);
    yw[j] = Pair<T>::put(q.x * c[2 * j] + p.x * s[2 * j], q.y * c[2 * j + 1] + p.y * s[2 * j + 1]);
  }
  x = make_uint4(xw[0], xw[1], xw[2], xw[3]);
  y = make_uint4(yw[0], yw[1], yw[2], yw[3]);
}
template <typename T>
__device__ __forceinline__ void turn_pairs(const float* cs, int half, int u, uint4& x) {
  const float4 c0 = *reinterpret_cast<const float4*>(cs + 4 * u), s0 = *reinterpret_cast<const float4*>(cs + half + 4 * u);
  const float c[4] = {c0.x, c0.y, c0.z, c0.w}, s[4] = {s0.x, s0.y, s0.z, s0.w};
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = Pair<T>::get(w[j]);
    w[j] = Pair<T>::put(p.x * c[j] - p.y * s[j], p.y * c[j] + p.x * s[j]);
  }
  x = make_uint4(w[0], w[1], w[2], w[3]);
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

// One CTA a token.  A thread takes pieces of heads: those of q, of k and of v, in turn.
template <typename T, bool HALVES>
__global__ void __launch_bounds__(kThreads) k_kv_append(AppendArgs a) {
  grid_dependents_launch();
  grid_dependency_wait();
  const int64_t n = blockIdx.x;
  const int b = a.by_slots.div((int)n), i = (int)n - b * a.slots, dim = a.c.dim;
  const int r = a.rows ? a.rows[n] : i;
  const int half = a.c.rot >> 1, pairs = HALVES ? half >> 3 : 0;
  const int ru = (dim >> 3) - pairs, vu = dim >> 3;  // pieces of a rotating head, each with its partner, and of a value head
  const bool has_k = r >= 0 && r < a.slots;
  const int nq = a.q ? a.c.q_heads * ru : 0, nk = has_k ? a.c.kv_heads * ru : 0, nv = has_k ? a.c.kv_heads * vu : 0;
  const int64_t k_row = (int64_t)b * a.slots + r;
  constexpr int kPer = 2;  // pieces in flight
  Token t;
  bool located = false;
  for (int w0 = threadIdx.x; w0 < nq + nk + nv || !located; w0 += kPer * kThreads) {
    uint4 x[kPer], y[kPer];
    int kind[kPer], head[kPer], u[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      int w = w0 + j * kThreads;
      kind[j] = w < nq ? 0 : w < nq + nk ? 1 : w < nq + nk + nv ? 2 : 3;
      if (kind[j] == 3) continue;
      const Divisor& by = kind[j] == 2 ? a.by_value : a.by_turn;
      w -= kind[j] == 0 ? 0 : kind[j] == 1 ? nq : nq + nk;
      head[j] = by.div(w);
      u[j] = w - head[j] * (int)by.d;
      const T* src = kind[j] == 0 ? static_cast<const T*>(a.q) + n * a.q_stride
                                  : kind[j] == 1 ? static_cast<const T*>(a.k) + k_row * a.k_stride : static_cast<const T*>(a.v) + k_row * a.v_stride;
      src += head[j] * dim;
      const int at = HALVES && kind[j] < 2 && u[j] >= pairs ? u[j] + pairs : u[j];
      x[j] = __ldcs(reinterpret_cast<const uint4*>(src) + at);
      if (HALVES && kind[j] < 2 && u[j] < pairs) y[j] = __ldcs(reinterpret_cast<const uint4*>(src) + u[j] + pairs);
    }
    if (!located) {
      t = locate(a, b, i, r);
      located = true;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (kind[j] == 3 || (kind[j] == 0 ? t.q_pos : t.k_pos) < 0) continue;
      T* dst = kind[j] == 0 ? static_cast<T*>(a.q_out) + n * a.q_out_stride + head[j] * dim
                            : static_cast<T*>(kind[j] == 1 ? a.k_cache : a.v_cache) + t.dst + head[j] * a.c.head_stride;
      uint4* out = reinterpret_cast<uint4*>(dst);
      if (kind[j] == 2) {
        out[u[j]] = x[j];
        continue;
      }
      const float* cs = a.rope + (int64_t)(kind[j] == 0 ? t.q_pos : t.k_pos) * a.c.rot;
      if (HALVES) {
        if (u[j] < pairs) {
          turn_halves<T>(cs, half, u[j], x[j], y[j]);
          out[u[j]] = x[j];
          out[u[j] + pairs] = y[j];
        } else {
          out[u[j] + pairs] = x[j];
        }
      } else {
        if (8 * u[j] < a.c.rot) turn_pairs<T>(cs, half, u[j], x[j]);
        out[u[j]] = x[j];
      }
    }
  }
}

// The same by elements and rotating pairs, for any alignment and any rot_dim.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_kv_append_elements(AppendArgs a) {
  grid_dependents_launch();
  grid_dependency_wait();
  const int64_t n = blockIdx.x;
  const int b = a.by_slots.div((int)n), i = (int)n - b * a.slots, dim = a.c.dim;
  const int r = a.rows ? a.rows[n] : i;
  const Token t = locate(a, b, i, r);
  const int64_t k_row = (int64_t)b * a.slots + r;
  const int ru = dim - (a.c.rot >> 1);
  const int nq = t.q_pos >= 0 ? a.c.q_heads * ru : 0, nk = t.k_pos >= 0 ? a.c.kv_heads * ru : 0;
  const int nv = t.k_pos >= 0 ? a.c.kv_heads * dim : 0;
  for (int w = threadIdx.x; w < nq + nk + nv; w += kThreads) {
    if (w < nq + nk) {
      const bool is_q = w < nq;
      const int x = is_q ? w : w - nq, head = x / ru, u = x - head * ru;
      const T* src = is_q ? static_cast<const T*>(a.q) + n * a.q_stride + head * dim
                          : static_cast<const T*>(a.k) + k_row * a.k_stride + head * dim;
      T* dst = is_q ? static_cast<T*>(a.q_out) + n * a.q_out_stride + head * dim
                    : static_cast<T*>(a.k_cache) + t.dst + head * a.c.head_stride;
      head_element<T>(a, src, dst, a.rope + (int64_t)(is_q ? t.q_pos : t.k_pos) * a.c.rot, u);
    } else {
      const int x = w - nq - nk, head = x / dim, u = x - head * dim;
      static_cast<T*>(a.v_cache)[t.dst + head * a.c.head_stride + u] = static_cast<const T*>(a.v)[k_row * a.v_stride + head * dim + u];
    }
  }
}

template <typename T>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.batch * a.slots));
  if (!a.vec) return launch_dependent(k_kv_append_elements<T>, grid, dim3(kThreads), 0, s, a);
  return launch_dependent(a.c.interleaved ? k_kv_append<T, false> : k_kv_append<T, true>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t s) {
  return dtype == GRAFT_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace graft
