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

template <bool EXT>
__device__ __forceinline__ Token locate(const AppendArgs& a, int b, int i, int r) {
  Token t{0, -1, -1};
  const int64_t first = (int64_t)b * a.slots;
  const int64_t ctx = a.ctx_len[b];
  const int64_t base = a.prefix_len + ctx;
  const int64_t limit = a.c.rot > 0 ? a.rope_len : INT32_MAX;
  // positions of the caller's take the place of base + depth, all axes inside the table of angles
  const bool given = EXT && a.position && a.c.rot > 0;
  auto inside = [&](int64_t row, int64_t pos) {
    if (!given) return pos < limit;
    bool in = true;
    for (int x = 0; x < a.axes; ++x) in = in && (uint32_t)a.position[x * a.tokens + row] < (uint32_t)a.rope_len;
    return in;
  };
  uint32_t bad = ctx < 0 || r >= a.slots ? GRAFT_ERR_RANGE : 0;
  if (ctx >= 0 && a.q) {
    const int32_t d = a.depth ? a.depth[first + i] : i;
    if (d >= 0 && !inside(first + i, base + d)) bad = GRAFT_ERR_RANGE;
    else if (d >= 0) t.q_pos = given ? 0 : (int32_t)(base + d);
  }
  if (ctx >= 0 && r >= 0 && r < a.slots) {
    const int32_t d = a.depth ? a.depth[first + r] : r;
    if (d >= 0) {
      const int64_t at = ctx + i, p = at >> a.c.page_shift;
      const int32_t page = p < a.table_stride ? a.page_table[(int64_t)b * a.table_stride + p] : -1;
      if (page >= 0 && page < a.c.num_pages && inside(first + r, base + d)) {
        t.k_pos = given ? 0 : (int32_t)(base + d);
        t.dst = page * a.c.page_stride + (at & (a.c.page_size - 1)) * a.c.token_stride;
      } else {
        bad = GRAFT_ERR_RANGE;
      }
    }
  }
  if (bad && threadIdx.x == 0) atomicOr(a.err, bad);
  return t;
}

// Cosines and sines of N pairs from p on: of one row of the table, or, with positions of several axes, of the row of each
// pair's own position (`row`: the token that has them).  Pairs of one axis take the same loads as without axes.
template <int N, bool EXT>
__device__ __forceinline__ void angles(const AppendArgs& a, int pos, int64_t row, int p, float* c, float* s) {
  const int half = a.c.rot >> 1;
  if (EXT && a.position) {
    int axis = a.pair_axis[p];
    bool one = true;
#pragma unroll
    for (int j = 1; j < N; ++j) one = one && a.pair_axis[p + j] == axis;
    if (!one) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float* cs = a.rope + (int64_t)a.position[a.pair_axis[p + j] * a.tokens + row] * a.c.rot + p + j;
        c[j] = cs[0];
        s[j] = cs[half];
      }
      return;
    }
    pos = a.position[axis * a.tokens + row];
  }
  const float* cs = a.rope + (int64_t)pos * a.c.rot + p;
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    const float4 x = *reinterpret_cast<const float4*>(cs + j), y = *reinterpret_cast<const float4*>(cs + half + j);
    c[j] = x.x; c[j + 1] = x.y; c[j + 2] = x.z; c[j + 3] = x.w;
    s[j] = y.x; s[j + 1] = y.y; s[j + 2] = y.z; s[j + 3] = y.w;
  }
}

// 16-byte pieces of a head.  Halves form: piece u < rot / 16 turns with its partner rot / 16 pieces on; interleaved form:
// a piece turns within itself; the rest is copied.  x: the piece, y: its partner, as 8 fp32 numbers.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float* f) {
  const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = Pair<T>::get(e[j]);
    f[2 * j] = p.x;
    f[2 * j + 1] = p.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float* f) {
  return make_uint4(Pair<T>::put(f[0], f[1]), Pair<T>::put(f[2], f[3]), Pair<T>::put(f[4], f[5]), Pair<T>::put(f[6], f[7]));
}
__device__ __forceinline__ void turn_halves(const float* c, const float* s, float* x, float* y) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float p = x[j], q = y[j];
    x[j] = p * c[j] - q * s[j];
    y[j] = q * c[j] + p * s[j];
  }
}
__device__ __forceinline__ void turn_pairs(const float* c, const float* s, float* x) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float p = x[2 * j], q = x[2 * j + 1];
    x[2 * j] = p * c[j] - q * s[j];
    x[2 * j + 1] = q * c[j] + p * s[j];
  }
}

// 8-bit caches: numbers over the head's scale, to the nearest e4m3 number (ties to even), at most 448 in magnitude.  The
// quotient is a division, so that what is stored follows from the definition bit for bit; 1 x 32768 is as fast with a
// product.
__device__ __forceinline__ uint32_t codes(const float* f, float scale) {  // four, in their order
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(__fdiv_rn(f[1], scale)), "f"(__fdiv_rn(f[0], scale)));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(__fdiv_rn(f[3], scale)), "f"(__fdiv_rn(f[2], scale)));
  return (uint32_t)hi << 16 | lo;
}
__device__ __forceinline__ uint8_t code(float x, float scale) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.f), "f"(__fdiv_rn(x, scale)));
  return (uint8_t)c;
}

// Any alignment and any rot_dim: one element, or one rotating pair (u < rot / 2).
template <typename T, bool EXT, typename Put>
__device__ __forceinline__ void head_element(const AppendArgs& a, const T* src, int pos, int64_t row, int u, Put put) {
  const int half = a.c.rot >> 1;
  if (u >= half) {
    put(u + half, Pair<T>::one(src[u + half]));
    return;
  }
  if (EXT && a.position) pos = a.position[a.pair_axis[u] * a.tokens + row];
  const float* cs = a.rope + (int64_t)pos * a.c.rot;
  const int i = a.c.interleaved ? 2 * u : u, j = a.c.interleaved ? 2 * u + 1 : u + half;
  const float x = Pair<T>::one(src[i]), y = Pair<T>::one(src[j]), c = cs[u], s = cs[half + u];
  put(i, x * c - y * s);
  put(j, y * c + x * s);
}

// One CTA a token.  A thread takes pieces of heads: those of q, of k and of v, in turn.
template <typename T, bool HALVES, bool EXT>
__global__ void __launch_bounds__(kThreads) k_kv_append(const __grid_constant__ AppendArgs a) {
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
      t = locate<EXT>(a, b, i, r);
      located = true;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (kind[j] == 3 || (kind[j] == 0 ? t.q_pos : t.k_pos) < 0) continue;
      const bool eight = EXT && a.c.eight && kind[j] != 0;
      const int64_t to = kind[j] == 0 ? n * a.q_out_stride + head[j] * dim : t.dst + head[j] * a.c.head_stride;
      void* base = kind[j] == 0 ? a.q_out : kind[j] == 1 ? a.k_cache : a.v_cache;
      const float scale = eight ? kv_scale(kind[j] == 1 ? a.k_scale : a.v_scale, head[j], a.err) : 1.f;
      auto put = [&](int piece, const float* f) {
        if (eight) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + to + 8 * piece) = make_uint2(codes(f, scale), codes(f + 4, scale));
        else *reinterpret_cast<uint4*>(static_cast<T*>(base) + to + 8 * piece) = pack<T>(f);
      };
      auto keep = [&](int piece, const uint4& w) {  // as it is
        if (eight) {
          float f[8];
          unpack<T>(w, f);
          put(piece, f);
        } else {
          *reinterpret_cast<uint4*>(static_cast<T*>(base) + to + 8 * piece) = w;
        }
      };
      if (kind[j] == 2) {
        keep(u[j], x[j]);
        continue;
      }
      const int pos = kind[j] == 0 ? t.q_pos : t.k_pos;
      const int64_t row = kind[j] == 0 ? n : k_row;
      float f[8], g[8], c[8], s[8];
      if (HALVES) {
        if (u[j] < pairs) {
          angles<8, EXT>(a, pos, row, 8 * u[j], c, s);
          unpack<T>(x[j], f);
          unpack<T>(y[j], g);
          turn_halves(c, s, f, g);
          put(u[j], f);
          put(u[j] + pairs, g);
        } else {
          keep(u[j] + pairs, x[j]);
        }
      } else if (8 * u[j] < a.c.rot) {
        angles<4, EXT>(a, pos, row, 4 * u[j], c, s);
        unpack<T>(x[j], f);
        turn_pairs(c, s, f);
        put(u[j], f);
      } else {
        keep(u[j], x[j]);
      }
    }
  }
}

// The same by elements and rotating pairs, for any alignment and any rot_dim.
template <typename T, bool EXT>
__global__ void __launch_bounds__(kThreads) k_kv_append_elements(const __grid_constant__ AppendArgs a) {
  grid_dependents_launch();
  grid_dependency_wait();
  const int64_t n = blockIdx.x;
  const int b = a.by_slots.div((int)n), i = (int)n - b * a.slots, dim = a.c.dim;
  const int r = a.rows ? a.rows[n] : i;
  const Token t = locate<EXT>(a, b, i, r);
  const int64_t k_row = (int64_t)b * a.slots + r;
  const int ru = dim - (a.c.rot >> 1);
  const int nq = t.q_pos >= 0 ? a.c.q_heads * ru : 0, nk = t.k_pos >= 0 ? a.c.kv_heads * ru : 0;
  const int nv = t.k_pos >= 0 ? a.c.kv_heads * dim : 0;
  for (int w = threadIdx.x; w < nq + nk + nv; w += kThreads) {
    const bool is_q = w < nq, is_v = w >= nq + nk;
    const int x = is_q ? w : is_v ? w - nq - nk : w - nq, head = x / (is_v ? dim : ru), u = x - head * (is_v ? dim : ru);
    const int64_t to = is_q ? n * a.q_out_stride + head * dim : t.dst + head * a.c.head_stride;
    void* base = is_q ? a.q_out : is_v ? a.v_cache : a.k_cache;
    const bool eight = EXT && a.c.eight && !is_q;
    const float scale = eight ? kv_scale(is_v ? a.v_scale : a.k_scale, head, a.err) : 1.f;
    auto put = [&](int at, float f) {
      if (eight) static_cast<uint8_t*>(base)[to + at] = code(f, scale);
      else static_cast<T*>(base)[to + at] = Pair<T>::round(f);
    };
    if (is_v) {
      const T v = static_cast<const T*>(a.v)[k_row * a.v_stride + head * dim + u];
      if (eight) put(u, Pair<T>::one(v));
      else static_cast<T*>(base)[to + u] = v;
    } else {
      const T* src = is_q ? static_cast<const T*>(a.q) + n * a.q_stride + head * dim
                          : static_cast<const T*>(a.k) + k_row * a.k_stride + head * dim;
      head_element<T, EXT>(a, src, is_q ? t.q_pos : t.k_pos, is_q ? n : k_row, u, put);
    }
  }
}

template <typename T, bool EXT>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.batch * a.slots));
  if (!a.vec) return launch_dependent(k_kv_append_elements<T, EXT>, grid, dim3(kThreads), 0, s, a);
  return launch_dependent(a.c.interleaved ? k_kv_append<T, false, EXT> : k_kv_append<T, true, EXT>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t s) {
  if (a.c.eight || a.position) return dtype == GRAFT_BF16 ? launch<__nv_bfloat16, true>(a, s) : launch<__half, true>(a, s);
  return dtype == GRAFT_BF16 ? launch<__nv_bfloat16, false>(a, s) : launch<__half, false>(a, s);
}

}  // namespace graft
