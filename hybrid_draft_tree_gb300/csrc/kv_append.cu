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
//
// Into an 8-bit cache keys and values are rounded to e4m3 over their head's
// scale on the way; with positions of several axes each pair turns by the angle
// of its own axis' position, which the CTA reads and judges once.  Bound by
// instructions then: 1 x 32768 in 8 bits 138 us (5.5 TB/s), three axes in 16 bits
// 145 us, both 158; 16 x 61 with both 8 us.
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

// Positions of the caller's, of the query's token and of the key's: read once by the CTA, which takes one verdict on them.
struct Given { int32_t q[8], k[8]; };
__device__ __forceinline__ uint32_t read_given(const AppendArgs& a, int64_t q_row, int64_t k_row, bool has_k, Given& s) {
  const int x = threadIdx.x;
  bool q_in = true, k_in = true;
  if (x < a.axes) {
    s.q[x] = a.position[x * a.tokens + q_row];
    q_in = (uint32_t)s.q[x] < (uint32_t)a.rope_len;
  } else if (x >= 8 && x < 8 + a.axes && has_k) {
    s.k[x - 8] = a.position[(x - 8) * a.tokens + k_row];
    k_in = (uint32_t)s.k[x - 8] < (uint32_t)a.rope_len;
  }
  const bool all_q = __syncthreads_and(q_in), all_k = __syncthreads_and(k_in);
  return (uint32_t)all_q | (uint32_t)all_k << 1;
}

// GIVEN: `given` is the verdict on positions of the caller's, which take the place of base + depth.
template <bool GIVEN>
__device__ __forceinline__ Token locate(const AppendArgs& a, int b, int i, int r, uint32_t given = 0) {
  Token t{0, -1, -1};
  const int64_t first = (int64_t)b * a.slots;
  const int64_t ctx = a.ctx_len[b];
  const int64_t base = a.prefix_len + ctx;
  const int64_t limit = a.c.rot > 0 ? a.rope_len : INT32_MAX;
  uint32_t bad = ctx < 0 || r >= a.slots ? GRAFT_ERR_RANGE : 0;
  if (ctx >= 0 && a.q) {
    const int32_t d = a.depth ? a.depth[first + i] : i;
    if (d >= 0 && (GIVEN ? !(given & 1) : base + d >= limit)) bad = GRAFT_ERR_RANGE;
    else if (d >= 0) t.q_pos = GIVEN ? 0 : (int32_t)(base + d);
  }
  if (ctx >= 0 && r >= 0 && r < a.slots) {
    const int32_t d = a.depth ? a.depth[first + r] : r;
    if (d >= 0) {
      const int64_t at = ctx + i, p = at >> a.c.page_shift;
      const int32_t page = p < a.table_stride ? a.page_table[(int64_t)b * a.table_stride + p] : -1;
      if (page >= 0 && page < a.c.num_pages && (GIVEN ? (given & 2) != 0 : base + d < limit)) {
        t.k_pos = GIVEN ? 0 : (int32_t)(base + d);
        t.dst = page * a.c.page_stride + (at & (a.c.page_size - 1)) * a.c.token_stride;
      } else {
        bad = GRAFT_ERR_RANGE;
      }
    }
  }
  if (bad && threadIdx.x == 0) atomicOr(a.err, bad);
  return t;
}

// Cosines and sines of the N pairs of piece u: of one row of the table, or, with pairs of several axes in the piece, of the
// row of each pair's own position.
template <int N, bool AXES>
__device__ __forceinline__ void angles(const AppendArgs& a, int pos, const int32_t* given, int u, float* c, float* s) {
  const int half = a.c.rot >> 1;
  if (AXES) {
    const int axis = (int)(a.piece_axis >> 4 * u) & 15;
    if (axis == kMixed) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float* cs = a.rope + (int64_t)given[a.pair_axis[N * u + j]] * a.c.rot + N * u + j;
        c[j] = cs[0];
        s[j] = cs[half];
      }
      return;
    }
    pos = given[axis];
  }
  const float* cs = a.rope + (int64_t)pos * a.c.rot + N * u;
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
// quotient is the correctly rounded one, so that what is stored follows from the definition bit for bit: with a correctly
// rounded reciprocal a product is within an ulp of it, and q + (x - q scale) / scale from there is it (Markstein).  All of
// that stays inside fp32 for scales from 2^-60 to 2^64 and quotients below 2^10, above which the result is 448 whatever the
// last bit; other scales get there by a power of two, with x.  (1 x 32768: 160 us with a division for each.)
struct Quotient {
  float up, scale, inverse;
  __device__ __forceinline__ explicit Quotient(float s) {
    up = s < 0x1p-60f ? 0x1p100f : s > 0x1p60f ? 0x1p-64f : 1.f;
    scale = s * up;
    inverse = 1.f / scale;
  }
  __device__ __forceinline__ float operator()(float x) const {
    x *= up;
    const float q = x * inverse;
    // a zero keeps its sign
    return fabsf(q) < 1024.f && q != 0.f ? fmaf(fmaf(-q, scale, x), inverse, q) : q;
  }
};
__device__ __forceinline__ uint32_t codes(const float* f, const Quotient& by) {  // four, in their order
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(by(f[1])), "f"(by(f[0])));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(by(f[3])), "f"(by(f[2])));
  return (uint32_t)hi << 16 | lo;
}
__device__ __forceinline__ uint8_t code(float x, const Quotient& by) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.f), "f"(by(x)));
  return (uint8_t)c;
}

// Any alignment and any rot_dim: one element, or one rotating pair (u < rot / 2).
template <typename T, bool AXES, typename Put>
__device__ __forceinline__ void head_element(const AppendArgs& a, const T* src, int pos, const int32_t* given, int u, Put put) {
  const int half = a.c.rot >> 1;
  if (u >= half) {
    put(u + half, Pair<T>::one(src[u + half]));
    return;
  }
  if (AXES) pos = given[a.pair_axis[u]];
  const float* cs = a.rope + (int64_t)pos * a.c.rot;
  const int i = a.c.interleaved ? 2 * u : u, j = a.c.interleaved ? 2 * u + 1 : u + half;
  const float x = Pair<T>::one(src[i]), y = Pair<T>::one(src[j]), c = cs[u], s = cs[half + u];
  put(i, x * c - y * s);
  put(j, y * c + x * s);
}

// One CTA a token.  A thread takes pieces of heads: those of q, of k and of v, in turn.
// Into an 8-bit cache, by positions of several axes, or both: more to compute and to hold, so eight CTAs an SM, or registers
// leave seven (1 x 32768 in 8 bits 138 us, 144 then).
template <typename T, bool HALVES, bool EIGHT, bool AXES>
__global__ void __launch_bounds__(kThreads, 8) k_kv_append_ext(const __grid_constant__ AppendArgs a) {
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
  __shared__ Given s_given;
  Token t;
  bool located = false;
  for (int w0 = threadIdx.x; w0 < nq + nk + nv || !located; w0 += kPer * kThreads) {
    uint4 x[kPer], y[kPer];
    int kind[kPer], head[kPer], u[kPer];
    float scale[kPer];
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
      if (EIGHT && kind[j] != 0) {  // the head's scale, on its way with the rows
        const float* of = kind[j] == 1 ? a.k_scale : a.v_scale;
        scale[j] = of ? of[head[j]] : 1.f;
      }
    }
    if (!located) {
      t = AXES ? locate<true>(a, b, i, r, read_given(a, n, k_row, has_k, s_given)) : locate<false>(a, b, i, r);
      located = true;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (kind[j] == 3 || (kind[j] == 0 ? t.q_pos : t.k_pos) < 0) continue;
      const int64_t to = kind[j] == 0 ? n * a.q_out_stride + head[j] * dim : t.dst + head[j] * a.c.head_stride;
      const int pos = kind[j] == 0 ? t.q_pos : t.k_pos;
      const int32_t* given = kind[j] == 0 ? s_given.q : s_given.k;
      float f[8], g[8], c[8], s[8];
      if (EIGHT && kind[j] != 0) {
        const Quotient by(checked_scale(scale[j], a.err));
        uint8_t* base = static_cast<uint8_t*>(kind[j] == 1 ? a.k_cache : a.v_cache) + to;
        auto put = [&](int piece, const float* f) { *reinterpret_cast<uint2*>(base + 8 * piece) = make_uint2(codes(f, by), codes(f + 4, by)); };
        unpack<T>(x[j], f);
        int at = u[j];
        if (kind[j] == 1 && HALVES) {
          if (u[j] < pairs) {
            angles<8, AXES>(a, pos, given, u[j], c, s);
            unpack<T>(y[j], g);
            turn_halves(c, s, f, g);
            put(u[j] + pairs, g);
          } else {
            at += pairs;
          }
        } else if (kind[j] == 1 && 8 * u[j] < a.c.rot) {
          angles<4, AXES>(a, pos, given, u[j], c, s);
          turn_pairs(c, s, f);
        }
        put(at, f);
        continue;
      }
      uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(kind[j] == 0 ? a.q_out : kind[j] == 1 ? a.k_cache : a.v_cache) + to);
      if (kind[j] == 2) {
        out[u[j]] = x[j];
      } else if (HALVES) {
        if (u[j] < pairs) {
          angles<8, AXES>(a, pos, given, u[j], c, s);
          unpack<T>(x[j], f);
          unpack<T>(y[j], g);
          turn_halves(c, s, f, g);
          out[u[j]] = pack<T>(f);
          out[u[j] + pairs] = pack<T>(g);
        } else {
          out[u[j] + pairs] = x[j];
        }
      } else {
        if (8 * u[j] < a.c.rot) {
          angles<4, AXES>(a, pos, given, u[j], c, s);
          unpack<T>(x[j], f);
          turn_pairs(c, s, f);
          x[j] = pack<T>(f);
        }
        out[u[j]] = x[j];
      }
    }
  }
}

// The same on pieces as they come, from the angles' row.
template <typename T>
__device__ __forceinline__ void turn_packed_halves(const float* cs, int half, int u, uint4& x, uint4& y) {
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
__device__ __forceinline__ void turn_packed_pairs(const float* cs, int half, int u, uint4& x) {
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

// Into a cache in the model's type, by the one position of a token: a kernel with a body of its own (1 x 32768: 127 us; as an
// instance of the body above 131).
template <typename T, bool HALVES>
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
      t = locate<false>(a, b, i, r);
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
          turn_packed_halves<T>(cs, half, u[j], x[j], y[j]);
          out[u[j]] = x[j];
          out[u[j] + pairs] = y[j];
        } else {
          out[u[j] + pairs] = x[j];
        }
      } else {
        if (8 * u[j] < a.c.rot) turn_packed_pairs<T>(cs, half, u[j], x[j]);
        out[u[j]] = x[j];
      }
    }
  }
}
// Both by elements and rotating pairs, for any alignment and any rot_dim.
template <typename T, bool EIGHT, bool AXES>
__global__ void __launch_bounds__(kThreads) k_kv_append_elements(const __grid_constant__ AppendArgs a) {
  grid_dependents_launch();
  grid_dependency_wait();
  const int64_t n = blockIdx.x;
  const int b = a.by_slots.div((int)n), i = (int)n - b * a.slots, dim = a.c.dim;
  const int r = a.rows ? a.rows[n] : i;
  const int64_t k_row = (int64_t)b * a.slots + r;
  __shared__ Given s_given;
  const Token t = AXES ? locate<true>(a, b, i, r, read_given(a, n, k_row, r >= 0 && r < a.slots, s_given)) : locate<false>(a, b, i, r);
  const int ru = dim - (a.c.rot >> 1);
  const int nq = t.q_pos >= 0 ? a.c.q_heads * ru : 0, nk = t.k_pos >= 0 ? a.c.kv_heads * ru : 0;
  const int nv = t.k_pos >= 0 ? a.c.kv_heads * dim : 0;
  for (int w = threadIdx.x; w < nq + nk + nv; w += kThreads) {
    const bool is_q = w < nq, is_v = w >= nq + nk;
    const int x = is_q ? w : is_v ? w - nq - nk : w - nq, head = x / (is_v ? dim : ru), u = x - head * (is_v ? dim : ru);
    const int64_t to = is_q ? n * a.q_out_stride + head * dim : t.dst + head * a.c.head_stride;
    void* base = is_q ? a.q_out : is_v ? a.v_cache : a.k_cache;
    const bool eight = EIGHT && !is_q;
    const Quotient by(eight ? kv_scale(is_v ? a.v_scale : a.k_scale, head, a.err) : 1.f);
    auto put = [&](int at, float f) {
      if (eight) static_cast<uint8_t*>(base)[to + at] = code(f, by);
      else static_cast<T*>(base)[to + at] = Pair<T>::round(f);
    };
    if (is_v) {
      const T v = static_cast<const T*>(a.v)[k_row * a.v_stride + head * dim + u];
      if (eight) put(u, Pair<T>::one(v));
      else static_cast<T*>(base)[to + u] = v;
    } else {
      const T* src = is_q ? static_cast<const T*>(a.q) + n * a.q_stride + head * dim
                          : static_cast<const T*>(a.k) + k_row * a.k_stride + head * dim;
      head_element<T, AXES>(a, src, is_q ? t.q_pos : t.k_pos, is_q ? s_given.q : s_given.k, u, put);
    }
  }
}

template <typename T, bool EIGHT, bool AXES>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.batch * a.slots));
  if (!a.vec) return launch_dependent(k_kv_append_elements<T, EIGHT, AXES>, grid, dim3(kThreads), 0, s, a);
  if constexpr (EIGHT || AXES)
    return launch_dependent(a.c.interleaved ? k_kv_append_ext<T, false, EIGHT, AXES> : k_kv_append_ext<T, true, EIGHT, AXES>, grid,
                            dim3(kThreads), 0, s, a);
  else
    return launch_dependent(a.c.interleaved ? k_kv_append<T, false> : k_kv_append<T, true>, grid, dim3(kThreads), 0, s, a);
}
template <typename T>
cudaError_t launch_type(const AppendArgs& a, cudaStream_t s) {
  const bool axes = a.position && a.c.rot > 0;
  if (a.c.eight) return axes ? launch<T, true, true>(a, s) : launch<T, true, false>(a, s);
  return axes ? launch<T, false, true>(a, s) : launch<T, false, false>(a, s);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t s) {
  return dtype == GRAFT_BF16 ? launch_type<__nv_bfloat16>(a, s) : launch_type<__half>(a, s);
}

}  // namespace graft
