// Penalties, biases and grammar masks on the tree's logits.
//
// A CTA takes one chunk of one request's vocabulary and some of its slots'
// rows.  It builds the chunk's rule table in shared memory once (occurrences in
// the history, the bias entry, whether a slot's token falls there) and streams
// the rows past it, so that the history is read once a chunk and not once a
// row.  Nearly every element has no rule: a bitmap tells which 16-byte pieces
// hold one that has, and the others are copied as they are, or masked by their
// bits of the grammar's row.  Bound by memory: a row is read and written once.
//
// Rows need not start on 16-byte boundaries: the pieces are those of the row's
// own alignment, so the table and the bits are read at the row's offset, and
// the few elements before its first and after its last piece go one by one.
#include <algorithm>

#include <cuda_bf16.h>

#include "logit_rules.cuh"

namespace graft {
namespace {

constexpr int kThreads = 512;
constexpr uint32_t COUNT = (1u << 19) - 1;  // occurrences in the output (the history is shorter than 2^19)
constexpr uint32_t PROMPT = 1u << 19;       // seen in the prompt
constexpr int BIAS_SHIFT = 20;              // index of the bias entry + 1, 11 bits
constexpr uint32_t BIAS = 0x7FFu << BIAS_SHIFT;
constexpr uint32_t TREE = 1u << 31;         // the token of a slot

// Elements in the words of a 16-byte piece.
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
  static __device__ __forceinline__ float at(const uint32_t* w, int e) {
    return __uint_as_float(e & 2 ? (e & 1 ? w[3] : w[2]) : (e & 1 ? w[1] : w[0]));
  }
  static __device__ __forceinline__ void set(uint32_t* w, int e, float x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = i == e ? __float_as_uint(x) : w[i];
  }
  // words of elements whose bit of `allowed` is 0 become -inf
  static __device__ __forceinline__ void forbid(uint32_t* w, uint32_t allowed) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (allowed >> i) & 1 ? w[i] : 0xFF800000u;
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ float at(const uint32_t* w, int e) {
    const uint32_t x = e & 4 ? (e & 2 ? w[3] : w[2]) : (e & 2 ? w[1] : w[0]);
    return __uint_as_float(e & 1 ? x & 0xFFFF0000u : x << 16);
  }
  static __device__ __forceinline__ void set(uint32_t* w, int e, float x) {
    const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(x));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t n = e & 1 ? (w[i] & 0xFFFFu) | h << 16 : (w[i] & 0xFFFF0000u) | h;
      w[i] = i == e >> 1 ? n : w[i];
    }
  }
  static __device__ __forceinline__ void forbid(uint32_t* w, uint32_t allowed) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = ((allowed >> (2 * i)) & 1 ? 0xFFFFu : 0u) | ((allowed >> (2 * i + 1)) & 1 ? 0xFFFF0000u : 0u);
      w[i] = (w[i] & m) | (0xFF80FF80u & ~m);
    }
  }
};

struct Shared {
  uint64_t path[MAX_S];     // ancestor masks without the root
  int32_t tok[MAX_S];       // tokens of the slots, -1 = pad
  int32_t gram[MAX_S];      // grammar row, -1 = all allowed
  int32_t rows[MAX_S];      // the CTA's slots that are no pads
  int32_t n_rows;
  float rep, freq, pres;
};

// The rules of one element: word = its table entry, i = the slot.
__device__ __forceinline__ float apply(const LogitArgs& a, const Shared& sh, const float* bias, uint32_t word, int i,
                                       int v, float x) {
  int n = word & COUNT;
  if (word & TREE) {
    uint64_t m = sh.path[i];
    while (m) {
      const int j = __ffsll((long long)m) - 1;
      m &= m - 1;
      n += sh.tok[j] == v;
    }
  }
  if (n > 0 || (word & PROMPT)) x = x > 0.f ? x / sh.rep : x * sh.rep;
  x -= sh.freq * (float)n;
  if (n > 0) x -= sh.pres;
  const uint32_t e = (word & BIAS) >> BIAS_SHIFT;
  if (e) x += bias[e - 1];
  return x;
}

// N bits from bit `at` on; `words` has at least one word more than those bits lie in, unless they end a word.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* words, int at, int n) {
  const int s = at & 31;
  const uint32_t lo = words[at >> 5], hi = s + n > 32 ? words[(at >> 5) + 1] : 0;
  return __funnelshift_r(lo, hi, s) & ((1u << n) - 1);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_logit_rules(LogitArgs a) {
  extern __shared__ uint32_t table[];  // [chunk], then the bitmap [chunk / 32 + 1]
  __shared__ Shared sh;
  constexpr int N = Elem<T>::N;
  const int b = blockIdx.y, t = threadIdx.x;
  const int c0 = blockIdx.x * a.chunk, c1 = min(a.V, c0 + a.chunk), len = c1 - c0;
  const int i0 = blockIdx.z * a.rows_per_cta, i1 = min(a.slots, i0 + a.rows_per_cta);
  uint32_t* bitmap = table + a.chunk;
  uint32_t bad = 0;
  // the slots, the request's penalties
  if (t < a.slots) {
    const int64_t at = (int64_t)b * a.slots + t;
    sh.tok[t] = a.tree_tok ? a.tree_tok[at] : 0;
    sh.path[t] = a.tree_tok ? a.tree_mask[at] & ~1ull : 0;
    if (a.slots < 64) sh.path[t] &= (1ull << a.slots) - 1;
    int g = a.r.d_grammar ? a.r.d_grammar_row[at] : -1;
    if (g < -1 || g >= a.r.n_grammar) { bad |= GRAFT_ERR_RULE; g = -1; }
    sh.gram[t] = g;
    if (a.tree_tok && sh.tok[t] >= a.V) bad |= GRAFT_ERR_TOKEN;
  }
  if (t == 0) {
    float r = 1.f, f = 0.f, p = 0.f;
    if (a.r.d_penalty) {
      r = a.r.d_penalty[3 * b]; f = a.r.d_penalty[3 * b + 1]; p = a.r.d_penalty[3 * b + 2];
      if (!(r > 0.f) || !isfinite(r) || !isfinite(f) || !isfinite(p)) { bad |= GRAFT_ERR_RULE; r = 1.f; f = p = 0.f; }
    }
    sh.rep = r; sh.freq = f; sh.pres = p;
  }
  for (int k = t; k < a.chunk; k += kThreads) table[k] = 0;
  if (t < 32) {  // the slots that are no pads, in order
    int n = 0;
    for (int i = i0; i < i1; i += 32) {
      const bool live = i + t < i1 && (!a.tree_tok || a.tree_tok[(int64_t)b * a.slots + i + t] >= 0);
      const uint32_t m = __ballot_sync(~0u, live);
      if (live) sh.rows[n + __popc(m & ((1u << t) - 1))] = i + t;
      n += __popc(m);
    }
    if (t == 0) sh.n_rows = n;
  }
  __syncthreads();
  const bool counts = sh.rep != 1.f || sh.freq != 0.f || sh.pres != 0.f;
  const float* bias = a.r.d_bias_val + (int64_t)b * a.r.n_bias;
  for (int k = t; k < a.r.n_bias; k += kThreads) {
    const int32_t v = a.r.d_bias_tok[(int64_t)b * a.r.n_bias + k];
    if (v >= a.V || v < -1) bad |= GRAFT_ERR_TOKEN;
    else if (v >= c0 && v < c1) atomicMax(&table[v - c0], (uint32_t)(k + 1) << BIAS_SHIFT);
  }
  __syncthreads();
  if (a.r.d_hist) {
    int64_t n = a.r.d_hist_len[b];
    if (n < 0 || n > a.r.hist_stride) { bad |= GRAFT_ERR_RULE; n = n < 0 ? 0 : a.r.hist_stride; }
    int64_t prompt = a.r.d_prompt_len ? a.r.d_prompt_len[b] : 0;
    if (prompt < 0) { bad |= GRAFT_ERR_RULE; prompt = 0; }
    const int32_t* hist = a.r.d_hist + (int64_t)b * a.r.hist_stride;
    for (int64_t k = t; k < n; k += kThreads) {
      const int32_t v = hist[k];
      if (v < 0 || v >= a.V) bad |= GRAFT_ERR_TOKEN;
      else if (counts && v >= c0 && v < c1) {
        if (k >= prompt) atomicAdd(&table[v - c0], 1u);
        else if (!(table[v - c0] & PROMPT)) atomicOr(&table[v - c0], PROMPT);
      }
    }
  }
  if (a.tree_tok && counts && t >= 1 && t < a.slots && sh.tok[t] >= c0 && sh.tok[t] < c1)
    atomicOr(&table[sh.tok[t] - c0], TREE);
  if (bad) atomicOr(a.err, bad);
  __syncthreads();
  for (int k = t; k < a.chunk + 32; k += kThreads) {
    const uint32_t w = __ballot_sync(~0u, k < a.chunk && table[k < a.chunk ? k : 0] != 0);
    if ((t & 31) == 0) bitmap[k >> 5] = w;
  }
  __syncthreads();
  // one element: its rules, then the grammar
  auto element = [&](int i, const uint32_t* gram, const T* in, T* out, int k) {
    float x = Elem<T>::get(in[k]);
    if (table[k]) x = apply(a, sh, bias, table[k], i, c0 + k, x);
    if (gram && !((gram[(c0 + k) >> 5] >> ((c0 + k) & 31)) & 1)) x = -INFINITY;
    out[k] = Elem<T>::put(x);
  };
  constexpr int R = 4;  // rows in flight
  const int n_rows = sh.n_rows;
  for (int r0 = 0; r0 < n_rows; r0 += R) {
    const T* in[R];
    T* out[R];
    const uint32_t* gram[R];
    int slot[R], off[R], pieces[R], most = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      slot[r] = sh.rows[min(r0 + r, n_rows - 1)];
      const int64_t row = (int64_t)b * a.slots + slot[r];
      in[r] = static_cast<const T*>(a.in) + row * a.in_stride + c0;
      out[r] = static_cast<T*>(a.out) + row * a.out_stride + c0;
      gram[r] = sh.gram[slot[r]] >= 0 ? a.r.d_grammar + (int64_t)sh.gram[slot[r]] * a.r.grammar_stride : nullptr;
      const uint32_t from = (uint32_t)reinterpret_cast<uintptr_t>(in[r]) & 15, to = (uint32_t)reinterpret_cast<uintptr_t>(out[r]) & 15;
      off[r] = from == to ? min(len, (int)(((16 - from) & 15) / sizeof(T))) : len;
      pieces[r] = r0 + r < n_rows ? (len - off[r]) / N : 0;
      most = max(most, pieces[r]);
      // the elements around the pieces
      const int loose = r0 + r < n_rows ? len - pieces[r] * N : 0;
      for (int k = t; k < loose; k += kThreads)
        element(slot[r], gram[r], in[r], out[r], k < off[r] ? k : k + pieces[r] * N);
    }
    for (int p = t; p < most; p += kThreads) {
      uint4 x[R];
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (p < pieces[r]) x[r] = __ldcs(reinterpret_cast<const uint4*>(in[r] + off[r] + p * N));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (p >= pieces[r]) continue;
        const int k = off[r] + p * N;
        uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
        uint32_t ruled = bits_at(bitmap, k, N);
        while (ruled) {
          const int e = __ffs(ruled) - 1;
          ruled &= ruled - 1;
          Elem<T>::set(w, e, apply(a, sh, bias, table[k + e], slot[r], c0 + k + e, Elem<T>::at(w, e)));
        }
        if (gram[r]) Elem<T>::forbid(w, bits_at(gram[r], c0 + k, N));
        __stcs(reinterpret_cast<uint4*>(out[r] + k), make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
}

}  // namespace

template <typename T>
static cudaError_t launch(LogitArgs a, int num_sms, cudaStream_t s) {
  // Every CTA reads the request's whole history: a chunk grows while that is more than an eighth of what its rows move
  // and two CTAs an SM remain; rows are split, four at least, when the chunks alone give fewer than four.
  const int pass = kThreads * Elem<T>::N;
  a.chunk = pass;
  auto ctas = [&](int chunk) { return (int64_t)a.batch * ((a.V + chunk - 1) / chunk); };
  while (a.chunk < 32768 && a.r.hist_stride * 32 > (int64_t)a.slots * a.chunk * (int)sizeof(T) * 2 &&
         ctas(2 * a.chunk) >= 2 * num_sms)
    a.chunk *= 2;
  const int64_t groups = std::max<int64_t>(1, std::min<int64_t>((a.slots + 3) / 4, 4 * num_sms / ctas(a.chunk)));
  a.rows_per_cta = (int)((a.slots + groups - 1) / groups);
  const dim3 grid((a.V + a.chunk - 1) / a.chunk, a.batch, (a.slots + a.rows_per_cta - 1) / a.rows_per_cta);
  const size_t smem = ((size_t)a.chunk + a.chunk / 32 + 1) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k_logit_rules<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != cudaSuccess) return e;
  }
  k_logit_rules<T><<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_logit_rules(const LogitArgs& a, int dtype, int num_sms, cudaStream_t s) {
  return dtype == GRAFT_BF16 ? launch<__nv_bfloat16>(a, num_sms, s) : launch<float>(a, num_sms, s);
}

}  // namespace graft
