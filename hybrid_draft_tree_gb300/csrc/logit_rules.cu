// Penalties, biases and grammar masks on the tree's logits.
//
// A CTA takes one chunk of one request's vocabulary and some of its slots'
// rows.  It builds the chunk's rule table in shared memory once (occurrences in
// the history, the bias entry, whether a slot's token falls there), so that the
// history is read once a chunk and not once a row, and turns it into what an
// element with a rule needs: what is taken off its logit, and whether it counts
// as seen.  Then its warps stream the rows past the table, four 16-byte pieces
// a lane at a time.  Nearly every element has no rule: a bitmap tells which
// pieces hold one that has, and the others are copied, or masked by their bits
// of the grammar's row.  Bound by memory: a row is read and written once.
//
// Rows need not start on 16-byte boundaries: the pieces are those of the row's
// own alignment, so the table and the bits are read at the row's offset, and
// the few elements before its first and after its last piece go one by one.
#include <algorithm>

#include <cuda_bf16.h>

#include "logit_rules.cuh"

namespace graft {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kUnit = 128;                  // pieces a warp takes at a time: four a lane
// a table entry while the rules are gathered
constexpr uint32_t COUNT = (1u << 19) - 1;  // occurrences in the output (the history is shorter than 2^19)
constexpr uint32_t PROMPT = 1u << 19;       // seen in the prompt
constexpr int BIAS_SHIFT = 20;              // index of the bias entry + 1, 11 bits
constexpr uint32_t BIAS = 0x7FFu << BIAS_SHIFT;
constexpr uint32_t TREE = 1u << 31;         // the token of a slot
// and then: the fp32 number taken off the logit, its lowest bit 1 for a token that was seen; or this NaN with the index
// of a token that some slots' paths hold, whose count depends on the slot
constexpr uint32_t PATH = 0xFFC00000u;

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
  static __device__ __forceinline__ void forbid(uint32_t* w, uint32_t allowed, const uint2*) {
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
  // spread[b]: the words' masks of four elements' bits b
  static __device__ __forceinline__ void forbid(uint32_t* w, uint32_t allowed, const uint2* spread) {
    const uint2 lo = spread[allowed & 15], hi = spread[allowed >> 4];
    const uint32_t m[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (w[i] & m[i]) | (0xFF80FF80u & ~m[i]);
  }
};

struct Shared {
  uint64_t path[MAX_S];     // ancestor masks without the root
  int32_t tok[MAX_S];       // tokens of the slots, -1 = pad
  int32_t gram[MAX_S];      // grammar row, -1 = all allowed
  int32_t rows[MAX_S];      // the CTA's slots that are no pads
  uint32_t path_word[MAX_S]; // gathered entries of the tokens that some paths hold
  uint2 spread[16];
  int32_t n_rows, n_paths;
  float rep, inv_rep, freq, pres;
};

// What a gathered entry takes off a logit, for a token with n occurrences.  The quotient by the repetition penalty is a
// product with its fp32 reciprocal and the differences are taken at once: a few fp32 roundings, far below the type's.
__device__ __forceinline__ float taken(const Shared& sh, const float* bias, uint32_t word, int n) {
  float x = sh.freq * (float)n;
  if (n > 0) x += sh.pres;
  const uint32_t e = (word & BIAS) >> BIAS_SHIFT;
  if (e) x -= bias[e - 1];
  return x;
}

// An element with a rule; i = the slot.
__device__ __forceinline__ float apply(const Shared& sh, const float* bias, uint32_t entry, int i, int v, float x) {
  bool seen = entry & 1;
  float off = __uint_as_float(entry);
  if (entry >= PATH) {
    const uint32_t word = sh.path_word[entry - PATH];
    int n = word & COUNT;
    for (uint64_t m = sh.path[i]; m; m &= m - 1) n += sh.tok[__ffsll((long long)m) - 1] == v;
    seen = n > 0 || (word & PROMPT);
    off = taken(sh, bias, word, n);
  }
  if (seen) x *= x > 0.f ? sh.inv_rep : sh.rep;
  return x - off;
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
    sh.rep = r; sh.inv_rep = 1.f / r; sh.freq = f; sh.pres = p;
    sh.n_paths = 0;
  }
  if (t < 16) sh.spread[t] = make_uint2((t & 1 ? 0xFFFFu : 0u) | (t & 2 ? 0xFFFF0000u : 0u), (t & 4 ? 0xFFFFu : 0u) | (t & 8 ? 0xFFFF0000u : 0u));
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
    const uint32_t word = k < a.chunk ? table[k] : 0;
    const uint32_t ruled = __ballot_sync(~0u, word != 0);
    if ((t & 31) == 0) bitmap[k >> 5] = ruled;
    if (word == 0) continue;
    uint32_t entry;
    if (word & TREE) {
      const int at = atomicAdd(&sh.n_paths, 1);
      sh.path_word[at] = word;
      entry = PATH + at;
    } else {
      const int n = word & COUNT;
      const float off = taken(sh, bias, word, n);
      entry = isnan(off) ? 0x7FC00000u : __float_as_uint(off) & ~1u;
      if (n > 0 || (word & PROMPT)) entry |= 1;
    }
    table[k] = entry;
  }
  __syncthreads();
  const int lane = t & 31, units = a.chunk / (kUnit * N), n_rows = sh.n_rows;
  for (int u = t >> 5; u < n_rows * units; u += kWarps) {
    const int r = u / units, part = u - r * units, i = sh.rows[r];
    const int64_t row = (int64_t)b * a.slots + i;
    const T* in = static_cast<const T*>(a.in) + row * a.in_stride + c0;
    T* out = static_cast<T*>(a.out) + row * a.out_stride + c0;
    const uint32_t* gram = sh.gram[i] >= 0 ? a.r.d_grammar + (int64_t)sh.gram[i] * a.r.grammar_stride : nullptr;
    auto element = [&](int k) {
      float x = Elem<T>::get(in[k]);
      if ((bitmap[k >> 5] >> (k & 31)) & 1) x = apply(sh, bias, table[k], i, c0 + k, x);
      if (gram && !((gram[(c0 + k) >> 5] >> ((c0 + k) & 31)) & 1)) x = -INFINITY;
      out[k] = Elem<T>::put(x);
    };
    const uint32_t from = (uint32_t)reinterpret_cast<uintptr_t>(in) & 15, to = (uint32_t)reinterpret_cast<uintptr_t>(out) & 15;
    if (from != to) {
      for (int k = part * kUnit * N + lane; k < min(len, (part + 1) * kUnit * N); k += 32) element(k);
      continue;
    }
    const int off = min(len, (int)(((16 - from) & 15) / sizeof(T))), pieces = (len - off) / N;
    if (part == 0)
      for (int k = lane; k < len - pieces * N; k += 32) element(k < off ? k : k + pieces * N);
    const int p0 = part * kUnit + lane;
    const uint4* src = reinterpret_cast<const uint4*>(in + off) + p0;
    uint4* dst = reinterpret_cast<uint4*>(out + off) + p0;
    uint4 x[4];
    uint32_t allowed[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (p0 + 32 * j < pieces) x[j] = __ldcs(src + 32 * j);
    const int k0 = off + p0 * N;
    if (gram) {
#pragma unroll
      for (int j = 0; j < 4; ++j) allowed[j] = p0 + 32 * j < pieces ? bits_at(gram, c0 + k0 + 32 * N * j, N) : 0;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p0 + 32 * j >= pieces) break;
      const int k = k0 + 32 * N * j;
      uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      for (uint32_t ruled = bits_at(bitmap, k, N); ruled; ruled &= ruled - 1) {
        const int e = __ffs(ruled) - 1;
        Elem<T>::set(w, e, apply(sh, bias, table[k + e], i, c0 + k + e, Elem<T>::at(w, e)));
      }
      if (gram) Elem<T>::forbid(w, allowed[j], sh.spread);
      __stcs(dst + 32 * j, make_uint4(w[0], w[1], w[2], w[3]));
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
