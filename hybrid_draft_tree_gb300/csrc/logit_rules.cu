// Penalties, biases and grammar masks on the tree's logits.
//
// A CTA takes one chunk of one request's vocabulary and some of its slots'
// rows.  It builds the chunk's rule table in shared memory once (occurrences in
// the history, the bias entry, whether a slot's token falls there) and streams
// the rows past it.  Nearly every element has no rule and is copied as it is
// (or masked by a bit): a bitmap tells which 16-byte pieces hold one that has.
#include "kv_internal.cuh"
#include "logit_rules.cuh"

namespace graft {
namespace {

constexpr int kThreads = 512;
constexpr uint32_t COUNT = (1u << 19) - 1;  // occurrences in the output (the history is shorter than 2^19)
constexpr uint32_t PROMPT = 1u << 19;       // seen in the prompt
constexpr int BIAS_SHIFT = 20;              // index of the bias entry + 1, 11 bits
constexpr uint32_t BIAS = 0x7FFu << BIAS_SHIFT;
constexpr uint32_t TREE = 1u << 31;         // the token of a slot

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int N = 4;
  static constexpr uint32_t NEG_INF = 0xFF800000u;
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

struct Shared {
  uint64_t path[MAX_S];     // ancestor masks without the root
  int32_t tok[MAX_S];       // tokens of the slots, -1 = pad
  int32_t gram[MAX_S];      // grammar row, -1 = all allowed
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

template <typename T>
__global__ void __launch_bounds__(kThreads) k_logit_rules(LogitArgs a) {
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
  for (int i = i0; i < i1; ++i) {
    if (sh.tok[i] < 0) continue;
    const int64_t row = (int64_t)b * a.slots + i;
    const T* in = static_cast<const T*>(a.in) + row * a.in_stride + c0;
    T* out = static_cast<T*>(a.out) + row * a.out_stride + c0;
    const uint32_t* gram = sh.gram[i] >= 0 ? a.r.d_grammar + (int64_t)sh.gram[i] * a.r.grammar_stride : nullptr;
    for (int k = t; k < len; k += kThreads) {
      float x = Elem<T>::get(in[k]);
      if (table[k]) x = apply(a, sh, bias, table[k], i, c0 + k, x);
      if (gram && !((gram[(c0 + k) >> 5] >> ((c0 + k) & 31)) & 1)) x = -INFINITY;
      out[k] = Elem<T>::put(x);
    }
  }
}

}  // namespace

cudaError_t launch_logit_rules(LogitArgs a, int dtype, int num_sms, cudaStream_t s) {
  a.chunk = 4096;
  const int chunks = (a.V + a.chunk - 1) / a.chunk;
  a.rows_per_cta = a.slots;
  const dim3 grid(chunks, a.batch, (a.slots + a.rows_per_cta - 1) / a.rows_per_cta);
  const size_t smem = (size_t)a.chunk * 4 + (a.chunk / 32 + 1) * 4;
  if (dtype == GRAFT_BF16) k_logit_rules<__nv_bfloat16><<<grid, kThreads, smem, s>>>(a);
  else k_logit_rules<float><<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace graft
