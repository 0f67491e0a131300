// Penalties, biases and grammar masks on the tree's logits.
//
// A CTA takes one chunk of one request's vocabulary and some of its slots'
// rows.  It builds the chunk's rule table in shared memory once (occurrences in
// the history, the bias entry, whether a slot's token falls there), so that the
// history is read once a chunk and not once a row, and turns it into what an
// element with a rule needs: what is taken off its logit, and whether it counts
// as seen.  Then its warps take the rows in units of four or eight 16-byte
// pieces a lane.  Nearly every element has no rule: a unit is masked by its bits
// of the grammar's row and stored; when some of its elements have rules, it
// passes through shared memory, where they are done a lane each (in the pieces
// they would cost the whole warp a pass for each of a lane's).  A row is read and
// written once; in place, units without a rule or a grammar are not touched.
// Bound by memory where a CTA has many rows (16 x 61 x 151936 bf16: 110 us, 5.3
// TB/s, 79% of the copy rate), by the table's building where it has few (64 x 17
// x 128256 behind 8192 tokens: 115 us, 4.7 TB/s), by latency for one row of 32000
// (5.3 us).
//
// Rows need not start on 16-byte boundaries: the pieces are those of the row's
// own alignment, so the bits are read at the row's offset, and the few elements
// before its first and after its last piece go one by one (so do rows whose input
// and output are aligned differently: 461 us instead of 110).
#include <algorithm>

#include <cuda_bf16.h>

#include "logit_rules.cuh"

namespace graft {
namespace {

// Threads of a CTA, 16-byte pieces that a lane takes at a time, CTAs an SM.
template <int THREADS, int LANE, int CTAS>
struct Shape {
  static constexpr int kThreads = THREADS, kWarps = THREADS / 32, kLane = LANE, kUnit = 32 * LANE, kCtas = CTAS;
  static size_t smem(int chunk) { return kWarps * kUnit * 16 + (size_t)chunk * 6 + 3 * (chunk / 32 + 1) * 4; }
};
using FewRows = Shape<384, 4, 3>;
using ManyRows = Shape<512, 8, 2>;
constexpr int kHeld = 8;                     // tokens of the history that a thread has in flight
// a table entry while the rules are gathered
constexpr uint32_t COUNT = (1u << 19) - 1;  // occurrences in the output (the history is shorter than 2^19)
constexpr uint32_t PROMPT = 1u << 19;       // seen in the prompt
constexpr int BIAS_SHIFT = 20;              // index of the bias entry + 1, 11 bits
constexpr uint32_t BIAS = 0x7FFu << BIAS_SHIFT;
constexpr uint32_t TREE = 1u << 31;         // the token of a slot
// and then: the fp32 number taken off the logit, all of its bits (a bias may be infinite, and f n beyond fp32; whether the
// token was seen is in a bitmap of its own); or this NaN with the index of a token that some slots' paths hold, whose count
// depends on the slot
constexpr uint32_t PATH = 0xFFC00000u;

// Elements and 16-byte pieces of them.
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
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
  // spread[b]: the words' masks of four elements' bits b
  static __device__ __forceinline__ void forbid(uint32_t* w, uint32_t allowed, const uint2* spread) {
    const uint2 lo = spread[allowed & 15], hi = spread[(allowed >> 4) & 15];
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
  float rep, freq, pres;
};

// What a gathered entry takes off a logit, for a token with n occurrences.  The differences are taken at once: four fp32
// roundings of their sizes' order, as many as one after the other would take.
__device__ __forceinline__ float taken(const Shared& sh, const float* bias, uint32_t word, int n) {
  float x = sh.freq * (float)n;
  if (n > 0) x += sh.pres;
  const uint32_t e = (word & BIAS) >> BIAS_SHIFT;
  if (e) x -= bias[e - 1];
  return x;
}

// An element with a rule; i = the slot, seen = the token occurs in the history (of a path's token the slot decides).
__device__ __forceinline__ float apply(const Shared& sh, const float* bias, uint32_t entry, bool seen, int i, int v, float x) {
  float off = __uint_as_float(entry);
  if (entry >= PATH) {
    const uint32_t word = sh.path_word[entry - PATH];
    int n = word & COUNT;
    for (uint64_t m = sh.path[i]; m; m &= m - 1) n += sh.tok[__ffsll((long long)m) - 1] == v;
    seen = n > 0 || (word & PROMPT);
    off = taken(sh, bias, word, n);
  }
  if (seen) x = x > 0.f ? x / sh.rep : x * sh.rep;
  return x - off;
}

// N bits from bit `at` on; `words` has at least one word more than those bits lie in, unless they end a word.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* words, int at, int n) {
  const int s = at & 31;
  const uint32_t lo = words[at >> 5], hi = s + n > 32 ? words[(at >> 5) + 1] : 0;
  return __funnelshift_r(lo, hi, s) & ((1u << n) - 1);
}

template <typename T, typename S>
__global__ void __launch_bounds__(S::kThreads, S::kCtas) k_logit_rules(LogitArgs a) {
  extern __shared__ uint4 space[];  // a unit a warp; the table [chunk]; two bitmaps, ranks [chunk / 32 + 1]; the list [chunk] of 16 bits
  __shared__ Shared sh;
  constexpr int N = Elem<T>::N, kThreads = S::kThreads, kWarps = S::kWarps, kLane = S::kLane, kUnit = S::kUnit;
  const int b = blockIdx.y, t = threadIdx.x;
  const int c0 = blockIdx.x * a.chunk, c1 = min(a.V, c0 + a.chunk), len = c1 - c0;
  const int i0 = blockIdx.z * a.rows_per_cta, i1 = min(a.slots, i0 + a.rows_per_cta);
  uint4* const stage = space + (t >> 5) * kUnit;
  uint32_t* const table = reinterpret_cast<uint32_t*>(space + kWarps * kUnit);
  uint32_t* const bitmap = table + a.chunk;            // elements with a rule
  uint32_t* const seen = bitmap + a.chunk / 32 + 1;    // elements whose token was seen
  uint32_t* const ranks = seen + a.chunk / 32 + 1;     // how many lie before a word of the bitmap
  uint16_t* const list = reinterpret_cast<uint16_t*>(ranks + a.chunk / 32 + 1);  // they, in order
  uint32_t bad = 0;
  grid_dependents_launch();
  grid_dependency_wait();
  // the first of the history on its way while the table is cleared
  const int32_t* const hist = a.r.d_hist + (int64_t)b * a.r.hist_stride;
  int n_hist = 0, prompt = 0;
  if (a.r.d_hist) {
    n_hist = a.r.d_hist_len[b];
    if (n_hist < 0 || n_hist > a.r.hist_stride) { bad |= GRAFT_ERR_RULE; n_hist = n_hist < 0 ? 0 : (int)a.r.hist_stride; }
    prompt = a.r.d_prompt_len ? a.r.d_prompt_len[b] : 0;
    if (prompt < 0) { bad |= GRAFT_ERR_RULE; prompt = 0; }
  }
  int32_t held[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) held[j] = t + j * kThreads < n_hist ? hist[t + j * kThreads] : -1;
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
  for (int k0 = 0; k0 < n_hist; k0 += kHeld * kThreads) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int k = k0 + t + j * kThreads, v = held[j];
      if (k >= n_hist) break;
      if (v < 0 || v >= a.V) bad |= GRAFT_ERR_TOKEN;
      else if (counts && v >= c0 && v < c1) {
        if (k >= prompt) atomicAdd(&table[v - c0], 1u);
        else if (!(table[v - c0] & PROMPT)) atomicOr(&table[v - c0], PROMPT);
      }
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int k = k0 + t + (kHeld + j) * kThreads;
      if (k < n_hist) held[j] = hist[k];
    }
  }
  if (a.tree_tok && counts && t >= 1 && t < a.slots && sh.tok[t] >= c0 && sh.tok[t] < c1)
    atomicOr(&table[sh.tok[t] - c0], TREE);
  if (bad) atomicOr(a.err, bad);
  __syncthreads();
  const int lane = t & 31, words = a.chunk / 32;
  for (int k = t; k < a.chunk; k += kThreads) {
    const uint32_t word = table[k], ruled = __ballot_sync(~0u, word != 0);
    const uint32_t was_seen = __ballot_sync(~0u, (word & (COUNT | PROMPT)) != 0);
    if (lane == 0) {
      bitmap[k >> 5] = ruled;
      seen[k >> 5] = was_seen;
    }
    if (word == 0) continue;
    uint32_t entry;
    if (word & TREE) {
      const int path = atomicAdd(&sh.n_paths, 1);
      sh.path_word[path] = word;
      entry = PATH + path;
    } else {
      const float off = taken(sh, bias, word, word & COUNT);
      entry = isnan(off) ? 0x7FC00000u : __float_as_uint(off);
    }
    table[k] = entry;
  }
  if (t == 0) bitmap[words] = 0;
  __syncthreads();
  if (t < 32) {
    uint32_t n = 0;
    for (int w = lane; w < (words / 32 + 1) * 32; w += 32) {
      const uint32_t mine = w < words ? __popc(bitmap[w]) : 0;
      uint32_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += v;
      }
      if (w <= words) ranks[w] = n + upto - mine;
      n += __shfl_sync(~0u, upto, 31);
    }
  }
  __syncthreads();
  auto rank = [&](int k) { return (int)(ranks[k >> 5] + __popc(bitmap[k >> 5] & ((1u << (k & 31)) - 1))); };
  for (int k = t; k < a.chunk; k += kThreads)
    if ((bitmap[k >> 5] >> (k & 31)) & 1) list[rank(k)] = (uint16_t)k;
  __syncthreads();

  const int n_rows = sh.n_rows, units = a.chunk / (kUnit * N);
  const bool in_place = a.in == a.out;
  struct Row { const T* in; T* out; const uint32_t* gram; int slot; };
  auto row_at = [&](int r) {
    const int i = sh.rows[r];
    const int64_t row = (int64_t)b * a.slots + i;
    return Row{static_cast<const T*>(a.in) + row * a.in_stride + c0, static_cast<T*>(a.out) + row * a.out_stride + c0,
               sh.gram[i] >= 0 ? a.r.d_grammar + (int64_t)sh.gram[i] * a.r.grammar_stride : nullptr, i};
  };
  auto ruled = [&](int k, int slot, T x) {
    return Elem<T>::put(apply(sh, bias, table[k], (seen[k >> 5] >> (k & 31)) & 1, slot, c0 + k, Elem<T>::get(x)));
  };
  auto forbidden = [&](const uint32_t* gram, int k) { return gram && !((gram[(c0 + k) >> 5] >> ((c0 + k) & 31)) & 1); };
  auto element = [&](const Row& r, int k) {
    if (forbidden(r.gram, k)) r.out[k] = Elem<T>::put(-INFINITY);
    else if ((bitmap[k >> 5] >> (k & 31)) & 1) r.out[k] = ruled(k, r.slot, r.in[k]);
    else r.out[k] = r.in[k];
  };
  auto offset = [](const T* p) { return (int)((uint32_t)reinterpret_cast<uintptr_t>(p) & 15); };
  for (int u = t >> 5; u < n_rows * units; u += kWarps) {
    const int r = u / units, part = u - r * units;
    const Row row = row_at(r);
    const T* const in = row.in;
    T* const out = row.out;
    const uint32_t* const gram = row.gram;
    const int i = row.slot, from = offset(in);
    if (from != offset(out)) {
      for (int k = part * kUnit * N + lane; k < min(len, (part + 1) * kUnit * N); k += 32) element(row, k);
      continue;
    }
    const int off = min(len, (int)(((16 - from) & 15) / sizeof(T))), pieces = (len - off) / N;
    const int k0 = off + min(pieces, part * kUnit) * N, k1 = off + min(pieces, (part + 1) * kUnit) * N;  // of the unit
    const int e0 = rank(k0), e1 = rank(k1);
    if (in_place && !gram) {
      for (int e = e0 + lane; e < e1; e += 32) element(row, list[e]);
      continue;
    }
    const int n = (k1 - k0) / N;
    const uint4* src = reinterpret_cast<const uint4*>(in + k0);
    uint4* dst = reinterpret_cast<uint4*>(out + k0);
    uint4 x[kLane];
#pragma unroll
    for (int j = 0; j < kLane; ++j) x[j] = lane + 32 * j < n ? __ldcs(src + lane + 32 * j) : make_uint4(0, 0, 0, 0);
    if (gram) {
      uint32_t allowed[kLane];
#pragma unroll
      for (int j = 0; j < kLane; ++j)
        allowed[j] = lane + 32 * j < n ? bits_at(gram, c0 + k0 + (lane + 32 * j) * N, N) : 0;
#pragma unroll
      for (int j = 0; j < kLane; ++j) {
        uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        Elem<T>::forbid(w, allowed[j], sh.spread);
        x[j] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (e0 < e1) {
#pragma unroll
      for (int j = 0; j < kLane; ++j) stage[lane + 32 * j] = x[j];
      __syncwarp();
      T* const values = reinterpret_cast<T*>(stage);
      for (int e = e0 + lane; e < e1; e += 32) {
        const int k = list[e];
        // what the grammar forbids is -inf already, and stays so whatever its rule takes off
        if (!forbidden(gram, k)) values[k - k0] = ruled(k, i, values[k - k0]);
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kLane; ++j) x[j] = stage[lane + 32 * j];
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < kLane; ++j)
      if (lane + 32 * j < n) __stcs(dst + lane + 32 * j, x[j]);
  }
  // elements before a row's first piece and after its last, from the end on: the last warps have the fewest units
  if ((len % N | offset(static_cast<const T*>(a.in) + c0) | (a.in_stride % N)) == 0) return;
  for (int e = kThreads - 1 - t; e < n_rows * 2 * N; e += kThreads) {
    const Row row = row_at(e / (2 * N));
    const int x = e & (2 * N - 1), from = offset(row.in);
    if (from != offset(row.out)) continue;
    const int off = min(len, (int)(((16 - from) & 15) / sizeof(T))), pieces = (len - off) / N;
    if (x < len - pieces * N) element(row, x < off ? x : x + pieces * N);
  }
}

}  // namespace

constexpr int kMaxChunk = 6144;

template <typename T, typename S>
static cudaError_t prepare() {
  return cudaFuncSetAttribute(k_logit_rules<T, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::smem(kMaxChunk));
}

cudaError_t prepare_logit_rules() {
  cudaError_t e = prepare<__nv_bfloat16, FewRows>();
  if (e == cudaSuccess) e = prepare<float, FewRows>();
  if (e == cudaSuccess) e = prepare<float, ManyRows>();
  return e;
}

static int64_t ctas_of(const LogitArgs& a, int chunk) { return (int64_t)a.batch * ((a.V + chunk - 1) / chunk); }

template <typename T, typename S>
static cudaError_t launch(LogitArgs a, int num_sms, cudaStream_t s) {
  // Every CTA reads the request's whole history: while that is more than an eighth of what its rows move, a chunk grows
  // as long as two CTAs an SM remain and three fit (64 x 17 behind 8192: 123 us with 3072 elements, 115 with 6144).  When the chunks alone are too few for the SMs, rows are split too, four at least, into one wave of CTAs
  // (1 x 61 behind 32768: 22 us; into 4 CTAs an SM 33, into one 26).
  const int pass = S::kThreads * Elem<T>::N;
  a.chunk = pass;
  while (2 * a.chunk <= kMaxChunk && a.r.hist_stride * 32 > (int64_t)a.slots * a.chunk * (int)sizeof(T) * 2 &&
         ctas_of(a, 2 * a.chunk) >= 2 * num_sms)
    a.chunk *= 2;
  const int64_t groups = std::max<int64_t>(1, std::min<int64_t>((a.slots + 3) / 4, 3 * num_sms / ctas_of(a, a.chunk)));
  a.rows_per_cta = (int)((a.slots + groups - 1) / groups);
  const dim3 grid((a.V + a.chunk - 1) / a.chunk, a.batch, (a.slots + a.rows_per_cta - 1) / a.rows_per_cta);
  return launch_dependent(k_logit_rules<T, S>, grid, dim3(S::kThreads), S::smem(a.chunk), s, a);
}

// How many CTAs build their tables at once counts most (bf16, 64 x 17 x 128256: 115 us with three an SM, 140 with two; one
// fp32 row of 32000: 5.3 and 6.0), for bf16 at every number of rows (16 x 61 x 151936: 110 and 111).  With many fp32 rows
// a CTA it is the pieces in flight: 16 x 32 x 151936 take 106 us with eight a lane and two CTAs, 109 with four and three;
// 16 x 28 96 either way, 16 x 17 65.4 and 64.9; where the chunks are less than two CTAs an SM, four (1 x 61 behind 32768:
// 27 us, 35 with eight).
cudaError_t launch_logit_rules(const LogitArgs& a, int dtype, int num_sms, cudaStream_t s) {
  if (dtype == GRAFT_BF16) return launch<__nv_bfloat16, FewRows>(a, num_sms, s);
  const bool many = a.slots >= 32 && ctas_of(a, ManyRows::kThreads * Elem<float>::N) >= 2 * num_sms;
  return many ? launch<float, ManyRows>(a, num_sms, s) : launch<float, FewRows>(a, num_sms, s);
}

}  // namespace graft
