// Attention of a step's slots over the paged cache (a shared prefix, each
// request's own context, the tree under its ancestor masks) on the tensor cores.
//
// A work item is up to 256 query rows of one kv head (a row is a slot and one
// of the head's query heads) against a range of key blocks of 128.  Its CTA:
//   warps 0-3, 4-7   two softmax groups, a thread a row: scores out of tensor
//                    memory, running maximum and sum, weights back into it;
//   warp 8           keys and values by tensor map, a page a copy, into a ring;
//   warp 9           S = Q K^T and O += P V, fp32 accumulators in tensor memory;
//   warp 10          values of places that no row may see, made harmless;
//   warp 11          nothing: registers move between groups of four warps.
// The groups alternate so that one's products run under the other's softmax.
// With more than 128 rows each group has its own 128 (every block's keys and
// values serve both); with fewer both share the rows and take the key blocks in
// turn, and their results are joined at the end.
//
// The online softmax keeps, per row, a base m, l = sum 2^(s-m) and O = sum
// 2^(s-m) v, s in units of log2.  m follows the maximum only when that has
// grown by 2^8: until then weights above 1 are as exact as below, and O, which
// lives in tensor memory, is not read and written back for every block.
//
// Rows of all requests against the prefix are packed into the same tiles
// ("packed"), so a prefix block is read once for up to 256 rows, when a
// request's own rows would leave a tile mostly empty; otherwise an item runs
// over prefix and own context in one pass ("joined").  Items are split along
// the keys until the SMs are full; partial results (normalised, with their
// log-sum-exp, fp32) are joined by a second kernel.
#include <algorithm>
#include <type_traits>

#include "kv_internal.cuh"
#include "tcgen05.cuh"

namespace graft {
namespace {

using namespace bulk;

constexpr int kSoftmaxThreads = 256, kThreads = 384;
// 384 threads start with 168 registers each; the softmax groups' 256 take 216, the rest keep 72: 64512 either way
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kCleanWarp = 10;
constexpr int BN = 128;                   // keys of a block
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.f;              // log2 of how far a maximum may run ahead of the base

template <int D>
struct Smem {
  static constexpr int kHalves = D / 64;              // tiles are stored in column halves of 64 elements (128 bytes)
  static constexpr int kTile = kHalves * 128 * 128;   // bytes of 128 rows
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kRing = 2 * kTile, kBytes = kRing + kStages * kTile + 1024;  // + alignment slack
};

struct Bars {
  unsigned long long full[8], empty[8], q_full, s_full[2], p_full[2], o_done[2], dirty, clean, drain;
  unsigned long long bad;        // slots whose value holds an element that is not finite
  uint32_t tmem;
  volatile uint32_t abort;
};

// One work item, the same in every thread of its CTA.
struct Item {
  int head;            // kv head
  int b;               // request, -1: rows of all requests (prefix only)
  int row0, rows;      // first row, number of rows of the row space
  int part;            // partial index, or -1: the item's rows are complete
  int nt;              // 128-row tiles: 2, or 1 shared by both groups
  int blocks;          // key blocks
  int first;           // first block, prefix blocks first
  int np;              // blocks below np are the prefix's
  int ctx;             // tokens of the request before the tree
  bool bad_ctx;
};

__device__ __forceinline__ Item decode(const AttendArgs& a) {
  const AttendPlan& p = a.plan;
  Item it{};
  int x = blockIdx.x;
  const int blocks_p = (a.prefix_len + BN - 1) / BN;
  if (x < p.items_a) {
    const int s = x % p.splits_a;
    x /= p.splits_a;
    it.head = x % a.c.kv_heads;
    const int tile = x / a.c.kv_heads;
    it.b = -1;
    it.nt = p.nt_a;
    it.row0 = tile * it.nt * 128;
    it.rows = a.batch * a.slots * a.group;
    it.np = blocks_p;
    const int per = (blocks_p + p.splits_a - 1) / p.splits_a;
    it.first = s * per;
    it.blocks = max(0, min(blocks_p, it.first + per) - it.first);
    it.part = s;
    return it;
  }
  x -= p.items_a;
  const int s = x % p.splits_b;
  x /= p.splits_b;
  it.head = x % a.c.kv_heads;
  x /= a.c.kv_heads;
  it.b = x % a.batch;
  const int tile = x / a.batch;
  it.nt = p.nt_b;
  it.row0 = tile * it.nt * 128;
  it.rows = a.slots * a.group;
  it.ctx = a.ctx_len[it.b];
  it.bad_ctx = it.ctx < 0 || it.ctx > a.max_ctx;
  it.ctx = min(max(it.ctx, 0), a.max_ctx);
  it.np = p.items_a > 0 ? 0 : blocks_p;
  const int total = it.np + (it.ctx + a.slots + BN - 1) / BN;
  const int per = (total + p.splits_b - 1) / p.splits_b;
  it.first = min(total, s * per);
  it.blocks = min(total, it.first + per) - it.first;
  it.part = p.parts > 1 ? (p.items_a > 0 ? p.splits_a : 0) + s : -1;
  return it;
}

// Keys of block j of the item: index of the first within its segment, how many are keys.
struct Block {
  bool prefix, masked;  // masked: some row does not see all 128
  int base, valid;
};
__device__ __forceinline__ Block block_of(const AttendArgs& a, const Item& it, int j) {
  const int x = it.first + j;
  Block k;
  k.prefix = x < it.np;
  k.base = (k.prefix ? x : x - it.np) * BN;
  k.valid = min(BN, (k.prefix ? a.prefix_len : it.ctx + a.slots) - k.base);
  k.masked = k.prefix ? k.valid < BN : k.base + BN > it.ctx;
  return k;
}

// Where a row's query, output and mask are: token row b * slots + slot, query head.
struct Row {
  int token, head;
};
__device__ __forceinline__ Row row_of(const AttendArgs& a, const Item& it, int r) {
  const int per = a.slots * a.group;
  const int b = it.b >= 0 ? it.b : r / per;
  const int in = it.b >= 0 ? r : r - b * per;
  const int slot = in / a.group;
  return Row{b * a.slots + slot, it.head * a.group + in - slot * a.group};
}

__device__ __forceinline__ uint64_t mask_of(const AttendArgs& a, int token) {
  const uint64_t all = a.slots == 64 ? ~0ull : (1ull << a.slots) - 1;
  if (a.tree_mask) return a.tree_mask[token] & all;
  const int slot = token % a.slots;
  return slot == 63 ? ~0ull : (1ull << (slot + 1)) - 1;
}

// A wait that another role's abort, or the poll limit, ends; false: the item's results are void.
__device__ __forceinline__ bool wait_bar(Bars& sh, const AttendArgs& a, unsigned long long* bar, uint32_t parity) {
  const uint32_t limit = a.wait_polls ? a.wait_polls : SPIN;
  for (uint32_t n = 0; n < limit; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if (sh.abort) return false;
  }
  atomicOr(a.err, GRAFT_ERR_TIMEOUT);
  sh.abort = 1;
  return false;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
      "l"(reinterpret_cast<uint64_t&>(c)));
  return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return reinterpret_cast<float2&>(d);
}

// ---- warp 8: keys and values into the ring ----------------------------------------------------------------------
template <int D>
__device__ void load_role(const AttendArgs& a, const Item& it, Bars& sh, uint8_t* ring, const CUtensorMap* kmap,
                          const CUtensorMap* vmap) {
  using S = Smem<D>;
  const int lane = threadIdx.x & 31;
  const int pages = BN >> a.c.page_shift;                   // of a block; a copy is a page's half
  const int page_bytes = a.c.page_size * 128;
  int loads = 0;
  uint32_t bad = it.bad_ctx ? GRAFT_ERR_RANGE : 0;
  // page of this lane's copy of block j: copy lane -> half lane % kHalves of page lane / kHalves
  auto page_of = [&](int j) -> int {
    const Block k = block_of(a, it, j);
    const int q = lane / S::kHalves;
    if (q >= pages || (q << a.c.page_shift) >= k.valid) return -1;
    const int at = (k.base >> a.c.page_shift) + q;
    int page = k.prefix ? a.prefix_pages[at] : a.page_table[(int64_t)it.b * a.table_stride + at];
    if (page < 0 || page >= a.c.num_pages) {                // reads as zeros
      bad = GRAFT_ERR_RANGE;
      page = a.c.num_pages;
    }
    return page;
  };
  int page = it.blocks > 0 ? page_of(0) : -1;
  bool ok = true;
  for (int j = 0; j < it.blocks && ok; ++j) {
    const int here = page;
    if (j + 1 < it.blocks) page = page_of(j + 1);
    const int copies = __popc(__ballot_sync(~0u, here >= 0));
    for (int v = 0; v < 2 && ok; ++v) {
      const int stage = loads % S::kStages;
      ok = loads < S::kStages || wait_bar(sh, a, &sh.empty[stage], ((loads / S::kStages) - 1) & 1);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      if (lane == 0) mbar_expect_tx(&sh.full[stage], copies * page_bytes);
      __syncwarp();
      if (here >= 0)
        tc::tma_4d(ring + stage * S::kTile + (lane % S::kHalves) * (128 * 128) + (lane / S::kHalves) * page_bytes,
                   v ? vmap : kmap, (lane % S::kHalves) * 64, 0, it.head, here, &sh.full[stage]);
      ++loads;
    }
  }
  if (bad) atomicOr(a.err, bad);
  if (sh.abort && lane == 0)  // the copies in flight land before the CTA ends
    for (int x = max(0, loads - S::kStages); x < loads; ++x)
      mbar_wait_drain(&sh.full[x % S::kStages], (x / S::kStages) & 1);
}

// ---- warp 10: values that no row may see -------------------------------------------------------------------------
// They must not reach a product as NaN or infinity (0 times them is NaN): rows past the last key are zeroed, and of the
// tree's rows (a key that some rows see and others do not) the elements that are not finite; their slots are recorded,
// and the rows that see them add those elements at the end.
template <typename T, int D>
__device__ void clean_role(const AttendArgs& a, const Item& it, Bars& sh, uint8_t* ring) {
  using S = Smem<D>;
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  uint32_t turn = 0;
  for (int j = 0; j < it.blocks; ++j) {
    const Block k = block_of(a, it, j);
    if (!k.masked) continue;
    // the issuing thread says when the block's values are there: only then is the stage's phase this block's
    const int x = 2 * j + 1, stage = x % S::kStages;
    bool ok = wait_bar(sh, a, &sh.dirty, turn++ & 1);
    ok = ok && wait_bar(sh, a, &sh.full[stage], (x / S::kStages) & 1);
    if (!__all_sync(~0u, ok)) return;
    const int tree = k.prefix ? k.valid : min(max(it.ctx - k.base, 0), k.valid);  // first row that is a slot
    for (int half = 0; half < S::kHalves; ++half) {
      uint4* p = reinterpret_cast<uint4*>(ring + stage * S::kTile + half * 128 * 128);
      for (int i = tree * 8 + lane; i < BN * 8; i += 32) {
        const int row = i >> 3;
        if (row >= k.valid) {
          p[i] = make_uint4(0, 0, 0, 0);
          continue;
        }
        const uint4 v = p[i];
        uint32_t e[4] = {v.x, v.y, v.z, v.w};
        bool any = false;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if ((e[c] & kExp) == kExp) { e[c] &= 0xFFFF0000u; any = true; }
          if (((e[c] >> 16) & kExp) == kExp) { e[c] &= 0xFFFFu; any = true; }
        }
        if (any) {
          p[i] = make_uint4(e[0], e[1], e[2], e[3]);
          atomicOr(&sh.bad, 1ull << (k.base + row - it.ctx));
        }
      }
    }
    tc::fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.clean);
  }
}

// ---- warp 9: the products ---------------------------------------------------------------------------------------
// One thread issues every product: its code has no warp-wide step in it.  Products run in the order they are issued, so
// the scores of a group's next block may follow its O += P V at once, although they overwrite P.
template <typename T, int D>
__device__ void mma_role(const AttendArgs& a, const Item& it, Bars& sh, uint8_t* q, uint8_t* ring) {
  using S = Smem<D>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kQK = tc::instr_desc(kBf16, 128, BN, false), kPV = tc::instr_desc(kBf16, 128, D, true);
  const uint32_t tmem = sh.tmem;
  const int units = it.blocks * it.nt;
  const uint64_t qd = tc::smem_desc(smem_u32(q), 16), kd = tc::smem_desc(smem_u32(ring), 16);
  const uint64_t vd = tc::smem_desc(smem_u32(ring), 128 * 128);
  constexpr int kTile16 = S::kTile / 16;
  // unit u is group u & 1 on key block u >> 1 (two tiles) or u (one)
  auto qk = [&](int u) -> bool {
    const int t = u & 1, x = it.nt == 2 ? u & ~1 : 2 * u, stage = x % S::kStages;
    if (!wait_bar(sh, a, &sh.full[stage], (x / S::kStages) & 1)) return false;
    tc::fence_after();
    const uint64_t qa = qd + (it.nt == 2 ? t : 0) * kTile16, kb = kd + stage * kTile16;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint64_t step = (k >> 2) * (128 * 128 / 16) + (k & 3) * 2;
      tc::mma_ss(tmem + t * 128, qa + step, kb + step, kQK, k > 0);
    }
    tc::commit(&sh.s_full[t]);
    if (it.nt == 1 || t == 1) tc::commit(&sh.empty[stage]);
    return true;
  };
  bool ok = wait_bar(sh, a, &sh.q_full, 0);
  for (int u = 0; u < 2 && u < units && ok; ++u) ok = qk(u);
  uint32_t cleaned = 0;
  for (int u = 0; u < units && ok; ++u) {
    const int t = u & 1, n = u >> 1, j = it.nt == 2 ? n : u, x = 2 * j + 1, stage = x % S::kStages;
    ok = wait_bar(sh, a, &sh.full[stage], (x / S::kStages) & 1);
    if (ok && (it.nt == 1 || t == 0) && block_of(a, it, j).masked) {
      mbar_arrive(&sh.dirty);
      ok = wait_bar(sh, a, &sh.clean, cleaned++ & 1);
    }
    ok = ok && wait_bar(sh, a, &sh.p_full[t], n & 1);
    if (!ok) break;
    tc::fence_after();
    const uint32_t o = tmem + 256 + t * D, p = tmem + (D == 128 ? t * 128 : 384 + t * 64);
    const uint64_t vb = vd + stage * kTile16;
#pragma unroll
    for (int k = 0; k < BN / 16; ++k) tc::mma_ts(o, p + k * 8, vb + k * (16 * 128 / 16), kPV, n > 0 || k > 0);
    if (it.nt == 1 || t == 1) tc::commit(&sh.empty[stage]);
    if (u + 2 >= units) tc::commit(&sh.o_done[t]);
    else ok = qk(u + 2);
  }
  if (sh.abort) {  // the products in flight finish before the tensor memory goes back
    tc::commit(&sh.drain);
    mbar_wait_drain(&sh.drain, 0);
  }
}

// ---- warps 0-7: softmax and results -----------------------------------------------------------------------------
template <typename T, int D>
__device__ void store_row(const AttendArgs& a, const Item& it, const Row& row, float lse2, const float* o, int c0, int n) {
  if (it.part >= 0) {
    float* dst = a.part_o + ((int64_t)it.part * a.plan.rows + (int64_t)row.token * a.c.q_heads + row.head) * D + c0;
    for (int c = 0; c < n; c += 4) *reinterpret_cast<float4*>(dst + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
    return;
  }
  T* dst = static_cast<T*>(a.out) + row.token * a.out_stride + row.head * D + c0;
  if (a.out_vec) {
#pragma unroll
    for (int c = 0; c < n; c += 8)
      *reinterpret_cast<uint4*>(dst + c) = make_uint4(Pair<T>::put(o[c], o[c + 1]), Pair<T>::put(o[c + 2], o[c + 3]),
                                                      Pair<T>::put(o[c + 4], o[c + 5]), Pair<T>::put(o[c + 6], o[c + 7]));
  } else {
#pragma unroll
    for (int c = 0; c < n; ++c) dst[c] = Pair<T>::round(o[c]);
  }
}

template <typename T, int D>
__device__ void softmax_role(const AttendArgs& a, const Item& it, Bars& sh, uint8_t* q) {
  using S = Smem<D>;
  const int tid = threadIdx.x, t = tid >> 7, lane_row = tid & 127;
  const uint32_t lanes = (uint32_t)(tid & 96) << 16;   // tensor-memory lanes of this warp
  const uint32_t tmem = sh.tmem + lanes;
  // queries into shared memory, 16 bytes a thread, in the swizzled order the products read
  for (int x = tid; x < it.nt * 128 * (D / 8); x += kSoftmaxThreads) {
    const int r = x / (D / 8), c = x % (D / 8);
    uint4 w = make_uint4(0, 0, 0, 0);
    if (it.row0 + r < it.rows) {
      const Row row = row_of(a, it, it.row0 + r);
      const T* src = static_cast<const T*>(a.q) + row.token * a.q_stride + row.head * D + c * 8;
      if (a.q_vec) {
        w = *reinterpret_cast<const uint4*>(src);
      } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
        w = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
      }
    }
    uint8_t* dst = q + (r >> 7) * S::kTile + (c >> 3) * (128 * 128) + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4);
    *reinterpret_cast<uint4*>(dst) = w;
  }
  tc::fence_async_smem();
  mbar_arrive(&sh.q_full);

  const int r = it.row0 + (it.nt == 2 ? t * 128 : 0) + lane_row;
  const bool live = r < it.rows;
  const Row row = live ? row_of(a, it, r) : Row{0, 0};
  const uint64_t mask = live ? mask_of(a, row.token) : 0;
  const bool warp_live = __any_sync(~0u, live);
  const float scale = a.scale * kLog2e;
  const int units = it.nt == 2 ? it.blocks : (it.blocks + 1 - t) >> 1;
  float m = -INFINITY;
  float2 l2 = make_float2(0.f, 0.f);
  bool ok = true;
  for (int n = 0; n < units && ok; ++n) {
    const Block k = block_of(a, it, it.nt == 2 ? n : 2 * n + t);
    ok = __all_sync(~0u, wait_bar(sh, a, &sh.s_full[t], n & 1));
    if (!ok) break;
    tc::fence_after();
    if (warp_live) {
      uint32_t s[BN];
#pragma unroll
      for (int c = 0; c < BN; c += 32) tc::ld32(tmem + t * 128 + c, s + c);
      tc::wait_ld();
      if (k.masked) {
        // bit c: the row sees key c of the block
        uint64_t lo, hi;
        if (k.prefix) {
          lo = k.valid >= 64 ? ~0ull : (1ull << k.valid) - 1;
          hi = k.valid >= 128 ? ~0ull : k.valid > 64 ? (1ull << (k.valid - 64)) - 1 : 0;
        } else {
          const int d = it.ctx - k.base;  // keys before the tree; negative: the tree began in an earlier block
          if (d >= 64) {
            lo = ~0ull;
            hi = d >= 128 ? ~0ull : ((1ull << (d - 64)) - 1) | mask << (d - 64);
          } else if (d > 0) {
            lo = ((1ull << d) - 1) | mask << d;
            hi = mask >> (64 - d);
          } else {
            lo = d > -64 ? mask >> -d : 0;
            hi = 0;
          }
        }
        const uint32_t w[4] = {(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
#pragma unroll
        for (int c = 0; c < BN; ++c)
          if (!((w[c >> 5] >> (c & 31)) & 1)) s[c] = 0xFF800000u;  // -inf
      }
      const float* sf = reinterpret_cast<const float*>(s);
      float mx[4] = {sf[0], sf[1], sf[2], sf[3]};
#pragma unroll
      for (int c = 4; c < BN; c += 4) {
        mx[0] = fmaxf(mx[0], sf[c]);
        mx[1] = fmaxf(mx[1], sf[c + 1]);
        mx[2] = fmaxf(mx[2], sf[c + 2]);
        mx[3] = fmaxf(mx[3], sf[c + 3]);
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
      if (__any_sync(~0u, top > m + kGrow)) {
        const float next = fmaxf(m, top);
        const float f = next == -INFINITY ? 1.f : ex2(m - next);
        m = next;
        l2.x *= f;
        l2.y *= f;
        if (n > 0) {  // the scores' arrival implies that the products before them are done: O is at rest
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tc::ld32(tmem + 256 + t * D + c, o);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tc::st32(tmem + 256 + t * D + c, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      const float2 sc = make_float2(scale, scale), mb = make_float2(-base, -base);
      float2 sum0 = l2, sum1 = make_float2(0.f, 0.f);
      const uint32_t p_at = tmem + (D == 128 ? t * 128 : 384 + t * 64);
#pragma unroll
      for (int c = 0; c < BN; c += 32) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float2 x = fma2(make_float2(sf[c + i], sf[c + i + 1]), sc, mb);
          float2 y = fma2(make_float2(sf[c + i + 2], sf[c + i + 3]), sc, mb);
          x = make_float2(ex2(x.x), ex2(x.y));
          y = make_float2(ex2(y.x), ex2(y.y));
          sum0 = add2(sum0, x);
          sum1 = add2(sum1, y);
          p[i / 2] = Pair<T>::put(x.x, x.y);
          p[i / 2 + 1] = Pair<T>::put(y.x, y.y);
        }
        tc::st16(p_at + c / 2, p);
      }
      l2 = add2(sum0, sum1);
      tc::wait_st();
    }
    tc::fence_before();
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(&sh.p_full[t]);
  }
  if (units > 0 && ok) ok = __all_sync(~0u, wait_bar(sh, a, &sh.o_done[t], 0));
  tc::fence_after();
  float l = l2.x + l2.y;
  const uint64_t bad = sh.bad;
  float* joint = reinterpret_cast<float*>(q);       // the queries' space, free once every product is done
  if (it.nt == 1) {
    // group 1 hands its maximum, sum and O over; both groups' products are done before the space is written, and both
    // take one decision when a wait has run out
    int all_ok;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, 256, p;\n selp.s32 %0, 1, 0, q;\n}"
        : "=r"(all_ok) : "r"((int)ok) : "memory");
    if (!all_ok) return;
    float* ml = joint + 128 * D;
    if (t == 1) {
      ml[lane_row] = m;
      ml[128 + lane_row] = l;
      if (warp_live && units > 0) {
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc::ld32(tmem + 256 + D + c, o);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(joint + ((c + i) / 4 * 128 + lane_row) * 4) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (t == 1) return;
  } else if (!ok) {
    return;
  }
  if (!warp_live) return;
  float f0 = 1.f, f1 = 0.f;
  bool other = false;
  if (it.nt == 1) {
    const float* ml = joint + 128 * D;
    const float m1 = ml[lane_row], l1 = ml[128 + lane_row];
    other = it.blocks > 1;
    const float both = fmaxf(m, m1);
    if (both != -INFINITY) {
      f0 = ex2(m - both);
      f1 = ex2(m1 - both);
    }
    l = l * f0 + (other ? l1 * f1 : 0.f);
    m = both;
  }
  const bool none = mask == 0 || l == 0.f;           // a pad, or a row that sees no key of the item (NaN is not none)
  const float inv = none ? 0.f : 1.f / l;
  const float lse2 = none ? -INFINITY : m + log2f(l);
#pragma unroll
  for (int c = 0; c < D; c += 32) {
    uint32_t o[32];
    if (units > 0) {
      tc::ld32(tmem + 256 + t * D + c, o);
      tc::wait_ld();
    }
    float f[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = units > 0 ? __uint_as_float(o[i]) * f0 : 0.f;
    if (other) {
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(joint + ((c + i) / 4 * 128 + lane_row) * 4);
        f[i] += v.x * f1; f[i + 1] += v.y * f1; f[i + 2] += v.z * f1; f[i + 3] += v.w * f1;
      }
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = none ? 0.f : f[i] * inv;
    if (bad && it.b >= 0) {
      for (uint64_t w = bad & mask; w; w &= w - 1) {
        const int at = it.ctx + __ffsll((long long)w) - 1;
        const int page = a.page_table[(int64_t)it.b * a.table_stride + (at >> a.c.page_shift)];
        const T* v = static_cast<const T*>(a.v_cache) + page * a.c.page_stride + it.head * a.c.head_stride +
                     (at & (a.c.page_size - 1)) * a.c.token_stride + c;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float x = Pair<T>::one(v[i]);
          if (!isfinite(x)) f[i] += x;
        }
      }
    }
    if (live) store_row<T, D>(a, it, row, lse2, f, c, 32);
  }
  if (live) {
    const int64_t at = (int64_t)row.token * a.c.q_heads + row.head;
    if (it.part >= 0) a.part_lse[(int64_t)it.part * a.plan.rows + at] = lse2;
    else if (a.lse) a.lse[at] = lse2 * 0.6931471805599453f;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_kv_attend(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<D>;
  extern __shared__ uint8_t raw[];
  __shared__ Bars sh;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5;
  const Item it = decode(a);
  grid_dependents_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) { mbar_init(&sh.full[i], 1); mbar_init(&sh.empty[i], 1); }
    for (int t = 0; t < 2; ++t) { mbar_init(&sh.s_full[t], 1); mbar_init(&sh.p_full[t], 4); mbar_init(&sh.o_done[t], 1); }
    mbar_init(&sh.q_full, kSoftmaxThreads);
    mbar_init(&sh.dirty, 1);
    mbar_init(&sh.clean, 1);
    mbar_init(&sh.drain, 1);
    sh.bad = 0;
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&sh.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp < kTmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_role<T, D>(a, it, sh, base);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTmaWarp) load_role<D>(a, it, sh, base + S::kRing, &kmap, &vmap);
    else if (warp == kMmaWarp) {
      if (tc::elect()) mma_role<T, D>(a, it, sh, base, base + S::kRing);
      __syncwarp();
    } else if (warp == kCleanWarp) clean_role<T, D>(a, it, sh, base + S::kRing);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::tmem_free(sh.tmem, 512);
}

// Joins the partial results of a row and head: a warp each.
template <typename T, int D>
__global__ void __launch_bounds__(256) k_kv_join(const __grid_constant__ AttendArgs a) {
  constexpr int N = D / 32;
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  if (at >= a.plan.rows) return;
  const int64_t token = at / a.c.q_heads;
  const int head = (int)(at - token * a.c.q_heads);
  float top = -INFINITY;
  for (int p = lane; p < a.plan.parts; p += 32) top = fmaxf(top, a.part_lse[(int64_t)p * a.plan.rows + at]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  // fmaxf drops a NaN: the sum keeps it
  float sum = 0.f, acc[N] = {};
  for (int p = 0; p < a.plan.parts; ++p) {
    const float z = a.part_lse[(int64_t)p * a.plan.rows + at];
    const float w = z == -INFINITY ? 0.f : ex2(z - (top == -INFINITY ? 0.f : top));
    sum += w;
    if (z != -INFINITY) {
      const float* o = a.part_o + ((int64_t)p * a.plan.rows + at) * D + lane * N;
      if (N == 4) {
        const float4 v = *reinterpret_cast<const float4*>(o);
        acc[0] += w * v.x; acc[1] += w * v.y; acc[N - 2] += w * v.z; acc[N - 1] += w * v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(o);
        acc[0] += w * v.x; acc[1] += w * v.y;
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* out = static_cast<T*>(a.out) + token * a.out_stride + head * D + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = Pair<T>::round(acc[i] * inv);
  if (lane == 0 && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

template <typename T, int D>
cudaError_t launch(const AttendArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s) {
  k_kv_attend<T, D><<<a.plan.items_a + a.plan.items_b, kThreads, Smem<D>::kBytes, s>>>(a, kmap, vmap);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && a.plan.parts > 1)
    e = launch_dependent(k_kv_join<T, D>, dim3((unsigned)((a.plan.rows + 7) / 8)), dim3(256), 0, s, a);
  return e;
}

template <typename T, int D>
cudaError_t prepare() {
  return cudaFuncSetAttribute(k_kv_attend<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
}

}  // namespace

cudaError_t prepare_kv_attend() {
  cudaError_t e = prepare<__nv_bfloat16, 128>();
  if (e == cudaSuccess) e = prepare<__nv_bfloat16, 64>();
  if (e == cudaSuccess) e = prepare<__half, 128>();
  if (e == cudaSuccess) e = prepare<__half, 64>();
  return e;
}

int64_t kv_attend_part_rows(int64_t rows, int num_sms) { return 3 * rows + 2LL * num_sms * 256; }

// Chooses tiles and splits from the sizes alone.  Times in units of a 128 x 128
// tile of scores and its two products: a group pair works through two tiles of
// a block in 2 units, one tile shared in 1; a block that no other item reads
// costs at least its 64 KB (D = 128) at the SM's share of the memory's rate,
// about 3 units; an item costs about 10 units before and after its blocks, the
// join of partial results about 6 and their bytes.
AttendPlan plan_kv_attend(int batch, int slots, int group, int kv_heads, int dim, int prefix_len, int max_ctx,
                          int num_sms, int64_t part_rows) {
  const int64_t R = (int64_t)slots * group, all = batch * R;
  const int np = (prefix_len + BN - 1) / BN, no = (int)(((int64_t)max_ctx + slots + BN - 1) / BN);
  AttendPlan best{};
  double best_t = 0;
  for (int packed = 0; packed < 2; ++packed) {
    if (packed && (np == 0 || batch == 1)) break;
    AttendPlan p{};
    p.rows = all * kv_heads;
    p.nt_a = all > 128 ? 2 : 1;
    p.nt_b = R > 128 ? 2 : 1;
    const int64_t tiles_a = (all + 128 * p.nt_a - 1) / (128 * p.nt_a), tiles_b = (R + 128 * p.nt_b - 1) / (128 * p.nt_b);
    const int nb = packed ? no : np + no;
    const double fill = (double)dim / 128;
    const double step_a = p.nt_a, step_b = p.nt_b > 3 * fill ? p.nt_b : (packed || np == 0 ? 3 * fill : std::max<double>(p.nt_b, 1.5 * fill));
    const int most = std::max(packed ? np : 0, nb);
    for (int len = most, last_a = 0, last_b = 0; len >= 1; len = len > 64 ? len * 15 / 16 : len - 1) {
      p.splits_a = packed ? (np + len - 1) / len : 0;
      p.splits_b = (nb + len - 1) / len;
      if (p.splits_a == last_a && p.splits_b == last_b) continue;
      last_a = p.splits_a;
      last_b = p.splits_b;
      p.parts = p.splits_a + p.splits_b;
      if (p.parts > 1 && p.parts * p.rows > part_rows) break;
      const int64_t ia = packed ? tiles_a * kv_heads * p.splits_a : 0, ib = batch * tiles_b * kv_heads * p.splits_b;
      if (ia + ib > 0x7FFFFFFF) break;
      p.items_a = (int)ia;
      p.items_b = (int)ib;
      const double da = packed ? 10 + step_a * ((np + p.splits_a - 1) / p.splits_a) : 0;
      const double db = 10 + step_b * ((nb + p.splits_b - 1) / p.splits_b);
      double t;
      if (packed) t = std::max(std::max(da, db), (ia * da + ib * db) / num_sms + 0.5 * std::min(da, db));
      else t = (double)((ib + num_sms - 1) / num_sms) * db;
      if (p.parts > 1) t += 6 + (double)p.parts * p.rows * dim * 8 / 2.0e6;
      if (best_t == 0 || t < best_t) {
        best_t = t;
        best = p;
      }
    }
  }
  return best;
}

cudaError_t launch_kv_attend(const AttendArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, int dtype,
                             cudaStream_t s) {
  if (a.c.dim == 128)
    return dtype == GRAFT_BF16 ? launch<__nv_bfloat16, 128>(a, kmap, vmap, s) : launch<__half, 128>(a, kmap, vmap, s);
  return dtype == GRAFT_BF16 ? launch<__nv_bfloat16, 64>(a, kmap, vmap, s) : launch<__half, 64>(a, kmap, vmap, s);
}

}  // namespace graft
