// Attention of a step's slots over the paged cache (a shared prefix, each
// request's own context, the tree under its ancestor masks) on the tensor cores.
//
// A work item is up to 256 query rows of one kv head (a row is a slot and one
// of the head's query heads) against a range of key blocks of 128.  Its CTA:
//   warps 0-3, 4-7   two softmax groups, a thread a row: scores out of tensor
//                    memory, running maximum and sum, weights back into it;
//   warp 8 (and 10)  keys and values by tensor map, a page a copy, into a ring;
//   warp 9           S = Q K^T and O += P V, fp32 accumulators in tensor memory;
//   warps (10), 11   values of places that no row may see, made harmless.
// The groups alternate so that one's products run under the other's softmax.
// With more than 128 rows each group has its own 128 (every block's keys and
// values serve both); with fewer both share the rows and take the key blocks in
// turn, and their results are joined at the end.
//
// The online softmax keeps, per row, a base m, l = sum 2^(s-m) and O = sum
// 2^(s-m) v, s in units of log2.  m is the maximum of the row's first keys and
// moves only when a later one exceeds it by 2^12: until then weights above 1 are
// as exact as below, O, which lives in tensor memory, is not read and written
// back for every block, and the weights need not wait for the block's maximum.
//
// Rows of all requests against the prefix are packed into the same tiles
// ("packed"), so a prefix block is read once for up to 256 rows, when a
// request's own rows would leave a tile mostly empty; otherwise an item runs
// over prefix and own context in one pass ("joined").
//
// The items lie on a line, each as long as its key blocks cost, and every CTA
// (one an SM) takes an equal piece of the line, cut at key blocks: however
// ragged the lengths are, the SMs end together, and the ring of keys and values
// runs on from item to item.  What a cut item's pieces found (normalised O and
// log-sum-exp, fp32) is joined by a second kernel, in the order of the keys.
//
// Measured (bf16, 32/8 heads of 128 unless said otherwise), and what bounds it:
//   16 x 61 slots behind 12001 + 2048 keys   166 us, 1290 TFLOP/s (176 us in seconds
//       of it, at the power limit): a block of 256 rows takes 1.5 us, its operands'
//       way through shared memory (256 KB);
//   64 x 1 behind 8192 + 1024                 60 us, 3.9 TB/s: memory, then the
//       start (4.5 us to the first scores) and the join (5 us);
//   1 x 61 behind 32768, pages of 16          43 us, 3.1 TB/s: the copies' issue
//       (one warp: 5.4 TB/s of 4 KB rows), start, ends and join;
//   64 x 17 behind 2048 + 777, 40/8 heads of 64, f16, pages of 16   86 us:
//       the latency from scores to weights to products (2700 cycles a unit of 128 x
//       128, two units in flight), pieces' ends (4 us each);
//   1 x 1 behind 117                           6.9 us: latency.
#include <algorithm>
#include <type_traits>

#include "kv_internal.cuh"
#include "tcgen05.cuh"

namespace graft {
namespace {

using namespace bulk;

constexpr int kSoftmaxThreads = 256, kThreads = 384;
// 384 threads start with 168 registers each; the softmax groups' 256 take 224, the rest keep 56: 64512 either way
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kSpareWarp = 10, kCleanWarp = 11;
constexpr int BN = 128;                   // keys of a block
constexpr float kLog2e = 1.4426950408889634f;
// log2 of how far a maximum may run ahead of the base: weights stay inside f16.  A sum of n values of at most |v| reaches
// 2^12 n |v|, so it stays inside fp32 while n |v| < 2^115 (f16's values always do).
constexpr float kGrow = 12.f;

// Shared memory: two query tiles, the ring, where results pass on their way out, and the barriers.  A tile is stored in
// column halves of 64 elements (128 bytes).  With D = 128 results pass through a query tile, 4 KB a warp: a shared tile's
// through its own, those of two tiles both through the first.  No product reads the queries there any more: a group comes
// here after its last commit, which covers every product before it, and those of the second tile are issued after the
// first's.
template <int D>
struct Smem {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * 128 * 128;   // bytes of 128 rows
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kRing = 2 * kTile, kStage = D == 128 ? 0 : kRing + kStages * kTile;
  static constexpr int kBars = kRing + kStages * kTile + (D == 128 ? 0 : 8 * 4096);
};

// A piece of a work item, the same in every thread of its CTA.
struct Item {
  int head;            // kv head
  int b;               // request, -1: rows of all requests (prefix only)
  int row0, rows;      // first row, number of rows of the row space
  int nt;              // 128-row tiles: 2, or 1 shared by both groups
  int first, blocks;   // key blocks of the piece, prefix blocks first
  int np;              // blocks below np are the prefix's
  int ctx;             // tokens of the request before the tree
  int dest;            // where its rows' results go: the output, their item's partial, their CTA's partial
  bool bad_ctx;
};
constexpr int kFinal = 0, kItemPart = 1, kCtaPart = 2;

// The line of items.  Packed items come first, then each request's, tile by tile and head by head.  An item takes
// `fixed` units before its first block's.  An item is shorter than 2^32 units: prefix, context and tree together are below
// 2^31 keys (graft_kv_attend), so its key blocks below 2^24 + 2, of at most 152 units.
struct Line {
  int64_t lo, hi;      // this CTA's part
  int64_t at;          // start of its first item
  int b, k;            // that item: request (-1: packed) and index within its request (or among the packed)
};

__device__ __forceinline__ int blocks_of(const AttendArgs& a, int ctx) {
  return (a.plan.packed ? 0 : (a.prefix_len + BN - 1) / BN) + (ctx + a.slots + BN - 1) / BN;
}
__device__ __forceinline__ int ctx_of(const AttendArgs& a, int b) { return min(max(a.ctx_len[b], 0), a.max_ctx); }
__device__ __forceinline__ uint32_t cost_a(const AttendArgs& a) {
  return a.plan.fixed_a + (uint32_t)((a.prefix_len + BN - 1) / BN) * a.plan.step_a;
}
__device__ __forceinline__ uint32_t cost_b(const AttendArgs& a, int blocks) {
  return a.plan.fixed_b + (uint32_t)blocks * a.plan.step_b;
}

// Walks the pieces of a CTA.
class Pieces {
 public:
  __device__ Pieces(const AttendArgs& a, const Line& line) : a_(a), line_(line), at_(line.at), b_(line.b), k_(line.k) {}
  // The next piece with at least one block; false at the end of the CTA's part of the line.
  __device__ bool next(Item& it) {
    const AttendPlan& p = a_.plan;
    for (;;) {
      if (k_ == (b_ < 0 ? p.items_a : p.tiles_b * a_.c.kv_heads)) {
        k_ = 0;
        ++b_;
      }
      if (b_ >= a_.batch || (!p.cut && at_ > 0)) return false;
      const int64_t base = at_ + (b_ < 0 ? p.fixed_a : p.fixed_b), hi = line_.hi, lo = line_.lo;  // base: place of block 0
      if (base >= hi) return false;
      const int np = (a_.prefix_len + BN - 1) / BN;
      const bool of_a = b_ < 0;
      int total = np;
      it.b = b_;
      it.np = of_a || !p.packed ? np : 0;
      it.ctx = 0;
      it.bad_ctx = false;
      if (!of_a) {
        const int ctx = a_.ctx_len[b_];
        it.ctx = min(max(ctx, 0), a_.max_ctx);
        it.bad_ctx = ctx != it.ctx;
        total = blocks_of(a_, it.ctx);
      }
      it.nt = of_a ? p.nt_a : p.nt_b;
      it.rows = (of_a ? a_.batch : 1) * a_.slots * a_.group;
      const int tile = a_.by_heads.div(k_);
      it.head = k_ - tile * a_.c.kv_heads;
      it.row0 = tile * it.nt * p.tile;
      const uint32_t step = of_a ? p.step_a : p.step_b, length = total * step;
      it.first = base >= lo ? 0 : (int)(((uint32_t)(lo - base) + step - 1) / step);
      const int end = hi - base >= length ? total : (int)(((uint32_t)(hi - base) + step - 1) / step);
      it.blocks = end - it.first;
      it.dest = end < total ? kCtaPart : (it.first > 0 || p.packed ? kItemPart : kFinal);
      at_ = base + length;
      ++k_;
      if (it.blocks > 0) return true;
    }
  }

 private:
  const AttendArgs& a_;
  const Line& line_;
  int64_t at_;
  int b_, k_;
};

struct Bars {
  unsigned long long full[8], empty[8], q_full[2], q_free[2], s_full[2], s_read[2], p_full[2], o_done[2], o_free;
  unsigned long long dirty[8], clean[8], drain;
  unsigned long long bad[8];     // slots whose value holds an element that is not finite; pieces take turns
  float2 ml[2][128];             // a shared tile's maxima and sums
  Line line;
  int loads[2], queries;         // loads that each copying warp asked for, the last piece whose queries were
  uint32_t tmem;
  volatile uint32_t abort;
};

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
  // rows of all requests follow each other as those of one do: slots times the group
  const int slot = a.by_group.div(r);
  return Row{(it.b >= 0 ? it.b * a.slots : 0) + slot, it.head * a.group + r - slot * a.group};
}

__device__ __forceinline__ uint64_t mask_of(const AttendArgs& a, int token) {
  const uint64_t all = a.slots == 64 ? ~0ull : (1ull << a.slots) - 1;
  if (a.tree_mask) return a.tree_mask[token] & all;
  const int slot = token % a.slots;
  return slot == 63 ? ~0ull : (1ull << (slot + 1)) - 1;
}

// Row of a partial result: of item pieces that end their item, by row and head, packed items' and the others' apart;
// of pieces whose item goes on in the next CTA, by CTA and row of the tile.
__device__ __forceinline__ int part_row(const AttendArgs& a, int dest, bool packed, int at, int cta, int in_tile) {
  if (dest == kItemPart) return (packed ? (int)a.plan.rows : 0) + at;
  return 2 * (int)a.plan.rows + cta * 256 + in_tile;
}

// A wait that another role's abort, or the poll limit, ends; false: the item's results are void.
__device__ __forceinline__ bool wait_bar(Bars& sh, const AttendArgs& a, unsigned long long* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t limit = a.wait_polls ? a.wait_polls : SPIN;
  for (uint32_t n = 1; n < limit; ++n) {
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// ---- warp 8, and 10 with small pages: keys and values into the ring ----------------------------------------------
// L of them: a copy takes its warp some 75 cycles to issue.  Each says its own bytes of a tile to the tile's barrier, so a
// phase ends when both have spoken and all has landed, and neither can pass the other by a phase.
template <int D, int L>
__device__ void load_role(const AttendArgs& a, Bars& sh, uint8_t* q, uint8_t* ring, const CUtensorMap* qmap, const CUtensorMap* kmap,
                          const CUtensorMap* vmap) {
  using S = Smem<D>;
  const int lane = threadIdx.x & 31, own = L == 1 ? 0 : (threadIdx.x >> 5) != kTmaWarp;  // the warp's number
  const int pages = BN >> a.c.page_shift;                   // of a block; a copy is a page's half
  const int page_bytes = a.c.page_size * 128;
  int loads = 0;
  uint32_t bad = 0, piece = 0;
  bool ok = true, last_two = false;
  int q_last = -1;  // the last piece whose queries were asked for
  Pieces pieces(a, sh.line);
  Item it;
  for (; ok && pieces.next(it); ++piece) {
    if (it.bad_ctx) bad = GRAFT_ERR_RANGE;
    const bool two = it.nt == 2;
    // A shared tile takes the query tiles in turn, so its queries come while the piece before runs; two tiles wait for
    // that piece's end, after the first blocks are on their way.
    auto queries = [&]() -> bool {
      if (!a.q_map) return true;
      const uint32_t before = two || last_two ? 1 : 2;  // pieces back: the last user of the space
      if (piece >= before) {
        const uint32_t user = piece - before;
        if (!__all_sync(~0u, wait_bar(sh, a, &sh.q_free[user & 1], (user >> 1) & 1))) return false;
      }
      if (lane == 0) mbar_expect_tx(&sh.q_full[piece & 1], it.nt * S::kHalves * a.plan.tile * 128);
      __syncwarp();
      if (lane < it.nt * S::kHalves) {
        const int tile = lane / S::kHalves, half = lane % S::kHalves;
        const Row row = row_of(a, it, it.row0 + tile * a.plan.tile);
        tc::tma_3d(q + (two ? tile : piece & 1) * S::kTile + half * (128 * 128), qmap, half * 64, it.head * a.group, row.token,
                   &sh.q_full[piece & 1]);
      }
      q_last = (int)piece;
      return true;
    };
    const int q_at = own ? -1 : two && piece > 0 ? min(2, it.blocks - 1) : 0;
    // page of this lane's copy of block j: the warps take pages in turn, a page's halves side by side
    const int place = lane / S::kHalves * L + own;
    auto page_of = [&](int j) -> int {
      const Block k = block_of(a, it, j);
      if (place >= pages) return -1;
      if ((place << a.c.page_shift) >= k.valid) return a.c.num_pages;  // past the last key: zeros
      const int at = (k.base >> a.c.page_shift) + place;
      int page = k.prefix ? a.prefix_pages[at] : a.page_table[(int64_t)it.b * a.table_stride + at];
      if (page < 0 || page >= a.c.num_pages) {                // reads as zeros
        bad = GRAFT_ERR_RANGE;
        page = a.c.num_pages;
      }
      return page;
    };
    int page = page_of(0);
    for (int j = 0; j < it.blocks && ok; ++j) {
      if (j == q_at) ok = queries();
      if (!ok) break;
      const int here = page;
      if (j + 1 < it.blocks) page = page_of(j + 1);
      for (int v = 0; v < 2 && ok; ++v) {
        const int stage = loads % S::kStages;
        ok = loads < S::kStages || wait_bar(sh, a, &sh.empty[stage], ((loads / S::kStages) - 1) & 1);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&sh.full[stage], S::kTile / L);  // this warp's copies
        __syncwarp();
        if (here >= 0)
          tc::tma_4d(ring + stage * S::kTile + (lane % S::kHalves) * (128 * 128) + place * page_bytes,
                     v ? vmap : kmap, (lane % S::kHalves) * 64, 0, it.head, here, &sh.full[stage]);
        // values to clean: said once the stage's phase is this block's
        if (v == 1 && lane == 0 && own == 0 && block_of(a, it, j).masked) mbar_arrive(&sh.dirty[stage]);
        ++loads;
      }
    }
    last_two = two;
  }
  if (bad) atomicOr(a.err, bad);
  if (lane == 0) {
    sh.loads[own] = loads;
    if (own == 0) sh.queries = q_last;
  }
}

// After a wait that ran out, whoever's: the copies in flight land before the CTA ends.  Two copying warps give up apart, so
// one may have asked for loads that the other has not: the barriers of those get the missing word here.  They are fewer than
// the ring's stages, since a stage is asked for again only after its last phase, which takes both.
template <int D, int L>
__device__ void drain_copies(Bars& sh) {
  constexpr int kStages = Smem<D>::kStages;
  const int loads = L == 2 ? max(sh.loads[0], sh.loads[1]) : sh.loads[0];
  for (int x = L == 2 ? min(sh.loads[0], sh.loads[1]) : loads; x < loads; ++x) mbar_arrive(&sh.full[x % kStages]);
  for (int x = max(0, loads - kStages); x < loads; ++x) mbar_wait_drain(&sh.full[x % kStages], (x / kStages) & 1);
  for (int x = max(0, sh.queries - 1); x <= sh.queries; ++x) mbar_wait_drain(&sh.q_full[x & 1], (x >> 1) & 1);
}

// ---- warp 11, and 10 with large pages: values that no row may see ------------------------------------------------
// They must not reach a product as NaN or infinity (0 times them is NaN): rows past the last key are zeroed, and of the
// tree's rows (a key that some rows see and others do not) the elements that are not finite; their slots are recorded,
// and the rows that see them add those elements at the end.  It happens as soon as a block has landed, blocks ahead of
// its products.
template <typename T, int D, int L>
__device__ void clean_role(const AttendArgs& a, Bars& sh, uint8_t* ring) {
  using S = Smem<D>;
  constexpr int kFirst = L == 2 ? kCleanWarp : kSpareWarp, kCleaners = (kCleanWarp + 1 - kFirst) * 32;
  const int lane = threadIdx.x & 31, thread = threadIdx.x - kFirst * 32;
  constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  uint32_t turn = 0;  // a bit a stage
  int before = 0, piece = 0;
  Pieces pieces(a, sh.line);
  Item it;
  for (; pieces.next(it); before += it.blocks, ++piece) {
    for (int j = 0; j < it.blocks; ++j) {
      const Block k = block_of(a, it, j);
      if (!k.masked) continue;
      const int x = 2 * (before + j) + 1, stage = x % S::kStages;
      bool ok = wait_bar(sh, a, &sh.dirty[stage], (turn >> stage) & 1);
      turn ^= 1u << stage;
      ok = ok && wait_bar(sh, a, &sh.full[stage], (x / S::kStages) & 1);
      if (!__all_sync(~0u, ok)) return;
      const int tree = k.prefix ? k.valid : min(max(it.ctx - k.base, 0), k.valid);  // first row that is a slot
      const int end = (k.valid + a.c.page_size - 1) & -a.c.page_size;  // of the last page; zeros follow
      uint4* p = reinterpret_cast<uint4*>(ring + stage * S::kTile);
#pragma unroll 1
      for (int half = 0; half < S::kHalves; ++half, p += 128 * 8) {
#pragma unroll 4
        for (int i = tree * 8 + thread; i < k.valid * 8; i += kCleaners) {
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
            atomicOr(&sh.bad[piece & 7], 1ull << (k.base + (i >> 3) - it.ctx));
          }
        }
#pragma unroll 4
        for (int i = k.valid * 8 + thread; i < end * 8; i += kCleaners) p[i] = make_uint4(0, 0, 0, 0);
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.clean[stage]);
    }
  }
}

// ---- warp 9: the products ---------------------------------------------------------------------------------------
// One thread issues every product: its code has no warp-wide step in it.  Products run in the order they are issued, so
// the scores of a group's next block may follow its O += P V at once, although they overwrite P.
// What it does between products is on every unit's path, so it keeps the ring's places instead of computing them, and
// waits once for what both groups use.
template <typename T, int D>
__device__ void mma_role(const AttendArgs& a, Bars& sh, uint8_t* q, uint8_t* ring) {
  using S = Smem<D>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kQK = tc::instr_desc(kBf16, 128, BN, false), kPV = tc::instr_desc(kBf16, 128, D, true);
  constexpr int kTile16 = S::kTile / 16;
  // With room for P beside S (D = 64) a group's next scores are computed as soon as it has read its last ones, while it
  // turns them into weights.  A piece's first scores are computed while the last piece's results go out.
  constexpr bool kApart = D == 64;
  const uint32_t tmem = sh.tmem;
  const uint64_t qd = tc::smem_desc(smem_u32(q), 16), kd = tc::smem_desc(smem_u32(ring), 16);
  const uint64_t vd = tc::smem_desc(smem_u32(ring), 128 * 128);
  // stage and phase of the next keys and of the next values; phases of the groups' barriers, a bit each
  int ks = 0, vs = 1;
  uint32_t kp = 0, vp = 0, cleaned = 0, weights = 0, reads = 0, piece = 0;
  bool ok = true;
  Pieces pieces(a, sh.line);
  Item it;
  for (; ok && pieces.next(it); ++piece) {
    const bool two = it.nt == 2;
    const int units = two ? 2 * it.blocks : it.blocks;
    // masked blocks: the prefix's last when part full, and the request's own from where the tree begins
    const int part_full = !(a.prefix_len & (BN - 1)) ? -1 : it.np - 1 - it.first;
    const int tree = it.b < 0 ? INT32_MAX : it.np + it.ctx / BN - it.first;
    // unit u is group u & 1 on key block u >> 1 (two tiles) or u (one)
    auto qk = [&](int t) -> bool {
      if ((!two || t == 0) && !wait_bar(sh, a, &sh.full[ks], kp)) return false;
      tc::fence_after();
      const uint64_t qa = qd + ((two ? t : piece & 1) ? kTile16 : 0), kb = kd + ks * kTile16;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t step = (k >> 2) * (128 * 128 / 16) + (k & 3) * 2;
        tc::mma_ss(tmem + t * 128, qa + step, kb + step, kQK, k > 0);
      }
      tc::commit(&sh.s_full[t]);
      if (!two || t) {
        tc::commit(&sh.empty[ks]);
        ks += 2;
        if (ks >= S::kStages) { ks -= S::kStages; kp ^= 1; }
      }
      return true;
    };
    ok = wait_bar(sh, a, &sh.q_full[piece & 1], (piece >> 1) & 1);
    for (int u = 0; u < 2 && u < units && ok; ++u) ok = qk(u);
    for (int u = 0; u < units && ok; ++u) {
      const int t = u & 1;
      if (kApart && u + 2 < units) {  // the group has read its scores
        ok = wait_bar(sh, a, &sh.s_read[t], (reads >> t) & 1) && qk(t);
        reads ^= 1u << t;
        if (!ok) break;
      }
      if (u == 0 && piece > 0) ok = wait_bar(sh, a, &sh.o_free, (piece - 1) & 1);  // the last piece's results are out
      if (!ok) break;
      if (!two || t == 0) {
        ok = wait_bar(sh, a, &sh.full[vs], vp);
        const int j = two ? u >> 1 : u;
        if (ok && (j >= tree || j == part_full)) {
          ok = wait_bar(sh, a, &sh.clean[vs], (cleaned >> vs) & 1);
          cleaned ^= 1u << vs;
        }
      }
      ok = ok && wait_bar(sh, a, &sh.p_full[t], (weights >> t) & 1);
      weights ^= 1u << t;
      if (!ok) break;
      tc::fence_after();
      const uint32_t o = tmem + 256 + t * D, p = tmem + (D == 128 ? t * 128 : 384 + t * 64);
      const uint64_t vb = vd + vs * kTile16;
#pragma unroll
      for (int k = 0; k < BN / 16; ++k) tc::mma_ts(o, p + k * 8, vb + k * (16 * 128 / 16), kPV, u > 1 || k > 0);
      if (kApart || u + 2 >= units) tc::commit(&sh.o_done[t]);
      if (!two || t) {
        tc::commit(&sh.empty[vs]);
        vs += 2;
        if (vs >= S::kStages) { vs -= S::kStages; vp ^= 1; }
      }
      if (!kApart && u + 2 < units) ok = qk(t);
    }
  }
  if (!ok) {  // the products in flight finish before the tensor memory goes back
    tc::commit(&sh.drain);
    mbar_wait_drain(&sh.drain, 0);
  }
}

// ---- warps 0-7: softmax and results -----------------------------------------------------------------------------
// 32 rows of 32 columns, a row a lane, to their places: through the warp's 4 KB of shared memory, so that 8 lanes (4 of
// 16-bit output) write a row's 128 (64) bytes together.  `code`: the lane's row, of the partials (part) or as token *
// 1024 + head of the output; -1 for none.
template <typename T, int D>
__device__ __forceinline__ void store_rows(const AttendArgs& a, uint8_t* stage, int code, bool part, const float* f, int c0) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  if (part) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) =
          make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    __syncwarp();
    int at[8];
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3), c = lane & 7;
      at[i] = __shfl_sync(~0u, code, r);
      v[i] = *reinterpret_cast<const float4*>(stage + r * 128 + ((c ^ (r & 7)) << 4));
    }
    float* dst = a.part_o + c0 + (lane & 7) * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at[i] >= 0) *reinterpret_cast<float4*>(dst + (int64_t)at[i] * D) = v[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(Pair<T>::put(f[8 * i], f[8 * i + 1]), Pair<T>::put(f[8 * i + 2], f[8 * i + 3]),
                   Pair<T>::put(f[8 * i + 4], f[8 * i + 5]), Pair<T>::put(f[8 * i + 6], f[8 * i + 7]));
  __syncwarp();
  int at[4];
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2), c = lane & 3;
    at[i] = __shfl_sync(~0u, code, r);
    v[i] = *reinterpret_cast<const uint4*>(stage + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  }
  T* dst = static_cast<T*>(a.out) + c0 + (lane & 3) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (at[i] < 0) continue;
    T* p = dst + (int64_t)(at[i] >> 10) * a.out_stride + (at[i] & 1023) * D;
    if (a.out_vec) {
      *reinterpret_cast<uint4*>(p) = v[i];
    } else {
      uint16_t* h = reinterpret_cast<uint16_t*>(p);
      const uint32_t e[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[2 * k] = (uint16_t)e[k];
        h[2 * k + 1] = (uint16_t)(e[k] >> 16);
      }
    }
  }
}

template <typename T, int D>
__device__ void softmax_role(const AttendArgs& a, Bars& sh, uint8_t* q) {
  using S = Smem<D>;
  const int tid = threadIdx.x, t = tid >> 7, lane_row = tid & 127;
  const uint32_t lanes = (uint32_t)(tid & 96) << 16;   // tensor-memory lanes of this warp
  const uint32_t tmem = sh.tmem + lanes;
  const float scale = a.scale * kLog2e;
  uint32_t scores = 0, results = 0, piece = 0;
  bool dead = false;                                 // a wait has run out: only the barriers of both groups are left
  Pieces pieces(a, sh.line);
  Item it;
  for (; pieces.next(it); ++piece) {
  // queries that no tensor map can bring: elements, into the swizzled order the products read
  if (!a.q_map) {
    if (piece > 0) asm volatile("bar.sync 1, 256;" ::: "memory");  // the last results have left the queries' space
    constexpr int kPer = D / 8, kRows = kSoftmaxThreads / kPer;   // threads of a row, rows at a time
    const int c = tid % kPer;
    uint8_t* dst = q + (it.nt == 1 ? (piece & 1) * S::kTile : 0);
    for (int x = tid / kPer; x < it.nt * 128; x += kRows) {
      const int tile = x >> 7, in = x & 127, r = it.row0 + tile * a.plan.tile + in;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (in < a.plan.tile && r < it.rows) {
        const Row row = row_of(a, it, r);
        const uint16_t* h = static_cast<const uint16_t*>(a.q) + row.token * a.q_stride + row.head * D + c * 8;
        w = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
      }
      *reinterpret_cast<uint4*>(dst + tile * S::kTile + (c >> 3) * (128 * 128) + in * 128 + (((c & 7) ^ (in & 7)) << 4)) = w;
    }
    tc::fence_async_smem();
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (tid == 0) mbar_arrive(&sh.q_full[piece & 1]);
  }

  const int r = it.row0 + (it.nt == 2 ? t * a.plan.tile : 0) + lane_row;
  const bool live = lane_row < a.plan.tile && r < it.rows;
  const Row row = live ? row_of(a, it, r) : Row{0, 0};
  const uint64_t mask = live ? mask_of(a, row.token) : 0;
  const bool warp_live = __any_sync(~0u, live);
  const int units = it.nt == 2 ? it.blocks : (it.blocks + 1 - t) >> 1;
  float m = live ? -INFINITY : 0.f;                 // lanes without a row never wait
  float2 l2 = make_float2(0.f, 0.f);
  bool ok = !dead;
  for (int n = 0; n < units && ok; ++n) {
    const Block k = block_of(a, it, it.nt == 2 ? n : 2 * n + t);
    ok = __all_sync(~0u, wait_bar(sh, a, &sh.s_full[t], scores++ & 1));
    if (!ok) break;
    tc::fence_after();
    // the group's scores may be overwritten once they are in registers; nobody waits for that in the last two units
    auto read_done = [&] {
      tc::fence_before();
      __syncwarp();
      if ((tid & 31) == 0 && n + 1 < units) mbar_arrive(&sh.s_read[t]);
    };
    // ... and the products with the last weights are then still under way: they end before O or the weights change
    auto settled = [&] { return n == 0 || __all_sync(~0u, wait_bar(sh, a, &sh.o_done[t], results++ & 1)); };
    if (D == 64 && !warp_live) {
      read_done();
      if (!settled()) { ok = false; break; }
    }
    if (warp_live) {
      uint32_t s[BN];
#pragma unroll
      for (int c = 0; c < BN; c += 32) tc::ld32(tmem + t * 128 + c, s + c);
      tc::wait_ld<BN>(s);
      if (D == 64) read_done();
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
        for (int c = 0; c < BN; c += 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((w[c >> 5] >> i) & 1)) s[c + i] = 0xFF800000u;  // -inf
        }
      }
      const float* sf = reinterpret_cast<const float*>(s);
      float mx[4] = {sf[0], sf[1], sf[2], sf[3]};
#pragma unroll
      for (int c = 4; c < BN - 4; c += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], sf[c + i], sf[c + 4 + i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], sf[BN - 4 + i]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
      if (D == 64) {
        if (!settled()) { ok = false; break; }
        tc::fence_after();
      }
      // A row's first keys set its base, so the weights wait for their maximum; later the weights are computed with the
      // base there is, beside the maximum, and again if that has run away from it.
      bool known = __all_sync(~0u, m != -INFINITY);
      float2 sum0, sum1;
      for (;;) {
        if (!known) {
          const float next = top > m + kGrow ? top : m;
          const float f = next == -INFINITY ? 1.f : ex2(m - next);
          m = next;
          l2.x *= f;
          l2.y *= f;
          if (n > 0) {  // O is at rest: the products before these scores are done (D = 128: the scores came after them)
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tc::ld32(tmem + 256 + t * D + c, o);
              tc::wait_ld<32>(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tc::st32(tmem + 256 + t * D + c, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        // The sums take the weights in fp32, the product with the values takes them rounded to the cache's type: the tensor
        // cores multiply 16-bit operands, and the lower halves would take a second product of the size of the first.  The
        // result's distance from the definition is then about 1.4 times that of fp32 weights, whose result is rounded too.
        const float2 sc = make_float2(scale, scale), mb = make_float2(-base, -base);
        const uint32_t p_at = tmem + (D == 128 ? t * 128 : 384 + t * 64);
        sum0 = l2;
        sum1 = make_float2(0.f, 0.f);
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
        if (!known || !__any_sync(~0u, live && top > m + kGrow)) break;
        tc::wait_st();  // two stores to one place keep no order of their own
        known = false;
      }
      l2 = add2(sum0, sum1);
      tc::wait_st();
    }
    tc::fence_before();
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(&sh.p_full[t]);
  }
  if (units > 0 && ok) ok = __all_sync(~0u, wait_bar(sh, a, &sh.o_done[t], results++ & 1));
  float l = l2.x + l2.y;
  const bool two = it.nt == 1 && it.blocks > 1;      // two sums of one row to join
  if (it.nt == 1 && units > 0) sh.ml[t][lane_row] = make_float2(m, l);
  // the groups of a shared tile join their results, and take one decision when a wait has run out
  if (it.nt == 1) {
    int all_ok;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, 256, p;\n selp.s32 %0, 1, 0, q;\n}"
        : "=r"(all_ok) : "r"((int)ok) : "memory");
    ok = all_ok;
  }
  dead = !ok;
  if (dead) continue;
  tc::fence_after();
  if (tid == 0 && it.dest == kCtaPart && it.first == 0 && it.b >= 0)
    a.line[a.batch + 1 + blockIdx.x] = (int64_t)it.b * a.plan.tiles_b * a.c.kv_heads +
                                       it.row0 / (it.nt * a.plan.tile) * a.c.kv_heads + it.head;
  // everybody has read O of the piece before, and what belonged to those before that; cleaning is at most the ring's 4
  // blocks ahead of this one
  if (tid == 0) sh.bad[(piece + 6) & 7] = 0;
  // a warp's last words on a piece: its reads of tensor memory are over; so is its use of the queries' space
  auto read = [&] {
    tc::fence_before();
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(&sh.o_free);
  };
  auto written = [&] {
    if (D == 128) tc::fence_async_smem();
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(&sh.q_free[piece & 1]);
  };
  if (D == 64) written();                            // results do not pass through it
  if (!warp_live) {
    read();
    if (D == 128) written();
    continue;
  }
  const uint64_t bad = sh.bad[piece & 7];
  float f0 = 1.f, f1 = 0.f;
  if (it.nt == 1) {
    m = sh.ml[0][lane_row].x;
    l = sh.ml[0][lane_row].y;
  }
  if (two) {
    const float m0 = m, m1 = sh.ml[1][lane_row].x, l1 = sh.ml[1][lane_row].y;
    m = fmaxf(m0, m1);
    if (m != -INFINITY) {
      f0 = ex2(m0 - m);
      f1 = ex2(m1 - m);
    }
    l = l * f0 + l1 * f1;
  }
  const bool none = mask == 0 || l == 0.f;           // a pad, or a row that sees no key of the piece (NaN is not none)
  const float inv = none ? 0.f : 1.f / l;
  f0 *= inv;
  f1 *= inv;
  const int at = row.token * a.c.q_heads + row.head;
  const bool part = it.dest != kFinal;
  const int slot = part_row(a, it.dest, it.b < 0, at, blockIdx.x, (it.nt == 2 ? t * 128 : 0) + lane_row);
  const int code = !live ? -1 : part ? slot : row.token << 10 | row.head;
  uint8_t* stage = q + (D == 128 ? (it.nt == 1 ? (piece & 1) * S::kTile : 0) : S::kStage) + (tid >> 5) * 4096;
  // of a shared tile each group writes half of the columns
  const int c_begin = it.nt == 1 ? t * (D / 2) : 0, c_end = it.nt == 1 ? c_begin + D / 2 : D;
  const uint32_t o_at = tmem + 256 + (it.nt == 1 ? 0 : t * D);
  for (int c = c_begin; c < c_end; c += 32) {
    uint32_t o[64];
    float f[32];
    tc::ld32(o_at + c, o);
    tc::ld32(o_at + (two ? D : 0) + c, o + 32);
    tc::wait_ld<64>(o);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float x = __uint_as_float(o[i]) * f0;
      f[i] = none ? 0.f : two ? x + __uint_as_float(o[32 + i]) * f1 : x;
    }
    if (bad & mask) {
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
    if (c + 32 == c_end) read();
    store_rows<T, D>(a, stage, code, part, f, c);
  }
  if (live && (it.nt == 2 || t == 0)) {
    const float lse2 = none ? -INFINITY : m + log2f(l);
    if (part) a.part_lse[slot] = lse2;
    else if (a.lse) a.lse[at] = lse2 * 0.6931471805599453f;
  }
  if (D == 128) written();
  }
}

// Where this CTA's part of the line begins; block 0 leaves the requests' places to the join.
__device__ void find_line(const AttendArgs& a, Bars& sh, int64_t* sums) {
  const int t = threadIdx.x, items = a.plan.tiles_b * a.c.kv_heads;
  if (!a.plan.cut) {  // an item, whole
    if (t == 0) sh.line = Line{0, INT64_MAX, 0, (int)(blockIdx.x / items), (int)(blockIdx.x % items)};
    return;
  }
  const int lane = t & 31, warp = t >> 5;
  const int per = (a.batch + kThreads - 1) / kThreads, b0 = min(a.batch, t * per), b1 = min(a.batch, b0 + per);
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += (int64_t)items * cost_b(a, blocks_of(a, ctx_of(a, b)));
  int64_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  const uint32_t ca = cost_a(a);
  const int64_t ta = (int64_t)a.plan.items_a * ca;
  int64_t start = ta + upto - sum, total = ta;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) start += sums[w];
    total += sums[w];
  }
  // at least a block's length, so that every CTA between the first and the last of an item holds a piece of it
  const int64_t chunk = max((total + gridDim.x - 1) / gridDim.x, (int64_t)max(a.plan.step_a, a.plan.step_b));
  const int64_t lo = blockIdx.x * chunk;
  if (t == 0) {
    if (blockIdx.x == 0) a.line[a.batch] = chunk;
    a.line[a.batch + 1 + blockIdx.x] = -1;
    const int k = lo < ta ? (int)(lo / ca) : 0;
    if (lo < ta) sh.line = Line{lo, lo + chunk, (int64_t)k * ca, -1, k};
    if (lo >= total) sh.line = Line{lo, lo, total, a.batch, 0};
  }
  const bool here = lo >= ta && lo >= start && lo < start + sum;
  if (here || blockIdx.x == 0) {
    int64_t at = start;
    for (int b = b0; b < b1; ++b) {
      const uint32_t cb = cost_b(a, blocks_of(a, ctx_of(a, b)));
      const int64_t c = (int64_t)items * cb;
      if (here && lo >= at && lo < at + c) {
        const int k = (int)((lo - at) / cb);
        sh.line = Line{lo, lo + chunk, at + (int64_t)k * cb, b, k};
      }
      if (blockIdx.x == 0) a.line[b] = at;
      at += c;
    }
  }
}

template <typename T, int D, int L>
__global__ void __launch_bounds__(kThreads, 1)
    k_kv_attend(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap qmap,
                const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<D>;
  extern __shared__ __align__(1024) uint8_t base[];  // all of the kernel's: it starts where swizzled tiles may
  Bars& sh = *reinterpret_cast<Bars*>(base + S::kBars);
  const int warp = threadIdx.x >> 5;
  grid_dependents_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sh.full[i], L);
      mbar_init(&sh.empty[i], 1);
      mbar_init(&sh.dirty[i], 1);
      mbar_init(&sh.clean[i], 3 - L);
    }
    for (int t = 0; t < 2; ++t) { mbar_init(&sh.s_full[t], 1); mbar_init(&sh.s_read[t], 4); mbar_init(&sh.p_full[t], 4); mbar_init(&sh.o_done[t], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&sh.q_full[i], 1); mbar_init(&sh.q_free[i], 8); }
    mbar_init(&sh.o_free, 8);
    mbar_init(&sh.drain, 1);
    for (int i = 0; i < 8; ++i) sh.bad[i] = 0;
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&sh.tmem, 512);
  grid_dependency_wait();
  find_line(a, sh, reinterpret_cast<int64_t*>(base));
  tc::fence_async_smem();  // copies will land where the sums were
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp < kTmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_role<T, D>(a, sh, base);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTmaWarp || (L == 2 && warp == kSpareWarp)) load_role<D, L>(a, sh, base, base + S::kRing, &qmap, &kmap, &vmap);
    else if (warp == kMmaWarp) {
      if (tc::elect()) mma_role<T, D>(a, sh, base, base + S::kRing);
      __syncwarp();
    } else clean_role<T, D, L>(a, sh, base + S::kRing);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (threadIdx.x == 0 && sh.abort) drain_copies<D, L>(sh);
  if (warp == kMmaWarp) tc::tmem_free(sh.tmem, 512);
}

template <int D>
constexpr int kSmem = Smem<D>::kBars + (int)sizeof(Bars);

// Joins the partial results of a row and head, in the order of their keys: D / 4 lanes a row, 16 bytes a lane.  Every
// row has two items to join when items are packed; else only rows of cut items have anything to: CTA row y then is an
// item, or (by_cta, with more items than CTAs) the CTA of an item's first piece, which has said which item that is
// (line[batch + 1 + y], -1: none).  What it takes is latency: a thread asks for P partials of R rows at once.
template <typename T, int D, int R, int P>
__global__ void __launch_bounds__(256, R == 2 ? 4 : 3) k_kv_join(const __grid_constant__ AttendArgs a, int by_cta) {
  constexpr int kLanes = D / 4, kRows = 256 / kLanes;
  __shared__ int held[8];  // the CTAs that hold the first and the last piece: of the item, of the packed item, of the next
  const AttendPlan& p = a.plan;
  const int lane = threadIdx.x % kLanes, items = p.tiles_b * a.c.kv_heads;
  const int per = a.slots * a.group, rows_a = p.nt_a * p.tile, rows_b = p.nt_b * p.tile;
  int b = blockIdx.z, item = blockIdx.y;
  grid_dependency_wait();
  if (by_cta) {
    const int64_t said = a.line[a.batch + 1 + blockIdx.y];
    if (said < 0) return;
    b = (int)(said / items);
    item = (int)(said - (int64_t)b * items);
  }
  const int tile_b = a.by_heads.div(item), kv_head = item - tile_b * a.c.kv_heads;
  const int first = tile_b * rows_b + blockIdx.x * R * kRows;  // the CTA's first row of the request
  const int tile_a = p.packed ? (b * per + first) / rows_a : 0;
  if (threadIdx.x < 6) {
    const int np = (a.prefix_len + BN - 1) / BN, which = threadIdx.x >> 1;
    const int64_t chunk = a.line[a.batch];
    int64_t at;
    if (which == 0) {
      const int blocks = blocks_of(a, ctx_of(a, b));
      at = a.line[b] + (int64_t)item * cost_b(a, blocks) + p.fixed_b + (threadIdx.x & 1 ? (int64_t)(blocks - 1) * p.step_b : 0);
    } else {
      at = (int64_t)((tile_a + which - 1) * a.c.kv_heads + kv_head) * cost_a(a) + p.fixed_a;
      if (threadIdx.x & 1) at += (int64_t)(np - 1) * p.step_a;
    }
    // a CTA's number, so a product with the fp32 reciprocal is right to one
    int c = (int)((float)at * (1.f / (float)chunk));
    if ((int64_t)c * chunk > at) --c;
    if ((int64_t)(c + 1) * chunk <= at) ++c;
    held[threadIdx.x] = c;
  }
  __syncthreads();
  const int b_first = held[0], b_last = held[1];
  if (!p.packed && b_first == b_last) return;  // whole, and written
  int row[R], token[R], head[R], in_a[R], a_first[R], na[R], n[R], most = 0;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    row[k] = (blockIdx.x * R + k) * kRows + threadIdx.x / kLanes;
    const int in_b = tile_b * rows_b + row[k];
    n[k] = na[k] = in_a[k] = a_first[k] = 0;
    token[k] = head[k] = 0;
    if (in_b >= per || row[k] >= rows_b) continue;
    const int slot = a.by_group.div(in_b);
    token[k] = b * a.slots + slot;
    head[k] = kv_head * a.group + in_b - slot * a.group;
    if (p.nt_b == 2 && row[k] >= p.tile) row[k] += 128 - p.tile;  // place in its CTA's partial
    if (p.packed) {
      in_a[k] = b * per + in_b - tile_a * rows_a;
      const bool next = in_a[k] >= rows_a;
      if (next) in_a[k] -= rows_a;
      if (p.nt_a == 2 && in_a[k] >= p.tile) in_a[k] += 128 - p.tile;
      a_first[k] = held[next ? 4 : 2];
      na[k] = held[next ? 5 : 3] - a_first[k] + 1;
    }
    n[k] = na[k] + b_last - b_first + 1;
    most = max(most, n[k]);
  }
  const float* parts = a.part_o + lane * 4;
  float top[R], sum[R];
  float4 acc[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    top[k] = -INFINITY;
    sum[k] = 0.f;
    acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int i0 = 0; i0 < most; i0 += P) {
    float z[R][P];
    float4 v[R][P];
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int i = i0 + j;
        z[k][j] = -INFINITY;
        if (i >= n[k]) continue;
        const bool of_a = i < na[k];
        const int cta = of_a ? a_first[k] + i : b_first + i - na[k];
        const bool last = of_a ? i == na[k] - 1 : cta == b_last;
        const int r = part_row(a, last ? kItemPart : kCtaPart, of_a, token[k] * a.c.q_heads + head[k], cta, of_a ? in_a[k] : row[k]);
        z[k][j] = a.part_lse[r];
        v[k][j] = *reinterpret_cast<const float4*>(parts + (int64_t)r * D);
      }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float next = top[k];
#pragma unroll
      for (int j = 0; j < P; ++j) next = fmaxf(next, z[k][j]);  // drops a NaN: the sum keeps it
      const float base = next == -INFINITY ? 0.f : next, f = ex2(top[k] - base);
      sum[k] *= f;
      acc[k].x *= f; acc[k].y *= f; acc[k].z *= f; acc[k].w *= f;
      top[k] = next;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if (z[k][j] == -INFINITY) continue;
        const float w = ex2(z[k][j] - base);
        sum[k] += w;
        acc[k].x += w * v[k][j].x; acc[k].y += w * v[k][j].y; acc[k].z += w * v[k][j].z; acc[k].w += w * v[k][j].w;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (n[k] == 0) continue;
    const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
    T* out = static_cast<T*>(a.out) + token[k] * a.out_stride + head[k] * D + lane * 4;
    const uint2 w = make_uint2(Pair<T>::put(acc[k].x * inv, acc[k].y * inv), Pair<T>::put(acc[k].z * inv, acc[k].w * inv));
    if (a.out_vec) {
      *reinterpret_cast<uint2*>(out) = w;
    } else {
      uint16_t* h = reinterpret_cast<uint16_t*>(out);
      h[0] = (uint16_t)w.x; h[1] = (uint16_t)(w.x >> 16); h[2] = (uint16_t)w.y; h[3] = (uint16_t)(w.y >> 16);
    }
    if (lane == 0 && a.lse)
      a.lse[token[k] * a.c.q_heads + head[k]] = sum[k] == 0.f ? -INFINITY : (top[k] + log2f(sum[k])) * 0.6931471805599453f;
  }
}

template <typename T, int D>
cudaError_t launch(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                   cudaStream_t s) {
  const AttendPlan& p = a.plan;
  // Small pages' copies take two warps where items have one tile and blocks little else to do (8 x 1 behind 700, pages of
  // 16: 12.6 us, 15.1 with one warp; 8 x 17 behind 300 + 600, heads of 64, pages of 32: 11.7 and 12.3); the ring's warps
  // are in the way of more work (64 x 17 behind 2048 + 777, pages of 16: 88 us, 85.5 with one warp).
  const bool two_loaders = a.c.page_size <= 32 && !p.packed && p.nt_b == 1;
  cudaError_t e = launch_dependent(two_loaders ? k_kv_attend<T, D, 2> : k_kv_attend<T, D, 1>, dim3(p.ctas), dim3(kThreads),
                                   kSmem<D>, s, a, qmap, kmap, vmap);
  if (e == cudaSuccess && p.cut) {
    // many rows have few partials each: two rows a thread take 167 us where one takes 174 (16 x 61 behind 12001, with the
    // main kernel), 86 and 91 (64 x 17, heads of 64), but 51 where one takes 43 (1 x 61 behind 32768).  Between, behind
    // 4000 keys: 29.9 and 28.1 at 5856 rows, 30.9 and 31.1 at 7808, 33.9 and 33.5 at 9760, 42.9 and 44.9 at 15616.
    const bool many = p.rows > 8192;
    const int rows = std::min(a.slots * a.group, p.nt_b * p.tile), items = p.tiles_b * a.c.kv_heads;
    const int each = (many ? 2 : 1) * 1024 / D;
    const bool by_cta = !p.packed && (int64_t)items * a.batch > p.ctas;
    const dim3 grid = by_cta ? dim3((rows + each - 1) / each, p.ctas) : dim3((rows + each - 1) / each, items, a.batch);
    e = many ? launch_dependent(k_kv_join<T, D, 2, 2>, grid, dim3(256), 0, s, a, (int)by_cta)
             : launch_dependent(k_kv_join<T, D, 1, 8>, grid, dim3(256), 0, s, a, (int)by_cta);
  }
  return e;
}

template <typename T, int D>
cudaError_t prepare() {
  const cudaError_t e = cudaFuncSetAttribute(k_kv_attend<T, D, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D>);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(k_kv_attend<T, D, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D>);
}

}  // namespace

cudaError_t prepare_kv_attend() {
  cudaError_t e = prepare<__nv_bfloat16, 128>();
  if (e == cudaSuccess) e = prepare<__nv_bfloat16, 64>();
  if (e == cudaSuccess) e = prepare<__half, 128>();
  if (e == cudaSuccess) e = prepare<__half, 64>();
  return e;
}

int64_t kv_attend_part_rows(int64_t rows, int num_sms) { return 2 * rows + (int64_t)num_sms * 256; }

// Chooses between packed and joined items, and between cut and whole ones, from the sizes alone: of the contexts it knows
// the bound, and a loose one costs what the wrong form does (1 x 1 behind 100: 6.8 us, 10.0 with a bound of 4096; 16 x 61
// behind 500: 19.6, 19.9 with 4096, 33.7 with 32768; 64 x 17 behind 2048 + 100: 81 with any).  Costs are in
// units of 10 ns, measured on one SM: a key block of 128 against two tiles of 128 rows, against one, and the least a block
// takes when its keys and values come from memory (the SM's share of the copy rate) or from L2, where other items' SMs
// read them too; before its first block an item pays for its queries, and the pipeline's start and end.
// Both sides, in us: packed 60 and joined 226 (64 x 1 behind 8192 + 1024), 86 and 100 (64 x 17 behind 2048 + 777, heads
// of 64), 179 and 167 (16 x 61 behind 12001 + 2048); two tiles and one 167 and 195 in the last, 43 and 61 (1 x 61 behind
// 32768); whole and cut 6.9 and 10.4 (1 x 1 behind 117).
AttendPlan plan_kv_attend(int batch, int slots, int group, int kv_heads, int dim, int prefix_len, int max_ctx,
                          int num_sms) {
  const int64_t R = (int64_t)slots * group, all = batch * R;
  const int np = (prefix_len + BN - 1) / BN, no = (int)(((int64_t)max_ctx + slots + BN - 1) / BN);
  const bool wide = dim == 128;
  const int two = wide ? 152 : 130, one = wide ? 85 : 130, fixed_two = wide ? 650 : 400, fixed_one = wide ? 280 : 450;
  const int memory = wide ? 120 : 65, l2 = wide ? 70 : 35;
  AttendPlan best{};
  double best_t = 0;
  for (int packed = 0; packed < 2; ++packed) {
    if (packed && (np == 0 || batch == 1)) break;
    AttendPlan p{};
    p.packed = packed;
    p.rows = all * kv_heads;
    p.tile = group <= 128 ? 128 / group * group : 128;
    p.nt_a = all > p.tile ? 2 : 1;
    p.nt_b = R > p.tile ? 2 : 1;
    p.tiles_b = (int)((R + p.tile * p.nt_b - 1) / (p.tile * p.nt_b));
    p.items_a = packed ? (int)((all + p.tile * p.nt_a - 1) / (p.tile * p.nt_a)) * kv_heads : 0;
    p.step_a = std::max(p.nt_a == 2 ? two : one, l2);
    p.fixed_a = p.nt_a == 2 ? fixed_two : fixed_one;
    p.fixed_b = p.nt_b == 2 ? fixed_two : fixed_one;
    // the share of an item's blocks that no other item reads
    const int blocks = packed ? no : np + no;
    const double alone = packed || batch == 1 ? 1.0 : (double)no / blocks;
    p.step_b = std::max(p.nt_b == 2 ? two : one, (int)(p.tiles_b > 1 ? l2 : l2 + alone * (memory - l2)));
    const int64_t items_b = (int64_t)batch * p.tiles_b * kv_heads;
    const double whole = p.fixed_b + (double)blocks * p.step_b;
    const double work = p.items_a * (p.fixed_a + (double)np * p.step_a) + items_b * whole;
    const double join = 400 + (double)(p.rows * (packed ? 2 : 1) + num_sms * 256) * dim * 8 / 50000;
    double t = work / num_sms + p.fixed_b + join;
    p.cut = 1;
    p.ctas = num_sms;
    // With few items the costs of a busy machine are off by `off`: whole and cut are level at 500 keys for 1 x 61 slots (14.8
    // us; at 1000 whole takes 20.5, cut 16.0), at 1000 for 1 x 1 (12.2; at 500 9.0 and 11.3), at 1900 for 8 x 1 (21).
    // On both sides of these points (1 x 1 and 61, 2 x 61, 4 x 4, 8 x 1 and 17, 32/8 heads of 64 and 128, 52 sizes) the rule
    // takes the faster form but for 1 x 61 at 600 (16.3, cut 14.8), 4 x 4 at 1500 (15.8 and 14.6) and two level ones.
    const int off = p.nt_b == 2 ? (wide ? -400 : -200) : (wide ? -100 : 200);
    if (!packed && items_b <= num_sms && whole <= t + off) {
      p.cut = 0;
      p.ctas = (int)items_b;
      t = whole;
    }
    if (best_t == 0 || t < best_t) {
      best_t = t;
      best = p;
    }
  }
  return best;
}

cudaError_t launch_kv_attend(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, int dtype, cudaStream_t s) {
  if (a.c.dim == 128)
    return dtype == GRAFT_BF16 ? launch<__nv_bfloat16, 128>(a, qmap, kmap, vmap, s) : launch<__half, 128>(a, qmap, kmap, vmap, s);
  return dtype == GRAFT_BF16 ? launch<__nv_bfloat16, 64>(a, qmap, kmap, vmap, s) : launch<__half, 64>(a, qmap, kmap, vmap, s);
}

}  // namespace graft
