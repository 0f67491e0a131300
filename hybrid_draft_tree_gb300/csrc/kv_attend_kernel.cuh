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
// 2^(s-m) v, s in units of log2.  m is the maximum of the row's first keys (2^6
// below it with f16 weights) and moves only when a later one exceeds it by 2^12
// (2^15.75): until then weights above 1 are as exact as below, O, which lives in
// tensor memory, is not read and written back for every block, and the weights
// need not wait for the block's maximum.
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
//   64 x 1 behind 8192 + 1024                 58 us, 4.0 TB/s: memory, then the
//       start (4.5 us to the first scores) and the join (5 us);
//   1 x 61 behind 32768, pages of 16          44.5 us, 3.0 TB/s: the copies' issue
//       (one warp: 5.4 TB/s of 4 KB rows), start, ends and join;
//   64 x 17 behind 2048 + 777, 40/8 heads of 64, f16, pages of 16   86 us:
//       the latency from scores to weights to products (2700 cycles a unit of 128 x
//       128, two units in flight), pieces' ends (4 us each);
//   1 x 1 behind 117                           6.9 us: latency.
//
// An 8-bit cache (EIGHT): four more warps turn copied tiles into 16-bit ones; items of
// few rows go another way, in CTAs of their own (kv_few.cuh).  Scores may be capped,
// windowed or biased (SHAPED).  Measured: 8 bits, 16 x 61 behind 12001 + 2048 218 us (1.9 us
// a block of 256 rows, 1.3 of 128, by shared memory); a block of 256 rows under a window as
// without, with biases 1.9 us, capped 2.4 (small scores) to 3, both 3.6.
#pragma once
#include <algorithm>
#include <type_traits>

#include "kv_internal.cuh"
#include "tcgen05.cuh"

namespace graft {
namespace {

using namespace bulk;

constexpr int kSoftmaxThreads = 256;
// 384 threads start with 168 registers each; the softmax groups' 256 take 224, the rest keep 56: 64512 either way.  With
// the converting warps of an 8-bit cache it is 512 threads with 128, then 208 and 48: 65536 either way.
template <bool EIGHT> constexpr int kThreads = EIGHT ? 512 : 384;
template <bool EIGHT> constexpr int kSoftmaxRegs = EIGHT ? 208 : 224;
template <bool EIGHT> constexpr int kOtherRegs = EIGHT ? 48 : 56;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kSpareWarp = 10, kCleanWarp = 11, kConvertWarp = 12;
constexpr int BN = 128;                   // keys of a block
constexpr float kLog2e = 1.4426950408889634f;
// log2 of how far a maximum lies above its base when it sets it, and of how far a later one may run ahead before the base
// moves, by the weights' type.  f16 weights (f16 models, 8-bit caches) use f16's whole range: the maximum's is 2^6, what lies
// down to 2^20 below it has all of its 11 bits, and further down a weight is off by 2^-31 of it at most.  A first key that
// outweighs the rest by that much is common, and its value often next to nothing: with the base at the maximum the rest lost
// 6 bits more.  Further down still, rows whose first keys say little of their largest would move their bases in many blocks (8
// bits, 16 x 61 behind 12001 with 0, 6 and 8: 216.4, 218.0 and 225 us; f16, 64 x 17, heads of 64: 85.6, 85.8 and 89).  A sum of n
// values of at most |v| reaches 2^16 n |v|, which stays inside fp32 for f16's values and e4m3's.  bf16 weights keep their 8 bits
// at any size; 2^12 n |v| stays inside fp32 while n |v| < 2^115.
template <typename P> constexpr float kLead = std::is_same<P, __half>::value ? 6.f : 0.f;
template <typename P> constexpr float kGrow = std::is_same<P, __half>::value ? 15.75f : 12.f;

// Shared memory: two query tiles, the ring, where results pass on their way out, and the barriers.  A tile is stored in
// column halves of 64 elements (128 bytes).  With D = 128 results pass through a query tile, 4 KB a warp: a shared tile's
// through its own, those of two tiles both through the first.  No product reads the queries there any more: a group comes
// here after its last commit, which covers every product before it, and those of the second tile are issued after the
// first's.
template <int D, bool EIGHT>
struct Smem {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * 128 * 128;   // bytes of 128 rows
  static constexpr int kStages = D == 128 ? 5 : 8;    // of the ring that copies fill
  static constexpr int kRing = 2 * kTile, kStage = D == 128 ? 0 : kRing + kStages * kTile;
  static constexpr int kBars = kRing + kStages * kTile + (D == 128 ? 0 : 8 * 4096);
  static constexpr int kCopied = kTile;               // bytes of a tile as it is copied
  static constexpr int kProducts = kRing, kReady = kStages;  // the ring that the products read: the same
};
// An 8-bit cache: copies fill a ring of 8-bit tiles, from which the converting warps fill a ring of 16-bit ones for the
// products.  What is in flight from memory (64 KB) is in the first; the second holds the three tiles that products need at
// once (the values under way, the keys and the values after them) with heads of 128.
template <int D>
struct Smem<D, true> {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * 128 * 128;
  static constexpr int kCopied = 128 * D;
  static constexpr int kReady = D == 128 ? 3 : 6, kStages = D == 128 ? 4 : 8;
  static constexpr int kProducts = 2 * kTile, kRing = kProducts + kReady * kTile;
  static constexpr int kStage = D == 128 ? 0 : kRing + kStages * kCopied;
  static constexpr int kBars = kRing + kStages * kCopied + (D == 128 ? 0 : 8 * 4096);
};

// A piece of a work item, the same in every thread of its CTA.
struct Item {
  int head;            // kv head
  int b;               // request, -1: rows of all requests (prefix only)
  int row0, rows;      // first row, number of rows of the row space
  int nt;              // 128-row tiles: 2, or 1 shared by both groups
  int first, blocks;   // key blocks of the piece, prefix blocks first
  int np;              // blocks below np are the prefix's
  int skip;            // blocks before the item's first, which no slot's window reaches
  int ctx;             // tokens of the request before the tree
  int dest;            // where its rows' results go: the output, their item's partial, their CTA's partial
  bool bad_ctx;
};
constexpr int kFinal = 0, kItemPart = 1, kCtaPart = 2;

// What becomes of scores, a kernel each (what the loop over the blocks does not use costs it registers and instruction
// fetches: 19 x 61 behind 2048 under a window takes 41 us in a kernel of its own, 45 in one that can do all of it): nothing;
// windows, which the others can do too; caps up to kWide, in units of log2; slopes; caps with slopes, or of any size (with what
// the latter take 16 x 61 behind 8192 under a window of 4096 and a cap of 50 is at 158 us, 148 without; 19 x 61 over 8 bits
// behind 6144 with slopes alone at 144, 132 without).
constexpr int kPlain = 0, kWindowed = 1, kCapped = 2, kBiased = 3, kAny = 4;
constexpr float kWide = 256.f;

// The line of items.  Packed items come first, then each request's, tile by tile and head by head.  An item takes
// `fixed` units before its first block's.  An item and a block are shorter than 2^32 units together (plan_kv_attend sees to
// it; prefix, context and tree together are below 2^31 keys, so key blocks below 2^24 + 2).
struct Line {
  int64_t lo, hi;      // this CTA's part
  int64_t at;          // start of its first item
  int b, k;            // that item: request (-1: packed) and index within its request (or among the packed)
};

// With a window (items are not packed then): the whole blocks before the first key that the root sees.  Slots sit one after
// the other behind the context, so no slot sees an earlier one.
template <int SHAPED>
__device__ __forceinline__ int skip_of(const AttendArgs& a, int ctx) {
  const int low = SHAPED && a.window ? a.prefix_len + ctx - a.window + 1 : 0;
  if (low <= 0) return 0;
  return low < a.prefix_len ? low / BN : (a.prefix_len + BN - 1) / BN + (low - a.prefix_len) / BN;
}
template <int SHAPED>
__device__ __forceinline__ int blocks_of(const AttendArgs& a, int ctx) {
  return (a.plan.packed ? 0 : (a.prefix_len + BN - 1) / BN) + (ctx + a.slots + BN - 1) / BN - skip_of<SHAPED>(a, ctx);
}
__device__ __forceinline__ int ctx_of(const AttendArgs& a, int b) { return min(max(a.ctx_len[b], 0), a.max_ctx); }
__device__ __forceinline__ uint32_t cost_a(const AttendArgs& a) {
  return a.plan.fixed_a + (uint32_t)((a.prefix_len + BN - 1) / BN) * a.plan.step_a;
}
__device__ __forceinline__ uint32_t cost_b(const AttendArgs& a, int blocks) {
  return a.plan.fixed_b + (uint32_t)blocks * a.plan.step_b;
}

// Walks the pieces of a CTA.
template <int SHAPED>
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
      it.skip = 0;
      it.bad_ctx = false;
      if (!of_a) {
        const int ctx = a_.ctx_len[b_];
        it.ctx = min(max(ctx, 0), a_.max_ctx);
        it.bad_ctx = ctx != it.ctx;
        total = blocks_of<SHAPED>(a_, it.ctx);
        it.skip = skip_of<SHAPED>(a_, it.ctx);
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
  unsigned long long dirty[8], clean[8], q_ready[2], drain;
  unsigned long long bad[8];     // slots whose value holds an element that is not finite; pieces take turns
  unsigned long long bad_edge[8];  // such keys where the slots' windows begin, from the root's first on
  uint8_t q_back[256];           // an 8-bit cache's queries: exponents of their rows' factors, of a shared tile by the piece's turn
  float2 ml[2][128];             // a shared tile's maxima and sums
  Line line;
  int few_loads[4];              // blocks up to and with the last that each copying warp of few rows asked for
  int loads[2], queries;         // loads that each copying warp asked for, the last piece whose queries were
  uint32_t tmem;
  volatile uint32_t abort;
};

// Where the slots' windows begin: the root sees keys from edge_begin on, a chain's last slot from edge_end on.
__device__ __forceinline__ int edge_begin(const AttendArgs& a, const Item& it) { return a.prefix_len + it.ctx - a.window + 1; }
__device__ __forceinline__ int edge_end(const AttendArgs& a, const Item& it) { return edge_begin(a, it) + a.slots - 1; }

// Keys of block j of the item: index of the first within its segment, how many are keys.
struct Block {
  bool prefix, masked;  // masked: some row does not see all 128
  int base, valid;
  int place;            // position of the first
};
template <int SHAPED>
__device__ __forceinline__ Block block_of(const AttendArgs& a, const Item& it, int j) {
  // with slopes the nearest keys first: their scores are the largest, so that bases are set once
  const int x = (SHAPED ? it.skip : 0) + it.first + (SHAPED >= kBiased ? it.blocks - 1 - j : j);
  Block k;
  k.prefix = x < it.np;
  k.base = (k.prefix ? x : x - it.np) * BN;
  k.valid = min(BN, (k.prefix ? a.prefix_len : it.ctx + a.slots) - k.base);
  k.place = (k.prefix ? 0 : a.prefix_len) + k.base;
  k.masked = (k.prefix ? k.valid < BN : k.base + BN > it.ctx) || (SHAPED && a.window && k.place < edge_end(a, it));
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
// Tiles of a piece come as K0 V0 K1 V1 ..., but of an 8-bit cache with one row tile an item in the order in which products
// take them, K0 K1 V0 K2 V1 ... V(n-1) of n blocks: few of them are held as 16-bit numbers at a time.  The block of tile t,
// times 2, plus 1 for values; and the places of a block's keys and values.
__device__ __forceinline__ int tile_of(bool ahead, int t, int n) {
  if (!ahead || t == 0 || t == 2 * n - 1) return t;
  return t & 1 ? t + 1 : t - 1;
}
__device__ __forceinline__ int keys_at(bool ahead, int j) { return ahead && j > 0 ? 2 * j - 1 : 2 * j; }
__device__ __forceinline__ int values_at(bool ahead, int j, int n) { return ahead && j + 1 < n ? 2 * j + 2 : 2 * j + 1; }

template <int D, int L, bool EIGHT, int SHAPED>
__device__ void load_role(const AttendArgs& a, Bars& sh, uint8_t* q, uint8_t* ring, const CUtensorMap* qmap, const CUtensorMap* kmap,
                          const CUtensorMap* vmap) {
  using S = Smem<D, EIGHT>;
  constexpr int kCopies = EIGHT ? 1 : S::kHalves;           // of a page: its halves, or (8 bits) all of it
  const int lane = threadIdx.x & 31, own = L == 1 ? 0 : (threadIdx.x >> 5) != kTmaWarp;  // the warp's number
  const int pages = BN >> a.c.page_shift;                   // of a block
  const int page_bytes = a.c.page_size * (EIGHT ? D : 128);
  int loads = 0;
  uint32_t bad = 0, piece = 0;
  bool ok = true, last_two = false;
  int q_last = -1;  // the last piece whose queries were asked for
  Pieces<SHAPED> pieces(a, sh.line);
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
    const int place = lane / kCopies * L + own;
    auto page_of = [&](int j) -> int {
      const Block k = block_of<SHAPED>(a, it, j);
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
    // a tile, from this lane's page
    auto load = [&](int j, int v, int from) {
      const int stage = loads % S::kStages;
      ok = loads < S::kStages || wait_bar(sh, a, &sh.empty[stage], ((loads / S::kStages) - 1) & 1);
      ok = __all_sync(~0u, ok);
      if (!ok) return;
      if (lane == 0) mbar_expect_tx(&sh.full[stage], S::kCopied / L);  // this warp's copies
      __syncwarp();
      if (from >= 0)
        tc::tma_4d(ring + stage * S::kCopied + (lane % kCopies) * (128 * 128) + place * page_bytes, v ? vmap : kmap,
                   (lane % kCopies) * 64, 0, it.head, from, &sh.full[stage]);
      // values to clean: said once the stage's phase is this block's
      if (!EIGHT && v == 1 && lane == 0 && own == 0 && block_of<SHAPED>(a, it, j).masked) mbar_arrive(&sh.dirty[stage]);
      ++loads;
    };
    int next = page_of(0);
    // Keys and values in a loop of two, which the compiler leaves one: 64 x 1 behind 8192 + 1024 58.2 us, 59.6 unrolled; 1 x 61
    // behind 32768, pages of 16 44.6 and 43.4; 64 x 17, heads of 64, pages of 16 86.0 and 85.6.
    if (!EIGHT || two) {
      for (int j = 0; j < it.blocks && ok; ++j) {
        if (j == q_at) ok = queries();
        if (!ok) break;
        const int here = next;
        if (j + 1 < it.blocks) next = page_of(j + 1);
        for (int v = 0; v < 2 && ok; ++v) load(j, v, here);
      }
    } else {
      int last = -1, before = -1;  // pages of the last keys, and of those before: values come a block behind
      for (int x = 0; x < 2 * it.blocks && ok; ++x) {
        const int tile = tile_of(true, x, it.blocks), j = tile >> 1, v = tile & 1;
        if (x == 2 * q_at) ok = queries();
        if (!ok) break;
        if (!v) {
          before = last;
          last = next;
          if (j + 1 < it.blocks) next = page_of(j + 1);
        }
        load(j, v, v && j + 1 < it.blocks ? before : last);
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
template <int D, int L, bool EIGHT>
__device__ void drain_copies(Bars& sh) {
  constexpr int kStages = Smem<D, EIGHT>::kStages;
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
// Rows of the block with key 0 at k.place: those before `unseen` no row of the item sees, neither those from k.valid on;
// those before `edge`, and from `tree` on, some rows see and others do not.
struct Unseen { int unseen, edge, tree; };
template <int SHAPED>
__device__ __forceinline__ Unseen unseen_of(const AttendArgs& a, const Item& it, const Block& k) {
  Unseen u{0, 0, k.prefix ? k.valid : min(max(it.ctx - k.base, 0), k.valid)};
  if (SHAPED && a.window) {
    u.unseen = min(max(edge_begin(a, it) - k.place, 0), u.tree);
    u.edge = min(max(edge_end(a, it) - k.place, 0), u.tree);
  }
  return u;
}
// A row whose value is not finite everywhere: a slot of the tree, or a key that some windows hold.
template <int SHAPED>
__device__ __forceinline__ void record_bad(const AttendArgs& a, const Item& it, const Block& k, const Unseen& u, Bars& sh, int piece, int row) {
  if (!SHAPED || row >= u.tree) atomicOr(&sh.bad[piece & 7], 1ull << (k.base + row - it.ctx));
  else atomicOr(&sh.bad_edge[piece & 7], 1ull << (k.place + row - edge_begin(a, it)));
}

template <typename T, int D, int L, int SHAPED>
__device__ void clean_role(const AttendArgs& a, Bars& sh, uint8_t* ring) {
  using S = Smem<D, false>;
  constexpr int kFirst = L == 2 ? kCleanWarp : kSpareWarp, kCleaners = (kCleanWarp + 1 - kFirst) * 32;
  const int lane = threadIdx.x & 31, thread = threadIdx.x - kFirst * 32;
  constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  uint32_t turn = 0;  // a bit a stage
  int before = 0, piece = 0;
  Pieces<SHAPED> pieces(a, sh.line);
  Item it;
  for (; pieces.next(it); before += it.blocks, ++piece) {
    for (int j = 0; j < it.blocks; ++j) {
      const Block k = block_of<SHAPED>(a, it, j);
      if (!k.masked) continue;
      const int x = 2 * (before + j) + 1, stage = x % S::kStages;
      bool ok = wait_bar(sh, a, &sh.dirty[stage], (turn >> stage) & 1);
      turn ^= 1u << stage;
      ok = ok && wait_bar(sh, a, &sh.full[stage], (x / S::kStages) & 1);
      if (!__all_sync(~0u, ok)) return;
      const Unseen u = unseen_of<SHAPED>(a, it, k);
      const int end = (k.valid + a.c.page_size - 1) & -a.c.page_size;  // of the last page; zeros follow
      uint4* p = reinterpret_cast<uint4*>(ring + stage * S::kTile);
#pragma unroll 1
      for (int half = 0; half < S::kHalves; ++half, p += 128 * 8) {
        auto clean = [&](int i) {
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
            record_bad<SHAPED>(a, it, k, u, sh, piece, i >> 3);
          }
        };
#pragma unroll 4
        for (int i = u.tree * 8 + thread; i < k.valid * 8; i += kCleaners) clean(i);
#pragma unroll 4
        for (int i = k.valid * 8 + thread; i < end * 8; i += kCleaners) p[i] = make_uint4(0, 0, 0, 0);
        if (SHAPED) {
#pragma unroll 1
          for (int i = thread; i < u.unseen * 8; i += kCleaners) p[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
          for (int i = u.unseen * 8 + thread; i < u.edge * 8; i += kCleaners) clean(i);
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.clean[stage]);
    }
  }
}

// ---- an 8-bit cache's tiles and queries as f16 ones ---------------------------------------------------------------
// Tiles, a thread a row: 16 bytes at a time become 32 at the places where the products look for them.  e4m3 numbers are f16
// numbers, so nothing is rounded; the head's scales join the scores and the results.  All products over an 8-bit cache are
// of f16 numbers: the step to bf16 takes three more instructions a pair (two tiles of 128 rows 2.26 us a block, 1.9 with f16).
// Values that no row may see are made harmless on the way, as above; an e4m3 number that is not finite is a NaN.
__device__ __forceinline__ uint4 widen(uint32_t lo, uint32_t hi) {  // 8 numbers
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t two = (uint16_t)((i < 2 ? lo : hi) >> 16 * (i & 1));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w[i]) : "h"(two));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The power of two, as an exponent, that brings a row's largest magnitude next to 2^11: its bf16 numbers down to 2^-28 of
// that stay exact as f16 ones.  Rows of zeros and such as are not finite stay as they are.
__device__ __forceinline__ int up_exponent(float top) {
  const int e = (int)(__float_as_uint(top) >> 23);
  return e == 0 || e == 255 ? 127 : min(max(265 - e, 1), 253);
}
__device__ __forceinline__ float power(int exponent) { return __uint_as_float((uint32_t)exponent << 23); }

// bf16 queries as f16 ones, in place; a thread a row.
template <int D>
__device__ __forceinline__ void convert_query(uint8_t* tile, int row, uint8_t* back) {
  auto at = [&](int c) { return reinterpret_cast<uint4*>(tile + (c >> 3) * (128 * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)); };
  uint32_t most = 0;  // magnitudes compare as whole numbers
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 v = *at(c);
    most = __vmaxu2(__vmaxu2(most, v.x & 0x7FFF7FFFu), __vmaxu2(v.y & 0x7FFF7FFFu, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
  }
  const float top = __uint_as_float(max(most << 16, most & 0xFFFF0000u));
  const int up = up_exponent(top);
  const float by = power(up);
  *back = (uint8_t)(254 - up);
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 v = *at(c);
    uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = Pair<__nv_bfloat16>::get(e[i]);
      e[i] = Pair<__half>::put(p.x * by, p.y * by);
    }
    *at(c) = make_uint4(e[0], e[1], e[2], e[3]);
  }
}

// kTeams teams of warps take the tiles in turn: a tile's way through a warp is latency (a wait, loads, stores, the word to
// the products), of which there are then as many under way.
constexpr int kTeams = 2, kTeamWarps = 2;

// ---- warps 10 and 11: an 8-bit cache's bf16 queries --------------------------------------------------------------
// Warps that have nothing else to do.  When the converting warps did this beside a piece's first tiles, 16 x 61 behind
// 12001 + 2048 took 224 us, 218 so, and 19 x 12 behind 6132 80, 75 so; contexts of a block or two lose by fewer threads
// (15 x 17 behind 91 12.9 us, 13.8 so).
template <int D, int SHAPED>
__device__ void query_role(const AttendArgs& a, Bars& sh, uint8_t* q) {
  constexpr int kThreadsHere = (kCleanWarp + 1 - kSpareWarp) * 32;
  const int lane = threadIdx.x & 31, thread = threadIdx.x - kSpareWarp * 32;
  int piece = 0;
  Pieces<SHAPED> pieces(a, sh.line);
  Item it;
  for (; pieces.next(it); ++piece) {
    if (!__all_sync(~0u, wait_bar(sh, a, &sh.q_full[piece & 1], (piece >> 1) & 1))) return;
    const int tile = it.nt == 1 ? piece & 1 : 0;
    for (int r = thread; r < it.nt * 128; r += kThreadsHere)
      convert_query<D>(q + (tile + (r >> 7)) * Smem<D, true>::kTile, r & 127, &sh.q_back[tile * 128 + r]);
    tc::fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.q_ready[piece & 1]);
  }
}

// ---- warps 12-15: an 8-bit cache's tiles as 16-bit ones ----------------------------------------------------------
template <typename T, int D, int SHAPED>
__device__ void convert_role(const AttendArgs& a, Bars& sh, const uint8_t* ring, uint8_t* products) {
  using S = Smem<D, true>;
  constexpr int kChunks = D / 16, kRows = kTeamWarps * 32;  // 16-byte places of a row; rows that a team takes at a time
  const int lane = threadIdx.x & 31, team = (threadIdx.x / 32 - kConvertWarp) / kTeamWarps;
  const int first = threadIdx.x - (kConvertWarp + team * kTeamWarps) * 32;
  int before = 0, piece = 0;
  Pieces<SHAPED> pieces(a, sh.line);
  Item it;
  for (; pieces.next(it); before += 2 * it.blocks, ++piece) {
    for (int x = (team + kTeams - before % kTeams) % kTeams; x < 2 * it.blocks; x += kTeams) {
      const int tile = tile_of(it.nt == 1, x, it.blocks), v = tile & 1, number = before + x;
      const int from = number % S::kStages, to = number % S::kReady;
      Block k{};
      Unseen u{};
      bool masked = false;
      if (v) {
        k = block_of<SHAPED>(a, it, tile >> 1);
        masked = k.masked;
        if (masked) u = unseen_of<SHAPED>(a, it, k);
      }
      // Teams take the places of an odd ring in turn, so the last tile here was the other's: its word is waited for first,
      // else this wait could be over by the phase before.  A fresh barrier passes for the phase before its first.
      const uint32_t phase = (number / S::kReady) & 1;
      bool ok = number < S::kReady || wait_bar(sh, a, &sh.clean[to], phase ^ 1);
      ok = ok && wait_bar(sh, a, &sh.dirty[to], phase ^ 1);
      ok = ok && wait_bar(sh, a, &sh.full[from], (number / S::kStages) & 1);
      if (!__all_sync(~0u, ok)) return;
#pragma unroll 1
      for (int row = first; row < 128; row += kRows) {
        const bool zero = masked && (row >= k.valid || row < u.unseen), check = masked && (row >= u.tree || row < u.edge);
        const uint8_t* src = ring + from * S::kCopied + row * D;
        uint8_t* dst = products + to * S::kTile + row * 128;
        // 16-byte places are exchanged as the copies' swizzle has it: of 128-byte rows by the row's last 3 bits, of 64-byte
        // rows by bits 1 and 2
        const int turn = D == 128 ? row & 7 : (row >> 1) & 3;
        bool any = false;
#pragma unroll
        for (int c0 = 0; c0 < kChunks; c0 += 4) {
          uint4 w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const uint4*>(src + (((c0 + c) ^ turn) << 4));
          if (zero || check) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t e[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t nan = ((e[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // a bit a NaN
                any |= nan != 0;
                e[i] = zero ? 0 : e[i] & ~((nan >> 7) * 0xFF);
              }
              w[c] = make_uint4(e[0], e[1], e[2], e[3]);
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int at = 2 * (c0 + c);  // 16-byte place in the 16-bit row, 8 of them a half
            uint8_t* half = dst + (at >> 3) * (128 * 128);
            *reinterpret_cast<uint4*>(half + (((at & 7) ^ (row & 7)) << 4)) = widen(w[c].x, w[c].y);
            *reinterpret_cast<uint4*>(half + ((((at + 1) & 7) ^ (row & 7)) << 4)) = widen(w[c].z, w[c].w);
          }
        }
        if (any && check && !zero) record_bad<SHAPED>(a, it, k, u, sh, piece, row);
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.empty[from]);
        mbar_arrive(&sh.clean[to]);
      }
    }
  }
}

// ---- warp 9: the products ---------------------------------------------------------------------------------------
// One thread issues every product: its code has no warp-wide step in it.  Products run in the order they are issued, so
// the scores of a group's next block may follow its O += P V at once, although they overwrite P.
// What it does between products is on every unit's path, so it keeps the ring's places instead of computing them, and
// waits once for what both groups use.
template <typename T, int D, bool EIGHT, int SHAPED>
__device__ void mma_role(const AttendArgs& a, Bars& sh, uint8_t* q, uint8_t* ring) {
  using S = Smem<D, EIGHT>;
  constexpr bool kBf16 = !EIGHT && std::is_same<T, __nv_bfloat16>::value;  // 8-bit caches: f16, and queries made so
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
  // an 8-bit cache's tiles are told ready, and given back, by their places in the products' ring: tile number `before` + t
  unsigned long long* const ready = EIGHT ? sh.clean : sh.full;
  unsigned long long* const free = EIGHT ? sh.dirty : sh.empty;
  int before = 0, kj = 0, vj = 0;
  auto place = [](int tile, int& stage, uint32_t& phase) {
    stage = tile % S::kReady;
    phase = (tile / S::kReady) & 1;
  };
  bool ok = true;
  Pieces<SHAPED> pieces(a, sh.line);
  Item it;
  for (; ok && pieces.next(it); ++piece) {
    const bool two = it.nt == 2;
    const int units = two ? 2 * it.blocks : it.blocks;
    // masked blocks: the prefix's last when part full, and the request's own from where the tree begins
    const int part_full = !(a.prefix_len & (BN - 1)) ? -1 : it.np - 1 - it.first - (SHAPED ? it.skip : 0);
    const int tree = it.b < 0 ? INT32_MAX : it.np + it.ctx / BN - it.first - (SHAPED ? it.skip : 0);
    // ... and, up to this one, where windows begin
    int edge = 0;
    if (SHAPED && a.window) {
      const int end = edge_end(a, it);
      if (end > 0) edge = (end <= a.prefix_len ? (end + BN - 1) / BN : it.np + (end - a.prefix_len + BN - 1) / BN) - it.first - it.skip;
    }
    if (EIGHT) {
      kj = vj = 0;
      place(before, ks, kp);
      place(before + values_at(!two, 0, it.blocks), vs, vp);
    }
    // unit u is group u & 1 on key block u >> 1 (two tiles) or u (one)
    auto qk = [&](int t) -> bool {
      if ((!two || t == 0) && !wait_bar(sh, a, &ready[ks], kp)) return false;
      tc::fence_after();
      const uint64_t qa = qd + ((two ? t : piece & 1) ? kTile16 : 0), kb = kd + ks * kTile16;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t step = (k >> 2) * (128 * 128 / 16) + (k & 3) * 2;
        tc::mma_ss(tmem + t * 128, qa + step, kb + step, kQK, k > 0);
      }
      tc::commit(&sh.s_full[t]);
      if (!two || t) {
        tc::commit(&free[ks]);
        if (EIGHT) {
          place(before + keys_at(!two, ++kj), ks, kp);
        } else {
          ks += 2;
          if (ks >= S::kStages) { ks -= S::kStages; kp ^= 1; }
        }
      }
      return true;
    };
    ok = wait_bar(sh, a, EIGHT && std::is_same<T, __nv_bfloat16>::value ? &sh.q_ready[piece & 1] : &sh.q_full[piece & 1], (piece >> 1) & 1);
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
        ok = wait_bar(sh, a, &ready[vs], vp);
        int j = two ? u >> 1 : u;
        if (SHAPED >= kBiased) j = it.blocks - 1 - j;
        if (!EIGHT && ok && (j >= tree || j == part_full || (SHAPED && j < edge))) {
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
        tc::commit(&free[vs]);
        if (EIGHT) {
          place(before + values_at(!two, ++vj, it.blocks), vs, vp);
        } else {
          vs += 2;
          if (vs >= S::kStages) { vs -= S::kStages; vp ^= 1; }
        }
      }
      if (!kApart && u + 2 < units) ok = qk(t);
    }
    before += 2 * it.blocks;
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

// A row's slots in the order of its mask, and where its window begins.
struct View {
  int place;       // position of the row's own, the last slot of its mask
  int low;         // of the first key that its window holds
  uint64_t mask;   // slots that it holds
};
__device__ __forceinline__ View view_of(const AttendArgs& a, const Item& it, int token, uint64_t mask) {
  View v{0, 0, mask};
  const int seen = __popcll(mask);
  v.place = a.prefix_len + (it.b >= 0 ? it.ctx : ctx_of(a, token / a.slots)) + seen - 1;
  if (a.window) {
    v.low = v.place - a.window + 1;
    for (int n = seen - a.window; n > 0; --n) v.mask &= v.mask - 1;
  }
  return v;
}
// Bit c of w: the row sees key c of an own block, d keys before the tree (negative: it began in an earlier block).
__device__ __forceinline__ void seen_keys(int d, uint64_t mask, uint64_t& lo, uint64_t& hi) {
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

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float min_nan(float a, float b) {  // a NaN stays one
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// cap tanh(x), x = s / softcap and cap in units of log2, as factors of a product: x = s f, cap tanh(x) = s g tanh(x) / x.
// Small x: tanh(x) / x by a polynomial in x^2 (fitted to |x| <= 1/2, off by 2^-25 of it).  Others: 1 - 2 / (1 + e^2x), off by
// some 2^-22 of the cap wherever x lies, which at a half of it and above is no more than such a score's own rounding steps
// (tanh.approx is off by 2^-11).  Under caps of up to kWide the same holds of small x: there 2^-22 of the cap is 2^-14 and less.
constexpr float kSmall = 0.5f, kTanh0 = 0.017135f, kTanh1 = -0.05298607f, kTanh2 = 0.13324779f, kTanh3 = -0.33333069f;
__device__ __forceinline__ float capped(float s, float f, float g, float cap) {
  const float x = s * f, z = x * x;
  const float far = fmaf(rcp(1.f + ex2(x * (2.f * kLog2e))), -2.f * cap, cap);
  const float near = s * g * fmaf(fmaf(fmaf(fmaf(kTanh0, z, kTanh1), z, kTanh2), z, kTanh3), z, 1.f);
  return fabsf(x) <= kSmall ? near : far;
}
// A block's.  A warp whose scores are all small takes the polynomial, with f and g in its coefficients (6 multiply-adds a
// score; f^8 has to stay inside fp32: beyond caps of 2^15 the scores are x themselves).  Any other takes the exponential and a
// reciprocal: one for two scores, 1 / a = b / (a b), in 16-bit caches' heads of 128, else one for each, which takes fewer
// instructions but more of the special-function unit (19 x 61 behind 6083, pairs and each: 161 and 174 us; heads of 64 157 and
// 157, 120 and 115 under a window; 8 bits 167 and 161.  Without a cap the first takes 88, with small scores 136); under caps
// above kWide each score by its own size, so that small ones lose nothing by larger ones in the rows beside them.  An
// exponential by multiply-adds for a quarter of the scores costs more than it saves (179), and so does a reciprocal for four (8
// bits 172).  Scores of keys that a row does not see are zeros here, and rows that see nothing do not vote: neither changes the
// choice, nor the score beside it.  A NaN is then of a key that the row sees, and may spoil the one beside it.
template <int D, bool EIGHT, bool WIDE>
__device__ __forceinline__ void cap_scores(const AttendArgs& a, float to_log2, bool votes, float* s) {
  const float cap = a.softcap * kLog2e;
  float g = to_log2, f = g / cap;
  // factors of the rows' own (an 8-bit cache's queries) or beyond the coefficients' range go into the scores
  if (EIGHT || !(f > 0x1p-15f && f < 0x1p15f)) {
    g = 1.f;
    f = 1.f / cap;
#pragma unroll
    for (int c = 0; c < BN; c += 2) {
      const float2 v = mul2(make_float2(s[c], s[c + 1]), both(to_log2));
      s[c] = v.x;
      s[c + 1] = v.y;
    }
  }
  if (WIDE && !(f > 0x1p-15f)) {  // the cap is beyond 2^15: what scores are in units of it
#pragma unroll
    for (int c = 0; c < BN; c += 2) {
      const float2 v = mul2(make_float2(s[c], s[c + 1]), both(f));
      s[c] = v.x;
      s[c + 1] = v.y;
    }
    g = cap;
    f = 1.f;
  }
  float top = 0.f;
#pragma unroll
  for (int c = 0; c < BN; c += 2) top = max3(top, fabsf(s[c]), fabsf(s[c + 1]));
  if (!votes) top = 0.f;
  if (__all_sync(~0u, top * f <= kSmall) && f < 0x1p15f) {
    const float f2 = f * f, f4 = f2 * f2;
    const float2 c3 = both(g * (kTanh3 * f2)), c2 = both(g * (kTanh2 * f4)), c1 = both(g * (kTanh1 * f4 * f2)), c0 = both(g * (kTanh0 * f4 * f4));
#pragma unroll
    for (int c = 0; c < BN; c += 2) {
      const float2 v = make_float2(s[c], s[c + 1]), z = mul2(v, v);
      const float2 p = mul2(fma2(fma2(fma2(fma2(c0, z, c1), z, c2), z, c3), z, both(g)), v);
      s[c] = p.x;
      s[c + 1] = p.y;
    }
    return;
  }
  if (WIDE && cap > kWide) {
#pragma unroll
    for (int c = 0; c < BN; ++c) s[c] = capped(s[c], f, g, cap);
    return;
  }
  const float2 to_e = both(f * (2.f * kLog2e));
#pragma unroll
  for (int c = 0; c < BN; c += 2) {
    const float2 y = mul2(make_float2(s[c], s[c + 1]), to_e);
    if (EIGHT || D == 64) {
      const float2 e = add2(make_float2(ex2(y.x), ex2(y.y)), both(1.f));  // of infinity: 0
      const float2 v = fma2(make_float2(rcp(e.x), rcp(e.y)), both(-2.f * cap), both(cap));
      s[c] = v.x;
      s[c + 1] = v.y;
    } else {
      // beyond 2^60 the quotient is 0 in all of the cap's bits; the product of two stays inside fp32
      const float2 e = add2(make_float2(ex2(min_nan(y.x, 60.f)), ex2(min_nan(y.y, 60.f))), both(1.f));
      const float r = rcp(e.x * e.y) * (-2.f * cap);
      s[c] = fmaf(r, e.y, cap);
      s[c + 1] = fmaf(r, e.x, cap);
    }
  }
}
// The bias takes distances as whole numbers, of a block that lies before the row's own key from its last key on: it is no
// further off than the bias of the block's nearest key is rounded, and exact next to the row's own key whatever the slope.
// Blocks that end inside, a prefix' last among them, take each key's own distance: from a last key that is none, and lies
// behind the row's own, a steep slope would lead beyond fp32.
__device__ __forceinline__ void bias_scores(const Item& it, const Block& k, int place, uint64_t mask, float slope, float factor, float* s) {
  const int d = k.prefix ? k.valid : it.ctx - k.base;  // keys before the tree
  if (d >= BN) {
    const float near = slope * (float)(k.place + (BN - 1) - place);
#pragma unroll
    for (int c = 0; c < BN; c += 2) {
      const float2 v = fma2(make_float2(s[c], s[c + 1]), both(factor), both(near));
      s[c] = fmaf(slope, (float)(c - (BN - 1)), v.x);
      s[c + 1] = fmaf(slope, (float)(c + 1 - (BN - 1)), v.y);
    }
    return;
  }
  // slots lie as far apart as the row's mask has them
  uint64_t lo, hi;
  seen_keys(d, mask, lo, hi);
  const uint32_t w[4] = {(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  float at = (float)(k.place + (d < 0 ? d + __popcll(d > -64 ? mask & ((1ull << -d) - 1) : mask) : 0) - place);
#pragma unroll
  for (int c = 0; c < BN; ++c) {
    s[c] = fmaf(slope, at, s[c] * factor);
    at += (w[c >> 5] >> (c & 31)) & 1 ? 1.f : 0.f;
  }
}

template <typename T, int D, bool EIGHT, int SHAPED>
__device__ void softmax_role(const AttendArgs& a, Bars& sh, uint8_t* q) {
  using S = Smem<D, EIGHT>;
  using P = typename std::conditional<EIGHT, __half, T>::type;  // of the weights
  const int tid = threadIdx.x, t = tid >> 7, lane_row = tid & 127;
  const uint32_t lanes = (uint32_t)(tid & 96) << 16;   // tensor-memory lanes of this warp
  const uint32_t tmem = sh.tmem + lanes;
  uint32_t scores = 0, results = 0, piece = 0;
  bool dead = false;                                 // a wait has run out: only the barriers of both groups are left
  Pieces<SHAPED> pieces(a, sh.line);
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
  // scores in units of log2; shaped ones get there before the softmax, whose own factor is 1 then
  bool ok = !dead;
  float to_log2 = a.scale * kLog2e;
  if (EIGHT) {
    to_log2 *= kv_scale(a.k_scale, it.head, a.err);
    if (std::is_same<T, __nv_bfloat16>::value && ok) {  // queries that were made f16
      ok = __all_sync(~0u, wait_bar(sh, a, &sh.q_ready[piece & 1], (piece >> 1) & 1));
      if (ok) to_log2 *= power(sh.q_back[(it.nt == 2 ? t : piece & 1) * 128 + lane_row]);
    }
  }
  const float scale = SHAPED >= kCapped ? 1.f : to_log2;
  float slope = 0.f;
  if (SHAPED >= kBiased && live) {
    slope = SHAPED == kAny && !a.slope ? 0.f : a.slope[row.head] * kLog2e;
    if (!(fabsf(slope) < INFINITY)) {
      slope = 0.f;
      atomicOr(a.err, GRAFT_ERR_RULE);
    }
  }
  const bool warp_live = __any_sync(~0u, live);
  const int units = it.nt == 2 ? it.blocks : (it.blocks + 1 - t) >> 1;
  float m = live ? -INFINITY : 0.f;                 // lanes without a row never wait
  float2 l2 = make_float2(0.f, 0.f);
  for (int n = 0; n < units && ok; ++n) {
    const Block k = block_of<SHAPED>(a, it, it.nt == 2 ? n : 2 * n + t);
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
      uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};  // bit c: the row sees key c of the block
      if (k.masked) {
        uint64_t lo, hi;
        const View view = SHAPED ? view_of(a, it, row.token, mask) : View{0, 0, mask};
        if (k.prefix) {
          lo = k.valid >= 64 ? ~0ull : (1ull << k.valid) - 1;
          hi = k.valid >= 128 ? ~0ull : k.valid > 64 ? (1ull << (k.valid - 64)) - 1 : 0;
        } else {
          seen_keys(it.ctx - k.base, view.mask, lo, hi);
        }
        if (SHAPED && a.window && view.low > k.place) {  // a slot never precedes its place in the row's order
          const int cut = view.low - k.place;
          lo = cut >= 64 ? 0 : lo & ~0ull << cut;
          hi = cut >= 128 ? 0 : cut > 64 ? hi & ~0ull << (cut - 64) : hi;
        }
        w[0] = (uint32_t)lo; w[1] = (uint32_t)(lo >> 32); w[2] = (uint32_t)hi; w[3] = (uint32_t)(hi >> 32);
      }
      auto fill = [&](uint32_t value) {  // scores of keys that the row does not see
#pragma unroll
        for (int c = 0; c < BN; c += 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((w[c >> 5] >> i) & 1)) s[c + i] = value;
        }
      };
      if (SHAPED == kCapped || SHAPED == kAny) {
        if (k.masked) fill(0);
        cap_scores<D, EIGHT, SHAPED == kAny>(a, to_log2, live && mask != 0, reinterpret_cast<float*>(s));
      }
      if (SHAPED == kBiased || (SHAPED == kAny && a.slope))
        bias_scores(it, k, view_of(a, it, row.token, mask).place, mask, slope, SHAPED == kAny ? 1.f : to_log2, reinterpret_cast<float*>(s));
      if (k.masked) fill(0xFF800000u);  // -inf
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
          const float next = top > m + kGrow<P> ? top - kLead<P> : m;
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
            p[i / 2] = Pair<P>::put(x.x, x.y);
            p[i / 2 + 1] = Pair<P>::put(y.x, y.y);
          }
          tc::st16(p_at + c / 2, p);
        }
        if (!known || !__any_sync(~0u, live && top > m + kGrow<P>)) break;
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
  if (tid == 0) {
    sh.bad[(piece + 6) & 7] = 0;
    if (SHAPED) sh.bad_edge[(piece + 6) & 7] = 0;
  }
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
  const View view = SHAPED ? view_of(a, it, row.token, mask) : View{0, 0, mask};
  const uint64_t bad = sh.bad[piece & 7] & view.mask;
  // of the keys where the windows begin, those that the row sees
  uint64_t bad_edge = 0;
  if (SHAPED && a.window && mask) bad_edge = sh.bad_edge[piece & 7] & ~0ull << (view.low - edge_begin(a, it));
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
  const float inv = none ? 0.f : (EIGHT ? kv_scale(a.v_scale, it.head, a.err) : 1.f) / l;
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
    // elements that are not finite, of keys that the row sees
    auto add = [&](int page, int at) {
      const int64_t from = page * a.c.page_stride + it.head * a.c.head_stride + (at & (a.c.page_size - 1)) * a.c.token_stride + c;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (EIGHT) {
          if ((static_cast<const uint8_t*>(a.v_cache)[from + i] & 0x7F) == 0x7F) f[i] = NAN;
        } else {
          const float x = Pair<T>::one(static_cast<const T*>(a.v_cache)[from + i]);
          if (!isfinite(x)) f[i] += x;
        }
      }
    };
    for (uint64_t w = bad; w; w &= w - 1) {
      const int at = it.ctx + __ffsll((long long)w) - 1;
      add(a.page_table[(int64_t)it.b * a.table_stride + (at >> a.c.page_shift)], at);
    }
    if (SHAPED)
      for (uint64_t w = bad_edge; w; w &= w - 1) {
        const int x = edge_begin(a, it) + __ffsll((long long)w) - 1, at = x - a.prefix_len;
        if (at < 0) add(a.prefix_pages[x >> a.c.page_shift], x);
        else add(a.page_table[(int64_t)it.b * a.table_stride + (at >> a.c.page_shift)], at);
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
template <int THREADS, int SHAPED>
__device__ void find_line(const AttendArgs& a, Bars& sh, int64_t* sums) {
  const AttendPlan& p = a.plan;
  const int t = threadIdx.x, items = p.tiles_b * a.c.kv_heads;
  if (!p.cut) {  // an item, whole
    if (t == 0) sh.line = Line{0, INT64_MAX, 0, (int)(blockIdx.x / items), (int)(blockIdx.x % items)};
    return;
  }
  const uint32_t ca = cost_a(a);
  // packed items on a line of their own, before the CTAs of few rows
  const int cta = (int)blockIdx.x - p.split, ctas = (int)gridDim.x - p.split;
  if (cta < 0) {
    const int64_t lo = blockIdx.x * p.chunk_a, end = (int64_t)p.items_a * ca;
    const int k = (int)(lo / ca);
    if (t == 0) {
      a.line[a.batch + 1 + blockIdx.x] = -1;
      sh.line = lo < end ? Line{lo, min(lo + p.chunk_a, end), (int64_t)k * ca, -1, k} : Line{lo, lo, end, a.batch, 0};
    }
    return;
  }
  const int lane = t & 31, warp = t >> 5;
  const int per = (a.batch + THREADS - 1) / THREADS, b0 = min(a.batch, t * per), b1 = min(a.batch, b0 + per);
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += (int64_t)items * cost_b(a, blocks_of<SHAPED>(a, ctx_of(a, b)));
  int64_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  const int64_t ta = p.split ? 0 : (int64_t)p.items_a * ca;
  int64_t start = ta + upto - sum, total = ta;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) start += sums[w];
    total += sums[w];
  }
  // at least a block's length, so that every CTA between the first and the last of an item holds a piece of it
  const int64_t chunk = max((total + ctas - 1) / ctas, (int64_t)(p.split ? p.step_b : max(p.step_a, p.step_b)));
  const int64_t lo = cta * chunk;
  if (t == 0) {
    if (cta == 0) a.line[a.batch] = chunk;
    a.line[a.batch + 1 + blockIdx.x] = -1;
    const int k = lo < ta ? (int)(lo / ca) : 0;
    if (lo < ta) sh.line = Line{lo, lo + chunk, (int64_t)k * ca, -1, k};
    if (lo >= total) sh.line = Line{lo, lo, total, a.batch, 0};
  }
  const bool here = lo >= ta && lo >= start && lo < start + sum;
  if (here || cta == 0) {
    int64_t at = start;
    for (int b = b0; b < b1; ++b) {
      const uint32_t cb = cost_b(a, blocks_of<SHAPED>(a, ctx_of(a, b)));
      const int64_t c = (int64_t)items * cb;
      if (here && lo >= at && lo < at + c) {
        const int k = (int)((lo - at) / cb);
        sh.line = Line{lo, lo + chunk, at + (int64_t)k * cb, b, k};
      }
      if (cta == 0) a.line[b] = at;
      at += c;
    }
  }
}

}  // namespace
}  // namespace graft

#include "kv_few.cuh"

namespace graft {
namespace {

// EIGHT: an 8-bit cache; SHAPED: capped, windowed or biased scores.
template <typename T, int D, int L, bool EIGHT, int SHAPED>
__global__ void __launch_bounds__(kThreads<EIGHT>, 1)
    k_kv_attend(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap qmap,
                const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<D, EIGHT>;
  extern __shared__ __align__(1024) uint8_t base[];  // all of the kernel's: it starts where swizzled tiles may
  Bars& sh = *reinterpret_cast<Bars*>(base + S::kBars);
  const int warp = threadIdx.x >> 5;
  grid_dependents_launch();
  if (EIGHT && a.plan.few && (int)blockIdx.x >= a.plan.split) {
    few_cta<T, D, SHAPED>(a, sh, base, &kmap, &vmap);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sh.full[i], L);
      mbar_init(&sh.empty[i], EIGHT ? kTeamWarps : 1);
    }
    for (int i = 0; i < S::kReady; ++i) {
      mbar_init(&sh.dirty[i], 1);
      mbar_init(&sh.clean[i], EIGHT ? kTeamWarps : 3 - L);
    }
    for (int t = 0; t < 2; ++t) { mbar_init(&sh.s_full[t], 1); mbar_init(&sh.s_read[t], 4); mbar_init(&sh.p_full[t], 4); mbar_init(&sh.o_done[t], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&sh.q_full[i], 1); mbar_init(&sh.q_free[i], 8); mbar_init(&sh.q_ready[i], 2); }
    mbar_init(&sh.o_free, 8);
    mbar_init(&sh.drain, 1);
    for (int i = 0; i < 8; ++i) sh.bad[i] = sh.bad_edge[i] = 0;
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&sh.tmem, 512);
  grid_dependency_wait();
  find_line<kThreads<EIGHT>, SHAPED>(a, sh, reinterpret_cast<int64_t*>(base));
  tc::fence_async_smem();  // copies will land where the sums were
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp < kTmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs<EIGHT>));
    softmax_role<T, D, EIGHT, SHAPED>(a, sh, base);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs<EIGHT>));
    if (warp == kTmaWarp || (L == 2 && warp == kSpareWarp)) load_role<D, L, EIGHT, SHAPED>(a, sh, base, base + S::kRing, &qmap, &kmap, &vmap);
    else if (warp == kMmaWarp) {
      if (tc::elect()) mma_role<T, D, EIGHT, SHAPED>(a, sh, base, base + S::kProducts);
      __syncwarp();
    } else if (EIGHT) {
      if (warp >= kConvertWarp) convert_role<T, D, SHAPED>(a, sh, base + S::kRing, base + S::kProducts);
      else if (std::is_same<T, __nv_bfloat16>::value) query_role<D, SHAPED>(a, sh, base);
    } else clean_role<T, D, L, SHAPED>(a, sh, base + S::kRing);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (threadIdx.x == 0 && sh.abort) drain_copies<D, L, EIGHT>(sh);
  if (warp == kMmaWarp) tc::tmem_free(sh.tmem, 512);
}

template <int D, bool EIGHT>
constexpr int kSmem = Smem<D, EIGHT>::kBars + (int)sizeof(Bars);
static_assert(kSmem<64, false> <= 227 * 1024 && kSmem<128, false> <= 227 * 1024 && kSmem<64, true> <= 227 * 1024 &&
              kSmem<128, true> <= 227 * 1024, "shared memory of a CTA");

// Small pages' copies take two warps where items have one tile and blocks little else to do (8 x 1 behind 700, pages of
// 16: 12.6 us, 15.1 with one warp; 8 x 17 behind 300 + 600, heads of 64, pages of 32: 11.7 and 12.3); the ring's warps
// are in the way of more work (64 x 17 behind 2048 + 777, pages of 16: 88 us, 85.5 with one warp).  Over an 8-bit cache, whose
// pages are a copy each, one warp: the second is worth more to its queries (8 x 17 behind 300, pages of 16: 14.1 us, 16.3 with
// two; 8 x 17 behind 3000 38.5 and 41.1; 1 x 20 behind 8000, pages of 8: 24.9 and 27.2; but heads of 64, pages of 8, 8 x 17
// behind 3000: 32.4 and 31.2).
template <typename T, int D, bool EIGHT, int SHAPED>
cudaError_t launch_one(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t s) {
  auto* kernel = k_kv_attend<T, D, 1, EIGHT, SHAPED>;
  if constexpr (!EIGHT)
    if (a.c.page_size <= 32 && !a.plan.packed && a.plan.nt_b == 1) kernel = k_kv_attend<T, D, 2, EIGHT, SHAPED>;
  return launch_dependent(kernel, dim3(a.plan.ctas), dim3(kThreads<EIGHT>), kSmem<D, EIGHT>, s, a, qmap, kmap, vmap);
}
template <bool EIGHT, int SHAPED>
cudaError_t launch_form(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap, int dtype, cudaStream_t s) {
  if (a.c.dim == 128)
    return dtype == GRAFT_BF16 ? launch_one<__nv_bfloat16, 128, EIGHT, SHAPED>(a, qmap, kmap, vmap, s)
                               : launch_one<__half, 128, EIGHT, SHAPED>(a, qmap, kmap, vmap, s);
  return dtype == GRAFT_BF16 ? launch_one<__nv_bfloat16, 64, EIGHT, SHAPED>(a, qmap, kmap, vmap, s)
                             : launch_one<__half, 64, EIGHT, SHAPED>(a, qmap, kmap, vmap, s);
}

template <typename T, int D, bool EIGHT, int SHAPED>
cudaError_t prepare_one() {
  cudaError_t e = cudaFuncSetAttribute(k_kv_attend<T, D, 1, EIGHT, SHAPED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D, EIGHT>);
  if constexpr (!EIGHT)
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_kv_attend<T, D, 2, EIGHT, SHAPED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D, EIGHT>);
  return e;
}
template <bool EIGHT, int SHAPED>
cudaError_t prepare_form(int dtype, int dim) {
  if (dim == 128) return dtype == GRAFT_BF16 ? prepare_one<__nv_bfloat16, 128, EIGHT, SHAPED>() : prepare_one<__half, 128, EIGHT, SHAPED>();
  return dtype == GRAFT_BF16 ? prepare_one<__nv_bfloat16, 64, EIGHT, SHAPED>() : prepare_one<__half, 64, EIGHT, SHAPED>();
}

}  // namespace
}  // namespace graft
