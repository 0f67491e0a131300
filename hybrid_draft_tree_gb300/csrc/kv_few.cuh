// Attention over an 8-bit cache where a kv head has few query rows (at most 16: a token or two of a request): part of the
// attention kernel, in CTAs of their own.
//
// What bounds it is the cache's bytes, so nothing is staged twice: copies fill a ring of blocks of 128 keys and their
// values, 128 KB in flight, and eight warps take 16 keys of a block each straight from it into the operands of
// mma.m16n8k16: an e4m3 number becomes an f16 one in registers, exactly.  The tiles of tcgen05 are 128 rows high, of which
// 4 or 8 would be in use, and its operands would have to be written back to shared memory as 16-bit numbers first: 1.9 us a
// block (heads of 128, bf16) where the copies take 0.75.
//   scores   S^T = K Q^T: keys are the rows of the first operand, as they lie in memory, query rows the columns;
//   weights  f16, turned over by movmatrix;
//   results  O^T += V^T P^T: a lane holds 16 consecutive d of its four keys, whose bytes are paired up by key.
// The order of d within a product is free as long as both operands have the same, and so is that of the keys: both are
// taken so that a lane's share is 16 consecutive bytes, and lanes that read together read other banks.
//
// A warp keeps a base, a sum and O of its own for each row; the base moves as in the other
// kernel, so there is no exchange between lanes in the loop.  Warps are joined at the piece's end, in their order.
// bf16 queries become f16 ones as in the other kernel.
#pragma once

namespace graft {
namespace {

template <int D>
struct FewSmem {
  static constexpr int kCopied = 128 * D, kBlock = 2 * kCopied, kStages = D == 128 ? 4 : 8, kMerge = kStages * kBlock;
  static constexpr int kLoaders = 4;  // warps; each owns every fourth block, so every fourth stage
};
constexpr int kFewWarps = 8;

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t turn_over(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t halves(uint32_t two) {  // the e4m3 numbers in the low 16 bits as f16
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}

// Lane's 8 bytes or 16 of a row: word i.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  }
}

// Blocks into the ring.
template <int D, int SHAPED>
__device__ void few_load(const AttendArgs& a, Bars& sh, uint8_t* ring, const CUtensorMap* kmap, const CUtensorMap* vmap, int loader) {
  using S = FewSmem<D>;
  const int lane = threadIdx.x & 31, place = lane & 15, pages = BN >> a.c.page_shift;
  int number = 0, mine = 0;
  uint32_t bad = 0;
  bool ok = true;
  Pieces<SHAPED> pieces(a, sh.line);
  Item it;
  for (; ok && pieces.next(it); number += it.blocks) {
    if (it.bad_ctx) bad = GRAFT_ERR_RANGE;
    for (int j = (loader - number) & (S::kLoaders - 1); j < it.blocks && ok; j += S::kLoaders) {
      const int n = number + j, stage = n % S::kStages;
      const Block k = block_of<SHAPED>(a, it, j);
      int page = -1;
      if (place < pages) {
        page = a.c.num_pages;  // past the last key: zeros
        if ((place << a.c.page_shift) < k.valid) {
          const int at = (k.base >> a.c.page_shift) + place;
          page = k.prefix ? a.prefix_pages[at] : a.page_table[(int64_t)it.b * a.table_stride + at];
          if (page < 0 || page >= a.c.num_pages) {
            bad = GRAFT_ERR_RANGE;
            page = a.c.num_pages;
          }
        }
      }
      ok = n < S::kStages || wait_bar(sh, a, &sh.empty[stage], ((n / S::kStages) - 1) & 1);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      if (lane == 0) mbar_expect_tx(&sh.full[stage], S::kBlock);
      __syncwarp();
      if (page >= 0)
        tc::tma_4d(ring + stage * S::kBlock + (lane >> 4) * S::kCopied + place * a.c.page_size * D, lane >> 4 ? vmap : kmap, 0, 0, it.head,
                   page, &sh.full[stage]);
      mine = n + 1;
    }
  }
  if (bad) atomicOr(a.err, bad);
  if (lane == 0) sh.few_loads[loader] = mine;
}
// After a wait that ran out: copies in flight land before the CTA ends.
template <int D>
__device__ void few_drain(Bars& sh) {
  using S = FewSmem<D>;
  for (int w = 0; w < S::kLoaders; ++w)
    for (int n = sh.few_loads[w] - 1, i = 0; n >= 0 && i < S::kStages / S::kLoaders; n -= S::kLoaders, ++i)
      mbar_wait_drain(&sh.full[n % S::kStages], (n / S::kStages) & 1);
}

template <typename T, int D, int NT, int SHAPED>
__device__ void few_compute(const AttendArgs& a, Bars& sh, const uint8_t* ring, float2* merge) {
  using S = FewSmem<D>;
  constexpr int kSteps = D / 16, kHalf = D / 64, kWords = D / 32;  // products over d; 64-byte parts of a key; words of a lane's values
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  // the keys that a lane's rows of the first operand are: g and g + 8 of the warp's 16 in an order in which lanes that read
  // together (two g, four t) read other banks; their values lie with the lanes t = g / 2
  auto key_of = [](int x) { return x ^ (x & 1) << 2; };
  const int key = warp * 16 + key_of(g);
  int value[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) value[i] = warp * 16 + key_of(2 * t + (i & 1)) + 8 * (i >> 1);
  auto chunk = [](int row, int c) { return row * D + ((c ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4); };
  uint64_t* const masks = reinterpret_cast<uint64_t*>(sh.ml[1]);  // of the piece's rows, for the joint
  int number = 0, piece = 0;
  Pieces<SHAPED> pieces(a, sh.line);
  // With 8 rows the next piece and its queries are asked for before the last one's results are joined (what a piece costs
  // beside its blocks is the way to these and back: 3.2 -> 1.6 us); with 16 there are no registers left for that (16 x 4
  // behind 4096 + 1024: 34 us, 41 with it).
  Item it, next;
  uint2 raw[NT][kSteps];
  float k_scale = 1.f, v_scale = 1.f;
  auto fetch = [&]() -> bool {
    if (!pieces.next(next)) return false;
    k_scale = kv_scale(a.k_scale, next.head, a.err);
    v_scale = kv_scale(a.v_scale, next.head, a.err);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      const bool live = r < next.rows;
      const Row row = live ? row_of(a, next, r) : Row{0, 0};
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + row.token * a.q_stride + row.head * D;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int d = 16 * (t + 4 * (s >> 2)) + 4 * (s & 3);
        raw[nt][s] = make_uint2(0, 0);
        if (live) {
          if (a.q_map) raw[nt][s] = *reinterpret_cast<const uint2*>(src + d);
          else raw[nt][s] = make_uint2(src[d] | src[d + 1] << 16, src[d + 2] | src[d + 3] << 16);
        }
      }
    }
    return true;
  };
  for (bool more = fetch(); more; ++piece) {
    it = next;
    const float to_log2 = a.scale * kLog2e * k_scale, to_value = v_scale;
    // rows 2t and 2t + 1 of a tile of 8, whose scores and results this lane holds; and row g, whose queries it holds
    uint32_t qf[NT][kSteps][2];
    float f[NT][2], m[NT][2], l[NT][2], slope[NT][2], o[NT][kSteps][4];
    uint64_t mask[NT][2];
    View view[NT][2];
    if (tid < 16) masks[tid] = tid < it.rows ? mask_of(a, row_of(a, it, tid).token) : 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[kSteps][4], top = 0.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint2 w = raw[nt][s];
        const float2 lo = Pair<T>::get(w.x), hi = Pair<T>::get(w.y);
        x[s][0] = lo.x; x[s][1] = lo.y; x[s][2] = hi.x; x[s][3] = hi.y;
        if (std::is_same<T, __half>::value) {
          qf[nt][s][0] = w.x;
          qf[nt][s][1] = w.y;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(x[s][i]));
        }
      }
      float back = 1.f;
      if (!std::is_same<T, __half>::value) {
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const int up = up_exponent(top);
        const float by = power(up);
        back = power(254 - up);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          qf[nt][s][0] = Pair<__half>::put(x[s][0] * by, x[s][1] * by);
          qf[nt][s][1] = Pair<__half>::put(x[s][2] * by, x[s][3] * by);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rr = nt * 8 + 2 * t + i;
        const bool on = rr < it.rows;
        const Row own = on ? row_of(a, it, rr) : Row{0, 0};
        f[nt][i] = __shfl_sync(~0u, back, (2 * t + i) * 4) * to_log2;
        m[nt][i] = on ? -INFINITY : 0.f;
        l[nt][i] = 0.f;
        mask[nt][i] = on ? mask_of(a, own.token) : 0;
        view[nt][i] = View{0, 0, mask[nt][i]};
        slope[nt][i] = 0.f;
        if (SHAPED && on) {
          view[nt][i] = view_of(a, it, own.token, mask[nt][i]);
          if (SHAPED >= kBiased) {
            slope[nt][i] = SHAPED == kAny && !a.slope ? 0.f : a.slope[own.head] * kLog2e;
            if (!(fabsf(slope[nt][i]) < INFINITY)) {
              slope[nt][i] = 0.f;
              atomicOr(a.err, GRAFT_ERR_RULE);
            }
          }
        }
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][s][i] = 0.f;
    }
    const float cap = SHAPED ? a.softcap * kLog2e : 0.f, of_cap = SHAPED && a.softcap > 0.f ? 1.f / cap : 0.f;
    // A block's words are read ahead: its keys under the softmax of the block before, its values under its own scores.
    uint32_t kw[kHalf][2][4], vw[4][kWords];
    auto wait_block = [&](int n) { return (bool)__all_sync(~0u, wait_bar(sh, a, &sh.full[n % S::kStages], (n / S::kStages) & 1)); };
    auto load_keys = [&](int n) {
      const uint8_t* keys = ring + n % S::kStages * S::kBlock;
#pragma unroll
      for (int h = 0; h < kHalf; ++h) {
        load_words<4>(keys + chunk(key, t + 4 * h), kw[h][0]);
        load_words<4>(keys + chunk(key + 8, t + 4 * h), kw[h][1]);
      }
    };
    auto load_values = [&](int n) {
      const uint8_t* values = ring + n % S::kStages * S::kBlock + S::kCopied;
#pragma unroll
      for (int i = 0; i < 4; ++i) load_words<kWords>(values + chunk(value[i], D == 128 ? g : g >> 1) + (D == 128 ? 0 : (g & 1) * 8), vw[i]);
    };
    bool ok = wait_block(number);
    if (ok) load_keys(number);
    for (int j = 0; j < it.blocks && ok; ++j, ++number) {
      const int stage = number % S::kStages;
      const Block k = block_of<SHAPED>(a, it, j);
      load_values(number);
      // two sums, of every other product, so that a product waits for the one before the last
      float s[NT][4], s1[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = s1[nt][i] = 0.f;
#pragma unroll
      for (int x = 0; x < kSteps; ++x) {
        const uint32_t w0 = kw[x >> 2][0][x & 3], w1 = kw[x >> 2][1][x & 3];
        const uint32_t a0 = halves(w0), a1 = halves(w1), a2 = halves(w0 >> 16), a3 = halves(w1 >> 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(x & 1 ? s1[nt] : s[nt], a0, a1, a2, a3, qf[nt][x][0], qf[nt][x][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] += s1[nt][i];
      if (j + 1 < it.blocks) {
        ok = wait_block(number + 1);
        if (!ok) break;
        load_keys(number + 1);
      }
      // s[nt][2 c + i]: key c of the lane's two, row i
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (SHAPED == kCapped || SHAPED == kAny) s[nt][i] = capped(s[nt][i], f[nt][i & 1] * of_cap, f[nt][i & 1], cap);
          else s[nt][i] *= f[nt][i & 1];
        }
      if (SHAPED == kBiased || (SHAPED == kAny && a.slope)) {
        const int d = k.prefix ? BN : it.ctx - k.base;  // keys before the tree
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = key + 8 * (i >> 1);
            int at = k.place + c;
            // slots lie as far apart as the row's mask has them
            if (c > d) at = k.place + d + __popcll(c - d >= 64 ? mask[nt][i & 1] : mask[nt][i & 1] & ((1ull << (c - d)) - 1));
            s[nt][i] = fmaf(slope[nt][i & 1], (float)(at - view[nt][i & 1].place), s[nt][i]);
          }
      }
      if (k.masked) {
        const Unseen u = unseen_of<SHAPED>(a, it, k);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = key + 8 * (i >> 1), node = c - u.tree;
            bool on = c < k.valid;
            if (node >= 0 && !k.prefix) on = on && view[nt][i & 1].mask >> (k.base + c - it.ctx) & 1;
            if (SHAPED && a.window) on = on && k.place + c >= view[nt][i & 1].low;
            if (!on) s[nt][i] = -INFINITY;
          }
        // values that no row sees, and numbers that are not finite where some do and others do not (an e4m3 one is a NaN)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = value[i];
          const bool zero = c >= k.valid || c < u.unseen, check = c >= u.tree || c < u.edge;
          bool any = false;
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            const uint32_t nan = ((vw[i][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            if (zero) {
              vw[i][w] = 0;
            } else if (check && nan) {
              vw[i][w] &= ~((nan >> 7) * 0xFF);
              any = true;
            }
          }
          if (any) record_bad<SHAPED>(a, it, k, u, sh, piece, c);
        }
      }
      bool grown = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) grown = grown || s[nt][i] > m[nt][i & 1] + kGrow<__half>;
      if (__any_sync(~0u, grown)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(s[nt][i], s[nt][2 + i]);
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
            const float next = top > m[nt][i] + kGrow<__half> ? top - kLead<__half> : m[nt][i];
            const float by = next == -INFINITY || next == m[nt][i] ? 1.f : ex2(m[nt][i] - next);
            m[nt][i] = next;
            l[nt][i] *= by;
#pragma unroll
            for (int x = 0; x < kSteps; ++x) {
              o[nt][x][i] *= by;
              o[nt][x][2 + i] *= by;
            }
          }
      }
      uint32_t b[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float base0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], base1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
        const float p0 = ex2(s[nt][0] - base0), p1 = ex2(s[nt][1] - base1), p2 = ex2(s[nt][2] - base0), p3 = ex2(s[nt][3] - base1);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        b[nt][0] = turn_over(Pair<__half>::put(p0, p1));
        b[nt][1] = turn_over(Pair<__half>::put(p2, p3));
      }
#pragma unroll
      for (int w = 0; w < kWords; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = __byte_perm(vw[0][w], vw[1][w], h ? 0x7362 : 0x5140), y = __byte_perm(vw[2][w], vw[3][w], h ? 0x7362 : 0x5140);
          const uint32_t a0 = halves(x), a1 = halves(x >> 16), a2 = halves(y), a3 = halves(y >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][2 * w + h], a0, a1, a2, a3, b[nt][0], b[nt][1]);
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[stage]);
    }
    if (NT == 1) more = ok && fetch();
    // the warps' results, by lane and product: element 2 x (+ 1) of the lane's D / 8, of row 2t (+ 1)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        for (int x = 4; x < 32; x <<= 1) l[nt][i] += __shfl_xor_sync(~0u, l[nt][i], x);
        if (g == 0) sh.ml[0][warp * 16 + nt * 8 + 2 * t + i] = make_float2(m[nt][i], l[nt][i]);
#pragma unroll
        for (int x = 0; x < kSteps; ++x) merge[(((warp * NT + nt) * kSteps + x) * 2 + i) * 33 + lane] = make_float2(o[nt][x][i], o[nt][x][2 + i]);
      }
    }
    int all_ok;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, 256, p;\n selp.s32 %0, 1, 0, q;\n}"
        : "=r"(all_ok) : "r"((int)ok) : "memory");
    if (!all_ok) return;
    if (tid == 0) {
      if (it.dest == kCtaPart && it.first == 0)
        a.line[a.batch + 1 + blockIdx.x] = (int64_t)it.b * a.plan.tiles_b * a.c.kv_heads + it.head;
      // everybody has read those of the piece before; loaded blocks are cleaned when they are computed, so none of a later
      // piece has been recorded
      sh.bad[(piece + 6) & 7] = 0;
      if (SHAPED) sh.bad_edge[(piece + 6) & 7] = 0;
    }
    for (int x = tid; x < it.rows * (D / 2); x += kFewWarps * 32) {
      const int r = x / (D / 2), d = 2 * (x - r * (D / 2)), nt = r >> 3;
      constexpr int kRun = D / 8;  // elements that a lane holds side by side
      const int from = ((nt * kSteps + d % kRun / 2) * 2 + (r & 1)) * 33 + d / kRun * 4 + (r & 7) / 2;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, sh.ml[0][w * 16 + r].x);
      const float base = top == -INFINITY ? 0.f : top;
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const float2 ml = sh.ml[0][w * 16 + r];
        const float by = ex2(ml.x - base);
        const float2 v = merge[w * NT * kSteps * 66 + from];
        sum += ml.y * by;
        acc.x += v.x * by;
        acc.y += v.y * by;
      }
      const Row row = row_of(a, it, r);
      const uint64_t own = masks[r];
      const bool none = own == 0 || sum == 0.f;
      const float inv = none ? 0.f : to_value / sum;
      acc.x = none ? 0.f : acc.x * inv;
      acc.y = none ? 0.f : acc.y * inv;
      View view = View{0, 0, own};
      if (SHAPED) view = view_of(a, it, row.token, own);
      auto add = [&](int page, int at) {
        const uint8_t* v = static_cast<const uint8_t*>(a.v_cache) + page * a.c.page_stride + it.head * a.c.head_stride +
                           (at & (a.c.page_size - 1)) * a.c.token_stride + d;
        if ((v[0] & 0x7F) == 0x7F) acc.x = NAN;
        if ((v[1] & 0x7F) == 0x7F) acc.y = NAN;
      };
      for (uint64_t w = sh.bad[piece & 7] & view.mask; w; w &= w - 1) {
        const int at = it.ctx + __ffsll((long long)w) - 1;
        add(a.page_table[(int64_t)it.b * a.table_stride + (at >> a.c.page_shift)], at);
      }
      if (SHAPED && a.window && own)
        for (uint64_t w = sh.bad_edge[piece & 7] & ~0ull << (view.low - edge_begin(a, it)); w; w &= w - 1) {
          const int p = edge_begin(a, it) + __ffsll((long long)w) - 1, at = p - a.prefix_len;
          if (at < 0) add(a.prefix_pages[p >> a.c.page_shift], p);
          else add(a.page_table[(int64_t)it.b * a.table_stride + (at >> a.c.page_shift)], at);
        }
      const int at = row.token * a.c.q_heads + row.head;
      const float lse2 = none ? -INFINITY : top + log2f(sum);
      if (it.dest != kFinal) {
        const int slot = part_row(a, it.dest, false, at, blockIdx.x, r);
        *reinterpret_cast<float2*>(a.part_o + (int64_t)slot * D + d) = acc;
        if (d == 0) a.part_lse[slot] = lse2;
      } else {
        uint16_t* out = static_cast<uint16_t*>(a.out) + row.token * a.out_stride + row.head * D + d;
        const uint32_t w = Pair<T>::put(acc.x, acc.y);
        if (a.out_vec) {
          *reinterpret_cast<uint32_t*>(out) = w;
        } else {
          out[0] = (uint16_t)w;
          out[1] = (uint16_t)(w >> 16);
        }
        if (d == 0 && a.lse) a.lse[at] = lse2 * 0.6931471805599453f;
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");  // what is joined has been read
    if (NT > 1) more = fetch();
  }
}

template <typename T, int D, int SHAPED>
__device__ void few_cta(const AttendArgs& a, Bars& sh, uint8_t* base, const CUtensorMap* kmap, const CUtensorMap* vmap) {
  using S = FewSmem<D>;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kFewWarps);
    }
    for (int i = 0; i < 8; ++i) sh.bad[i] = sh.bad_edge[i] = 0;
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  grid_dependency_wait();
  find_line<kThreads<true>, SHAPED>(a, sh, reinterpret_cast<int64_t*>(base));
  tc::fence_async_smem();  // copies will land where the sums were
  __syncthreads();
  if (warp < kFewWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    float2* merge = reinterpret_cast<float2*>(base + S::kMerge);
    if (a.plan.few == 1) few_compute<T, D, 1, SHAPED>(a, sh, base, merge);
    else few_compute<T, D, 2, SHAPED>(a, sh, base, merge);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp < kFewWarps + S::kLoaders) few_load<D, SHAPED>(a, sh, base, kmap, vmap, warp - kFewWarps);
  }
  __syncthreads();
  if (threadIdx.x == 0 && sh.abort) few_drain<D>(sh);
}

static_assert(FewSmem<128>::kMerge + kFewWarps * 2 * 8 * 66 * 8 <= Smem<128, true>::kBars, "the joint's space");
static_assert(FewSmem<64>::kMerge + kFewWarps * 2 * 4 * 66 * 8 <= Smem<64, true>::kBars, "the joint's space");

}  // namespace
}  // namespace graft
