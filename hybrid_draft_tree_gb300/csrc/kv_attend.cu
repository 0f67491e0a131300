// Attention over a cache in the model's type with plain scores; the join of cut items' pieces, and the choice of how a
// call's work is laid out, for every form.
#include "kv_attend_kernel.cuh"

namespace graft {
namespace {

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
    const int64_t chunk = which && p.split ? p.chunk_a : a.line[a.batch];
    int64_t at;
    if (which == 0) {
      const int blocks = blocks_of<true>(a, ctx_of(a, b));
      at = a.line[b] + (int64_t)item * cost_b(a, blocks) + p.fixed_b + (threadIdx.x & 1 ? (int64_t)(blocks - 1) * p.step_b : 0);
    } else {
      at = (int64_t)((tile_a + which - 1) * a.c.kv_heads + kv_head) * cost_a(a) + p.fixed_a;
      if (threadIdx.x & 1) at += (int64_t)(np - 1) * p.step_a;
    }
    // a CTA's number, so a product with the fp32 reciprocal is right to one
    int c = (int)((float)at * (1.f / (float)chunk));
    if ((int64_t)c * chunk > at) --c;
    if ((int64_t)(c + 1) * chunk <= at) ++c;
    held[threadIdx.x] = which ? c : c + p.split;
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
cudaError_t join(const AttendArgs& a, cudaStream_t s) {
  const AttendPlan& p = a.plan;
  // many rows have few partials each: two rows a thread take 167 us where one takes 174 (16 x 61 behind 12001, with the
  // main kernel), 86 and 91 (64 x 17, heads of 64), but 51 where one takes 43 (1 x 61 behind 32768).  Between, behind
  // 4000 keys: 29.9 and 28.1 at 5856 rows, 30.9 and 31.1 at 7808, 33.9 and 33.5 at 9760, 42.9 and 44.9 at 15616.
  const bool many = p.rows > 8192;
  const int rows = std::min(a.slots * a.group, p.nt_b * p.tile), items = p.tiles_b * a.c.kv_heads;
  const int each = (many ? 2 : 1) * 1024 / D;
  const bool by_cta = !p.packed && (int64_t)items * a.batch > p.ctas;
  const dim3 grid = by_cta ? dim3((rows + each - 1) / each, p.ctas) : dim3((rows + each - 1) / each, items, a.batch);
  return many ? launch_dependent(k_kv_join<T, D, 2, 2>, grid, dim3(256), 0, s, a, (int)by_cta)
           : launch_dependent(k_kv_join<T, D, 1, 8>, grid, dim3(256), 0, s, a, (int)by_cta);
}

}  // namespace

const AttendForm kAttendPlain = {prepare_form<false, kPlain>, launch_form<false, kPlain>};

namespace {
const AttendForm* const kForms[2][5] = {
    {&kAttendPlain, &kAttendWindowed, &kAttendCapped, &kAttendBiased, &kAttendAny},
    {&kAttendEightPlain, &kAttendEightWindowed, &kAttendEightCapped, &kAttendEightBiased, &kAttendEightAny}};
}  // namespace

int kv_attend_form(const float* slope, float softcap, int window) {
  if (softcap > 0.f) return slope || softcap * kLog2e > kWide ? kAny : kCapped;
  return slope ? kBiased : window > 0 ? kWindowed : kPlain;
}
cudaError_t prepare_kv_attend(int form, int dtype, int dim, bool eight) { return kForms[eight][form]->prepare(dtype, dim); }

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
//
// The kernels hold an item's length in 32 bits.  Where costs of 10 ns would pass them (some 1.8e9 keys and more, at up to 300
// a block), the plan that is chosen counts in a larger unit.
AttendPlan plan_kv_attend(int batch, int slots, int group, int kv_heads, int dim, int prefix_len, int max_ctx,
                          int window, bool eight, bool capped, int num_sms) {
  const int64_t R = (int64_t)slots * group, all = batch * R;
  const int np = (prefix_len + BN - 1) / BN, no = (int)(((int64_t)max_ctx + slots + BN - 1) / BN);
  const bool wide = dim == 128;
  int two = wide ? 152 : 130, one = wide ? 85 : 130, fixed_two = wide ? 650 : 400, fixed_one = wide ? 280 : 450;
  int memory = wide ? 120 : 65, l2 = wide ? 70 : 35;
  const bool few = eight && R <= 16;
  const int step_few = R <= 8 ? (wide ? 47 : 29) : (wide ? 61 : 41), fixed_few = 280;
  const int item_few = R <= 8 ? 260 : wide ? 720 : 600, busy_few = R <= 8 ? (wide ? 67 : 40) : (wide ? 74 : 31);
  if (eight) {
    two = wide ? 190 : 140;
    one = wide ? 125 : 115;
    memory = wide ? 75 : 40;
    l2 = wide ? 40 : 20;
  }
  if (capped) {
    two += wide ? 110 : 120;
    one += wide ? 60 : 65;
  }
  AttendPlan best{};
  double best_t = 0;
  for (int packed = 0; packed < 2; ++packed) {
    if (packed && (np == 0 || batch == 1 || window)) break;
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
    int blocks = packed ? no : np + no;
    if (window) blocks = std::min(blocks, (int)(((int64_t)window + slots + BN - 1) / BN) + 1);
    const double alone = packed || batch == 1 ? 1.0 : (double)no / blocks;
    p.few = few ? (R > 8 ? 2 : 1) : 0;
    if (few) p.fixed_b = fixed_few;
    p.step_b = std::max(few ? step_few : p.nt_b == 2 ? two : one, (int)(p.tiles_b > 1 ? l2 : l2 + alone * (memory - l2)));
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
    if (few && packed) {
      // As many CTAs for the packed items as end with the others.  Beside CTAs that keep memory busy both are slower than
      // alone: what the packed ones pay before and after their blocks was 9 to 27 us, an item of the others up to 8 rows 2.6 us
      // and 0.67 a block, up to 16 rows 7.2 and 0.74 (heads of 64 6 and 0.3: it waits for its queries where the other asks for
      // them ahead).  In us, by the number of CTAs for the packed items:
      //   64 x 1 behind 8192 + 1024, 32/8 heads of 128   55.8 with 40, 57.3 with 47 (the rule), 55.3 with 60, 72 with 30, 64 with 80
      //   16 x 1 behind 8192 + 4000                      41.8 with 40 or 60, 42.7 with 55 (the rule), 62 with 30 or 80
      //   64 x 1 behind 8192 + 100, heads of 64          29.6 with 70, 36.4 with 96 (the rule), 44 with 30
      //   64 x 1 behind 2000 + 4000, heads of 64         58.5 with 10, 67 with 7 (the rule), 71 with 40
      //   64 x 3 behind 8192 + 1024                      97.3 with 50, 96.6 with 60 (the rule 57), 136 with 30, 110 with 80
      //   the same, heads of 64                          60.0 with 70 (the rule 69), 72 with 50, 66 with 80
      //   64 x 4 behind 8192 + 100                       81 with 80, 97 with 60 or 100 (the rule 90)
      //   16 x 3 behind 8192 + 2000                      47.2 with 70, 51.6 with 80 (the rule 78), 71 with 50
      const double line = p.items_a * (p.fixed_a + (double)np * p.step_a);
      double best_end = 0;
      for (int n = 1; n < num_sms; ++n) {
        const double end = std::max(line / n + 2000, items_b * (item_few + (double)blocks * busy_few) / (num_sms - n));
        if (best_end == 0 || end < best_end) {
          best_end = end;
          p.split = n;
        }
      }
      t = best_end + join;
    }
    if (best_t == 0 || t < best_t) {
      best_t = t;
      best = p;
    }
  }
  // an item's length and a block more, which a place is rounded up by
  auto longest = [&](int64_t fixed, int64_t step) { return fixed + ((int64_t)np + no + 1) * step; };
  while (std::max(longest(best.fixed_a, best.step_a), longest(best.fixed_b, best.step_b)) > UINT32_MAX)
    for (int32_t* cost : {&best.fixed_a, &best.step_a, &best.fixed_b, &best.step_b}) *cost = (*cost + 1) / 2;
  if (best.split) {
    const int64_t line = best.items_a * (best.fixed_a + (int64_t)np * best.step_a);
    best.chunk_a = std::max((line + best.split - 1) / best.split, (int64_t)best.step_a);
  }
  return best;
}

cudaError_t launch_kv_attend(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, int dtype, cudaStream_t s) {
  const int form = kv_attend_form(a.slope, a.softcap, a.window);
  const cudaError_t e = kForms[a.c.eight != 0][form]->launch(a, qmap, kmap, vmap, dtype, s);
  if (e != cudaSuccess || !a.plan.cut) return e;
  if (a.c.dim == 128) return dtype == GRAFT_BF16 ? join<__nv_bfloat16, 128>(a, s) : join<__half, 128>(a, s);
  return dtype == GRAFT_BF16 ? join<__nv_bfloat16, 64>(a, s) : join<__half, 64>(a, s);
}

}  // namespace graft
