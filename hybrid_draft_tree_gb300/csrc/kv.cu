// C ABI of the paged-cache calls (graft_kv_*): handle, argument checks and launches.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>

#include <nvtx3/nvToolsExt.h>

#include "kv_internal.cuh"

struct graft_kv {
  graft_kv_config cfg;
  graft::KvLayout layout;
  int device = 0, num_sms = 0;
  uint32_t* err = nullptr;      // [1]
  float* part_o = nullptr;      // [part_rows][head_dim] partial results of the attention
  float* part_lse = nullptr;    // [part_rows]
  int64_t* line = nullptr;      // [max_batch + 1 + SMs]
  int64_t part_rows = 0;
  uint32_t wait_polls = 0;
  int32_t axes = 1;             // of positions that the caller gives
  uint8_t pair_axis[64] = {0};  // axis whose position turns a pair
  uint32_t prepared = 0;        // forms of the attention, a bit each
  int32_t last_launches = 0;
  char msg[256] = {0};
};

namespace {

using graft::misaligned;

constexpr int32_t kMaxKeys = 0x7FFFFFFF - 256;  // of a row: key counts rounded up to blocks stay below 2^31

int fail(graft_kv* h, int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(h->msg, sizeof h->msg, fmt, ap);
  va_end(ap);
  return code;
}

int cuda_fail(graft_kv* h, cudaError_t e, const char* what) {
  return fail(h, GRAFT_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

int check_cfg(const graft_kv_config* c, graft_kv* h) {
  if (c->kv_heads < 1 || c->q_heads < 1 || c->q_heads % c->kv_heads != 0 || c->q_heads > 1024)
    return fail(h, GRAFT_EINVAL, "q_heads must be a multiple of kv_heads, both in [1, 1024]");
  if (c->head_dim != 64 && c->head_dim != 128) return fail(h, GRAFT_EINVAL, "head_dim must be 64 or 128");
  if (c->rot_dim < 0 || c->rot_dim > c->head_dim || c->rot_dim % 2 != 0)
    return fail(h, GRAFT_EINVAL, "rot_dim must be even and in [0, head_dim]");
  if (c->rot_interleaved != 0 && c->rot_interleaved != 1) return fail(h, GRAFT_EINVAL, "rot_interleaved must be 0 or 1");
  const int ps = c->page_size;
  if (ps < 8 || ps > 128 || (ps & (ps - 1)) != 0) return fail(h, GRAFT_EINVAL, "page_size must be 8, 16, 32, 64 or 128");
  if (c->num_pages < 1 || (int64_t)c->num_pages * ps > 0x7FFFFFFF)
    return fail(h, GRAFT_EINVAL, "num_pages * page_size must be in [1, 2^31)");
  if (c->max_slots < 1 || c->max_slots > graft::MAX_S) return fail(h, GRAFT_EINVAL, "max_slots must be in [1, 64]");
  if (c->max_batch < 1 || (int64_t)c->max_batch * c->max_slots > 65535)
    return fail(h, GRAFT_EINVAL, "max_batch * max_slots must be in [1, 65535]");
  const int type = c->dtype & ~GRAFT_CACHE_E4M3, piece = c->dtype & GRAFT_CACHE_E4M3 ? 16 : 8;
  if (type != GRAFT_BF16 && type != GRAFT_F16)
    return fail(h, GRAFT_EINVAL, "dtype must be GRAFT_BF16 or GRAFT_F16, for an 8-bit cache with GRAFT_CACHE_E4M3");
  const int64_t D = c->head_dim, T = c->token_stride, H = c->head_stride, P = c->page_stride;
  const int64_t top = (int64_t)1 << 38;  // bytes of a stride stay below 2^40
  if (T < D || H < D || P < D || T % piece != 0 || H % piece != 0 || P % piece != 0 || T >= top || H >= top || P >= top)
    return fail(h, GRAFT_EINVAL, "strides must be multiples of 8 elements (16 of an 8-bit cache), at least head_dim and below 2^38");
  // tokens, heads and pages nest in the order of their strides, whichever that is: each steps over all that lies within
  struct Axis { int64_t stride, count; };
  Axis axes[3] = {{T, ps}, {H, c->kv_heads}, {P, c->num_pages}};
  std::sort(axes, axes + 3, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
  int64_t extent = D;
  for (const Axis& x : axes) {
    if (x.count == 1) continue;
    if (x.stride < extent) return fail(h, GRAFT_EINVAL, "the strides make tokens, heads or pages overlap");
    extent = x.count - 1 > top / x.stride ? top : extent + (x.count - 1) * x.stride;  // top: no further stride reaches it
  }
  return GRAFT_OK;
}

int check_cache(graft_kv* h, const void* k, const void* v) {
  if (!k || !v) return fail(h, GRAFT_EINVAL, "null pointer");
  if (misaligned(k, 16) || misaligned(v, 16)) return fail(h, GRAFT_EINVAL, "a cache buffer is not aligned to 16 bytes");
  return GRAFT_OK;
}

// Scales and scores of the calls that take them.
int check_scales(graft_kv* h, const graft_kv_scales* s) {
  if (!s) return GRAFT_OK;
  if (!h->layout.eight && (s->d_k_scale || s->d_v_scale)) return fail(h, GRAFT_EINVAL, "only 8-bit caches have scales");
  if (misaligned(s->d_k_scale, 4) || misaligned(s->d_v_scale, 4))
    return fail(h, GRAFT_EINVAL, "a buffer is not aligned to its element size");
  return GRAFT_OK;
}
int check_scores(graft_kv* h, const graft_kv_scores* s, float scale) {
  if (!s) return GRAFT_OK;
  if (!(s->softcap >= 0.f) || !std::isfinite(s->softcap) || s->window < 0)
    return fail(h, GRAFT_EINVAL, "softcap must be finite and >= 0, window >= 0");
  // the score in units of the cap, and the cap in those of the exponential, in fp32
  if (s->softcap > 0.f && (!std::isfinite(4.f * scale / s->softcap) || !std::isfinite(4.f * s->softcap) || 4.f * s->softcap < 1e-30f))
    return fail(h, GRAFT_EINVAL, "softcap %g is too far from scale %g", s->softcap, scale);
  if (misaligned(s->d_slope, 4)) return fail(h, GRAFT_EINVAL, "a buffer is not aligned to its element size");
  return GRAFT_OK;
}

// Work goes to the device that holds the workspace, which has to be the current one.
int check_device(graft_kv* h) {
  int device = -1;
  if (cudaGetDevice(&device) != cudaSuccess || device != h->device)
    return fail(h, GRAFT_EINVAL, "the handle is of device %d, the current one is %d", h->device, device);
  return GRAFT_OK;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up through the runtime (the library links no libcuda).
EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// A cache buffer as [page][kv head][token][d]; a copy is 64 elements of one page's tokens of one head, in rows of 128
// bytes under the 128-byte swizzle; of an 8-bit cache all of a head's elements, in rows of 128 or 64 bytes under theirs.
bool cache_map(const graft::KvLayout& c, int dtype, const void* base, CUtensorMap* map) {
  const cuuint64_t size = c.eight ? 1 : 2;
  const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride * size, (cuuint64_t)c.head_stride * size, (cuuint64_t)c.page_stride * size};
  const cuuint32_t box[4] = {c.eight ? (cuuint32_t)c.dim : 64, (cuuint32_t)c.page_size, 1, 1}, step[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type = c.eight ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : dtype == GRAFT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const EncodeTiled encode = encoder();
  return encode && encode(map, type, 4, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          c.eight && c.dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as [token][head][d]; a copy is 64 elements of one group's heads of as many tokens as make a row tile.
bool query_map(const graft::KvLayout& c, int dtype, const void* base, int64_t tokens, int64_t stride, int group, CUtensorMap* map) {
  const cuuint64_t dims[3] = {(cuuint64_t)c.dim, (cuuint64_t)c.q_heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)c.dim * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(128 / group)}, step[3] = {1, 1, 1};
  const EncodeTiled encode = encoder();
  return encode && encode(map, dtype == GRAFT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                          const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

void free_all(graft_kv* h) {
  cudaFree(h->err);
  cudaFree(h->part_o);
  cudaFree(h->part_lse);
  cudaFree(h->line);
}

// The kernels of a form are loaded when a handle first needs them: the plain form's with the handle, a shaped one's in its
// first call, which may be under capture (a process' first handle takes 1.2 ms so over 16-bit caches and 1.6 over 8-bit ones; with
// every form of every type and head size 4.5 and 23).
cudaError_t prepare(graft_kv* h, int form) {
  if (h->prepared >> form & 1) return cudaSuccess;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return e;
  e = graft::prepare_kv_attend(form, h->cfg.dtype, h->layout.dim, h->layout.eight != 0);
  const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e == cudaSuccess) e = back;
  if (e == cudaSuccess) h->prepared |= 1u << form;
  return e;
}

// graft_kv_append and graft_kv_append_ext
int append(graft_kv* h, int32_t batch, int32_t slots, const void* d_q, int64_t q_stride, const void* d_k, int64_t k_stride,
           const void* d_v, int64_t v_stride, const int32_t* d_depth, const int32_t* d_rows, const int32_t* d_position,
           const float* d_rope, int32_t rope_len, int32_t prefix_len, const int32_t* d_page_table, int32_t table_stride,
           const int32_t* d_ctx_len, void* d_q_out, int64_t q_out_stride, void* d_k_cache, void* d_v_cache,
           const graft_kv_scales* scales, void* stream) {
  if (!h) return GRAFT_EINVAL;
  h->last_launches = 0;
  const graft::KvLayout& c = h->layout;
  if (batch < 0 || slots < 1 || (int64_t)batch * slots > 0x7FFFFFFF)
    return fail(h, GRAFT_EINVAL, "batch %d and slots %d: batch >= 0, slots >= 1, batch * slots < 2^31", batch, slots);
  if (prefix_len < 0 || rope_len < 0 || table_stride < 0)
    return fail(h, GRAFT_EINVAL, "prefix_len, rope_len and table_stride must be >= 0");
  if (batch == 0) return GRAFT_OK;
  if (!d_k || !d_v || !d_page_table || !d_ctx_len || (c.rot > 0 && !d_rope)) return fail(h, GRAFT_EINVAL, "null pointer");
  if (!d_q != !d_q_out) return fail(h, GRAFT_EINVAL, "d_q and d_q_out go together");
  if (const int rc = check_cache(h, d_k_cache, d_v_cache)) return rc;
  if (const int rc = check_scales(h, scales)) return rc;
  const int64_t qw = (int64_t)c.q_heads * c.dim, kw = (int64_t)c.kv_heads * c.dim;
  if (k_stride < kw || v_stride < kw || (d_q && (q_stride < qw || q_out_stride < qw)))
    return fail(h, GRAFT_EINVAL, "a row stride is less than the row");
  if (misaligned(d_q, 2) || misaligned(d_q_out, 2) || misaligned(d_k, 2) || misaligned(d_v, 2) ||
      misaligned(d_depth, 4) || misaligned(d_rows, 4) || misaligned(d_position, 4) || misaligned(d_rope, 4) || misaligned(d_page_table, 4) ||
      misaligned(d_ctx_len, 4))
    return fail(h, GRAFT_EINVAL, "a buffer is not aligned to its element size");
  graft::AppendArgs a{};
  a.c = c;
  a.batch = batch; a.slots = slots;
  a.q = d_q; a.k = d_k; a.v = d_v;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride; a.q_out_stride = q_out_stride;
  a.depth = d_depth; a.rows = d_rows; a.rope = d_rope; a.rope_len = rope_len; a.prefix_len = prefix_len;
  a.page_table = d_page_table; a.table_stride = table_stride; a.ctx_len = d_ctx_len;
  a.q_out = d_q_out; a.k_cache = d_k_cache; a.v_cache = d_v_cache;
  a.err = h->err;
  a.position = d_position; a.tokens = (int64_t)batch * slots; a.axes = h->axes;
  std::memcpy(a.pair_axis, h->pair_axis, sizeof a.pair_axis);
  const int per = c.interleaved ? 4 : 8;
  for (int i = 0; d_position && i < c.rot / 2; i += per) {
    uint64_t axis = a.pair_axis[i];
    for (int j = 1; j < per && i + j < c.rot / 2; ++j) axis = a.pair_axis[i + j] == axis ? axis : graft::kMixed;
    a.piece_axis |= axis << 4 * (i / per);
  }
  if (scales) { a.k_scale = scales->d_k_scale; a.v_scale = scales->d_v_scale; }
  const bool rows16 = !misaligned(d_k, 16) && !misaligned(d_v, 16) && k_stride % 8 == 0 && v_stride % 8 == 0 &&
                      (!d_q || (!misaligned(d_q, 16) && !misaligned(d_q_out, 16) && q_stride % 8 == 0 &&
                                q_out_stride % 8 == 0));
  // 16-byte pieces where rows and rotating halves allow them, else elements (1 x 32768: 127 and 427 us; 16 x 61: 6.5 and 26)
  a.vec = rows16 && c.rot % (c.interleaved ? 8 : 16) == 0 && !misaligned(d_rope, 16);
  a.by_slots = graft::Divisor(slots);
  a.by_turn = graft::Divisor(c.dim / 8 - (c.interleaved ? 0 : c.rot / 16));
  a.by_value = graft::Divisor(c.dim / 8);
  const cudaError_t e = graft::launch_kv_append(a, h->cfg.dtype, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(h, e, "graft_kv_append launch");
  h->last_launches = 1;
  return GRAFT_OK;
}

// graft_kv_attend and graft_kv_attend_ext
int attend(graft_kv* h, int32_t batch, int32_t slots, const void* d_q, int64_t q_stride, const void* d_k_cache,
           const void* d_v_cache, const int32_t* d_prefix_pages, int32_t prefix_len, const int32_t* d_page_table,
           int32_t table_stride, const int32_t* d_ctx_len, int32_t max_ctx, const uint64_t* d_tree_mask, float scale,
           void* d_out, int64_t out_stride, float* d_lse, const graft_kv_scales* scales, const graft_kv_scores* scores,
           void* stream) {
  if (!h) return GRAFT_EINVAL;
  h->last_launches = 0;
  const graft::KvLayout& c = h->layout;
  if (batch < 0 || batch > h->cfg.max_batch) return fail(h, GRAFT_EINVAL, "batch %d outside [0, %d]", batch, h->cfg.max_batch);
  if (slots < 1 || slots > h->cfg.max_slots) return fail(h, GRAFT_EINVAL, "slots %d outside [1, %d]", slots, h->cfg.max_slots);
  if (prefix_len < 0 || max_ctx < 0 || table_stride < 0 ||
      (int64_t)max_ctx + slots > (int64_t)table_stride * c.page_size)
    return fail(h, GRAFT_EINVAL, "prefix_len and max_ctx must be >= 0, max_ctx + slots <= table_stride * page_size");
  if ((int64_t)prefix_len + max_ctx + slots > kMaxKeys)
    return fail(h, GRAFT_EINVAL, "prefix_len + max_ctx + slots is more than %d", kMaxKeys);
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(h, GRAFT_EINVAL, "scale must be finite and > 0");
  if (const int rc = check_scores(h, scores, scale)) return rc;
  if (batch == 0) return GRAFT_OK;
  if (!d_q || !d_out || !d_page_table || !d_ctx_len || (prefix_len > 0 && !d_prefix_pages))
    return fail(h, GRAFT_EINVAL, "null pointer");
  if (const int rc = check_cache(h, d_k_cache, d_v_cache)) return rc;
  if (const int rc = check_scales(h, scales)) return rc;
  const int64_t qw = (int64_t)c.q_heads * c.dim;
  if (q_stride < qw || out_stride < qw) return fail(h, GRAFT_EINVAL, "a row stride is less than the row");
  if (misaligned(d_q, 2) || misaligned(d_out, 2) || misaligned(d_prefix_pages, 4) || misaligned(d_page_table, 4) ||
      misaligned(d_ctx_len, 4) || misaligned(d_tree_mask, 8) || misaligned(d_lse, 4))
    return fail(h, GRAFT_EINVAL, "a buffer is not aligned to its element size");
  graft::AttendArgs a{};
  a.c = c;
  a.batch = batch; a.slots = slots; a.group = c.q_heads / c.kv_heads;
  a.q = d_q; a.k_cache = d_k_cache; a.v_cache = d_v_cache;
  a.q_stride = q_stride; a.out_stride = out_stride;
  a.prefix_pages = d_prefix_pages; a.prefix_len = prefix_len;
  a.page_table = d_page_table; a.table_stride = table_stride; a.ctx_len = d_ctx_len; a.max_ctx = max_ctx;
  a.tree_mask = d_tree_mask; a.scale = scale; a.out = d_out; a.lse = d_lse; a.err = h->err;
  if (scales) { a.k_scale = scales->d_k_scale; a.v_scale = scales->d_v_scale; }
  if (scores) {
    a.softcap = scores->softcap; a.slope = scores->d_slope;
    // one that holds all there may be changes nothing
    a.window = scores->window < prefix_len + max_ctx + slots ? scores->window : 0;
  }
  a.out_vec = !misaligned(d_out, 16) && out_stride % 8 == 0;
  a.plan = graft::plan_kv_attend(batch, slots, a.group, c.kv_heads, c.dim, prefix_len, max_ctx, a.window, c.eight != 0, a.softcap > 0.f,
                                 h->num_sms);
  a.part_o = h->part_o; a.part_lse = h->part_lse; a.line = h->line; a.wait_polls = h->wait_polls;
  a.by_group = graft::Divisor(a.group);
  a.by_heads = graft::Divisor(c.kv_heads);
  // A tensor map needs rows on 16-byte boundaries; other queries come by elements (16 x 61 behind 12001 + 2048: 167 us by
  // map, 181 by elements; 64 x 1 behind 8192 + 1024: 60 and 72).
  a.q_map = !misaligned(d_q, 16) && q_stride % 8 == 0 && a.group <= 128 && q_stride < ((int64_t)1 << 38);
  CUtensorMap qmap{}, kmap, vmap;
  if (a.q_map && !query_map(c, h->cfg.dtype, d_q, (int64_t)batch * slots, q_stride, a.group, &qmap))
    return fail(h, GRAFT_ECUDA, "the driver refused the queries' tensor map");
  if (!cache_map(c, h->cfg.dtype, d_k_cache, &kmap) || !cache_map(c, h->cfg.dtype, d_v_cache, &vmap))
    return fail(h, GRAFT_ECUDA, "the driver refused the cache's tensor map");
  if (const cudaError_t e = prepare(h, graft::kv_attend_form(a.slope, a.softcap, a.window))) return cuda_fail(h, e, "loading the attention");
  const cudaError_t e = graft::launch_kv_attend(a, qmap, kmap, vmap, h->cfg.dtype, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(h, e, "graft_kv_attend launch");
  h->last_launches = a.plan.cut ? 2 : 1;
  return GRAFT_OK;
}

}  // namespace

extern "C" {

void graft_kv_default_config(graft_kv_config* c, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                             int32_t page_size, int32_t num_pages, int32_t max_batch, int32_t max_slots,
                             int32_t dtype) {
  std::memset(c, 0, sizeof *c);
  c->q_heads = q_heads;
  c->kv_heads = kv_heads;
  c->head_dim = head_dim;
  c->rot_dim = head_dim;
  c->page_size = page_size;
  c->num_pages = num_pages;
  c->max_batch = max_batch;
  c->max_slots = max_slots;
  c->dtype = dtype;
  c->token_stride = head_dim;
  c->head_stride = (int64_t)page_size * head_dim;
  c->page_stride = c->head_stride * kv_heads;
}

int graft_kv_init(const graft_kv_config* cfg, graft_kv** out) {
  if (!cfg || !out) return GRAFT_EINVAL;
  *out = nullptr;
  graft_kv* h = new (std::nothrow) graft_kv();
  if (!h) return GRAFT_ENOMEM;
  const int rc = check_cfg(cfg, h);
  if (rc) { delete h; return rc; }
  h->cfg = *cfg;
  graft::KvLayout& c = h->layout;
  c.q_heads = cfg->q_heads; c.kv_heads = cfg->kv_heads; c.dim = cfg->head_dim; c.rot = cfg->rot_dim;
  c.interleaved = cfg->rot_interleaved; c.page_size = cfg->page_size; c.num_pages = cfg->num_pages;
  while ((1 << c.page_shift) < cfg->page_size) ++c.page_shift;
  c.page_stride = cfg->page_stride; c.head_stride = cfg->head_stride; c.token_stride = cfg->token_stride;
  c.eight = (cfg->dtype & GRAFT_CACHE_E4M3) != 0;
  h->cfg.dtype &= ~GRAFT_CACHE_E4M3;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e != cudaSuccess) { delete h; return GRAFT_ECUDA; }
  h->part_rows = graft::kv_attend_part_rows((int64_t)cfg->max_batch * cfg->max_slots * cfg->q_heads, h->num_sms);
  e = cudaMalloc(reinterpret_cast<void**>(&h->err), 16);
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&h->part_o), (size_t)h->part_rows * cfg->head_dim * 4);
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&h->part_lse), (size_t)h->part_rows * 4);
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&h->line), ((size_t)cfg->max_batch + 1 + h->num_sms) * 8);
  if (e != cudaSuccess) { free_all(h); delete h; return GRAFT_ENOMEM; }
  e = cudaMemset(h->err, 0, 16);
  if (e == cudaSuccess) e = prepare(h, 0);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) { free_all(h); delete h; return GRAFT_ECUDA; }
  *out = h;
  return GRAFT_OK;
}

int graft_kv_destroy(graft_kv* h) {
  if (!h) return GRAFT_EINVAL;
  cudaDeviceSynchronize();
  free_all(h);
  delete h;
  return GRAFT_OK;
}

int graft_kv_set_axes(graft_kv* h, int32_t axes, const int32_t* pair_axis) {
  if (!h) return GRAFT_EINVAL;
  if (axes < 1 || axes > 8) return fail(h, GRAFT_EINVAL, "axes must be in [1, 8]");
  const int pairs = h->layout.rot / 2;
  if (pairs > 0 && !pair_axis) return fail(h, GRAFT_EINVAL, "null pointer");
  for (int i = 0; i < pairs; ++i)
    if (pair_axis[i] < 0 || pair_axis[i] >= axes) return fail(h, GRAFT_EINVAL, "pair %d: axis %d outside [0, %d)", i, pair_axis[i], axes);
  h->axes = axes;
  for (int i = 0; i < pairs; ++i) h->pair_axis[i] = (uint8_t)pair_axis[i];
  return GRAFT_OK;
}

int graft_kv_append(graft_kv* h, int32_t batch, int32_t slots, const void* d_q, int64_t q_stride, const void* d_k,
                    int64_t k_stride, const void* d_v, int64_t v_stride, const int32_t* d_depth,
                    const int32_t* d_rows, const float* d_rope, int32_t rope_len, int32_t prefix_len,
                    const int32_t* d_page_table, int32_t table_stride, const int32_t* d_ctx_len, void* d_q_out,
                    int64_t q_out_stride, void* d_k_cache, void* d_v_cache, void* stream) {
  NvtxRange nvtx("graft_kv_append");
  return append(h, batch, slots, d_q, q_stride, d_k, k_stride, d_v, v_stride, d_depth, d_rows, nullptr, d_rope, rope_len,
                prefix_len, d_page_table, table_stride, d_ctx_len, d_q_out, q_out_stride, d_k_cache, d_v_cache, nullptr, stream);
}

int graft_kv_append_ext(graft_kv* h, int32_t batch, int32_t slots, const void* d_q, int64_t q_stride, const void* d_k,
                        int64_t k_stride, const void* d_v, int64_t v_stride, const int32_t* d_depth,
                        const int32_t* d_rows, const int32_t* d_position, const float* d_rope, int32_t rope_len,
                        int32_t prefix_len, const int32_t* d_page_table, int32_t table_stride,
                        const int32_t* d_ctx_len, void* d_q_out, int64_t q_out_stride, void* d_k_cache,
                        void* d_v_cache, const graft_kv_scales* scales, void* stream) {
  NvtxRange nvtx("graft_kv_append_ext");
  if (!h) return GRAFT_EINVAL;
  h->last_launches = 0;
  if (const int rc = check_device(h)) return rc;
  return append(h, batch, slots, d_q, q_stride, d_k, k_stride, d_v, v_stride, d_depth, d_rows, d_position, d_rope, rope_len,
                prefix_len, d_page_table, table_stride, d_ctx_len, d_q_out, q_out_stride, d_k_cache, d_v_cache, scales, stream);
}

int graft_kv_read(graft_kv* h, int32_t batch, int32_t slots, const void* d_k_cache, const void* d_v_cache,
                  const int32_t* d_page_table, int32_t table_stride, const int32_t* d_first, const int32_t* d_count,
                  const graft_kv_scales* scales, void* d_k_out, int64_t k_stride, void* d_v_out, int64_t v_stride,
                  void* stream) {
  NvtxRange nvtx("graft_kv_read");
  if (!h) return GRAFT_EINVAL;
  h->last_launches = 0;
  const graft::KvLayout& c = h->layout;
  if (batch < 0 || slots < 1 || (int64_t)batch * slots > 0x7FFFFFFF)
    return fail(h, GRAFT_EINVAL, "batch %d and slots %d: batch >= 0, slots >= 1, batch * slots < 2^31", batch, slots);
  if (table_stride < 0) return fail(h, GRAFT_EINVAL, "table_stride must be >= 0");
  if (const int rc = check_device(h)) return rc;
  if (batch == 0) return GRAFT_OK;
  if (!d_page_table || !d_first || !d_count || !d_k_out || !d_v_out) return fail(h, GRAFT_EINVAL, "null pointer");
  if (const int rc = check_cache(h, d_k_cache, d_v_cache)) return rc;
  if (const int rc = check_scales(h, scales)) return rc;
  const int64_t kw = (int64_t)c.kv_heads * c.dim;
  if (k_stride < kw || v_stride < kw) return fail(h, GRAFT_EINVAL, "a row stride is less than the row");
  if (misaligned(d_page_table, 4) || misaligned(d_first, 4) || misaligned(d_count, 4) || misaligned(d_k_out, 2) ||
      misaligned(d_v_out, 2))
    return fail(h, GRAFT_EINVAL, "a buffer is not aligned to its element size");
  graft::ReadArgs a{};
  a.c = c;
  a.batch = batch; a.slots = slots;
  a.vec = !misaligned(d_k_out, 16) && !misaligned(d_v_out, 16) && k_stride % 8 == 0 && v_stride % 8 == 0;
  a.k_cache = d_k_cache; a.v_cache = d_v_cache;
  a.page_table = d_page_table; a.table_stride = table_stride; a.first = d_first; a.count = d_count;
  if (scales) { a.k_scale = scales->d_k_scale; a.v_scale = scales->d_v_scale; }
  a.k_out = d_k_out; a.v_out = d_v_out; a.k_stride = k_stride; a.v_stride = v_stride;
  a.by_slots = graft::Divisor(slots);
  a.by_head = graft::Divisor(c.dim / (c.eight ? 16 : 8));
  a.err = h->err;
  const cudaError_t e = graft::launch_kv_read(a, h->cfg.dtype, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(h, e, "graft_kv_read launch");
  h->last_launches = 1;
  return GRAFT_OK;
}

int graft_kv_attend(graft_kv* h, int32_t batch, int32_t slots, const void* d_q, int64_t q_stride,
                    const void* d_k_cache, const void* d_v_cache, const int32_t* d_prefix_pages, int32_t prefix_len,
                    const int32_t* d_page_table, int32_t table_stride, const int32_t* d_ctx_len, int32_t max_ctx,
                    const uint64_t* d_tree_mask, float scale, void* d_out, int64_t out_stride, float* d_lse,
                    void* stream) {
  NvtxRange nvtx("graft_kv_attend");
  return attend(h, batch, slots, d_q, q_stride, d_k_cache, d_v_cache, d_prefix_pages, prefix_len, d_page_table, table_stride,
                d_ctx_len, max_ctx, d_tree_mask, scale, d_out, out_stride, d_lse, nullptr, nullptr, stream);
}

int graft_kv_attend_ext(graft_kv* h, int32_t batch, int32_t slots, const void* d_q, int64_t q_stride,
                        const void* d_k_cache, const void* d_v_cache, const int32_t* d_prefix_pages,
                        int32_t prefix_len, const int32_t* d_page_table, int32_t table_stride,
                        const int32_t* d_ctx_len, int32_t max_ctx, const uint64_t* d_tree_mask, float scale,
                        void* d_out, int64_t out_stride, float* d_lse, const graft_kv_scales* scales,
                        const graft_kv_scores* scores, void* stream) {
  NvtxRange nvtx("graft_kv_attend_ext");
  if (!h) return GRAFT_EINVAL;
  h->last_launches = 0;
  if (const int rc = check_device(h)) return rc;
  return attend(h, batch, slots, d_q, q_stride, d_k_cache, d_v_cache, d_prefix_pages, prefix_len, d_page_table, table_stride,
                d_ctx_len, max_ctx, d_tree_mask, scale, d_out, out_stride, d_lse, scales, scores, stream);
}

int graft_kv_sync(graft_kv* h, void* stream, uint32_t* out_flags) {
  if (!h) return GRAFT_EINVAL;
  uint32_t flags = 0;
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaMemcpy(&flags, h->err, sizeof flags, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && flags) e = cudaMemset(h->err, 0, sizeof flags);
  if (out_flags) *out_flags = flags;
  if (e != cudaSuccess) return cuda_fail(h, e, "graft_kv_sync");
  if (flags) return fail(h, GRAFT_EDEVICE, "device error flags 0x%x (range %d, timeout %d, rule %d)", flags,
                         !!(flags & GRAFT_ERR_RANGE), !!(flags & GRAFT_ERR_TIMEOUT), !!(flags & GRAFT_ERR_RULE));
  return GRAFT_OK;
}

const char* graft_kv_last_error(const graft_kv* h) { return h ? h->msg : "null handle"; }

int32_t graft_kv_last_launch_count(const graft_kv* h) { return h ? h->last_launches : 0; }

int graft_kv_set_wait_limit(graft_kv* h, uint32_t polls) {
  if (!h) return GRAFT_EINVAL;
  h->wait_polls = polls;
  return GRAFT_OK;
}

}  // extern "C"
