// C entry points of the paged KV cache and of the norm + rotation pass
// (declared in include/arl2.h): handles, argument checks, work space and
// kernel dispatch.  Batches are read by the kernels alone: nothing here waits
// for the device, so every call may be captured into a CUDA graph.

#include <cmath>
#include <cstdint>
#include <mutex>
#include <new>
#include <set>

#include "layer.h"
#include "paged.h"

using namespace arl2;

namespace {

constexpr uint64_t kPagedMagic = 0x41524c3250414745ull;  // "ARL2PAGE"
constexpr uint64_t kDefaultWaitNs = 1000000000ull;
constexpr int32_t kMaxLen = 1 << 30;  // of a cache or a batch's tokens: key and row indices stay in 32 bits

std::mutex g_paged_mu;
std::set<const void*> g_paged;

size_t esize(int dtype) { return dtype == ARL2_F32 ? 4 : 2; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// `rows` runs of `width` bytes, `pitch` bytes apart.
struct Span {
  const void* p;
  size_t rows, width, pitch;
  size_t bytes() const { return rows ? (rows - 1) * pitch + width : 0; }
};
Span flat(const void* p, size_t bytes) { return Span{p, bytes ? size_t(1) : 0, bytes, bytes}; }

// Whether two spans share a byte (for unequal pitches: whether their extents do).
bool clash(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.rows || !b.rows) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (x >= y + b.bytes() || y >= x + a.bytes()) return false;
  if (a.pitch != b.pitch || a.rows < 2 || b.rows < 2) return true;
  // rows of one pitch: b's runs begin `off` bytes behind a's
  const size_t off = y >= x ? (y - x) % a.pitch : (a.pitch - (x - y) % a.pitch) % a.pitch;
  return off < a.width || off + b.width > a.pitch;
}

bool check_prep(const arl2_qk_prep* p, int dtype, int d, arl2_status* s) {
  *s = ARL2_ERR_INVALID_ARGUMENT;
  if (!p || p->n_axes < 0 || p->n_axes > 3 || (p->halves != 0 && p->halves != 1)) return false;
  if (!std::isfinite(p->eps) || p->eps < 0.f) return false;
  if ((p->w_q == nullptr) != (p->w_k == nullptr) || !aligned(p->w_q, 16) || !aligned(p->w_k, 16)) return false;
  int64_t R = 0;
  for (int a = 0; a < p->n_axes; ++a) {
    if (p->axis_dim[a] < 2 || p->axis_dim[a] % 2) return false;
    R += p->axis_dim[a];
  }
  if (R > d) return false;
  if (p->n_axes > 0 && !(p->theta >= 1.f && p->theta <= 1e12f)) return false;
  *s = ARL2_ERR_UNSUPPORTED;
  if (p->halves && R / 2 % int64_t(16 / esize(dtype))) return false;
  *s = ARL2_OK;
  return true;
}

arl2_status check_head_dim(int dtype, int d) {
  if (dtype != ARL2_F32 && dtype != ARL2_BF16) return ARL2_ERR_UNSUPPORTED;
  if (d < 1) return ARL2_ERR_INVALID_ARGUMENT;
  return d > 128 || d % int(16 / esize(dtype)) ? ARL2_ERR_UNSUPPORTED : ARL2_OK;
}

// Rotation frequencies in fractions of a turn per position: theta^(-2 i / n) /
// (2 pi) in units of 2^-64.  The powers are products of one ratio in 64-bit
// mantissas: at most 64 roundings, 2^-58 of a frequency, so 2^-29 of a turn at
// the largest position.
void fill_prep(PrepParams& p, const arl2_qk_prep& prep) {
  p.w_q = prep.w_q;
  p.w_k = prep.w_k;
  p.norm = prep.w_q != nullptr;
  p.eps = prep.eps;
  p.n_axes = prep.n_axes;
  p.halves = prep.halves;
  p.rot = 0;
  int at = 0;
  for (int a = 0; a < 3; ++a) {
    p.axis_dim[a] = a < prep.n_axes ? prep.axis_dim[a] : 0;
    p.rot += p.axis_dim[a];
    if (a >= prep.n_axes) continue;
    const long double ratio = std::pow((long double)prep.theta, -2.0L / prep.axis_dim[a]);
    long double f = 18446744073709551616.0L / 6.283185307179586476925286766559L;
    for (int i = 0; i < prep.axis_dim[a] / 2; ++i, f *= ratio) p.freq[at++] = uint64_t(f + 0.5L);
  }
}

struct Device {
  int prev = -1, ok = 0;
  explicit Device(int dev) {
    ok = cudaGetDevice(&prev) == cudaSuccess && (prev == dev || cudaSetDevice(dev) == cudaSuccess);
    if (prev == dev) prev = -1;
  }
  ~Device() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

}  // namespace

struct arl2_paged {
  uint64_t magic;
  arl2_paged_config cfg;
  int device, sms;
  float scale;
  void *k_pool, *v_pool;
  uint64_t wait_ns;
  float* part_o;   // pieces of items that CTAs share, and their statistics (PagedAttnParams)
  float2* part_ml;
  uint32_t* joined;
  int grid;        // CTAs of the attention launch
  uint32_t* err;
  int64_t bytes;
  cudaStream_t last_stream;
  int l2_bytes;
  FastDiv page;
  int box;
  CUtensorMap tm_k, tm_v;  // over the pools (bf16)
};

namespace {

bool live(const arl2_paged* h) {
  if (!h) return false;
  std::lock_guard<std::mutex> g(g_paged_mu);
  return g_paged.count(h) && h->magic == kPagedMagic;
}

void free_paged(arl2_paged* h) {
  for (void* p : {(void*)h->part_o, (void*)h->part_ml, (void*)h->joined, (void*)h->err})
    if (p) cudaFree(p);
  h->magic = 0;
  delete h;
}

size_t joined_bytes(const arl2_paged* h) { return size_t(h->grid) * 8 * sizeof(uint32_t); }

int group_of(const arl2_paged* h) { return h->cfg.heads / h->cfg.kv_heads; }

Span pool_span(const arl2_paged* h, const void* p) {
  const arl2_paged_config& c = h->cfg;
  return flat(p, size_t(c.n_pages) * c.kv_heads * c.page_size * c.head_dim * esize(c.dtype));
}
// [tokens, heads, head_dim] rows ld elements apart (0: contiguous)
Span rows_span(const void* p, int64_t tokens, int heads, int d, int64_t ld, int dtype) {
  const size_t row = size_t(heads) * d;
  return Span{p, size_t(tokens), row * esize(dtype), size_t(ld ? ld : int64_t(row)) * esize(dtype)};
}

arl2_status check_batch(const arl2_paged* h, const arl2_paged_batch* b, bool rows) {
  if (!b || b->n_seqs < 0) return ARL2_ERR_INVALID_ARGUMENT;
  if (b->n_seqs == 0) return ARL2_OK;
  if (b->max_kv < 0 || b->pages_ld < 0 || !b->kv_len || !aligned(b->kv_len, 4)) return ARL2_ERR_INVALID_ARGUMENT;
  if (b->pages_ld > 0 && (!b->pages || !aligned(b->pages, 4))) return ARL2_ERR_INVALID_ARGUMENT;
  if (b->max_kv > kMaxLen || int64_t(b->n_seqs) * h->cfg.kv_heads > kMaxLen) return ARL2_ERR_UNSUPPORTED;
  if (rows) {
    if (b->tokens < 0 || b->max_q < 0 || !b->q_start || !aligned(b->q_start, 4)) return ARL2_ERR_INVALID_ARGUMENT;
    if (b->tokens > kMaxLen || b->max_q > kMaxLen) return ARL2_ERR_UNSUPPORTED;
  }
  return ARL2_OK;
}

bool check_ld(int64_t ld, int64_t row, int dtype) {
  return ld == 0 || (ld >= row && ld % int64_t(16 / esize(dtype)) == 0);
}

PagedSeqs seqs_of(const arl2_paged* h, const arl2_paged_batch* b) {
  PagedSeqs s{};
  s.q_start = b->q_start;
  s.kv_len = b->kv_len;
  s.pages = b->pages;
  s.n_seqs = b->n_seqs;
  s.tokens = b->tokens;
  s.max_q = b->max_q;
  s.max_kv = b->max_kv;
  s.pages_ld = b->pages_ld;
  s.page_size = h->cfg.page_size;
  s.n_pages = h->cfg.n_pages;
  s.page = h->page;
  s.box = h->box;
  return s;
}

// The spans that a batch's own arrays take.
struct BatchSpans {
  Span s[3];
  bool clash_any(const Span& o) const { return clash(o, s[0]) || clash(o, s[1]) || clash(o, s[2]); }
};
BatchSpans batch_spans(const arl2_paged_batch* b) {
  return BatchSpans{{flat(b->q_start, (size_t(b->n_seqs) + 1) * 4), flat(b->kv_len, size_t(b->n_seqs) * 4),
                     flat(b->pages, size_t(b->n_seqs) * b->pages_ld * 4)}};
}

}  // namespace

#define PAGED_TRY(expr)                               \
  do {                                                \
    cudaError_t e_ = (expr);                          \
    if (e_ != cudaSuccess) return status_of_cuda(e_); \
  } while (0)

extern "C" {

arl2_status arl2_qk_norm_rope(const arl2_qk_prep* prep, int32_t dtype, int32_t heads, int32_t kv_heads,
                              int32_t head_dim, int64_t tokens, const void* q, const void* k, int64_t ld,
                              const int32_t* pos, void* q_out, void* k_out, int64_t ld_out, void* stream) {
  if (heads < 1 || kv_heads < 1 || tokens < 0) return ARL2_ERR_INVALID_ARGUMENT;
  arl2_status s = check_head_dim(dtype, head_dim);
  if (s != ARL2_OK) return s;
  if (!check_prep(prep, dtype, head_dim, &s)) return s;
  if (heads > 65536 || kv_heads > 65536 || tokens > kMaxLen) return ARL2_ERR_UNSUPPORTED;
  const int64_t row_q = int64_t(heads) * head_dim, row_k = int64_t(kv_heads) * head_dim;
  const int64_t row = row_q > row_k ? row_q : row_k;
  if (!check_ld(ld, row, dtype) || !check_ld(ld_out, row, dtype)) return ARL2_ERR_INVALID_ARGUMENT;
  if (tokens == 0) return ARL2_OK;
  for (const void* p : {q, k, (const void*)q_out, (const void*)k_out})
    if (!p || !aligned(p, 16)) return ARL2_ERR_INVALID_ARGUMENT;
  if (prep->n_axes > 0 && (!pos || !aligned(pos, 4))) return ARL2_ERR_INVALID_ARGUMENT;
  {
    const Span in[2] = {rows_span(q, tokens, heads, head_dim, ld, dtype),
                        rows_span(k, tokens, kv_heads, head_dim, ld, dtype)};
    const Span out[2] = {rows_span(q_out, tokens, heads, head_dim, ld_out, dtype),
                         rows_span(k_out, tokens, kv_heads, head_dim, ld_out, dtype)};
    const Span small[3] = {flat(prep->w_q, size_t(head_dim) * esize(dtype)),
                           flat(prep->w_k, size_t(head_dim) * esize(dtype)),
                           flat(prep->n_axes > 0 ? pos : nullptr, size_t(tokens) * prep->n_axes * 4)};
    if (clash(out[0], out[1])) return ARL2_ERR_INVALID_ARGUMENT;
    for (int o = 0; o < 2; ++o) {
      for (int i = 0; i < 2; ++i) {
        const bool in_place = o == i && out[o].p == in[i].p && (out[o].pitch == in[i].pitch || tokens == 1);
        if (!in_place && clash(out[o], in[i])) return ARL2_ERR_INVALID_ARGUMENT;
      }
      for (const Span& w : small)
        if (clash(out[o], w)) return ARL2_ERR_INVALID_ARGUMENT;
    }
  }
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return ARL2_ERR_NO_DEVICE;
  PrepParams p{};
  fill_prep(p, *prep);
  p.q = q;
  p.k = k;
  p.ld_q = ld ? ld : row_q;
  p.ld_k = ld ? ld : row_k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.ld_qo = ld_out ? ld_out : row_q;
  p.ld_ko = ld_out ? ld_out : row_k;
  p.pos = pos;
  p.tokens = tokens;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.d = head_dim;
  p.inv_d = 1.f / float(head_dim);
  PAGED_TRY(launch_prep(p, dtype, false, sms, static_cast<cudaStream_t>(stream)));
  return ARL2_OK;
}

arl2_status arl2_paged_init(const arl2_paged_config* cfg, void* k_pool, void* v_pool, void* stream,
                            arl2_paged_t* out) {
  if (!out) return ARL2_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  if (!cfg || cfg->heads < 1 || cfg->kv_heads < 1 || cfg->heads % cfg->kv_heads || cfg->page_size < 1 ||
      cfg->n_pages < 1)
    return ARL2_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(cfg->softmax_scale) || cfg->softmax_scale < 0.f) return ARL2_ERR_INVALID_ARGUMENT;
  arl2_status s = check_head_dim(cfg->dtype, cfg->head_dim);
  if (s != ARL2_OK) return s;
  if (cfg->dtype == ARL2_BF16 && cfg->head_dim != 128) return ARL2_ERR_UNSUPPORTED;
  if (cfg->heads / cfg->kv_heads > kPagedMaxGroup || cfg->heads > 65536 || cfg->page_size % 8 ||
      cfg->page_size > 4096 || int64_t(cfg->n_pages) * cfg->kv_heads >= (int64_t(1) << 31) / cfg->page_size)
    return ARL2_ERR_UNSUPPORTED;
  if (!k_pool || !v_pool || !aligned(k_pool, 16) || !aligned(v_pool, 16)) return ARL2_ERR_INVALID_ARGUMENT;
  const size_t pool = size_t(cfg->n_pages) * cfg->kv_heads * cfg->page_size * cfg->head_dim * esize(cfg->dtype);
  if (clash(flat(k_pool, pool), flat(v_pool, pool))) return ARL2_ERR_INVALID_ARGUMENT;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ARL2_ERR_NO_DEVICE;
  arl2_paged* h = new (std::nothrow) arl2_paged();
  if (!h) return ARL2_ERR_OUT_OF_MEMORY;
  h->cfg = *cfg;
  h->device = dev;
  h->scale = cfg->softmax_scale > 0.f ? cfg->softmax_scale : 1.f / std::sqrt(float(cfg->head_dim));
  h->k_pool = k_pool;
  h->v_pool = v_pool;
  h->wait_ns = kDefaultWaitNs;
  if (cudaDeviceGetAttribute(&h->l2_bytes, cudaDevAttrL2CacheSize, dev) != cudaSuccess) h->l2_bytes = 0;
  h->page = FastDiv(cfg->page_size);
  h->box = box_keys(cfg->page_size);
  h->last_stream = static_cast<cudaStream_t>(stream);
  if (cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || h->sms < 1) h->sms = 1;
  if (cfg->dtype == ARL2_BF16) {
    const int64_t rows = int64_t(cfg->n_pages) * cfg->kv_heads * cfg->page_size;
    if (!tensor_map_encoder() || !paged_pool_map(&h->tm_k, k_pool, rows, cfg->page_size) ||
        !paged_pool_map(&h->tm_v, v_pool, rows, cfg->page_size)) {
      free_paged(h);
      return ARL2_ERR_NO_DEVICE;
    }
  }
  h->grid = paged_attn_grid(cfg->dtype, h->sms);
  const size_t pieces = 2 * size_t(h->grid), rows = paged_piece_rows(cfg->dtype);
  const size_t po = pieces * rows * cfg->head_dim * sizeof(float), pm = pieces * rows * sizeof(float2);
  cudaError_t e = device_alloc(reinterpret_cast<void**>(&h->part_o), po);
  if (e == cudaSuccess) e = device_alloc(reinterpret_cast<void**>(&h->part_ml), pm);
  if (e == cudaSuccess) e = device_alloc(reinterpret_cast<void**>(&h->joined), joined_bytes(h));
  if (e == cudaSuccess) e = cudaMemsetAsync(h->joined, 0, joined_bytes(h), h->last_stream);
  if (e == cudaSuccess) e = device_alloc(reinterpret_cast<void**>(&h->err), 256);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->err, 0, 256, h->last_stream);
  // the first call may come on a stream that does not wait for this one
  if (e == cudaSuccess) e = cudaStreamSynchronize(h->last_stream);
  if (e != cudaSuccess) {
    free_paged(h);
    return status_of_cuda(e);
  }
  h->bytes = int64_t(po + pm + joined_bytes(h) + 256);
  h->magic = kPagedMagic;
  {
    std::lock_guard<std::mutex> g(g_paged_mu);
    g_paged.insert(h);
  }
  *out = h;
  return ARL2_OK;
}

arl2_status arl2_paged_append(arl2_paged_t h, const arl2_paged_batch* batch, const arl2_qk_prep* prep, const void* q,
                              const void* k, const void* v, int64_t ld, const int32_t* pos, void* q_out,
                              void* stream) {
  if (!live(h)) return ARL2_ERR_INVALID_ARGUMENT;
  const arl2_paged_config& c = h->cfg;
  arl2_status s = check_batch(h, batch, true);
  if (s != ARL2_OK) return s;
  if (prep && !check_prep(prep, c.dtype, c.head_dim, &s)) return s;
  if ((q == nullptr) != (q_out == nullptr) || (!prep && q)) return ARL2_ERR_INVALID_ARGUMENT;
  const int64_t row_q = int64_t(c.heads) * c.head_dim, row_k = int64_t(c.kv_heads) * c.head_dim;
  if (!check_ld(ld, q ? row_q : row_k, c.dtype)) return ARL2_ERR_INVALID_ARGUMENT;
  if (batch->n_seqs == 0 || batch->tokens == 0) return ARL2_OK;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16))
    return ARL2_ERR_INVALID_ARGUMENT;
  const bool turn = prep && prep->n_axes > 0;
  if (turn && (!pos || !aligned(pos, 4))) return ARL2_ERR_INVALID_ARGUMENT;
  {
    const Span in[3] = {rows_span(q, batch->tokens, c.heads, c.head_dim, ld, c.dtype),
                        rows_span(k, batch->tokens, c.kv_heads, c.head_dim, ld, c.dtype),
                        rows_span(v, batch->tokens, c.kv_heads, c.head_dim, ld, c.dtype)};
    const Span small[3] = {flat(prep ? prep->w_q : nullptr, size_t(c.head_dim) * esize(c.dtype)),
                           flat(prep ? prep->w_k : nullptr, size_t(c.head_dim) * esize(c.dtype)),
                           flat(turn ? pos : nullptr, size_t(batch->tokens) * (turn ? prep->n_axes : 0) * 4)};
    const Span out[3] = {rows_span(q_out, batch->tokens, c.heads, c.head_dim, 0, c.dtype), pool_span(h, h->k_pool),
                         pool_span(h, h->v_pool)};
    const BatchSpans bs = batch_spans(batch);
    if (clash(out[0], out[1]) || clash(out[0], out[2])) return ARL2_ERR_INVALID_ARGUMENT;
    for (int o = 0; o < 3; ++o) {
      for (int i = 0; i < 3; ++i) {
        const bool in_place = o == 0 && i == 0 && q_out == q && (out[0].pitch == in[0].pitch || batch->tokens == 1);
        if (!in_place && clash(out[o], in[i])) return ARL2_ERR_INVALID_ARGUMENT;
      }
      for (const Span& w : small)
        if (clash(out[o], w)) return ARL2_ERR_INVALID_ARGUMENT;
      if (bs.clash_any(out[o])) return ARL2_ERR_INVALID_ARGUMENT;
    }
  }
  Device dev(h->device);
  if (!dev.ok) return ARL2_ERR_CUDA;
  h->last_stream = static_cast<cudaStream_t>(stream);
  PrepParams p{};
  if (prep) fill_prep(p, *prep);
  p.q = q;
  p.k = k;
  p.v = v;
  p.ld_q = ld ? ld : row_q;
  p.ld_k = p.ld_v = ld ? ld : row_k;
  p.q_out = q_out;
  p.ld_qo = row_q;
  p.pos = pos;
  p.tokens = batch->tokens;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.d = c.head_dim;
  p.inv_d = 1.f / float(c.head_dim);
  p.s = seqs_of(h, batch);
  p.k_pool = h->k_pool;
  p.v_pool = h->v_pool;
  p.err = h->err;
  PAGED_TRY(launch_prep(p, c.dtype, true, h->sms, h->last_stream));
  return ARL2_OK;
}

arl2_status arl2_paged_attend(arl2_paged_t h, const arl2_paged_batch* batch, const void* q, int64_t ld_q,
                              int32_t mask_block, void* o, float* lse, void* stream) {
  if (!live(h)) return ARL2_ERR_INVALID_ARGUMENT;
  const arl2_paged_config& c = h->cfg;
  arl2_status s = check_batch(h, batch, true);
  if (s != ARL2_OK) return s;
  const int64_t row = int64_t(c.heads) * c.head_dim;
  if (mask_block < 0 || !check_ld(ld_q, row, c.dtype)) return ARL2_ERR_INVALID_ARGUMENT;
  if (batch->n_seqs == 0 || batch->tokens == 0 || batch->max_q == 0) return ARL2_OK;
  if (!q || !o || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4)) return ARL2_ERR_INVALID_ARGUMENT;
  {
    const Span in[3] = {rows_span(q, batch->tokens, c.heads, c.head_dim, ld_q, c.dtype), pool_span(h, h->k_pool),
                        pool_span(h, h->v_pool)};
    const Span out[2] = {rows_span(o, batch->tokens, c.heads, c.head_dim, 0, c.dtype),
                         flat(lse, size_t(batch->tokens) * c.heads * 4)};
    const BatchSpans bs = batch_spans(batch);
    if (clash(out[0], out[1])) return ARL2_ERR_INVALID_ARGUMENT;
    for (const Span& x : out) {
      for (const Span& y : in)
        if (clash(x, y)) return ARL2_ERR_INVALID_ARGUMENT;
      if (bs.clash_any(x)) return ARL2_ERR_INVALID_ARGUMENT;
    }
  }
  Device dev(h->device);
  if (!dev.ok) return ARL2_ERR_CUDA;
  h->last_stream = static_cast<cudaStream_t>(stream);
  PagedAttnParams p{};
  p.s = seqs_of(h, batch);
  p.q = q;
  p.ld_q = ld_q ? ld_q : row;
  p.k_pool = h->k_pool;
  p.v_pool = h->v_pool;
  p.o = o;
  p.lse = lse;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.group = group_of(h);
  p.d = c.head_dim;
  p.mask_block = mask_block;
  p.scale_log2 = h->scale * 1.4426950408889634f;
  p.part_o = h->part_o;
  p.part_ml = h->part_ml;
  p.joined = h->joined;
  p.err = h->err;
  p.wait_limit_ns = h->wait_ns;
  if (!paged_plan(p, c.dtype == ARL2_BF16 ? 128 : 64, c.dtype == ARL2_BF16 ? 2 : 1, c.dtype == ARL2_BF16 ? 128 : 64))
    return ARL2_ERR_UNSUPPORTED;
  // Units of a range at least: one of 256 keys takes about 1.5 us, a piece more in
  // the join 0.09 for every 8 rows, so that sqrt(0.06 units rows / 8) a range costs
  // least.  16 tokens of 8 heads a key head on 3000 keys take 31 us (47 with one at
  // least), one on 20000 keys 24 (28); one token of a head of its own on 1561 keys
  // 16, and 17.2 with two.  (float32's join is a whole block's: one.)
  p.min_cost = 1;
  if (c.dtype == ARL2_BF16) {
    const int rows = (batch->max_q < p.qt ? batch->max_q : p.qt) * p.group;
    p.min_cost = int(std::sqrt(0.06 * (batch->max_kv / 256 + 1) * ((rows + 7) / 8)));
    if (p.min_cost < 1) p.min_cost = 1;
  }
  // Several blocks of rows on the keys of a pool that L2 does not hold: a frame of
  // 1560 tokens on 201 MB reads 513 MB from memory instead of 945 and takes 4 %
  // less time.  With 33 MB of keys the rotation costs 7 %.
  const bool rotate = batch->max_q > 2 * p.qt && 2 * pool_span(h, h->k_pool).bytes() > size_t(h->l2_bytes);
  PAGED_TRY(c.dtype == ARL2_BF16 ? launch_paged_attn_bf16(p, h->tm_k, h->tm_v, h->grid, rotate, h->last_stream)
                                 : launch_paged_attn_f32(p, h->grid, h->last_stream));
  return ARL2_OK;
}

arl2_status arl2_paged_weights(arl2_paged_t h, const arl2_paged_batch* batch, const void* q, int64_t ld_q,
                               int32_t mask_block, const float* lse, float decay, const float* w_in, float* w_out,
                               int64_t w_ld, void* stream) {
  if (!live(h)) return ARL2_ERR_INVALID_ARGUMENT;
  const arl2_paged_config& c = h->cfg;
  arl2_status s = check_batch(h, batch, true);
  if (s != ARL2_OK) return s;
  const int64_t row = int64_t(c.heads) * c.head_dim;
  if (mask_block < 0 || !std::isfinite(decay) || !check_ld(ld_q, row, c.dtype)) return ARL2_ERR_INVALID_ARGUMENT;
  if (batch->n_seqs == 0) return ARL2_OK;
  if (w_ld < batch->max_kv || w_ld < 0) return ARL2_ERR_INVALID_ARGUMENT;
  if (w_ld > kMaxLen) return ARL2_ERR_UNSUPPORTED;
  if (w_ld == 0) return ARL2_OK;
  if (!w_in || !w_out || !aligned(w_in, 4) || !aligned(w_out, 4)) return ARL2_ERR_INVALID_ARGUMENT;
  if (batch->tokens > 0 && (!q || !lse || !aligned(q, 16) || !aligned(lse, 4))) return ARL2_ERR_INVALID_ARGUMENT;
  {
    const size_t wb = size_t(batch->n_seqs) * c.kv_heads * size_t(w_ld) * 4;
    const Span out = flat(w_out, wb);
    const Span in[4] = {rows_span(q, batch->tokens, c.heads, c.head_dim, ld_q, c.dtype), pool_span(h, h->k_pool),
                        pool_span(h, h->v_pool), flat(lse, size_t(batch->tokens) * c.heads * 4)};
    for (const Span& x : in)
      if (clash(out, x)) return ARL2_ERR_INVALID_ARGUMENT;
    if (w_in != w_out && clash(out, flat(w_in, wb))) return ARL2_ERR_INVALID_ARGUMENT;
    if (batch_spans(batch).clash_any(out)) return ARL2_ERR_INVALID_ARGUMENT;
  }
  Device dev(h->device);
  if (!dev.ok) return ARL2_ERR_CUDA;
  h->last_stream = static_cast<cudaStream_t>(stream);
  PagedWeightParams p{};
  p.s = seqs_of(h, batch);
  p.q = q;
  p.ld_q = ld_q ? ld_q : row;
  p.k_pool = h->k_pool;
  p.lse = lse;
  p.w_in = w_in;
  p.w_out = w_out;
  p.w_ld = w_ld;
  p.decay = decay;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.group = group_of(h);
  p.d = c.head_dim;
  p.mask_block = mask_block;
  p.scale_log2 = h->scale * 1.4426950408889634f;
  p.err = h->err;
  p.wait_limit_ns = h->wait_ns;
  p.mask = FastDiv(mask_block);
  p.per_group = FastDiv(p.group);
  const int keys = c.dtype == ARL2_BF16 ? 256 : 64;
  p.per_tile = FastDiv((c.dtype == ARL2_BF16 ? 128 : 64) / p.group);
  if (most_blocks(p.s, p.per_tile.by) * (batch->max_kv / keys + 1) * c.kv_heads >= double(kMaxUnits))
    return ARL2_ERR_UNSUPPORTED;
  p.part_w = h->part_o;
  p.joined = h->joined;
  PAGED_TRY(c.dtype == ARL2_BF16 ? launch_paged_weights_bf16(p, h->tm_k, h->sms, h->last_stream)
                                 : launch_paged_weights_f32(p, h->sms, h->last_stream));
  return ARL2_OK;
}

arl2_status arl2_paged_evict(arl2_paged_t h, const arl2_paged_batch* batch, const float* w_in, int64_t w_ld,
                             int32_t budget, int32_t sink, int32_t recent, const int32_t* dst_pages, int32_t dst_ld,
                             float* w_out, int32_t* kept, int32_t* kv_len_out, void* stream) {
  if (!live(h)) return ARL2_ERR_INVALID_ARGUMENT;
  const arl2_paged_config& c = h->cfg;
  arl2_status s = check_batch(h, batch, false);
  if (s != ARL2_OK) return s;
  if (budget < 1 || sink < 0 || recent < 0 || int64_t(sink) + recent > budget) return ARL2_ERR_INVALID_ARGUMENT;
  if (batch->n_seqs == 0) return ARL2_OK;
  if (w_ld < batch->max_kv || w_ld < 1 || dst_ld < 0) return ARL2_ERR_INVALID_ARGUMENT;
  if (w_ld > kMaxLen || budget > kMaxLen) return ARL2_ERR_UNSUPPORTED;
  if (!w_in || !w_out || !kept || !kv_len_out || (dst_ld > 0 && !dst_pages)) return ARL2_ERR_INVALID_ARGUMENT;
  for (const void* p : {(const void*)w_in, (const void*)w_out, (const void*)kept, (const void*)kv_len_out,
                        (const void*)dst_pages})
    if (!aligned(p, 4)) return ARL2_ERR_INVALID_ARGUMENT;
  {
    const size_t n = size_t(batch->n_seqs), wb = n * c.kv_heads * size_t(w_ld) * 4;
    const Span out[5] = {flat(w_out, wb), flat(kept, n * c.kv_heads * size_t(budget) * 4), flat(kv_len_out, n * 4),
                         pool_span(h, h->k_pool), pool_span(h, h->v_pool)};
    const Span in[2] = {flat(w_in, wb), flat(dst_pages, n * dst_ld * 4)};
    BatchSpans bs = batch_spans(batch);
    bs.s[0] = Span{};  // q_start is not used
    for (int i = 0; i < 5; ++i) {
      for (int j = i + 1; j < 5; ++j)
        if (clash(out[i], out[j])) return ARL2_ERR_INVALID_ARGUMENT;
      for (const Span& x : in)
        if (clash(out[i], x)) return ARL2_ERR_INVALID_ARGUMENT;
      if (bs.clash_any(out[i])) return ARL2_ERR_INVALID_ARGUMENT;
    }
  }
  Device dev(h->device);
  if (!dev.ok) return ARL2_ERR_CUDA;
  h->last_stream = static_cast<cudaStream_t>(stream);
  PagedEvictParams p{};
  p.s = seqs_of(h, batch);
  p.k_pool = h->k_pool;
  p.v_pool = h->v_pool;
  p.w_in = w_in;
  p.w_out = w_out;
  p.w_ld = w_ld;
  p.kept = kept;
  p.kv_len_out = kv_len_out;
  p.dst_pages = dst_pages;
  p.dst_ld = dst_ld;
  p.kv_heads = c.kv_heads;
  p.row_bytes = int(size_t(c.head_dim) * esize(c.dtype));
  p.budget = budget;
  p.sink = sink;
  p.recent = recent;
  p.err = h->err;
  PAGED_TRY(launch_paged_evict(p, h->sms, h->last_stream));
  return ARL2_OK;
}

arl2_status arl2_paged_last_error(arl2_paged_t h) {
  if (!live(h)) return ARL2_ERR_INVALID_ARGUMENT;
  Device dev(h->device);
  if (!dev.ok) return ARL2_ERR_CUDA;
  // the whole device: a captured call's replays run on streams that the handle never saw
  PAGED_TRY(cudaDeviceSynchronize());
  uint32_t w = 0;
  PAGED_TRY(cudaMemcpy(&w, h->err, sizeof(w), cudaMemcpyDeviceToHost));
  if (w) {
    // A kernel that gave up may have left pieces counted.  A memset of device memory may
    // return before it has run, and not every stream waits for the default one: it is
    // waited for here, so that no later launch meets it.
    PAGED_TRY(cudaMemset(h->err, 0, sizeof(w)));
    PAGED_TRY(cudaMemset(h->joined, 0, joined_bytes(h)));
    PAGED_TRY(cudaStreamSynchronize(nullptr));
  }
  return static_cast<arl2_status>(w);
}

int64_t arl2_paged_device_bytes(arl2_paged_t h) { return live(h) ? h->bytes : -1; }

arl2_status arl2_paged_set_wait_limit(arl2_paged_t h, uint64_t limit_ns) {
  if (!live(h)) return ARL2_ERR_INVALID_ARGUMENT;
  h->wait_ns = limit_ns ? limit_ns : kDefaultWaitNs;
  return ARL2_OK;
}

arl2_status arl2_paged_destroy(arl2_paged_t h) {
  if (!live(h)) return ARL2_ERR_INVALID_ARGUMENT;
  {
    std::lock_guard<std::mutex> g(g_paged_mu);
    g_paged.erase(h);
  }
  Device dev(h->device);
  cudaStreamSynchronize(h->last_stream);
  free_paged(h);
  return ARL2_OK;
}

}  // extern "C"
