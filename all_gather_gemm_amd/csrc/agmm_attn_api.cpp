// Host side of the C ABI declared in include/agmm_attn.h: validation, plans, launches.
#include <float.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "agmm_attn_internal.h"

using agmm::AttnParams;
using agmm::CacheParams;
using agmm::CacheView;
using agmm::RopeParams;

struct ag_rope_handle {
  ag_rope_desc desc;
  int device;
  uint64_t* turns;  // device
};

struct ag_attn_handle {
  ag_attn_desc desc;
  int device, num_wgs;
  char* ws;
  bool own_ws;
};

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr int kRotMax = 512;
constexpr int kDefaultCus = 256;
constexpr uint32_t kMaxThreads = 1u << 30;  // of one launch, so that thread numbers fit FastDiv

int hip_failed(hipError_t e) {
  agmm::set_last_hip_error((int)e);
  return e == hipErrorOutOfMemory ? AGMM_ERR_OOM : AGMM_ERR_HIP;
}
#define ATTN_HIP(x)                               \
  do {                                            \
    const hipError_t e_ = (x);                    \
    if (e_ != hipSuccess) return hip_failed(e_);  \
  } while (0)

bool aligned(const void* p, uintptr_t n) { return p != nullptr && ((uintptr_t)p & (n - 1)) == 0; }

int64_t align256(int64_t x) { return (x + 255) & ~(int64_t)255; }

// The handle's device has to be the current one.
int check_device(int device) {
  int cur = -1;
  ATTN_HIP(hipGetDevice(&cur));
  return cur == device ? AGMM_OK : AGMM_ERR_WRONG_DEVICE;
}

bool valid_rope(const ag_rope_desc* d) {
  if (!d || (d->dtype != AGMM_F16 && d->dtype != AGMM_BF16)) return false;
  if (d->head_dim < 2 || d->head_dim > 1024) return false;
  if (d->rot_dim < 2 || d->rot_dim > std::min(d->head_dim, kRotMax) || d->rot_dim % 2) return false;
  if (d->rot_start < 0 || d->rot_start > d->head_dim - d->rot_dim) return false;
  if (d->pairing != AG_ROPE_HALF && d->pairing != AG_ROPE_INTERLEAVED) return false;
  if (!isfinite((float)d->magnitude)) return false;  // as the kernels take it
  if (d->thetas) {
    for (int i = 0; i < d->rot_dim / 2; ++i)
      if (!isfinite(d->thetas[i])) return false;
    return true;
  }
  if (d->scaling < AG_ROPE_NONE || d->scaling > AG_ROPE_INDEX) return false;
  if (!(d->base > 1.0) || !isfinite(d->base)) return false;
  if (d->scaling != AG_ROPE_NONE && (!(d->factor > 0.0) || !isfinite(d->factor))) return false;
  if (d->scaling == AG_ROPE_BASE && d->rot_dim == 2) return false;
  if (d->scaling == AG_ROPE_TURNS || d->scaling == AG_ROPE_INDEX)
    if (!(d->original_len > 0.0) || !isfinite(d->original_len) || !(d->low > 0.0) ||
        !(d->high > d->low) || !isfinite(d->high))
      return false;
  return true;
}

void make_thetas(const ag_rope_desc& d, double* out) {
  const int n = d.rot_dim / 2;
  if (d.thetas) {
    memcpy(out, d.thetas, n * sizeof(double));
    return;
  }
  double base = d.base;
  if (d.scaling == AG_ROPE_BASE) base *= pow(d.factor, d.rot_dim / (d.rot_dim - 2.0));
  auto index_of = [&](double turns) {
    return d.rot_dim * log(d.original_len / (kTwoPi * turns)) / (2.0 * log(d.base));
  };
  const double i0 = std::max(floor(index_of(d.high)), 0.0);
  const double i1 = std::min(ceil(index_of(d.low)), d.rot_dim - 1.0);
  for (int i = 0; i < n; ++i) {
    const double t = pow(base, -2.0 * i / d.rot_dim);
    double g = 1.0;
    if (d.scaling == AG_ROPE_LINEAR) g = 0.0;
    if (d.scaling == AG_ROPE_TURNS)
      g = std::min(1.0, std::max(0.0, (d.original_len * t / kTwoPi - d.low) / (d.high - d.low)));
    if (d.scaling == AG_ROPE_INDEX)
      g = 1.0 - std::min(1.0, std::max(0.0, (i - i0) / std::max(i1 - i0, 0.001)));
    out[i] = d.scaling == AG_ROPE_NONE || d.scaling == AG_ROPE_BASE ? t
                                                                    : t * (g + (1.0 - g) / d.factor);
  }
}

agmm::RopePlan plan_of(const ag_rope_handle& h) {
  agmm::RopePlan r;
  r.turns = h.turns;
  r.magnitude = (float)h.desc.magnitude;
  r.head_dim = h.desc.head_dim;
  r.rot_dim = h.desc.rot_dim;
  r.rot_start = h.desc.rot_start;
  return r;
}

// Whether two strides lead to the same n places: that of a dimension of one says nothing.
bool same_step(int64_t n, int64_t a, int64_t b) { return n <= 1 || a == b; }

// The units that threads take of a head.
void rope_units(const ag_rope_desc& d, int64_t heads, RopeParams* p) {
  p->rot_units = d.pairing == AG_ROPE_HALF ? (d.rot_dim / 2 + 7) / 8 : (d.rot_dim / 2 + 3) / 4;
  p->pass_units0 = (d.rot_start + 7) / 8;
  const int behind = (d.head_dim - d.rot_start - d.rot_dim + 7) / 8;
  const int pass = p->in_place ? 0 : p->pass_units0 + behind;
  p->units = agmm::fast_div((uint32_t)(p->rot_units + pass));
  p->heads = agmm::fast_div((uint32_t)heads);
}

int check_cache(const ag_kv_cache* c) {
  if (!c) return AGMM_ERR_INVALID_ARG;
  if (c->dtype != AGMM_F16 && c->dtype != AGMM_BF16) return AGMM_ERR_INVALID_ARG;
  if (c->storage < AG_KV_16BIT || c->storage > AG_KV_MXFP4) return AGMM_ERR_INVALID_ARG;
  if (c->head_dim < 1 || c->kv_heads < 1 || c->page_size < 1 || c->num_pages < 0)
    return AGMM_ERR_INVALID_ARG;
  if (c->head_dim > 256 || c->head_dim % (c->storage == AG_KV_16BIT ? 8 : 32))
    return AGMM_ERR_UNSUPPORTED;
  if (c->num_pages >= ((int64_t)1 << 31) || c->num_pages * c->page_size >= ((int64_t)1 << 31))
    return AGMM_ERR_UNSUPPORTED;
  if (c->page_stride < 0 || c->head_stride < 0 || c->row_stride < 0 ||
      (c->page_stride | c->head_stride | c->row_stride) & 15)
    return AGMM_ERR_INVALID_ARG;
  const int64_t wide = (int64_t)1 << 32;
  if (c->page_stride >= wide || c->row_stride >= wide) return AGMM_ERR_UNSUPPORTED;
  if (c->num_pages > 0 && (!aligned(c->k, 16) || !aligned(c->v, 16))) return AGMM_ERR_INVALID_ARG;
  if (c->storage != AG_KV_16BIT) {
    if (c->scale_page < 0 || c->scale_head < 0 || c->scale_row < 0 ||
        (c->scale_page | c->scale_head | c->scale_row) & 3)
      return AGMM_ERR_INVALID_ARG;
    if (c->scale_page >= wide || c->scale_row >= wide) return AGMM_ERR_UNSUPPORTED;
    if (c->num_pages > 0 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
      return AGMM_ERR_INVALID_ARG;
  } else if (c->k_scale || c->v_scale) {
    return AGMM_ERR_INVALID_ARG;
  }
  return AGMM_OK;
}

CacheView view_of(const ag_kv_cache& c) {
  CacheView v;
  v.k = (char*)c.k;
  v.v = (char*)c.v;
  v.ks = (char*)c.k_scale;
  v.vs = (char*)c.v_scale;
  v.page = (uint32_t)c.page_stride;
  v.head = c.head_stride;
  v.row = (uint32_t)c.row_stride;
  v.s_page = (uint32_t)c.scale_page;
  v.s_head = c.scale_head;
  v.s_row = (uint32_t)c.scale_row;
  v.page_size = agmm::fast_div((uint32_t)c.page_size);
  v.rows = (uint32_t)(c.num_pages * c.page_size);
  v.head_dim = c.head_dim;
  v.kv_heads = c.kv_heads;
  return v;
}

// Tokens of one launch for `per_token` threads each.
int64_t tokens_per_launch(uint64_t per_token) {
  return std::max<int64_t>(1, (int64_t)(kMaxThreads / std::max<uint64_t>(1, per_token)));
}

// The two directions of the cache's traffic share their arguments.
struct Traffic {
  const uint16_t *k, *v;
  uint16_t *k_out, *v_out;
  int64_t k_token, k_head, v_token, v_head;
  const int64_t *slots, *positions;
};

CacheParams traffic_of(const ag_kv_cache& c, const Traffic& t, int64_t t0, int64_t n) {
  CacheParams p;
  memset(&p, 0, sizeof(p));
  p.c = view_of(c);
  p.k = t.k ? t.k + t0 * t.k_token : nullptr;
  p.v = t.v ? t.v + t0 * t.v_token : nullptr;
  p.k_out = t.k_out ? t.k_out + t0 * t.k_token : nullptr;
  p.v_out = t.v_out ? t.v_out + t0 * t.v_token : nullptr;
  p.k_token = t.k_token;
  p.k_head = t.k_head;
  p.v_token = t.v_token;
  p.v_head = t.v_head;
  p.slots = t.slots + t0;
  p.positions = t.positions ? t.positions + t0 : nullptr;
  p.chunks = agmm::fast_div((uint32_t)c.head_dim / 8);
  p.heads = agmm::fast_div((uint32_t)c.kv_heads);
  p.total = (uint32_t)(n * c.kv_heads * (c.head_dim / 8));
  return p;
}

int check_attn(const ag_attn_desc* d) {
  if (!d) return AGMM_ERR_INVALID_ARG;
  if (d->dtype != AGMM_F16 && d->dtype != AGMM_BF16) return AGMM_ERR_INVALID_ARG;
  if (d->storage < AG_KV_16BIT || d->storage > AG_KV_MXFP4) return AGMM_ERR_INVALID_ARG;
  if (d->head_dim < 1 || d->q_heads < 1 || d->kv_heads < 1 || d->q_heads % d->kv_heads ||
      d->window < 0 || d->num_wgs < 0 || d->num_wgs > agmm::kAttnMaxWgs)
    return AGMM_ERR_INVALID_ARG;
  if (!(d->scale >= 0.0f) || !isfinite(d->scale) || !(d->soft_cap >= 0.0f) ||
      !isfinite(d->soft_cap))
    return AGMM_ERR_INVALID_ARG;
  if (d->head_dim > 256 || d->head_dim % (d->storage == AG_KV_16BIT ? 8 : 32))
    return AGMM_ERR_UNSUPPORTED;
  if (d->q_heads > (1 << 20)) return AGMM_ERR_UNSUPPORTED;
  return AGMM_OK;
}

// Workgroups of a run: as many as the compute units hold at once.
int workgroups(const ag_attn_desc& d, int num_cus) {
  return d.num_wgs ? d.num_wgs
                   : agmm::attn_per_cu(d.storage, agmm::attn_padded(d.head_dim)) * num_cus;
}

// Two partial results for each wave of a run, and three counters.
int attn_rows(const ag_attn_desc& d) { return std::min(16, d.q_heads / d.kv_heads); }
int64_t partials_bytes(const ag_attn_desc& d, int wgs) {
  return align256((int64_t)2 * 4 * wgs * attn_rows(d) * (agmm::attn_padded(d.head_dim) + 2) * 4);
}
int64_t attn_bytes(const ag_attn_desc& d, int wgs) {
  return partials_bytes(d, wgs) + align256((int64_t)3 * 4 * wgs * 4);
}

}  // namespace

extern "C" {

void ag_rope_desc_init(ag_rope_desc* d) {
  if (!d) return;
  memset(d, 0, sizeof(*d));
  d->dtype = AGMM_BF16;
  d->head_dim = d->rot_dim = 128;
  d->base = 10000.0;
  d->factor = 1.0;
  d->low = 1.0;
  d->high = 4.0;
  d->magnitude = 1.0;
}

int ag_rope_thetas(const ag_rope_desc* desc, double* out) {
  if (!valid_rope(desc) || !out) return AGMM_ERR_INVALID_ARG;
  make_thetas(*desc, out);
  return AGMM_OK;
}

int ag_rope_create(const ag_rope_desc* desc, ag_rope_handle** out_handle) {
  if (!valid_rope(desc) || !out_handle) return AGMM_ERR_INVALID_ARG;
  *out_handle = nullptr;
  double th[kRotMax / 2];
  make_thetas(*desc, th);
  uint64_t turns[kRotMax / 2] = {};
  for (int i = 0; i < desc->rot_dim / 2; ++i) {
    // the fraction of a turn, in 64 bits: the long double's mantissa holds all of them
    long double t = (long double)th[i] / 6.283185307179586476925286766559006L;
    t -= floorl(t);
    const long double f = roundl(t * 18446744073709551616.0L);
    turns[i] = f >= 18446744073709551616.0L ? 0 : (uint64_t)f;
  }
  ag_rope_handle* h = new (std::nothrow) ag_rope_handle;
  if (!h) return AGMM_ERR_OOM;
  h->desc = *desc;
  h->desc.thetas = nullptr;
  h->turns = nullptr;
  const size_t bytes = (size_t)((desc->rot_dim / 2 + 7) & ~7) * sizeof(uint64_t);
  hipError_t e = hipGetDevice(&h->device);
  if (e == hipSuccess) e = hipMalloc((void**)&h->turns, bytes);
  if (e == hipSuccess) e = hipMemcpy(h->turns, turns, bytes, hipMemcpyHostToDevice);
  if (e != hipSuccess) {
    if (h->turns) (void)hipFree(h->turns);
    delete h;
    return hip_failed(e);
  }
  *out_handle = h;
  return AGMM_OK;
}

int ag_rope_destroy(ag_rope_handle* h) {
  if (!h) return AGMM_OK;
  const int rc = check_device(h->device);
  if (rc != AGMM_OK) return rc;
  const hipError_t a = hipDeviceSynchronize(), b = hipFree(h->turns);
  delete h;
  if (a != hipSuccess || b != hipSuccess) return hip_failed(a != hipSuccess ? a : b);
  return AGMM_OK;
}

int ag_rope_run(ag_rope_handle* h, const void* x, int64_t x_batch, int64_t x_token, int64_t x_head,
                void* y, int64_t y_batch, int64_t y_token, int64_t y_head, const int64_t* positions,
                int64_t pos_batch, int64_t batch, int64_t tokens, int64_t heads, int gradient,
                void* hip_stream) {
  if (!h || batch < 0 || tokens < 0 || heads < 0 || (gradient != 0 && gradient != 1))
    return AGMM_ERR_INVALID_ARG;
  if (batch == 0 || tokens == 0 || heads == 0) return AGMM_OK;
  if (!aligned(x, 2) || !aligned(y, 2) || !aligned(positions, 8)) return AGMM_ERR_INVALID_ARG;
  if (heads > (1 << 20)) return AGMM_ERR_UNSUPPORTED;
  const int rc = check_device(h->device);
  if (rc != AGMM_OK) return rc;
  RopeParams p;
  memset(&p, 0, sizeof(p));
  p.plan = plan_of(*h);
  p.x_batch = x_batch;
  p.x_token = x_token;
  p.x_head = x_head;
  p.y_batch = y_batch;
  p.y_token = y_token;
  p.y_head = y_head;
  p.pos_batch = pos_batch;
  p.in_place = x == y && same_step(batch, x_batch, y_batch) && same_step(tokens, x_token, y_token) &&
               same_step(heads, x_head, y_head);
  rope_units(h->desc, heads, &p);
  const uint64_t per_token = (uint64_t)p.units.d * p.heads.d;
  const int64_t step = tokens_per_launch(per_token), bstep = 65535;
  for (int64_t b0 = 0; b0 < batch; b0 += bstep)
    for (int64_t t0 = 0; t0 < tokens; t0 += step) {
      const int64_t n = std::min(step, tokens - t0);
      p.x = (const uint16_t*)x + b0 * x_batch + t0 * x_token;
      p.y = (uint16_t*)y + b0 * y_batch + t0 * y_token;
      p.positions = positions + b0 * pos_batch + t0;
      p.total = (uint32_t)(n * (int64_t)per_token);
      ATTN_HIP(agmm::launch_rope(p, h->desc.dtype, h->desc.pairing, gradient,
                                 std::min(bstep, batch - b0), (hipStream_t)hip_stream));
    }
  return AGMM_OK;
}

int ag_kv_append(const ag_kv_cache* cache, const void* k, int64_t k_token, int64_t k_head,
                 const void* v, int64_t v_token, int64_t v_head, const int64_t* slots,
                 int64_t tokens, void* hip_stream) {
  const int rc = check_cache(cache);
  if (rc != AGMM_OK) return rc;
  if (tokens < 0) return AGMM_ERR_INVALID_ARG;
  if (tokens == 0) return AGMM_OK;
  if (!aligned(k, 2) || !aligned(v, 2) || !aligned(slots, 8)) return AGMM_ERR_INVALID_ARG;
  if (cache->kv_heads > (1 << 20)) return AGMM_ERR_UNSUPPORTED;
  const Traffic t = {(const uint16_t*)k, (const uint16_t*)v, nullptr, nullptr, k_token, k_head,
                     v_token, v_head, slots, nullptr};
  const int64_t step = tokens_per_launch((uint64_t)cache->kv_heads * (cache->head_dim / 8));
  for (int64_t t0 = 0; t0 < tokens; t0 += step) {
    const CacheParams p = traffic_of(*cache, t, t0, std::min(step, tokens - t0));
    ATTN_HIP(agmm::launch_append(p, nullptr, cache->dtype, cache->storage, 0,
                                 (hipStream_t)hip_stream));
  }
  return AGMM_OK;
}

int ag_kv_append_rope(const ag_kv_cache* cache, ag_rope_handle* rope, const void* q,
                      int64_t q_token, int64_t q_head, int64_t q_heads, void* q_out,
                      int64_t qo_token, int64_t qo_head, const void* k, int64_t k_token,
                      int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                      const int64_t* positions, const int64_t* slots, int64_t tokens,
                      void* hip_stream) {
  int rc = check_cache(cache);
  if (rc != AGMM_OK) return rc;
  if (!rope || rope->desc.dtype != cache->dtype || rope->desc.head_dim != cache->head_dim ||
      tokens < 0 || q_heads < 0)
    return AGMM_ERR_INVALID_ARG;
  if (tokens == 0) return AGMM_OK;
  if (!aligned(k, 2) || !aligned(v, 2) || !aligned(slots, 8) || !aligned(positions, 8) ||
      (q_heads > 0 && (!aligned(q, 2) || !aligned(q_out, 2))))
    return AGMM_ERR_INVALID_ARG;
  if (cache->kv_heads > (1 << 20) || q_heads > (1 << 20)) return AGMM_ERR_UNSUPPORTED;
  rc = check_device(rope->device);
  if (rc != AGMM_OK) return rc;
  const Traffic t = {(const uint16_t*)k, (const uint16_t*)v, nullptr, nullptr, k_token, k_head,
                     v_token, v_head, slots, positions};
  RopeParams r;
  memset(&r, 0, sizeof(r));
  r.plan = plan_of(*rope);
  r.x_token = q_token;
  r.x_head = q_head;
  r.y_token = qo_token;
  r.y_head = qo_head;
  r.in_place = q == q_out && same_step(tokens, q_token, qo_token) && same_step(q_heads, q_head, qo_head);
  rope_units(rope->desc, std::max<int64_t>(1, q_heads), &r);
  const uint64_t q_threads = q_heads ? (uint64_t)r.units.d * r.heads.d : 0;
  const int64_t step = tokens_per_launch(
      std::max(q_threads, (uint64_t)cache->kv_heads * (cache->head_dim / 8)));
  for (int64_t t0 = 0; t0 < tokens; t0 += step) {
    const int64_t n = std::min(step, tokens - t0);
    CacheParams p = traffic_of(*cache, t, t0, n);
    p.plan = r.plan;
    r.x = (const uint16_t*)q + t0 * q_token;
    r.y = (uint16_t*)q_out + t0 * qo_token;
    r.positions = positions + t0;
    r.total = (uint32_t)(n * (int64_t)q_threads);
    p.q_blocks = (r.total + 255) / 256;
    ATTN_HIP(agmm::launch_append(p, &r, cache->dtype, cache->storage, rope->desc.pairing,
                                 (hipStream_t)hip_stream));
  }
  return AGMM_OK;
}

int ag_kv_read(const ag_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k_out,
               int64_t k_token, int64_t k_head, void* v_out, int64_t v_token, int64_t v_head,
               void* hip_stream) {
  const int rc = check_cache(cache);
  if (rc != AGMM_OK) return rc;
  if (tokens < 0) return AGMM_ERR_INVALID_ARG;
  if (tokens == 0) return AGMM_OK;
  if (!aligned(k_out, 2) || !aligned(v_out, 2) || !aligned(slots, 8)) return AGMM_ERR_INVALID_ARG;
  if (cache->kv_heads > (1 << 20)) return AGMM_ERR_UNSUPPORTED;
  const Traffic t = {nullptr, nullptr, (uint16_t*)k_out, (uint16_t*)v_out, k_token, k_head,
                     v_token, v_head, slots, nullptr};
  const int64_t step = tokens_per_launch((uint64_t)cache->kv_heads * (cache->head_dim / 8));
  for (int64_t t0 = 0; t0 < tokens; t0 += step) {
    const CacheParams p = traffic_of(*cache, t, t0, std::min(step, tokens - t0));
    ATTN_HIP(agmm::launch_read(p, cache->dtype, cache->storage, (hipStream_t)hip_stream));
  }
  return AGMM_OK;
}

void ag_attn_desc_init(ag_attn_desc* d) {
  if (!d) return;
  memset(d, 0, sizeof(*d));
  d->dtype = AGMM_BF16;
  d->head_dim = 128;
  d->q_heads = d->kv_heads = 1;
}

int64_t ag_attn_workspace_bytes(const ag_attn_desc* desc) {
  const int rc = check_attn(desc);
  return rc != AGMM_OK ? rc : attn_bytes(*desc, workgroups(*desc, kDefaultCus));
}

int ag_attn_create(const ag_attn_desc* desc, void* workspace, size_t workspace_bytes,
                   ag_attn_handle** out_handle) {
  const int rc = check_attn(desc);
  if (rc != AGMM_OK) return rc;
  if (!out_handle) return AGMM_ERR_INVALID_ARG;
  *out_handle = nullptr;
  int device = -1, cus = 0;
  ATTN_HIP(hipGetDevice(&device));
  ATTN_HIP(hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device));
  const int wgs = workgroups(*desc, std::min(cus, kDefaultCus));
  const int64_t bytes = attn_bytes(*desc, wgs), counters = partials_bytes(*desc, wgs);
  if (workspace && (!aligned(workspace, 256) || workspace_bytes < (size_t)bytes))
    return AGMM_ERR_INVALID_ARG;
  ag_attn_handle* h = new (std::nothrow) ag_attn_handle;
  if (!h) return AGMM_ERR_OOM;
  h->desc = *desc;
  h->device = device;
  h->num_wgs = wgs;
  h->own_ws = !workspace;
  h->ws = (char*)workspace;
  hipError_t e = hipSuccess;
  if (h->own_ws) e = hipMalloc((void**)&h->ws, (size_t)bytes);
  if (e == hipSuccess) e = hipMemset(h->ws + counters, 0, (size_t)(bytes - counters));
  if (e == hipSuccess) e = hipStreamSynchronize(nullptr);
  if (e != hipSuccess) {
    if (h->own_ws && h->ws) (void)hipFree(h->ws);
    delete h;
    return hip_failed(e);
  }
  *out_handle = h;
  return AGMM_OK;
}

int ag_attn_destroy(ag_attn_handle* h) {
  if (!h) return AGMM_OK;
  const int rc = check_device(h->device);
  if (rc != AGMM_OK) return rc;
  const hipError_t a = hipDeviceSynchronize();
  const hipError_t b = h->own_ws ? hipFree(h->ws) : hipSuccess;
  delete h;
  if (a != hipSuccess || b != hipSuccess) return hip_failed(a != hipSuccess ? a : b);
  return AGMM_OK;
}

int ag_attn_run(ag_attn_handle* h, const ag_kv_cache* cache, const void* q, int64_t q_batch,
                int64_t q_head, const int32_t* page_table, int64_t table_row, int64_t table_len,
                const int32_t* lens, int64_t batch, void* out, int64_t o_batch, int64_t o_head,
                float* lse, void* hip_stream) {
  if (!h) return AGMM_ERR_INVALID_ARG;
  int rc = check_cache(cache);
  if (rc != AGMM_OK) return rc;
  const ag_attn_desc& d = h->desc;
  if (cache->dtype != d.dtype || cache->storage != d.storage || cache->head_dim != d.head_dim ||
      cache->kv_heads != d.kv_heads || batch < 0 || table_len < 0)
    return AGMM_ERR_INVALID_ARG;
  if (batch == 0) return AGMM_OK;
  if (!aligned(q, 2) || !aligned(out, 2) || !aligned(lens, 4) ||
      (table_len > 0 && !aligned(page_table, 4)) || (lse && !aligned(lse, 4)))
    return AGMM_ERR_INVALID_ARG;
  const int64_t most = (int64_t)1 << 31;
  if (batch >= most || table_len >= most || table_len * cache->page_size >= most)
    return AGMM_ERR_UNSUPPORTED;
  AttnParams p;
  memset(&p, 0, sizeof(p));
  p.c = view_of(*cache);
  p.group = d.q_heads / d.kv_heads;
  p.q_groups = (p.group + 15) / 16;
  p.rows = attn_rows(d);
  p.capacity = cache->num_pages > 0 ? (int32_t)(table_len * cache->page_size) : 0;
  // every tile has a 32-bit number
  const int64_t seen = d.window ? std::min(d.window, (int64_t)p.capacity) : p.capacity;
  const int64_t tiles = (seen + 15 + agmm::kAttnTile - 1) / agmm::kAttnTile;
  const int64_t heads = (int64_t)d.kv_heads * p.q_groups;
  if ((double)tiles * heads * batch >= (double)most) return AGMM_ERR_UNSUPPORTED;
  rc = check_device(h->device);
  if (rc != AGMM_OK) return rc;
  p.q = (const uint16_t*)q;
  p.out = (uint16_t*)out;
  p.lse = lse;
  p.table = page_table;
  p.lens = lens;
  p.q_batch = q_batch;
  p.q_head = q_head;
  p.o_batch = o_batch;
  p.o_head = o_head;
  p.table_row = table_row;
  p.partials = (float*)h->ws;
  p.counters = (uint32_t*)(h->ws + partials_bytes(d, h->num_wgs));
  p.window = d.window;
  p.num_pages = (int32_t)cache->num_pages;
  p.batch = (int32_t)batch;
  p.q_heads = d.q_heads;
  const double log2e = 1.4426950408889634073599;
  const double scale = d.scale != 0.0f ? d.scale : 1.0 / sqrt((double)d.head_dim);
  // (finite, and the cap's above 0, at the ends of their ranges)
  p.scale = (float)std::min(scale * log2e, (double)FLT_MAX);
  p.cap = (float)std::min(d.soft_cap * log2e, (double)FLT_MAX);
  p.inv_cap = d.soft_cap != 0.0f
                  ? (float)std::min(std::max(2.0 * log2e * scale / d.soft_cap, (double)FLT_MIN),
                                    (double)FLT_MAX)
                  : 0.0f;
  const int64_t grid = std::min<int64_t>(h->num_wgs, std::max<int64_t>(1, tiles * heads * batch));
  ATTN_HIP(agmm::launch_attn(p, d.dtype, d.storage, (int)grid, (hipStream_t)hip_stream));
  return AGMM_OK;
}

}  // extern "C"
