// Host side of the C ABI declared in include/agmm_long.h: validation, launches.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "agmm_long_internal.h"

using namespace agmm;

namespace {

constexpr int kCompute = 256;  // compute units
constexpr int64_t kWide = (int64_t)1 << 31;
constexpr int64_t kReach = kWide - (1 << 20);  // of a table: loops go past their ends, in 32 bits
constexpr int64_t kHeads = 1 << 21;  // sequences times kv heads: each has a workgroup of up to 1024 threads

// ---- prefixes ----

struct Scratch {
  int64_t slots, sums, stats, own, own_stats, bytes;  // offsets behind the groups
};

int prefix_wgs(const ag_attn_desc& d) {
  return d.num_wgs ? std::max(2, d.num_wgs) : prefix_per_cu(attn_padded(d.head_dim)) * kCompute;
}

// A strip for every 128 rows of a kv head, and an unfilled one for each group; a piece for each strip and for
// each workgroup. (Doubles: sizes past 2^31 are refused, so what they round does not count.)
int scratch_of(const ag_attn_desc& d, int64_t batch, int64_t groups, Scratch* s) {
  if (batch < 0 || groups < 0) return AGMM_ERR_INVALID_ARG;
  const int64_t group = d.q_heads / d.kv_heads;
  if (batch >= kWide || groups >= kWide || (double)batch * group >= (double)kWide) return AGMM_ERR_UNSUPPORTED;
  const int64_t strips = batch * group / kPrefixRows + std::min(batch, groups);
  if ((double)strips * d.kv_heads >= (double)kWide / 2) return AGMM_ERR_UNSUPPORTED;
  // (threads of the joining: numbers of 32 bits)
  if ((double)batch * d.q_heads * (d.head_dim / 4) >= (double)kWide) return AGMM_ERR_UNSUPPORTED;
  s->slots = strips * d.kv_heads + prefix_wgs(d);
  s->sums = align256(groups * (int64_t)sizeof(PrefixGroup));
  s->stats = s->sums + s->slots * kPrefixRows * attn_padded(d.head_dim) * 4;
  s->own = s->stats + align256(s->slots * kPrefixRows * 2 * 4);
  s->own_stats = s->own + batch * d.q_heads * attn_padded(d.head_dim) * 4;
  s->bytes = align256(s->own_stats + batch * d.q_heads * 2 * 4);
  return AGMM_OK;
}

// ---- what the others share ----

// Page tables and lengths of a batch.
int check_tables(const ag_kv_cache& c, const int32_t* table, int64_t table_len, const int32_t* lens,
                 int64_t batch) {
  if (batch < 0 || table_len < 0) return AGMM_ERR_INVALID_ARG;
  if (batch == 0) return AGMM_OK;
  if (!aligned(lens, 4) || (table_len > 0 && !aligned(table, 4))) return AGMM_ERR_INVALID_ARG;
  if (batch >= kWide || table_len >= kWide || table_len * c.page_size >= kReach ||
      batch > kHeads / c.kv_heads)
    return AGMM_ERR_UNSUPPORTED;
  return AGMM_OK;
}

int check_index(const ag_kv_cache* cache, const ag_page_index* x) {
  const int rc = check_cache(cache);
  if (rc != AGMM_OK) return rc;
  if (!x || (cache->num_pages > 0 && (!aligned(x->codes, 16) || !x->scales))) return AGMM_ERR_INVALID_ARG;
  return AGMM_OK;
}

IndexParams index_params(const ag_kv_cache& c, const ag_page_index& x, const int32_t* table, int64_t table_row,
                         int64_t table_len, const int32_t* lens) {
  IndexParams p;
  memset(&p, 0, sizeof(p));
  p.c = view_of(c);
  p.codes = x.codes;
  p.scales = x.scales;
  p.table = table;
  p.lens = lens;
  p.table_row = table_row;
  p.num_pages = (int32_t)c.num_pages;
  p.pages = (int32_t)table_len;
  return p;
}

// Workgroups for each of `n` sequences, or their heads: `wgs` in all, as long as each has an item for its waves.
int splits_of(int64_t wgs, int64_t n, int64_t items) {
  const int64_t most = std::max<int64_t>(1, (items + 3) / 4);
  n = std::min(std::max<int64_t>(1, wgs / std::max<int64_t>(1, n)), most);
  return (int)n;
}

int check_choice(int64_t budget, int64_t sink, int64_t recent) {
  if (budget < 1 || sink < 0 || recent < 0 || sink > budget || recent > budget - sink)
    return AGMM_ERR_INVALID_ARG;
  return budget >= kWide ? AGMM_ERR_UNSUPPORTED : AGMM_OK;
}

int64_t key_stride(int64_t table_len) { return (table_len + 3) & ~(int64_t)3; }

}  // namespace

extern "C" {

int64_t ag_prefix_scratch_bytes(const ag_attn_desc* desc, int64_t batch, int64_t groups) {
  int rc = check_attn(desc);
  if (rc != AGMM_OK) return rc;
  Scratch s;
  rc = scratch_of(*desc, batch, groups, &s);
  return rc != AGMM_OK ? rc : s.bytes;
}

int ag_prefix_run(ag_attn_handle* h, const ag_kv_cache* cache, const void* q, int64_t q_batch,
                  int64_t q_head, const int32_t* prefix_table, int64_t prefix_row, int64_t prefix_pages,
                  const int32_t* prefix_lens, const int32_t* starts, int64_t groups,
                  const int32_t* page_table, int64_t table_row, int64_t table_len, const int32_t* lens,
                  int64_t batch, void* out, int64_t o_batch, int64_t o_head, float* lse, void* scratch,
                  int64_t scratch_bytes, void* hip_stream) {
  if (!h || groups < 0 || prefix_pages < 0) return AGMM_ERR_INVALID_ARG;
  const ag_attn_desc& d = attn_desc(h);
  if (d.window != 0) return AGMM_ERR_UNSUPPORTED;
  AttnParams a;
  int grid = 0;
  int rc = attn_params(h, cache, q, q_batch, q_head, page_table, table_row, table_len, lens, batch, out,
                       o_batch, o_head, lse, &a, &grid);
  if (rc != AGMM_OK || grid == 0) return rc;
  if (a.cap == 0.0f && a.scale > 0x1p64f) return AGMM_ERR_UNSUPPORTED;
  Scratch s;
  rc = scratch_of(d, batch, groups, &s);
  if (rc != AGMM_OK) return rc;
  if (groups == 0) {
    ATTN_HIP(launch_attn(a, d.dtype, d.storage, grid, (hipStream_t)hip_stream));
    return AGMM_OK;
  }
  if (!aligned(prefix_lens, 4) || (prefix_pages > 0 && !aligned(prefix_table, 4)) ||
      (starts ? !aligned(starts, 4) : groups != 1) || !aligned(scratch, 256) || scratch_bytes < s.bytes)
    return AGMM_ERR_INVALID_ARG;
  if (prefix_pages >= kWide || prefix_pages * cache->page_size >= kReach) return AGMM_ERR_UNSUPPORTED;
  PrefixParams p;
  memset(&p, 0, sizeof(p));
  a.prefix.info = (PrefixGroup*)scratch;
  a.prefix.sums = (float*)((char*)scratch + s.sums);
  a.prefix.stats = (float*)((char*)scratch + s.stats);
  a.prefix.own = (float*)((char*)scratch + s.own);
  a.prefix.own_stats = (float*)((char*)scratch + s.own_stats);
  a.prefix.groups = (uint32_t)groups;
  p.own = a;
  p.table = prefix_table;
  p.table_row = prefix_row;
  p.capacity = cache->num_pages > 0 ? (int32_t)(prefix_pages * cache->page_size) : 0;
  p.lens = prefix_lens;
  p.starts = starts;
  p.least = 2;
  const int64_t tokens = 8192 / attn_padded(d.head_dim);
  const int64_t strips = s.slots - prefix_wgs(d);
  const int64_t tiles = (p.capacity + tokens - 1) / tokens;
  if ((double)tiles * strips >= (double)kWide) return AGMM_ERR_UNSUPPORTED;
  p.own_wgs = (uint32_t)attn_workgroups(h);   // that their workspace is for
  const int wgs = (int)std::min<int64_t>(prefix_wgs(d), std::max<int64_t>(2, tiles * strips + grid));
  ATTN_HIP(d.dtype == AGMM_F16 ? launch_prefix_f16(p, d.storage, wgs, (hipStream_t)hip_stream)
                               : launch_prefix_bf16(p, d.storage, wgs, (hipStream_t)hip_stream));
  ATTN_HIP(launch_prefix_join(p, d.dtype, (hipStream_t)hip_stream));
  return AGMM_OK;
}

int ag_attn_run_heads(ag_attn_handle* h, const ag_kv_cache* cache, const void* q, int64_t q_batch,
                      int64_t q_head, const int32_t* page_table, int64_t table_row, int64_t table_head,
                      int64_t table_len, const int32_t* lens, int64_t batch, void* out, int64_t o_batch,
                      int64_t o_head, float* lse, void* hip_stream) {
  AttnParams a;
  int grid = 0;
  const int rc = attn_params(h, cache, q, q_batch, q_head, page_table, table_row, table_len, lens, batch, out,
                             o_batch, o_head, lse, &a, &grid);
  if (rc != AGMM_OK || grid == 0) return rc;
  a.table_head = table_head;
  const ag_attn_desc& d = attn_desc(h);
  ATTN_HIP(launch_attn_heads(a, d.dtype, d.storage, grid, (hipStream_t)hip_stream));
  return AGMM_OK;
}

int ag_index_update(const ag_kv_cache* cache, const ag_page_index* index, const int32_t* page_table,
                    int64_t table_row, int64_t table_len, const int32_t* starts, const int32_t* lens,
                    int64_t batch, void* hip_stream) {
  int rc = check_index(cache, index);
  if (rc != AGMM_OK) return rc;
  rc = check_tables(*cache, page_table, table_len, lens, batch);
  if (rc != AGMM_OK) return rc;
  if (starts && !aligned(starts, 4)) return AGMM_ERR_INVALID_ARG;
  if (batch == 0 || table_len == 0 || cache->num_pages == 0) return AGMM_OK;
  IndexParams p = index_params(*cache, *index, page_table, table_row, table_len, lens);
  p.starts = starts;
  p.batch = fast_div((uint32_t)batch);
  p.step = fast_div((uint32_t)(4 * splits_of(8 * kCompute, batch, table_len * cache->kv_heads)));
  p.heads = fast_div((uint32_t)cache->kv_heads);
  ATTN_HIP(launch_index_update(p, cache->dtype, cache->storage, batch, (hipStream_t)hip_stream));
  return AGMM_OK;
}

int64_t ag_index_scratch_bytes(const ag_kv_cache* cache, int64_t table_len, int64_t batch) {
  const int rc = check_cache(cache);
  if (rc != AGMM_OK) return rc;
  if (table_len < 0 || batch < 0) return AGMM_ERR_INVALID_ARG;
  if (table_len >= kWide || batch > kHeads / cache->kv_heads) return AGMM_ERR_UNSUPPORTED;
  return table_len <= kFew ? 0 : batch * cache->kv_heads * key_stride(table_len) * 4;
}

int ag_index_select(const ag_kv_cache* cache, const ag_page_index* index, const void* q, int64_t q_batch,
                    int64_t q_head, int64_t q_heads, const int32_t* page_table, int64_t table_row,
                    int64_t table_len, const int32_t* lens, int64_t batch, int64_t budget, int64_t sink,
                    int64_t recent, int32_t* out_table, int32_t* out_lens, void* scratch,
                    int64_t scratch_bytes, void* hip_stream) {
  int rc = check_index(cache, index);
  if (rc != AGMM_OK) return rc;
  rc = check_choice(budget, sink, recent);
  if (rc != AGMM_OK) return rc;
  if (recent < 1 || q_heads < 1 || q_heads % cache->kv_heads) return AGMM_ERR_INVALID_ARG;
  if (q_heads / cache->kv_heads > 128) return AGMM_ERR_UNSUPPORTED;
  rc = check_tables(*cache, page_table, table_len, lens, batch);
  if (rc != AGMM_OK) return rc;
  if (batch == 0) return AGMM_OK;
  const int64_t bytes = ag_index_scratch_bytes(cache, table_len, batch);
  if (!aligned(q, 2) || !aligned(out_table, 4) || !aligned(out_lens, 4) ||
      (bytes > 0 && (!aligned(scratch, 16) || scratch_bytes < bytes)))
    return AGMM_ERR_INVALID_ARG;
  const int64_t heads = batch * cache->kv_heads;
  IndexParams p = index_params(*cache, *index, page_table, table_row, table_len, lens);
  if (cache->num_pages == 0) p.pages = 0;   // (nothing to read behind the index's pointers)
  p.q = (const uint16_t*)q;
  p.q_batch = q_batch;
  p.q_head = q_head;
  p.group = (int32_t)(q_heads / cache->kv_heads);
  p.keys = (uint32_t*)scratch;
  const int64_t at_once = 64 / (attn_padded(cache->head_dim) / 8);
  // (32 sequences of up to 32768 tokens, 8 kv heads: 17.4 us with 4 a compute unit, 12.3 with 8, 13.6 with 16)
  p.splits = splits_of(8 * kCompute, heads, (table_len + at_once - 1) / at_once);
  ChooseParams c;
  memset(&c, 0, sizeof(c));
  c.keys = p.keys;
  c.table = page_table;
  c.lens = lens;
  c.table_row = table_row;
  c.page_size = p.c.page_size;
  c.num_pages = p.num_pages;
  c.pages = c.items = p.pages;
  c.heads = cache->kv_heads;
  c.key_stride = (int32_t)key_stride(table_len);
  c.budget = (int32_t)budget;
  c.sink = (int32_t)sink;
  c.recent = (int32_t)recent;
  c.out = out_table;
  c.out_lens = out_lens;
  if (table_len <= kFew) {
    ATTN_HIP(launch_select(p, c, cache->dtype, batch, (hipStream_t)hip_stream));
    return AGMM_OK;
  }
  if (p.pages > 0) ATTN_HIP(launch_index_score(p, cache->dtype, batch, (hipStream_t)hip_stream));
  ATTN_HIP(launch_choose_pages(c, batch, (hipStream_t)hip_stream));
  return AGMM_OK;
}

int ag_mass_add(const ag_attn_desc* desc, const ag_kv_cache* cache, const void* q, int64_t q_batch,
                int64_t q_head, const float* lse, const int32_t* page_table, int64_t table_row,
                int64_t table_len, const int32_t* lens, int64_t batch, const float* mass,
                int64_t mass_batch, int64_t mass_head, float* out, int64_t out_batch, int64_t out_head,
                int64_t tokens, float decay, void* hip_stream) {
  int rc = check_attn(desc);
  if (rc != AGMM_OK) return rc;
  rc = check_cache(cache);
  if (rc != AGMM_OK) return rc;
  const ag_attn_desc& d = *desc;
  if (cache->dtype != d.dtype || cache->storage != d.storage || cache->head_dim != d.head_dim ||
      cache->kv_heads != d.kv_heads || tokens < 0 || !isfinite(decay))
    return AGMM_ERR_INVALID_ARG;
  rc = check_tables(*cache, page_table, table_len, lens, batch);
  if (rc != AGMM_OK) return rc;
  if (batch == 0 || tokens == 0) return AGMM_OK;
  if (!aligned(q, 2) || !aligned(lse, 4) || !aligned(mass, 4) || !aligned(out, 4)) return AGMM_ERR_INVALID_ARG;
  if (mass == out && ((batch > 1 && mass_batch != out_batch) || (d.kv_heads > 1 && mass_head != out_head)))
    return AGMM_ERR_INVALID_ARG;
  if (tokens >= kWide) return AGMM_ERR_UNSUPPORTED;
  MassParams m;
  memset(&m, 0, sizeof(m));
  AttnParams& p = m.a;
  p.c = view_of(*cache);
  p.q = (const uint16_t*)q;
  p.q_batch = q_batch;
  p.q_head = q_head;
  p.table = page_table;
  p.table_row = table_row;
  p.lens = lens;
  p.window = d.window;
  p.capacity = cache->num_pages > 0 ? (int32_t)(table_len * cache->page_size) : 0;
  p.num_pages = (int32_t)cache->num_pages;
  p.batch = (int32_t)batch;
  p.q_heads = d.q_heads;
  p.group = d.q_heads / d.kv_heads;
  p.q_groups = (p.group + 15) / 16;
  attn_scales(d, &p);
  m.mass = mass;
  m.out = out;
  m.lse = lse;
  m.mass_batch = mass_batch;
  m.mass_head = mass_head;
  m.out_batch = out_batch;
  m.out_head = out_head;
  m.tokens = (int32_t)tokens;
  m.decay = decay;
  const int64_t heads = batch * d.kv_heads;
  m.splits = splits_of(16 * kCompute, heads, (tokens + 63) / 64);
  ATTN_HIP(launch_mass(m, d.dtype, d.storage, (hipStream_t)hip_stream));
  return AGMM_OK;
}

int ag_evict_choose(const ag_kv_cache* cache, const float* mass, int64_t mass_batch, int64_t mass_head,
                    int64_t tokens, const int32_t* page_table, int64_t table_row, int64_t table_len,
                    const int32_t* lens, int64_t batch, int64_t budget, int64_t sink, int64_t recent,
                    int32_t* kept, float* out_mass, int32_t* out_lens, void* hip_stream) {
  int rc = check_cache(cache);
  if (rc != AGMM_OK) return rc;
  rc = check_choice(budget, sink, recent);
  if (rc != AGMM_OK) return rc;
  if (tokens < 0) return AGMM_ERR_INVALID_ARG;
  rc = check_tables(*cache, page_table, table_len, lens, batch);
  if (rc != AGMM_OK) return rc;
  if (batch == 0) return AGMM_OK;
  if ((tokens > 0 && !aligned(mass, 4)) || !aligned(kept, 4) || !aligned(out_lens, 4) ||
      (out_mass && !aligned(out_mass, 4)))
    return AGMM_ERR_INVALID_ARG;
  if (tokens >= kWide) return AGMM_ERR_UNSUPPORTED;
  ChooseParams c;
  memset(&c, 0, sizeof(c));
  c.mass = mass;
  c.mass_batch = mass_batch;
  c.mass_head = mass_head;
  c.table = page_table;
  c.lens = lens;
  c.table_row = table_row;
  c.page_size = fast_div((uint32_t)cache->page_size);
  c.num_pages = (int32_t)cache->num_pages;
  c.pages = (int32_t)table_len;
  c.items = (int32_t)std::min(tokens, table_len * cache->page_size);
  c.heads = cache->kv_heads;
  c.budget = (int32_t)budget;
  c.sink = (int32_t)sink;
  c.recent = (int32_t)recent;
  c.out = kept;
  c.out_mass = out_mass;
  c.out_lens = out_lens;
  ATTN_HIP(launch_choose_tokens(c, batch, (hipStream_t)hip_stream));
  return AGMM_OK;
}

int ag_evict_move(const ag_kv_cache* from, const int32_t* from_table, int64_t from_row, int64_t from_len,
                  const ag_kv_cache* to, const int32_t* to_table, int64_t to_row, int64_t to_len,
                  const int32_t* kept, int64_t budget, const int32_t* lens, int64_t batch,
                  void* hip_stream) {
  int rc = check_cache(from);
  if (rc != AGMM_OK) return rc;
  rc = check_cache(to);
  if (rc != AGMM_OK) return rc;
  if (from->dtype != to->dtype || from->storage != to->storage || from->head_dim != to->head_dim ||
      from->kv_heads != to->kv_heads || budget < 0)
    return AGMM_ERR_INVALID_ARG;
  rc = check_tables(*from, from_table, from_len, lens, batch);
  if (rc != AGMM_OK) return rc;
  rc = check_tables(*to, to_table, to_len, lens, batch);
  if (rc != AGMM_OK) return rc;
  if (batch == 0 || budget == 0 || from->num_pages == 0 || to->num_pages == 0) return AGMM_OK;
  if (!aligned(kept, 4)) return AGMM_ERR_INVALID_ARG;
  MoveParams m;
  memset(&m, 0, sizeof(m));
  const int row = from->storage == AG_KV_16BIT   ? 2 * from->head_dim
                  : from->storage == AG_KV_MXFP8 ? from->head_dim
                                                 : from->head_dim / 2;
  if (budget >= kWide / 2 / (row / 16)) return AGMM_ERR_UNSUPPORTED;
  m.from = view_of(*from);
  m.to = view_of(*to);
  m.from_table = from_table;
  m.to_table = to_table;
  m.from_row = from_row;
  m.to_row = to_row;
  m.from_len = (int32_t)from_len;
  m.to_len = (int32_t)to_len;
  m.from_pages = (int32_t)from->num_pages;
  m.to_pages = (int32_t)to->num_pages;
  m.kept = kept;
  m.lens = lens;
  m.budget = (int32_t)budget;
  m.chunks = fast_div((uint32_t)(row / 16));
  m.scale_bytes = from->storage == AG_KV_16BIT ? 0 : (from->head_dim / 32 + 3) / 4 * 4;
  ATTN_HIP(launch_move(m, batch, (hipStream_t)hip_stream));
  return AGMM_OK;
}

}  // extern "C"
