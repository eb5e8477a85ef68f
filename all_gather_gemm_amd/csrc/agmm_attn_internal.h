// Internal interface between the C ABI of agmm_attn.h and its gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "agmm_attn.h"
#include "agmm_internal.h"

namespace agmm {

// n / d for 0 <= n < 2^31 by one multiplication: with 2^(s-1) < d <= 2^s and
// mul = floor(2^32 (2^s - d) / d) + 1, n / d = (umulhi(mul, n) + n) >> s.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f;
  f.d = d;
  f.shift = 0;
  while ((1ull << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)((((1ull << 32) * ((1ull << f.shift) - d)) / d) + 1);
  return f;
}

// The rotation's plan, as the kernels see it.
struct RopePlan {
  const uint64_t* turns;  // [rot_dim / 2, padded to 8]: theta_i / 2 pi as fractions of 2^64
  float magnitude;
  int32_t head_dim, rot_dim, rot_start;
};

// Heads to rotate, of one batch entry (blockIdx.y): element strides.
struct RopeParams {
  RopePlan plan;
  const uint16_t* x;
  uint16_t* y;
  const int64_t* positions;
  int64_t x_batch, x_token, x_head, y_batch, y_token, y_head, pos_batch;
  int32_t in_place;         // the elements that pass through need no copy
  int32_t rot_units;        // units of a head that rotate (8 half pairs or 4 interleaved ones),
  int32_t pass_units0;      // and units of 8 elements in front of the rotated part
  FastDiv units;            // all units of a head
  FastDiv heads;
  uint32_t total;           // threads: tokens * heads * units
};

struct CacheView {
  char *k, *v, *ks, *vs;
  int64_t head, s_head;              // bytes
  uint32_t page, row, s_page, s_row;
  FastDiv page_size;
  uint32_t rows;                                   // num_pages * page_size
  int32_t head_dim, kv_heads;
};

struct CacheParams {
  CacheView c;
  const uint16_t *k, *v;     // append
  uint16_t *k_out, *v_out;   // read
  int64_t k_token, k_head, v_token, v_head;  // elements
  const int64_t* slots;
  const int64_t* positions;  // with a rotation
  RopePlan plan;
  FastDiv chunks, heads;     // 8-element chunks of a head; heads
  uint32_t total;            // threads: tokens * heads * chunks
  uint32_t q_blocks;         // leading workgroups that rotate q (RopeParams beside)
};

// What the kernel of shared prefixes leaves for the joining (agmm_prefix_kernel.h). The rows of a prefix are the q
// heads of one kv head of all the sequences, kPrefixRows of them a strip; a strip's tiles of tokens, strip
// after strip, are cut into runs of `quota`, one for each workgroup that works on prefixes. Workgroup w's piece of
// strip s is in slot w + s.
constexpr int kPrefixRows = 128;
struct PrefixGroup {
  int32_t first, end;       // sequences
  uint32_t tiles;           // of a strip
  uint32_t row_tiles;       // strips of a kv head
  uint32_t strip0, tile0;   // the first strip and tile
  uint32_t quota;
  uint32_t reserved;        // (two loads of 16 bytes)
};
struct PrefixView {
  PrefixGroup* info;        // [groups]
  float* sums;              // [slots][padded head_dim / 8][kPrefixRows][8]
  float* stats;             // [slots][kPrefixRows][2]: reference of the weights, and their sum
  float* own;               // [batch][q_heads][padded head_dim]: the average of the own tokens' values
  float* own_stats;         // [batch][q_heads][2]: maximum and sum
  uint32_t groups;
};
constexpr int64_t prefix_at(int64_t row, int e) { return ((int64_t)(e / 8) * kPrefixRows + row) * 8 + e % 8; }

struct AttnParams {
  CacheView c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const int32_t* table;
  const int32_t* lens;
  int64_t q_batch, q_head, o_batch, o_head, table_row;
  float* partials;         // [2 * 4 * workgroups]: rows x (padded head_dim + 2)
  uint32_t* counters;      // [3 * 4 * workgroups]
  int64_t window;          // 0 = all
  int32_t capacity;        // tokens that the table reaches
  int32_t num_pages;
  int32_t batch, q_heads;
  int32_t group, q_groups; // q heads of a kv head; 16-wide groups of them
  int32_t rows;            // of a partial result: q heads in the largest of these groups
  float scale;             // times log2 e
  float cap, inv_cap;      // cap * log2 e, and 2 log2 e * scale / cap; cap 0 = none
  int64_t table_head;      // from one kv head's page table to the next (launch_attn_heads)
  PrefixView prefix;       // (launch_prefix)
};

hipError_t launch_rope(const RopeParams& p, int dtype, int pairing, int gradient, int64_t batch,
                       hipStream_t s);
// rope: nullptr, or the rotation of q (its threads come in the leading q_blocks workgroups)
hipError_t launch_append(const CacheParams& p, const RopeParams* rope, int dtype, int storage,
                         int pairing, hipStream_t s);
hipError_t launch_read(const CacheParams& p, int dtype, int storage, hipStream_t s);
// padded head_dim of the attention kernels: 64, 128 or 256
inline int attn_padded(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
constexpr int kAttnTile = 128;     // tokens of a tile, the unit of the workgroups' shares
constexpr int kAttnMaxWgs = 1024;  // workgroups of a run
// Workgroups of the attention kernel that share a compute unit, by the registers of a tile: 16-bit
// rows of 256 spill with two (32 x 8192 tokens: 353 us with one, 394 with two).
constexpr int attn_per_cu(int storage, int padded) {
  return storage == AG_KV_16BIT && padded == 256 ? 1 : 2;
}
hipError_t launch_attn(const AttnParams& p, int dtype, int storage, int grid, hipStream_t s);
hipError_t launch_attn_heads(const AttnParams& p, int dtype, int storage, int grid, hipStream_t s);

// Of agmm_attn_api.cpp, for the rest of the host side.
int hip_failed(hipError_t e);                // remembers it; the ABI's code for it
int check_device(int device);                // has to be the current one
int check_cache(const ag_kv_cache* c);
int check_attn(const ag_attn_desc* d);
CacheView view_of(const ag_kv_cache& c);
void attn_scales(const ag_attn_desc& d, AttnParams* p);
// A run's arguments, checked, and its grid (0: nothing to do).
int attn_params(ag_attn_handle* h, const ag_kv_cache* cache, const void* q, int64_t q_batch, int64_t q_head,
                const int32_t* page_table, int64_t table_row, int64_t table_len, const int32_t* lens,
                int64_t batch, void* out, int64_t o_batch, int64_t o_head, float* lse, AttnParams* p,
                int* grid);
const ag_attn_desc& attn_desc(const ag_attn_handle* h);
int attn_workgroups(const ag_attn_handle* h);
inline bool aligned(const void* p, uintptr_t n) { return p != nullptr && ((uintptr_t)p & (n - 1)) == 0; }
inline int64_t align256(int64_t x) { return (x + 255) & ~(int64_t)255; }
#define ATTN_HIP(x)                                    \
  do {                                                 \
    const hipError_t e_ = (x);                         \
    if (e_ != hipSuccess) return agmm::hip_failed(e_); \
  } while (0)

}  // namespace agmm
