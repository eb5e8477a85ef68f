// Internal interface between the C ABI of agmm_long.h and its gfx950 kernels.
#pragma once

#include "agmm_attn_internal.h"
#include "agmm_long.h"

namespace agmm {

struct PrefixParams {
  AttnParams own;          // the sequences' own tokens; prefix: where the pieces go
  const int32_t* table;    // of the prefixes
  int64_t table_row;
  int32_t capacity;        // tokens that it reaches
  const int32_t* lens;     // of the prefixes
  const int32_t* starts;   // or nullptr: one group
  uint32_t least;          // tiles of a workgroup's run
  uint32_t own_wgs;        // workgroups on own tokens, at most
};
// Workgroups that share a compute unit, by their registers
constexpr int prefix_per_cu(int padded) { return padded == 256 ? 1 : 2; }
hipError_t launch_prefix_f16(const PrefixParams& p, int storage, int grid, hipStream_t s);
hipError_t launch_prefix_bf16(const PrefixParams& p, int storage, int grid, hipStream_t s);
hipError_t launch_prefix_join(const PrefixParams& p, int dtype, hipStream_t s);

struct IndexParams {
  CacheView c;
  int8_t* codes;
  uint8_t* scales;
  const int32_t* table;
  const int32_t* starts;   // or nullptr
  const int32_t* lens;
  int64_t table_row;
  int32_t num_pages, pages;  // of the cache; of a sequence's table
  // update
  FastDiv batch, step, heads;  // step: entries of a sequence at once, 4 a workgroup; heads: kv heads
  // select
  int32_t splits;            // workgroups of one sequence and head
  const uint16_t* q;
  int64_t q_batch, q_head;
  int32_t group;
  uint32_t* keys;            // [batch][kv_heads][pages rounded up to 4]
};
hipError_t launch_index_update(const IndexParams& p, int dtype, int storage, int64_t batch, hipStream_t s);
hipError_t launch_index_score(const IndexParams& p, int dtype, int64_t batch, hipStream_t s);

// Which of a sequence and head's items (pages or tokens) are kept.
struct ChooseParams {
  const uint32_t* keys;      // pages: [batch][heads][stride]; or
  const float* mass;         // tokens: their masses
  int64_t mass_batch, mass_head;
  const int32_t* table;
  const int32_t* lens;
  int64_t table_row;
  FastDiv page_size;
  int32_t num_pages, pages;  // of the cache; of a sequence's table
  int32_t items;             // of the keys or masses
  int32_t heads, key_stride;
  int32_t budget, sink, recent;
  int32_t* out;              // [batch][heads][budget]
  float* out_mass;           // or nullptr
  int32_t* out_lens;
};
// Tables that one workgroup scores and chooses from in one launch
constexpr int kFew = 256;
hipError_t launch_select(const IndexParams& p, const ChooseParams& c, int dtype, int64_t batch, hipStream_t s);
hipError_t launch_choose_pages(const ChooseParams& p, int64_t batch, hipStream_t s);
hipError_t launch_choose_tokens(const ChooseParams& p, int64_t batch, hipStream_t s);

struct MoveParams {
  CacheView from, to;
  const int32_t *from_table, *to_table;
  int64_t from_row, to_row;
  int32_t from_len, to_len;    // pages of the tables
  int32_t from_pages, to_pages;  // of the caches
  const int32_t* kept;
  const int32_t* lens;
  int32_t budget;
  FastDiv chunks;              // of 16 bytes of a row
  int32_t scale_bytes;
  int64_t bh0;                 // first sequence and head of a launch
};
hipError_t launch_move(MoveParams p, int64_t batch, hipStream_t s);

struct MassParams {
  AttnParams a;
  const float* mass;
  float* out;
  const float* lse;
  int64_t mass_batch, mass_head, out_batch, out_head;
  int32_t tokens;
  int32_t splits;              // workgroups of one sequence and head
  float decay;
};
hipError_t launch_mass(const MassParams& p, int dtype, int storage, hipStream_t s);

}  // namespace agmm
