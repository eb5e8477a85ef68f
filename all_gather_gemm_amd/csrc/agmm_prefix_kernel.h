// gfx950 kernel of the attention over prefixes that sequences share (agmm_long.h).
//
// Mathematics: for one prefix and kv head the q heads of all its sequences are the rows of one matrix Q
// (rows x dim), and the prefix is read once for all of them: S^T = K Q^T (tokens x rows), a softmax over
// the tokens with a running maximum and sum in 32 bits, O^T = V^T P^T. That is 4 rows x tokens x dim
// operations for 4 tokens x dim bytes (16-bit cache), so from a few hundred rows on the matrix units bound
// it, and the vector units, which make rows x tokens weights meanwhile.
//
//  - A workgroup has 128 rows, 32 a wave, and goes through tiles of tokens (8192 elements of K, as many of
//    V), which all of its waves read from LDS. A wave whose rows do not exist leaves the products out.
//  - Matrix instructions of 32 tokens x 32 rows: S^T's accumulators (lane = row, 4 consecutive tokens) are
//    P^T's operands for O^T, in the order of tokens {16 s + 4 h ..+3, 16 s + 8 + 4 h ..+3} for lane half h, so
//    P never moves between lanes. V^T's operands in that order are two transposing reads of LDS each.
//  - Weights enter the product in two parts of the 16-bit type, as in the attention of single tokens, so that
//    a shared prefix gives what its tokens give unshared. One rounded part alone: 390 us against 472 (256 sequences
//    behind 32768 tokens, one run), and where values average out 1.4 times as far off, bf16's own rounding counted in.
//  - 16-bit rows of whole padded width go from memory to LDS directly; others, and codes, through registers, where
//    they become values of the 16-bit type, so all storages share the rest.
//  - The next tile is under way to the other half of LDS while one is worked on: one barrier a tile.
//  - Operands are read from LDS some instructions ahead, and the weights of 16 tokens are made between the products
//    of the 16 before: the order of instructions is given, as the compiler's waits for each read (518 us, 402).
//
// Work: a strip is 128 rows of one kv head and prefix; strips' tiles, strip after strip, are cut into equal runs,
// one for each workgroup that works on prefixes, from the lengths on the device. Every piece of a strip leaves its
// sums, references and sums of weights in the scratch. The other workgroups of the launch attend to the sequences'
// own tokens (agmm_attn_kernel.h) and leave theirs. A second kernel joins them all, in the order of the pieces, so
// results do not depend on timing.
//
// Measured, with the joining: 256 sequences behind 32768 tokens, 64/8 heads of 128, bf16: 429 to 468 us, from card to
// card; the prefix by itself 393: 0.70 PFLOP/s counted once, 1.05 with both parts of the weights (the card's large
// products run at 1.2, at its power limit; the clock is 1.9 GHz here). The matrix units are busy half of the cycles,
// the vector units 60%, and 2192 MB are read, for 289 MB of prefix and own tokens, at 5 TB/s: every 128 rows read the
// prefix again.
// 64 sequences behind 8192 tokens: 51 us, of which products and weights take 28, launch, lengths and pages 10, the
// writing of the pieces' 33 MB 8, the joining 8; a call of 4 behind 2000 tokens 14 + the host.
// Kernels that spill registers, all of width 64 and 128: those with a cap 34 to 98 (64 sequences behind 8192 tokens, in a
// graph: 64 us, 55.5 without), 16-bit rows through registers at width 128 10 and 11, e4m3's 6 and 7, e2m1's 1 or none.
#pragma once

#include "agmm_attn_kernel.h"
#include "agmm_long_internal.h"

namespace agmm {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int DT>
__device__ inline f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (DT == AGMM_F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8_t, a), __builtin_bit_cast(h8_t, b), c,
                                                  0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8_t, a), __builtin_bit_cast(b8_t, b),
                                                   c, 0, 0, 0);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <int DP>
struct Tile {
  static constexpr int kTokens = 8192 / DP;       // 128, 64 or 32
  static constexpr int kRow = 2 * DP;             // bytes of a row
  static constexpr int kChunks = DP / 8;          // of 16 bytes a row
  static constexpr int kSub = kTokens / 32;       // blocks of 32 tokens
  static constexpr int kMasks = (kTokens + 63) / 64;
  static constexpr int kLines = 64 / kChunks;     // rows that a wave fills at once
  static constexpr int kBytes = 16384;            // of K's tile, and of V's

  // Chunk c of row t is in place c ^ key(t), or c ^ value(t). Keys are read by 16 lanes at once, one chunk of
  // 16 rows; values by 32 lanes, two neighbouring chunks of 4 rows twice. Rows are 32, 64 and 128 words: the
  // places are such that the lanes that read together find different banks.
  __device__ static inline int key(int t) { return DP == 64 ? (t >> 1) & 7 : t & 15; }
  __device__ static inline int value(int t) { return DP == 64 ? 4 * ((t >> 1) & 1) : 4 * (t & 3); }
};

template <int DP>
struct alignas(16) TileShared {
  char k[2][Tile<DP>::kBytes], v[2][Tile<DP>::kBytes];
  int64_t at[4][Tile<DP>::kTokens][2];  // the tokens' places: data and scale offsets, for each wave
};

// 16 bytes a lane from `from` into LDS at byte m0 + 16 * lane (m0 is wave-uniform). Written as inline asm so that
// the compiler adds no waits for it: it cannot tell which half of LDS is written, and would wait before every
// read of the other. (The load needs one wait state behind the write of m0, which the compiler does not keep in front
// of inline asm.)
__device__ inline void dma16(const char* from, uint32_t m0) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "{m0}"(m0) : "memory");
}
__device__ inline void dma_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A thread's chunks of a tile as they come from memory, where they do not go to LDS directly.
template <int ST>
struct Staged {
  static constexpr int kWords = ST == AG_KV_16BIT ? 4 : ST == AG_KV_MXFP8 ? 2 : 1;
  uint32_t k[4][kWords], v[4][kWords];
  uint32_t ks[4], vs[4];
};

struct PrefixScan {  // of one lane's group
  int32_t first, end;
  uint32_t tiles, row_tiles, strips, strip0, tile0;
  int32_t len;
};

// What one wave of the workgroup knows about groups base .. base + 63, given what came before.
struct PrefixCarry {
  int32_t last;            // the sequences up to here are in some group
  uint32_t strips, tiles;
};

__device__ inline uint32_t last_lane(uint32_t x) { return (uint32_t)__builtin_amdgcn_readlane((int)x, 63); }

template <int DP>
__device__ inline PrefixScan scan_groups(const PrefixParams& p, uint32_t base, PrefixCarry& c) {
  const int lane = threadIdx.x & 63;
  const uint32_t g = base + lane;
  const AttnParams& a = p.own;
  PrefixScan r = {};
  // A group ends where the next begins, and none begins before another's end: whatever `starts` holds,
  // sequences are in one group at most.
  int32_t end = 0;
  if (g < a.prefix.groups) {
    end = p.starts ? max(0, min(p.starts[g + 1], a.batch)) : a.batch;
    r.len = max(0, min(p.lens[g], p.capacity));
  }
  int32_t run = end;  // the largest end up to this lane
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int32_t o = __shfl_up(run, d);
    if (lane >= d) run = max(run, o);
  }
  int32_t before = __shfl_up(run, 1);
  before = lane == 0 ? 0 : before;
  const int32_t floor0 = base == 0 && p.starts ? max(0, min(p.starts[0], a.batch)) : 0;
  const int32_t lowest = max(c.last, floor0);
  r.first = max(before, lowest);
  r.end = max(run, lowest);
  if (g < a.prefix.groups && r.len > 0 && r.end > r.first) {
    r.tiles = (uint32_t)((r.len + Tile<DP>::kTokens - 1) / Tile<DP>::kTokens);
    r.row_tiles = ((uint32_t)(r.end - r.first) * a.group + kPrefixRows - 1) / kPrefixRows;
    r.strips = r.row_tiles * a.c.kv_heads;
  }
  const uint32_t s = wave_scan(r.strips), t = wave_scan(r.strips * r.tiles);
  r.strip0 = c.strips + s - r.strips;
  r.tile0 = c.tiles + t - r.strips * r.tiles;
  c.last = max(c.last, (int32_t)last_lane((uint32_t)r.end));
  c.strips += last_lane(s);
  c.tiles += last_lane(t);
  return r;
}

// The next `n` instructions of this kind, in the order of these calls.
constexpr int kAlu = 0x402, kMatrix = 0x8, kReads = 0x100;
#define ORDER(kind, n) __builtin_amdgcn_sched_group_barrier(kind, n, 0)

// DMA: 16-bit rows of all of DP elements, which go from memory to LDS directly.
template <int DT, int ST, int DP, bool CAP, bool DMA>
struct PrefixWave {
  typedef Tile<DP> T;
  typedef Staged<ST> S;
  static constexpr int kSteps = DP / 16;   // matrix instructions over the head for 32 tokens
  static constexpr int kParts = DP / 32;   // accumulators
  static constexpr int kKeys = kSteps < 8 ? kSteps : 8, kValues = kParts < 4 ? kParts : 4;

  u32x4 q[kSteps];
  f32x16 acc[kParts];
  float m, l;  // of this lane's row: weights are 2^(score - m), base 2; their sum over this lane's tokens
  uint32_t k_at[kKeys], v_at[kValues];  // LDS bytes of this lane's operands

  __device__ inline void start(const AttnParams& p, int32_t first, int kv, int row, int rows) {
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int i = row < rows ? row : 0;
    const int b = first + i / p.group, head = kv * p.group + i % p.group;
    const uint16_t* from = p.q + b * p.q_batch + head * p.q_head;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int e = 16 * s + 8 * h;
      q[s] = u32x4{0, 0, 0, 0};
      if (row < rows && e < p.c.head_dim) q[s] = load16(from + e);
    }
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
      for (int w = 0; w < 16; ++w) acc[i][w] = 0.0f;
    m = -INFINITY;
    l = 0.0f;
    const int t = lane & 31, i16 = lane & 15, half = (lane >> 4) & 1;
#pragma unroll
    for (int s = 0; s < kKeys; ++s) k_at[s] = (uint32_t)(t * T::kRow + 16 * ((2 * s + h) ^ T::key(t)));
    // transposing reads: 16 lanes get 16 elements of 4 tokens from addresses of 4 elements of one
#pragma unroll
    for (int i = 0; i < kValues; ++i)
      v_at[i] = (uint32_t)((4 * h + i16 / 4) * T::kRow +
                           16 * ((4 * i + 2 * half + i16 % 4 / 2) ^ T::value(i16 / 4)) + 8 * (i16 % 2));
  }

  // Rows line(i) of a tile are this lane's to fetch, chunk lane % kChunks.
  __device__ static inline int line(int i) {
    return (((int)threadIdx.x >> 6) * 4 + i) * T::kLines + (int)(threadIdx.x & 63) / T::kChunks;
  }
  __device__ static inline int bytes_of(int e) { return ST == AG_KV_16BIT ? 2 * e : ST == AG_KV_MXFP8 ? e : e / 2; }

  // The loads of the tile whose tokens' places are in `at`; tokens that are absent have the place of the
  // pools' first row, and chunks past the head's end read its first. k and v: LDS bytes of the tile's halves.
  __device__ static inline void load(S& r, const AttnParams& p, const int64_t (*at)[2], int64_t head,
                                     int64_t s_head, uint32_t k, uint32_t v) {
    const int c = (int)(threadIdx.x & 63) % T::kChunks, hd = p.c.head_dim;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = line(i);
      const int64_t data = head + at[t][0];
      if constexpr (DMA) {
        const uint32_t to = (uint32_t)(1024 * (4 * wave + i));
        dma16(p.c.k + data + 16 * (c ^ T::key(t)), k + to);
        dma16(p.c.v + data + 16 * (c ^ T::value(t)), v + to);
      } else {
        const int e = 8 * c < hd ? 8 * c : 0;
        load_words<S::kWords>(r.k[i], p.c.k + data + bytes_of(e));
        load_words<S::kWords>(r.v[i], p.c.v + data + bytes_of(e));
        if (ST != AG_KV_16BIT) {
          const int64_t scale = s_head + at[t][1] + e / 32;
          r.ks[i] = *(const uint8_t*)(p.c.ks + scale);
          r.vs[i] = *(const uint8_t*)(p.c.vs + scale);
        }
      }
    }
  }

  __device__ static inline u32x4 chunk(const uint32_t (&w)[S::kWords], uint32_t scale) {
    if constexpr (ST == AG_KV_16BIT)
      return u32x4{w[0], w[1], w[2], w[3]};
    else if constexpr (ST == AG_KV_MXFP8)
      return from_fp8x8<DT>(w[0], w[1], scale_of(scale));
    else
      return from_fp4x8<DT>(w[0], scale_of(scale));
  }

  // The loaded tile in LDS; the values of absent tokens, and all elements past the head's end, are zeros.
  __device__ static inline void store(const S& r, const AttnParams& p, const uint64_t (&there)[T::kMasks],
                                      bool all, lds_char* k, lds_char* v) {
    const int c = (int)(threadIdx.x & 63) % T::kChunks;
    const u32x4 zero = {0, 0, 0, 0};
    if constexpr (DMA) {
      dma_done();
      if (all) return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = line(i);
      const uint64_t mask = T::kMasks == 2 && t >= 64 ? there[T::kMasks - 1] : there[0];
      const bool ok = mask >> (t & 63) & 1;
      if constexpr (DMA) {
        if (!ok) *(lds_u32x4*)(v + t * T::kRow + 16 * c) = zero;
      } else {
        const bool in = 8 * c < p.c.head_dim;
        const u32x4 x = chunk(r.k[i], r.ks[i]), y = chunk(r.v[i], r.vs[i]);
        *(lds_u32x4*)(k + t * T::kRow + 16 * (c ^ T::key(t))) = in ? x : zero;
        *(lds_u32x4*)(v + t * T::kRow + 16 * (c ^ T::value(t))) = in && ok ? y : zero;
      }
    }
  }

  // k, v: the tile.
  __device__ __attribute__((always_inline)) inline void work(const AttnParams& p, const uint64_t (&there)[T::kMasks], bool all, int up,
                              const lds_char* k, const lds_char* v) {
    const int h = (int)(threadIdx.x & 63) >> 5;
    f32x16 st[T::kSub];
#pragma unroll
    for (int u = 0; u < T::kSub; ++u)
#pragma unroll
      for (int w = 0; w < 16; ++w) st[u][w] = 0.0f;
    // Operands kAhead instructions ahead, so that the matrix unit does not wait for LDS.
    constexpr int kAll = kSteps * T::kSub, kAhead = 6;
    u32x4 key[kAll];
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int u = 0; u < T::kSub; ++u)
        key[s * T::kSub + u] =
            *(const lds_u32x4*)(k + k_at[s % kKeys] + 16 * 16 * (s / kKeys) + 32 * u * T::kRow);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int u = 0; u < T::kSub; ++u) st[u] = mfma32<DT>(key[s * T::kSub + u], q[s], st[u]);
    ORDER(kReads, kAhead);
#pragma unroll
    for (int i = 0; i < kAll - kAhead; ++i) {
      ORDER(kMatrix, 1);
      ORDER(kReads, 1);
    }
    ORDER(kMatrix, kAhead);
    float scale = p.scale;
    if constexpr (CAP) {
      scale = 1.0f;
      float most = 0.0f;
#pragma unroll
      for (int u = 0; u < T::kSub; ++u)
#pragma unroll
        for (int w = 0; w < 16; ++w) most = fmaxf(most, fabsf(st[u][w]));
      if (__any(most * p.inv_cap >= kFar)) {
#pragma unroll
        for (int u = 0; u < T::kSub; ++u)
#pragma unroll
          for (int w = 0; w < 16; ++w) st[u][w] = capped<false>(p, st[u][w]);
      } else {
#pragma unroll
        for (int u = 0; u < T::kSub; ++u)
#pragma unroll
          for (int w = 0; w < 16; ++w) st[u][w] = capped<true>(p, st[u][w]);
      }
    }
    if (!all) {
#pragma unroll
      for (int u = 0; u < T::kSub; ++u) {
        const uint32_t mine = (uint32_t)(there[u / 2] >> (32 * (u & 1))) >> (4 * here(h));
#pragma unroll
        for (int w = 0; w < 16; ++w)
          st[u][w] = __builtin_bit_cast(
              float, here(__builtin_bit_cast(int, mine >> (8 * (w / 4) + w % 4) & 1u ? st[u][w] : -INFINITY)));
      }
    }
    float top = st[0][0];
#pragma unroll
    for (int u = 0; u < T::kSub; ++u)
#pragma unroll
      for (int w = 0; w < 16; ++w) top = fmaxf(top, st[u][w]);
    {
      const auto x = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, top),
                                                      __builtin_bit_cast(uint32_t, top), false, false);
      top = fmaxf(__builtin_bit_cast(float, (uint32_t)x[0]), __builtin_bit_cast(float, (uint32_t)x[1]));
    }
    // Weights are 2^(score - m) with a whole number m, `up` below the largest score so far (or less: it is raised
    // only when that is left behind by 2^kRaise). One multiply-add then gives an exponent that is off by its own
    // rounding alone, however large the scores are, and what is summed is rescaled by powers of 2. Past 2^23 not
    // every whole number is a 32-bit float: there m is the score itself. (One past the range of floats gives NaN.)
    top *= scale;
    const float head = (float)up;
    if (__any(top - m > (float)kRaise + head)) {
      const float whole = fminf(ceilf(top), 0x1.fffffep127f);
      const float raised = fmaxf(m, fabsf(whole) < 0x1p23f ? whole - head : whole);
      const float f = weight(m, raised, 1.0f);
#pragma unroll
      for (int i = 0; i < kParts; ++i)
#pragma unroll
        for (int w = 0; w < 16; ++w) acc[i][w] *= f;
      l *= f;
      m = raised;
    }
    const float less = m == -INFINITY ? 0.0f : -m;
    // 16 tokens at a time; the weights of the next ones are made between the products of these.
    // (A wave that is here goes first on its SIMD: the other one's scores have no vector work between them. 256
    // sequences behind 32768 tokens: 393 us of prefixes, 403 without.)
    __builtin_amdgcn_s_setprio(1);
    constexpr int kTimes = 2 * T::kSub, kVector = 56 / (2 * kParts);
    u32x4 hi[2], lo[2], value[2][kParts];
    auto weigh = [&](int g) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[i] = __builtin_amdgcn_exp2f(fmaf(st[g / 2][8 * (g % 2) + 2 * j + i], scale, less));
          l += w[i];
        }
        const u32x2 x = T16<DT>::split(w[0], w[1]);
        hi[g % 2][j] = x[0];
        lo[g % 2][j] = x[1];
      }
    };
    auto read = [&](int g) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const lds_char* at = v + v_at[i % kValues] + 16 * 16 * (i / kValues) + 16 * g * T::kRow;
        const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at));
        const u32x2 y =
            __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 8 * T::kRow)));
        value[g % 2][i] = u32x4{x[0], x[1], y[0], y[1]};
      }
    };
    read(0);
    weigh(0);
    ORDER(kReads, 2 * kParts);
    ORDER(kAlu, 56);
#pragma unroll
    for (int g = 0; g < kTimes; ++g) {
      if (g + 1 < kTimes) {
        read(g + 1);
        weigh(g + 1);
      }
#pragma unroll
      for (int i = 0; i < kParts; ++i) acc[i] = mfma32<DT>(value[g % 2][i], hi[g % 2], acc[i]);
#pragma unroll
      for (int i = 0; i < kParts; ++i) acc[i] = mfma32<DT>(value[g % 2][i], lo[g % 2], acc[i]);
#pragma unroll
      for (int i = 0; i < 2 * kParts; ++i) {
        ORDER(kMatrix, 1);
        if (g + 1 < kTimes) {
          ORDER(kReads, 1);
          ORDER(kAlu, kVector);
        }
      }
    }
    __builtin_amdgcn_s_setprio(0);
  }

  // The piece's sums, maxima and sums of weights.
  __device__ inline void leave(const PrefixParams& p, uint32_t slot, int row) const {
    const int h = (threadIdx.x & 63) >> 5;
    float* to = p.own.prefix.sums + (int64_t)slot * kPrefixRows * DP;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w)
        *reinterpret_cast<f32x4*>(to + prefix_at(row, 32 * i + 8 * w + 4 * h)) =
            f32x4{acc[i][4 * w], acc[i][4 * w + 1], acc[i][4 * w + 2], acc[i][4 * w + 3]};
    const auto x = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, l),
                                                    __builtin_bit_cast(uint32_t, l), false, false);
    const float sum = __builtin_bit_cast(float, (uint32_t)x[0]) + __builtin_bit_cast(float, (uint32_t)x[1]);
    if (h == 0) {
      float* s = p.own.prefix.stats + ((int64_t)slot * kPrefixRows + row) * 2;
      s[0] = m;
      s[1] = sum;
    }
  }
};

// The share of workgroup `me` of those that work on prefixes, of which each has a run of `quota` of all tiles.
template <int DT, int ST, int DP, bool CAP, bool DMA>
__device__ inline void prefix_share(const PrefixParams& p, TileShared<DP>& sh, const PrefixScan* scan0,
                                    const PrefixCarry& carry0, uint32_t me, uint32_t total, uint32_t quota) {
  typedef Tile<DP> T;
  typedef PrefixWave<DT, ST, DP, CAP, DMA> W;
  const AttnParams& a = p.own;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  uint32_t cur = me * quota;
  if (cur >= total) return;
  const uint32_t end = min(cur + quota, total);

  while (cur < end) {
    // the group and strip of tile `cur`
    PrefixScan r = {};
    uint32_t group = 0;
    PrefixCarry c = carry0;
    for (uint32_t g = 0; g < a.prefix.groups; g += 64) {
      const PrefixScan s = g == 0 ? scan0[lane] : scan_groups<DP>(p, g, c);
      const uint64_t hit = __ballot(s.strips * s.tiles != 0 && cur >= s.tile0 &&
                                    cur < s.tile0 + s.strips * s.tiles);
      if (hit) {
        const int at = __builtin_ctzll(hit);
        group = g + at;
        r.first = __shfl(s.first, at);
        r.end = __shfl(s.end, at);
        r.tiles = __shfl(s.tiles, at);
        r.row_tiles = __shfl(s.row_tiles, at);
        r.strip0 = __shfl(s.strip0, at);
        r.tile0 = __shfl(s.tile0, at);
        r.strips = __shfl(s.strips, at);
        r.len = __shfl(s.len, at);
        break;
      }
    }
    group = __builtin_amdgcn_readfirstlane(group);
    const uint32_t tiles = __builtin_amdgcn_readfirstlane(r.tiles);
    const uint32_t tile0 = __builtin_amdgcn_readfirstlane(r.tile0);
    const uint32_t strip0 = __builtin_amdgcn_readfirstlane(r.strip0);
    const uint32_t strips = __builtin_amdgcn_readfirstlane(r.strips);
    const uint32_t row_tiles = __builtin_amdgcn_readfirstlane(r.row_tiles);
    const int32_t first = __builtin_amdgcn_readfirstlane(r.first);
    const int32_t rows = (__builtin_amdgcn_readfirstlane(r.end) - first) * a.group;
    const int32_t len = __builtin_amdgcn_readfirstlane(r.len);
    const int32_t* table = p.table + (int64_t)group * p.table_row;
    const int up = head_of<DT>(len);
    for (uint32_t strip = (cur - tile0) / tiles; strip < strips && cur < end; ++strip) {
      const uint32_t begin = tile0 + strip * tiles, stop = min(end, begin + tiles);
      const int kv = (int)(strip / row_tiles);
      const int row0 = (int)(strip - kv * row_tiles) * kPrefixRows;
      const int row = 32 * wave + (lane & 31);
      const bool some = row0 + 32 * wave < rows;
      const int64_t head = kv * a.c.head, s_head = kv * a.c.s_head;
      W w;
      w.start(a, first, kv, row0 + row, rows);
      int64_t(*at)[2] = sh.at[wave];
      auto page_of = [&](int64_t t) { return table[(uint32_t)min(t, (int64_t)len - 1) / a.c.page_size]; };
      // Puts the places of a tile's tokens into LDS; bit t: token base + t is attended to.
      auto place = [&](int64_t base, const int32_t (&page)[T::kMasks], uint64_t (&there)[T::kMasks]) {
#pragma unroll
        for (int i = 0; i < T::kMasks; ++i) {
          const int64_t tok = base + 64 * i + lane;
          const bool ok = (uint32_t)page[i] < (uint32_t)a.num_pages && tok < len &&
                          (T::kTokens >= 64 || lane < T::kTokens);
          there[i] = __ballot(ok);
          const uint32_t t = (uint32_t)tok;
          const uint32_t r = t - (t / a.c.page_size) * a.c.page_size.d;
          if (T::kTokens >= 64 || lane < T::kTokens) {
            at[64 * i + lane][0] = ok ? row_at(a.c, page[i], r) : 0;
            if (ST != AG_KV_16BIT) at[64 * i + lane][1] = ok ? scales_at(a.c, page[i], r) : 0;
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      };
      auto pages = [&](int64_t base, int32_t (&page)[T::kMasks]) {
#pragma unroll
        for (int i = 0; i < T::kMasks; ++i) page[i] = page_of(base + 64 * i + lane);
      };
      constexpr uint64_t kAll = T::kTokens >= 64 ? ~0ull : (1ull << (T::kTokens & 63)) - 1;
      int64_t base = (int64_t)(cur - begin) * T::kTokens;
      const int64_t behind = (int64_t)(stop - begin) * T::kTokens;
      int32_t page[T::kMasks];
      uint64_t there[T::kMasks], next[T::kMasks];
      typename W::S staged;
      auto whole = [&](const uint64_t (&x)[T::kMasks]) {
        bool all = x[0] == kAll;
        if (T::kMasks == 2) all = all && x[T::kMasks - 1] == kAll;
        return all;
      };
      lds_char* const k = (lds_char*)&sh.k[0][0];
      lds_char* const v = (lds_char*)&sh.v[0][0];
      auto fetch = [&](int buf) {
        W::load(staged, a, at, head, s_head, (uint32_t)(size_t)k + buf * T::kBytes,
                (uint32_t)(size_t)v + buf * T::kBytes);
      };
      pages(base, page);
      place(base, page, there);
      pages(base + T::kTokens, page);
      fetch(0);
      W::store(staged, a, there, whole(there), k, v);
      __syncthreads();
      // The next tile is under way to one half of LDS while the other is worked on.
      auto step = [&](auto buf) __attribute__((always_inline)) {
        constexpr int now = decltype(buf)::value, after = 1 - now;
        base += T::kTokens;
        const bool more_tiles = base < behind;
        if (more_tiles) {
          place(base, page, next);
          pages(base + T::kTokens, page);
          fetch(after);
        }
        if (some) w.work(a, there, whole(there), up, k + now * T::kBytes, v + now * T::kBytes);
        if (more_tiles) {
          W::store(staged, a, next, whole(next), k + after * T::kBytes, v + after * T::kBytes);
#pragma unroll
          for (int i = 0; i < T::kMasks; ++i) there[i] = next[i];
        }
        __syncthreads();
        return more_tiles;
      };
      while (step(std::integral_constant<int, 0>{}) && step(std::integral_constant<int, 1>{})) {
      }
      if (some) w.leave(p, me + strip0 + strip, row);
      cur = stop;
    }
  }
}

// The length of the runs that prefixes' `total` tiles are cut into, so that the workgroups that are left for the
// `own` tiles take as long. Each lane works out one length, with a prefix's tile at kTile of an own one, whatever the
// width, the storage and the rows that the strip has. Runs have at least `least` tiles, as long as every compute unit
// gets one.
// kTile 0.65, 0.8, 0.9, 1.0, in graphs: 256 sequences behind 32768 tokens 435, 431, 432, 432 us; 64 of 2048 behind 8192
// tokens, 64/8 heads, e4m3 61.6, 61.2, 60.5, 60.5, e2m1 61.0, 60.4, 60.2, 60.0; 32/8 heads of 256, 16 bits 105, 104, 111, 111.
__device__ inline uint32_t run_length(uint32_t total, uint32_t own, uint32_t wgs, uint32_t least) {
  constexpr float kTile = 0.8f;
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t shortest = max(max(1u, min(least, (total + kCus - 1) / kCus)), (total + wgs - 1) / wgs);
  // (the last lane's is all of it in one run: that always leaves a workgroup)
  const uint32_t quota = lane < 63 ? shortest + lane * max(1u, shortest / 64) : max(shortest, total);
  const uint32_t x = (total + quota - 1) / quota;
  float t = (float)quota * kTile;
  if (own) t = x < wgs ? fmaxf(t, (float)((own + wgs - x - 1) / max(wgs - x, 1u))) : INFINITY;
  float best = t;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) best = fminf(best, __shfl_xor(best, d));
  const int at = __builtin_ctzll(__ballot(t == best));
  return (uint32_t)__builtin_amdgcn_readlane((int)quota, at);
}

// Prefixes and own tokens in one launch, so that the products of the ones run beside the loads of the others: of the
// workgroups, which are all on the chip at once, each part has as many as its share of the work, in every XCD alike.
template <int DT, int ST, int DP, bool CAP, bool DMA>
__global__ __launch_bounds__(kThreads, prefix_per_cu(DP)) void prefix_kernel(PrefixParams p) {
  __shared__ union {
    TileShared<DP> tiles;
    AttnShared<DP> own;
  } sh;
  __shared__ PrefixScan scan0[64];
  const AttnParams& a = p.own;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // (what the first 64 groups' scan gives is kept: most calls have no more)
  PrefixCarry carry0 = {0, 0, 0};
  scan0[lane] = scan_groups<DP>(p, 0, carry0);   // (every wave writes the same)
  __syncthreads();
  PrefixCarry c = carry0;
  for (uint32_t g = 64; g < a.prefix.groups; g += 64) scan_groups<DP>(p, g, c);
  const uint32_t total = c.tiles;
  const Census own = census(a);
  const uint32_t own_tiles = own.tiles * (uint32_t)(a.c.kv_heads * a.q_groups);
  const uint32_t wgs = gridDim.x;
  const uint32_t quota = run_length(total, own_tiles, wgs, p.least);
  const uint32_t x = (total + quota - 1) / quota;   // workgroups that have a run
  if (blockIdx.x == 0 && wave == 0) {
    c = carry0;
    for (uint32_t g = 0; g < a.prefix.groups; g += 64) {
      const PrefixScan r = g == 0 ? scan0[lane] : scan_groups<DP>(p, g, c);
      if (g + lane < a.prefix.groups)
        a.prefix.info[g + lane] =
            PrefixGroup{r.first, r.end, r.tiles, r.row_tiles, r.strip0, r.tile0, quota, 0};
    }
  }
  // Consecutive numbers to the workgroups of an XCD, which are 8 apart, so that neighbouring runs share an L2 (strips of
  // one kv head whose runs are a strip or so long read the same tiles; of a long prefix they are at other tokens);
  // the first of each XCD's are the prefixes'.
  const uint32_t xcd = blockIdx.x % 8, local = blockIdx.x / 8;
  const uint32_t from = xcd * (wgs / 8) + min(xcd, wgs % 8), size = wgs / 8 + (xcd < wgs % 8 ? 1 : 0);
  const uint32_t first = (uint32_t)((uint64_t)x * from / wgs);
  const uint32_t mine = (uint32_t)((uint64_t)x * (from + size) / wgs) - first;
  if (local < mine) {
    prefix_share<DT, ST, DP, CAP, DMA>(p, sh.tiles, scan0, carry0, first + local, total, quota);
  } else {
    const uint32_t other = from - first + local - mine, others = min(wgs - x, p.own_wgs);
    if (other < others) share_of<DT, ST, DP, CAP, kPieces>(a, sh.own, own, other, others);
  }
}

template <int DT, int ST, int DP, bool DMA>
void prefix_by_cap(const PrefixParams& p, int grid, hipStream_t s) {
  if (p.own.cap != 0.0f)
    prefix_kernel<DT, ST, DP, true, DMA><<<grid, kThreads, 0, s>>>(p);
  else
    prefix_kernel<DT, ST, DP, false, DMA><<<grid, kThreads, 0, s>>>(p);
}

template <int DT, int ST, int DP>
void prefix_by_rows(const PrefixParams& p, int grid, hipStream_t s) {
  if constexpr (ST == AG_KV_16BIT) {
    if (p.own.c.head_dim == DP) {
      prefix_by_cap<DT, ST, DP, true>(p, grid, s);
      return;
    }
  }
  prefix_by_cap<DT, ST, DP, false>(p, grid, s);
}

template <int DT, int ST>
void prefix_by_width(const PrefixParams& p, int grid, hipStream_t s) {
  const int dp = attn_padded(p.own.c.head_dim);
  if (dp == 64)
    prefix_by_rows<DT, ST, 64>(p, grid, s);
  else if (dp == 128)
    prefix_by_rows<DT, ST, 128>(p, grid, s);
  else
    prefix_by_rows<DT, ST, 256>(p, grid, s);
}

template <int DT>
hipError_t prefix_by_storage(const PrefixParams& p, int storage, int grid, hipStream_t s) {
  if (storage == AG_KV_16BIT)
    prefix_by_width<DT, AG_KV_16BIT>(p, grid, s);
  else if (storage == AG_KV_MXFP8)
    prefix_by_width<DT, AG_KV_MXFP8>(p, grid, s);
  else
    prefix_by_width<DT, AG_KV_MXFP4>(p, grid, s);
  return hipGetLastError();
}

}  // namespace
}  // namespace agmm
