// gfx950 kernel of the attention of one new token over a paged key-value cache (agmm_attn.h).
//
// Mathematics, for one sequence and one kv head with its G q heads: S = K Q^T (tokens x G), a
// softmax over the tokens with a running maximum m and sum l in 32 bits, O^T = V^T P^T. Each cached
// byte is used for G <= 16 q heads, 4 G flop per 16-bit value, so the bound is the memory
// bandwidth and the kernel is built around keeping loads in flight:
//
//  - Matrix instructions of 16 tokens x 16 q heads read K straight from global memory: a lane's
//    operand is 8 values of one token's row, which is 16 contiguous bytes. The order of the inner
//    dimension is free as long as Q has the same, so 8-bit and 4-bit rows are read 16 bytes a lane
//    too. Nothing passes through LDS on the way.
//  - S^T's accumulator layout (lane = q head, 4 consecutive tokens) is, for a pair of 16-token
//    tiles, the operand layout of P^T for 32 tokens in the order {4 g .. 4 g + 3, 16 + 4 g ..}, so
//    P never moves between lanes.
//  - V^T needs 8 tokens of one element in a lane. A lane loads 8 elements of each of its 8 tokens (4
//    where rows have 64), 16 lanes covering whole rows, and transposes in registers with v_perm_b32;
//    matrix instruction e takes element e of every lane's chunk, so a lane's accumulators end up
//    holding 32 consecutive elements of the output.
//  - Codes are turned into the 16-bit type, scale included, by one v_cvt_scalef32_pk per pair.
//  - Weights enter the product in two parts of the 16-bit type, 22 bits (fp16) or 16 (bf16) in all.
//  - The maximum is raised only when a tile's exceeds it by 2^4 or more, so the accumulators are
//    rescaled a few times a sequence. Weights are 2^(s - m + head). fp16: head 11, so up to 2^15, where
//    both parts have their full precision and room below. bf16, whose values reach to the end of 32 bits:
//    low enough that all of a sequence's weights add up to 1 at most, and with them no sum exceeds the
//    largest value, which 32 bits hold.
//  - Past 16 q heads to a kv head, groups of 16 take the cache one after the other.
//
// Work: the tiles (128 tokens) of all sequences and heads, in that order, are cut into equal runs, one
// for each worker, from the lengths on the device. A worker is a workgroup's 4 waves, or each wave by
// itself where many heads are short. A run may begin and end inside a sequence's head; such a head's
// pieces are joined by the last worker to finish one, in the order of the pieces (over 32 of them: 16
// at a time, and then the groups of 16), so results do not depend on timing.
//
// Measured, warm, the same call again and again: 64 sequences of 8192 tokens, 64/8 heads of 128, bf16:
// 355 us, 6.05 TB/s of cache read once (a copy of 4 GiB runs at 4.7 TB/s, reads and writes together); 32
// such sequences in e4m3 107 us, 5.2 TB/s, in e2m1 58 us, 4.9 TB/s, where turning codes into values bounds
// it: over half of the vector unit's issue slots, and its waits. In a trace one token takes 5.8 us
// (launch, length, page, keys and values, output: four reads that each wait for the one before), 300 8.5;
// 2048 tokens of e4m3, which workgroups share and join, 11.4. Times beside the constants and rules below
// are of the step that chose them, both sides in one run; since then they have moved by up to 3%.
#pragma once

#include "agmm_attn_device.h"

namespace agmm {
namespace {

constexpr int kCus = 256;
// What a kernel's tokens and results are: kPlain, those of ag_attn_run; kHeads, with a page table for each kv
// head; kPieces, the tokens behind a shared prefix, whose results are left for the joining with it.
constexpr int kPlain = 0, kHeads = 1, kPieces = 2;
// Tiles of a workgroup's share, at least, as long as every compute unit gets one, where sequences have more
// than kLong tiles on the average: fewer pieces to join (131072 tokens, one kv head, e4m3: 17.7 us, 20.8
// with 2). Of shorter ones a share would hold ends of two heads more often than it saves pieces (32
// ragged up to 4000, 8 kv heads, e4m3: 21.5 us, 24.6 with 4; 16 up to 2000, 8 kv heads, bf16 9.4,
// 14.4; but 8 of 700 11.2, 10.3). One sequence of 5000, 8 kv heads: 12.1, one tile at least 14.5.
constexpr uint32_t kLong = 16;
constexpr uint32_t kLeast = 4;
// Pieces that are joined at once; more are joined in groups of kJoin first (64 pieces of 8 q heads:
// 17.3 us for the run at once, 14.0 in groups; 32: 13.0 at once, 14.0 in groups)
constexpr int kSingle = 32;
constexpr int kJoin = 16;
constexpr int kChunk = 16;           // pieces whose loads are in flight together
constexpr int kRaise = 4;            // raise the maximum when a tile's is above it by this

// Partial results pass between workgroups that may sit on different XCDs, whose L2s are not coherent.
// They are stored and loaded as relaxed atomics of agent scope, which write through and read past
// the L2: once a store is acknowledged (vmcnt 0) every later agent-scope load sees it, so no
// workgroup has to write its L2 back or invalidate it, which costs far more than the few kilobytes.
__device__ inline void store_shared(float* p, f32x4 x) {
  uint64_t* w = reinterpret_cast<uint64_t*>(p);
  const u32x4 b = __builtin_bit_cast(u32x4, x);
  __hip_atomic_store(w, (uint64_t)b[1] << 32 | b[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(w + 1, (uint64_t)b[3] << 32 | b[2], __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline void store_shared2(float* p, float x, float y) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p),
                     (uint64_t)__builtin_bit_cast(uint32_t, y) << 32 | __builtin_bit_cast(uint32_t, x),
                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline f32x4 load_shared4(const float* p) {
  const uint64_t* w = reinterpret_cast<const uint64_t*>(p);
  const uint64_t a = __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint64_t b = __hip_atomic_load(w + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return __builtin_bit_cast(f32x4, u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b,
                                         (uint32_t)(b >> 32)});
}
__device__ inline void load_shared2(const float* p, float& x, float& y) {
  const uint64_t a = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
  x = __builtin_bit_cast(float, (uint32_t)a);
  y = __builtin_bit_cast(float, (uint32_t)(a >> 32));
}

// What works on a run of tiles: a workgroup's 4 waves together, or (NW = 1) each wave by itself, for
// which the barriers below are none and threads are counted in the wave.
template <int NW>
__device__ inline void sync() {
  if constexpr (NW == 1) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  } else {
    __syncthreads();
  }
}
template <int NW>
__device__ inline int thread() {
  return NW == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
}

// The factor that brings a sum with maximum m to the maximum `top` >= m, units of `scale` in base 2. A
// sum without a finite score keeps its own: it is 0, or NaN.
__device__ inline float weight(float m, float top, float scale) {
  return m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - top) * scale);
}

// What a unit of the maxima is in base 2: they are products q . k, or capped scores.
__device__ inline float unit(const AttnParams& p) { return p.cap != 0.0f ? 1.0f : p.scale; }

// Sum or maximum over the 4 lane groups of 16 (lanes l, l ^ 16, l ^ 32, l ^ 48), by exchanges of rows
// between registers; a shuffle through LDS takes some 100 clocks, and every tile waits for one.
template <class F>
__device__ inline float across(float x, F f) {
  const auto h = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x),
                                                  __builtin_bit_cast(uint32_t, x), false, false);
  x = f(__builtin_bit_cast(float, (uint32_t)h[0]), __builtin_bit_cast(float, (uint32_t)h[1]));
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x),
                                                  __builtin_bit_cast(uint32_t, x), false, false);
  return f(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ inline float across_max(float x) {
  return across(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ inline float across_sum(float x) {
  return across(x, [](float a, float b) { return a + b; });
}

// Stops the compiler from moving what is computed from x out of a loop, into registers that the loop
// needs for its loads.
__device__ inline int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// cap * tanh(s / cap) of a product x = q . k, in base 2, to ten roundings of the score itself however far
// the cap is from it. With u = s / cap: from |u| = 5/16 on as 1 - 2 / (e^2u + 1), where the subtraction
// loses two bits at most; below, where it would lose them all, as s times the series of tanh(u) / u, whose
// first term left out is 8e-8 there. z is 2u in base 2. ALL: no lane has a |u| from 5/16 on (or NaN,
// which the series keeps).
constexpr float kPerU = 2.88539008177792681f, kFar = 0.3125f * kPerU;  // 2 log2 e
template <bool ALL>
__device__ inline float capped(const AttnParams& p, float x) {
  constexpr float k2 = kPerU * kPerU;
  const float z = x * p.inv_cap, y = z * z;
  float r = fmaf(y, 62.0f / 2835.0f / (k2 * k2 * k2 * k2), -17.0f / 315.0f / (k2 * k2 * k2));
  r = fmaf(y, r, 2.0f / 15.0f / (k2 * k2));
  r = fmaf(y, r, -1.0f / 3.0f / k2);
  r = fmaf(y, r, 1.0f) * (x * p.scale);
  if constexpr (!ALL) {
    const float e = __builtin_amdgcn_exp2f(z);
    const float far = fmaf(__builtin_amdgcn_rcpf(e + 1.0f), -2.0f, 1.0f) * p.cap;
    r = fabsf(z) >= kFar ? far : r;
  }
  return r;
}

// The head of a sequence's weights by the tokens that are attended to. (The other end, bf16: the
// products of values below 2^-122, and 2^-105 of 131072 tokens, are subnormal and lose bits one by one:
// a sharp softmax over 9000 values is exact to the output's rounding down to 2^-120, to 3% at 2^-126.)
template <int DT>
__device__ inline int head_of(int64_t tokens) {
  if (DT == AGMM_F16) return 11;
  return -kRaise - (tokens > 1 ? 32 - __builtin_clz((uint32_t)(tokens - 1)) : 0);
}

// What one wave loads of a tile of tokens, as it comes from memory.
template <int ST, int DP>
struct Raw {
  // Sub-tiles of 16 tokens. 64 tokens share the cost of placing a tile and of its softmax; a tile's
  // registers are loaded again while it is worked on (32 x 8192 tokens, e2m1: rows of 64 44 us, 58 with
  // 32 tokens; of 128 61, 67). kTwo: for 16-bit rows of 128 those registers spill (4.6 TB/s); 32
  // tokens in each of two tiles' registers reach 6.0. e4m3 rows of 256 spill with 64 tokens too. Rows of
  // 256 in e4m3 and e2m1 spill 8 and 13 registers as they are (5.4 and 4.7 TB/s, rows of 128 5.2 and 4.9).
  static constexpr bool kTwo = ST == AG_KV_16BIT && DP == 128;
  static constexpr int kSub = kTwo || (ST == AG_KV_MXFP8 && DP == 256) ? 2 : 4;
  static constexpr int kTokens = 16 * kSub;
  static constexpr int kSteps = DP / 32;  // matrix instructions over the head for 16 tokens
  // K: loads a lane makes for one token, and words in each
  static constexpr int kWords = ST == AG_KV_MXFP4 && DP == 64 ? 2 : 4;
  static constexpr int kLoads = ST == AG_KV_16BIT ? DP / 32
                                : ST == AG_KV_MXFP8 ? DP / 64 : (DP == 64 ? 1 : DP / 128);
  static constexpr int kPer = kSteps / kLoads;  // matrix instructions a load feeds
  static constexpr int kScales = ST == AG_KV_16BIT ? 0 : (DP == 256 ? 2 : 1);  // scale words a row
  static constexpr int kScaleRegs = kScales ? kScales : 1;
  // V: chunks of kElems elements a lane takes of each token, and bytes of a chunk
  static constexpr int kElems = DP == 64 ? 4 : 8;
  static constexpr int kChunks = DP == 256 ? 2 : 1;
  static constexpr int kBytes = ST == AG_KV_16BIT ? 2 * kElems : ST == AG_KV_MXFP8 ? kElems : kElems / 2;
  static constexpr int kVWords = (kBytes + 3) / 4;

  uint32_t k[kSub][kLoads][kWords];
  uint32_t v[kSub][4][kChunks][kVWords];    // of tokens 4 g .. 4 g + 3 of each sub-tile
  uint32_t ks[kScaleRegs], vs[kScaleRegs];  // of token `lane`

  // First element of a lane's operand in matrix instruction `step`, lane group g.
  __device__ static inline int first(int step, int g) {
    const int load = step / kPer, part = step % kPer;
    return load * 32 * kPer + g * 8 * kPer + part * 8;
  }
  __device__ static inline int bytes_of(int e) {
    return ST == AG_KV_16BIT ? 2 * e : ST == AG_KV_MXFP8 ? e : e / 2;
  }
};

template <int N>
__device__ inline void load_words(uint32_t (&w)[N], const char* p) {
  if constexpr (N == 4) {
    const u32x4 t = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = t[i];
  } else if constexpr (N == 2) {
    const u32x2 t = *reinterpret_cast<const u32x2*>(p);
    w[0] = t[0];
    w[1] = t[1];
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

template <int DP>
constexpr int kScalesOf = 64 * (DP == 256 ? 2 : 1);
template <int DP, int NW>
struct Shared {
  int64_t at[NW][64][2];                  // the tokens' places: data and scale offsets
  uint32_t scales[NW][2][kScalesOf<DP>];  // the tokens' scale words, keys' and values'
  float m[NW][16], l[NW][16];
  float acc[NW][16][DP + 4];
  uint32_t last[2];
};

template <int DT, int ST, int DP, bool CAP>
struct Wave {
  typedef Raw<ST, DP> R;
  static constexpr int kAcc = R::kElems * R::kChunks;
  static constexpr uint64_t kAll = R::kTokens == 64 ? ~0ull : (1ull << (R::kTokens & 63)) - 1;

  u32x4 q[R::kSteps];
  f32x4 acc[kAcc];
  float m, l;  // of this lane's q head, m in unit()s; l of this lane's tokens alone

  __device__ inline void start(const AttnParams& p, int64_t b, int head0, int n) {
    const int lane = here(threadIdx.x) & 63, col = lane & 15, g = lane >> 4;
    const uint16_t* row = p.q + b * p.q_batch + (int64_t)(head0 + (col < n ? col : 0)) * p.q_head;
#pragma unroll
    for (int i = 0; i < R::kSteps; ++i) {
      const int e = R::first(i, g);
      q[i] = u32x4{0, 0, 0, 0};
      if (col < n && e < p.c.head_dim) q[i] = load16(row + e);
    }
#pragma unroll
    for (int i = 0; i < kAcc; ++i) acc[i] = f32x4{0, 0, 0, 0};
    m = -INFINITY;
    l = 0.0f;
  }

  // The loads of the tile whose tokens' places are in `at`. A token that is not attended to has the
  // place of the pools' first row, and lanes past the head's end read its first elements: what comes
  // back there is thrown away below, and the loads need no branches.
  __device__ static inline void load_k(R& r, const AttnParams& p, const int64_t (*at)[2],
                                       int64_t head, int64_t s_head) {
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int hd = p.c.head_dim;
#pragma unroll
    for (int t = 0; t < R::kSub; ++t) {
      const char* row = p.c.k + head + at[16 * t + col][0];
#pragma unroll
      for (int i = 0; i < R::kLoads; ++i) {
        const int e = R::first(i * R::kPer, g);
        load_words<R::kWords>(r.k[t][i], row + R::bytes_of(e < hd ? e : 0));
      }
    }
    if (R::kScales) load_scales(r.ks, p.c.ks + s_head, hd, at);
  }

  __device__ static inline void load_v(R& r, const AttnParams& p, const int64_t (*at)[2],
                                       int64_t head, int64_t s_head) {
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int hd = p.c.head_dim;
#pragma unroll
    for (int t = 0; t < R::kSub; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const char* row = p.c.v + head + at[16 * t + 4 * g + j][0];
#pragma unroll
        for (int c = 0; c < R::kChunks; ++c) {
          const int e = 128 * c + R::kElems * col;
          const char* from = row + R::bytes_of(e < hd ? e : 0);
          if constexpr (R::kBytes == 2)
            r.v[t][j][c][0] = *reinterpret_cast<const uint16_t*>(from);
          else
            load_words<R::kVWords>(r.v[t][j][c], from);
        }
      }
    if (R::kScales) load_scales(r.vs, p.c.vs + s_head, hd, at);
  }

  __device__ static inline void load_scales(uint32_t (&w)[R::kScaleRegs], const char* pool, int hd,
                                            const int64_t (*at)[2]) {
    const char* row = pool + at[threadIdx.x & 63][1];
#pragma unroll
    for (int i = 0; i < R::kScales; ++i)
      w[i] = *reinterpret_cast<const uint32_t*>(row + (128 * i < hd ? 4 * i : 0));
  }

  // Scale words from the lane that loaded them to where the other lanes find them.
  __device__ static inline void share(uint32_t* to, const uint32_t (&w)[R::kScaleRegs]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < R::kScales; ++i) to[lane * R::kScales + i] = w[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }

  // The K operand of matrix instruction `step` for sub-tile t, whose scale words are w.
  __device__ static inline u32x4 key(const R& r, int t, int step, int g, const uint32_t* w) {
    const int i = step / R::kPer, part = step % R::kPer;
    if constexpr (ST == AG_KV_16BIT) {
      return u32x4{r.k[t][i][0], r.k[t][i][1], r.k[t][i][2], r.k[t][i][3]};
    } else {
      const int block = R::first(step, 0) / 32 + (g * R::kPer * 8) / 32;
      const uint32_t word = R::kScales == 2 && block >= 4 ? w[R::kScales - 1] : w[0];
      const float s = scale_of((word >> (8 * (block & 3))) & 255u);
      if constexpr (ST == AG_KV_MXFP8)
        return from_fp8x8<DT>(r.k[t][i][2 * part], r.k[t][i][2 * part + 1], s);
      else
        return from_fp4x8<DT>(r.k[t][i][part], s);
    }
  }

  // S^T of the tile, or (HEADS) S: lane = token, 4 consecutive q heads; `sc`: the wave's place for the keys'
  // scale words.
  template <bool HEADS = false>
  __device__ inline void scores(R& r, const AttnParams& p, uint32_t* sc, f32x4 (&st)[R::kSub]) const {
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int hd = p.c.head_dim;
    uint32_t kw[R::kSub][R::kScaleRegs];
    if (R::kScales) {
      share(sc, r.ks);
#pragma unroll
      for (int t = 0; t < R::kSub; ++t)
#pragma unroll
        for (int i = 0; i < R::kScales; ++i) kw[t][i] = sc[(16 * t + col) * R::kScales + i];
    }
    if (hd != DP) {  // the keys' elements past the head's end are zeros
      const int me = here(g);
#pragma unroll
      for (int i = 0; i < R::kLoads; ++i)
        if (R::first(i * R::kPer, me) >= hd) {
#pragma unroll
          for (int t = 0; t < R::kSub; ++t)
#pragma unroll
            for (int w = 0; w < R::kWords; ++w) r.k[t][i][w] = 0;
        }
      // (the scale bytes behind the row's last block hold anything: 255 would make those zeros NaN)
#pragma unroll
      for (int i = 0; i < R::kScales; ++i) {
        const int left = hd - 128 * i;
        const uint32_t mask = left >= 128 ? ~0u : left <= 0 ? 0u : (1u << left / 4) - 1u;
#pragma unroll
        for (int t = 0; t < R::kSub; ++t) kw[t][i] &= mask;
      }
    }
#pragma unroll
    for (int t = 0; t < R::kSub; ++t) st[t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < R::kSteps; ++i)
#pragma unroll
      for (int t = 0; t < R::kSub; ++t)
        st[t] = HEADS ? T16<DT>::mfma(q[i], key(r, t, i, g, kw[t]), st[t])
                      : T16<DT>::mfma(key(r, t, i, g, kw[t]), q[i], st[t]);
  }

  // Scores to weights: st, products or capped scores, becomes 2^((st - m) scale + up), with m raised and
  // what is summed rescaled first where needed.
  __device__ inline void weights(const AttnParams& p, uint64_t there, int up, f32x4 (&st)[R::kSub]) {
    float scale = p.scale;
    if constexpr (CAP) {
      // Most scores are far below the cap: one branch for the wave leaves the exponential out (96 ragged
      // sequences, e2m1 rows of 64, a cap of 30: 27.0 us, one of 2: 29.7; none: 24.4). The other side is
      // expected less so that it does not make rows of 256 spill more (32 x 8192 tokens, e2m1, a cap of
      // 30: 122 us, 128).
      scale = 1.0f;
      float most = 0.0f;
#pragma unroll
      for (int t = 0; t < R::kSub; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) most = fmaxf(most, fabsf(st[t][j]));
      if (__builtin_expect(__any(most * p.inv_cap >= kFar), 0)) {
#pragma unroll
        for (int t = 0; t < R::kSub; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) st[t][j] = capped<false>(p, st[t][j]);
      } else {
#pragma unroll
        for (int t = 0; t < R::kSub; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) st[t][j] = capped<true>(p, st[t][j]);
      }
    }
    if (there != kAll) {
      const int g = here(threadIdx.x & 63) >> 4;
#pragma unroll
      for (int t = 0; t < R::kSub; ++t) {
        const uint32_t mine = (uint32_t)(there >> (16 * t)) >> (4 * g);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          st[t][j] = __builtin_bit_cast(
              float, here(__builtin_bit_cast(int, (mine >> j) & 1u ? st[t][j] : -INFINITY)));
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < R::kSub; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, st[t][j]);
    top = across_max(top);
    if (__any((top - m) * scale > (float)kRaise)) {
      const float raised = fmaxf(m, top);
      const float f = weight(m, raised, scale);
#pragma unroll
      for (int i = 0; i < kAcc; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) acc[i][w] *= f;
      l *= f;
      m = raised;
    }
    // The maximum is taken away before the scale comes in: rounded to base 2 first it would be up to half
    // an ulp off, from 2^27 on more than all of a weight's head.
    const float ref = m == -INFINITY ? 0.0f : m, head = (float)up;
#pragma unroll
    for (int t = 0; t < R::kSub; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        st[t][j] = __builtin_amdgcn_exp2f(fmaf(st[t][j] - ref, scale, head));
        l += st[t][j];
      }
  }

  // O^T += V^T P^T; `sc`: the wave's place for the values' scale words.
  __device__ inline void values(R& r, uint64_t there, uint32_t* sc, const f32x4 (&st)[R::kSub]) {
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    if (R::kScales) share(sc, r.vs);
#pragma unroll
    for (int h = 0; h < R::kSub; h += 2) {  // 32 tokens
      u32x4 hi, lo;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x2 w = T16<DT>::split(st[h + j / 2][2 * j % 4], st[h + j / 2][2 * j % 4 + 1]);
        hi[j] = w[0];
        lo[j] = w[1];
      }
#pragma unroll
      for (int c = 0; c < R::kChunks; ++c) {
        uint32_t v[8][R::kElems / 2];  // 8 tokens x kElems elements
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const auto& w = r.v[h + j / 4][j % 4][c];
          if constexpr (ST == AG_KV_16BIT) {
#pragma unroll
            for (int i = 0; i < R::kElems / 2; ++i) v[j][i] = w[i];
          } else {
            // the scale of this lane's elements: block kElems * col / 32 of these 128
            const uint32_t word = sc[(16 * (h + j / 4) + 4 * g + j % 4) * R::kScales + c];
            const float s = scale_of((word >> (8 * (R::kElems * col >> 5))) & 255u);
            if constexpr (ST == AG_KV_MXFP8) {
#pragma unroll
              for (int i = 0; i < R::kVWords; ++i) {
                v[j][2 * i] = T16<DT>::template from_fp8<0>(w[i], s);
                v[j][2 * i + 1] = T16<DT>::template from_fp8<1>(w[i], s);
              }
            } else {
              v[j][0] = T16<DT>::template from_fp4<0>(w[0], s);
              v[j][1] = T16<DT>::template from_fp4<1>(w[0], s);
              if constexpr (R::kElems == 8) {
                v[j][2] = T16<DT>::template from_fp4<2>(w[0], s);
                v[j][3] = T16<DT>::template from_fp4<3>(w[0], s);
              }
            }
          }
        }
        // the values of tokens that are not attended to count as zeros (the results go through here()
        // so that this stays a branch, which all but the last tiles skip)
        if (there != kAll) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const bool keep = (uint32_t)(there >> (16 * (h + j / 4))) >> (4 * here(g) + j % 4) & 1u;
#pragma unroll
            for (int i = 0; i < R::kElems / 2; ++i) v[j][i] = here(keep ? v[j][i] : 0);
          }
        }
#pragma unroll
        for (int e = 0; e < R::kElems; ++e) {
          u32x4 a;  // 8 tokens of element e
#pragma unroll
          for (int j = 0; j < 4; ++j)
            a[j] = __builtin_amdgcn_perm(v[2 * j + 1][e / 2], v[2 * j][e / 2],
                                         e % 2 ? 0x07060302u : 0x05040100u);
          f32x4& o = acc[R::kElems * c + e];
          o = T16<DT>::mfma(a, hi, o);
          o = T16<DT>::mfma(a, lo, o);
        }
      }
    }
  }
};

// A partial result: p.rows rows of DP sums, then the rows' maxima and sums in pairs.
template <int DP>
__device__ inline float* partial(const AttnParams& p, uint32_t slot) {
  return p.partials + (int64_t)slot * (p.rows * (DP + 2));
}

struct Range {  // tokens [first, end) of a sequence; tiles begin at `from`, a multiple of 16
  int64_t from, first, end;
};
__device__ inline Range range_of(const AttnParams& p, int32_t len) {
  const int64_t n = max(len, 0), end = min(n, (int64_t)p.capacity);
  const int64_t first = p.window > 0 ? min(max((int64_t)0, n - p.window), end) : 0;
  return Range{first & ~(int64_t)15, first, end};
}
__device__ inline uint32_t tiles_of(const AttnParams& p, int32_t len) {
  const Range r = range_of(p, len);
  return r.first == r.end ? 0 : (uint32_t)((r.end - r.from + kAttnTile - 1) / kAttnTile);
}

template <int CTRL, int ROWS>
__device__ inline uint32_t add_from(uint32_t x) {
  return x + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false);
}
// Sum over the lanes up to and with this one: within rows of 16 lanes, then the rows' sums.
__device__ inline uint32_t wave_scan(uint32_t x) {
  x = add_from<0x111, 0xf>(x);
  x = add_from<0x112, 0xf>(x);
  x = add_from<0x114, 0xf>(x);
  x = add_from<0x118, 0xf>(x);
  x = add_from<0x142, 0xa>(x);
  return add_from<0x143, 0xc>(x);
}
__device__ inline uint32_t wave_sum(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_readlane((int)wave_scan(x), 63);
}

// Elements e .. e + 3 of a row: o over the row's sum l, and the row's lse with element 0.
template <int DT, int DP, int WAY>
__device__ inline void finish(const AttnParams& p, int64_t b, int head, int e, f32x4 o, float m,
                              float l, int up) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // 0: nothing was attended to
  if constexpr (WAY == kPieces) {
    const int64_t row = b * p.q_heads + head;
#pragma unroll
    for (int w = 0; w < 4; ++w) o[w] *= inv;
    *reinterpret_cast<f32x4*>(p.prefix.own + row * DP + e) = o;
    if (e == 0) {
      p.prefix.own_stats[2 * row] = m;
      p.prefix.own_stats[2 * row + 1] = ldexpf(l, -up);
    }
    return;
  }
  typedef u32x2 u32x2_any __attribute__((aligned(2)));
  *reinterpret_cast<u32x2_any*>(p.out + b * p.o_batch + (int64_t)head * p.o_head + e) =
      u32x2{T16<DT>::pack(o[0] * inv, o[1] * inv), T16<DT>::pack(o[2] * inv, o[3] * inv)};
  if (e == 0 && p.lse)
    p.lse[b * p.q_heads + head] =
        l == 0.0f ? -INFINITY
                  : (m * unit(p) + __builtin_amdgcn_logf(ldexpf(l, -up))) * 0.69314718055994531f;
}

// A head's part that a workgroup does not have all of.
struct Piece {
  int b, head0, n;          // sequence, first q head, q heads
  int up;                   // head of the sequence's weights
  uint32_t begin, pieces;   // workgroup that has the head's first tile; workgroups that have any
};

// Joins `count` partial results of a head: of workgroups wg0, wg0 + stride, ..., the one of the
// workgroup where the head begins in slot 1 and the others in slot 0. final: the output; else a
// partial result again, in the place of the first.
template <int DT, int DP, int WAY, int NW>
__device__ inline void join(const AttnParams& p, Shared<DP, NW>& sh, const Piece& h, uint32_t wg0,
                            uint32_t stride, uint32_t count, bool final) {
  auto slot = [&](uint32_t i) {
    const uint32_t wg = wg0 + i * stride;
    return partial<DP>(p, 2 * wg + (wg == h.begin ? 1 : 0));
  };
  const int d4 = p.c.head_dim / 4, tid = here(thread<NW>());
#pragma unroll 1
  for (int idx = tid; idx < h.n * d4; idx += NW * 64) {
    const int row = idx / d4, e = (idx - row * d4) * 4;
    f32x4 o = {0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (uint32_t c = 0; c < count; c += kChunk) {
      f32x4 x[kChunk];
      float mi[kChunk], li[kChunk];
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {  // (past the last: the last again, not counted below)
        const float* s = slot(min(c + i, count - 1));
        load_shared2(s + p.rows * DP + 2 * row, mi[i], li[i]);
        x[i] = load_shared4(s + row * DP + e);
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < kChunk; ++i) top = fmaxf(top, mi[i]);
      const float f = weight(m, top, unit(p));
      l *= f;
#pragma unroll
      for (int w = 0; w < 4; ++w) o[w] *= f;
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        if (c + i < count) {
          const float g = weight(mi[i], top, unit(p));
          l = fmaf(g, li[i], l);
#pragma unroll
          for (int w = 0; w < 4; ++w) o[w] = fmaf(g, x[i][w], o[w]);
        }
      }
      m = top;
    }
    if (final) {
      finish<DT, DP, WAY>(p, h.b, h.head0 + row, e, o, m, l, h.up);
    } else {
#pragma unroll
      for (int w = 0; w < 4; ++w) sh.acc[0][row][e + w] = o[w];
      if (e == 0) {
        sh.m[0][row] = m;
        sh.l[0][row] = l;
      }
    }
  }
  if (final) return;
  sync<NW>();  // every piece has been read: the first one's place is free
#pragma unroll 1
  for (int idx = tid; idx < h.n * d4; idx += NW * 64) {
    const int row = idx / d4, e = (idx - row * d4) * 4;
    float* s = slot(0);
    const float* o = &sh.acc[0][row][e];
    store_shared(s + row * DP + e, f32x4{o[0], o[1], o[2], o[3]});
    if (e == 0) store_shared2(s + p.rows * DP + 2 * row, sh.m[0][row], sh.l[0][row]);
  }
}

// Counts a partial result in; true for the one that comes last of `size`, which leaves the counter
// cleared for the next run. The partial result's stores have been acknowledged.
__device__ inline bool count_in(uint32_t* counter, uint32_t size) {
  const uint32_t before =
      __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (before + 1 != size) return false;
  __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return true;
}
// All stores so far are acknowledged.
template <int NW>
__device__ inline void settle() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  sync<NW>();
}

// The waves' results of tokens of one head, put together: the output if that was all of the head,
// else a partial result in the workgroup's slot.
template <int DT, int ST, int DP, bool CAP, int WAY, int NW>
__device__ inline void combine(const AttnParams& p, const Wave<DT, ST, DP, CAP>& w,
                               Shared<DP, NW>& sh, const Piece& h,
                               uint32_t me) {
  const int tid = here(thread<NW>());
  const int lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
  const float l = across_sum(w.l);
  if (g == 0) {
    sh.m[wave][col] = w.m;
    sh.l[wave][col] = l;
  }
  sync<NW>();
  float m = sh.m[0][col];
#pragma unroll
  for (int i = 1; i < NW; ++i) m = fmaxf(m, sh.m[i][col]);
  const float f = weight(w.m, m, unit(p));
  if (col < h.n) {
    constexpr int kElems = Raw<ST, DP>::kElems;
#pragma unroll
    for (int c = 0; c < Raw<ST, DP>::kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < kElems; ++k)
          sh.acc[wave][col][128 * c + kElems * (4 * g + i) + k] = w.acc[kElems * c + k][i] * f;
  }
  sync<NW>();
  const bool whole = h.pieces == 1;
  float* slot = partial<DP>(p, 2 * me + (me == h.begin ? 1 : 0));
  const int d4 = p.c.head_dim / 4;
  for (int idx = tid; idx < h.n * d4; idx += NW * 64) {
    const int row = idx / d4, e = (idx - row * d4) * 4;
    float rm = sh.m[0][row], rl = 0.0f;
#pragma unroll
    for (int i = 1; i < NW; ++i) rm = fmaxf(rm, sh.m[i][row]);
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      rl += sh.l[i][row] * weight(sh.m[i][row], rm, unit(p));
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] += sh.acc[i][row][e + k];
    }
    if (whole) {
      finish<DT, DP, WAY>(p, h.b, h.head0 + row, e, o, rm, rl, h.up);
    } else {
      store_shared(slot + row * DP + e, o);
      if (e == 0) store_shared2(slot + p.rows * DP + 2 * row, rm, rl);
    }
  }
  sync<NW>();  // sh is free again
}

// The run of tiles of worker `me` of `wgs` (NW = 4: workgroups, NW = 1: waves), out of the `total` tiles
// of all sequences and heads.
template <int DT, int ST, int DP, bool CAP, int WAY, int NW>
__device__ inline void work(const AttnParams& p, Shared<DP, NW>& sh, uint32_t me, uint32_t wgs,
                            uint32_t total, uint32_t least, uint32_t whole) {
  typedef Wave<DT, ST, DP, CAP> W;
  typedef typename W::R R;
  const int tid = thread<NW>(), lane = threadIdx.x & 63;
  const int wave = NW == 1 ? 0 : __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const uint32_t heads = (uint32_t)(p.c.kv_heads * p.q_groups);
  // an equal share, but at least `least` tiles once that gives every compute unit 4 waves, and never
  // less than `whole`
  constexpr uint32_t kFill = 4 * kCus / NW;
  const uint32_t quota = max(max((total + wgs - 1) / wgs, whole), min(least, (total + kFill - 1) / kFill));
  uint32_t cur = me * quota;
  if (cur >= total) return;
  const uint32_t end = min(cur + quota, total);

  // the sequence and head where it begins
  int b = 0;
  uint32_t before = 0;  // tiles of one head of the sequences in front
  for (int c = 0; c < p.batch; c += 64) {
    const uint32_t t = c + lane < p.batch ? tiles_of(p, p.lens[c + lane]) : 0;
    const uint32_t scan = wave_scan(t);
    const uint64_t hit = __ballot((before + scan) * heads > cur);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      b = c + at;
      before += (uint32_t)__builtin_amdgcn_readlane((int)(scan - t), at);
      break;
    }
    before += (uint32_t)__builtin_amdgcn_readlane((int)scan, 63);
  }
  Range seq = range_of(p, p.lens[b]);
  uint32_t tiles = (uint32_t)((seq.end - seq.from + kAttnTile - 1) / kAttnTile);
  uint32_t head = (cur - before * heads) / tiles;
  uint32_t start = before * heads + head * tiles;  // first tile of the head

  Piece part[2];  // what it has of heads shared with others: one that began before, one that goes on
  part[0].pieces = part[1].pieces = 0;
  while (true) {
    const uint32_t stop = min(end, start + tiles);
    const int64_t t0 = seq.from + (int64_t)(cur - start) * kAttnTile;
    const int64_t t1 = min(seq.end, seq.from + (int64_t)(stop - start) * kAttnTile);
    const int kv = (int)head / p.q_groups, group = (int)head - kv * p.q_groups;
    const int64_t hoff = kv * p.c.head, shoff = kv * p.c.s_head;
    Piece h;
    h.b = b;
    h.head0 = kv * p.group + 16 * group;
    h.n = min(16, p.group - 16 * group);
    h.up = head_of<DT>(seq.end - seq.first);
    h.begin = start / quota;
    h.pieces = (start + tiles - 1) / quota - h.begin + 1;

    W w;
    w.start(p, b, h.head0, h.n);
    const int32_t* table = p.table + (int64_t)b * p.table_row + (WAY == kHeads ? kv * p.table_head : 0);
    int64_t(*at)[2] = sh.at[wave];
    // The page of token base + lane; past the end, the last token's.
    auto page_of = [&](int64_t base) {
      const uint32_t t = (uint32_t)min(base + lane, t1 - 1);
      return table[t / p.c.page_size];
    };
    // Puts the tokens' places into LDS; bit t of the result: token base + t is attended to.
    auto place = [&](int64_t base, int32_t page) {
      const int64_t tok = base + lane;
      const bool ok = (uint32_t)page < (uint32_t)p.num_pages && tok >= seq.first && tok < t1;
      const uint64_t there = __ballot(ok) & W::kAll;
      const uint32_t t = (uint32_t)tok;
      const uint32_t row = t - (t / p.c.page_size) * p.c.page_size.d;
      at[lane][0] = ok ? row_at(p.c, page, row) : 0;
      if (R::kScales) at[lane][1] = ok ? scales_at(p.c, page, row) : 0;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      return there;
    };
    // Tiles of the wave, t0 + (wave + NW * i) * kTokens. (Past the last tile the loads read the
    // pools' first row.)
    constexpr int kStep = NW * R::kTokens;
    int64_t base = t0 + wave * R::kTokens;
    if (base < t1) {
      uint64_t there = place(base, page_of(base));
      int32_t page = page_of(base + kStep);
      uint32_t(*sc)[kScalesOf<DP>] = sh.scales[wave];
      if constexpr (R::kTwo) {
        // a tile is loaded while the one in front of it is worked on
        R r0, r1;
        auto load = [&](R& r) {
          W::load_k(r, p, at, hoff, shoff);
          W::load_v(r, p, at, hoff, shoff);
        };
        auto step = [&](R& now, R& after) {
          base += kStep;
          const uint64_t next = place(base, page);
          page = page_of(base + kStep);
          load(after);
          f32x4 st[R::kSub];
          w.scores(now, p, sc[0], st);
          w.weights(p, there, h.up, st);
          w.values(now, there, sc[1], st);
          there = next;
        };
        load(r0);
        while (true) {
          step(r0, r1);
          if (base >= t1) break;
          step(r1, r0);
          if (base >= t1) break;
        }
      } else {
        // The next tile's keys are loaded into their registers as soon as the scores are made, the
        // next values once theirs are used, so that loads are under way all the time.
        R r;
        W::load_k(r, p, at, hoff, shoff);
        W::load_v(r, p, at, hoff, shoff);
        while (true) {
          f32x4 st[R::kSub];
          w.scores(r, p, sc[0], st);
          base += kStep;
          const uint64_t next = place(base, page);
          page = page_of(base + kStep);
          W::load_k(r, p, at, hoff, shoff);
          w.weights(p, there, h.up, st);
          w.values(r, there, sc[1], st);
          if (base >= t1) break;
          W::load_v(r, p, at, hoff, shoff);
          there = next;
        }
      }
    }
    combine<DT, ST, DP, CAP, WAY>(p, w, sh, h, me);
    if (h.pieces > 1) (h.begin == me ? part[1] : part[0]) = h;

    cur = stop;
    if (cur >= end) break;
    start += tiles;  // the next head, and after the last the next sequence with a tile
    if (++head == heads) {
      head = 0;
      do {
        seq = range_of(p, p.lens[++b]);
        tiles = seq.first == seq.end
                    ? 0
                    : (uint32_t)((seq.end - seq.from + kAttnTile - 1) / kAttnTile);
      } while (tiles == 0);
    }
  }

  if (part[0].pieces == 0 && part[1].pieces == 0) return;
  settle<NW>();
  // A workgroup begins at most one head that goes on, and at most one later group of 16 pieces: a
  // counter for either, and one for the groups of a head.
  auto group_of = [&](const Piece& h) { return (me - h.begin) / kJoin; };
  if (tid < 2) {
    const Piece h = tid ? part[1] : part[0];
    bool last = false;
    if (h.pieces > kSingle) {
      const uint32_t g = group_of(h);
      last = count_in(p.counters + (g == 0 ? wgs : 2 * wgs) + h.begin + g * kJoin,
                      min((uint32_t)kJoin, h.pieces - g * kJoin));
    } else if (h.pieces) {
      last = count_in(p.counters + h.begin, h.pieces);
    }
    sh.last[tid] = last;
  }
  sync<NW>();
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    if (!sh.last[i]) continue;
    const Piece h = i ? part[1] : part[0];
    const uint32_t g = group_of(h), groups = (h.pieces + kJoin - 1) / kJoin;
    bool final = h.pieces <= kSingle;
    uint32_t first = final ? h.begin : h.begin + g * kJoin, stride = 1;
    uint32_t count = final ? h.pieces : min((uint32_t)kJoin, h.pieces - g * kJoin);
    while (true) {
      join<DT, DP, WAY>(p, sh, h, first, stride, count, final);
      if (final) break;
      settle<NW>();
      if (tid == 0) sh.last[i] = count_in(p.counters + h.begin, groups);
      sync<NW>();
      if (!sh.last[i]) break;
      final = true;
      first = h.begin;
      stride = kJoin;
      count = groups;
    }
    sync<NW>();  // sh is free again
  }
}

// What the lengths say about the work: tiles of one head; sequences with one or two, with three, with any.
struct Census {
  uint32_t tiles, short_ones, threes, sequences;
};
__device__ inline Census census(const AttnParams& p) {
  const int lane = threadIdx.x & 63;
  uint32_t sum = 0, few = 0, mid = 0, some = 0;
  for (int b = lane; b < p.batch; b += 64) {
    const uint32_t t = tiles_of(p, p.lens[b]);
    sum += t;
    few += t == 1 || t == 2 ? 1 : 0;
    mid += t == 3 ? 1 : 0;
    some += t ? 1 : 0;
  }
  return Census{wave_sum(sum), wave_sum(few), wave_sum(mid), wave_sum(some)};
}

template <int DP>
union AttnShared {
  Shared<DP, 4> together;
  Shared<DP, 1> alone[4];
};

// The share of workgroup `me` of `wgs`.
template <int DT, int ST, int DP, bool CAP, int WAY>
__device__ inline void share_of(const AttnParams& p, AttnShared<DP>& sh, const Census& c, uint32_t me,
                                uint32_t wgs) {
  const uint32_t heads = (uint32_t)(p.c.kv_heads * p.q_groups);
  // Heads that all have 2 or all have 3 tiles are not cut: one workgroup's second step costs less than
  // joining (300 tokens, bf16 8.6 us, cut 9.5; 200 7.6, 9.5). With 4 tiles neither wins (9.7, 9.6). All
  // shares are alike, so none leaves heads of 2 and of 3 tiles whole both: those are cut as any others.
  const bool twos = c.short_ones == c.sequences && c.tiles == 2 * c.sequences;
  const uint32_t whole = c.threes == c.sequences ? 3 : twos ? 2 : 1;
  // Where many heads have but a tile or two, a workgroup's waves would wait for each other at every
  // one of them: each wave works by itself then, on two tiles or more unless no head has more than one.
  // 96 ragged sequences (8 kv heads, e2m1, window) 26.5 us, together 45; 256 of 50 tokens (bf16) 15 us,
  // together 20. Else together: 64 of 512 (e2m1) 12 us, by themselves 17; 64 of 8192 (bf16) 355, 376;
  // and where the compute units suffice for a workgroup each: 32 of 200 (bf16, 8 kv heads) 8.0, 13.5.
  // (Behind a shared prefix `wgs` are part of the chip's: where each has a tile at most they work together.)
  const uint32_t enough = WAY == kPieces ? max(wgs, kCus * whole) : kCus * whole;
  if (c.tiles * heads > enough && 3 * c.short_ones * heads >= wgs) {
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    work<DT, ST, DP, CAP, WAY, 1>(p, sh.alone[wave], 4 * me + wave, 4 * wgs, c.tiles * heads,
                                  c.tiles == c.sequences ? 1 : 2, 1);
  } else {
    work<DT, ST, DP, CAP, WAY, 4>(p, sh.together, me, wgs, c.tiles * heads,
                                  c.tiles > kLong * c.sequences ? kLeast : 1, whole);
  }
}

template <int DT, int ST, int DP, bool CAP, int WAY>
__global__ __launch_bounds__(kThreads, attn_per_cu(ST, DP)) void attn_kernel(AttnParams p) {
  __shared__ AttnShared<DP> sh;
  const Census c = census(p);
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x)
    if (tiles_of(p, p.lens[b]) == 0) {
      const int d4 = p.c.head_dim / 4;
      for (int i = threadIdx.x; i < p.q_heads * d4; i += kThreads) {
        const int h = i / d4;
        finish<DT, DP, WAY>(p, b, h, (i - h * d4) * 4, f32x4{0, 0, 0, 0}, 0.0f, 0.0f, 0);
      }
    }
  share_of<DT, ST, DP, CAP, WAY>(p, sh, c, blockIdx.x, gridDim.x);
}

// Kernels with a cap are their own: its code in the others' way costs a call of one token 0.3 us of 5.7, and
// ragged sequences to 9000, f16, 39.6 us instead of 39.2.
template <int DT, int ST, int DP, int WAY>
void by_cap(const AttnParams& p, int grid, hipStream_t s) {
  if (p.cap != 0.0f)
    attn_kernel<DT, ST, DP, true, WAY><<<grid, kThreads, 0, s>>>(p);
  else
    attn_kernel<DT, ST, DP, false, WAY><<<grid, kThreads, 0, s>>>(p);
}

template <int DT, int ST, int WAY>
void by_width(const AttnParams& p, int grid, hipStream_t s) {
  const int dp = attn_padded(p.c.head_dim);
  if (dp == 64)
    by_cap<DT, ST, 64, WAY>(p, grid, s);
  else if (dp == 128)
    by_cap<DT, ST, 128, WAY>(p, grid, s);
  else
    by_cap<DT, ST, 256, WAY>(p, grid, s);
}

template <int DT, int WAY>
void by_storage(const AttnParams& p, int storage, int grid, hipStream_t s) {
  if (storage == AG_KV_16BIT)
    by_width<DT, AG_KV_16BIT, WAY>(p, grid, s);
  else if (storage == AG_KV_MXFP8)
    by_width<DT, AG_KV_MXFP8, WAY>(p, grid, s);
  else
    by_width<DT, AG_KV_MXFP4, WAY>(p, grid, s);
}

}  // namespace
}  // namespace agmm
