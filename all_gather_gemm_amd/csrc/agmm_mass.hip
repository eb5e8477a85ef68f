// gfx950 kernel that adds up the attention weights of cached tokens (agmm_long.h).
//
// Mathematics, for one sequence and kv head with its G q heads: S = Q K^T (heads x tokens), weights exp(s - lse)
// with the log-sum-exp that the attention has given, and their sum over the heads. Keys are read once, 2 G
// flop a 16-bit value, so the bound is the memory bandwidth; values are not read at all.
//
// Matrix instructions of 16 q heads x 16 tokens read K straight from global memory, as the attention's do
// (agmm_attn_kernel.h), with the operands the other way round: a lane's accumulators are 4 heads of one
// token, so the sum over the heads is 3 additions and two exchanges of rows. Tiles do not depend on each
// other, so each wave goes through its own; the next tile's keys are loaded as soon as the products have used
// the last one's.
//
// Measured, warm: 32 sequences of 16384 tokens, 64/8 heads of 128, bf16: 205 us, 5.5 TB/s; one of 4096, 8/1 heads: 6.3 us
// (launch, length, page, keys, each waiting for the one before). Past 16 q heads to a kv head, q and log-sum-exp are read
// again for every tile and group of 16: 32 sequences of 16384, one kv head, 16, 17, 32, 64 q heads 28, 34, 39, 53 us.
#include "agmm_attn_kernel.h"
#include "agmm_long_internal.h"

namespace agmm {
namespace {

template <int DP>
struct MassShared {
  int64_t at[4][64][2];
  uint32_t scales[4][kScalesOf<DP>];
};

template <int DT, int ST, int DP, bool CAP>
__global__ __launch_bounds__(kThreads, DP == 256 ? 2 : 4) void mass_kernel(MassParams m) {
  typedef Wave<DT, ST, DP, CAP> W;
  typedef typename W::R R;
  __shared__ MassShared<DP> sh;
  const AttnParams& p = m.a;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const uint32_t bh = blockIdx.x / (uint32_t)m.splits, split = blockIdx.x - bh * (uint32_t)m.splits;
  const int b = (int)(bh / (uint32_t)p.c.kv_heads), kv = (int)(bh - (uint32_t)b * p.c.kv_heads);
  const int32_t len = max(p.lens[b], 0);
  const int32_t held = min(len, m.tokens);       // entries that get decayed and added to; the others are copied
  const Range seq = range_of(p, len);            // tokens that are attended to
  const float* from = m.mass + b * m.mass_batch + kv * m.mass_head;
  float* to = m.out + b * m.out_batch + kv * m.out_head;
  const int32_t* table = p.table + (int64_t)b * p.table_row;
  const int64_t hoff = kv * p.c.head, shoff = kv * p.c.s_head;
  int64_t(*at)[2] = sh.at[wave];
  uint32_t* sc = sh.scales[wave];

  constexpr int kTile = R::kTokens;
  const int64_t step = (int64_t)m.splits * 4 * kTile;
  int64_t base = ((int64_t)split * 4 + wave) * kTile;

  W w;
  float lse[4], rest[4];   // in base 2, and what its rounding leaves
  bool none[4];            // adds nothing, whatever its score: 0 * infinity in a row without a head is NaN
  auto heads = [&](int group) {
    const int head0 = kv * p.group + 16 * group, count = min(16, p.group - 16 * group);
    w.start(p, b, head0, count);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int h = 4 * g + j;
      const float x = h < count ? m.lse[(int64_t)b * p.q_heads + head0 + h] : -INFINITY;
      const float log2e = 1.44269504088896340736f;
      none[j] = x == -INFINITY;
      lse[j] = none[j] ? 0.0f : x * log2e;
      rest[j] = fabsf(lse[j]) < INFINITY ? fmaf(x, log2e, -lse[j]) + x * 1.92596299e-8f : 0.0f;
    }
  };
  // Puts the places of a tile's tokens into LDS; bit t: token base + t is attended to. Loads of tiles without
  // one are left out.
  auto place = [&](int64_t base) {
    const int64_t tok = base + lane;
    bool ok = lane < kTile && tok >= seq.first && tok < min(seq.end, (int64_t)held);
    if (__ballot(ok) == 0) return (uint64_t)0;
    const uint32_t t = (uint32_t)tok, j = t / p.c.page_size;
    const int32_t page = ok ? table[j] : -1;
    ok = (uint32_t)page < (uint32_t)p.num_pages;
    const uint32_t row = t - j * p.c.page_size.d;
    at[lane][0] = ok ? row_at(p.c, page, row) : 0;
    if (R::kScales) at[lane][1] = ok ? scales_at(p.c, page, row) : 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return (uint64_t)__ballot(ok);
  };
  heads(0);   // (in front of what waits for the length)
  if (base < held) {
    R r;
    uint64_t there = place(base);
    if (there) W::load_k(r, p, at, hoff, shoff);
    while (true) {
      const int64_t tok = base + lane;
      const bool mine = lane < kTile && tok < held;
      const float old = mine ? from[tok] : 0.0f;
      float sum[R::kSub];
#pragma unroll
      for (int t = 0; t < R::kSub; ++t) sum[t] = 0.0f;
      const uint64_t now = there;
      auto add = [&](const f32x4 (&st)[R::kSub]) {
#pragma unroll
        for (int t = 0; t < R::kSub; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float s = st[t][j], scale = p.scale;
            if constexpr (CAP) {
              s = capped<false>(p, s);
              scale = 1.0f;
            }
            const float w = __builtin_amdgcn_exp2f(fmaf(s, scale, -lse[j]) - rest[j]);
            sum[t] += none[j] ? 0.0f : w;
          }
      };
      f32x4 st[R::kSub];
      for (int group = 1; group < p.q_groups; ++group) {   // (more than 16 heads: the last groups first)
        if (now == 0) break;
        heads(group);
        w.template scores<true>(r, p, sc, st);
        add(st);
      }
      if (now != 0) {
        if (p.q_groups > 1) heads(0);
        w.template scores<true>(r, p, sc, st);
      }
      base += step;
      there = 0;
      if (base < held) {
        there = place(base);
        if (there) W::load_k(r, p, at, hoff, shoff);
      }
      float x = 0.0f;
      if (now != 0) {
        add(st);
#pragma unroll
        for (int t = 0; t < R::kSub; ++t) {
          const float s = across_sum(sum[t]);
          x = g == t ? s : x;
        }
        x = now >> lane & 1 ? x : 0.0f;
      }
      if (mine) to[tok] = fmaf(m.decay, old, x);
      if (base >= held) break;
    }
  }

  // The entries behind the sequence, all threads over the row and 4 each, those without tiles first. (32 sequences of up
  // to 16384 tokens, 62516 in all, in rows of 16384, 64/8 heads: 49 us, 63 with tiles of these as of the others.)
  if (m.out == m.mass) return;
  typedef f32x4 f32x4_any __attribute__((aligned(4)));
  const int64_t each = (int64_t)4 * kThreads * m.splits;
  for (int64_t t = held + each - 4 - 4 * (int64_t)(split * kThreads + threadIdx.x); t < m.tokens; t += each) {
    if (t + 4 <= m.tokens)
      *reinterpret_cast<f32x4_any*>(to + t) = *reinterpret_cast<const f32x4_any*>(from + t);
    else
      for (int64_t i = t; i < m.tokens; ++i) to[i] = from[i];
  }
}

template <int DT, int ST, int DP>
void mass_by_cap(const MassParams& p, hipStream_t s) {
  const int grid = p.a.batch * p.a.c.kv_heads * p.splits;
  if (p.a.cap != 0.0f)
    mass_kernel<DT, ST, DP, true><<<grid, kThreads, 0, s>>>(p);
  else
    mass_kernel<DT, ST, DP, false><<<grid, kThreads, 0, s>>>(p);
}

template <int DT, int ST>
void mass_by_width(const MassParams& p, hipStream_t s) {
  const int dp = attn_padded(p.a.c.head_dim);
  if (dp == 64)
    mass_by_cap<DT, ST, 64>(p, s);
  else if (dp == 128)
    mass_by_cap<DT, ST, 128>(p, s);
  else
    mass_by_cap<DT, ST, 256>(p, s);
}

template <int DT>
void mass_by_storage(const MassParams& p, int storage, hipStream_t s) {
  if (storage == AG_KV_16BIT)
    mass_by_width<DT, AG_KV_16BIT>(p, s);
  else if (storage == AG_KV_MXFP8)
    mass_by_width<DT, AG_KV_MXFP8>(p, s);
  else
    mass_by_width<DT, AG_KV_MXFP4>(p, s);
}

}  // namespace

hipError_t launch_mass(const MassParams& p, int dtype, int storage, hipStream_t s) {
  if (dtype == AGMM_F16)
    mass_by_storage<AGMM_F16>(p, storage, s);
  else
    mass_by_storage<AGMM_BF16>(p, storage, s);
  return hipGetLastError();
}

}  // namespace agmm
