// The kernels of agmm_prefix_kernel.h for fp16, and the joining of what they leave.
#include "agmm_prefix_kernel.h"

namespace agmm {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// A thread joins 4 elements of one row: the prefix's pieces, in their order, and the own tokens' average. The two
// come in over their own sums: what joins them is an average again, so finite values cannot leave the type's
// range on the way.
//
// What takes the time are loads that wait for loads, so all that can be is loaded at once: the lengths, the
// own part and the group's plan; then the pieces, 16 at a time.
template <int DT, int DP>
__global__ __launch_bounds__(kThreads) void join_kernel(PrefixParams p, FastDiv d4, FastDiv heads, FastDiv group) {
  const AttnParams& a = p.own;
  const PrefixView& x = a.prefix;
  const uint32_t i = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  const uint32_t at = i / d4;
  const int e = 4 * (int)(i - at * d4.d);
  const uint32_t b = at / heads;
  if (b >= (uint32_t)a.batch) return;
  const uint32_t head = at - b * heads.d, kv = head / group;
  const int64_t own_row = (int64_t)b * a.q_heads + head;
  const int32_t len = a.lens[b];
  f32x4 mine = *reinterpret_cast<const f32x4*>(x.own + own_row * DP + e);
  float own_m = x.own_stats[2 * own_row], own_l = x.own_stats[2 * own_row + 1];
  // the last group that begins at b or before
  uint32_t lo = 0, hi = x.groups;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    (x.info[mid].first <= (int32_t)b ? lo : hi) = mid;
  }
  const u32x4 g0 = *reinterpret_cast<const u32x4*>(&x.info[lo]);
  const u32x4 g1 = *(reinterpret_cast<const u32x4*>(&x.info[lo]) + 1);
  const PrefixGroup g = {(int32_t)g0[0], (int32_t)g0[1], g0[2], g0[3], g1[0], g1[1], g1[2], 0};
  const uint32_t r = (b - g.first) * a.group + (head - kv * a.group);
  const uint32_t strip = kv * g.row_tiles + r / kPrefixRows, row = r % kPrefixRows;
  const uint32_t start = g.tile0 + strip * g.tiles, begin = start / g.quota;
  const bool shares = (int32_t)b >= g.first && (int32_t)b < g.end && g.tiles != 0;
  const uint32_t pieces = shares ? (start + g.tiles - 1) / g.quota - begin + 1 : 0;
  const int64_t slot = begin + g.strip0 + strip;
  const float* const sums = x.sums + slot * (kPrefixRows * DP) + prefix_at(row, e);
  const float* const stats = x.stats + (slot * kPrefixRows + row) * 2;
  constexpr int kIn = 16;
  f32x4 o = {0, 0, 0, 0};
  float m = -INFINITY, l = 0.0f;
#pragma unroll 1
  for (uint32_t c = 0; c < pieces; c += kIn) {
    f32x4 y[kIn];
    f32x2 t[kIn];
#pragma unroll
    for (int k = 0; k < kIn; ++k) {  // (past the last: the last again, not counted below)
      const uint32_t s = min(c + k, pieces - 1);
      t[k] = *reinterpret_cast<const f32x2*>(stats + (uint64_t)s * (2 * kPrefixRows));
      y[k] = *reinterpret_cast<const f32x4*>(sums + (uint64_t)s * (kPrefixRows * DP));
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kIn; ++k) top = fmaxf(top, t[k][0]);
    const float f = weight(m, top, 1.0f);
    l *= f;
#pragma unroll
    for (int w = 0; w < 4; ++w) o[w] *= f;
#pragma unroll
    for (int k = 0; k < kIn; ++k) {
      const bool in = c + k < pieces;
      const float f = in ? weight(t[k][0], top, 1.0f) : 0.0f;
      l = fmaf(f, in ? t[k][1] : 0.0f, l);
#pragma unroll
      for (int w = 0; w < 4; ++w) o[w] = fmaf(f, in ? y[k][w] : 0.0f, o[w]);
    }
    m = top;
  }
  if (tiles_of(a, len) == 0) {   // nothing was left there
    mine = f32x4{0, 0, 0, 0};
    own_m = -INFINITY;
    own_l = 0.0f;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  // (the prefix's reference is in base 2, the other in unit()s of it)
  const float u = unit(a), top = fmaxf(own_m * u, m);
  const float ours = own_m == -INFINITY ? own_l : own_l * __builtin_amdgcn_exp2f(fmaf(own_m, u, -top));
  const float theirs = l * weight(m, top, 1.0f);
  const float all = ours + theirs;
  const float fo = all == 0.0f ? 0.0f : ours / all, fp = all == 0.0f ? 0.0f : theirs / all;
  float y[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) y[w] = fmaf(mine[w], fo, o[w] * inv * fp);
  typedef u32x2 u32x2_any __attribute__((aligned(2)));
  *reinterpret_cast<u32x2_any*>(a.out + (int64_t)b * a.o_batch + (int64_t)head * a.o_head + e) =
      u32x2{T16<DT>::pack(y[0], y[1]), T16<DT>::pack(y[2], y[3])};
  if (e == 0 && a.lse)
    a.lse[own_row] = all == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(all)) * 0.69314718055994531f;
}

template <int DT>
void join_by_width(const PrefixParams& p, hipStream_t s) {
  const AttnParams& a = p.own;
  const FastDiv d4 = fast_div((uint32_t)a.c.head_dim / 4), heads = fast_div((uint32_t)a.q_heads),
                group = fast_div((uint32_t)a.group);
  const uint32_t threads = (uint32_t)a.batch * a.q_heads * d4.d, grid = (threads + kThreads - 1) / kThreads;
  const int dp = attn_padded(a.c.head_dim);
  if (dp == 64)
    join_kernel<DT, 64><<<grid, kThreads, 0, s>>>(p, d4, heads, group);
  else if (dp == 128)
    join_kernel<DT, 128><<<grid, kThreads, 0, s>>>(p, d4, heads, group);
  else
    join_kernel<DT, 256><<<grid, kThreads, 0, s>>>(p, d4, heads, group);
}

}  // namespace

hipError_t launch_prefix_f16(const PrefixParams& p, int storage, int grid, hipStream_t s) {
  return prefix_by_storage<AGMM_F16>(p, storage, grid, s);
}

hipError_t launch_prefix_join(const PrefixParams& p, int dtype, hipStream_t s) {
  if (dtype == AGMM_F16)
    join_by_width<AGMM_F16>(p, s);
  else
    join_by_width<AGMM_BF16>(p, s);
  return hipGetLastError();
}

}  // namespace agmm
