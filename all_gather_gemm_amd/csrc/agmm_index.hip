// gfx950 kernels of the page index, of choosing what is kept, and of moving rows (agmm_long.h).
//
// All of them read a stream of bytes and compute little on each, so many pages or tokens are bound by memory
// bandwidth and few by the chain of a launch, the length, the page and its rows.
//
// Measured, warm: entries of a prompt of 16384 tokens (8 kv heads of 128, bf16, pages of 16) 7.8 us, 4.6 TB/s; scores of
// 32 sequences of up to 32768 tokens, 8 kv heads: 12 us, of one of 131072 tokens, one kv head, pages of 64: 4.6; choosing
// from 2048 pages 6.4 us, from 16384 tokens (one workgroup each, 256 of them) 26; moving 4096 rows of 32 sequences and 8
// kv heads 216 us, 4.9 TB/s of reads and writes (a copy of 4 GiB runs at 4.7; four rows to a thread: 220).
#include "agmm_attn_kernel.h"
#include "agmm_long_internal.h"

namespace agmm {
namespace {

// ---------------------------------------------------------------- the index's entries

template <int DT>
__device__ inline float value_of(uint32_t w, int half) {
  return half ? T16<DT>::hi(w) : T16<DT>::lo(w);
}

// Sum of whole numbers, or another combination, over the N lanes (8, 16 or 32) that work on one page.
template <int N, class F>
__device__ inline uint32_t over_lanes(uint32_t x, F f) {
  x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xf, 0xf, true));   // pairs
  x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xf, 0xf, true));   // fours
  x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xf, 0xf, true));  // eights, mirrored
  if constexpr (N >= 16) x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xf, 0xf, true));
  if constexpr (N >= 32) x = f(x, (uint32_t)__shfl_xor((int)x, 16));
  return x;
}
__device__ inline uint32_t as_u(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ inline float as_f(uint32_t x) { return __builtin_bit_cast(float, x); }
template <int N>
__device__ inline float max_over_lanes(float x) {
  return as_f(over_lanes<N>(as_u(x), [](uint32_t a, uint32_t b) { return as_u(fmaxf(as_f(a), as_f(b))); }));
}

// 127 + the least e from -126 on with most <= 127 * 2^e, for most >= 0 and finite. With most = x 2^k, 1 <= x
// < 2, 127 * 2^(k - 6) is enough for x <= 127 / 64.
__device__ inline uint32_t least_exponent(float most) {
  const uint32_t w = as_u(most);
  const int e = (int)(w >> 23) - 6 + ((w & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return (uint32_t)max(e, 1);
}
// 2^(127 - s), that is 1 / 2^e, exactly: s is 1..248.
__device__ inline float one_over(uint32_t s) { return as_f((254u - s) << 23); }

// Pairs of 16-bit floats as pairs of 16-bit whole numbers of the same order, and back. What is past infinity is NaN.
typedef short s16x2 __attribute__((ext_vector_type(2)));
__device__ inline s16x2 ordered(uint32_t w) {
  const s16x2 x = __builtin_bit_cast(s16x2, w);
  return x ^ ((x >> 15) & (short)0x7fff);
}
__device__ inline s16x2 larger(s16x2 a, s16x2 b) { return __builtin_elementwise_max(a, b); }
__device__ inline s16x2 smaller(s16x2 a, s16x2 b) { return __builtin_elementwise_min(a, b); }

// Pages of sequence b whose entries are made: [first, end), and the tokens of the last.
struct Renewed {
  int32_t first, end, used;
};
__device__ inline Renewed renewed(const IndexParams& p, int64_t b) {
  const int32_t ps = (int32_t)p.c.page_size.d;
  const int32_t len = min(max(p.lens[b], 0), p.pages * ps), start = p.starts ? max(p.starts[b], 0) : 0;
  if (start >= len) return Renewed{0, 0, 0};
  const int32_t last = (int32_t)((uint32_t)(len - 1) / p.c.page_size);
  return Renewed{(int32_t)((uint32_t)start / p.c.page_size), last + 1, len - last * ps};
}

struct HeldShared {
  int32_t first[kThreads], last[kThreads];
  uint64_t some[kThreads / 64];   // threads whose sequence has full pages
  int32_t found;
};

// Whether any place of the call holds this page with more than `used` tokens, for the whole workgroup. Pages in front
// of a sequence's last are full, so the last ones are compared by their tokens and the others by their number alone:
// a thread has one sequence's last page, and all of them go through the full ones of one sequence after the other.
__device__ inline bool held_longer(const IndexParams& p, HeldShared& sh, int32_t page, int32_t used) {
  constexpr int kUnroll = 8;
  const int tid = threadIdx.x;
  bool longer = false;
  if (tid == 0) sh.found = 0;
  for (int32_t base = 0; base < (int32_t)p.batch.d; base += kThreads) {
    const int32_t b = base + tid;
    Renewed r = {0, 0, 0};
    if (b < (int32_t)p.batch.d) r = renewed(p, b);
    if (base) __syncthreads();
    if (r.used > used) longer = longer || p.table[b * p.table_row + r.end - 1] == page;
    sh.first[tid] = r.first;
    sh.last[tid] = r.end - 1;
    const uint64_t some = __ballot(r.first < r.end - 1);
    if ((tid & 63) == 0) sh.some[tid >> 6] = some;
    __syncthreads();
    for (int w = 0; w < kThreads / 64; ++w)
      for (uint64_t left = sh.some[w]; left; left &= left - 1) {
        const int s = 64 * w + __builtin_ctzll(left);
        const int32_t* table = p.table + (int64_t)(base + s) * p.table_row;
        const int32_t last = sh.last[s];
        for (int32_t j = sh.first[s] + tid; j < last; j += kUnroll * kThreads) {
          int32_t x[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) x[u] = table[min(j + u * kThreads, last - 1)];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) longer = longer || x[u] == page;
        }
      }
  }
  if (longer) sh.found = 1;
  __syncthreads();
  return sh.found != 0;
}

// A page may be in several places of the call's tables. Where it is full, all of them make the same entry; where a
// sequence ends in it, its workgroup looks whether another place has more of its tokens, and leaves the entry to that
// (those with as many make the same bytes). That takes a step of one sequence from 2.7 to 3.4 us and of 4096 from 31
// to 39 (1000 tokens, 8 kv heads of 128, bf16), 32 prompts of 8001 tokens from 124 to 134.
//
// A wave makes one entry at a time: LC = padded dim / 8 lanes on 8 elements each, 64 / LC rows at once. Largest and
// least are found among 16-bit whole numbers, two at once; ~x turns the order round, so both are maxima. The rows are
// put together by exchanges of registers that leave the largest to the lower half of the wave and the least to the
// upper, and (LC < 32) half of the elements to every other 16 lanes: each lane then has kLeft words of the result.
template <int DT, int ST, int LC>
__global__ __launch_bounds__(kThreads) void update_kernel(IndexParams p) {
  constexpr int kRows = 64 / LC, kUnroll = 4, kLeft = LC == 32 ? 4 : 2;
  const int lane = threadIdx.x & 63, c = lane % LC, r0 = lane / LC;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // (all sequences' first workgroups come first: the others have nothing in a step)
  const uint32_t heads = p.heads.d, split = blockIdx.x / p.batch, b = blockIdx.x - split * p.batch.d;
  const int32_t ps = (int32_t)p.c.page_size.d, hd = p.c.head_dim;
  const Renewed mine = renewed(p, b);
  const uint32_t first = (uint32_t)mine.first, end = (uint32_t)mine.end;
  if (first >= end) return;
  const bool in = 8 * c < hd;
  const int e = in ? 8 * c : 0;
  const int bytes = ST == AG_KV_16BIT ? 2 * e : ST == AG_KV_MXFP8 ? e : e / 2;
  constexpr int kWords = ST == AG_KV_16BIT ? 4 : ST == AG_KV_MXFP8 ? 2 : 1;
  const bool upper = lane >= 32;                                  // has the least
  const int part = LC == 32 ? 0 : (lane >> 4) & 1;                // and which elements of its 8
  const int32_t* table = p.table + (int64_t)b * p.table_row;
  // entries of one sequence: heads of a page, page after page, 4 a workgroup at once
  const uint32_t begin = split * 4 + wave, step = p.step.d, wgs = step / 4;
  const uint32_t step_j = step / p.heads, step_h = step - step_j * heads;
  uint32_t j = begin / p.heads, kv = begin - j * heads;
  j += first;
  int32_t page = j < end ? table[j] : -1;
  __shared__ HeldShared sh;
  uint32_t left = end;   // the page that is left to another place
  if (mine.used < ps) {
    // its entries begin at number (end - 1 - first) * heads, of which only the rest over `step` counts
    const auto rest = [&](uint32_t x) { return x - x / p.step * step; };
    const uint32_t at = rest(rest(end - 1 - first) * rest(heads));
    if ((split >= at / 4 ? split - at / 4 : split + wgs - at / 4) <= (at % 4 + heads - 1) / 4) {
      if (held_longer(p, sh, table[end - 1], mine.used)) left = end - 1;
    }
  }
  for (uint32_t next_j, next_kv; j < end; j = next_j, kv = next_kv) {
    const int32_t now = page;
    next_j = j + step_j;
    next_kv = kv + step_h;
    if (next_kv >= heads) {
      next_kv -= heads;
      ++next_j;
    }
    page = next_j < end ? table[next_j] : -1;
    if ((uint32_t)now >= (uint32_t)p.num_pages || j == left) continue;
    const int used = j + 1 == end ? mine.used : ps;
    s16x2 hi[4], lo[4];   // lo: the largest of ~x
#pragma unroll
    for (int k = 0; k < 4; ++k) hi[k] = lo[k] = s16x2{-0x8000, -0x8000};
    for (int r = r0; r - r0 < used; r += kUnroll * kRows) {
      uint32_t w[kUnroll][kWords], s[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {   // (past the last row: the last again)
        const uint32_t row = (uint32_t)min(r + u * kRows, used - 1);
        load_words<kWords>(w[u], p.c.k + kv * p.c.head + row_at(p.c, now, row) + bytes);
        if (ST != AG_KV_16BIT)
          s[u] = *(const uint8_t*)(p.c.ks + kv * p.c.s_head + scales_at(p.c, now, row) + e / 32);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        u32x4 x;
        if constexpr (ST == AG_KV_16BIT)
          x = u32x4{w[u][0], w[u][1], w[u][2], w[u][3]};
        else if constexpr (ST == AG_KV_MXFP8)
          x = from_fp8x8<DT>(w[u][0], w[u][1], scale_of(s[u]));
        else
          x = from_fp4x8<DT>(w[u][0], scale_of(s[u]));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const s16x2 o = ordered(x[k]);
          hi[k] = larger(hi[k], o);
          lo[k] = larger(lo[k], ~o);
        }
      }
    }
    if constexpr (LC == 8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // lanes 8 apart
        const int x = __builtin_bit_cast(int, hi[k]), y = __builtin_bit_cast(int, lo[k]);
        hi[k] = larger(hi[k], __builtin_bit_cast(s16x2, __builtin_amdgcn_update_dpp(0, x, 0x128, 0xf, 0xf, true)));
        lo[k] = larger(lo[k], __builtin_bit_cast(s16x2, __builtin_amdgcn_update_dpp(0, y, 0x128, 0xf, 0xf, true)));
      }
    }
    s16x2 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const auto x = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, hi[k]),
                                                      __builtin_bit_cast(uint32_t, lo[k]), false, false);
      v[k] = larger(__builtin_bit_cast(s16x2, (uint32_t)x[0]), __builtin_bit_cast(s16x2, (uint32_t)x[1]));
    }
    if constexpr (LC < 32) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const auto x = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v[k]),
                                                        __builtin_bit_cast(uint32_t, v[k + 2]), false, false);
        v[k] = larger(__builtin_bit_cast(s16x2, (uint32_t)x[0]), __builtin_bit_cast(s16x2, (uint32_t)x[1]));
      }
    }
    float f[2 * kLeft], most = 0.0f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kLeft; ++i) {
      const uint32_t w = __builtin_bit_cast(uint32_t, ordered(__builtin_bit_cast(uint32_t, upper ? ~v[i] : v[i])));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x = value_of<DT>(w, h);
        odd = odd || !(fabsf(x) < INFINITY);
        most = fmaxf(most, fabsf(x));
        f[2 * i + h] = upper ? -x : x;   // (rounded up, either)
      }
    }
    const bool bad = __ballot(odd && in) != 0;
    most = max_over_lanes<16>(in ? most : 0.0f);
    const uint32_t s = bad ? 255u : least_exponent(across_max(most));
    const float unit = bad ? 0.0f : one_over(s);
    uint32_t code[kLeft / 2];
#pragma unroll
    for (int i = 0; i < kLeft / 2; ++i) code[i] = 0;
#pragma unroll
    for (int k = 0; k < 2 * kLeft; ++k) {
      // (a product that underflows is still above 0)
      const int h = bad ? 0 : max((int)ceilf(f[k] * unit), f[k] > 0.0f ? 1 : -128);
      code[k / 4] |= (uint32_t)((upper ? -h : h) & 255) << (8 * (k % 4));
    }
    const int64_t entry = (int64_t)now * p.c.kv_heads + kv;
    int8_t* to = p.codes + entry * 2 * hd + (upper ? hd : 0) + e + 4 * part;
    if (in && (LC != 8 || !(lane & 8))) {
      if constexpr (LC == 32)
        *reinterpret_cast<u32x2*>(to) = u32x2{code[0], code[kLeft / 2 - 1]};
      else
        *reinterpret_cast<uint32_t*>(to) = code[0];
    }
    if (lane == 0) p.scales[entry] = (uint8_t)s;
  }
}

// ---------------------------------------------------------------- scores

// Floats as whole numbers of the same order, from 1 on. -0 is 0; NaN, and what comes before all others, is
// kMost; 0 is left for what cannot be chosen and kForced for what has to be.
constexpr uint32_t kMost = 0xfffffffeu, kForced = 0xffffffffu;
__device__ inline uint32_t order_key(float x) {
  if (!(x == x)) return kMost;
  const uint32_t w = as_u(x + 0.0f);
  return w >> 31 ? ~w : w | 0x80000000u;
}

template <int LC>
struct alignas(16) ScoreShared {
  uint8_t code[2][16 * LC];   // the sums' low and high parts
  int sum[16 * LC];           // of the elements' positive codes, and of the negative ones
  float most[kThreads / 64];
};

// What a page's codes are multiplied by, for one sequence and kv head: the sums over the q heads of the positive
// codes of each element, and of the negative ones, in two parts of 8 bits, 128 x + y, for v_dot4_i32_i8 (they are
// within 127 * 128). The workgroup makes them together, a thread some heads of one element; a lane gets its 16.
template <int DT, int LC>
__device__ inline void weights_of(const IndexParams& p, int64_t b, int kv, ScoreShared<LC>& sh,
                                  u32x4& w0, u32x4& w1) {
  constexpr int kDim = 8 * LC, kPer = kThreads / kDim, kIn = 4;
  const int tid = threadIdx.x, e = tid % kDim, part = tid / kDim, hd = p.c.head_dim;
  const uint16_t* q = p.q + b * p.q_batch + (int64_t)kv * p.group * p.q_head + (e < hd ? e : 0);
  uint16_t x[kIn];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kIn; ++i) x[i] = q[(int64_t)min(h0 + i * kPer, p.group - 1) * p.q_head];
  };
  auto value = [&](int h, int i) {
    const float f = value_of<DT>(x[i], 0);
    return fabsf(f) < INFINITY && h < p.group && e < hd ? f : 0.0f;
  };
  float most = 0.0f;
  for (int h0 = part; h0 < p.group; h0 += kIn * kPer) {
    load(h0);
#pragma unroll
    for (int i = 0; i < kIn; ++i) most = fmaxf(most, fabsf(value(h0 + i * kPer, i)));
  }
  most = max_over_lanes<32>(most);
  most = fmaxf(most, __shfl_xor(most, 32));
  for (int i = tid; i < 16 * LC; i += kThreads) sh.sum[i] = 0;
  if ((tid & 63) == 0) sh.most[tid >> 6] = most;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) most = fmaxf(most, sh.most[i]);
  const float unit = one_over(least_exponent(most));
  int up = 0, down = 0;
  for (int h0 = part; h0 < p.group; h0 += kIn * kPer) {
    if (p.group > kIn * kPer) load(h0);
#pragma unroll
    for (int i = 0; i < kIn; ++i) {
      const int code = (int)rintf(value(h0 + i * kPer, i) * unit);
      up += max(code, 0);
      down += min(code, 0);
    }
  }
  if (e < hd) {
    atomicAdd(&sh.sum[e], up);
    atomicAdd(&sh.sum[hd + e], down);
  }
  __syncthreads();
  for (int i = tid; i < 16 * LC; i += kThreads) {   // (0 past 2 * hd)
    const int s = sh.sum[i], hi = s / 128;
    sh.code[0][i] = (uint8_t)(s - 128 * hi);
    sh.code[1][i] = (uint8_t)hi;
  }
  __syncthreads();
  const int c = (tid & 63) % LC;   // chunk: 16 of the 2 * hd codes
  w0 = *reinterpret_cast<const u32x4*>(sh.code[0] + 16 * c);
  w1 = *reinterpret_cast<const u32x4*>(sh.code[1] + 16 * c);
}

// The keys of pages j0, j0 + 1 .. and so on in steps of `step` for one sequence and kv head, LC lanes to a page:
// put(page, key).
template <int DT, int LC, class F>
__device__ inline void score(const IndexParams& p, int64_t b, int kv, ScoreShared<LC>& sh, int32_t j0, int32_t step,
                             int32_t end, F put) {
  constexpr int kUnroll = 4;
  const int lane = threadIdx.x & 63, c = lane % LC, r0 = lane / LC;
  const int32_t hd = p.c.head_dim;
  u32x4 w0, w1;
  weights_of<DT, LC>(p, b, kv, sh, w0, w1);
  const bool in = c < hd / 8;
  const int32_t* table = p.table + b * p.table_row;
  for (; j0 < end; j0 += kUnroll * step) {
    int32_t page[kUnroll];
    u32x4 x[kUnroll];
    uint32_t s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t j = j0 + u * step + r0;
      page[u] = j < end ? table[j] : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const bool ok = (uint32_t)page[u] < (uint32_t)p.num_pages;
      const int64_t entry = (int64_t)(ok ? page[u] : 0) * p.c.kv_heads + kv;
      x[u] = *reinterpret_cast<const u32x4*>(p.codes + entry * 2 * hd + (in ? 16 * c : 0));
      s[u] = p.scales[entry];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      int t0 = 0, t1 = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t0 = __builtin_amdgcn_sdot4((int)x[u][i], (int)w0[i], t0, false);
        t1 = __builtin_amdgcn_sdot4((int)x[u][i], (int)w1[i], t1, false);
      }
      const int total =
          (int)over_lanes<LC>((uint32_t)(128 * t1 + t0), [](uint32_t a, uint32_t b) { return a + b; });
      const int32_t j = j0 + u * step + r0;
      if (c == 0 && j < end) {
        const bool ok = (uint32_t)page[u] < (uint32_t)p.num_pages;
        const uint32_t key = s[u] == 255u ? kMost : order_key((float)total * as_f(s[u] << 23));
        put(j, ok ? key : 0u);
      }
    }
  }
}

// Pages with tokens of sequence b.
__device__ inline int32_t pages_of(const IndexParams& p, int64_t b) {
  const int32_t ps = (int32_t)p.c.page_size.d;
  const int64_t len = min((int64_t)max(p.lens[b], 0), (int64_t)p.pages * ps);
  return (int32_t)((len + ps - 1) / ps);
}

template <int DT, int LC>
__global__ __launch_bounds__(kThreads) void score_kernel(IndexParams p) {
  constexpr int kPages = 64 / LC;
  __shared__ ScoreShared<LC> sh;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const uint32_t bh = blockIdx.x / (uint32_t)p.splits, split = blockIdx.x - bh * (uint32_t)p.splits;
  const int64_t b = bh / (uint32_t)p.c.kv_heads;
  const int kv = (int)(bh - (uint32_t)b * p.c.kv_heads);
  const int32_t end = pages_of(p, b);
  if ((int32_t)split * 4 * kPages >= end) return;   // (nothing for the whole workgroup)
  uint32_t* keys = p.keys + (int64_t)bh * ((p.pages + 3) & ~3);
  score<DT, LC>(p, b, kv, sh, (int32_t)(split * 4 + wave) * kPages, (int32_t)p.splits * 4 * kPages, end,
                [&](int32_t j, uint32_t key) { keys[j] = key; });
}

// ---------------------------------------------------------------- choosing

template <int T>
struct ChooseShared {
  uint32_t hist[2048];
  uint32_t waves[T / 64];
  uint32_t bin, left, held;
};

// Sum over the workgroup's threads in front of this one, and over all.
template <int T>
__device__ inline uint32_t block_scan(uint32_t x, uint32_t* waves, uint32_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t s = wave_scan(x);
  if (lane == 63) waves[wave] = s;
  __syncthreads();
  uint32_t before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < T / 64; ++i) {
    const uint32_t w = waves[i];
    before += i < wave ? w : 0;
    total += w;
  }
  __syncthreads();
  all = total;
  return before + s - x;
}

// One workgroup chooses for one sequence and head: the keys of all items, the `budget`-th largest found by
// histograms of 11, 11 and 10 bits (as many as it takes), then the chosen items written in order. A thread has K
// consecutive items, in registers where the workgroup has all of them at once.
//
// One workgroup's time is what counts, and of that the instructions for each item. What is past T * K items is read again
// for every histogram and for writing: 8 heads of 16384, 32768 and 131072 tokens take 14, 25 and 91 us, 256 of 16384 and 16400
// 20 and 49 (in graphs).
// keys: in global memory or, K = 1, in LDS.
template <int T, int K, bool TOKENS>
__device__ inline void choose_items(const ChooseParams& p, ChooseShared<T>& sh, const uint32_t* keys) {
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x / (uint32_t)p.heads;
  const int head = (int)(blockIdx.x - (uint32_t)b * p.heads);
  const int32_t ps = (int32_t)p.page_size.d;
  const int64_t len = min((int64_t)max(p.lens[b], 0), (int64_t)p.pages * ps);
  const int32_t n = TOKENS ? (int32_t)min(len, (int64_t)p.items) : (int32_t)((len + ps - 1) / ps);
  const int32_t* table = p.table + b * p.table_row;
  const float* mass = TOKENS ? p.mass + b * p.mass_batch + head * p.mass_head : nullptr;
  auto there = [&](int32_t page) { return (uint32_t)page < (uint32_t)p.num_pages; };
  constexpr int kBins = 2048 / T;

  // a thread's keys, and what it writes with the chosen ones: tokens' masses or the pages' numbers
  uint32_t k[K], with[K];
  auto load = [&](int32_t base) {
    typedef u32x4 u32x4_four __attribute__((aligned(4)));
    const int32_t i0 = base + tid * K;
    const uint32_t* from = TOKENS ? reinterpret_cast<const uint32_t*>(mass) : reinterpret_cast<const uint32_t*>(table);
    if (K > 1 && i0 + K <= n) {
#pragma unroll
      for (int i = 0; i < K / 4 * 4; i += 4) {
        const u32x4 x = *reinterpret_cast<const u32x4_four*>(from + i0 + i);
#pragma unroll
        for (int u = 0; u < 4; ++u) with[i + u] = x[u];
      }
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i) with[i] = i0 + i < n ? from[i0 + i] : 0u;
    }
    if constexpr (TOKENS) {
      if (ps >= K) {   // a thread's tokens are in two pages at most
        const uint32_t j = (uint32_t)min(i0, n - 1) / p.page_size;   // (n > 0)
        const int32_t left = (int32_t)(j + 1) * ps - i0;   // tokens of the first
        const int32_t p0 = table[j], p1 = table[min((int32_t)j + 1, p.pages - 1)];
        const bool ok0 = there(p0), ok1 = there(p1);
#pragma unroll
        for (int i = 0; i < K; ++i)
          k[i] = i0 + i < n && (i < left ? ok0 : ok1) ? order_key(as_f(with[i])) : 0u;
      } else {
#pragma unroll
        for (int i = 0; i < K; ++i) {
          const int32_t page = table[(uint32_t)min(i0 + i, n - 1) / p.page_size];
          k[i] = i0 + i < n && there(page) ? order_key(as_f(with[i])) : 0u;
        }
      }
    } else if constexpr (K == 1) {
      k[0] = i0 < n ? keys[i0] : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < K; i += 4) {   // (the keys' rows are filled up to fours)
        u32x4 x = {0, 0, 0, 0};
        if (i0 + i < n) x = *reinterpret_cast<const u32x4*>(keys + i0 + i);
#pragma unroll
        for (int u = 0; u < 4; ++u) k[i + u] = i0 + i + u < n ? x[u] : 0;
      }
    }
    if (i0 < p.sink || i0 + K > n - p.recent)
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (k[i] != 0 && (i0 + i < p.sink || i0 + i >= n - p.recent)) k[i] = kForced;
  };
  const bool once = n <= T * K;
#pragma unroll
  for (int i = 0; i < kBins; ++i) sh.hist[tid + i * T] = 0;
  if (once && n > 0) load(0);   // (nothing may be read of a sequence without a token)
  __syncthreads();
  // Chosen: keys above `least`, and the first `ties` that equal it. What cannot be chosen, key 0, has bin 0 of the
  // first histogram to itself (the least other key, minus infinity's, is in bin 3).
  uint32_t least = 0, ties = 0, keep = (uint32_t)p.budget, left = 0;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int32_t base = 0; base < n; base += T * K) {
      if (!once) load(base);
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (pass == 0 || (k[i] ^ least) >> (shift + bits) == 0)
          atomicAdd(&sh.hist[k[i] >> shift & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    const int top = (1 << bits) - 1;
    uint32_t h[kBins], mine = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kBins; ++i) {   // from the largest down
      const int bin = top - (tid * kBins + i);
      h[i] = bin >= 0 && (pass != 0 || bin > 0) ? sh.hist[bin] : 0;
      mine += h[i];
    }
    uint32_t before = block_scan<T>(mine, sh.waves, all);
    if (pass == 0) {   // all: what can be chosen
      if (all <= keep) {
        keep = all;
        break;
      }
      left = keep;
    }
#pragma unroll
    for (int i = 0; i < kBins; ++i) {
      if (before < left && left <= before + h[i]) {
        sh.bin = (uint32_t)(top - (tid * kBins + i));
        sh.left = left - before;
        sh.held = h[i];
      }
      before += h[i];
      sh.hist[tid + i * T] = 0;   // (block_scan's barriers are behind every read)
    }
    __syncthreads();
    least |= sh.bin << shift;
    left = sh.left;
    const bool whole = left == sh.held;
    __syncthreads();
    if (whole) {   // all of the bin's
      least -= 1;   // (no bin is 0: keys above this are those of the bin and more)
      break;
    }
    if (pass == 2) ties = left;
  }
  int32_t* out = p.out + (int64_t)blockIdx.x * p.budget;
  float* out_mass = TOKENS && p.out_mass ? p.out_mass + (int64_t)blockIdx.x * p.budget : nullptr;
  uint32_t above = 0, equal = 0;   // so far
  for (int32_t base = 0; base < n; base += T * K) {
    if (!once) load(base);
    uint32_t mine = 0, all = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) mine += (k[i] > least ? 1u : 0u) + (k[i] == least ? 0x10000u : 0u);
    const uint32_t before = block_scan<T>(mine, sh.waves, all);
    uint32_t a = above + (before & 0xffffu), e = equal + (before >> 16);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const bool more = k[i] > least, same = k[i] == least;
      if (more || (same && e < ties)) {
        const int32_t item = base + tid * K + i;
        const uint32_t at = a + min(e, ties);
        out[at] = TOKENS ? item : (int32_t)with[i];
        if (TOKENS && out_mass) out_mass[at] = as_f(with[i]);
      }
      a += more ? 1 : 0;
      e += same ? 1 : 0;
    }
    above += all & 0xffffu;
    equal += all >> 16;
  }
  for (uint32_t i = keep + tid; i < (uint32_t)p.budget; i += T) {
    out[i] = -1;
    if (TOKENS && out_mass) out_mass[i] = 0.0f;
  }
  if (head == 0 && tid == 0) {
    if (TOKENS) {
      p.out_lens[b] = (int32_t)keep;
    } else {
      // all pages are full but the sequence's last, which is chosen if it is there
      const bool last = n > 0 && there(table[n - 1]);
      p.out_lens[b] = (int32_t)((int64_t)keep * ps - (last ? (int64_t)n * ps - len : 0));
    }
  }
}

template <int T, int K, bool TOKENS>
__global__ __launch_bounds__(T) void choose_kernel(ChooseParams p) {
  __shared__ ChooseShared<T> sh;
  choose_items<T, K, TOKENS>(p, sh, TOKENS ? nullptr : p.keys + (int64_t)blockIdx.x * p.key_stride);
}

// Scores and choice in one launch, for tables of up to kFew pages: the keys stay in LDS.
template <int DT, int LC>
__global__ __launch_bounds__(kThreads) void select_kernel(IndexParams p, ChooseParams c) {
  constexpr int kPages = 64 / LC;
  __shared__ union {
    ScoreShared<LC> score;
    ChooseShared<kThreads> choose;
  } sh;
  __shared__ uint32_t keys[kFew];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t b = blockIdx.x / (uint32_t)p.c.kv_heads;
  const int kv = (int)(blockIdx.x - (uint32_t)b * p.c.kv_heads);
  score<DT, LC>(p, b, kv, sh.score, wave * kPages, 4 * kPages, pages_of(p, b),
                [&](int32_t j, uint32_t key) { keys[j] = key; });
  __syncthreads();
  choose_items<kThreads, 1, false>(c, sh.choose, keys);
}

// ---------------------------------------------------------------- moving

// A thread moves one 16-byte chunk of a row's keys and of its values; the first ones also the scales.
__global__ __launch_bounds__(kThreads) void move_kernel(MoveParams p) {
  const int64_t bh = p.bh0 + blockIdx.y;
  const uint32_t i = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  const uint32_t j = i / p.chunks, chunk = i - j * p.chunks.d;
  const int64_t b = bh / p.from.kv_heads;
  const int kv = (int)(bh - b * p.from.kv_heads);
  if (j >= (uint32_t)max(0, min(p.lens[b], p.budget))) return;
  const int32_t t = p.kept[bh * p.budget + j];
  const uint32_t fj = (uint32_t)t / p.from.page_size, tj = j / p.to.page_size;
  if (t < 0 || fj >= (uint32_t)p.from_len || tj >= (uint32_t)p.to_len) return;
  const int32_t fp = p.from_table[b * p.from_row + fj], tp = p.to_table[b * p.to_row + tj];
  if ((uint32_t)fp >= (uint32_t)p.from_pages || (uint32_t)tp >= (uint32_t)p.to_pages) return;
  const uint32_t fr = (uint32_t)t - fj * p.from.page_size.d, tr = j - tj * p.to.page_size.d;
  const int64_t src = kv * p.from.head + row_at(p.from, fp, fr) + 16 * chunk;
  const int64_t dst = kv * p.to.head + row_at(p.to, tp, tr) + 16 * chunk;
  const u32x4 k = *reinterpret_cast<const u32x4*>(p.from.k + src);
  const u32x4 v = *reinterpret_cast<const u32x4*>(p.from.v + src);
  *reinterpret_cast<u32x4*>(p.to.k + dst) = k;
  *reinterpret_cast<u32x4*>(p.to.v + dst) = v;
  if (4 * (int)chunk < p.scale_bytes) {
    const int64_t s = kv * p.from.s_head + scales_at(p.from, fp, fr) + 4 * chunk;
    const int64_t d = kv * p.to.s_head + scales_at(p.to, tp, tr) + 4 * chunk;
    *reinterpret_cast<uint32_t*>(p.to.ks + d) = *reinterpret_cast<const uint32_t*>(p.from.ks + s);
    *reinterpret_cast<uint32_t*>(p.to.vs + d) = *reinterpret_cast<const uint32_t*>(p.from.vs + s);
  }
}

template <int DT, int ST>
void update_by_width(const IndexParams& p, int grid, hipStream_t s) {
  const int dp = attn_padded(p.c.head_dim);
  if (dp == 64)
    update_kernel<DT, ST, 8><<<grid, kThreads, 0, s>>>(p);
  else if (dp == 128)
    update_kernel<DT, ST, 16><<<grid, kThreads, 0, s>>>(p);
  else
    update_kernel<DT, ST, 32><<<grid, kThreads, 0, s>>>(p);
}

template <int DT>
void update_by_storage(const IndexParams& p, int storage, int grid, hipStream_t s) {
  if (storage == AG_KV_16BIT)
    update_by_width<DT, AG_KV_16BIT>(p, grid, s);
  else if (storage == AG_KV_MXFP8)
    update_by_width<DT, AG_KV_MXFP8>(p, grid, s);
  else
    update_by_width<DT, AG_KV_MXFP4>(p, grid, s);
}

template <int DT>
void select_by_width(const IndexParams& p, const ChooseParams& c, int grid, hipStream_t s) {
  const int dp = attn_padded(p.c.head_dim);
  if (dp == 64)
    select_kernel<DT, 8><<<grid, kThreads, 0, s>>>(p, c);
  else if (dp == 128)
    select_kernel<DT, 16><<<grid, kThreads, 0, s>>>(p, c);
  else
    select_kernel<DT, 32><<<grid, kThreads, 0, s>>>(p, c);
}

template <int DT>
void score_by_width(const IndexParams& p, int grid, hipStream_t s) {
  const int dp = attn_padded(p.c.head_dim);
  if (dp == 64)
    score_kernel<DT, 8><<<grid, kThreads, 0, s>>>(p);
  else if (dp == 128)
    score_kernel<DT, 16><<<grid, kThreads, 0, s>>>(p);
  else
    score_kernel<DT, 32><<<grid, kThreads, 0, s>>>(p);
}

template <bool TOKENS>
hipError_t choose(const ChooseParams& p, int64_t batch, hipStream_t s) {
  const int grid = (int)(batch * p.heads);
  if (p.items <= 256 * 8)
    choose_kernel<256, 8, TOKENS><<<grid, 256, 0, s>>>(p);
  else
    choose_kernel<1024, 16, TOKENS><<<grid, 1024, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_index_update(const IndexParams& p, int dtype, int storage, int64_t batch, hipStream_t s) {
  const int grid = (int)(batch * (p.step.d / 4));
  if (dtype == AGMM_F16)
    update_by_storage<AGMM_F16>(p, storage, grid, s);
  else
    update_by_storage<AGMM_BF16>(p, storage, grid, s);
  return hipGetLastError();
}

hipError_t launch_index_score(const IndexParams& p, int dtype, int64_t batch, hipStream_t s) {
  const int grid = (int)(batch * p.c.kv_heads * p.splits);
  if (dtype == AGMM_F16)
    score_by_width<AGMM_F16>(p, grid, s);
  else
    score_by_width<AGMM_BF16>(p, grid, s);
  return hipGetLastError();
}

hipError_t launch_select(const IndexParams& p, const ChooseParams& c, int dtype, int64_t batch, hipStream_t s) {
  const int grid = (int)(batch * p.c.kv_heads);
  if (dtype == AGMM_F16)
    select_by_width<AGMM_F16>(p, c, grid, s);
  else
    select_by_width<AGMM_BF16>(p, c, grid, s);
  return hipGetLastError();
}

hipError_t launch_choose_pages(const ChooseParams& p, int64_t batch, hipStream_t s) {
  return choose<false>(p, batch, s);
}
hipError_t launch_choose_tokens(const ChooseParams& p, int64_t batch, hipStream_t s) {
  return choose<true>(p, batch, s);
}

hipError_t launch_move(MoveParams p, int64_t batch, hipStream_t s) {
  const uint32_t blocks = ((uint32_t)p.budget * p.chunks.d + kThreads - 1) / kThreads;
  const int64_t heads = batch * p.from.kv_heads, most = 65535;
  for (p.bh0 = 0; p.bh0 < heads; p.bh0 += most)
    move_kernel<<<dim3(blocks, (uint32_t)min(most, heads - p.bh0)), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace agmm
