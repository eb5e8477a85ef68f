// gfx950 kernels of the rotary positions and of the paged key-value cache (agmm_attn.h).
//
// All of them move each byte once and compute little, so they are bound by memory bandwidth for
// many tokens and by one launch for few. Work is cut into units of 16 bytes a lane, consecutive
// lanes on consecutive units of a head, then heads, then tokens, so a wave's loads are runs of a
// whole head or more.
//
// Measured, warm, bytes read and written: 16384 tokens x 72 heads of 128 rotated 100 us, 6.0 TB/s; 16384 x 8
// heads of 128 into the cache 20.8 us in 16 bits (6.5 TB/s), 19.4 in e4m3 (5.3), 17.5 in e2m1 (4.9), and
// back 21.3 (6.3), 18.7 (5.4), 19.0 (4.5). A copy of 4 GiB runs at 4.7 TB/s, a kernel of one token takes
// 1.8 us.
#include "agmm_attn_device.h"

namespace agmm {
namespace {

// cos and sin of a position's angle for one pair, times the magnitude. The angle in turns is
// position * theta / 2 pi; with theta / 2 pi held as a fraction of 2^64 the product modulo 2^64 is
// its fractional part, exact but for the fraction's own rounding (2^-65 turns a position), however
// long the context. The top 32 bits as a signed number are turns in [-1/2, 1/2), which is what
// v_sin_f32 and v_cos_f32 take. No table of cosines is read: one would cost 8 bytes a pair
// of cache or memory traffic beside the 8 bytes of the pair itself.
__device__ inline void turn(uint64_t f, int64_t pos, float mag, float& c, float& s) {
  const uint64_t phase = f * (uint64_t)pos;
  const float t = (float)(int32_t)(phase >> 32) * 0x1p-32f;
  c = mag * __builtin_amdgcn_cosf(t);
  s = mag * __builtin_amdgcn_sinf(t);
}

// The empty asm keeps the results 32-bit values that are rounded to 16 bits afterwards: folded into a
// mixed-precision multiply-add in some places and not in others, the same pair would differ in its
// last bit between them.
__device__ inline void rotate(float a, float b, float c, float s, float& ya, float& yb) {
  ya = fmaf(a, c, -(b * s));
  yb = fmaf(b, c, a * s);
  asm("" : "+v"(ya), "+v"(yb));
}

template <int DT>
__device__ inline float value(const uint16_t* p) {
  return T16<DT>::lo(*p);
}
template <int DT>
__device__ inline void put(uint16_t* p, float x) {
  *p = (uint16_t)T16<DT>::pack(x, 0.0f);
}

// One unit of a head's rotated part: 8 pairs (half) or 4 (interleaved). The last unit of a rotated
// part that is no multiple of that begins earlier, and what two units share is written twice, the
// same; in place, where a pair has to be read and written by one thread only, it takes its n pairs
// one by one (4096 tokens x 72 heads of 128, 24 rotated: 33 us so, 47 us pair by pair).
//
// A thread takes one unit of one head and makes its own angles. Four heads to a thread, which share
// them, measured slower: 16384 x 72 heads of 128 108 us against 100, 4097 x 28 of 80 9.5 against 8.7.
template <int DT, bool HALF, bool GRAD>
__device__ inline void rotate_unit(const RopeParams& p, uint32_t u, int64_t pos,
                                   const uint16_t* x, uint16_t* y) {
  constexpr int NP = HALF ? 8 : 4;
  const int r2 = p.plan.rot_dim / 2;
  int i0 = (int)u * NP;
  if (!p.in_place && r2 >= NP) i0 = min(i0, r2 - NP);
  const int n = min(NP, r2 - i0);
  const int e1 = p.plan.rot_start + (HALF ? i0 : 2 * i0);
  x += e1;
  y += e1;
  float c[NP], s[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    turn(p.plan.turns[i0 + k], pos, p.plan.magnitude, c[k], s[k]);  // (the table is padded)
    if (GRAD) s[k] = -s[k];
  }
  if (n == NP) {
    const u32x4 a = load16(x), b = HALF ? load16(x + r2) : a;
    u32x4 ya, yb;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float y0, y1, z0, z1;
      if (HALF) {
        rotate(T16<DT>::lo(a[k]), T16<DT>::lo(b[k]), c[2 * k % NP], s[2 * k % NP], y0, z0);
        rotate(T16<DT>::hi(a[k]), T16<DT>::hi(b[k]), c[(2 * k + 1) % NP], s[(2 * k + 1) % NP], y1,
               z1);
        yb[k] = T16<DT>::pack(z0, z1);
      } else {
        rotate(T16<DT>::lo(a[k]), T16<DT>::hi(a[k]), c[k], s[k], y0, y1);
      }
      ya[k] = T16<DT>::pack(y0, y1);
    }
    store16(y, ya);
    if (HALF) store16(y + r2, yb);
  } else {
#pragma unroll
    for (int k = 0; k < NP; ++k)
      if (k < n) {
        const int ia = HALF ? k : 2 * k, ib = HALF ? k + r2 : 2 * k + 1;
        float ya, yb;
        rotate(value<DT>(x + ia), value<DT>(x + ib), c[k], s[k], ya, yb);
        put<DT>(y + ia, ya);
        put<DT>(y + ib, yb);
      }
  }
}

// One unit of the elements that pass through (never in place): 8 of them, the last unit of a run
// beginning earlier where needed, or all n of a run shorter than that.
__device__ inline void pass_unit(const RopeParams& p, uint32_t u, const uint16_t* x, uint16_t* y) {
  const bool front = u < (uint32_t)p.pass_units0;
  const int begin = front ? 0 : p.plan.rot_start + p.plan.rot_dim;
  const int end = front ? p.plan.rot_start : p.plan.head_dim;
  const int n = min(8, end - begin);
  const int e = min(begin + 8 * (int)(front ? u : u - p.pass_units0), end - n);
  if (n == 8) {
    store16(y + e, load16(x + e));
  } else {
    for (int k = 0; k < n; ++k) y[e + k] = x[e + k];
  }
}

template <int DT, bool HALF, bool GRAD>
__device__ inline void rope_thread(const RopeParams& p, uint32_t idx, int64_t b) {
  if (idx >= p.total) return;
  const uint32_t r = idx / p.units, u = idx - r * p.units.d;
  const uint32_t t = r / p.heads, h = r - t * p.heads.d;
  const uint16_t* x = p.x + b * p.x_batch + (int64_t)t * p.x_token + (int64_t)h * p.x_head;
  uint16_t* y = p.y + b * p.y_batch + (int64_t)t * p.y_token + (int64_t)h * p.y_head;
  if (u < (uint32_t)p.rot_units)
    rotate_unit<DT, HALF, GRAD>(p, u, p.positions[b * p.pos_batch + t], x, y);
  else
    pass_unit(p, u - p.rot_units, x, y);
}

template <int DT, bool HALF, bool GRAD>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeParams p) {
  rope_thread<DT, HALF, GRAD>(p, blockIdx.x * kThreads + threadIdx.x, blockIdx.y);
}

// ---- the cache ----

template <int DT, int ST>
struct Mx {
  static constexpr bool kFp8 = ST == AG_KV_MXFP8;
  // The largest code M = 1.75 * 2^8 or 1.5 * 2^2, and the largest whose value the 16-bit type holds
  // at the scales (exponents kEdge and above) where M's would not: 240 or 3.
  static constexpr int kExp = kFp8 ? 8 : 2;
  static constexpr uint32_t kMant = kFp8 ? 0x600000u : 0x400000u;
  static constexpr float kM = kFp8 ? 448.0f : 6.0f;
  static constexpr float kMEdge = kFp8 ? 240.0f : 3.0f;
  static constexpr int kEdge = (DT == AGMM_F16 ? 16 : 128) - (kFp8 ? 8 : 2);
};

// Maximum over the 4 lanes of a quad.
__device__ inline uint32_t quad_max(uint32_t a) {
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xf, 0xf, true));  // lanes ^ 1
  return max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xf, 0xf, true));  // lanes ^ 2
}

// Writes the 8 elements x of chunk `ch` of a row. 4 neighbouring lanes hold a block of 32.
template <int DT, int ST>
__device__ inline void write_chunk(char* row, char* srow, uint32_t ch, u32x4 x) {
  if (ST == AG_KV_16BIT) {
    *reinterpret_cast<u32x4*>(row + 16 * ch) = x;
    return;
  }
  typedef Mx<DT, ST> M;
  float v[8];
  uint32_t amax = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = T16<DT>::lo(x[k]);
    v[2 * k + 1] = T16<DT>::hi(x[k]);
  }
  // magnitudes compare as their bits do, NaN above infinity above the rest
#pragma unroll
  for (int k = 0; k < 8; ++k) amax = max(amax, __builtin_bit_cast(uint32_t, v[k]) & 0x7fffffffu);
  amax = quad_max(amax);
  const bool odd = amax >= 0x7f800000u;
  int e = (int)(amax >> 23) - 127 - M::kExp + ((amax & 0x7fffffu) > M::kMant ? 1 : 0);
  e = odd ? 0 : max(e, -126);
  const float inv = odd ? 0.0f : __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
  const float top = e >= M::kEdge ? M::kMEdge : M::kM;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = odd ? 0.0f : __builtin_amdgcn_fmed3f(v[k] * inv, -top, top);  // the product is exact
  }
  if (M::kFp8) {
    u32x2 w;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k], v[4 * k + 1], 0, false);
      w[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k + 2], v[4 * k + 3], b, true);
    }
    *reinterpret_cast<u32x2*>(row + 8 * ch) = w;
  } else {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.0f, 3);
    *reinterpret_cast<uint32_t*>(row + 4 * ch) = w;
  }
  if (ch % 4 == 0) srow[ch / 4] = (char)(odd ? 255 : e + 127);
}

// Chunk `ch` of a row, as 8 packed 16-bit values.
template <int DT, int ST>
__device__ inline u32x4 read_chunk(const char* row, const char* srow, uint32_t ch) {
  if (ST == AG_KV_16BIT) return *reinterpret_cast<const u32x4*>(row + 16 * ch);
  const float s = scale_of(*reinterpret_cast<const uint8_t*>(srow + ch / 4));
  if (ST == AG_KV_MXFP8) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(row + 8 * ch);
    return from_fp8x8<DT>(w[0], w[1], s);
  }
  return from_fp4x8<DT>(*reinterpret_cast<const uint32_t*>(row + 4 * ch), s);
}

// The 8 elements from e0 of a head, rotated as rotate_unit() would: each element's partner of its
// pair is read beside it (from the caches, its own chunk's thread reads it too), so that a thread
// ends with 8 consecutive elements and a quad of lanes with a block.
template <int DT, bool HALF>
__device__ inline u32x4 rotated_chunk(const RopePlan& r, int64_t pos, const uint16_t* head, int e0) {
  const u32x4 own = load16(head + e0);
  const int r2 = r.rot_dim / 2, r0 = r.rot_start;
  if (e0 + 8 <= r0 || e0 >= r0 + r.rot_dim) return own;
  u32x4 y;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = e0 + k - r0;  // in the rotated part
    const uint32_t bits = (own[k / 2] >> (16 * (k % 2))) & 0xffffu;
    uint32_t w = bits;
    if (i >= 0 && i < r.rot_dim) {
      const bool second = HALF ? i >= r2 : (i & 1) != 0;
      const int pair = HALF ? (second ? i - r2 : i) : i / 2;
      const float z = value<DT>(head + e0 + k + (HALF ? (second ? -r2 : r2) : (second ? -1 : 1)));
      float c, s, ya, yb;
      turn(r.turns[pair], pos, r.magnitude, c, s);
      const float x = T16<DT>::lo(bits);
      rotate(second ? z : x, second ? x : z, c, s, ya, yb);
      w = T16<DT>::pack(second ? yb : ya, 0.0f) & 0xffffu;
    }
    y[k / 2] = (k % 2) ? (y[k / 2] | (w << 16)) : w;
  }
  return y;
}

template <int DT, int ST, bool ROPE, bool HALF>
__device__ inline void append_thread(const CacheParams& p, uint32_t idx) {
  if (idx >= p.total) return;
  const uint32_t r = idx / p.chunks, ch = idx - r * p.chunks.d;
  const uint32_t t = r / p.heads, h = r - t * p.heads.d;
  const int64_t slot = p.slots[t];
  if (slot < 0 || slot >= (int64_t)p.c.rows) return;  // the same for a block's 4 lanes
  const uint32_t page = (uint32_t)slot / p.c.page_size;
  const uint32_t row = (uint32_t)slot - page * p.c.page_size.d;
  const uint16_t* kh = p.k + (int64_t)t * p.k_token + (int64_t)h * p.k_head;
  const uint16_t* vh = p.v + (int64_t)t * p.v_token + (int64_t)h * p.v_head;
  const u32x4 v = load16(vh + 8 * ch);
  const u32x4 k = ROPE ? rotated_chunk<DT, HALF>(p.plan, p.positions[t], kh, 8 * (int)ch)
                       : load16(kh + 8 * ch);
  const int64_t at = row_at(p.c, page, row) + (int64_t)h * p.c.head;
  const int64_t sat = scales_at(p.c, page, row) + (int64_t)h * p.c.s_head;
  write_chunk<DT, ST>(p.c.k + at, p.c.ks + sat, ch, k);
  write_chunk<DT, ST>(p.c.v + at, p.c.vs + sat, ch, v);
}

template <int DT, int ST>
__global__ __launch_bounds__(kThreads) void append_kernel(CacheParams p) {
  append_thread<DT, ST, false, false>(p, blockIdx.x * kThreads + threadIdx.x);
}

template <int DT, int ST, bool HALF>
__global__ __launch_bounds__(kThreads) void append_rope_kernel(CacheParams p, RopeParams q) {
  if (blockIdx.x < p.q_blocks)
    rope_thread<DT, HALF, false>(q, blockIdx.x * kThreads + threadIdx.x, 0);
  else
    append_thread<DT, ST, true, HALF>(p, (blockIdx.x - p.q_blocks) * kThreads + threadIdx.x);
}

template <int DT, int ST>
__global__ __launch_bounds__(kThreads) void read_kernel(CacheParams p) {
  const uint32_t idx = blockIdx.x * kThreads + threadIdx.x;
  if (idx >= p.total) return;
  const uint32_t r = idx / p.chunks, ch = idx - r * p.chunks.d;
  const uint32_t t = r / p.heads, h = r - t * p.heads.d;
  const int64_t slot = p.slots[t];
  u32x4 k = {0, 0, 0, 0}, v = {0, 0, 0, 0};
  if (slot >= 0 && slot < (int64_t)p.c.rows) {
    const uint32_t page = (uint32_t)slot / p.c.page_size;
    const uint32_t row = (uint32_t)slot - page * p.c.page_size.d;
    const int64_t at = row_at(p.c, page, row) + (int64_t)h * p.c.head;
    const int64_t sat = scales_at(p.c, page, row) + (int64_t)h * p.c.s_head;
    k = read_chunk<DT, ST>(p.c.k + at, p.c.ks + sat, ch);
    v = read_chunk<DT, ST>(p.c.v + at, p.c.vs + sat, ch);
  }
  store16(p.k_out + (int64_t)t * p.k_token + (int64_t)h * p.k_head + 8 * ch, k);
  store16(p.v_out + (int64_t)t * p.v_token + (int64_t)h * p.v_head + 8 * ch, v);
}

inline uint32_t blocks(uint32_t threads) { return (threads + kThreads - 1) / kThreads; }

}  // namespace

hipError_t launch_rope(const RopeParams& p, int dtype, int pairing, int gradient, int64_t batch,
                       hipStream_t s) {
  const dim3 grid(blocks(p.total), (uint32_t)batch);
  auto by = [&](auto dt, auto half) {
    constexpr int DT = decltype(dt)::value;
    constexpr bool HALF = decltype(half)::value;
    if (gradient)
      rope_kernel<DT, HALF, true><<<grid, kThreads, 0, s>>>(p);
    else
      rope_kernel<DT, HALF, false><<<grid, kThreads, 0, s>>>(p);
  };
  auto pairs = [&](auto dt) {
    if (pairing == AG_ROPE_HALF)
      by(dt, std::true_type());
    else
      by(dt, std::false_type());
  };
  if (dtype == AGMM_F16)
    pairs(std::integral_constant<int, AGMM_F16>());
  else
    pairs(std::integral_constant<int, AGMM_BF16>());
  return hipGetLastError();
}

namespace {

template <class F>
void by_type(int dtype, int storage, F f) {
  auto st = [&](auto dt) {
    if (storage == AG_KV_16BIT)
      f(dt, std::integral_constant<int, AG_KV_16BIT>());
    else if (storage == AG_KV_MXFP8)
      f(dt, std::integral_constant<int, AG_KV_MXFP8>());
    else
      f(dt, std::integral_constant<int, AG_KV_MXFP4>());
  };
  if (dtype == AGMM_F16)
    st(std::integral_constant<int, AGMM_F16>());
  else
    st(std::integral_constant<int, AGMM_BF16>());
}

}  // namespace

hipError_t launch_append(const CacheParams& p, const RopeParams* rope, int dtype, int storage,
                         int pairing, hipStream_t s) {
  const uint32_t grid = p.q_blocks + blocks(p.total);
  by_type(dtype, storage, [&](auto dt, auto st) {
    constexpr int DT = decltype(dt)::value, ST = decltype(st)::value;
    if (!rope)
      append_kernel<DT, ST><<<grid, kThreads, 0, s>>>(p);
    else if (pairing == AG_ROPE_HALF)
      append_rope_kernel<DT, ST, true><<<grid, kThreads, 0, s>>>(p, *rope);
    else
      append_rope_kernel<DT, ST, false><<<grid, kThreads, 0, s>>>(p, *rope);
  });
  return hipGetLastError();
}

hipError_t launch_read(const CacheParams& p, int dtype, int storage, hipStream_t s) {
  by_type(dtype, storage, [&](auto dt, auto st) {
    read_kernel<decltype(dt)::value, decltype(st)::value>
        <<<blocks(p.total), kThreads, 0, s>>>(p);
  });
  return hipGetLastError();
}

}  // namespace agmm
