// Pieces that the MXFP4 product kernels share: expert row ranges, row-major scale
// fetches, the epilogue's stores.
#pragma once
#include "fn_device.cuh"
#include "mg_params.h"
#include "tc_device.cuh"

namespace fn {

// Row range [lo, lo + cnt) of expert e, kept inside [0, M) whatever the
// offsets hold.
__device__ __forceinline__ void mg_range(const MGParams& p, int e, int* lo, int* cnt) {
  const int a = min(max(p.offsets[e], 0), p.M), b = min(max(p.offsets[e + 1], 0), p.M);
  *lo = a;
  *cnt = max(b - a, 0);
}

// The tile table in shared memory, by one warp: cum [E + 1] tiles before each
// expert (`each` for every piece of `tok` rows, at most `most` pieces in
// all), lo [E] first rows, cnt [E] rows.  A running sum over 32 experts at a time.
__device__ __forceinline__ void mg_table(const MGParams& p, int* table, int lane, int tok, int each,
                                         int most) {
  int* cum = table;
  int* lo = table + p.E + 1;
  int* cnt = table + 2 * p.E + 1;
  int64_t before = 0;  // (offsets that break the contract can add up to any number of rows)
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    int a = 0, c = 0;
    if (e0 + lane < p.E) {
      mg_range(p, e0 + lane, &a, &c);
      lo[e0 + lane] = a;
      cnt[e0 + lane] = c;
    }
    int64_t sum = c / tok + (c % tok != 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (e0 + lane < p.E) cum[e0 + lane + 1] = each * (int)min(before + sum, (int64_t)most);
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (lane == 0) cum[0] = 0;
}

__device__ __forceinline__ uint4 ld_scales16(const uint8_t* p) {
  uint4 v;
  asm("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p));
  return v;
}

// The 16 scale bytes of groups 16 c .. 16 c + 15 of a row-major row (zeros past
// the last group).  `wide`: every row is whole aligned vectors.  Otherwise the
// aligned words that hold at least one of the bytes are read and shifted.
__device__ __forceinline__ uint4 mg_scales(const uint8_t* row, int c, int groups, bool wide) {
  const int left = groups - 16 * c;
  if (left <= 0) return make_uint4(0, 0, 0, 0);
  const uint8_t* p = row + 16 * c;
  if (wide) return ld_scales16(p);
  const int n = min(left, 16), a = (int)(reinterpret_cast<uintptr_t>(p) & 3);
  const uint32_t* w = reinterpret_cast<const uint32_t*>(p - a);
  uint32_t v[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = 4 * i < a + n ? __ldg(w + i) : 0;
  uint4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x = __funnelshift_r(v[i], v[i + 1], 8 * a);
    const int have = n - 4 * i;  // bytes of this word inside the row
    if (have < 4) x = have <= 0 ? 0 : x & ((1u << (8 * have)) - 1);
    set_word(r, i, x);
  }
  return r;
}

// The same from the 32x4x4 tiling (the last K step of rows whose padding the
// MMA would read).
__device__ __forceinline__ uint4 mg_tiled_scales(const uint8_t* base, int64_t row, int c,
                                                 int groups) {
  const int kts = (groups + 3) >> 2;
  uint4 r = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int kt = 4 * c + i;
    if (kt >= kts) continue;
    uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(
        base + ((row >> 7) * kts + kt) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4));
    const int have = groups - 4 * kt;
    if (have < 4) x &= (1u << (8 * have)) - 1;
    set_word(r, i, x);
  }
  return r;
}

// Transposes 4 rows x 4 features over groups of four lanes: in, the lane's
// feature for rows 0..3 (packed pairs a = rows 0, 1, b = rows 2, 3); out, four
// neighbouring features of row (lane & 3).
__device__ __forceinline__ uint2 mg_transpose4(uint32_t a, uint32_t b, int lane) {
  const bool upper = lane & 2, odd = lane & 1;
  const uint32_t keep = upper ? b : a;
  const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? a : b, 2);  // feature ^ 2, same rows
  const uint32_t mine = __byte_perm(keep, got, odd ? 0x7632 : 0x5410);
  const uint32_t other =
      __shfl_xor_sync(0xffffffffu, __byte_perm(keep, got, odd ? 0x5410 : 0x7632), 1);
  const uint32_t x = odd ? other : mine, y = odd ? mine : other;
  const uint32_t l = __byte_perm(x, y, 0x5410), h = __byte_perm(x, y, 0x7632);
  return upper ? make_uint2(h, l) : make_uint2(l, h);
}

__device__ __forceinline__ void mg_store_one(const MGParams& p, float a, int64_t row, int f) {
  if (p.out_type == MG_OUT_FP32)
    static_cast<float*>(p.out)[row * p.ldo + f] = a;
  else
    static_cast<uint16_t*>(p.out)[row * p.ldo + f] =
        (uint16_t)(p.out_type == MG_OUT_BF16 ? pack_bf16x2(a, 0.f) : pack_f16x2(a, 0.f));
}

// Whether out holds NaN there.
__device__ __forceinline__ bool mg_is_nan(const MGParams& p, int64_t row, int f) {
  if (p.out_type == MG_OUT_FP32)
    return (reinterpret_cast<const uint32_t*>(p.out)[row * p.ldo + f] & 0x7fffffffu) > 0x7f800000u;
  return (static_cast<const uint16_t*>(p.out)[row * p.ldo + f] & 0x7fffu) >
         (p.out_type == MG_OUT_BF16 ? 0x7f80u : 0x7c00u);
}

// Stores `n` rows (of at most C) of a chunk; the lane holds feature f.
template <int C>
__device__ __forceinline__ void mg_store(const MGParams& p, uint32_t (&v)[C], int64_t row, int n,
                                         int f, int lane) {
  if (p.out_type == MG_OUT_FP32) {
    if (p.out_pairs) {  // neighbouring lanes trade rows for pairs of features
      const int odd = lane & 1, pair = f & ~1;
      float* o = static_cast<float*>(p.out) + (row + odd) * p.ldo + pair;
      float2 w[C / 2];
#pragma unroll
      for (int i = 0; i < C / 2; ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[2 * i] : v[2 * i + 1], 1);
        w[i] = odd ? make_float2(__uint_as_float(got), __uint_as_float(v[2 * i + 1]))
                   : make_float2(__uint_as_float(v[2 * i]), __uint_as_float(got));
      }
      const int mine = pair < p.N ? n - odd : 0;
#pragma unroll
      for (int i = 0; i < C / 2; ++i)
        if (2 * i < mine) *reinterpret_cast<float2*>(o + 2 * i * p.ldo) = w[i];
      return;
    }
    float* o = static_cast<float*>(p.out) + row * p.ldo + f;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < n && f < p.N) o[i * p.ldo] = __uint_as_float(v[i]);
    return;
  }
  const bool bf = p.out_type == MG_OUT_BF16;
  if (p.out_quads) {
    const int quad = f & ~3;
    uint16_t* o = static_cast<uint16_t*>(p.out) + (row + (lane & 3)) * p.ldo + quad;
    // all transposes first, without a branch between them: their shuffles overlap
    // (a loop that left at n ran them one after another, 3.6 us of a tile's 10)
    uint2 w[C / 4];
#pragma unroll
    for (int i = 0; i < C / 4; ++i) {
      const float a = __uint_as_float(v[4 * i]), b = __uint_as_float(v[4 * i + 1]),
                  c = __uint_as_float(v[4 * i + 2]), d = __uint_as_float(v[4 * i + 3]);
      w[i] = bf ? mg_transpose4(pack_bf16x2(a, b), pack_bf16x2(c, d), lane)
                : mg_transpose4(pack_f16x2(a, b), pack_f16x2(c, d), lane);
    }
    const int mine = quad < p.N ? n - (lane & 3) : 0;
#pragma unroll
    for (int i = 0; i < C / 4; ++i)
      if (4 * i < mine) *reinterpret_cast<uint2*>(o + 4 * i * p.ldo) = w[i];
    return;
  }
  uint16_t* o = static_cast<uint16_t*>(p.out) + row * p.ldo + f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const float a = __uint_as_float(v[i]);
    if (i < n && f < p.N)
      o[i * p.ldo] = (uint16_t)(bf ? pack_bf16x2(a, 0.f) : pack_f16x2(a, 0.f));
  }
}

}  // namespace fn
