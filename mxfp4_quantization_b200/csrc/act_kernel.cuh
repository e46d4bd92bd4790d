// silu(gate) * up with the quantization of its result, sm_100a.
//
// y = round16(g u / (1 + e^-g)), correctly rounded, then the quantization stage
// of the row kernels (rq_kernel.cuh) on y: the same codes and scales as the
// stand-alone quantization of that row.
#pragma once
#include "rq_kernel.cuh"

namespace fn {

struct ActParams {
  const uint4* x;           // [M, 2H] as 16-byte vectors, rows ldv vectors apart
  const int32_t* num_rows;  // rows in use, or nullptr
  uint8_t* out_q;
  void* out_scale;
  uint4* out_y;             // [M, H] or nullptr
  int64_t M, ldv;
  int nvec;                 // H / 8
  int scale_layout;
  int64_t scale_ld;
  // ceil(2^64 / n) and ceil(2^32 / n) for the n >= 2 units of a row (group modes): the high
  // half of their product with i is i / n, exactly, while i (n - 1) < 2^64 (2^32)
  uint64_t recip64;
  uint32_t recip32;
};

// The real value's nearest 16-bit neighbour through fp64.  p = g u (and p / 2) is
// exact: 16 or 22 bits.  Between -2^-20 and 2^-20 the value is (p / 2)(1 + c), c =
// tanh(g / 2) = g/2 - g^3/24 + ..., above 20 it is p (1 + c), c = -e^-g / (1 + e^-g):
// p / 2 or p may be the midpoint of two 16-bit values, and c, below 2^-20, then
// decides however small it is, so its sign stays with the sum (`side`) where
// the fp64 addition loses it.  Elsewhere the fp64 quotient, within a few 2^-53
// of the real value, is no midpoint (e^-g is transcendental).  fp64 -> fp32
// rounds to odd (the last bit marks what was cut off), so that the rounding to
// 16 bits is the only one.
template <class IO>
__device__ __noinline__ uint32_t silu_mul_fp64(float g, float u) {
  const double gd = g;
  double p = gd * (double)u, v;
  int side = 0;  // the real magnitude is above (1) or below (-1) that of v
  if ((fabsf(g) < 0x1p-20f || g > 20.f) && isfinite(p)) {
    double c;
    if (g > 20.f) {
      const double e = exp(-gd);
      c = -e / (1.0 + e);
      side = -1;
    } else {
      c = gd * (0.5 - gd * gd / 24.0);
      p *= 0.5;
      side = g > 0.f ? 1 : -1;
    }
    v = p == 0.0 ? p : p + p * c;
    if (v != p || p == 0.0) side = 0;
  } else {
    v = p / (1.0 + exp(-gd));
  }
  float f = __double2float_rz(v);
  if (f == f && !isinf(f)) {
    if ((double)f != v || side > 0)
      f = __uint_as_float(__float_as_uint(f) | 1u);
    else if (side < 0)
      f = __uint_as_float((__float_as_uint(f) - 1u) | 1u);
  }
  return IO::pack(f, 0.f) & 0xFFFFu;
}

// The same for the elements that fp32 leaves open, in about 50 instructions (the
// form above takes 300): e^-g as 2^n 2^f, the Taylor polynomial of e^(f ln 2) to
// degree 11 (|f ln 2| <= 0.347: 2^-47), the reciprocal of 1 + e^-g by two
// Newton-Raphson steps on the fp32 approximation; 2^-45 in all.  Where the result
// is that near a midpoint (twice over), outside the type's normal range, or g < -87,
// the form above decides.
template <class IO>
__device__ __forceinline__ uint32_t silu_mul_mid(float g, float u) {
  const double gd = g, t = gd * -1.4426950408889634074;
  const double n = rint(t), x = (t - n) * 0.69314718055994530942;
  double e = 1.0 / 39916800;
  e = fma(e, x, 1.0 / 3628800);
  e = fma(e, x, 1.0 / 362880);
  e = fma(e, x, 1.0 / 40320);
  e = fma(e, x, 1.0 / 5040);
  e = fma(e, x, 1.0 / 720);
  e = fma(e, x, 1.0 / 120);
  e = fma(e, x, 1.0 / 24);
  e = fma(e, x, 1.0 / 6);
  e = fma(e, x, 0.5);
  e = fma(e, x, 1.0);
  e = fma(e, x, 1.0);
  const int ni = g >= -87.f && g <= 700.f ? (int)n : 0;
  const double d = 1.0 + __hiloint2double(__double2hiint(e) + (ni << 20), __double2loint(e));
  float rf;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rf) : "f"((float)d));
  double r = rf;
  r = fma(fma(-d, r, 1.0), r, r);
  r = fma(fma(-d, r, 1.0), r, r);
  const double v = gd * (double)u * r;
  constexpr int kCut = IO::kF16 ? 42 : 45;  // mantissa bits beyond the 16-bit type's
  const uint64_t rest = (uint64_t)__double_as_longlong(v) & ((1ull << kCut) - 1);
  const int64_t off = (int64_t)rest - (int64_t)(1ull << (kCut - 1));
  const double mag = fabs(v);
  const bool sure = g >= -87.f && g <= 700.f && (off > 1 << 10 || off < -(1 << 10)) &&
                    mag >= (IO::kF16 ? 0x1p-14 : 0x1p-100) && mag < (IO::kF16 ? 65504.0 : 0x1p127);
  if (!sure) return silu_mul_fp64<IO>(g, u);
  // cut to fp32 with the last bit set: on the same side of every midpoint
  const float f = __uint_as_float(__float_as_uint(__double2float_rz(v)) | 1u);
  return IO::pack(f, 0.f) & 0xFFFFu;
}

// The lower end of an interval that holds g u / (1 + e^-g); its product with
// kSiluWidth is the upper one (g >= -87, |g r| >= 2^-126, |result| >= 2^-100).  e^-g = 2^t
// with t = -g log2(e) in two parts: the rounded product and its remainder, which scales
// the result by 1 + t_lo ln 2.
// Errors, in units of 2^-24: ex2.approx 4 (2^-22), the remainder's terms 1, their
// product 1, the sum 1 + e^-g 1 (and it passes on at most the 6 before), the
// approximate reciprocal 2, two products 2: below 12 in all.  The sum comes scaled by
// 1 + 14 units, so the result is 2 to 26 below the real value, and 28 more, less
// the rounding of that product, are above it.  (The .ftz forms: an e^-g below 2^-126 adds nothing to 1, and 1 + e^-g stays below 2^126,
// so neither result that matters is subnormal.  The product g r is a .ftz form too: a
// bf16 gate below 2^-125 makes it subnormal, whose spacing swallows the 14 units, and a
// large u would bring such a result back to any size; flushed, it stays 0 and counts
// as outside the range.  It takes no time; a second minimum over the gates took 62 us
// instead of 60, 32768 x 2048, MXFP4.)
constexpr float kSiluUp = 1.f + 14 * 0x1p-24f;
constexpr float kSiluWidth = 1.f + 28 * 0x1p-24f;

__device__ __forceinline__ float2 mul_ftz_f32x2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.ftz.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 silu_mul_fp32(float2 g, float2 u) {
  constexpr float kLog2e = 1.44269504088896340736f;
  constexpr float kLog2eLo = 1.92596299112661746887e-8f;  // log2(e) - kLog2e
  constexpr float kLn2 = 0.693147180559945309417f;
  // t = -g log2(e), lo what t lacks, with the other sign (no negations)
  const float2 t = mul_f32x2(g, make_float2(-kLog2e, -kLog2e));
  float2 lo = fma_f32x2(g, make_float2(kLog2e, kLog2e), t);
  lo = fma_f32x2(g, make_float2(kLog2eLo, kLog2eLo), lo);
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = fma_f32x2(e, mul_f32x2(lo, make_float2(-kLn2, -kLn2)), e);
  const float2 d = fma_f32x2(e, make_float2(kSiluUp, kSiluUp), make_float2(kSiluUp, kSiluUp));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return mul_f32x2(mul_ftz_f32x2(g, r), u);  // g u alone can overflow where the result does not
}

// The smallest value, NaN if one is.
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int N>
struct SiluVecs {
  uint4 y[N];
};

// Recomputes the elements of `mask` (8 bits a vector) of N vectors, their gates at src
// and every `step` vectors on, their ups nvec vectors behind (read again, 2 bytes
// each, from L1): every lane its own next one, so lanes that missed different elements share
// a pass.
template <class IO, int N>
__device__ __noinline__ SiluVecs<N> silu_mul_redo(SiluVecs<N> s, const uint4* src, int step,
                                                  int nvec, uint32_t mask) {
  const uint16_t* g = reinterpret_cast<const uint16_t*>(src);
  while (mask) {
    const int i = __ffs(mask) - 1, w = i >> 1, sh = 16 * (i & 1);
    mask &= mask - 1;
    const uint16_t* at = g + (w >> 2) * step * 8 + (i & 7);
    const uint32_t r = silu_mul_mid<IO>(IO::lo(__ldg(at)), IO::lo(__ldg(at + nvec * 8)));
    const uint32_t keep = ~(0xFFFFu << sh);
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (w == 4 * k + j) set_word(s.y[k], j, (word(s.y[k], j) & keep) | r << sh);
    }
  }
  return s;
}

// y of 8 elements.  The two ends of the interval that holds the real value
// round to one 16-bit value unless a midpoint lies between them; one test
// covers all 8.  Returns the mask of the elements that stay open.
template <class IO>
__device__ __forceinline__ uint32_t silu_mul_fast(const uint4& gv, const uint4& uv, uint4& out) {
  uint32_t a[4], y[4], differ = 0;
  float2 v[4];
  float vmin = 1.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 g = make_float2(IO::lo(word(gv, i)), IO::hi(word(gv, i)));
    const float2 u = make_float2(IO::lo(word(uv, i)), IO::hi(word(uv, i)));
    v[i] = silu_mul_fp32(g, u);
    const float2 h = mul_f32x2(v[i], make_float2(kSiluWidth, kSiluWidth));
    a[i] = IO::pack(v[i].x, v[i].y);
    y[i] = IO::pack(h.x, h.y);
    differ |= a[i] ^ y[i];
    vmin = min_nan(vmin, fabsf(v[i].x), fabsf(v[i].y));
  }
  out = make_uint4(y[0], y[1], y[2], y[3]);
  uint32_t mask = 0;
  // (g below -87.3, where 1 / (1 + e^-g) leaves the normal range, gives 0 here)
  const bool far = !(vmin >= 0x1p-100f);
  if (differ != 0 || far) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = a[i] ^ y[i];
      if (x & 0xFFFFu) mask |= 1u << (2 * i);
      if (x >> 16) mask |= 2u << (2 * i);
    }
    if (far) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float g0 = IO::lo(word(gv, i)), g1 = IO::hi(word(gv, i));
        // outside the interval's range (a zero is exact, or far below every 16-bit value,
        // if g r was not flushed)
        const bool in0 = fabsf(v[i].x) >= 0x1p-100f ||
                         (v[i].x == 0.f && (g0 == 0.f || fabsf(g0) >= 0x1p-100f));
        const bool in1 = fabsf(v[i].y) >= 0x1p-100f ||
                         (v[i].y == 0.f && (g1 == 0.f || fabsf(g1) >= 0x1p-100f));
        if (!(g0 >= -87.f) || !in0) mask |= 1u << (2 * i);
        if (!(g1 >= -87.f) || !in1) mask |= 2u << (2 * i);
      }
    }
  }
  return mask;
}

// y of N vectors, `step` apart from src on; `skip`: the mask of elements not asked for.
template <class IO, int N>
__device__ __forceinline__ void silu_mul_vecs(const uint4 (&g)[N], const uint4 (&u)[N], uint4* y,
                                              const uint4* src, int step, int nvec,
                                              uint32_t skip = 0) {
  uint32_t mask = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) mask |= silu_mul_fast<IO>(g[k], u[k], y[k]) << (8 * k);
  mask &= ~skip;
  if (mask) {
    SiluVecs<N> s;
#pragma unroll
    for (int k = 0; k < N; ++k) s.y[k] = y[k];
    s = silu_mul_redo<IO, N>(s, src, step, nvec, mask);
#pragma unroll
    for (int k = 0; k < N; ++k) y[k] = s.y[k];
  }
}

__device__ __forceinline__ int64_t act_rows(const ActParams& p) {
  if (p.num_rows == nullptr) return p.M;
  const int64_t n = *p.num_rows;
  return n < 0 ? 0 : n < p.M ? n : p.M;
}

// Group modes (MXFP4, FP8 per 128): the rows laid end to end, N neighbouring 8-element
// vectors a thread (two where there is work for it, one for decode-sized calls);
// groups are 4 / N or 16 / N neighbouring lanes.  Bound by instructions (24 an element:
// two special-function operations, five packed fp32, the interval test, the
// quantization; 70 % of the issue slots) and the loads' latency in front of them.
// 32768 x 2048: MXFP4 from bf16 60 us (5.1 TB/s), FP8 per 128 67 us; from
// binary16, whose midpoints lie eight times as close, 76 and 83 us.  Loads past L1
// 60, 68, 76 and 84 us, with a thread's 32 bytes in one load (aligned rows only) the
// same; five blocks an SM 62, 70, 76 and 83; vectors 256 apart instead of neighbours
// (their own scales, twice the shuffles), each one's open elements on their own 73,
// 85, 94 and 106.
template <int MODE, class IO, int N>
__global__ void __launch_bounds__(256, 6) act_groups_kernel(const ActParams p) {
  pdl_enter();
  constexpr int kLanes = (MODE == MODE_MX ? 4 : 16) / N;
  const int lane = threadIdx.x & 31;
  const int units = p.nvec / N;
  const int64_t rows = act_rows(p), i0 = (int64_t)blockIdx.x * 256;
  if (i0 >= rows * units) return;
  // a unit is at most 255 past (r0, v0), v0 < units <= 4096
  const int64_t r0 = (int64_t)__umul64hi((uint64_t)i0, p.recip64);
  const unsigned at = (unsigned)(i0 - r0 * units) + threadIdx.x;
  const unsigned down = __umulhi(at, p.recip32);
  int64_t row = r0 + down;
  int v = (int)(at - down * (unsigned)units) * N;
  const bool ok = row < rows;
  if (!ok) row = 0, v = 0;
  uint4 g[N], u[N], y[N];
  const uint4* src = p.x + row * p.ldv + v;
  // (through L1: each of a thread's loads takes half of every 32-byte sector)
#pragma unroll
  for (int k = 0; k < N; ++k) {
    g[k] = __ldg(src + k);
    u[k] = __ldg(src + p.nvec + k);
  }
  silu_mul_vecs<IO, N>(g, u, y, src, 1, p.nvec);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (p.out_y && ok) st_stream(p.out_y + row * p.nvec + v + k, y[k]);
  }
  float a = vec_absmax<IO>(y[0]);
  if constexpr (MODE == MODE_MX) {
    if constexpr (N == 2) a = fmaxf(a, vec_absmax<IO>(y[1]));
    float inv;
    const uint32_t e8 = mx_scale(group_max<kLanes>(a), inv);
    uint32_t q[N];
#pragma unroll
    for (int k = 0; k < N; ++k) q[k] = e2m1_codes<IO>(y[k], inv);
    if (!ok) return;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out_q + row * (int64_t)(p.nvec * 4)) + v;
    if constexpr (N == 2)
      st_stream(reinterpret_cast<uint2*>(dst), make_uint2(q[0], q[1]));
    else
      st_stream(dst, q[0]);
    if (lane % kLanes == 0)
      static_cast<uint8_t*>(p.out_scale)[scale_index(p.scale_layout, p.scale_ld, row, v / 4,
                                                     p.nvec / 4)] = (uint8_t)e8;
  } else {
    // (as bits: a vector of NaN counts as the largest, as in quant_vec)
    uint32_t am = __float_as_uint(a);
    if constexpr (N == 2) am = max(am, __float_as_uint(vec_absmax<IO>(y[1])));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
    const Fp8Scale s = fp8_scale_direct(__uint_as_float(am));
    const bool exact = __any_sync(0xffffffffu, s.exact_div);
    uint2 q[N];
#pragma unroll
    for (int k = 0; k < N; ++k) q[k] = e4m3_codes_uniform<IO>(y[k], s, exact);
    if (!ok) return;
    uint2* dst = reinterpret_cast<uint2*>(p.out_q + row * (int64_t)(p.nvec * 8)) + v;
    if constexpr (N == 2)
      st_stream(reinterpret_cast<uint4*>(dst), make_uint4(q[0].x, q[0].y, q[1].x, q[1].y));
    else
      st_stream(dst, q[0]);
    if (lane % kLanes == 0)
      static_cast<float*>(p.out_scale)[scale_index(p.scale_layout, p.scale_ld, row, v / 16,
                                                   p.nvec / 16)] = s.s;
  }
}

// Per-token mode: a block per row, the row in registers (V vectors a thread)
// between the maximum and the codes.  bf16, 67 M elements: 64 us at H = 1024 and 2048
// (5.2 TB/s), 67 us at 8192, 74 us at 16384, 99 us at 32768; the sizes of the blocks,
// both ways, are at the launch.  Three blocks of 512 threads an SM where four
// vectors take two: 77 us at 2048 (spills).
template <int V, class IO>
__global__ void __launch_bounds__(512, V == 1 ? 4 : V == 2 ? 3 : V == 4 ? 2 : 1)
    act_row_kernel(const ActParams p) {
  pdl_enter();
  __shared__ float red[16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  const int64_t rows = act_rows(p);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    constexpr int B = V < 4 ? V : 4;  // vectors whose loads are in flight together
    uint4 y[V];
    float am = 0.f;
#pragma unroll
    for (int k0 = 0; k0 < V; k0 += B) {
      uint4 g[B], u[B];
      uint32_t skip = 0;
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int v = threadIdx.x + (k0 + k) * blockDim.x;
        const uint4* src = p.x + row * p.ldv + (v < p.nvec ? v : 0);
        if (v >= p.nvec) skip |= 0xFFu << (8 * k);
        g[k] = __ldg(src);
        u[k] = __ldg(src + p.nvec);
      }
      silu_mul_vecs<IO, B>(g, u, y + k0, p.x + row * p.ldv + threadIdx.x + k0 * blockDim.x,
                           blockDim.x, p.nvec, skip);
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int v = threadIdx.x + (k0 + k) * blockDim.x;
        if (v < p.nvec) {
          if (p.out_y) st_stream(p.out_y + row * p.nvec + v, y[k0 + k]);
          am = fmaxf(am, vec_absmax<IO>(y[k0 + k]));
        }
      }
    }
    am = warp_max(am);
    __syncthreads();
    if (lane == 0) red[warp] = am;
    __syncthreads();
    am = warp_max(lane < warps ? red[lane] : 0.f);
    const Fp8Scale s = fp8_scale_direct(am);
    if (threadIdx.x == 0) static_cast<float*>(p.out_scale)[row] = s.s;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int v = threadIdx.x + k * blockDim.x;
      quant_store<MODE_TOKEN, IO>(y[k], v < p.nvec, lane, row, v, p.nvec * 8, s, p.out_q,
                                  p.out_scale, p.scale_layout, p.scale_ld);
    }
  }
}

using ActKernel = void (*)(const ActParams);

}  // namespace fn
