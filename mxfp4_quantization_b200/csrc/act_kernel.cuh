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

// fp32 value of g u / (1 + e^-g), relative error below kSiluErr where it is used
// (g >= -87, |result| >= 2^-100).  e^-g = 2^t with t = -g log2(e) in two parts:
// the rounded product and its remainder, which scales the result by 1 + t_lo ln 2.
// Errors, in units of 2^-24: ex2.approx 4 (2^-22), the remainder's terms 1, their
// product 1, the sum 1 + e^-g 1 (and it passes on at most the 6 before), the
// approximate reciprocal 2, two products 2: 12 in all, below 2^-20.4.
constexpr float kSiluErr = 0x1p-20f;

__device__ __forceinline__ float silu_mul_fp32(float g, float u) {
  constexpr float kLog2e = 1.44269504088896340736f;
  constexpr float kLog2eLo = 1.92596299112661746887e-8f;  // log2(e) - kLog2e
  const float t = -g * kLog2e;
  const float lo = fmaf(-g, kLog2eLo, fmaf(-g, kLog2e, -t));
  float e, r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
  e = fmaf(e, lo * 0.693147180559945309417f, e);
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return (g * r) * u;  // g u alone can overflow where the result does not
}

// y of one element pair (gate word, up word).
template <class IO>
__device__ __forceinline__ uint32_t silu_mul_pair(uint32_t gw, uint32_t uw) {
  const float g0 = IO::lo(gw), g1 = IO::hi(gw), u0 = IO::lo(uw), u1 = IO::hi(uw);
  const float v0 = silu_mul_fp32(g0, u0), v1 = silu_mul_fp32(g1, u1);
  // the two ends of the interval that holds the real value round to one
  // 16-bit value unless a midpoint lies between them
  const uint32_t a = IO::pack(v0 * (1.f - kSiluErr), v1 * (1.f - kSiluErr));
  uint32_t y = IO::pack(v0 * (1.f + kSiluErr), v1 * (1.f + kSiluErr));
  // outside the interval's range (a zero is exact, or far below every 16-bit value)
  const bool far0 = !(g0 >= -87.f) || !(fabsf(v0) >= 0x1p-100f || v0 == 0.f),
             far1 = !(g1 >= -87.f) || !(fabsf(v1) >= 0x1p-100f || v1 == 0.f);
  if (((a ^ y) & 0xFFFFu) || far0) y = (y & 0xFFFF0000u) | silu_mul_fp64<IO>(g0, u0);
  if (((a ^ y) >> 16) || far1) y = (y & 0xFFFFu) | silu_mul_fp64<IO>(g1, u1) << 16;
  return y;
}

template <class IO>
__device__ __forceinline__ uint4 silu_mul_vec(const uint4& g, const uint4& u) {
  return make_uint4(silu_mul_pair<IO>(g.x, u.x), silu_mul_pair<IO>(g.y, u.y),
                    silu_mul_pair<IO>(g.z, u.z), silu_mul_pair<IO>(g.w, u.w));
}

__device__ __forceinline__ int64_t act_rows(const ActParams& p) {
  if (p.num_rows == nullptr) return p.M;
  const int64_t n = *p.num_rows;
  return n < 0 ? 0 : n < p.M ? n : p.M;
}

// Group modes (MXFP4, FP8 per 128): a thread per 8-element vector of the rows
// laid end to end; groups are 4 or 16 neighbouring lanes.
template <int MODE, class IO>
__global__ void __launch_bounds__(256) act_groups_kernel(const ActParams p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t total = act_rows(p) * p.nvec;
  for (int64_t i0 = (int64_t)blockIdx.x * blockDim.x; i0 < total;
       i0 += (int64_t)gridDim.x * blockDim.x) {
    const int64_t i = i0 + threadIdx.x;
    const bool ok = i < total;
    const int64_t row = ok ? i / p.nvec : 0;
    const int v = ok ? (int)(i - row * p.nvec) : 0;
    uint4 y = make_uint4(0, 0, 0, 0);
    if (ok) {
      const uint4* src = p.x + row * p.ldv + v;
      y = silu_mul_vec<IO>(ld_stream_nc(src), ld_stream_nc(src + p.nvec));
      if (p.out_y) st_stream(p.out_y + row * p.nvec + v, y);
    }
    quant_store<MODE, IO>(y, ok, lane, row, v, p.nvec * 8, Fp8Scale{1.f, 1.f, 0.f, false},
                          p.out_q, p.out_scale, p.scale_layout, p.scale_ld);
  }
}

// Per-token mode: a block per row, the row in registers (V vectors a thread)
// between the maximum and the codes.
template <int V, class IO>
__global__ void __launch_bounds__(1024) act_row_kernel(const ActParams p) {
  pdl_enter();
  __shared__ float red[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  const int64_t rows = act_rows(p);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    uint4 y[V];
    float am = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int v = threadIdx.x + k * blockDim.x;
      y[k] = make_uint4(0, 0, 0, 0);
      if (v < p.nvec) {
        const uint4* src = p.x + row * p.ldv + v;
        y[k] = silu_mul_vec<IO>(ld_stream_nc(src), ld_stream_nc(src + p.nvec));
        if (p.out_y) st_stream(p.out_y + row * p.nvec + v, y[k]);
        am = fmaxf(am, vec_absmax<IO>(y[k]));
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
