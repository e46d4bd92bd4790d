// Weighted sum of expert rows in token order, sm_100a: out[t] = round16(base[t] +
// sum_j w[t,j] y[pos[t,j]]), fp32, j ascending.
#pragma once
#include "fn_device.cuh"

namespace fn {

struct CombineParams {
  const void* y;
  const int32_t* pos;
  const float* weight;
  const void* base;  // or nullptr; may be out
  void* out;
  int64_t R, T;
  int k, n;          // n: vectors (wide) or elements (narrow) of a row
  int per_row;       // blocks of a row
};

// Bound by memory: k rows read, one written.  B choices' rows are in flight together;
// four, or two where there are no more (more registers then only cost blocks
// an SM).  4096 tokens x 8 rows of 7168: 78 us (6.7 TB/s, part of it from L2)
// with four, 80 with two, 85 with eight or with each load behind its position;
// 1024 x 2 of 8192: 8.5 us with two, 10.3 with four.
template <class IO, int kCombineBatch>
__global__ void __launch_bounds__(256) combine_kernel(const CombineParams p) {
  pdl_enter();
  const int64_t t = blockIdx.x / p.per_row;
  const int v = (int)(blockIdx.x % p.per_row) * blockDim.x + threadIdx.x;
  if (v >= p.n) return;
  const uint4* y = static_cast<const uint4*>(p.y);
  float2 a[4] = {};
  if (p.base) {
    const uint4 b = ld_stream(static_cast<const uint4*>(p.base) + t * p.n + v);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = make_float2(IO::lo(word(b, i)), IO::hi(word(b, i)));
  }
  for (int j0 = 0; j0 < p.k; j0 += kCombineBatch) {
    int64_t r[kCombineBatch];
    float w[kCombineBatch];
    uint4 x[kCombineBatch];
#pragma unroll
    for (int j = 0; j < kCombineBatch; ++j) {
      r[j] = j0 + j < p.k ? p.pos[t * p.k + j0 + j] : -1;
      if (r[j] >= p.R) r[j] = -1;
    }
#pragma unroll
    for (int j = 0; j < kCombineBatch; ++j)
      if (r[j] >= 0) {
        w[j] = p.weight[t * p.k + j0 + j];
        x[j] = ld_stream_nc(y + r[j] * p.n + v);
      }
#pragma unroll
    for (int j = 0; j < kCombineBatch; ++j)
      if (r[j] >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = fma_f32x2(make_float2(w[j], w[j]),
                           make_float2(IO::lo(word(x[j], i)), IO::hi(word(x[j], i))), a[i]);
      }
  }
  st_stream(static_cast<uint4*>(p.out) + t * p.n + v,
            make_uint4(IO::pack(a[0].x, a[0].y), IO::pack(a[1].x, a[1].y),
                       IO::pack(a[2].x, a[2].y), IO::pack(a[3].x, a[3].y)));
}

// Rows that are not made of aligned 16-byte vectors: a thread per element, each
// choice's load behind its position's.  Bound by that latency and by instructions: 4096
// tokens x 8 rows of 7167 take 303 us (1.7 TB/s), 4 x 8 of them 2.3 us.
template <class IO>
__global__ void __launch_bounds__(256) combine_narrow_kernel(const CombineParams p) {
  pdl_enter();
  const int64_t t = blockIdx.x / p.per_row;
  const int v = (int)(blockIdx.x % p.per_row) * blockDim.x + threadIdx.x;
  if (v >= p.n) return;
  const uint16_t* y = static_cast<const uint16_t*>(p.y);
  float a = p.base ? IO::lo(static_cast<const uint16_t*>(p.base)[t * p.n + v]) : 0.f;
  for (int j = 0; j < p.k; ++j) {
    const int64_t r = p.pos[t * p.k + j];
    if (r < 0 || r >= p.R) continue;
    a = fmaf(p.weight[t * p.k + j], IO::lo(y[r * p.n + v]), a);
  }
  static_cast<uint16_t*>(p.out)[t * p.n + v] = (uint16_t)IO::pack(a, 0.f);
}

using CombineKernel = void (*)(const CombineParams);

}  // namespace fn
