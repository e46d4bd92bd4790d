// Product of MXFP4 operands on the block-scaled tensor cores, sm_100a.
//
//   out[r, f] = round( sum_g 2^(sx[r,g] + sw[f,g] - 254) sum_{k in g} X[r,k] W[f,k] )
//
// with groups g of 32 elements, E2M1 values X and W, E8M0 bytes sx and sw, the
// sums in fp32 in tensor memory and one rounding to the output type.
//
// The weights are the M side of the MMA (128 features a tile), the token rows
// the N side (up to TOK rows a tile, cut at run time to the rows that are
// there, in steps of 16): a tile of few rows costs few MMA columns, whether the
// call has one row or an expert's row range ends inside a tile.  A feature is
// then a TMEM lane and a row a TMEM column.
//
// One persistent block per SM, one role per warp:
//   warp 0      TMA: the weight tile and the row tile of each K step of 256
//               elements (128 bytes a row, 128-byte swizzle); rows by index
//               with gather4
//   warp 1      one thread issues per K step the copies of the scales to TMEM
//               and the four 64-element MMAs
//   warps 2, 3  the scales of the rows / of the weights, brought to the
//               512-byte tiles that the copies read (a row's scales are a few
//               bytes at any offset, below what a TMA box can fetch)
//   warps 4-7   epilogue: TMEM to registers, rounding, stores
#pragma once
#include "fn_device.cuh"
#include "mg_params.h"
#include "tc_device.cuh"

namespace fn {

template <int TOK>
struct MGShape {
  static constexpr int kXBlocks = (TOK + 127) / 128;  // 512-byte scale tiles per 128 elements
  static constexpr int kWBytes = kMgFeat * 128;
  static constexpr int kXBytes = TOK * 128;
  static constexpr int kSwBytes = 2 * 512;
  static constexpr int kSxBytes = 2 * 512 * kXBlocks;
  static constexpr int kStage = kWBytes + kXBytes + kSwBytes + kSxBytes;
  static constexpr int kStages = TOK >= 256 ? 4 : TOK >= 128 ? 6 : TOK >= 64 ? 8 : 10;
  static constexpr int kAcc = TOK <= 128 ? 2 : 1;  // accumulators in TMEM
  static constexpr int kColSw = kAcc * TOK;        // TMEM columns of the scales
  static constexpr int kColSx = kColSw + 8;
  static constexpr int kColEnd = kColSx + 8 * kXBlocks;
  static constexpr int kCols = kColEnd <= 64 ? 64 : kColEnd <= 128 ? 128 : kColEnd <= 256 ? 256 : 512;
  // 1024 bytes: the operand tiles' alignment
  static constexpr int kSmem = kStages * kStage + 1024;
};

struct MGTile {
  int e, f0, row0, n;
};

// The tiles in order: expert, then feature tile, then row tile (the row tiles
// that share a weight tile are next to each other).  Every role walks the same
// sequence blockIdx.x, blockIdx.x + gridDim.x, ...
template <int TOK>
struct MGTiles {
  const int* cum;  // [E + 1] tiles before expert e   (offsets given)
  const int* lo;   // [E] first row
  const int* cnt;  // [E] rows
  int t, e, total, feat, M;

  __device__ MGTiles(const MGParams& p, const int* table)
      : cum(table), lo(table + p.E + 1), cnt(table + 2 * p.E + 1), t(blockIdx.x), e(0), M(p.M) {
    feat = (p.N + kMgFeat - 1) / kMgFeat;
    total = p.offsets ? cum[p.E] : feat * ((M + TOK - 1) / TOK);
    if (!p.offsets) cum = nullptr;
  }
  __device__ bool next(MGTile& o) {
    if (t >= total) return false;
    int rel = t, rows = M, first = 0;
    if (cum) {
      while (t >= cum[e + 1]) ++e;
      rel = t - cum[e];
      rows = cnt[e];
      first = lo[e];
    }
    const int nt = (rows + TOK - 1) / TOK;
    const int f = rel / nt, m = rel - f * nt;
    o.e = e;
    o.f0 = f * kMgFeat;
    o.row0 = first + m * TOK;
    o.n = min(TOK, rows - m * TOK);
    t += gridDim.x;
    return true;
  }
};

// Row range [lo, lo + cnt) of expert e, kept inside [0, M) whatever the
// offsets hold.
__device__ __forceinline__ void mg_range(const MGParams& p, int e, int* lo, int* cnt) {
  const int a = min(max(p.offsets[e], 0), p.M), b = min(max(p.offsets[e + 1], 0), p.M);
  *lo = a;
  *cnt = max(b - a, 0);
}

// The 32-bit scale word (groups 4 kt .. 4 kt + 3) of a row, zeros past the last
// group, by byte loads: rows whose words are not aligned, and the last word of
// a row with a number of groups that is no multiple of 4.
__device__ __forceinline__ uint32_t mg_scale_word(const uint8_t* base, int64_t row, int kt,
                                                  int groups, int swizzled) {
  const int kts = (groups + 3) >> 2;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int g = kt * 4 + i;
    if (g < groups) {
      const int64_t at = swizzled ? ((row >> 7) * kts + kt) * 512 + (row & 31) * 16 +
                                        ((row >> 5) & 3) * 4 + i
                                  : row * groups + g;
      w |= (uint32_t)base[at] << (8 * i);
    }
  }
  return w;
}

template <int TOK>
__global__ void __launch_bounds__(kMgThreads, 1)
    mg_kernel(const __grid_constant__ MGParams p, const __grid_constant__ CUtensorMap x_map,
              const __grid_constant__ CUtensorMap w_map) {
  using S = MGShape<TOK>;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[3 * S::kStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t stop;

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const uint32_t tiles0 = (smem_addr(dyn) + 1023) & ~1023u;
  int* table = reinterpret_cast<int*>(dyn + (tiles0 - smem_addr(dyn)) + S::kStages * S::kStage);
  const uint32_t full = smem_addr(bars), sfull = full + 8 * S::kStages,
                 empty = sfull + 8 * S::kStages, tfull = empty + 8 * S::kStages,
                 tempty = tfull + 16, drain = tempty + 16;
  auto w_tile = [&](int s) { return tiles0 + s * (S::kWBytes + S::kXBytes); };
  auto x_tile = [&](int s) { return w_tile(s) + S::kWBytes; };
  const uint32_t scales0 = tiles0 + S::kStages * (S::kWBytes + S::kXBytes);
  auto sw_tile = [&](int s) { return scales0 + s * (S::kSwBytes + S::kSxBytes); };
  auto sx_tile = [&](int s) { return sw_tile(s) + S::kSwBytes; };

  if (threadIdx.x == 0) {
    stop = 0;
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(sfull + 8 * s, 2);
      mbar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + 8 * b, 1);
      mbar_init(tempty + 8 * b, 4);
    }
    mbar_init(drain, 1);
    fence_async_smem();
    tma_prefetch_map(&x_map);
    tma_prefetch_map(&w_map);
  }
  if (warp == 3) tmem_alloc(smem_addr(&tmem_slot), S::kCols);
  pdl_enter();
  if (p.offsets && warp == 0) {
    // tiles before each expert: a running sum over 32 experts at a time
    int* cum = table;
    int* lo = table + p.E + 1;
    int* cnt = table + 2 * p.E + 1;
    const int feat = (p.N + kMgFeat - 1) / kMgFeat;
    int before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      int a = 0, c = 0;
      if (e0 + lane < p.E) {
        mg_range(p, e0 + lane, &a, &c);
        lo[e0 + lane] = a;
        cnt[e0 + lane] = c;
      }
      int sum = feat * ((c + TOK - 1) / TOK);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (e0 + lane < p.E) cum[e0 + lane + 1] = before + sum;
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) cum[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int steps = (p.K + kMgStageK - 1) / kMgStageK;
  MGTiles<TOK> tiles(p, table);
  MGTile t;

  if (warp == 0) {
    // ---- operands -----------------------------------------------------------------------
    int s = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (ok && tiles.next(t)) {
      const int wrow = t.e * p.N + t.f0;
      int4 src[(TOK + 127) / 128];
      if (p.rows) {
#pragma unroll
        for (int b = 0; b < (TOK + 127) / 128; ++b) {
          int r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // rows past the tile's end and indices outside the operand fetch row 0
            const int j = (b * 32 + lane) * 4 + i;
            const int v = j < t.n ? p.rows[t.row0 + j] : 0;
            r[i] = (unsigned)v < (unsigned)p.x_rows ? v : 0;
          }
          src[b] = make_int4(r[0], r[1], r[2], r[3]);
        }
      }
      const int pieces = p.rows ? (t.n + 3) / 4 : (t.n + p.box - 1) / p.box;
      const uint32_t bytes = S::kWBytes + (uint32_t)pieces * (p.rows ? 4 : p.box) * 128;
      for (int kb = 0; kb < steps; ++kb) {
        ok = mbar_wait(empty + 8 * s, ph ^ 1, &stop);
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(full + 8 * s, bytes);
          tma_load(w_tile(s), &w_map, kb * 128, wrow, full + 8 * s);
        }
        __syncwarp();
        if (p.rows) {
#pragma unroll
          for (int b = 0; b < (TOK + 127) / 128; ++b)
            if (b * 32 + lane < pieces)
              tma_gather4(x_tile(s) + (b * 32 + lane) * 512, &x_map, kb * 128, src[b].x, src[b].y,
                          src[b].z, src[b].w, full + 8 * s);
        } else if (lane < pieces) {
          tma_load(x_tile(s) + lane * p.box * 128, &x_map, kb * 128, t.row0 + lane * p.box,
                   full + 8 * s);
        }
        ++issued;
        if (++s == S::kStages) s = 0, ph ^= 1;
      }
    }
    if (!ok) {  // the copies in flight land before the block goes
      for (int i = 0; i < min(issued, S::kStages); ++i) {
        if (--s < 0) s = S::kStages - 1, ph ^= 1;
        for (int n = 0; n < kWaitTries && !mbar_try(full + 8 * s, ph); ++n) {
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA ----------------------------------------------------------------------------
    if (lane == 0) {
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      while (ok && tiles.next(t)) {
        const uint32_t d = tmem + acc * TOK;
        const int n16 = (t.n + 15) / 16 * 16;
        const uint32_t id0 = mxf4_idesc(kMgFeat, n16, 0), id1 = mxf4_idesc(kMgFeat, n16, 1);
        ok = mbar_wait(tempty + 8 * acc, aph ^ 1, &stop);
        tc_fence_after();
        for (int kb = 0; ok && kb < steps; ++kb) {
          ok = mbar_wait(sfull + 8 * s, ph, &stop) && mbar_wait(full + 8 * s, ph, &stop);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            tc_copy_scales(tmem + S::kColSw + 4 * i, scale_desc(sw_tile(s) + 512 * i));
#pragma unroll
            for (int b = 0; b < S::kXBlocks; ++b)
              tc_copy_scales(tmem + S::kColSx + 4 * (i * S::kXBlocks + b),
                             scale_desc(sx_tile(s) + 512 * (i * S::kXBlocks + b)));
          }
          const uint64_t a = operand_desc(w_tile(s)), b = operand_desc(x_tile(s));
          const int mmas = min(4, (p.K - kb * kMgStageK + 63) / 64);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < mmas)
              tc_mma_mxf4(d, a + 2 * j, b + 2 * j, j & 1 ? id1 : id0,
                          tmem + S::kColSw + 4 * (j / 2),
                          tmem + S::kColSx + 4 * S::kXBlocks * (j / 2), kb > 0 || j > 0);
          tc_commit(empty + 8 * s);
          if (++s == S::kStages) s = 0, ph ^= 1;
        }
        if (ok) tc_commit(tfull + 8 * acc);
        if (++acc == S::kAcc) acc = 0, aph ^= 1;
      }
      if (!ok) {  // MMAs in flight end before the block goes
        tc_commit(drain);
        for (int n = 0; n < kWaitTries && !mbar_try(drain, 0); ++n) {
        }
      }
    }
  } else if (warp < 4) {
    // ---- scales ---------------------------------------------------------------------------
    const bool is_x = warp == 2;
    const uint8_t* scale = is_x ? p.x_scale : p.w_scale;
    const int swz = is_x ? p.x_swizzled : p.w_swizzled;
    const int kts = (p.groups + 3) >> 2;
    const bool words = swz || (p.groups % 4 == 0 && (reinterpret_cast<uintptr_t>(scale) & 3) == 0);
    constexpr int RX = (TOK + 31) / 32;
    constexpr int kAhead = 3;  // stages whose copies are in flight
    int s = 0, as = 0, pending = 0;
    uint32_t ph = 0;
    bool ok = true;
    auto arrive = [&] {
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(sfull + 8 * as);
      if (++as == S::kStages) as = 0;
      --pending;
    };
    while (ok && tiles.next(t)) {
      const uint8_t* base = is_x ? scale : scale + t.e * p.w_scale_stride;
      int64_t row[RX > 4 ? RX : 4];
      bool in[RX > 4 ? RX : 4];
#pragma unroll
      for (int i = 0; i < (RX > 4 ? RX : 4); ++i) {
        const int j = i * 32 + lane;
        if (is_x) {
          in[i] = j < t.n;
          int v = t.row0 + j;
          if (p.rows && in[i]) {
            v = p.rows[v];
            in[i] = (unsigned)v < (unsigned)p.x_rows;
          }
          row[i] = in[i] ? v : 0;
        } else {
          in[i] = i < 4 && t.f0 + j < p.N;
          row[i] = in[i] ? t.f0 + j : 0;
        }
      }
      for (int kb = 0; kb < steps; ++kb) {
        ok = mbar_wait(empty + 8 * s, ph ^ 1, &stop);
        if (!ok) break;
        const uint32_t dst0 = is_x ? sx_tile(s) : sw_tile(s);
        const bool fast = words && (kb * 8 + 8 <= p.groups || p.groups % 4 == 0);
#pragma unroll
        for (int i = 0; i < (RX > 4 ? RX : 4); ++i) {
          if (i >= (is_x ? RX : 4)) continue;
          const int nblk = is_x ? S::kXBlocks : 1;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int kt = kb * 2 + h;
            const uint32_t dst = dst0 + (h * nblk + i / 4) * 512 + lane * 16 + (i & 3) * 4;
            if (fast) {
              const bool have = in[i] && kt < kts;
              const int64_t at = swz ? ((row[i] >> 7) * kts + kt) * 512 + (row[i] & 31) * 16 +
                                           ((row[i] >> 5) & 3) * 4
                                     : row[i] * p.groups + kt * 4;
              cp_async4(dst, have ? base + at : base, have);
            } else {
              const uint32_t w = in[i] ? mg_scale_word(base, row[i], kt, p.groups, swz) : 0;
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst), "r"(w) : "memory");
            }
          }
        }
        cp_async_commit();
        if (++pending == kAhead) {
          cp_async_wait<kAhead - 1>();
          arrive();
        }
        if (++s == S::kStages) s = 0, ph ^= 1;
      }
    }
    cp_async_wait<0>();
    while (pending > 0) arrive();
  } else {
    // ---- epilogue ---------------------------------------------------------------------------
    const int quad = warp - 4;
    int acc = 0;
    uint32_t aph = 0;
    bool ok = true;
    while (tiles.next(t)) {
      if (ok) ok = mbar_wait(tfull + 8 * acc, aph, &stop);
      tc_fence_after();
      const int f = t.f0 + quad * 32 + lane;
      for (int c = 0; c < t.n; c += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + ((uint32_t)(quad * 32) << 16) + acc * TOK + c, v);
        tmem_wait_ld();
        uint32_t keep = 0xffffffffu;  // rows whose source index is inside the operand
        if (p.rows) {
          const int src = lane < 16 && c + lane < t.n ? p.rows[t.row0 + c + lane] : 0;
          keep = __ballot_sync(0xffffffffu, (unsigned)src < (unsigned)p.x_rows);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (c + i < t.n && f < p.N) {
            const float val = !ok ? __uint_as_float(0x7fffffffu)
                              : (keep >> i) & 1 ? __uint_as_float(v[i]) : 0.f;
            const int64_t at = (int64_t)(t.row0 + c + i) * p.ldo + f;
            if (p.out_type == MG_OUT_FP32)
              static_cast<float*>(p.out)[at] = val;
            else
              static_cast<uint16_t*>(p.out)[at] =
                  (uint16_t)(p.out_type == MG_OUT_BF16 ? pack_bf16x2(val, 0.f)
                                                       : pack_f16x2(val, 0.f));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty + 8 * acc);
      if (++acc == S::kAcc) acc = 0, aph ^= 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) tmem_dealloc(tmem, S::kCols);
}

}  // namespace fn
