// Product of MXFP4 operands on the block-scaled tensor cores, sm_100a.
//
//   out[r, f] = round( sum_g 2^(sx[r,g] + sw[f,g] - 254) sum_{k in g} X[r,k] W[f,k] )
//
// with groups g of 32 elements, E2M1 values X and W, E8M0 bytes sx and sw, the
// sums in fp32 in tensor memory and one rounding to the output type.
//
// The weights are the M side of the MMA (128 features a block), the token rows
// the N side (up to TOK rows a tile, cut at run time to the rows that are
// there, in steps of 16): a tile of few rows costs few MMA columns, whether the
// call has one row or an expert's row range ends inside a tile.  A feature is
// then a TMEM lane and a row a TMEM column.
//
// CG = 2: a cluster of two blocks shares a tile of 256 features (cta_group::2).
// Each block holds 128 features and half of the rows' codes, so an operand
// byte in shared memory feeds twice the products: a 128 x 256 tile of one
// block would need 12 KB of reads and 12 KB of fills per 128-cycle MMA, above
// what shared memory gives, the pair's blocks 8 KB and 8 KB each.
//
// Persistent blocks, one role per warp:
//   warp 0      TMA: the weight tile and the row tile of each K step of 256
//               elements (128 bytes a row, 128-byte swizzle; rows by index
//               with gather4), and scales that are in the 32x4x4 tiling
//   warp 1      one thread (of the pair's first block) issues per K step the
//               copies of the scales to TMEM and the four 64-element MMAs
//   warps 2-4   scales that are row-major (2, 3: the rows', 128 each; 4: the
//               weights'): a row's scales are a few bytes at any offset, below
//               what a TMA box can fetch.  They come as 16-byte vectors, two K
//               steps at once and two fetches ahead, and leave as the 512-byte
//               tiles that the copies to TMEM read
//   warps 5-8   epilogue: TMEM to registers, rounding, stores
#pragma once
#include "fn_device.cuh"
#include "mg_params.h"
#include "tc_device.cuh"

namespace fn {

template <int TOK, int CG>
struct MGShape {
  static constexpr int kXBlocks = (TOK + 127) / 128;  // 512-byte scale tiles per 128 elements
  static constexpr int kXRows = TOK / CG;             // rows' codes in one block
  static constexpr int kWBytes = kMgFeat * 128;
  static constexpr int kXBytes = kXRows * 128;
  static constexpr int kSwBytes = 2 * 512;
  static constexpr int kSxBytes = 2 * 512 * kXBlocks;
  static constexpr int kStage = kWBytes + kXBytes + kSwBytes + kSxBytes;
  static constexpr int kStages = kXRows >= 128 ? 6 : kXRows >= 64 ? 8 : 10;
  // Two accumulators in TMEM.  For 256 rows they overlap, or no columns would be
  // left for the scales: the epilogue drains the shared columns first, and the
  // next tile's MMAs start then.
  static constexpr bool kOverlap = TOK == 256;
  static constexpr int kAcc1 = kOverlap ? 232 : TOK;
  static constexpr int kColSw = kAcc1 + TOK;
  static constexpr int kColSx = kColSw + 8;
  static constexpr int kColEnd = kColSx + 8 * kXBlocks;
  static constexpr int kCols = kColEnd <= 64 ? 64 : kColEnd <= 128 ? 128 : kColEnd <= 256 ? 256 : 512;
  static_assert(kColEnd <= 512, "tensor memory");
  static constexpr int kChunk = TOK >= 32 ? 32 : 16;  // columns the epilogue takes at once
  // 1024 bytes: the operand tiles' alignment
  static constexpr int kSmem = kStages * kStage + 1024;
};

struct MGTile {
  int e, f0, row0, n;
};

// The tiles in order: expert, then feature tile, then row tile (the row tiles
// that share a weight tile are next to each other).  Every role walks the same
// sequence: the cluster's index, then one cluster grid further each time.
template <int TOK, int CG>
struct MGTiles {
  const int* cum;  // [E + 1] tiles before expert e   (offsets given)
  const int* lo;   // [E] first row
  const int* cnt;  // [E] rows
  int t, e, total, M;

  __device__ MGTiles(const MGParams& p, const int* table)
      : cum(table), lo(table + p.E + 1), cnt(table + 2 * p.E + 1), t(blockIdx.x / CG), e(0),
        M(p.M) {
    const int feat = (p.N + CG * kMgFeat - 1) / (CG * kMgFeat);
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
    o.f0 = f * CG * kMgFeat;
    o.row0 = first + m * TOK;
    o.n = min(TOK, rows - m * TOK);
    t += gridDim.x / CG;
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

// Stores `n` rows (of at most C) of a chunk; the lane holds feature f.
template <int C>
__device__ __forceinline__ void mg_store(const MGParams& p, uint32_t (&v)[C], int64_t row, int n,
                                         int f, int lane) {
  if (p.out_type == MG_OUT_FP32) {
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
#pragma unroll
    for (int i = 0; i < C; i += 4) {
      if (i >= n) break;
      const float a = __uint_as_float(v[i]), b = __uint_as_float(v[i + 1]),
                  c = __uint_as_float(v[i + 2]), d = __uint_as_float(v[i + 3]);
      const uint2 w = bf ? mg_transpose4(pack_bf16x2(a, b), pack_bf16x2(c, d), lane)
                         : mg_transpose4(pack_f16x2(a, b), pack_f16x2(c, d), lane);
      if (i + (lane & 3) < n && quad < p.N)
        *reinterpret_cast<uint2*>(o + i * p.ldo) = w;
    }
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

template <int TOK, int CG>
__global__ void __launch_bounds__(kMgThreads, 1)
    mg_kernel(const __grid_constant__ MGParams p, const __grid_constant__ MGMaps maps) {
  using S = MGShape<TOK, CG>;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[3 * S::kStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t stop;

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : cluster_rank();
  const uint32_t tiles0 = (smem_addr(dyn) + 1023) & ~1023u;
  int* table = reinterpret_cast<int*>(dyn + (tiles0 - smem_addr(dyn)) + S::kStages * S::kStage);
  const uint32_t full = smem_addr(bars), sfull = full + 8 * S::kStages,
                 empty = sfull + 8 * S::kStages, tfull = empty + 8 * S::kStages,
                 tempty = tfull + 16, drain = tempty + 16;
  auto w_tile = [&](int s) { return tiles0 + s * (S::kWBytes + S::kXBytes); };
  auto x_tile = [&](int s) { return w_tile(s) + S::kWBytes; };
  const uint32_t scales0 = tiles0 + S::kStages * (S::kWBytes + S::kXBytes);
  auto sw_tile = [&](int s) { return scales0 + s * (S::kSwBytes + S::kSxBytes); };
  // per 128 rows: the tiles of the step's two halves
  auto sx_tile = [&](int s) { return sw_tile(s) + S::kSwBytes; };
  // barriers that the MMA thread waits on live in the pair's first block
  auto first = [&](uint32_t bar) { return CG == 1 ? bar : cluster_map(bar, 0); };
  auto arrive_first = [&](uint32_t bar) {
    if constexpr (CG == 1)
      mbar_arrive(bar);
    else
      mbar_arrive_cluster(cluster_map(bar, 0));
  };
  const int scale_warps = (p.x_mode != MG_SCALE_TMA ? S::kXBlocks : 0) + (p.w_mode != MG_SCALE_TMA);

  if (threadIdx.x == 0) {
    stop = 0;
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(sfull + 8 * s, max(1, scale_warps * CG));
      mbar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + 8 * b, 1);
      mbar_init(tempty + 8 * b, 4 * CG);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    tma_prefetch_map(&maps.x);
    tma_prefetch_map(&maps.w);
  }
  if (warp == 1) tmem_alloc<CG>(smem_addr(&tmem_slot), S::kCols);
  pdl_enter();
  if (p.offsets && warp == 0) {
    // tiles before each expert: a running sum over 32 experts at a time
    int* cum = table;
    int* lo = table + p.E + 1;
    int* cnt = table + 2 * p.E + 1;
    const int feat = (p.N + CG * kMgFeat - 1) / (CG * kMgFeat);
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
  if constexpr (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int steps = (p.K + kMgStageK - 1) / kMgStageK;
  const int kts = (p.groups + 3) >> 2;
  MGTiles<TOK, CG> tiles(p, table);
  MGTile t;

  if (warp == 0) {
    // ---- operands -----------------------------------------------------------------------
    int s = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    constexpr int G = (S::kXRows + 127) / 128;
    while (ok && tiles.next(t)) {
      const int f0 = t.f0 + (int)rank * kMgFeat;
      const int wrow = t.e * p.N + f0;
      const int half = (t.n + 15) / 16 * 16 / CG;  // rows' codes of this block
      const int x0 = (int)rank * half;             // first of them in the tile
      int4 src[G];
      if (p.rows) {
#pragma unroll
        for (int b = 0; b < G; ++b) {
          int r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // rows past the tile's end and indices outside the operand fetch row 0
            const int j = x0 + (b * 32 + lane) * 4 + i;
            const int v = j < t.n ? p.rows[t.row0 + j] : 0;
            r[i] = (unsigned)v < (unsigned)p.x_rows ? v : 0;
          }
          src[b] = make_int4(r[0], r[1], r[2], r[3]);
        }
      }
      const int each = p.rows ? 4 : p.box;
      const int pieces = (half + each - 1) / each;
      const uint32_t codes = CG * (S::kWBytes + (uint32_t)(pieces * each) * 128);
      const int64_t ws0 = (int64_t)t.e * (p.w_scale_stride / 512) + (int64_t)(f0 / 128) * kts;
      const int64_t xs0 = (int64_t)(t.row0 / 128) * kts;
      for (int kb = 0; kb < steps; ++kb) {
        ok = mbar_wait<CG>(empty + 8 * s, ph ^ 1, &stop);
        if (!ok) break;
        const bool last = kb == steps - 1;
        const bool tw = p.w_mode == MG_SCALE_TMA || (p.w_mode == MG_SCALE_TMA_TAIL && !last);
        const bool tx = p.x_mode == MG_SCALE_TMA || (p.x_mode == MG_SCALE_TMA_TAIL && !last);
        const uint32_t bar = first(full + 8 * s);
        if (lane == 0) {
          if (rank == 0)
            mbar_expect_tx(full + 8 * s,
                           codes + CG * ((tw ? S::kSwBytes : 0) + (tx ? S::kSxBytes : 0)));
          tma_load<CG>(w_tile(s), &maps.w, kb * 128, wrow, bar);
          if (tw) tma_load<CG>(sw_tile(s), &maps.ws, 0, (int)(ws0 + 2 * kb), bar);
          if (tx) {
#pragma unroll
            for (int b = 0; b < S::kXBlocks; ++b)
              tma_load<CG>(sx_tile(s) + 1024 * b, &maps.xs, 0,
                           (int)(xs0 + (int64_t)b * kts + 2 * kb), bar);
          }
        }
        __syncwarp();
        if (p.rows) {
#pragma unroll
          for (int b = 0; b < G; ++b)
            if (b * 32 + lane < pieces)
              tma_gather4<CG>(x_tile(s) + (b * 32 + lane) * 512, &maps.x, kb * 128, src[b], bar);
        } else if (lane < pieces) {
          tma_load<CG>(x_tile(s) + lane * p.box * 128, &maps.x, kb * 128,
                       t.row0 + x0 + lane * p.box, bar);
        }
        ++issued;
        if (++s == S::kStages) s = 0, ph ^= 1;
      }
    }
    // the last MMAs' arrivals on this block's barriers come before it goes
    for (int i = 0; ok && i < min(issued, S::kStages); ++i) {
      ok = mbar_wait<CG>(empty + 8 * s, ph ^ 1, &stop);
      if (++s == S::kStages) s = 0, ph ^= 1;
    }
    if (!ok && rank == 0) {  // the copies in flight land before the blocks go
      for (int i = 0; i < min(issued, S::kStages); ++i) {
        if (--s < 0) s = S::kStages - 1, ph ^= 1;
        for (int n = 0; n < kWaitTries && !mbar_try<CG>(full + 8 * s, ph); ++n) {
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA ----------------------------------------------------------------------------
    if (lane == 0 && rank == 0) {
      int s = 0, i = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (; ok && tiles.next(t); ++i) {
        const int acc = i & 1;
        const uint32_t d = tmem + (acc ? S::kAcc1 : 0);
        const int n16 = (t.n + 15) / 16 * 16;
        const uint32_t id0 = mxf4_idesc(CG * kMgFeat, n16, 0), id1 = mxf4_idesc(CG * kMgFeat, n16, 1);
        // overlapping accumulators: the shared columns of the tile before are
        // drained (and all of the one before that); else this accumulator is
        ok = S::kOverlap ? mbar_wait<CG>(tempty, (i & 1) ^ 1, &stop)
                         : mbar_wait<CG>(tempty + 8 * acc, ((i >> 1) & 1) ^ 1, &stop);
        tc_fence_after();
        for (int kb = 0; ok && kb < steps; ++kb) {
          ok = mbar_wait<CG>(full + 8 * s, ph, &stop) &&
               (scale_warps == 0 || mbar_wait<CG>(sfull + 8 * s, ph, &stop));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tc_copy_scales<CG>(tmem + S::kColSw + 4 * h, scale_desc(sw_tile(s) + 512 * h));
#pragma unroll
            for (int b = 0; b < S::kXBlocks; ++b)
              tc_copy_scales<CG>(tmem + S::kColSx + 4 * (h * S::kXBlocks + b),
                                 scale_desc(sx_tile(s) + 512 * (2 * b + h)));
          }
          const uint64_t a = operand_desc(w_tile(s)), b = operand_desc(x_tile(s));
          const int mmas = min(4, (p.K - kb * kMgStageK + 63) / 64);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < mmas)
              tc_mma_mxf4<CG>(d, a + 2 * j, b + 2 * j, j & 1 ? id1 : id0,
                              tmem + S::kColSw + 4 * (j / 2),
                              tmem + S::kColSx + 4 * S::kXBlocks * (j / 2), kb > 0 || j > 0);
          tc_commit<CG>(empty + 8 * s);
          if (++s == S::kStages) s = 0, ph ^= 1;
        }
        if (ok) tc_commit<CG>(tfull + 8 * acc);
      }
      if (!ok) {  // MMAs in flight end before the blocks go
        tc_commit<CG>(drain);
        for (int n = 0; n < kWaitTries && !mbar_try<CG>(drain, 0); ++n) {
        }
      }
    }
  } else if (warp < 5) {
    // ---- scales ---------------------------------------------------------------------------
    const bool is_x = warp < 4;
    const int mode = is_x ? p.x_mode : p.w_mode;
    if (mode != MG_SCALE_TMA && (!is_x || warp - 2 < S::kXBlocks)) {
      const bool wide = is_x ? p.x_wide : p.w_wide;
      const int blk = is_x ? warp - 2 : 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      while (ok && tiles.next(t)) {
        const uint8_t* base = is_x ? p.x_scale : p.w_scale + t.e * p.w_scale_stride;
        const uint8_t* src[4];
        int64_t row[4];
        bool in[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = blk * 128 + i * 32 + lane;
          if (is_x) {
            in[i] = j < t.n;
            int v = t.row0 + j;
            if (p.rows && in[i]) {
              v = p.rows[v];
              in[i] = (unsigned)v < (unsigned)p.x_rows;
            }
            row[i] = in[i] ? v : 0;
          } else {
            const int f = t.f0 + (int)rank * kMgFeat + j;
            in[i] = f < p.N;
            row[i] = in[i] ? f : 0;
          }
          src[i] = base + row[i] * p.groups;
        }
        auto fetch = [&](uint4 (&b)[4], int c) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            b[i] = !in[i] || 2 * c >= steps ? make_uint4(0, 0, 0, 0)
                   : mode == MG_SCALE_WARP  ? mg_scales(src[i], c, p.groups, wide)
                   : 2 * c + 2 >= steps     ? mg_tiled_scales(base, row[i], c, p.groups)
                                            : make_uint4(0, 0, 0, 0);
        };
        uint4 b0[4], b1[4], b2[4];
        fetch(b0, 0);
        fetch(b1, 1);
        for (int c = 0; 2 * c < steps; ++c) {
          fetch(b2, c + 2);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int kb = 2 * c + h;
            if (kb < steps && ok) {
              ok = mbar_wait<CG>(empty + 8 * s, ph ^ 1, &stop);
              if (ok && (mode == MG_SCALE_WARP || kb == steps - 1)) {
                const uint32_t dst =
                    (is_x ? sx_tile(s) + 1024 * blk : sw_tile(s)) + lane * 16;
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 512 * k),
                               "r"(word(b0[0], 2 * h + k)), "r"(word(b0[1], 2 * h + k)),
                               "r"(word(b0[2], 2 * h + k)), "r"(word(b0[3], 2 * h + k))
                               : "memory");
                fence_async_smem();
              }
              __syncwarp();
              if (ok && lane == 0) arrive_first(sfull + 8 * s);
              if (++s == S::kStages) s = 0, ph ^= 1;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) b0[i] = b1[i], b1[i] = b2[i];
        }
      }
    }
  } else {
    // ---- epilogue ---------------------------------------------------------------------------
    const int quad = warp & 3;  // the TMEM lanes a warp can read
    constexpr int C = S::kChunk;
    bool ok = true;
    for (int i = 0; tiles.next(t); ++i) {
      const int acc = i & 1;
      if (ok) ok = mbar_wait<CG>(tfull + 8 * acc, (i >> 1) & 1, &stop);
      tc_fence_after();
      const int f = t.f0 + (int)rank * kMgFeat + quad * 32 + lane;
      const uint32_t src = tmem + ((uint32_t)(quad * 32) << 16) + (acc ? S::kAcc1 : 0);
      const int chunks = (t.n + C - 1) / C;
      // the chunk with the columns that both accumulators use goes first
      const int lead = S::kOverlap && acc == 0 && chunks == TOK / C ? chunks - 1 : 0;
      const bool free_now = S::kOverlap && acc == 0 && lead == 0;  // not in use by this tile
      auto release = [&](int b) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(tempty + 8 * b);
      };
      if (free_now) release(0);
      for (int k = 0; k < chunks; ++k) {
        const int c = lead == 0 ? k : k == 0 ? lead : k - 1;
        uint32_t v[C];
        tmem_ld(src + c * C, v);
        tmem_wait_ld();
        if (S::kOverlap && k == 0 && !free_now) release(0);
        if (!ok) {
#pragma unroll
          for (int q = 0; q < C; ++q) v[q] = 0x7fffffffu;
        } else if (p.rows) {  // rows whose source index is outside the operand are zero
          const int j = c * C + lane;
          const int r = lane < C && j < t.n ? p.rows[t.row0 + j] : 0;
          const uint32_t keep = __ballot_sync(0xffffffffu, (unsigned)r < (unsigned)p.x_rows);
          if (keep != 0xffffffffu) {
#pragma unroll
            for (int q = 0; q < C; ++q)
              if (!((keep >> q) & 1)) v[q] = 0;
          }
        }
        mg_store<C>(p, v, (int64_t)t.row0 + c * C, min(C, t.n - c * C), f, lane);
      }
      if (!S::kOverlap) release(acc);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  if (warp == 1) tmem_dealloc<CG>(tmem, S::kCols);
}

}  // namespace fn
