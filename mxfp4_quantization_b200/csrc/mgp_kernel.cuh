// Product of MXFP4 operands over pairs of blocks, for calls of many rows, sm_100a.
//
// The mathematics and the operands' sides are those of mg_kernel.cuh.  A cluster
// of two blocks shares a tile of 256 features and up to 240 rows (cta_group::2):
// each block holds 128 features and half of the rows' codes, so an operand byte
// in shared memory feeds twice the products.  A 128 x 256 tile of one block needs
// 12 KB of reads and 12 KB of fills in the 128 cycles of an MMA, above what
// shared memory gives; the pair's blocks need 8 KB and 8 KB.
//
// TMEM: two accumulators of 240 columns and one K step's scales (24 columns).
// 256-row tiles leave room for two accumulators only if they overlap, and the
// next tile's first MMA then waits for the epilogue: 1.6 us a tile (*).
//
// All operands come by TMA.  Scales have to be 512-byte tiles aligned to the row
// tiles, which start anywhere (an expert's first row, a multiple of the tile
// height): mgp_arrange_kernel writes them to the workspace first, with zeros in
// the padding, and gathers the codes of rows given by index once instead of once
// per feature tile (with gather4 in the product itself, 32768 rows x 4096 features
// took 1140 us against 800 us without an index (*); 32 experts' 32768 gathered rows
// take 407 us, the same rows in place 390).
// Warps that fetched the row-major scales inside the product cost 60 us of 320
// (8192 x 8192 x 7168 (*)): their tiles pass a fence and a release to the other block
// in every K step.
//
// (*) Measured while the MMAs were still issued from a one-lane branch, which set the
// pace (251 us instead of 170); not measured again on this form.
//
// What bounds it: 8192 x 8192 x 7168 takes 166-182 us (5300-5800 TFLOP/s; the arranging
// kernel's 6 us in front included), tensor pipe 77 % busy, L2 to shared memory 13 TB/s,
// at the power limit when calls follow each other (215 us).  The scale copies, in
// order with the MMAs, cost the rest of a K step.  Measured and not kept: copies a K
// step ahead into a second buffer (*); scales stored four times and copied 128 rows at
// a time (same time); warps that store the words to TMEM (tcgen05.st: 474 us (*));
// heights of 208 and 192 rows (184 us); rows' codes in one box instead of three.
//
//   warp 0       TMA
//   warp 1       one thread of the first block: scale copies and MMAs
//   warp 2       looks for rows without a source
//   warps 4-11   epilogue, two per TMEM lane quadrant
#pragma once
#include "mg_common.cuh"

namespace fn {

struct MGPShape {
  static constexpr int kXRows = kMgPairRows / 2;
  static constexpr int kWBytes = kMgFeat * 128;
  static constexpr int kXBytes = kXRows * 128;
  static constexpr int kSwBytes = 2 * 512;
  static constexpr int kSxBytes = 2 * kMgXTile;
  static constexpr int kStage = kWBytes + kXBytes + kSwBytes + kSxBytes;
  static constexpr int kStages = 6;
  static constexpr int kColSw = 2 * kMgPairRows;
  static constexpr int kColSx = kColSw + 8;
  static constexpr int kCols = 512;
  static_assert(kColSx + 16 <= kCols && kXBytes % 1024 == 0, "layout");
  static constexpr int kSmem = kStages * kStage + 1024;
};

// Rows of the row tiles of an expert (or of the product): as even as steps of 16
// allow, so that no tile is left with a few rows.
__device__ __forceinline__ int mgp_height(int rows, int tok) {
  const int nt = (rows + tok - 1) / tok;
  return (rows / nt + (rows % nt != 0) + 15) / 16 * 16;
}

struct MGPTile {
  int e, f0, row0, n, piece;
};

// The tiles in order: expert, group of eight row tiles, feature tile, row tile.  The
// 74 pairs then work on about 9 x 8 tiles at a time, whose operands stay in L2
// (with all row tiles in one group 32768 x 4096 x 7168 reads its 117 MB of rows once
// per feature tile: 405 us against 323).
struct MGPTiles {
  static constexpr int kGroup = 8;
  const int* cum;  // [E + 1] row tiles before expert e   (offsets given)
  const int* lo;
  const int* cnt;
  int t, e, total, feat, M, tok, stride;

  __device__ MGPTiles(const MGParams& p, const int* table)
      : cum(p.offsets ? table : nullptr), lo(table + p.E + 1), cnt(table + 2 * p.E + 1),
        t(blockIdx.x / 2), e(0), M(p.M), tok(p.tok), stride(gridDim.x / 2) {
    feat = (p.N + kMgPairFeat - 1) / kMgPairFeat;
    total = feat * (cum ? cum[p.E] : (M + tok - 1) / tok);
  }
  __device__ bool next(MGPTile& o) {
    while (t < total) {
      int rel = t, rows = M, first = 0, before = 0, nt;
      if (cum) {
        while (t >= feat * cum[e + 1]) ++e;
        before = cum[e];
        nt = cum[e + 1] - before;
        rel = t - feat * before;
        rows = cnt[e];
        first = lo[e];
      } else {
        nt = (rows + tok - 1) / tok;
      }
      // groups of kGroup row tiles, all their feature tiles in turn
      const int g = rel / (feat * kGroup) * kGroup, in = min(kGroup, nt - g);
      rel -= g * feat;
      const int f = rel / in, m = g + rel - f * in;
      const int h = mgp_height(rows, tok);
      o.e = e;
      o.f0 = f * kMgPairFeat;
      o.row0 = first + m * h;
      o.n = min(h, rows - m * h);
      o.piece = before + m;
      t += stride;
      if (o.n > 0) return true;  // (even tiles can be one fewer)
    }
    return false;
  }
};

__global__ void __launch_bounds__(kMgPairThreads, 1)
    mgp_kernel(const __grid_constant__ MGParams p, const __grid_constant__ MGMaps maps) {
  using S = MGPShape;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[2 * S::kStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t stop;
  __shared__ uint32_t outside;  // a tile of this block has rows whose index is outside the operand

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t tiles0 = (smem_addr(dyn) + 1023) & ~1023u;
  int* table = reinterpret_cast<int*>(dyn + (tiles0 - smem_addr(dyn)) + S::kStages * S::kStage);
  const uint32_t full = smem_addr(bars), empty = full + 8 * S::kStages,
                 tfull = empty + 8 * S::kStages, tempty = tfull + 16, drain = tempty + 16;
  auto w_tile = [&](int s) { return tiles0 + s * (S::kWBytes + S::kXBytes); };
  auto x_tile = [&](int s) { return w_tile(s) + S::kWBytes; };
  const uint32_t scales0 = tiles0 + S::kStages * (S::kWBytes + S::kXBytes);
  auto sw_tile = [&](int s) { return scales0 + s * (S::kSwBytes + S::kSxBytes); };
  auto sx_tile = [&](int s) { return sw_tile(s) + S::kSwBytes; };

  if (threadIdx.x == 0) {
    stop = 0;
    outside = 0;
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + 8 * b, 1);
      mbar_init(tempty + 8 * b, 16);  // eight epilogue warps of each block
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    tma_prefetch_map(&maps.x);
    tma_prefetch_map(&maps.w);
    tma_prefetch_map(&maps.xs);
    tma_prefetch_map(&maps.ws);
  }
  if (warp == 1) tmem_alloc<2>(smem_addr(&tmem_slot), S::kCols);
  pdl_enter();
  if (p.offsets && warp == 0) mg_table(p, table, lane, p.tok, 1, p.pieces);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);  // (known to be uniform)
  const int steps = (p.K + kMgStageK - 1) / kMgStageK;
  const int kts = (p.groups + 3) >> 2;
  MGPTiles tiles(p, table);
  MGPTile t;

  // warps 0 and 1 loop with all lanes and issue from one (as in mg_kernel.cuh)
  const bool leader = elect_one();
  if (warp == 0) {
    // ---- operands: each block its own features' and its half of the rows' codes, and
    // all scales that its MMA half reads; all bytes count on the first block's
    // barrier
    int s = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (ok && tiles.next(t)) {
      const int f0 = t.f0 + (int)rank * kMgFeat;
      const int half = (t.n + 15) / 16 * 8;
      const int x0 = t.row0 + (int)rank * half;
      const int pieces = (half + p.box - 1) / p.box;
      const uint32_t bytes = 2 * (S::kWBytes + pieces * p.box * 128 + S::kSwBytes + S::kSxBytes);
      const int ws0 = t.e * ((p.N + 127) / 128 * kts) + f0 / 128 * kts;
      const int xs0 = t.piece * kts;
      for (int kb = 0; kb < steps; ++kb) {
        ok = mbar_wait<2>(empty + 8 * s, ph ^ 1, &stop);
        if (!ok) break;
        const uint32_t bar = cluster_map(full + 8 * s, 0);
        if (leader) {
          if (rank == 0) mbar_expect_tx(full + 8 * s, bytes);
          tma_load<2>(w_tile(s), &maps.w, kb * 128, t.e * p.N + f0, bar);
          tma_load<2>(sw_tile(s), &maps.ws, 0, ws0 + 2 * kb, bar);
          tma_load<2>(sx_tile(s), &maps.xs, 0, (xs0 + 2 * kb) * 2, bar);
          for (int i = 0; i < pieces; ++i)
            tma_load<2>(x_tile(s) + i * p.box * 128, &maps.x, kb * 128, x0 + i * p.box, bar);
        }
        __syncwarp();
        ++issued;
        if (++s == S::kStages) s = 0, ph ^= 1;
      }
    }
    // the last MMAs' arrivals on this block's barriers come before it goes
    for (int i = 0; ok && i < min(issued, S::kStages); ++i) {
      ok = mbar_wait<2>(empty + 8 * s, ph ^ 1, &stop);
      if (++s == S::kStages) s = 0, ph ^= 1;
    }
    if (!ok && rank == 0) {  // the copies in flight land before the blocks go
      for (int i = 0; i < min(issued, S::kStages); ++i) {
        if (--s < 0) s = S::kStages - 1, ph ^= 1;
        for (int n = 0; n < kWaitTries && !mbar_try<2>(full + 8 * s, ph); ++n) {
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA ----------------------------------------------------------------------------
    if (rank == 0) {
      int s = 0, i = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (; ok && tiles.next(t); ++i) {
        const int acc = i & 1;
        const uint32_t d = tmem + acc * kMgPairRows;
        const int n16 = (t.n + 15) / 16 * 16;
        const uint32_t id0 = mxf4_idesc(kMgPairFeat, n16, 0), id1 = mxf4_idesc(kMgPairFeat, n16, 1);
        ok = mbar_wait<2>(tempty + 8 * acc, ((i >> 1) & 1) ^ 1, &stop);
        tc_fence_after();
        for (int kb = 0; ok && kb < steps; ++kb) {
          ok = mbar_wait<2>(full + 8 * s, ph, &stop);
          if (!ok) break;
          tc_fence_after();
          const int mmas = min(4, (p.K - kb * kMgStageK + 63) / 64);
          const uint64_t a = operand_desc(w_tile(s)), b = operand_desc(x_tile(s));
          const uint64_t sw = scale_desc(sw_tile(s)), sx = scale_desc(sx_tile(s));
          if (leader) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              tc_copy_scales<2>(tmem + S::kColSw + 4 * h, sw + 32 * h);
#pragma unroll
              for (int b = 0; b < 2; ++b)
                tc_copy_scales<2>(tmem + S::kColSx + 4 * (2 * h + b), sx + 32 * (2 * h + b));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < mmas)
                tc_mma_mxf4<2>(d, a + 2 * j, b + 2 * j, j & 1 ? id1 : id0,
                               tmem + S::kColSw + 4 * (j / 2), tmem + S::kColSx + 8 * (j / 2),
                               kb > 0 || j > 0);
            tc_commit<2>(empty + 8 * s);
          }
          __syncwarp();
          if (++s == S::kStages) s = 0, ph ^= 1;
        }
        if (ok && leader) tc_commit<2>(tfull + 8 * acc);
        __syncwarp();
      }
      if (!ok) {  // MMAs in flight end before the blocks go
        if (leader) tc_commit<2>(drain);
        __syncwarp();
        for (int n = 0; n < kWaitTries && !mbar_try<2>(drain, 0); ++n) {
        }
      }
    }
  } else if (warp == 2) {
    // ---- rows without a source ------------------------------------------------------------
    bool out = false;
    while (p.rows && tiles.next(t))
      for (int r = lane; r < t.n; r += 32) out |= (unsigned)p.rows[t.row0 + r] >= (unsigned)p.x_rows;
    if (out) outside = 1;
  } else if (warp >= 4) {
    // ---- epilogue ---------------------------------------------------------------------------
    const int quad = warp & 3;  // the TMEM lanes a warp can read
    bool ok = true;
    for (int i = 0; tiles.next(t); ++i) {
      const int acc = i & 1;
      if (ok) ok = mbar_wait<2>(tfull + 8 * acc, (i >> 1) & 1, &stop);
      tc_fence_after();
      const int f = t.f0 + (int)rank * kMgFeat + quad * 32 + lane;
      // the two warps of a quadrant take turns with 32 rows each
      for (int c = (warp - 4) / 4 * 32; c < t.n; c += 64) {
        uint32_t v[32];
        tmem_ld(tmem + ((uint32_t)(quad * 32) << 16) + acc * kMgPairRows + c, v);
        tmem_wait_ld();
        if (!ok) {
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = 0x7fffffffu;
        }
        mg_store<32>(p, v, (int64_t)t.row0 + c, min(32, t.n - c), f, lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_map(tempty + 8 * acc, 0));
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) tmem_dealloc<2>(tmem, S::kCols);
  // A row without a source is zero.  Its codes are, so its sums are zero or, for a feature
  // whose weight has a NaN scale, NaN, in all such rows of a tile alike: where the first
  // one shows NaN, zeros are stored over all of them.  At the end, a warp a tile, so that
  // the epilogue's loop stays as it is: 4096 gathered rows, 4096 x 2048, 46 us, 48 where a
  // quarter of the rows has no source (50 and 52 with masks in that loop; 45 and 80 with
  // zeros stored over every such row behind its tile).
  if (outside) {
    constexpr int kWarps = kMgPairThreads / 32, kParts = (kMgPairRows + 31) / 32;
    MGPTiles own(p, table);  // every kWarps-th tile of the block
    own.t += warp * own.stride;
    own.stride *= kWarps;
    while (own.next(t)) {
      uint32_t out[kParts];
      int first = -1;
#pragma unroll
      for (int j = 0; j < kParts; ++j) {
        const int r = j * 32 + lane;
        const int src = r < t.n ? p.rows[t.row0 + r] : 0;
        out[j] = __ballot_sync(0xffffffffu, (unsigned)src >= (unsigned)p.x_rows);
      }
#pragma unroll
      for (int j = kParts - 1; j >= 0; --j)
        if (out[j]) first = j * 32 + __ffs(out[j]) - 1;
      if (first < 0) continue;
      const int f0 = t.f0 + (int)rank * kMgFeat + lane;
      bool nan = false;
#pragma unroll
      for (int f = 0; f < kMgFeat; f += 32)
        if (f0 + f < p.N) nan |= mg_is_nan(p, (int64_t)t.row0 + first, f0 + f);
      if (!__any_sync(0xffffffffu, nan)) continue;
#pragma unroll
      for (int j = 0; j < kParts; ++j) {
        for (; out[j]; out[j] &= out[j] - 1) {
          const int64_t row = (int64_t)t.row0 + j * 32 + __ffs(out[j]) - 1;
#pragma unroll
          for (int f = 0; f < kMgFeat; f += 32)
            if (f0 + f < p.N) mg_store_one(p, 0.f, row, f0 + f);
        }
      }
    }
  }
}

// Brings row-major (or row-tiled) scales into 512-byte tiles aligned to the pair
// kernel's row tiles and to 128 weights, zeros in the padding, and gathers codes.
// A warp handles 128 rows x 16 groups at a time: a 16-byte vector of four
// rows a lane, four tiles' words of each.  Bound by memory latency: 2 MB of scales
// for 8192 rows of 7168.
__global__ void __launch_bounds__(256)
    mgp_arrange_kernel(const __grid_constant__ MGParams p, const __grid_constant__ MGArrange a) {
  extern __shared__ int table[];
  pdl_enter();
  const int lane = threadIdx.x & 31;
  if (p.offsets && threadIdx.x < 32) mg_table(p, table, lane, p.tok, 1, p.pieces);
  __syncthreads();
  const int* cum = table;
  const int kts = (p.groups + 3) >> 2, chunks = (kts + 3) / 4;
  const int pieces = p.offsets ? cum[p.E] : (p.M + p.tok - 1) / p.tok;
  const int64_t warps = (int64_t)gridDim.x * 8;
  const int64_t first = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;

  // the words of tiles 4 c ... 4 c + 3, `step` bytes apart
  auto put = [&](uint8_t* tile, int64_t step, const uint4 (&v)[4], int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * c + i < kts)
        reinterpret_cast<uint4*>(tile + (4 * c + i) * step)[lane] =
            make_uint4(word(v[0], i), word(v[1], i), word(v[2], i), word(v[3], i));
  };
  int e = 0;
  for (int64_t w = first; w < (int64_t)pieces * 2 * chunks; w += warps) {
    const int c = (int)(w % chunks), blk = (int)(w / chunks) & 1, piece = (int)(w / chunks / 2);
    int rows = p.M, lo = 0, m = piece;
    if (p.offsets) {
      while (piece >= cum[e + 1]) ++e;
      rows = table[2 * p.E + 1 + e];
      lo = table[p.E + 1 + e];
      m = piece - cum[e];
    }
    const int h = mgp_height(rows, p.tok), n = min(h, rows - m * h);
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = blk * 128 + i * 32 + lane;
      int r = lo + m * h + j;
      bool in = j < n;
      if (in && p.rows) {
        r = p.rows[r];
        in = (unsigned)r < (unsigned)p.x_rows;
      }
      v[i] = !in            ? make_uint4(0, 0, 0, 0)
             : a.x_swizzled ? mg_tiled_scales(p.x_scale, r, c, p.groups)
                            : mg_scales(p.x_scale + (int64_t)r * p.groups, c, p.groups, p.x_wide);
    }
    put(a.x_tiles + (int64_t)piece * kts * kMgXTile + blk * (kMgXTile / 2), kMgXTile, v, c);
  }
  if (a.w_tiles) {
    const int blocks = (p.N + 127) / 128;
    for (int64_t w = first; w < (int64_t)p.E * blocks * chunks; w += warps) {
      const int c = (int)(w % chunks), b = (int)(w / chunks % blocks);
      const int64_t ex = w / chunks / blocks;
      const uint8_t* base = p.w_scale + ex * p.w_scale_stride;
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t r = b * 128 + i * 32 + lane;
        v[i] = r >= p.N       ? make_uint4(0, 0, 0, 0)
               : a.w_swizzled ? mg_tiled_scales(base, r, c, p.groups)
                              : mg_scales(base + r * p.groups, c, p.groups, p.w_wide);
      }
      put(a.w_tiles + (ex * blocks + b) * kts * 512, 512, v, c);
    }
  }
  if (a.codes) {  // rows by index; an index outside the operand gives zeros
    const int vecs = p.groups;  // 16 bytes hold 32 codes
    // a warp a row, or, for short rows, neighbouring lanes a row
    const int per = vecs >= 32 ? 32 : vecs >= 8 ? 8 : 1, mine = lane % per;
    const int64_t step = warps * (32 / per);
    for (int64_t r = first * (32 / per) + lane / per; r < p.M; r += step) {
      const int src = p.rows[r];
      const bool in = (unsigned)src < (unsigned)p.x_rows;
      const uint4* from = a.x_codes + (in ? (int64_t)src * vecs : 0);
      uint4* to = a.codes + r * vecs;
      for (int v0 = mine; v0 < vecs; v0 += 4 * per) {
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (v0 + i * per < vecs)
            x[i] = in ? ld_stream_nc(from + v0 + i * per) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (v0 + i * per < vecs) to[v0 + i * per] = x[i];
      }
    }
  }
}

}  // namespace fn
