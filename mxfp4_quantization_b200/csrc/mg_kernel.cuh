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
// This kernel takes calls of few rows (a product of up to 64, experts of 16 on
// average); the pair kernel (mgp_kernel.cuh) the others.  Persistent blocks, one role per
// warp:
//   warp 0      TMA: the weight tile and the row tile of each K step of 256
//               elements (128 bytes a row, 128-byte swizzle; rows by index
//               with gather4), and scales that are in the 32x4x4 tiling
//   warp 1      one thread issues per K step the copies of the scales to TMEM
//               and the four 64-element MMAs
//   warps 2, 3  scales that are row-major (2: the rows'; 3: the weights'): a
//               row's scales are a few bytes at any offset, below what a TMA
//               box can fetch.  They come as 16-byte vectors, two K steps at
//               once and two fetches ahead, and leave as the 512-byte tiles that
//               the copies to TMEM read
//   warps 4-7   epilogue: TMEM to registers, rounding, stores
#pragma once
#include "mg_common.cuh"

namespace fn {

template <int TOK>
struct MGShape {
  static constexpr int kWBytes = kMgFeat * 128;
  static constexpr int kXBytes = TOK * 128;
  static constexpr int kScaleBytes = 2 * 512;  // of either operand
  static constexpr int kStage = kWBytes + kXBytes + 2 * kScaleBytes;
  // two blocks an SM
  static constexpr int kStages = TOK >= 64 ? 4 : 5;
  // TMEM: two accumulators, then the scales (4 columns per 128 elements each)
  static constexpr int kColSw = 2 * TOK;
  static constexpr int kColSx = kColSw + 8;
  static constexpr int kColEnd = kColSx + 8;
  static constexpr int kCols = kColEnd <= 64 ? 64 : kColEnd <= 256 ? 256 : 512;
  static constexpr int kChunk = TOK >= 32 ? 32 : 16;  // columns the epilogue takes at once
  static constexpr int kXLaneRows = (TOK + 31) / 32;  // rows whose scales a lane brings
  // a split's partial sums of the smallest tile: [block][row / split][feature]
  static constexpr bool kPush = TOK == 16;
  static constexpr int kPushBytes = kPush ? TOK * kMgFeat * 4 : 0;
  // 1024 bytes: the operand tiles' alignment
  static constexpr int kSmem = kStages * kStage + kPushBytes + 1024;
  static_assert(kStages * kStage >= TOK * kMgFeat * 4, "a split's partial sums");
};

template <int R>
struct MGRows {
  static constexpr int value = R;
};

struct MGTile {
  int e, f0, row0, n;
};

// The tiles in order: expert, then feature tile, then row tile (the row tiles
// that share a weight tile are next to each other).  Every role walks the same
// sequence: the block's (or the split's) index, then one grid further each time.
template <int TOK>
struct MGTiles {
  const int* cum;  // [E + 1] tiles before expert e   (offsets given)
  const int* lo;   // [E] first row
  const int* cnt;  // [E] rows
  int t, e, total, M, stride;

  __device__ MGTiles(const MGParams& p, const int* table)
      : cum(table), lo(table + p.E + 1), cnt(table + 2 * p.E + 1), t(blockIdx.x >> p.split_log2), e(0),
        M(p.M), stride(gridDim.x >> p.split_log2) {
    const int feat = (p.N + kMgFeat - 1) / kMgFeat;
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
    const int f = nt == 1 ? rel : rel / nt, m = rel - f * nt;
    o.e = e;
    o.f0 = f * kMgFeat;
    o.row0 = first + m * TOK;
    o.n = min(TOK, rows - m * TOK);
    t += stride;
    return true;
  }
};

template <int TOK>
__global__ void __launch_bounds__(kMgThreads, 2)
    mg_kernel(const __grid_constant__ MGParams p, const __grid_constant__ MGMaps maps) {
  using S = MGShape<TOK>;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t bars[3 * S::kStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t stop;

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const uint32_t tiles0 = (smem_addr(dyn) + 1023) & ~1023u;
  uint8_t* const tiles_p = dyn + (tiles0 - smem_addr(dyn));
  int* table = reinterpret_cast<int*>(tiles_p + S::kStages * S::kStage + S::kPushBytes);
  const uint32_t part0 = tiles0 + S::kStages * S::kStage;
  const uint32_t full = smem_addr(bars), sfull = full + 8 * S::kStages,
                 empty = sfull + 8 * S::kStages, tfull = empty + 8 * S::kStages,
                 tempty = tfull + 16, drain = tempty + 16;
  auto w_tile = [&](int s) { return tiles0 + s * (S::kWBytes + S::kXBytes); };
  auto x_tile = [&](int s) { return w_tile(s) + S::kWBytes; };
  const uint32_t scales0 = tiles0 + S::kStages * (S::kWBytes + S::kXBytes);
  auto sw_tile = [&](int s) { return scales0 + s * 2 * S::kScaleBytes; };
  auto sx_tile = [&](int s) { return sw_tile(s) + S::kScaleBytes; };
  const int scale_warps = (p.x_mode != MG_SCALE_TMA) + (p.w_mode != MG_SCALE_TMA);

  // Warp 0 sets the barriers up (one a lane), makes the tile table and goes on to
  // its loads; the others wait for that and for the TMEM allocation.
  if (warp == 0) {
    if (lane == 0) {
      stop = 0;
      tma_prefetch_map(&maps.w);
      tma_prefetch_map(&maps.x);
    }
    constexpr int kBars = 3 * S::kStages + 5;
    static_assert(kBars <= 32, "a barrier a lane");
    if (lane < kBars) {
      const int s = lane / S::kStages;  // 0 full, 1 sfull, 2 empty, then tfull, tempty, drain
      const int last = lane - 3 * S::kStages;
      mbar_init(full + 8 * lane, s == 1                     ? max(1, scale_warps)
                                 : last == 2 || last == 3 ? 4
                                                            : 1);
    }
    fence_async_smem();
  }
  if (warp == 1) tmem_alloc<1>(smem_addr(&tmem_slot), S::kCols);
  if (p.prefetch && warp == 0) {
    // A programmatic dependent: this block's first weights start towards L2 while the
    // kernel before is still at work (a hint: what that kernel writes is seen all
    // the same).
    const int tile = blockIdx.x >> p.split_log2, part = blockIdx.x & (p.split - 1);
    const int f0 = tile / p.pieces * kMgFeat, steps = (p.K + kMgStageK - 1) / kMgStageK;
    const int first = steps * part >> p.split_log2, end = steps * (part + 1) >> p.split_log2;
    const int kb = first + lane;
    if (kb < min(end, first + S::kStages) && f0 < p.N) tma_prefetch(&maps.w, kb * 128, f0);
  }
  pdl_enter();
  if (p.offsets && warp == 0) mg_table(p, table, lane, TOK, (p.N + kMgFeat - 1) / kMgFeat, p.pieces);
  if (warp == 0) {
    __syncwarp();
    named_arrive<1>(kMgThreads);
  } else {
    tc_fence_before();
    named_sync<1>(kMgThreads);
    tc_fence_after();
  }
  const uint32_t tmem = warp == 0 ? 0 : __shfl_sync(0xffffffffu, tmem_slot, 0);  // (uniform)
  if (S::kPush && p.split > 1) cluster_arrive_started();
  // a split's blocks share the K steps of their tile
  const uint32_t rank = p.split > 1 ? cluster_rank() : 0;
  const int all = (p.K + kMgStageK - 1) / kMgStageK, shift = p.split_log2;
  const int kb0 = all * (int)rank >> shift, kb1 = all * ((int)rank + 1) >> shift;
  const int kts = (p.groups + 3) >> 2;
  MGTiles<TOK> tiles(p, table);
  MGTile t;

  // The scales of one operand, for warps 2 and 3.
  auto scale_role = [&](auto lane_rows, bool is_x) {
    constexpr int R = decltype(lane_rows)::value;
    const int mode = is_x ? p.x_mode : p.w_mode;
    const bool wide = is_x ? p.x_wide : p.w_wide;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (ok && tiles.next(t)) {
      const uint8_t* base = is_x ? p.x_scale : p.w_scale + t.e * p.w_scale_stride;
      const uint8_t* src[R];
      int64_t row[R];
      bool in[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int j = i * 32 + lane;
        int v;
        if (is_x) {
          in[i] = j < t.n;
          v = t.row0 + j;
          if (p.rows && in[i]) {
            v = p.rows[v];
            in[i] = (unsigned)v < (unsigned)p.x_rows;
          }
        } else {
          v = t.f0 + j;
          in[i] = v < p.N;
        }
        row[i] = in[i] ? v : 0;
        src[i] = base + row[i] * p.groups;
      }
      // the chunk of 16 groups with K steps 2 c, 2 c + 1
      auto fetch = [&](uint4 (&b)[R], int c) {
        const bool use = 2 * c < kb1 && (mode == MG_SCALE_WARP || 2 * c + 2 >= all);
#pragma unroll
        for (int i = 0; i < R; ++i)
          b[i] = !in[i] || !use          ? make_uint4(0, 0, 0, 0)
                 : mode == MG_SCALE_WARP ? mg_scales(src[i], c, p.groups, wide)
                                         : mg_tiled_scales(base, row[i], c, p.groups);
      };
      auto emit = [&](const uint4 (&b)[R], int c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int kb = 2 * c + h;
          if (kb >= kb0 && kb < kb1 && ok) {
            ok = mbar_wait<1>(empty + 8 * s, ph ^ 1, &stop);
            if (ok && (mode == MG_SCALE_WARP || kb == all - 1)) {
              const uint32_t dst = (is_x ? sx_tile(s) : sw_tile(s)) + lane * 16;
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int w = 2 * h + k;
                // (rows beyond the lane's are beyond the tile: their words are not read)
                st_shared_words(dst + 512 * k, word(b[0], w), word(b[R > 1 ? 1 : 0], w),
                                word(b[R > 2 ? 2 : 0], w), word(b[R > 3 ? 3 : 0], w));
              }
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(sfull + 8 * s);
            if (++s == S::kStages) s = 0, ph ^= 1;
          }
        }
      };
      // three buffers by name: a copy from one to the next would wait for its load
      const int c0 = kb0 / 2;
      uint4 b0[R], b1[R], b2[R];
      fetch(b0, c0);
      fetch(b1, c0 + 1);
      for (int c = c0; 2 * c < kb1 && ok; c += 3) {
        fetch(b2, c + 2);
        emit(b0, c);
        fetch(b0, c + 3);
        emit(b1, c + 1);
        fetch(b1, c + 4);
        emit(b2, c + 2);
      }
    }
  };

  // Warps 0 and 1 run their loops with all lanes and only issue from one: their
  // operands then stay in uniform registers (inside a one-lane branch every
  // instruction moved its descriptors there first: 630 cycles for the eight
  // tcgen05 instructions of a K step).
  const bool leader = elect_one();
  if (warp == 0) {
    // ---- operands -----------------------------------------------------------------------
    int s = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (ok && tiles.next(t)) {
      const int wrow = t.e * p.N + t.f0;
      int4 src = make_int4(0, 0, 0, 0);
      if (p.rows) {
        int r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // rows past the tile's end and indices outside the operand fetch row 0
          const int j = lane * 4 + i;
          const int v = j < t.n ? p.rows[t.row0 + j] : 0;
          r[i] = (unsigned)v < (unsigned)p.x_rows ? v : 0;
        }
        src = make_int4(r[0], r[1], r[2], r[3]);
      }
      const int pieces = (t.n + 3) / 4;  // rows by index come four at a time
      const uint32_t codes = S::kWBytes + (p.rows ? pieces * 512 : S::kXBytes);
      const int ws0 = t.e * p.w_tiles + t.f0 / 128 * kts;
      const int xs0 = t.row0 / 128 * kts;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = mbar_wait<1>(empty + 8 * s, ph ^ 1, &stop);
        if (!ok) break;
        const bool last = kb == all - 1;
        const bool tw = p.w_mode == MG_SCALE_TMA || (p.w_mode == MG_SCALE_TMA_TAIL && !last);
        const bool tx = p.x_mode == MG_SCALE_TMA || (p.x_mode == MG_SCALE_TMA_TAIL && !last);
        const uint32_t bar = full + 8 * s;
        if (leader) {
          mbar_expect_tx(bar, codes + (tw ? S::kScaleBytes : 0) + (tx ? S::kScaleBytes : 0));
          tma_load<1>(w_tile(s), &maps.w, kb * 128, wrow, bar);
          if (tw) tma_load<1>(sw_tile(s), &maps.ws, 0, ws0 + 2 * kb, bar);
          if (tx) tma_load<1>(sx_tile(s), &maps.xs, 0, xs0 + 2 * kb, bar);
          if (!p.rows) tma_load<1>(x_tile(s), &maps.x, kb * 128, t.row0, bar);
        }
        if (p.rows) {
          __syncwarp();
          if (lane < pieces) tma_gather4(x_tile(s) + lane * 512, &maps.x, kb * 128, src, bar);
        }
        ++issued;
        if (++s == S::kStages) s = 0, ph ^= 1;
      }
    }
    if (!ok) {  // the copies in flight land before the block goes
      for (int i = 0; i < min(issued, S::kStages); ++i) {
        if (--s < 0) s = S::kStages - 1, ph ^= 1;
        for (int n = 0; n < kWaitTries && !mbar_try<1>(full + 8 * s, ph); ++n) {
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA ----------------------------------------------------------------------------
    int s = 0, i = 0, fenced = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (; ok && tiles.next(t); ++i) {
      const int acc = i & 1;
      const uint32_t d = tmem + acc * TOK;
      const int n16 = (t.n + 15) / 16 * 16;
      const uint32_t id0 = mxf4_idesc(kMgFeat, n16, 0), id1 = mxf4_idesc(kMgFeat, n16, 1);
      ok = mbar_wait<1>(tempty + 8 * acc, ((i >> 1) & 1) ^ 1, &stop);
      tc_fence_after();
      for (int kb = kb0; ok && kb < kb1; ++kb) {
        ok = mbar_wait<1>(full + 8 * s, ph, &stop);
        // The fence for the scale warps' writes is made here, where no loads are in
        // flight: it waits for a thread's own, and the scale warps always have
        // some (with the fence in those warps a K step took 1.2 us).  It covers
        // every stage whose scales are there already.
        if (ok && scale_warps > 0 && fenced == 0) {
          ok = mbar_wait<1>(sfull + 8 * s, ph, &stop);
          int n = s;
          uint32_t nph = ph;
          do {
            ++fenced;
            if (++n == S::kStages) n = 0, nph ^= 1;
          } while (fenced < S::kStages &&
                   __all_sync(0xffffffffu, mbar_test(sfull + 8 * n, nph)));
          fence_async_smem();
        }
        if (!ok) break;
        --fenced;
        tc_fence_after();
        const int mmas = min(4, (p.K - kb * kMgStageK + 63) / 64);
        const uint64_t a = operand_desc(w_tile(s)), b = operand_desc(x_tile(s));
        const uint64_t sw = scale_desc(sw_tile(s)), sx = scale_desc(sx_tile(s));
        if (leader) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tc_copy_scales<1>(tmem + S::kColSw + 4 * h, sw + 32 * h);
            tc_copy_scales<1>(tmem + S::kColSx + 4 * h, sx + 32 * h);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < mmas)
              tc_mma_mxf4<1>(d, a + 2 * j, b + 2 * j, j & 1 ? id1 : id0,
                             tmem + S::kColSw + 4 * (j / 2), tmem + S::kColSx + 4 * (j / 2),
                             kb > kb0 || j > 0);
          tc_commit<1>(empty + 8 * s);
        }
        __syncwarp();
        if (++s == S::kStages) s = 0, ph ^= 1;
      }
      if (ok && leader) tc_commit<1>(tfull + 8 * acc);
      __syncwarp();
    }
    if (!ok) {  // MMAs in flight end before the block goes
      if (leader) tc_commit<1>(drain);
      __syncwarp();
      for (int n = 0; n < kWaitTries && !mbar_try<1>(drain, 0); ++n) {
      }
    }
  } else if (warp < 4) {
    // ---- scales ---------------------------------------------------------------------------
    // rows a lane brings: the tile's, or the weights' 128
    if (warp == 2 && p.x_mode != MG_SCALE_TMA) scale_role(MGRows<S::kXLaneRows>(), true);
    if (warp == 3 && p.w_mode != MG_SCALE_TMA) scale_role(MGRows<4>(), false);
  } else {
    // ---- epilogue ---------------------------------------------------------------------------
    const int quad = warp & 3;  // the TMEM lanes a warp can read
    constexpr int C = S::kChunk;
    if (S::kPush && p.split > 1) cluster_wait_started();
    bool ok = true;
    for (int i = 0; tiles.next(t); ++i) {
      const int acc = i & 1;
      if (ok) ok = mbar_wait<1>(tfull + 8 * acc, (i >> 1) & 1, &stop);
      tc_fence_after();
      const int f = t.f0 + quad * 32 + lane;
      for (int c = 0; c < t.n; c += C) {
        uint32_t v[C];
        tmem_ld(tmem + ((uint32_t)(quad * 32) << 16) + acc * TOK + c, v);
        tmem_wait_ld();
        if (!ok) {
#pragma unroll
          for (int q = 0; q < C; ++q) v[q] = 0x7fffffffu;
        } else if (p.rows) {  // rows whose source index is outside the operand are zero
          const int r = lane < C && c + lane < t.n ? p.rows[t.row0 + c + lane] : 0;
          const uint32_t keep = __ballot_sync(0xffffffffu, (unsigned)r < (unsigned)p.x_rows);
          if (keep != 0xffffffffu) {
#pragma unroll
            for (int q = 0; q < C; ++q)
              if (!((keep >> q) & 1)) v[q] = 0;
          }
        }
        if (p.split > 1 && S::kPush) {  // to the block that sums the row
          const uint32_t to = part0 + (rank * (TOK / p.split) * kMgFeat + quad * 32 + lane) * 4;
#pragma unroll
          for (int q = 0; q < C; ++q)
            if (c + q < t.n)
              st_cluster(cluster_map(to + ((c + q) >> shift) * kMgFeat * 4, (c + q) & (p.split - 1)),
                         __uint_as_float(v[q]));
        } else if (p.split > 1) {  // this block's partial sums, over the operand tiles (all read)
          float* part = reinterpret_cast<float*>(tiles_p) + quad * 32 + lane;
#pragma unroll
          for (int q = 0; q < C; ++q)
            if (c + q < t.n) part[(c + q) * kMgFeat] = __uint_as_float(v[q]);
        } else {
          mg_store<C>(p, v, (int64_t)t.row0 + c, min(C, t.n - c), f, lane);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty + 8 * acc);
    }
  }
  __syncwarp();
  tc_fence_before();
  if (p.split > 1) {
    if (S::kPush && warp < 4) cluster_wait_started();
    // One tile a split.  Block r sums rows r, r + split, ... over the blocks, in
    // order.  The smallest tile's partial sums were pushed there (one barrier of
    // the cluster); the others are fetched, and the blocks wait for each other
    // again before they go.
    cluster_sync_all();
    MGTiles<TOK> again(p, table);
    if (again.next(t)) {
      const int f = threadIdx.x & (kMgFeat - 1);
      const int half = threadIdx.x / kMgFeat, next = TOK / p.split * kMgFeat * 4;
      constexpr int R = TOK / 16;  // rows whose loads are in flight together
      for (int j0 = 0; j0 << shift < t.n; j0 += 2 * R) {  // slots of this block's rows
        float sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) sum[r] = 0.f;
        for (int q = 0; q < p.split; ++q) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const int slot = j0 + half * R + r, j = (slot << shift) + (int)rank;
            if (j < t.n)
              sum[r] += S::kPush ? ld_shared(part0 + q * next + (slot * kMgFeat + f) * 4)
                                 : ld_cluster(cluster_map(tiles0 + (j * kMgFeat + f) * 4, q));
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int j = ((j0 + half * R + r) << shift) + (int)rank;
          if (j < t.n && t.f0 + f < p.N) mg_store_one(p, sum[r], (int64_t)t.row0 + j, t.f0 + f);
        }
      }
    }
    if (!S::kPush) cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (warp == 1) tmem_dealloc<1>(tmem, S::kCols);
}

}  // namespace fn
