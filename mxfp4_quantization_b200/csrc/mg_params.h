// Parameter block and instance table of the MXFP4 product kernels
// (mg_kernel.cuh), shared by the host dispatch and the instantiation unit.
#pragma once
#include <cuda.h>

#include <cstdint>

namespace fn {

enum : int { MG_OUT_BF16 = 0, MG_OUT_FP16 = 1, MG_OUT_FP32 = 2 };

// Who brings an operand's scales to shared memory.
enum : int {
  MG_SCALE_TMA = 0,       // TMA boxes of the 32x4x4 tiling
  MG_SCALE_TMA_TAIL = 1,  // the same, but the last K step by a warp (it masks padding)
  MG_SCALE_WARP = 2,      // a warp, from row-major bytes
};

constexpr int kMgFeat = 128;         // output features of a block's tile
constexpr int kMgStageK = 256;       // elements of a K step (128 bytes of codes a row)
constexpr int kMgThreads = 256;      // 4 role warps, 4 epilogue warps

struct MGParams {
  const uint8_t* x_scale;   // token rows' scales
  const uint8_t* w_scale;   // weights' scales
  void* out;
  const int32_t* offsets;   // [E + 1] row ranges of the experts, or nullptr (one product)
  const int32_t* rows;      // source row of each row, or nullptr
  int64_t ldo;              // row stride of out, elements
  int64_t w_scale_stride;   // bytes of one expert's weight scales
  int M;                    // rows (of out)
  int x_rows;               // rows of the token operand
  int N, K, E;
  int groups;               // K / 32
  int x_mode, w_mode;       // MG_SCALE_*
  int x_wide, w_wide;       // row-major scale rows are whole aligned 16-byte vectors
  int out_type;
  int out_quads;            // 16-bit output whose rows are whole aligned groups of 4
  int out_pairs;            // fp32 output in aligned pairs
  int tok;                  // pair kernel: rows of a tile, a multiple of 16
  int box;                  // rows of a token TMA box (1: gather)
  int pieces;               // row tiles there can be, over all experts
  int split, split_log2;    // blocks (a cluster) that share a tile's K steps: 1, 2, 4 or 8
  int prefetch;             // single blocks: weights towards L2 before the launch wait
  int w_tiles;              // 512-byte scale tiles of one expert's weights
};

constexpr int kMgPairFeat = 256;     // features of a pair's tile
constexpr int kMgPairRows = 240;     // rows of a pair's tile, at most
constexpr int kMgPairThreads = 384;  // 4 role warps, 8 epilogue warps

constexpr int kMgXTile = 1024;       // a row tile's scales of 128 elements, 512 bytes per 128 rows

// What the arranging kernel prepares for the pair kernel, in the workspace.
struct MGArrange {
  uint8_t* x_tiles;         // [pieces][groups / 4][2 x 128 rows] 512-byte tiles
  uint8_t* w_tiles;         // [E][N / 128][groups / 4] tiles of the weights', or nullptr
  uint4* codes;             // [M, K / 32] gathered codes, or nullptr
  const uint4* x_codes;
  int x_swizzled, w_swizzled;
};

struct MGMaps {
  CUtensorMap x, w;        // codes
  CUtensorMap xs, ws;      // scale tiles (512 bytes each), where a TMA mode reads them
};

using MGKernel = void (*)(const MGParams, const MGMaps);

struct MGInstance {
  MGKernel kernel;
  int tok;       // token rows of a tile
  int smem;      // dynamic shared memory without the tile table
  int per_sm;    // blocks an SM holds
  int id;        // 0 .. kMgInstances - 1
};
constexpr int kMgInstances = 3;

// The single-block instance for a token tile of `tok` rows (16 or 64), and
// the pair kernel with the kernel that arranges its scales.
using MGArrangeKernel = void (*)(const MGParams, const MGArrange);
MGInstance mg_pick(int tok);
MGInstance mg_pair();
MGArrangeKernel mg_arrange();

}  // namespace fn
