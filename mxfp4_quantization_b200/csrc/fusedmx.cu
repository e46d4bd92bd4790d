// Host side of libfusedmx.so: argument checks, dispatch, launches.
// The C ABI and its contract are declared in include/fusedmx.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "fusedmx.h"
#include "act_kernel.cuh"
#include "combine_kernel.cuh"
#include "mg_params.h"

namespace {

thread_local int tl_variant = MX_VARIANT_NONE;
thread_local int32_t tl_launch[4] = {0, 0, 0, 0};
thread_local int tl_pdl = 0;

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

Range range_of(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + static_cast<uintptr_t>(bytes)};
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return -1;
  }
  return n;
}

// `pdl`: as a programmatic dependent of the work before it on the stream (every
// kernel waits for that work before it touches memory).
template <typename... KArgs, typename... Args>
int launch(void (*k)(KArgs...), unsigned grid, unsigned threads, size_t smem, void* stream,
           int cluster, bool pdl, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = (unsigned)n;
  if (cudaLaunchKernelEx(&cfg, k, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return FN_ERR_CUDA;
  }
  return FN_OK;
}

void record(int variant, int64_t a, int64_t b, int64_t c, int64_t d) {
  tl_variant = variant;
  tl_launch[0] = (int32_t)a;
  tl_launch[1] = (int32_t)b;
  tl_launch[2] = (int32_t)c;
  tl_launch[3] = (int32_t)d;
}

// ---- the products -----------------------------------------------------------------------

// The driver's encoder of TMA descriptors, looked up once (the library does not
// link against libcuda).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static std::atomic<EncodeTiled> cached{nullptr};
  EncodeTiled f = cached.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult res;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                       &res) != cudaSuccess ||
      res != cudaDriverEntryPointSuccess || !p) {
    (void)cudaGetLastError();
    return nullptr;
  }
  f = reinterpret_cast<EncodeTiled>(p);
  cached.store(f, std::memory_order_release);
  return f;
}

// Scale tiles of the 32x4x4 tiling, 512 bytes each; boxes of `box`.
bool scale_map(CUtensorMap* m, const void* s, int64_t tiles, int box = 2) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {128, (cuuint64_t)tiles};
  const cuuint64_t strides[1] = {512};
  const cuuint32_t boxes[2] = {128, (cuuint32_t)box};
  const cuuint32_t elem[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(s), dims, strides, boxes,
             elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Code rows [rows, K/2] bytes; boxes of 128 bytes x `box` rows, swizzled.
bool code_map(CUtensorMap* m, const void* q, int64_t rows, int64_t K, int box) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
  const cuuint32_t boxes[2] = {128, (cuuint32_t)box};
  const cuuint32_t elem[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(q), dims, strides, boxes, elem,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared memory of a product kernel (`id`: its place in the record), allowed once per
// kernel and device (function attributes belong to a device's context).  Plain
// atomics: nothing here can throw through the C entries, and two threads that meet
// set the same attribute twice.
bool allow_smem(const fn::MGInstance& k, int bytes) {
  constexpr int kDevices = 64;
  static std::atomic<int> done[fn::kMgInstances][kDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  std::atomic<int>* have = dev >= 0 && dev < kDevices ? &done[k.id][dev] : nullptr;
  if (have && have->load(std::memory_order_acquire) >= bytes) return true;
  // the most that any call of the kernel asks for, so that it is set once
  const int most = std::max(bytes, k.smem + (3 * MX_MAX_EXPERTS + 1) * 4);
  if (cudaFuncSetAttribute(reinterpret_cast<const void*>(k.kernel),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  if (have) have->store(most, std::memory_order_release);
  return true;
}

struct Product {
  const void *a_q, *a_scale, *b_q, *b_scale;
  const int32_t *rows, *offsets;
  int64_t a_rows, E, M, N, K, ldo;
  int flags;
  void* out;
  void* workspace;
};

constexpr int64_t kMaxRows = INT32_MAX - 256;  // row coordinates with a tile's reach on top
constexpr int64_t kMaxK = 1 << 24;

int64_t scale_bytes(int64_t rows, int64_t K, bool swizzled) {
  return swizzled ? round_up(rows, 128) * round_up(K / 32, 4) : rows * (K / 32);
}

int out_size(int flags) { return (flags & 0xF) == MX_OUT_FP32 ? 4 : 2; }

int check_product(const Product& q, bool grouped) {
  const int known = 0xF | MX_A_SCALE_SWIZZLE | MX_B_SCALE_SWIZZLE;
  if ((q.flags & ~known) || (q.flags & 0xF) > MX_OUT_FP32) return FN_ERR_INVALID;
  if (q.M < 0 || q.N < 1 || q.K < 32 || q.K % 32 || q.ldo < q.N) return FN_ERR_INVALID;
  if (grouped && (q.E < 1 || q.a_rows < 0)) return FN_ERR_INVALID;
  if (q.M > kMaxRows || q.N > kMaxRows || q.K > kMaxK) return FN_ERR_UNSUPPORTED;
  if (grouped) {
    if (q.flags & MX_A_SCALE_SWIZZLE) return FN_ERR_UNSUPPORTED;
    if (q.E > MX_MAX_EXPERTS || q.a_rows > kMaxRows || q.E * q.N > kMaxRows)
      return FN_ERR_UNSUPPORTED;
  }
  // every address stays below 2^62 bytes from its pointer
  if (q.ldo > ((int64_t)1 << 28)) return FN_ERR_UNSUPPORTED;
  return FN_OK;
}

int check_product_pointers(const Product& q, bool grouped, int64_t ws_bytes) {
  if (!q.a_q || !q.a_scale || !q.b_q || !q.b_scale || !q.out) return FN_ERR_INVALID;
  if (ws_bytes > 0 && !q.workspace) return FN_ERR_INVALID;
  if (grouped && !q.offsets) return FN_ERR_INVALID;
  if (grouped && (q.rows ? q.a_rows < 1 : q.a_rows < q.M)) return FN_ERR_INVALID;
  if (!aligned(q.a_q, 16) || !aligned(q.b_q, 16) || !aligned(q.out, out_size(q.flags)) ||
      (ws_bytes > 0 && !aligned(q.workspace, 16)))
    return FN_ERR_ALIGN;
  if ((q.flags & MX_A_SCALE_SWIZZLE && !aligned(q.a_scale, 16)) ||
      (q.flags & MX_B_SCALE_SWIZZLE && !aligned(q.b_scale, 16)))
    return FN_ERR_ALIGN;
  if (grouped && (!aligned(q.offsets, 4) || !aligned(q.rows, 4))) return FN_ERR_ALIGN;
  const int64_t E = grouped ? q.E : 1;
  const Range in[6] = {
      range_of(q.a_q, q.a_rows * q.K / 2),
      range_of(q.a_scale, scale_bytes(q.a_rows, q.K, q.flags & MX_A_SCALE_SWIZZLE)),
      range_of(q.b_q, E * q.N * q.K / 2),
      range_of(q.b_scale, E * scale_bytes(q.N, q.K, q.flags & MX_B_SCALE_SWIZZLE)),
      range_of(q.offsets, grouped ? (q.E + 1) * 4 : 0),
      range_of(q.rows, q.rows ? q.M * 4 : 0)};
  const Range out = range_of(q.out, ((q.M - 1) * q.ldo + q.N) * out_size(q.flags));
  const Range ws = range_of(q.workspace, ws_bytes);
  for (const Range& r : in)
    if (overlap(out, r) || (ws_bytes > 0 && overlap(ws, r))) return FN_ERR_INVALID;
  if (ws_bytes > 0 && overlap(ws, out)) return FN_ERR_INVALID;
  return FN_OK;
}

// How a product runs: a function of its sizes and flags alone, so that the
// workspace query and the call agree.
struct Plan {
  bool pair = false;
  int tok = 0;             // rows of a tile
  int split = 1;           // single-block kernel: blocks that share a tile's K steps
  int64_t feat = 0;        // feature tiles
  int64_t pieces = 0;      // row tiles, at most
  int64_t x_bytes = 0, w_bytes = 0, code_bytes = 0;  // workspace
  int64_t workspace() const { return x_bytes + w_bytes + code_bytes; }
};

constexpr int kSms = 148;  // B200 (a constant, so that a plan follows from the sizes alone)

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// `gather`: rows by index.  FN_ERR_UNSUPPORTED beyond the kernels' index range.
int plan_product(int64_t M, int64_t E, int64_t N, int64_t K, int flags, bool grouped, bool gather,
                 Plan* out) {
  Plan p;
  const int64_t each = grouped ? ceil_div(M, E) : M;
  const int64_t more = grouped ? std::min(E, M) : 0;  // a partly filled tile an expert
  const int64_t groups = K / 32, kts = ceil_div(groups, 4);
  // Pairs of blocks from here on.  Measured, us a call of single blocks / of pairs,
  // 8192 x 7168: 64 rows 13.1 / 14.0, 96 rows 15.4 / 14.5, 128 rows 15.6 / 14.6;
  // experts of 4096 x 7168 with 16 rows on average 157 / 162 (64 experts), 25 / 29 (8
  // experts), with 32 rows 157-167 / 165-170 and 27 / 30, with 48 rows 168 / 167;
  // 2048 x 2048 with 50 rows 10.1 / 9.4 (4 experts).  (Between 17 and 48 rows single
  // blocks are up to a tenth ahead; the border of 16, above which a call takes a
  // workspace, is part of the header's contract and dates from an earlier form of them.)
  p.pair = each > (grouped ? MX_SMALL_EXPERT_ROWS : MX_SMALL_ROWS);
  if (p.pair) {
    p.feat = ceil_div(N, fn::kMgPairFeat);
    // the tile height with the least rows times waves of pairs, as if the rows were
    // spread evenly over the experts; a tile also costs about as much as 32 more
    // rows (its weights, its epilogue)
    int64_t best = INT64_MAX;
    for (int tok = fn::kMgPairRows; tok >= 48; tok -= 16) {
      const int64_t nt = ceil_div(each, tok), rows = ceil_div(ceil_div(each, nt), 16) * 16;
      const int64_t waves = ceil_div(nt * (grouped ? E : 1) * p.feat, kSms / 2);
      if (waves * (rows + 32) < best) best = waves * (rows + 32), p.tok = tok;
    }
    p.pieces = M / p.tok + (grouped ? more : M % p.tok != 0);
    p.x_bytes = p.pieces * kts * fn::kMgXTile;
    // weights' tiles are taken as they are, unless a padding byte would be read
    if (!(flags & MX_B_SCALE_SWIZZLE) || groups & 1)
      p.w_bytes = (grouped ? E : 1) * ceil_div(N, 128) * kts * 512;
    if (gather) p.code_bytes = M * (K / 2);
  } else {
    p.feat = ceil_div(N, fn::kMgFeat);
    p.tok = each <= 16 ? 16 : 64;
    p.pieces = M / p.tok + (grouped ? more : M % p.tok != 0);
    // few tiles: the blocks of a cluster share the K steps of one, while all of them
    // fit the GPU at once, two an SM.  16 x 8192 x 7168: 14.1 us whole, 11.4 in two,
    // 10.8 in four, 15.8 in eight parts (512 blocks); 1 x 7168 x 7168: 14.0, 10.4, 9.7,
    // 14.5.
    const int64_t steps = ceil_div(K, fn::kMgStageK), tiles = p.feat * p.pieces;
    while (p.split < 8 && tiles * p.split * 2 <= 2 * kSms && p.split * 4 <= steps) p.split *= 2;
  }
  if (p.feat * p.pieces > INT32_MAX / 16 || p.pieces * kts > kMaxRows / 2 ||
      (grouped ? E : 1) * ceil_div(N, 128) * kts > kMaxRows || ceil_div(M, 128) * kts > kMaxRows)
    return FN_ERR_UNSUPPORTED;
  *out = p;
  return FN_OK;
}

int launch_product(const Product& q, bool grouped, const Plan& plan, void* stream) {
  fn::MGParams p;
  std::memset(&p, 0, sizeof p);
  p.x_scale = static_cast<const uint8_t*>(q.a_scale);
  p.w_scale = static_cast<const uint8_t*>(q.b_scale);
  p.out = q.out;
  p.offsets = q.offsets;
  p.rows = q.rows;
  p.ldo = q.ldo;
  p.w_scale_stride = scale_bytes(q.N, q.K, q.flags & MX_B_SCALE_SWIZZLE);
  p.M = (int)q.M;
  p.x_rows = (int)q.a_rows;
  p.N = (int)q.N;
  p.K = (int)q.K;
  p.E = grouped ? (int)q.E : 1;
  p.groups = (int)(q.K / 32);
  // an odd number of groups: the last MMA reads a byte of the tiling's padding
  const int tiled = p.groups & 1 ? fn::MG_SCALE_TMA_TAIL : fn::MG_SCALE_TMA;
  p.x_mode = q.flags & MX_A_SCALE_SWIZZLE ? tiled : fn::MG_SCALE_WARP;
  p.w_mode = q.flags & MX_B_SCALE_SWIZZLE ? tiled : fn::MG_SCALE_WARP;
  p.x_wide = p.groups % 16 == 0 && aligned(q.a_scale, 16);
  p.w_wide = p.groups % 16 == 0 && aligned(q.b_scale, 16);
  p.out_type = q.flags & 0xF;
  p.out_quads = p.out_type != MX_OUT_FP32 && q.N % 4 == 0 && q.ldo % 4 == 0 && aligned(q.out, 8);
  // fp32 rows in 8-byte stores where the epilogue sets the pace, in 4-byte stores where
  // the MMAs do and its shuffles cost them issue slots: 8192 x 7168, K = 2048
  // 78 us / 86 us, 8192 x 8192, K = 7168 221 us / 201 us
  p.out_pairs = p.out_type == MX_OUT_FP32 && q.K <= 4096 && q.N % 2 == 0 && q.ldo % 2 == 0 &&
                aligned(q.out, 8);
  p.tok = plan.tok;
  p.pieces = (int)plan.pieces;
  p.split = plan.split;
  while (1 << p.split_log2 < p.split) ++p.split_log2;
  const int sms = sm_count();
  if (sms <= 0) return FN_ERR_CUDA;
  const int table = grouped ? (3 * p.E + 1) * 4 : 0;
  const int64_t tiles_w = p.E * ceil_div(q.N, 128) * ceil_div(p.groups, 4);
  p.w_tiles = (int)(tiles_w / p.E);
  const int64_t tiles_x = ceil_div(q.a_rows, 128) * ceil_div(p.groups, 4);
  const fn::MGInstance k = plan.pair ? fn::mg_pair() : fn::mg_pick(plan.tok);
  fn::MGMaps maps;
  std::memset(&maps, 0, sizeof maps);
  if (!code_map(&maps.w, q.b_q, p.E * q.N, q.K, fn::kMgFeat) ||
      !allow_smem(k, k.smem + table))
    return FN_ERR_CUDA;
  if (!plan.pair) {
    p.box = q.rows ? 1 : plan.tok;
    p.prefetch = tl_pdl && !grouped ? 1 : 0;  // (an expert's rows are not known before the wait)
    if (!code_map(&maps.x, q.a_q, q.a_rows, q.K, p.box) ||
        (p.x_mode != fn::MG_SCALE_WARP && !scale_map(&maps.xs, q.a_scale, tiles_x)) ||
        (p.w_mode != fn::MG_SCALE_WARP && !scale_map(&maps.ws, q.b_scale, tiles_w)))
      return FN_ERR_CUDA;
    const int64_t tiles = plan.feat * plan.pieces;
    const unsigned grid = (unsigned)(plan.split > 1
                                         ? tiles * plan.split
                                         : std::min<int64_t>(tiles, (int64_t)sms * k.per_sm));
    const int st = launch(k.kernel, grid, fn::kMgThreads, k.smem + table, stream, plan.split,
                          tl_pdl != 0, p, maps);
    if (st == FN_OK) record(MX_VARIANT_GEMM, grid, fn::kMgThreads, plan.tok, plan.split);
    return st;
  }
  fn::MGArrange a;
  std::memset(&a, 0, sizeof a);
  uint8_t* ws = static_cast<uint8_t*>(q.workspace);
  a.x_tiles = ws;
  a.w_tiles = plan.w_bytes ? ws + plan.x_bytes : nullptr;
  a.codes = plan.code_bytes ? reinterpret_cast<uint4*>(ws + plan.x_bytes + plan.w_bytes) : nullptr;
  a.x_codes = static_cast<const uint4*>(q.a_q);
  a.x_swizzled = q.flags & MX_A_SCALE_SWIZZLE ? 1 : 0;
  a.w_swizzled = q.flags & MX_B_SCALE_SWIZZLE ? 1 : 0;
  p.box = fn::kMgPairRows / 6;
  if (!code_map(&maps.x, a.codes ? static_cast<const void*>(a.codes) : q.a_q,
                a.codes ? q.M : q.a_rows, q.K, p.box) ||
      !scale_map(&maps.xs, a.x_tiles, plan.x_bytes / 512, 4) ||
      !scale_map(&maps.ws, a.w_tiles ? a.w_tiles : q.b_scale, tiles_w))
    return FN_ERR_CUDA;
  const int64_t items = std::max(plan.pieces * 2, a.w_tiles ? p.E * ceil_div(q.N, 128) : 0) *
                        ceil_div(ceil_div(p.groups, 4), 4);
  const int64_t blocks =
      std::max(ceil_div(items, 8), a.codes ? ceil_div(q.M * p.groups, 1024) : 0);
  const unsigned agrid = (unsigned)std::min<int64_t>(blocks, (int64_t)sms * 8);
  if (launch(fn::mg_arrange(), agrid, 256, table, stream, 1, tl_pdl != 0, p, a) != FN_OK)
    return FN_ERR_CUDA;
  const unsigned grid = (unsigned)(std::min<int64_t>(plan.feat * plan.pieces, sms / 2) * 2);
  const int st = launch(k.kernel, grid, fn::kMgPairThreads, k.smem + table, stream, 2, true, p, maps);
  if (st == FN_OK) record(MX_VARIANT_GEMM_PAIR, grid, fn::kMgPairThreads, plan.tok, 2);
  return st;
}

// Bytes of workspace, -1 for sizes or flags that the call refuses.
int64_t workspace_bytes(const Product& q, bool grouped, bool gather) {
  Plan plan;
  if (check_product(q, grouped) != FN_OK) return -1;
  if (q.M == 0) return 0;
  if (plan_product(q.M, q.E, q.N, q.K, q.flags, grouped, gather, &plan) != FN_OK) return -1;
  return plan.workspace();
}

int run_product(const Product& q, bool grouped, void* stream) {
  if (int st = check_product(q, grouped)) return st;
  if (q.M == 0) return FN_OK;
  Plan plan;
  if (int st = plan_product(q.M, q.E, q.N, q.K, q.flags, grouped, q.rows != nullptr, &plan))
    return st;
  if (int st = check_product_pointers(q, grouped, plan.workspace())) return st;
  return launch_product(q, grouped, plan, stream);
}

// ---- silu_mul_quant ---------------------------------------------------------------------

struct ModeInfo {
  int q = -1, layout = 0;
  bool f16 = false;
};

int parse_mode(int mode, ModeInfo* mi) {
  const int q = mode & FN_MODE_MASK, flags = mode & ~(FN_MODE_MASK | FN_IO_FP16);
  if (q < FN_FP8_PER_TOKEN || q > FN_MXFP4) return FN_ERR_INVALID;
  mi->q = q;
  mi->f16 = (mode & FN_IO_FP16) != 0;
  mi->layout = fn::SCALE_ROW_MAJOR;
  if (flags == FN_SCALE_SWIZZLE_32_4_4 && q == FN_MXFP4)
    mi->layout = fn::SCALE_SWIZZLE_32_4_4;
  else if (flags == FN_SCALE_MN_MAJOR && q == FN_FP8_PER_GROUP128)
    mi->layout = fn::SCALE_MN_MAJOR;
  else if (flags != 0)
    return FN_ERR_INVALID;
  return FN_OK;
}

template <int MODE>
fn::ActKernel act_groups(bool f16, int vecs) {
  return vecs == 1 ? (f16 ? fn::act_groups_kernel<MODE, fn::F16, 1>
                          : fn::act_groups_kernel<MODE, fn::Bf16, 1>)
                   : (f16 ? fn::act_groups_kernel<MODE, fn::F16, 2>
                          : fn::act_groups_kernel<MODE, fn::Bf16, 2>);
}

template <class IO>
fn::ActKernel act_row(int V) {
  return V == 1   ? fn::act_row_kernel<1, IO>
         : V == 2 ? fn::act_row_kernel<2, IO>
         : V == 4 ? fn::act_row_kernel<4, IO>
                  : fn::act_row_kernel<8, IO>;
}

}  // namespace

extern "C" {

int mx_version(void) { return 100; }

int mx_last_variant(void) { return tl_variant; }

void mx_last_launch(int32_t out[4]) {
  if (out) std::memcpy(out, tl_launch, sizeof tl_launch);
}

int mx_programmatic_launch(int on) {
  const int old = tl_pdl;
  tl_pdl = on ? 1 : 0;
  return old;
}

const char* mx_status_string(int status) {
  switch (status) {
    case FN_OK: return "ok";
    case FN_ERR_INVALID: return "invalid argument (null pointer, size, flag or overlap)";
    case FN_ERR_ALIGN: return "misaligned pointer or stride";
    case FN_ERR_UNSUPPORTED: return "shape outside the built kernels";
    case FN_ERR_CUDA: return "CUDA launch failed";
    default: return "unknown status";
  }
}

int64_t mx_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int flags) {
  Product q = {};
  q.a_rows = q.M = M, q.E = 1, q.N = q.ldo = N, q.K = K, q.flags = flags;
  return workspace_bytes(q, false, false);
}

int mx_gemm(const void* a_q, const void* a_scale, const void* b_q, const void* b_scale, int64_t M,
            int64_t N, int64_t K, int flags, void* out, int64_t ldo, void* workspace,
            void* stream) {
  tl_variant = MX_VARIANT_NONE;
  const Product q = {a_q, a_scale, b_q, b_scale, nullptr, nullptr, M,        1,
                     M,   N,       K,   ldo,     flags,   out,     workspace};
  return run_product(q, false, stream);
}

int64_t mx_grouped_gemm_workspace_bytes(int64_t R, int64_t E, int64_t N, int64_t K, int flags,
                                        int gather) {
  Product q = {};
  q.a_rows = q.M = R, q.E = E, q.N = q.ldo = N, q.K = K, q.flags = flags;
  return workspace_bytes(q, true, gather != 0);
}

int mx_grouped_gemm(const void* a_q, const void* a_scale, int64_t a_rows, const int32_t* rows,
                    const int32_t* offsets, int64_t E, const void* b_q, const void* b_scale,
                    int64_t R, int64_t N, int64_t K, int flags, void* out, int64_t ldo,
                    void* workspace, void* stream) {
  tl_variant = MX_VARIANT_NONE;
  const Product q = {a_q, a_scale, b_q, b_scale, rows,  offsets, a_rows,   E,
                     R,   N,       K,   ldo,     flags, out,     workspace};
  return run_product(q, true, stream);
}

int mx_silu_mul_quant(const void* x, int64_t ldx, int mode, int64_t M, int64_t H,
                      const int32_t* num_rows, void* out_q, void* out_scale, void* out_y,
                      void* stream) {
  tl_variant = MX_VARIANT_NONE;
  ModeInfo mi;
  if (int st = parse_mode(mode, &mi)) return st;
  if (M < 0 || H <= 0 || H % 8 || ldx < 2 * H) return FN_ERR_INVALID;
  if (mi.q == FN_FP8_PER_GROUP128 && H % 128) return FN_ERR_INVALID;
  if (mi.q == FN_MXFP4 && H % 32) return FN_ERR_INVALID;
  if (H > FN_MAX_H || M > (int64_t)INT32_MAX / 8 || ldx > ((int64_t)1 << 31))
    return FN_ERR_UNSUPPORTED;
  if (M == 0) return FN_OK;
  if (!x || !out_q || !out_scale) return FN_ERR_INVALID;
  if (!aligned(x, 16) || ldx % 8 || !aligned(out_y, 16) || !aligned(num_rows, 4) ||
      !aligned(out_q, mi.q == FN_MXFP4 ? 4 : 8) || (mi.q != FN_MXFP4 && !aligned(out_scale, 4)))
    return FN_ERR_ALIGN;
  const int64_t sb = mi.q == FN_FP8_PER_TOKEN ? M * 4
                     : mi.q == FN_FP8_PER_GROUP128
                         ? (mi.layout == fn::SCALE_MN_MAJOR ? round_up(M, 4) : M) * (H / 128) * 4
                         : scale_bytes(M, H, mi.layout == fn::SCALE_SWIZZLE_32_4_4);
  const Range in[2] = {range_of(x, ((M - 1) * ldx + 2 * H) * 2),
                       range_of(num_rows, num_rows ? 4 : 0)};
  const Range outs[3] = {range_of(out_q, mi.q == FN_MXFP4 ? M * H / 2 : M * H),
                         range_of(out_scale, sb), range_of(out_y, out_y ? M * H * 2 : 0)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in)
      if (overlap(outs[i], r)) return FN_ERR_INVALID;
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return FN_ERR_INVALID;
  }
  fn::ActParams p;
  std::memset(&p, 0, sizeof p);
  p.x = static_cast<const uint4*>(x);
  p.num_rows = num_rows;
  p.out_q = static_cast<uint8_t*>(out_q);
  p.out_scale = out_scale;
  p.out_y = static_cast<uint4*>(out_y);
  p.M = M;
  p.ldv = ldx / 8;
  p.nvec = (int)(H / 8);
  p.scale_layout = mi.layout;
  p.scale_ld = mi.layout == fn::SCALE_SWIZZLE_32_4_4 ? round_up(H / 32, 4) / 4
               : mi.layout == fn::SCALE_MN_MAJOR     ? round_up(M, 4)
                                                     : 0;
  const int sms = sm_count();
  if (sms <= 0) return FN_ERR_CUDA;
  if (mi.q == FN_FP8_PER_TOKEN) {
    // Few rows: one vector a thread up to 512 threads.  Many: up to four, in blocks as
    // small as a warp (the barriers of a row then hold up few warps), unless more
    // than an eighth of the lanes would idle.  32768 x 2048: 65 us with four
    // (64 threads), 70 with two, 89 with one; 4097 x 2560: 14.5 with four (96 threads,
    // a sixth idle), 13.4 with two.
    const auto threads_of = [&](int v) { return round_up(ceil_div(p.nvec, v), 32); };
    int V = 1;
    while (M > (int64_t)sms * 4 && V < 4 && p.nvec > 32 * V &&
           (threads_of(2 * V) * 2 * V - p.nvec) * 8 <= p.nvec)
      V *= 2;
    while (p.nvec > 512 * V) V *= 2;
    const unsigned threads = (unsigned)threads_of(V);
    const unsigned grid = (unsigned)std::min<int64_t>(M, (int64_t)sms * 64);
    const int st = launch(mi.f16 ? act_row<fn::F16>(V) : act_row<fn::Bf16>(V), grid, threads, 0,
                          stream, 1, tl_pdl != 0, p);
    if (st == FN_OK) record(MX_VARIANT_SILU_ROW, grid, threads, V, 1);
    return st;
  }
  // two vectors a thread once every SM has eight blocks of one, and where a thread's 16
  // codes are aligned to one store
  // (MXFP4, 32768 x 2048: 60 us, with one vector 80 us)
  const int vecs =
      M * p.nvec > (int64_t)sms * 8 * 256 && aligned(out_q, mi.q == FN_MXFP4 ? 8 : 16) ? 2 : 1;
  const int units = p.nvec / vecs;
  p.recip64 = UINT64_MAX / (uint64_t)units + 1;
  p.recip32 = UINT32_MAX / (uint32_t)units + 1;
  const int64_t blocks = ceil_div(M * units, 256);
  if (blocks > INT32_MAX) return FN_ERR_UNSUPPORTED;  // (above 8 TB of rows)
  const unsigned grid = (unsigned)blocks;
  const int st = launch(mi.q == FN_MXFP4 ? act_groups<fn::MODE_MX>(mi.f16, vecs)
                                         : act_groups<fn::MODE_G128>(mi.f16, vecs),
                        grid, 256, 0, stream, 1, tl_pdl != 0, p);
  if (st == FN_OK) record(MX_VARIANT_SILU_GROUPS, grid, 256, vecs, 1);
  return st;
}

int mx_combine(const void* y, int64_t R, const int32_t* pos, const float* weight, const void* base,
               int64_t T, int k, int64_t N, int flags, void* out, void* stream) {
  tl_variant = MX_VARIANT_NONE;
  if (flags & ~FN_IO_FP16) return FN_ERR_INVALID;
  if (T < 0 || R < 0 || k < 0 || N < 1) return FN_ERR_INVALID;
  if (k > MX_MAX_TOP || N > (1 << 24) || R > INT32_MAX) return FN_ERR_UNSUPPORTED;
  const bool f16 = (flags & FN_IO_FP16) != 0;
  if (T > INT32_MAX || T * ((N + 255) / 256) > INT32_MAX) return FN_ERR_UNSUPPORTED;  // grid size
  if (T == 0) return FN_OK;
  if (!out || (k > 0 && (!pos || !weight)) || (k > 0 && R > 0 && !y)) return FN_ERR_INVALID;
  if (!aligned(y, 2) || !aligned(base, 2) || !aligned(out, 2) || !aligned(pos, 4) ||
      !aligned(weight, 4))
    return FN_ERR_ALIGN;
  const Range o = range_of(out, T * N * 2);
  if (overlap(o, range_of(y, R * N * 2)) || overlap(o, range_of(pos, T * k * 4)) ||
      overlap(o, range_of(weight, T * k * 4)) ||
      (base && base != out && overlap(o, range_of(base, T * N * 2))))
    return FN_ERR_INVALID;
  const bool wide = N % 8 == 0 && aligned(y, 16) && aligned(base, 16) && aligned(out, 16);
  fn::CombineParams p;
  std::memset(&p, 0, sizeof p);
  p.y = y;
  p.pos = pos;
  p.weight = weight;
  p.base = base;
  p.out = out;
  p.R = R;
  p.T = T;
  p.k = k;
  p.n = (int)(wide ? N / 8 : N);
  const unsigned threads = (unsigned)std::min<int64_t>(256, round_up(p.n, 32));
  p.per_row = (p.n + (int)threads - 1) / (int)threads;
  const unsigned grid = (unsigned)(T * p.per_row);
  fn::CombineKernel kern =
      !wide   ? (f16 ? fn::combine_narrow_kernel<fn::F16> : fn::combine_narrow_kernel<fn::Bf16>)
      : k > 2 ? (f16 ? fn::combine_kernel<fn::F16, 4> : fn::combine_kernel<fn::Bf16, 4>)
              : (f16 ? fn::combine_kernel<fn::F16, 2> : fn::combine_kernel<fn::Bf16, 2>);
  const int st = launch(kern, grid, threads, 0, stream, 1, tl_pdl != 0, p);
  if (st == FN_OK)
    record(wide ? MX_VARIANT_COMBINE : MX_VARIANT_COMBINE_NARROW, grid, threads, 1, 1);
  return st;
}

}  // extern "C"
