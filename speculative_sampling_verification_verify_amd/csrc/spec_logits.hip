// The operators between a model and the verify / sampling calls, for MI355X
// (gfx950): kernels and their C ABI (see spec_logits.h).

#include "sl_w4.h"
#include "sl_f8.h"
#include "sl_process.h"

#include <stdio.h>
#include <string.h>

#include <mutex>

namespace sl {

static thread_local char g_errbuf[256];

static int hip_status(hipError_t e) {
  if (e == hipSuccess) return SV_OK;
  snprintf(g_errbuf, sizeof g_errbuf, "HIP error: %s", hipGetErrorString(e));
  return SV_ERR_HIP;
}

static bool known(int dtype) { return dtype == SV_BF16 || dtype == SV_FP32; }
static size_t size_of(int dtype) { return dtype == SV_BF16 ? 2 : 4; }
static bool misaligned(const void* p, size_t n) { return (uintptr_t)p % n != 0; }

static bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  return (uintptr_t)p < (uintptr_t)q + nq && (uintptr_t)q < (uintptr_t)p + np;
}

// A launch holds fewer than 2^32 threads.
static bool fits(long long groups, int threads) { return groups * threads < (1LL << 32); }

// ---------------------------------------------------------------------------
// spec_logits_w4
// ---------------------------------------------------------------------------

constexpr int W4S_GRID = 256;   // one workgroup per CU

template <typename XT, typename ST, int SUB, int MT>
static hipError_t launch_stream(W4Args a, hipStream_t st) {
  const int tiles = (a.N + 15) / 16;
  hipLaunchKernelGGL((w4_stream_kernel<XT, ST, SUB, MT>), dim3((unsigned)(tiles < W4S_GRID ? tiles : W4S_GRID)),
                     dim3(W4S_NT), 0, st, a);
  return hipGetLastError();
}

template <typename XT, typename ST, int SUB, int MT, int U, int KC>
static hipError_t launch_tile(W4Args a, hipStream_t st) {
  a.row_tiles = (a.R + 32 * MT - 1) / (32 * MT);
  const int cols = W4_WAVES * 32;
  const long long sets = (long long)((a.N + cols - 1) / cols) * a.row_tiles;
  a.per_xcd = (int)((sets + 7) / 8);
  hipLaunchKernelGGL((w4_tile_kernel<XT, ST, SUB, MT, U, KC>), dim3((unsigned)a.per_xcd * 8), dim3(W4_NT), 0, st, a);
  return hipGetLastError();
}

// The plan of a call, a function of its sizes and types alone.  The rows of x
// stay in LDS where they fit it.  In us, LDS and tiles, at N=32000 and 128256:
//   R=16, K=4096, groups of 32:   29.5, 43.4   80.8, 100
//                 groups of 128:  24.0, 33.8   64.0, 70.1
//   R=32, K=2048, groups of 32:   25.5, 26.1   62.3, 54.4
//                 groups of 64:   20.0, 22.3   47.7, 45.5
//                 groups of 128:  17.4, 19.3   43.4, 39.9
//   R=32, K=1024, fp32 states:    18.3, 18.6   39.0, 39.4 (groups of 128)
// (17 to 32 rows lose a little where N is large, most with groups of 32, whose
// kernel keeps 44 to 84 bytes a lane in scratch; N does not enter the workspace's
// size, so it does not decide.)
struct W4Plan {
  int stream;        // row tiles of the streaming kernel (1, 2), 0: two launches
  int rp;            // rows staged of a tile (streaming kernel)
  int row_tiles;     // row tiles of 32 in the workspace, whole workgroup tiles
  size_t op_bytes, bytes;
};

// Row tiles of 32 of a workgroup in the two-launch form: two above 32 rows, which
// expand a weight once for 64 rows (one at R=64, K=4096: 133 us instead of 106 at
// N=128256; but 36 instead of 50 at N=32000, where two fill half of the CUs).
static int w4_tile_rows(int R) { return R > 32 ? 2 : 1; }

static W4Plan w4_plan(int hidden_dtype, int group, int R, int K) {
  W4Plan p;
  memset(&p, 0, sizeof p);
  const int sub = group == 32 ? 4 : group == 64 ? 2 : 1, nblk = (K + 127) / 128;
  const int parts = hidden_dtype == SV_BF16 ? 1 : 3;
  p.rp = 16;
  while (p.rp / 2 >= R) p.rp /= 2;
  const int mt = R <= 16 ? 1 : 2;
  const long long lds = (long long)nblk * mt * (4 * parts * 64 * p.rp + sub * 64);
  if (R <= 32 && lds <= W4S_LDS) {
    p.stream = mt;
    return p;
  }
  const int tile = w4_tile_rows(R);
  p.row_tiles = (R + 32 * tile - 1) / (32 * tile) * tile;
  p.op_bytes = (size_t)p.row_tiles * w4_blocks(K) * 8 * parts * 1024;
  p.bytes = p.op_bytes + (size_t)p.row_tiles * w4_blocks(K) * sub * 128;
  return p;
}

template <typename XT, typename ST, int SUB>
static hipError_t launch_w4(W4Args a, const W4Plan& p, hipStream_t st) {
  a.rp = p.rp;
  if (p.stream == 1) return launch_stream<XT, ST, SUB, 1>(a, st);
  if (p.stream == 2) return launch_stream<XT, ST, SUB, 2>(a, st);
  hipLaunchKernelGGL((w4_order_kernel<XT, SUB>), dim3((unsigned)(p.row_tiles * w4_blocks(a.K))), dim3(512), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (w4_tile_rows(a.R) == 1) return launch_tile<XT, ST, SUB, 1, 2, 2>(a, st);
  return launch_tile<XT, ST, SUB, 2, 1, 1>(a, st);
}

template <typename XT, typename ST>
static hipError_t launch_w4(const W4Args& a, int group, const W4Plan& p, hipStream_t st) {
  if (group == 32) return launch_w4<XT, ST, 4>(a, p, st);
  return group == 64 ? launch_w4<XT, ST, 2>(a, p, st) : launch_w4<XT, ST, 1>(a, p, st);
}

// R * K and R * N stay below it, so that both launches hold fewer than 2^32
// threads: one for 8 values of x, 512 for 32 rows and 256 columns.
constexpr long long W4_MOST = 1LL << 34;

static int w4_sizes(int hidden_dtype, int group, int R, int K) {
  if (!known(hidden_dtype) || R > SL_MAX_ROWS || K > SL_MAX_K) return SV_ERR_UNSUPPORTED;
  if (R < 0 || K < 1 || group < 1) return SV_ERR_ARG;
  if (group != 32 && group != 64 && group % 128 != 0) return SV_ERR_UNSUPPORTED;
  if (K % group != 0) return SV_ERR_ARG;
  return (long long)R * K < W4_MOST ? SV_OK : SV_ERR_UNSUPPORTED;
}

}  // namespace sl

using namespace sl;

extern "C" size_t spec_logits_w4_workspace_bytes(int hidden_dtype, int group, int R, int K) {
  return w4_sizes(hidden_dtype, group, R, K) == SV_OK && R > 0 ? w4_plan(hidden_dtype, group, R, K).bytes : 0;
}

extern "C" int spec_logits_w4(const void* hidden, int hidden_dtype, const uint8_t* weights, const void* scales,
                              int scale_dtype, const uint8_t* zeros, int group, int R, int K, int N, void* out,
                              int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!known(scale_dtype) || !known(out_dtype) || N > SV_MAX_VOCAB) return SV_ERR_UNSUPPORTED;
  const int rc = w4_sizes(hidden_dtype, group, R, K);
  if (rc != SV_OK) return rc;
  if (N < 1) return SV_ERR_ARG;
  if ((long long)R * N >= W4_MOST) return SV_ERR_UNSUPPORTED;
  if (R == 0) return SV_OK;
  if (!hidden || !weights || !scales || !out) return SV_ERR_ARG;
  if (misaligned(hidden, 16) || misaligned(weights, 16) || misaligned(scales, size_of(scale_dtype)) ||
      misaligned(out, size_of(out_dtype)))
    return SV_ERR_ARG;
  const W4Plan p = w4_plan(hidden_dtype, group, R, K);
  if (p.bytes && (!workspace || workspace_bytes < p.bytes || misaligned(workspace, 256))) return SV_ERR_WORKSPACE;
  const size_t no = (size_t)R * N * size_of(out_dtype), groups = (size_t)N * (K / group);
  if (overlap(out, no, hidden, (size_t)R * K * size_of(hidden_dtype)) || overlap(out, no, weights, (size_t)N * (K / 2)) ||
      overlap(out, no, scales, groups * size_of(scale_dtype)) || (zeros && overlap(out, no, zeros, groups)))
    return SV_ERR_ARG;
  W4Args a;
  memset(&a, 0, sizeof a);
  a.x = hidden;
  a.w = weights;
  a.s = scales;
  a.z = zeros;
  a.out = out;
  a.R = R;
  a.K = K;
  a.N = N;
  a.G = K / group;
  a.gb = group >= 128 ? group / 128 : 1;
  a.out_bf16 = out_dtype == SV_BF16;
  a.xop = (char*)workspace;
  a.xsum = (char*)workspace + p.op_bytes;
  hipStream_t st = (hipStream_t)stream;
  hipError_t e;
  if (hidden_dtype == SV_BF16)
    e = scale_dtype == SV_BF16 ? launch_w4<uint16_t, uint16_t>(a, group, p, st) : launch_w4<uint16_t, float>(a, group, p, st);
  else
    e = scale_dtype == SV_BF16 ? launch_w4<float, uint16_t>(a, group, p, st) : launch_w4<float, float>(a, group, p, st);
  return hip_status(e);
}

// ---------------------------------------------------------------------------
// spec_quantize_f8, spec_logits_f8
// ---------------------------------------------------------------------------
namespace sl {

// Raises a kernel's dynamic-LDS limit on the current device, once for each
// kernel and device: what is known of it is kept in a small table.
constexpr int MAX_DEVICES = 64;
static hipError_t lds_limit(const void* kernel, int bytes) {
  static std::mutex mu;
  static struct { const void* kernel; uint64_t devices; } done[32];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= MAX_DEVICES) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  int i = 0;
  while (i < 31 && done[i].kernel && done[i].kernel != kernel) ++i;
  if (done[i].kernel == kernel && (done[i].devices >> dev & 1)) return hipSuccess;
  if ((e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes)) != hipSuccess) return e;
  if (done[i].kernel != kernel) done[i].devices = 0;
  done[i].kernel = kernel;
  done[i].devices |= 1ull << dev;
  return hipSuccess;
}

static int f8_sizes(int R, int K) {
  if (R > SL_MAX_ROWS || K > SL_MAX_K) return SV_ERR_UNSUPPORTED;
  if (R < 0 || K < 1) return SV_ERR_ARG;
  return (long long)R * K < W4_MOST ? SV_OK : SV_ERR_UNSUPPORTED;
}

template <typename XT, bool WIDE>
static int launch_quantize(const F8QuantArgs& a, int rows, hipStream_t st) {
  const long long blocks = (long long)(rows == 1 ? a.R : (a.R + 127) / 128) * a.KB;
  const long long grid = rows == 1 ? (blocks + FQ_NT / 16 - 1) / (FQ_NT / 16) : blocks;
  if (!fits(grid, FQ_NT)) return SV_ERR_UNSUPPORTED;
  if (rows == 1) hipLaunchKernelGGL((quantize_rows_kernel<XT, WIDE>), dim3((unsigned)grid), dim3(FQ_NT), 0, st, a);
  else hipLaunchKernelGGL((quantize_tiles_kernel<XT, WIDE>), dim3((unsigned)grid), dim3(FQ_NT), 0, st, a);
  return hip_status(hipGetLastError());
}

// The plan of a product, a function of its sizes and types alone: few rows go to
// the streaming kernel where they fit LDS.  In us, streamed and in tiles (K = 4096):
//   N=32000:   R=1 23, 32   R=8 28, 31   R=16 34, 31
//   N=128255:  R=1 100, 113 R=8 109, 114 R=16 118, 115
// products8: the caller takes the matrix cores' 8-bit products.  They halve the time
// only where one tile does not hold all rows; up to F8_EXACT_ROWS sums stay in float32.
// In us, expanded and 8-bit:
//   N=32000:   R=64  33,  26   R=65  49,  31   R=320 120,  55
//   N=128255:  R=64 126, 116   R=65 156, 119   R=320 405, 200
constexpr int F8_EXACT_ROWS = 64;

struct F8Plan {
  int stream, rp, f8;
  int cn, mt, row_tiles;   // 128 cn weight rows and 64 mt rows of x a workgroup
  size_t op_bytes, bytes;
};

// Tiles of the expanded form: whichever takes the least time in whole rounds of the
// chip, a workgroup a CU.  A tile (cn, mt) takes about, in us at K = 4096,
// (1,1) 25, (2,1) 44, (1,2) 42, (2,2) 65; calls, in that order, bf16:
//   N=32000:   R=64   33,  45,  46,  61   R=128   57,  49,  47,  61   R=192   81,  85,  82,  66
//              R=320 128, 124, 118, 120   R=448  173, 159, 155, 125   R=2048 799, 673, 656, 523
//   N=128255:  R=64  126, 120, 177, 145   R=128  216, 195, 186, 157   R=192  310, 278, 340, 269
//              R=320 494, 443, 503, 397   R=448  683, 603, 669, 527   R=2048 3229, 2767, 2706, 2120
static void f8_expanded_tiles(F8Plan& p, int R, int N) {
  static const struct { int cn, mt, us; } tile[] = {{2, 2, 65}, {1, 2, 42}, {2, 1, 44}, {1, 1, 25}};
  long long best = 0;
  for (const auto& t : tile) {
    const int rows = (R + 64 * t.mt - 1) / (64 * t.mt);
    const long long sets = (long long)((N + 128 * t.cn - 1) / (128 * t.cn)) * rows, us = (sets + 255) / 256 * t.us;
    if (best && us >= best) continue;
    best = us;
    p.cn = t.cn;
    p.mt = t.mt;
    p.row_tiles = rows;
  }
}

// Column tiles of the 8-bit products, of 256 or 128 weight rows, the same way: a tile
// of 128 counted as 0.55 of one of 256, from four row tiles a wavefront on (whose
// operands it reads for half the products) as 0.62.  In us, 256 and 128 (K = 4096):
//   N=32000:   R=128  60.2, 39.5   R=320  83.4, 65.4
//   N=152064:  R=128   194,  170   R=320   279,  297
static bool f8_wide(int row_tiles, int mt, int N) {
  const long long wide = (long long)((N + 255) / 256) * row_tiles, narrow = (long long)((N + 127) / 128) * row_tiles;
  return (wide + 255) / 256 * 100 <= (narrow + 255) / 256 * (mt >= 4 ? 62 : 55);
}

// N only chooses among tiles: `bytes` is enough for every N.
static F8Plan f8_plan(bool products8, int R, int K, int N) {
  F8Plan p;
  memset(&p, 0, sizeof p);
  const int KB = (K + 127) / 128;
  p.rp = 16;
  while (p.rp / 2 >= R) p.rp /= 2;
  if (R <= 16 && f8_stream_lds(KB, p.rp) <= F8S_LDS) {
    p.stream = 1;
    return p;
  }
  p.f8 = products8 && R > F8_EXACT_ROWS;
  size_t units;   // of 64 rows
  if (p.f8) {
    // The widest tile that pads the fewest rows.  For 7, 11, 13 and 17 units of 64 rows
    // that is the narrowest one, where a wider one would take less time.  In us, as it is
    // and at its best, N = 128255:  R=448 394, 282 (mt 4)   R=640 367, 353 (mt 5)
    //   R=704 609, 418 (mt 4)   R=832 698, 504 (mt 5)   R=1088 921, 674 (mt 5)   R=2048 1140, 1140
    p.mt = 1;
    for (int mt = 2; mt <= 5; ++mt)
      if ((R + 64 * mt - 1) / (64 * mt) * mt <= (R + 64 * p.mt - 1) / (64 * p.mt) * p.mt) p.mt = mt;
    p.row_tiles = (R + 64 * p.mt - 1) / (64 * p.mt);
    p.cn = f8_wide(p.row_tiles, p.mt, N) ? 2 : 1;
    units = (size_t)p.row_tiles * p.mt;
  } else {
    f8_expanded_tiles(p, R, N);
    units = (size_t)(R + 127) / 128 * 2;
  }
  const size_t blocks = units * 2 * KB;
  p.op_bytes = blocks * (p.f8 ? f8_block_bytes<true>() : f8_block_bytes<false>());
  p.bytes = p.op_bytes + blocks * 128;
  return p;
}

// The kernel's LDS limit is raised once per device, whatever call comes first.
template <int CN, int MT, bool F8>
static hipError_t launch_f8_tile(F8Args a, hipStream_t st) {
  typedef F8Tile<CN, MT, F8> T;
  const hipError_t e = lds_limit(reinterpret_cast<const void*>(&f8_tile_kernel<CN, MT, F8>), T::LDS);
  if (e != hipSuccess) return e;
  const long long sets = (long long)((a.N + T::N - 1) / T::N) * a.row_tiles;
  a.per_xcd = (int)((sets + 7) / 8);
  hipLaunchKernelGGL((f8_tile_kernel<CN, MT, F8>), dim3((unsigned)a.per_xcd * 8), dim3(F8T_NT), T::LDS, st, a);
  return hipGetLastError();
}

template <int MT, bool F8>
static hipError_t launch_f8_tile(const F8Args& a, int cn, hipStream_t st) {
  return cn == 2 ? launch_f8_tile<2, MT, F8>(a, st) : launch_f8_tile<1, MT, F8>(a, st);
}

template <typename XT>
static hipError_t launch_f8(F8Args a, const F8Plan& p, hipStream_t st) {
  a.rp = p.rp;
  a.row_tiles = p.row_tiles;
  if (p.stream) {
    const int tiles = (a.N + 15) / 16;
    hipLaunchKernelGGL((f8_stream_kernel<XT>), dim3((unsigned)(tiles < W4S_GRID ? tiles : W4S_GRID)), dim3(F8S_NT), 0, st, a);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(p.row_tiles * 2 * p.mt * a.KB));
  if (p.f8) hipLaunchKernelGGL((f8_order_kernel<XT, true>), grid, dim3(512), 0, st, a);
  else hipLaunchKernelGGL((f8_order_kernel<XT, false>), grid, dim3(512), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.f8) {
    switch (p.mt) {
      case 1: return launch_f8_tile<1, true>(a, p.cn, st);
      case 2: return launch_f8_tile<2, true>(a, p.cn, st);
      case 3: return launch_f8_tile<3, true>(a, p.cn, st);
      case 4: return launch_f8_tile<4, true>(a, p.cn, st);
      default: return launch_f8_tile<5, true>(a, p.cn, st);
    }
  }
  return p.mt == 1 ? launch_f8_tile<1, false>(a, p.cn, st) : launch_f8_tile<2, false>(a, p.cn, st);
}

}  // namespace sl

extern "C" int spec_quantize_f8(const void* x, int x_dtype, int rows, int R, int K, uint8_t* codes, float* scales,
                                void* stream) {
  if (!known(x_dtype) || (rows != 1 && rows != SL_F8_BLOCK)) return SV_ERR_UNSUPPORTED;
  const int rc = f8_sizes(R, K);
  if (rc != SV_OK) return rc;
  if (R == 0) return SV_OK;
  if (!x || !codes || !scales) return SV_ERR_ARG;
  if (misaligned(x, size_of(x_dtype)) || misaligned(scales, 4)) return SV_ERR_ARG;
  F8QuantArgs a;
  memset(&a, 0, sizeof a);
  a.x = x;
  a.q = codes;
  a.s = scales;
  a.R = R;
  a.K = K;
  a.KB = (K + 127) / 128;
  const size_t nx = (size_t)R * K * size_of(x_dtype), ns = (size_t)((R + rows - 1) / rows) * a.KB * 4;
  if (overlap(codes, (size_t)R * K, x, nx) || overlap(scales, ns, x, nx) || overlap(scales, ns, codes, (size_t)R * K))
    return SV_ERR_ARG;
  const bool wide = K % 8 == 0 && !misaligned(x, 16) && !misaligned(codes, 8);
  hipStream_t st = (hipStream_t)stream;
  if (x_dtype == SV_BF16) return wide ? launch_quantize<uint16_t, true>(a, rows, st) : launch_quantize<uint16_t, false>(a, rows, st);
  return wide ? launch_quantize<float, true>(a, rows, st) : launch_quantize<float, false>(a, rows, st);
}

extern "C" size_t spec_logits_f8_workspace_bytes(int out_dtype, int R, int K) {
  const bool products8 = out_dtype == SL_BF16_F8;
  return (known(out_dtype) || products8) && f8_sizes(R, K) == SV_OK && K % 16 == 0 && R > 0 ? f8_plan(products8, R, K, 1).bytes : 0;
}

extern "C" int spec_logits_f8(const void* hidden, int hidden_dtype, const float* hidden_scales, const uint8_t* weights,
                              const float* scales, int R, int K, int N, void* out, int out_dtype, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const bool products8 = out_dtype == SL_BF16_F8;
  if (products8) out_dtype = SV_BF16;
  if ((!known(hidden_dtype) && hidden_dtype != SL_F8) || !known(out_dtype) || N > SV_MAX_VOCAB) return SV_ERR_UNSUPPORTED;
  const int rc = f8_sizes(R, K);
  if (rc != SV_OK) return rc;
  if (N < 1 || K % 16 != 0) return SV_ERR_ARG;
  if ((long long)R * N >= W4_MOST) return SV_ERR_UNSUPPORTED;
  if ((hidden_dtype == SL_F8) != (hidden_scales != nullptr)) return SV_ERR_ARG;
  if (R == 0) return SV_OK;
  if (!hidden || !weights || !scales || !out) return SV_ERR_ARG;
  if (misaligned(hidden, 16) || misaligned(weights, 16) || misaligned(scales, 4) || misaligned(hidden_scales, 4) ||
      misaligned(out, size_of(out_dtype)))
    return SV_ERR_ARG;
  const F8Plan p = f8_plan(products8, R, K, N);
  if (p.bytes && (!workspace || workspace_bytes < p.bytes || misaligned(workspace, 256))) return SV_ERR_WORKSPACE;
  F8Args a;
  memset(&a, 0, sizeof a);
  a.KB = (K + 127) / 128;
  const size_t no = (size_t)R * N * size_of(out_dtype), nx = (size_t)R * K * (hidden_dtype == SL_F8 ? 1 : size_of(hidden_dtype));
  if (overlap(out, no, hidden, nx) || overlap(out, no, weights, (size_t)N * K) ||
      overlap(out, no, scales, (size_t)((N + 127) / 128) * a.KB * 4) ||
      (hidden_scales && overlap(out, no, hidden_scales, (size_t)R * a.KB * 4)))
    return SV_ERR_ARG;
  a.x = hidden;
  a.xs = hidden_scales;
  a.w = weights;
  a.s = scales;
  a.out = out;
  a.R = R;
  a.K = K;
  a.N = N;
  a.out_bf16 = out_dtype == SV_BF16;
  a.xop = (char*)workspace;
  a.xsc = (float*)((char*)workspace + p.op_bytes);
  hipStream_t st = (hipStream_t)stream;
  if (hidden_dtype == SL_F8) return hip_status(launch_f8<uint8_t>(a, p, st));
  return hip_status(hidden_dtype == SV_BF16 ? launch_f8<uint16_t>(a, p, st) : launch_f8<float>(a, p, st));
}

// ---------------------------------------------------------------------------
// The token history
// ---------------------------------------------------------------------------

// The checks of both calls; SV_OK with *run = false: nothing to do.
static int check_history(const void* counts, const void* ids, const void* num, int S, int V, const void* slots, int B,
                         bool* run) {
  *run = false;
  if (V > SV_MAX_VOCAB || B > SL_MAX_ROWS) return SV_ERR_UNSUPPORTED;
  if (S < 0 || V < 1 || B < 0) return SV_ERR_ARG;
  if (!slots && B > S) return SV_ERR_ARG;
  if (B == 0 || S == 0) return SV_OK;
  if (!counts || !ids || !num) return SV_ERR_ARG;
  if (misaligned(counts, 4) || misaligned(ids, 4) || misaligned(num, 4) || misaligned(slots, 4)) return SV_ERR_ARG;
  *run = true;
  return SV_OK;
}

extern "C" int spec_history_append(int32_t* counts, int32_t* ids, int32_t* num, int S, int V, const int32_t* slots,
                                   const int32_t* tokens, int B, int T, int prompt, void* stream) {
  if (T < 1) return SV_ERR_ARG;
  if (T > (1 << 24)) return SV_ERR_UNSUPPORTED;
  bool run;
  const int rc = check_history(counts, ids, num, S, V, slots, B, &run);
  if (rc != SV_OK || !run) return rc;
  if (!tokens || misaligned(tokens, 4)) return SV_ERR_ARG;
  const int chunks = (T + HA_NT - 1) / HA_NT;
  const long long grid = (long long)B * chunks;
  if (!fits(grid, HA_NT)) return SV_ERR_UNSUPPORTED;
  const HistoryArgs a = {(uint32_t*)counts, ids, num, slots, tokens, S, V, B, T, prompt != 0, chunks};
  hipLaunchKernelGGL(history_append_kernel, dim3((unsigned)grid), dim3(HA_NT), 0, (hipStream_t)stream, a);
  return hip_status(hipGetLastError());
}

extern "C" int spec_history_reset(int32_t* counts, const int32_t* ids, int32_t* num, int S, int V,
                                  const int32_t* slots, int B, void* stream) {
  bool run;
  const int rc = check_history(counts, ids, num, S, V, slots, B, &run);
  if (rc != SV_OK || !run) return rc;
  const HistoryArgs a = {(uint32_t*)counts, const_cast<int32_t*>(ids), num, slots, nullptr, S, V, B, 0, 0, 1};
  hipLaunchKernelGGL(history_reset_kernel, dim3((unsigned)B), dim3(HR_NT), 0, (hipStream_t)stream, a);
  return hip_status(hipGetLastError());
}

// ---------------------------------------------------------------------------
// spec_process_logits
// ---------------------------------------------------------------------------

// Workgroups to spread a call over.  Where each reads lists and streams, few:
// with 1024 instead of 512, B=1000, J=5, V=1000 in fp32 takes two groups of rows
// to a sequence and 25 us, not 21.  Where it only streams, many: 2048, 4096 and
// 8192 give 142, 121 and 114 us for a masked copy (B=128, J=9, V=128256), and 27,
// 24 and 24.5 in place (B=64, J=5).  Where it only walks lists: 512 and 2048 give
// 106 and 97 us (B=256, J=8, V=152064, 2000 tokens held).
constexpr int PR_TARGET = 512;
constexpr int PR_TARGET_PLAIN = 4096;
constexpr int PR_TARGET_LISTS = 2048;
// The least elements of a piece worth a workgroup (2048: the same).
constexpr int PR_MIN_PIECE = 4096;

template <typename ET>
static int launch_process(ProcessArgs a, hipStream_t st) {
  constexpr int VEC = Elem<ET>::VEC, TILE = PR_TILE * VEC;
  const int names = a.NB + (a.drafts ? a.first + a.J - 1 : 0);
  a.hmask = 63;
  while (a.hmask + 1 < names + names / 2) a.hmask = 2 * a.hmask + 1;
  int lds = Specials::bytes(names, a.hmask);
  const bool stream = a.in != a.out || a.mask_rows, lists = names || a.counts;
  const int target = !stream ? PR_TARGET_LISTS : lists ? PR_TARGET : PR_TARGET_PLAIN;
  // With lists, a piece goes through a tile (half a tile: 390 us instead of 294 at B=256, J=8, V=152064; two to
  // four tiles a workgroup: 338).
  const int most = (a.V + PR_MIN_PIECE - 1) / PR_MIN_PIECE, least = (a.V + TILE - 1) / TILE;
  // Pieces of the vocabulary (shares of the lists), then groups of rows; with
  // no lists to read, every row by itself.
  a.groups = stream && !lists ? a.J : 1;
  const long long per = (long long)a.B * a.groups;
  const long long want = (target + per - 1) / per;
  a.pieces = (int)(want < 1 ? 1 : want);
  if (stream) {
    if (a.pieces > most) a.pieces = most;
    if (lists && a.pieces < least) a.pieces = least;
    // Whole 128-byte lines, or a whole row in whole units.
    const int round = a.pieces > 1 ? 128 / (int)sizeof(ET) : VEC;
    a.piece = ((a.V + a.pieces - 1) / a.pieces + round - 1) / round * round;
    a.pieces = (a.V + a.piece - 1) / a.piece;
    if (lists) {
      a.tile_off = (PR_ENTRIES * (int)sizeof(int2) + lds + 15) / 16 * 16;
      a.tile_rows = TILE / (a.piece + 2 * VEC);
      if (a.tile_rows > a.J) a.tile_rows = a.J;
      if (a.tile_rows < 1) a.tile_rows = 1;
      lds = a.tile_off + a.tile_rows * (a.piece + 2 * VEC) * (int)sizeof(ET);
    }
  } else if (a.pieces > 8) {
    a.pieces = 8;
  }
  if (a.groups < a.J) {
    const long long g = (target + (long long)a.B * a.pieces - 1) / ((long long)a.B * a.pieces);
    a.groups = (int)(g > a.J ? a.J : g);
  }
  const long long grid = (long long)a.B * a.pieces * a.groups;
  if (!fits(grid, PR_NT)) return SV_ERR_UNSUPPORTED;
  if (stream && lists) hipLaunchKernelGGL((process_stream_kernel<ET, true>), dim3((unsigned)grid), dim3(PR_NT), lds, st, a);
  else if (stream) hipLaunchKernelGGL((process_stream_kernel<ET, false>), dim3((unsigned)grid), dim3(PR_NT), 0, st, a);
  else hipLaunchKernelGGL((process_lists_kernel<ET>), dim3((unsigned)grid), dim3(PR_NT), lds, st, a);
  return hip_status(hipGetLastError());
}

extern "C" int spec_process_logits(const void* logits, void* out, int dtype, const int32_t* counts, const int32_t* ids,
                                   const int32_t* num, int S, const int32_t* slots, const int32_t* draft_tokens,
                                   int draft_stride, int first, const float* repetition, const float* presence,
                                   const float* frequency, const int32_t* bias_ids, const float* bias_values, int NB,
                                   const uint32_t* masks, int M, const int32_t* mask_rows, const int32_t* rows, int B,
                                   int J, int V, void* stream) {
  if (!known(dtype)) return SV_ERR_UNSUPPORTED;
  if (V > SV_MAX_VOCAB || NB > SL_MAX_BIAS || M > SL_MAX_MASKS) return SV_ERR_UNSUPPORTED;
  if (B < 0 || J < 1 || V < 1 || S < 0 || NB < 0 || M < 0 || first < 0) return SV_ERR_ARG;
  if ((long long)B * J > SL_MAX_ROWS) return SV_ERR_UNSUPPORTED;
  if (B == 0) return SV_OK;
  if (!logits || !out) return SV_ERR_ARG;
  if ((counts != nullptr) != (ids != nullptr) || (counts != nullptr) != (num != nullptr)) return SV_ERR_ARG;
  if ((counts == nullptr) != (S == 0)) return SV_ERR_ARG;
  if (counts && !slots && B > S) return SV_ERR_ARG;
  if (draft_tokens && (long long)first + J - 1 > draft_stride) return SV_ERR_ARG;
  if (draft_tokens && (long long)first + J - 1 > SL_MAX_DRAFT) return SV_ERR_UNSUPPORTED;
  if ((bias_ids != nullptr) != (NB > 0) || (bias_values != nullptr) != (NB > 0)) return SV_ERR_ARG;
  if ((masks != nullptr) != (M > 0) || (mask_rows != nullptr) != (M > 0)) return SV_ERR_ARG;
  const void* words[] = {counts, ids, num, slots, draft_tokens, repetition, presence, frequency, bias_ids, bias_values,
                         masks, mask_rows, rows};
  for (const void* p : words)
    if (misaligned(p, 4)) return SV_ERR_ARG;
  if (misaligned(logits, size_of(dtype)) || misaligned(out, size_of(dtype))) return SV_ERR_ARG;
  const size_t bytes = (size_t)B * J * V * size_of(dtype);
  if (out != logits && overlap(logits, bytes, out, bytes)) return SV_ERR_ARG;

  ProcessArgs a;
  memset(&a, 0, sizeof a);
  a.in = logits;
  a.out = out;
  a.counts = (const uint32_t*)counts;
  a.ids = ids;
  a.num = num;
  a.S = S;
  a.slots = slots;
  a.drafts = draft_tokens;
  a.draft_stride = draft_stride;
  a.first = first;
  a.rep = repetition;
  a.pres = presence;
  a.freq = frequency;
  a.bias_ids = bias_ids;
  a.bias_vals = bias_values;
  a.NB = NB;
  a.masks = masks;
  a.M = M;
  a.mask_rows = mask_rows;
  a.rows = rows;
  a.B = B;
  a.J = J;
  a.V = V;
  a.W = (V + 31) / 32;
  a.wide = !misaligned(logits, 16) && !misaligned(out, 16);
  hipStream_t st = (hipStream_t)stream;
  return dtype == SV_BF16 ? launch_process<uint16_t>(a, st) : launch_process<float>(a, st);
}

extern "C" const char* spec_logits_strerror(int code) {
  switch (code) {
    case SV_OK: return "ok";
    case SV_ERR_ARG: return "invalid argument (null pointer, size out of range or misaligned pointer)";
    case SV_ERR_UNSUPPORTED: return "unsupported dtype, group or size";
    case SV_ERR_WORKSPACE: return "workspace missing, too small or not 256-byte aligned";
    case SV_ERR_HIP: return g_errbuf[0] ? g_errbuf : "HIP error";
    default: return "unknown error code";
  }
}
