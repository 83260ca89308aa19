// The operators between a model and the verify / sampling calls, for MI355X
// (gfx950): kernels and their C ABI (see spec_logits.h).

#include "sl_w4.h"
#include "sl_process.h"

#include <stdio.h>
#include <string.h>

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
