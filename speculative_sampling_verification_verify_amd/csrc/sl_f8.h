// 8-bit floating point (e4m3, 4 exponent bits, largest finite value 448) with a
// scale for each block of 128, and logits from a head of such weights:
//
//   q = e4m3(x / s),  s = max(max |x| of the block * float(1 / 448), 2^-126)
//   out[r][n] = sum_b sx[r][b] * sw[n / 128][b] * sum_{k in b} qx[r][k] * qw[n][k]
//
// The matrix cores multiply such codes at twice the rate of bf16, but they align
// the products of 8 consecutive codes to the largest and cut off what lies below
// 2^-13 of its binade (measured, the same for every instruction that takes these
// codes); only sums of those have 24 bits.  For sums of N(0, 1) values that is an
// error of about 2.5e-4 of their norm, and beside large products that cancel small
// ones are lost altogether.  Expanded to bf16, which is exact, the products are
// summed as float32.  So the codes are multiplied as they are only where the caller
// asks for it (SL_BF16_F8) and the products' rate bounds.  Everywhere else they are
// expanded.
//
// Up to 16 rows the weight bytes bound: the rows of x are quantised into LDS by
// every workgroup and the weights are streamed (f8_stream_kernel).  With more
// rows x is quantised into operand order first (f8_order_kernel), then tiles
// over rows and columns (f8_tile_kernel).  At K = 4096, bf16:
//   1 row,     N = 152064: 115 us a call, 5.4 TB/s of weight bytes (a 1 GiB copy: 5.05)
//   320 rows,  N = 128255: 405 us, 0.83 PFLOP/s; with 8-bit products 200 us, 1.68
//                          PFLOP/s (the library's product of such codes with one scale
//                          for everything, N = 128256: 260 us)
//   2048 rows, N = 152064: 2.50 ms, 1.02 PFLOP/s; with 8-bit products 1.30 ms, 1.96
//                          PFLOP/s (such a library product: 1.09 ms)
#pragma once

#include "sl_common.h"

namespace sl {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr float F8_TINY = 0x1p-126f;

struct F8Args {
  const void* x;
  const float* xs;    // scales of x where x is given as codes, else null
  const uint8_t* w;
  const float* s;
  void* out;
  int R, K, N;
  int KB;             // blocks of 128 along k
  int out_bf16;
  int rp;             // few rows: rows staged of a tile (a power of two, 16 unless R is smaller)
  int row_tiles;      // more rows: workgroup tiles over the rows
  int per_xcd;        // workgroups of one XCD
  char* xop;          // x in operand order and its scales (workspace)
  float* xsc;
};

// Eight consecutive values as float32.
__device__ __forceinline__ void f8_load(const uint16_t* p, float (&v)[8]) {
  uint32_t d[4];
  __builtin_memcpy(d, p, 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(d[i] << 16);
    v[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void f8_load(const float* p, float (&v)[8]) { __builtin_memcpy(v, p, 32); }

// The largest over 16 consecutive lanes, in every one of them.
__device__ __forceinline__ float f8_max16(float v) {
  const auto step = [](float a, int b) { return fmaxf(a, __uint_as_float((uint32_t)b)); };
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x121, 0xF, 0xF, false));   // row_ror:1
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x122, 0xF, 0xF, false));
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x124, 0xF, 0xF, false));
  return step(v, __builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x128, 0xF, 0xF, false));
}

__device__ __forceinline__ float f8_amax(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

__device__ __forceinline__ float f8_scale(float amax) { return fmaxf(amax * (1.0f / 448.0f), F8_TINY); }

// Eight codes.  The quotients are at most 448 (1 + 2^-22), which rounds to 448.
__device__ __forceinline__ uint2 f8_codes(const float (&v)[8], float s) {
  uint2 c;
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] / s, v[1] / s, 0, false);
  c.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] / s, v[3] / s, a, true);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] / s, v[5] / s, 0, false);
  c.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[6] / s, v[7] / s, a, true);
  return c;
}

// ---------------------------------------------------------------------------
// The quantiser.
// ---------------------------------------------------------------------------
constexpr int FQ_NT = 256;

struct F8QuantArgs {
  const void* x;
  uint8_t* q;
  float* s;
  int R, K, KB;
};

// Eight values from column k of a row on, zeros behind its end.  WIDE: rows of whole
// units of eight, aligned bases.
template <typename XT, bool WIDE>
__device__ __forceinline__ void fq_load(const XT* row, int k, int K, float (&v)[8]) {
  if (WIDE) {
    if (k < K) {
      f8_load(row + k, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < K ? load_in(row + k + i) : 0.0f;
  }
}

template <bool WIDE>
__device__ __forceinline__ void fq_store(uint8_t* row, int k, int K, uint2 c) {
  if (WIDE) {
    if (k < K) *reinterpret_cast<uint2*>(row + k) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) row[k + i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// A scale for each row and 128 of k: 16 lanes to a block, whose values are in
// registers from the one read to the write.  Memory bounds it: 128256 x 4096 in bf16
// with a scale a tile (below) takes 298 us, 1.58 GB at 5.3 TB/s.  Where K is no multiple of
// 8 or a base not aligned (WIDE false) values and codes go one by one: 1048 us at
// 128256 x 4095 in tiles; 4096 rows of 4096 and of 4095 with a scale a row: 12 and 27 us.
template <typename XT, bool WIDE>
__global__ __launch_bounds__(FQ_NT) void quantize_rows_kernel(F8QuantArgs a) {
  const int u = threadIdx.x & 15;
  const long long block = (long long)blockIdx.x * (FQ_NT / 16) + (threadIdx.x >> 4);
  if (block >= (long long)a.R * a.KB) return;   // 16 lanes together
  const int r = (int)(block / a.KB), b = (int)(block % a.KB), k = b * 128 + u * 8;
  float v[8];
  fq_load<XT, WIDE>(reinterpret_cast<const XT*>(a.x) + (size_t)r * a.K, k, a.K, v);
  const float s = f8_scale(f8_max16(f8_amax(v)));
  fq_store<WIDE>(a.q + (size_t)r * a.K, k, a.K, f8_codes(v, s));
  if (u == 0) a.s[block] = s;
}

// A scale for each tile of 128 x 128: one workgroup, its values in registers.
template <typename XT, bool WIDE>
__global__ __launch_bounds__(FQ_NT) void quantize_tiles_kernel(F8QuantArgs a) {
  __shared__ float part[FQ_NT / 64];
  const int u = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int rb = (int)(blockIdx.x / (unsigned)a.KB), b = (int)(blockIdx.x % (unsigned)a.KB), k = b * 128 + u * 8;
  float v[8][8], m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rb * 128 + i * 16 + r0;
    if (r < a.R) {
      fq_load<XT, WIDE>(reinterpret_cast<const XT*>(a.x) + (size_t)r * a.K, k, a.K, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, f8_amax(v[i]));
  m = f8_max16(m);
  m = fmaxf(m, __shfl_xor(m, 16, 64));
  m = fmaxf(m, __shfl_xor(m, 32, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FQ_NT / 64; ++i) m = fmaxf(m, part[i]);
  const float s = f8_scale(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rb * 128 + i * 16 + r0;
    if (r < a.R) fq_store<WIDE>(a.q + (size_t)r * a.K, k, a.K, f8_codes(v[i], s));
  }
  if (threadIdx.x == 0) a.s[blockIdx.x] = s;
}

// ---------------------------------------------------------------------------
// The rows of x as codes: eight values from column k of a row, quantised over
// the 16 lanes that hold a block (codes as they are, with their scale).
// ---------------------------------------------------------------------------
template <typename XT>
__device__ __forceinline__ uint2 f8_take(const F8Args& a, int row, int b, int k, float* s) {
  float v[8];
  fq_load<XT, true>(reinterpret_cast<const XT*>(a.x) + (size_t)row * a.K, k, a.K, v);
  *s = f8_scale(f8_max16(f8_amax(v)));
  return f8_codes(v, *s);
}
template <>
__device__ __forceinline__ uint2 f8_take<uint8_t>(const F8Args& a, int row, int b, int k, float* s) {
  uint2 c = make_uint2(0, 0);
  if (k < a.K) c = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(a.x) + (size_t)row * a.K + k);
  *s = a.xs[(size_t)row * a.KB + b];
  return c;
}

// Eight codes as bf16 values, exactly.
__device__ __forceinline__ bf16x8 f8_expand(uint32_t lo, uint32_t hi) {
  const auto pair = [](uint32_t c, bool high) {
    return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
  };
  return __builtin_bit_cast(bf16x8, u32x4{pair(lo, false), pair(lo, true), pair(hi, false), pair(hi, true)});
}

__device__ __forceinline__ i32x8 f8_join(i32x4 a, i32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// ---------------------------------------------------------------------------
// Few rows: one workgroup per CU with a run of tiles of 16 weight rows, whose
// steps of U blocks its 16 wavefronts share out evenly.  A wavefront streams
// its share without a barrier, one step ahead across tile borders; a tile that
// lies in several shares is added up at the end, in the order of the
// wavefronts.
//
// A block takes four v_mfma_f32_16x16x32_bf16: lane l holds 8 values of row /
// column l % 16 of either operand, and rows 4 * (l / 16) + 0..3 of column l % 16 of
// the result.  Which k a lane's values are is free, as long as both operands
// agree: in product t 64 (t / 2) + 16 (l / 16) + 8 (t % 2) + 0..7, so that a load of
// 16 bytes a lane takes 64 consecutive bytes of a row.
// ---------------------------------------------------------------------------
constexpr int F8S_NT = 1024;
constexpr int F8S_WAVES = F8S_NT / 64;
constexpr int F8S_LDS = 156 * 1024;
constexpr int F8S_U = 2;

template <int U> struct F8Ahead {
  i32x4 w[U][2];
  float s[U];
};

// LDS bytes of the staged rows: values [block][t][quad][rp] 16 bytes, then scales [block][16].
__host__ __device__ __forceinline__ long long f8_stream_lds(int KB, int rp) { return (long long)KB * (256 * rp + 64); }

template <typename XT>
__global__ __launch_bounds__(F8S_NT) void f8_stream_kernel(F8Args a) {
  constexpr int U = F8S_U;
  __shared__ __align__(16) char smem[F8S_LDS];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63, l16 = lane & 15,
            quad = lane >> 4;
  const int KB = a.KB, rp = a.rp;
  float* sx = reinterpret_cast<float*>(smem + KB * 256 * rp);
  const int tiles = (a.N + 15) / 16, steps = (KB + U - 1) / U;
  const int t0 = (int)((long long)tiles * blockIdx.x / gridDim.x), t1 = (int)((long long)tiles * (blockIdx.x + 1) / gridDim.x);
  const long long all = (long long)(t1 - t0) * steps;
  const int first = (int)(all * wave / F8S_WAVES), last = (int)(all * (wave + 1) / F8S_WAVES);
  int tile = t0 + first / steps, step = first % steps;
  int ftile = tile, fstep = step;

  // What lies beyond K repeats the row's end: it meets zeros of x.
  auto fetch = [&](F8Ahead<U>& h) {
    const int n0 = min(ftile * 16, a.N - 1);
    const uint8_t* w = a.w + (size_t)n0 * a.K;
    const uint32_t row = (uint32_t)min(l16, a.N - 1 - n0) * (uint32_t)a.K;
    const float* s = a.s + (size_t)(n0 / 128) * KB;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = fstep * U + u;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        h.w[u][c] = *reinterpret_cast<const i32x4*>(w + (row + (uint32_t)min(b * 128 + c * 64 + quad * 16, a.K - 16)));
      h.s[u] = s[min(b, KB - 1)];
    }
    if (++fstep == steps) {
      fstep = 0;
      ++ftile;
    }
  };
  auto store = [&](int t, const f32x4& v) {
    const int n = t * 16 + l16;
    if (n >= a.N) return;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = quad * 4 + r;
      if (row >= a.R) continue;
      const size_t o = (size_t)row * a.N + n;
      if (a.out_bf16) store_out(reinterpret_cast<uint16_t*>(a.out) + o, v[r]);
      else store_out(reinterpret_cast<float*>(a.out) + o, v[r]);
    }
  };
  f32x4 tot = {0, 0, 0, 0}, head = {0, 0, 0, 0};
  bool begun = step == 0;   // the current tile's first block is this wavefront's
  const int loff = (quad * rp + min(l16, rp - 1)) * 16;
  auto compute = [&](const F8Ahead<U>& h) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = step * U + u;
      if (b < KB) {
        const char* x = smem + b * 256 * rp + loff;
        f32x4 p = {0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < 4; ++t)
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*reinterpret_cast<const bf16x8*>(x + t * 64 * rp),
                                                      f8_expand((uint32_t)h.w[u][t >> 1][2 * (t & 1)], (uint32_t)h.w[u][t >> 1][2 * (t & 1) + 1]), p, 0, 0, 0);
        const f32x4 s4 = *reinterpret_cast<const f32x4*>(sx + b * 16 + quad * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) tot[r] = __builtin_fmaf(h.s[u] * s4[r], p[r], tot[r]);
      }
    }
    if (++step == steps) {
      if (begun) store(tile, tot);
      else head = tot;
      tot = f32x4{0, 0, 0, 0};
      step = 0;
      ++tile;
      begun = true;
    }
  };

  F8Ahead<U> ha, hb;
  const int n = last - first;
  if (n > 0) fetch(ha);
  for (int q = threadIdx.x; q < KB * rp * 16; q += F8S_NT) {
    const int u = q & 15, r = q >> 4 & (rp - 1), b = (q >> 4) / rp, k = b * 128 + u * 8;
    float s;
    const uint2 c = f8_take<XT>(a, min(r, a.R - 1), b, k, &s);
    const int t = (u >> 3) * 2 + (u & 1);
    *reinterpret_cast<bf16x8*>(smem + b * 256 * rp + ((t * 4 + (u >> 1 & 3)) * rp + r) * 16) = f8_expand(c.x, c.y);
    if (u == 0) sx[b * 16 + r] = s;
  }
  __syncthreads();
  for (int i = 0; i < n; i += 2) {
    if (i + 1 < n) fetch(hb);
    compute(ha);
    if (i + 1 >= n) break;
    if (i + 2 < n) fetch(ha);
    compute(hb);
  }

  // What is left in tot: a tile that the next wavefronts go on with, begun
  // here, or all of this share is inside a tile.
  if (n > 0 && step > 0 && !begun) head = tot;
  f32x4* part = reinterpret_cast<f32x4*>(smem);   // [wave][lane], over the staged rows
  __syncthreads();
  part[wave * 64 + lane] = head;
  __syncthreads();
  if (n > 0 && step > 0 && begun) {
    const long long end = (long long)(tile - t0 + 1) * steps;
    for (int w = wave + 1; w < F8S_WAVES && all * w / F8S_WAVES < end; ++w) tot += part[w * 64 + lane];
    store(tile, tot);
  }
}

// ---------------------------------------------------------------------------
// More rows: x into operand order first.  A block of 128 k is two products
// v_mfma_f32_32x32x64_f8f6f4 (F8) or eight v_mfma_f32_32x32x16_bf16: lane l holds 32
// or 8 values of row / column l % 32 of either operand, and rows 8 * (r / 4) +
// 4 * (l / 32) + r % 4 of column l % 32 of the result.  A lane's values of a block
// are k = 64 (l / 32) + 0..63, in their order.
//
// One workgroup per 32 rows and block.  xop: [row tile][block] of 4 KB, [16 codes][lane] (F8),
// or of 8 KB, [8 values][lane]; xsc: [row tile][block][row].  Rows beyond R and k beyond K
// are zeros.
// ---------------------------------------------------------------------------
template <bool F8> __host__ __device__ constexpr int f8_block_bytes() { return F8 ? 4096 : 8192; }

template <typename XT, bool F8>
__global__ __launch_bounds__(512) void f8_order_kernel(F8Args a) {
  const int rt = (int)(blockIdx.x / (unsigned)a.KB), b = (int)(blockIdx.x % (unsigned)a.KB);
  const int r = threadIdx.x >> 4, u = threadIdx.x & 15;
  const int row = rt * 32 + r;
  uint2 c = make_uint2(0, 0);
  float s = 0.0f;
  if (row < a.R) c = f8_take<XT>(a, row, b, b * 128 + u * 8, &s);   // 16 lanes together
  const int lane = (u >> 3) * 32 + r;
  char* o = a.xop + (size_t)blockIdx.x * f8_block_bytes<F8>();
  if (F8) *reinterpret_cast<uint2*>(o + (u >> 1 & 3) * 1024 + lane * 16 + (u & 1) * 8) = c;
  else *reinterpret_cast<bf16x8*>(o + (u & 7) * 1024 + lane * 16) = f8_expand(c.x, c.y);
  if (u == 0) a.xsc[(size_t)blockIdx.x * 32 + r] = s;
}

// 16 (or 4) bytes a lane from memory (base + a lane's offset) into consecutive LDS
// from byte `at` on, past the registers.  In assembly, because the compiler lets
// any later read of LDS wait for such a load: who uses this waits himself
// (f8_landed), before he reads what it brings, and has read what lay there before.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // (m0 named as written: that the compiler then sets it again is meant)
__device__ __forceinline__ void f8_to_lds(const void* base, uint32_t off, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void f8_word_to_lds(const void* base, uint32_t off, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(at), "v"(off), "s"(base) : "memory", "m0");
}
#pragma clang diagnostic pop
// All but the last N of this wavefront's loads have landed.
template <int N> __device__ __forceinline__ void f8_landed() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// What this wavefront's lanes wrote to LDS before is there for all of them after it.
__device__ __forceinline__ void f8_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Eight wavefronts, four along the weight rows (32 CN of them each) by two along
// the rows of x (32 MT each).  Weight rows are the products' rows, rows of x
// their columns: a lane's results share a row of x, hence one scale a block.
// Both come from memory into LDS without registers in between, in as many
// buffers as fit, all but one block ahead, with one barrier a block.  The weights
// are loaded in whole lines and read in operand order; position q of a row holds
// its 16-byte unit q ^ (row / 2 % 8), so that the reads do not conflict (4 cycles a
// 16-byte read of a wavefront, measured alone; with row % 8, 8).
// At R = 2048, N = 152064, K = 4096: 8-bit products, matrix cores busy 46% of the time,
// vector units 40% (mostly the scaling), at 2.0 GHz, without its loads 1.03 ms of 1.30;
// expanded, matrix cores 45%, vector units 39% (the expansion and the scaling), and two
// row tiles a wavefront are what LDS holds twice beside 256 weight rows.
constexpr int F8T_NT = 512;
constexpr int F8T_SW = 4096;   // bytes of the weights' scales: SL_MAX_K / 128 blocks, twice

template <int CN, int MT, bool F8> struct F8Tile {
  static constexpr int N = 128 * CN;                                       // weight rows of a workgroup
  static constexpr int WL = N * 128, XB = f8_block_bytes<F8>(), XL = 2 * MT * XB, SL = F8T_NT * 4;
  static constexpr int STAGE = WL + XL + SL;                               // weights, operands of x, their scales
  static constexpr int FIT = (160 * 1024 - F8T_SW) / STAGE, STAGES = FIT > 6 ? 6 : FIT;
  static constexpr int WI = WL / 8192, XI = XL / 8192, LOADS = WI + XI + 1;   // of 1 KB; loads a wavefront and block
  static constexpr int PITCH = 32 * CN * 4 + 16, OUT = 8 * 32 * PITCH;     // results on their way out
  static constexpr int LDS = F8T_SW + (STAGES * STAGE > OUT ? STAGES * STAGE : OUT);
  static_assert(STAGES >= 2 && LDS <= 160 * 1024 && LOADS * (STAGES - 2) < 64, "a workgroup's LDS, the count of loads");
};

template <int CN, int MT, bool F8>
__global__ __launch_bounds__(F8T_NT, 2) void f8_tile_kernel(F8Args a) {
  typedef F8Tile<CN, MT, F8> T;
  constexpr int N = T::N, WL = T::WL, XB = T::XB, WI = T::WI, XI = T::XI, AHEAD = T::STAGES - 1;
  extern __shared__ __align__(16) char lds[];              // the weights' scales, then the stages
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wave & 3, wr = wave >> 2;
  int lane = tid & 63;
  const int KB = a.KB;
  const long long sets = (long long)((a.N + N - 1) / N) * a.row_tiles;
  // The row tiles of a column tile run on one XCD, one after the other.
  const long long set = (long long)(blockIdx.x & 7) * a.per_xcd + (blockIdx.x >> 3);
  if (set >= sets) return;
  const int rt = (int)(set % a.row_tiles) * 2 * MT;        // of 32 rows
  const int n0 = (int)(set / a.row_tiles) * N;
  const char* xop = a.xop + (size_t)rt * KB * XB;
  const char* xsc = reinterpret_cast<const char*>(a.xsc + (size_t)rt * KB * 32);
  const uint8_t* wbase = a.w + (size_t)n0 * a.K;
  // What lies behind the last weight row repeats it; what lies beyond K repeats
  // the row's end, and meets zeros of x.
  const int wlast = a.N - 1 - n0;
  const uint32_t xlen = (uint32_t)KB * XB;   // bytes of a row tile
  auto load = [&](int b, int stage) __attribute__((always_inline)) {
    const uint32_t to = lds0 + F8T_SW + (uint32_t)(stage * T::STAGE);
#pragma unroll
    for (int i = 0; i < WI; ++i) {
      const int unit = (lane & 7) ^ (((i & 1) << 2) + (lane >> 4));   // rows (wave WI + i) 8 + lane / 8
      f8_to_lds(wbase, (uint32_t)min((wave * WI + i) * 8 + (lane >> 3), wlast) * (uint32_t)a.K + (uint32_t)min(b * 128 + unit * 16, a.K - 16),
                to + (wave * WI + i) * 1024);
    }
    const char* from = xop + (size_t)b * XB;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int at = (i * 8 + wave) * 1024, m = at / XB;
      f8_to_lds(from + ((size_t)m * xlen + at % XB), lane * 16, to + WL + at);
    }
    // The scales of two row tiles (every wavefront loads some, so that all wait for the same number of loads).
    const int st = min(wave, MT - 1) * 2;
    f8_word_to_lds(xsc + ((size_t)st * KB + b) * 128, (uint32_t)(lane >> 5) * (uint32_t)KB * 128 + (lane & 31) * 4, to + WL + T::XL + wave * 256);
  };
  f32x16 tot[CN][MT];
#pragma unroll
  for (int c = 0; c < CN; ++c)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) tot[c][m][r] = 0.0f;
  f32x16 zero;
#pragma unroll
  for (int r = 0; r < 16; ++r) zero[r] = 0.0f;

  // The weights' scales of the workgroup's one or two blocks of 128 rows.
  float* sws = reinterpret_cast<float*>(lds);
  for (int i = tid; i < CN * KB; i += F8T_NT) sws[i] = a.s[(size_t)min(n0 / 128 + i / KB, (a.N - 1) / 128) * KB + i % KB];
  f8_landed<0>();
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (i < KB) load(i, i);
  int stage = 0;
  for (int b = 0; b < KB; ++b) {
    // This wavefront's loads of the block have landed, and everyone's; the buffer
    // of the block before has been read.
    if (b + AHEAD <= KB) f8_landed<T::LOADS * (AHEAD - 1)>();
    else f8_landed<0>();
    __syncthreads();
    const float swb = sws[(CN > 1 ? wn >> 1 : 0) * KB + b];
    asm volatile("" : "+v"(lane));   // what follows from it is formed again in each block: registers are short
    const int l32 = lane & 31, half = lane >> 5;
    const uint32_t at = (uint32_t)(F8T_SW + stage * T::STAGE);
    // Unit 4 half + q of a row, q = 0..3, lies at position (4 half ^ row / 2 % 8) ^ q.
    const uint32_t wl = at + (uint32_t)((wn * 32 * CN + l32) * 128), wq = (uint32_t)(((half * 4) ^ (l32 >> 1 & 7)) << 4);
    const char* xl = lds + at + WL + wr * MT * XB + lane * 16;
    const float* sl = reinterpret_cast<const float*>(lds + at + WL + T::XL + wr * MT * 128) + l32;
    i32x4 wv[CN][4];
    auto read_w = [&](int c, int q) __attribute__((always_inline)) {
      wv[c][q] = *reinterpret_cast<const i32x4*>(lds + wl + (wq ^ (q << 4)) + c * 4096);
    };
    auto next = [&]() __attribute__((always_inline)) {   // the loads of the block furthest ahead
      if (b + AHEAD < KB) load(b + AHEAD, stage == 0 ? AHEAD : stage - 1);
      stage = stage == AHEAD ? 0 : stage + 1;
    };
    if constexpr (F8) {
      // What the first products need is read first, then the next block's loads
      // go out.  Step (m, c): two products, and in their shade the scaling of the
      // step before.
      constexpr int XD = MT < 5 ? 2 : 1;   // the operands of a row tile are read while those of the last one are in use
      f32x16 p[2];
      i32x8 xv[XD][2];
      auto read_x = [&](int m) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          xv[m % XD][j] = f8_join(*reinterpret_cast<const i32x4*>(xl + m * XB + j * 2048), *reinterpret_cast<const i32x4*>(xl + m * XB + j * 2048 + 1024));
      };
      read_w(0, 0);
      read_w(0, 1);
      read_x(0);
      read_w(0, 2);
      read_w(0, 3);
      float sx[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) sx[m] = sl[m * 32];
      __builtin_amdgcn_sched_barrier(0);
      next();
#pragma unroll
      for (int c = 1; c < CN; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) read_w(c, q);
#pragma unroll
      for (int q = 0; q <= CN * MT; ++q) {
        const int m = q / CN, c = q % CN, mb = (q - 1) / CN, cb = (q - 1) % CN;
        if (q > 0 && cb == 0) sx[mb] *= swb;
        if (q < CN * MT) {
          if (XD == 1 && c == 0 && m > 0) read_x(m);
          p[q & 1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f8_join(wv[c][0], wv[c][1]), xv[m % XD][0], zero, 0, 0, 0, 0, 0, 0);
          p[q & 1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f8_join(wv[c][2], wv[c][3]), xv[m % XD][1], p[q & 1], 0, 0, 0, 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
          if (XD == 2 && c == 0 && m + 1 < MT) read_x(m + 1);
        }
        if (q > 0) {
#pragma unroll
          for (int r = 0; r < 16; ++r) tot[cb][mb][r] = __builtin_fmaf(sx[mb], p[(q - 1) & 1][r], tot[cb][mb][r]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      next();
#pragma unroll
      for (int c = 0; c < CN; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) read_w(c, q);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x16 p[CN];
#pragma unroll
        for (int c = 0; c < CN; ++c) p[c] = zero;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const bf16x8 xv = *reinterpret_cast<const bf16x8*>(xl + m * XB + t * 1024);
#pragma unroll
          for (int c = 0; c < CN; ++c)
            p[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f8_expand((uint32_t)wv[c][t >> 1][2 * (t & 1)], (uint32_t)wv[c][t >> 1][2 * (t & 1) + 1]), xv, p[c], 0, 0, 0);
        }
        const float sx = sl[m * 32] * swb;
#pragma unroll
        for (int c = 0; c < CN; ++c)
#pragma unroll
          for (int r = 0; r < 16; ++r) tot[c][m][r] = __builtin_fmaf(sx, p[c][r], tot[c][m][r]);
      }
    }
  }

  // The results through LDS, so that whole lines are written: a wavefront's
  // 32 rows of 32 CN values at a time.
  __syncthreads();
  const int l32 = lane & 31, half = lane >> 5;
  const int nw = n0 + wn * 32 * CN, cols = min(a.N - nw, 32 * CN);
  const int es = a.out_bf16 ? 2 : 4, pitch = 32 * CN * es + 16;
  char* mine = lds + F8T_SW + wave * 32 * T::PITCH;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    char* put = mine + l32 * pitch;
#pragma unroll
    for (int c = 0; c < CN; ++c)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = c * 32 + 8 * g + 4 * half;
        const f32x4 v = {tot[c][m][4 * g], tot[c][m][4 * g + 1], tot[c][m][4 * g + 2], tot[c][m][4 * g + 3]};
        if (a.out_bf16) {
          const uint2 h = make_uint2(to_bf16(v[0]) | (uint32_t)to_bf16(v[1]) << 16, to_bf16(v[2]) | (uint32_t)to_bf16(v[3]) << 16);
          *reinterpret_cast<uint2*>(put + n * 2) = h;
        } else {
          *reinterpret_cast<f32x4*>(put + n * 4) = v;
        }
      }
    f8_wave_sync();   // the lanes read what others wrote
    const int row0 = (rt + wr * MT + m) * 32, unit = 16 / es, per = 32 * CN / unit;   // 16-byte units of a row
    char* out = reinterpret_cast<char*>(a.out);
    for (int u = lane; u < 32 * per; u += 64) {
      const int r = u / per, n = u % per * unit;
      if (row0 + r >= a.R) continue;
      const char* from = mine + r * pitch + n * es;
      char* to = out + ((size_t)(row0 + r) * a.N + nw + n) * es;
      if (n + unit <= cols) {
        __builtin_memcpy(to, from, 16);
      } else {
        for (int e = 0; n + e < cols; ++e) {
          if (a.out_bf16) __builtin_memcpy(to + e * 2, from + e * 2, 2);
          else __builtin_memcpy(to + e * 4, from + e * 4, 4);
        }
      }
    }
    f8_wave_sync();   // and have read it before the next row tile's are written
  }
}

}  // namespace sl
