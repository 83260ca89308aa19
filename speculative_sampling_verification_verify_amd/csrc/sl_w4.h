// Logits from a head of 4-bit weights with group scales:
//
//   out[r][n] = sum_g s[n][g] * sum_{k in g} (w[n][k] - z[n][g]) * x[r][k].
//
// The inner sums run on the matrix cores in bf16 with float32 accumulators: a
// weight enters as the bf16 number w, the products w x are exact, and what the
// zero point is too much, z times the sum of the x, is taken out in float32
// within 256 of k.  As the fp8 (e4m3) number with its code, a nibble is w * 2^-9
// (codes 0..7 are the subnormals, 8..15 the binade above them, in the same
// steps), so one conversion with a scale of 2^9 gives two weights: with the
// nibbles taken apart, seven operations for eight.  (16 + w, as 0x4180 + 8 w,
// takes eight, and its sums are three times as large.)  fp32 hidden states are
// split into three bf16 parts (8 + 8 + 8 significand bits, truncated, so the
// parts add up to the value exactly) that take a product each: of 8 consecutive
// k, an instruction cuts off what lies below the last bit of the largest
// product, so parts of different size do not share one.
//
// Two forms.  Up to 16 rows (32 where K is short) the weight bytes bound: the
// rows of x stay in LDS and the weights are streamed (w4_stream_kernel).  With
// more rows the products count too: tiles over rows and columns, x brought into
// operand order first (w4_order_kernel, w4_tile_kernel).  Rows of x are the
// products' rows, rows of the weight matrix their columns: the results that a
// lane holds share one weight row, hence one scale.
#pragma once

#include "sl_common.h"

namespace sl {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct W4Args {
  const void* x;
  const uint8_t* w;
  const void* s;
  const uint8_t* z;   // or null
  void* out;
  int R, K, N;
  int G;              // groups per weight row
  int gb;             // 128-k blocks per group (1 where the group is 32 or 64)
  int out_bf16;
  int rp;             // few rows: rows staged of a tile (a power of two, 16 unless R is smaller)
  int row_tiles;      // more rows: tiles of MT * 32 rows
  int per_xcd;        // workgroups of one XCD
  char* xop;          // x in operand order and its sums per group (workspace)
  char* xsum;
};

// The eight weights of a word as bf16 numbers, in the order 0 2 4 6 1 3 5 7.
__device__ __forceinline__ uint32_t w4_pair(uint32_t codes) {        // of the lower two bytes
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 512.0f, false));
}
__device__ __forceinline__ uint32_t w4_pair_high(uint32_t codes) {   // of the upper two
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 512.0f, true));
}
__device__ __forceinline__ bf16x8 w4_expand(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  return __builtin_bit_cast(bf16x8, u32x4{w4_pair(even), w4_pair_high(even), w4_pair(odd), w4_pair_high(odd)});
}

// Eight consecutive bf16 values in the same order.
__device__ __forceinline__ bf16x8 w4_order(uint4 a) {
  uint4 v;
  v.x = __builtin_amdgcn_perm(a.y, a.x, 0x05040100u);
  v.y = __builtin_amdgcn_perm(a.w, a.z, 0x05040100u);
  v.z = __builtin_amdgcn_perm(a.y, a.x, 0x07060302u);
  v.w = __builtin_amdgcn_perm(a.w, a.z, 0x07060302u);
  return __builtin_bit_cast(bf16x8, v);
}

template <typename XT> struct W4Hidden;

template <> struct W4Hidden<uint16_t> {
  static constexpr int PARTS = 1;
  __device__ __forceinline__ static void load(const uint16_t* p, bf16x8 (&f)[1]) {
    f[0] = w4_order(*reinterpret_cast<const uint4*>(p));
  }
};

template <> struct W4Hidden<float> {
  static constexpr int PARTS = 3;
  __device__ __forceinline__ static void load(const float* p, bf16x8 (&f)[3]) {
    uint32_t h[8], m[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = p[i];
      h[i] = __float_as_uint(v) & 0xFFFF0000u;
      const float r = v - __uint_as_float(h[i]);
      m[i] = __float_as_uint(r) & 0xFFFF0000u;
      l[i] = __float_as_uint(r - __uint_as_float(m[i]));
    }
    f[0] = pack(h);
    f[1] = pack(m);
    f[2] = pack(l);
  }
  // The upper halves of eight words in the order 0 2 4 6 1 3 5 7.
  __device__ __forceinline__ static bf16x8 pack(const uint32_t (&u)[8]) {
    uint4 v;
    v.x = __builtin_amdgcn_perm(u[2], u[0], 0x07060302u);
    v.y = __builtin_amdgcn_perm(u[6], u[4], 0x07060302u);
    v.z = __builtin_amdgcn_perm(u[3], u[1], 0x07060302u);
    v.w = __builtin_amdgcn_perm(u[7], u[5], 0x07060302u);
    return __builtin_bit_cast(bf16x8, v);
  }
};

// The words of the four lanes that share a weight row, transposed: a lane's
// word i becomes word (lane / 16) of the quarter i, so that word i of all four
// lanes together is the 32 consecutive k of quarter i.
__device__ __forceinline__ void w4_transpose(uint32_t (&d)[4]) {
  auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  d[0] = c[0];
  d[1] = c[1];
  d[2] = e[0];
  d[3] = e[1];
}


// What a wavefront fetches ahead of one column tile: U blocks of 128 k with
// their scales and zeros.
template <typename ST, int SUB, int U>
struct W4Ahead {
  static constexpr int NS = U * SUB;                               // scales
  static constexpr int SW = (NS * (int)sizeof(ST) + 3) / 4, ZW = (NS + 3) / 4;
  u32x4 w[U];
  uint32_t s[SW], z[ZW];
};

__device__ __forceinline__ float w4_get(const uint32_t* w, int i, const uint16_t*) {
  return __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
}
__device__ __forceinline__ float w4_get(const uint32_t* w, int i, const float*) { return __uint_as_float(w[i]); }
__device__ __forceinline__ void w4_put(uint32_t* w, int i, uint16_t v) { w[i >> 1] |= (uint32_t)v << (16 * (i & 1)); }
__device__ __forceinline__ void w4_put(uint32_t* w, int i, float v) { w[i] = __float_as_uint(v); }

// The zero point of entry i.
__device__ __forceinline__ float w4_zero(const W4Args& a, const uint32_t* z, int i) {
  return (float)(a.z ? (z[i >> 2] >> (8 * (i & 3))) & 15u : 8u);
}

// Sixteen weight rows of a column tile: their first row (uniform over the
// wavefront), and the lane's row from there on (the last one of the matrix
// where the tile goes on behind it).
struct W4Rows {
  size_t first;
  uint32_t local;
};
__device__ __forceinline__ W4Rows w4_rows(const W4Args& a, int n0, int l16) {
  W4Rows r;
  const int n = min(n0, a.N - 1);
  r.first = (size_t)n;
  r.local = (uint32_t)min(l16, a.N - 1 - n);
  return r;
}

// The group of entry j (an entry: 128 / SUB of k).
__device__ __forceinline__ uint32_t w4_group(const W4Args& a, int j) {
  return (uint32_t)min(a.gb == 1 ? j : j / a.gb, a.G - 1);
}

// COUNT scales of the lane's row from entry j on.  TOGETHER: they lie side by
// side inside the row; else one by one, and entries behind the row's end repeat
// its last.
template <typename ST, int COUNT, bool TOGETHER, int SW>
__device__ __forceinline__ void w4_fetch_scales(const W4Args& a, uint32_t (&sw)[SW], const W4Rows& r, int j) {
  const ST* s = reinterpret_cast<const ST*>(a.s) + r.first * a.G;
  const uint32_t row = r.local * (uint32_t)a.G;
  if (TOGETHER) {
    __builtin_memcpy(sw, s + (row + (uint32_t)j), COUNT * sizeof(ST));
  } else {
#pragma unroll
    for (int i = 0; i < SW; ++i) sw[i] = 0;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) w4_put(sw, i, s[row + w4_group(a, j + i)]);
  }
}

// The same for the zero points, where there are any.
template <int COUNT, bool TOGETHER, int ZW>
__device__ __forceinline__ void w4_fetch_zeros(const W4Args& a, uint32_t (&zw)[ZW], const W4Rows& r, int j) {
  if (!a.z) return;
  const uint8_t* z = a.z + r.first * a.G;
  const uint32_t row = r.local * (uint32_t)a.G;
  if (TOGETHER) {
    __builtin_memcpy(zw, z + (row + (uint32_t)j), COUNT);
  } else {
#pragma unroll
    for (int i = 0; i < ZW; ++i) zw[i] = 0;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) zw[i >> 2] |= (uint32_t)z[row + w4_group(a, j + i)] << (8 * (i & 3));
  }
}

// Blocks b .. b + U - 1 of a column tile.  What lies beyond K repeats the
// row's end: it meets zeros of x.
template <typename ST, int SUB, int U>
__device__ __forceinline__ void w4_fetch(const W4Args& a, W4Ahead<ST, SUB, U>& h, const W4Rows& r, int quad, int b) {
  constexpr int NS = W4Ahead<ST, SUB, U>::NS;
  const uint8_t* w = a.w + r.first * (size_t)(a.K / 2);
  const uint32_t row = r.local * (uint32_t)(a.K / 2);
#pragma unroll
  for (int u = 0; u < U; ++u)
    h.w[u] = *reinterpret_cast<const u32x4*>(w + (row + (uint32_t)min((b + u) * 64 + quad * 16, a.K / 2 - 16)));
  if (a.gb == 1 && (b + U) * SUB <= a.G) {
    w4_fetch_scales<ST, NS, true>(a, h.s, r, b * SUB);
    w4_fetch_zeros<NS, true>(a, h.z, r, b * SUB);
  } else {
    w4_fetch_scales<ST, NS, false>(a, h.s, r, b * SUB);
    w4_fetch_zeros<NS, false>(a, h.z, r, b * SUB);
  }
}

// Block u of what was fetched, times the rows of x in LDS, onto tot.  x: the
// operands of this block and lane, `mx` bytes from one row tile to the next,
// `frag` from one operand to the next; xsum: the sums of this block and lane,
// `ms` bytes from one row tile to the next.
template <typename XT, typename ST, int SUB, int MT, int U>
__device__ __forceinline__ void w4_block(const W4Args& a, const W4Ahead<ST, SUB, U>& h, int u, const char* x, int mx, int frag,
                                         const char* xsum, int ms, f32x4 (&tot)[MT]) {
  constexpr int P = W4Hidden<XT>::PARTS, IG = 4 / SUB;   // operands of 32 k in a group
  uint32_t d[4] = {h.w[u].x, h.w[u].y, h.w[u].z, h.w[u].w};
  if (SUB > 1) w4_transpose(d);
#pragma unroll
  for (int sg = 0; sg < SUB; ++sg) {
    f32x4 blk[MT];
#pragma unroll
    for (int i = 0; i < IG; ++i) {
      const bf16x8 wv = w4_expand(d[sg * IG + i]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int p = P - 1; p >= 0; --p) {
          const bf16x8 f = *reinterpret_cast<const bf16x8*>(x + m * mx + ((sg * IG + i) * P + p) * frag);
          blk[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, wv, i == 0 && p == P - 1 ? f32x4{0, 0, 0, 0} : blk[m], 0, 0, 0);
        }
      }
    }
    const float sc = w4_get(h.s, u * SUB + sg, (const ST*)nullptr), zz = w4_zero(a, h.z, u * SUB + sg);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const f32x4 x4 = *reinterpret_cast<const f32x4*>(xsum + m * ms + sg * 64);
#pragma unroll
      for (int r = 0; r < 4; ++r) tot[m][r] = __builtin_fmaf(sc, __builtin_fmaf(-zz, x4[r], blk[m][r]), tot[m][r]);
    }
  }
}

// The rows of x into LDS as the products' operands: [MT][block][i][part][quad][rp] 16 bytes, and their sums per group
// (products with ones): [MT][block][SUB][16].  The rows
// are ready when this returns.
template <typename XT, int SUB, int MT, int NTHR>
__device__ __forceinline__ void w4_stage(const W4Args& a, int nblk, int rp, char* xs, float* sums) {
  constexpr int P = W4Hidden<XT>::PARTS;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, l16 = lane & 15, quad = lane >> 4;
  const int frag = 64 * rp, loff = (quad * rp + min(l16, rp - 1)) * 16;
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
  const XT* x = reinterpret_cast<const XT*>(a.x);
  const int units = nblk * 4 * MT * 4 * rp;
  for (int q = tid; q < units; q += NTHR) {
    const int r = q & (rp - 1), rest0 = q / rp, qd = rest0 & 3, rest = rest0 >> 2;
    const int m = rest % MT, i = rest / MT & 3, lb = rest / MT >> 2;
    const int k = lb * 128 + (SUB > 1 ? i * 32 + qd * 8 : qd * 32 + i * 8);
    const int row = min(m * 16 + r, a.R - 1);
    bf16x8 f[P];
    if (k < a.K) {
      W4Hidden<XT>::load(x + (size_t)row * a.K + k, f);
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) f[p] = __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0});
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
      *reinterpret_cast<bf16x8*>(xs + (((m * nblk + lb) * 4 + i) * P + p) * frag + (qd * rp + r) * 16) = f[p];
  }
  __syncthreads();
  for (int q = wave; q < nblk * MT; q += NTHR / 64) {
    const int m = q % MT, lb = q / MT;
    f32x4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int p = P - 1; p >= 0; --p)
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            *reinterpret_cast<const bf16x8*>(xs + (((m * nblk + lb) * 4 + i) * P + p) * frag + loff), ones, sum, 0, 0, 0);
      if (SUB == 4 || (SUB == 2 && (i & 1)) || i == 3) {
        const int sg = SUB == 4 ? i : SUB == 2 ? i >> 1 : 0;
        if (l16 == 0) *reinterpret_cast<f32x4*>(sums + ((m * nblk + lb) * SUB + sg) * 16 + quad * 4) = sum;
        sum = f32x4{0, 0, 0, 0};
      }
    }
  }
  __syncthreads();
}

template <int MT>
__device__ __forceinline__ void w4_store(const W4Args& a, int n0, const f32x4 (&tot)[MT]) {
  const int n = n0 + (threadIdx.x & 15), quad = (threadIdx.x >> 4) & 3;
  if (n >= a.N) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = m * 16 + quad * 4 + r;
      if (row >= a.R) continue;
      const size_t o = (size_t)row * a.N + n;
      if (a.out_bf16) store_out(reinterpret_cast<uint16_t*>(a.out) + o, tot[m][r]);
      else store_out(reinterpret_cast<float*>(a.out) + o, tot[m][r]);
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows, all of them in LDS for the whole call: one workgroup per CU with a
// run of column tiles, whose blocks its 16 wavefronts share out evenly, U at a
// time.  A wavefront streams its share without a barrier, fetching one step
// ahead across tile borders; a tile that lies in several shares is added up at
// the end, in the order of the wavefronts.
//
// v_mfma_f32_16x16x32_bf16: lane l holds row / column l % 16 of either operand
// at k = 8 * (l / 16) + 0..7, and rows 4 * (l / 16) + 0..3 of column l % 16 of
// the result.
//
// Bound by the weight bytes.  R=1, K=4096, N=152064, groups of 128 with zeros:
// 65 us, 5.0 TB/s (a 1 GiB copy moves 5.1 TB/s), 12% of the matrix cores; R=16:
// 78 us.  A first form, one wavefront to 16 columns with x from the cache, took
// 187 us; one with x in LDS, a barrier for each set of columns and no even
// shares, 129 us.  R=1, K=2048, N=32000, groups of 64: 11.6 us for 34.9 MB, of
// which filling the 256 CUs' pipelines once is about half.
// ---------------------------------------------------------------------------
constexpr int W4S_NT = 1024;
constexpr int W4S_WAVES = W4S_NT / 64;
constexpr int W4S_LDS = 156 * 1024;
constexpr int W4S_U = 4;

template <typename XT, typename ST, int SUB, int MT>
__global__ __launch_bounds__(W4S_NT) void w4_stream_kernel(W4Args a) {
  constexpr int P = W4Hidden<XT>::PARTS, U = W4S_U;
  __shared__ __align__(16) char smem[W4S_LDS];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l16 = lane & 15, quad = lane >> 4;
  const int nblk = (a.K + 127) / 128, rp = a.rp;
  const int frag = 64 * rp, loff = (quad * rp + min(l16, rp - 1)) * 16;
  float* sums = reinterpret_cast<float*>(smem + nblk * 4 * P * MT * frag);

  const int tiles = (a.N + 15) / 16, steps = (nblk + U - 1) / U;   // steps of U blocks per tile
  const int t0 = (int)((long long)tiles * blockIdx.x / gridDim.x), t1 = (int)((long long)tiles * (blockIdx.x + 1) / gridDim.x);
  const long long all = (long long)(t1 - t0) * steps;
  const int first = (int)(all * wave / W4S_WAVES), last = (int)(all * (wave + 1) / W4S_WAVES);
  int tile = t0 + first / steps, step = first % steps;             // of what is computed
  int ftile = tile, fstep = step;                                  // of what is fetched

  auto fetch = [&](W4Ahead<ST, SUB, U>& h) {
    w4_fetch<ST, SUB, U>(a, h, w4_rows(a, ftile * 16, l16), quad, fstep * U);
    if (++fstep == steps) {
      fstep = 0;
      ++ftile;
    }
  };
  f32x4 tot[MT], head[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) tot[m] = head[m] = f32x4{0, 0, 0, 0};
  bool begun = step == 0;   // the current tile's first block is this wavefront's
  auto compute = [&](const W4Ahead<ST, SUB, U>& h) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (step * U + u < nblk) {
        const int b = step * U + u;
        w4_block<XT, ST, SUB, MT, U>(a, h, u, smem + b * 4 * P * frag + loff, nblk * 4 * P * frag, frag,
                                     reinterpret_cast<const char*>(sums + b * SUB * 16 + quad * 4), nblk * SUB * 64, tot);
      }
      __builtin_amdgcn_sched_barrier(0);   // no block's operands are loaded ahead: 128 registers for 16 wavefronts
    }
    if (++step == steps) {
      if (begun) {
        w4_store<MT>(a, tile * 16, tot);
      } else {
#pragma unroll
        for (int m = 0; m < MT; ++m) head[m] = tot[m];
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) tot[m] = f32x4{0, 0, 0, 0};
      step = 0;
      ++tile;
      begun = true;
    }
  };

  W4Ahead<ST, SUB, U> ha, hb;
  const int n = last - first;
  if (n > 0) fetch(ha);
  w4_stage<XT, SUB, MT, W4S_NT>(a, nblk, rp, smem, sums);
  for (int i = 0; i < n; i += 2) {
    if (i + 1 < n) fetch(hb);
    compute(ha);
    if (i + 1 >= n) break;
    if (i + 2 < n) fetch(ha);
    compute(hb);
  }

  // What is left in tot: a tile that the next wavefronts go on with, begun
  // here, or all of this share is inside a tile.
  if (n > 0 && step > 0 && !begun) {
#pragma unroll
    for (int m = 0; m < MT; ++m) head[m] = tot[m];
  }
  f32x4* part = reinterpret_cast<f32x4*>(smem);   // [wave][MT][lane], over the staged rows
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; ++m) part[(wave * MT + m) * 64 + lane] = head[m];
  __syncthreads();
  if (n > 0 && step > 0 && begun) {
    const long long end = (long long)(tile - t0 + 1) * steps;
    for (int w = wave + 1; w < W4S_WAVES && all * w / W4S_WAVES < end; ++w)
#pragma unroll
      for (int m = 0; m < MT; ++m) tot[m] += part[(w * MT + m) * 64 + lane];
    w4_store<MT>(a, tile * 16, tot);
  }
}

// ---------------------------------------------------------------------------
// More rows than that: two launches.  The first puts the rows of x into the
// order of the products' operands in a workspace (small: it stays in the L2);
// the second is tiled over rows and columns.
//
// Here a vector operation for each result and group would cost more than it
// may, so the zero points are taken out by products of their own, in float32,
// one for two entries (an entry: 128 k, or a group where that is less): tot -=
// sum s * z * X.  So no sum holds more than two entries' zero points: an error of
// 1e-7 to 5e-7 of the results' norm at K = 4096 and 8192, in either type, with
// states of mean 0 or half of their spread, where torch's float32 product has
// 2e-7 to 1.5e-6.  (With the zero points of all of K taken out at the start, in bf16
// parts, 1e-6 to 1e-5.)
//
// R=320, K=4096, N=128256, groups of 128 with zeros: 381-388 us, 870 TFLOP/s, where
// the library's bf16 product of the same shape, with 4 times the weight bytes,
// takes 470 us (715) and its best on 8192^3 is 1198.  On the way: 16x16x32
// products with a shift of each group, 942 us; with zero points by products,
// 566; the checks out of the loop, 433; 32x32x16 products, two column tiles a
// wavefront, 390; one column tile, which two workgroups of a CU then share, 380.
// Scales and zero points fetched for each block by itself: 443 (a lane's lie in
// a cache line of their own, so a fetch of one byte takes as long as one of 16).
// Chunks of two blocks, two blocks ahead and workgroups of four wavefronts were
// slower.  Groups of 64: 410 us, of 32: 518 (16 scalings for 4 products).  R=64:
// 98 us; R=32, N=128255: 69-75 us (3.8-4.1 TB/s, of which the first launch is 5 us).
// Counters at R=320: the matrix cores are busy 46% of the SIMDs' time, the vector
// units 41% (with groups of 32, 45% and 59%), the LDS 27%, at 2.0 GHz where R=64
// runs at 2.5: what bounds it is the SIMDs' instructions, expanding and scaling
// among them, and the clock that this load leaves.
// ---------------------------------------------------------------------------

// Blocks of 128 k in the workspace: an even number.
__host__ __device__ __forceinline__ int w4_blocks(int K) { return (K + 255) / 256 * 2; }

// The products here are v_mfma_f32_32x32x16_bf16 (lane l holds row / column
// l % 32 of either operand at k = 8 * (l / 32) + 0..7, and rows 8 * (r / 4) +
// 4 * (l / 32) + r % 4 of column l % 32 of the result): with two wavefronts on
// a SIMD and two vector operations for each 16 x 16 x 32 of product between
// them, they were measured at 2170 TFLOP/s over the chip, 16x16x32 at 1260.
//
// A block of 128 k is eight products t.  A lane's two 16-byte loads of a weight
// row hold 32 consecutive k each, at 64 j + 32 h (h = l / 32); word i of load j
// is product t = 4 j + i, at k = 64 j + 32 h + 8 i.  With groups of 32 the
// halves of the wavefront exchange words, so that a product stays in one group:
// t = 4 j + 2 g + q at k = 64 j + 32 g + 16 q + 8 h.

template <int SUB>
__device__ __forceinline__ void w4_place(int u, int& t, int& h) {   // of the block's k = 8 u
  if (SUB == 4) {
    t = (u >> 3) * 4 + ((u >> 2) & 1) * 2 + ((u >> 1) & 1);
    h = u & 1;
  } else {
    t = (u >> 3) * 4 + (u & 3);
    h = (u >> 2) & 1;
  }
}

// One workgroup per 32 rows and 128 k.  xop: [row tile][block][t][part] of 1 KB
// ([h][row] 16 bytes), the rows' values; xsum: [row tile][block][SUB][row] float,
// their sums over each 128 / SUB of k.  Rows beyond R and k beyond K are zeros, so
// that the product needs no checks: what it reads of the weights there meets
// zeros.
template <typename XT, int SUB>
__global__ __launch_bounds__(512) void w4_order_kernel(W4Args a) {
  constexpr int P = W4Hidden<XT>::PARTS;
  __shared__ float part[16][33];
  const int nblk = w4_blocks(a.K);
  const int rt = (int)(blockIdx.x / (unsigned)nblk), b = (int)(blockIdx.x % (unsigned)nblk);
  const int r = threadIdx.x >> 4, u = threadIdx.x & 15;   // u: 8 of the block's 128 k
  const int row = rt * 32 + r, k = b * 128 + u * 8;
  int t, h;
  w4_place<SUB>(u, t, h);
  bf16x8 f[P];
  float sum = 0.0f;
  if (row < a.R && k < a.K) {
    const XT* x = reinterpret_cast<const XT*>(a.x) + (size_t)row * a.K + k;
    W4Hidden<XT>::load(x, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += load_in(x + e);
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p) f[p] = __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0});
  }
  char* o = a.xop + (((size_t)blockIdx.x * 8 + t) * P) * 1024 + (h * 32 + r) * 16;
#pragma unroll
  for (int p = 0; p < P; ++p) *reinterpret_cast<bf16x8*>(o + p * 1024) = f[p];
  part[u][r] = sum;
  __syncthreads();
  if (threadIdx.x < SUB * 32) {
    const int sg = threadIdx.x >> 5, rr = threadIdx.x & 31;
    float x = 0.0f;
#pragma unroll
    for (int e = 0; e < 16 / SUB; ++e) x += part[sg * (16 / SUB) + e][rr];
    reinterpret_cast<float*>(a.xsum)[(size_t)blockIdx.x * SUB * 32 + threadIdx.x] = x;
  }
}

template <int NL> struct W4Stage {
  u32x4 v[NL];
  float sum;
};

// What a wavefront fetches ahead of one column tile of 32: U blocks of 128 k.
template <int U> struct W4Wide { u32x4 w[U][2]; };

constexpr int W4_NT = 512;                 // threads per workgroup
constexpr int W4_WAVES = W4_NT / 64;

// MT * 32 rows by 32 columns a wavefront, eight wavefronts side by side.
// Operands of x come KC blocks at a time through two LDS buffers: the next
// chunk's are loaded into registers before this one is computed and written
// after it, one barrier a chunk.  Weights go from memory to registers, U
// blocks ahead.
template <typename XT, typename ST, int SUB, int MT, int U, int KC>
__global__ __launch_bounds__(W4_NT, W4Hidden<XT>::PARTS == 1 ? 4 : 2) void w4_tile_kernel(W4Args a) {
  constexpr int P = W4Hidden<XT>::PARTS;
  constexpr int ROW = KC * 8 * P * 1024, OPS = MT * ROW;   // bytes of a chunk: one row tile's, all
  constexpr int NL = OPS / 16 / W4_NT;                     // 16-byte loads a thread
  constexpr int CE = KC * SUB < 2 ? 2 : KC * SUB;          // entries of a chunk, or of it and its neighbour
  constexpr int SROW = CE * 32, SUMS = MT * SROW;          // their sums
  static_assert(OPS % (16 * W4_NT) == 0 && KC % U == 0 && SUMS <= W4_NT, "chunk does not fit the workgroup");
  typedef W4Wide<U> Wide;
  // A lane's row is a line of its own, so a fetch of a few bytes takes as long as one of 16: scales and zero points come
  // for several blocks at a time.
  constexpr int SE = U * SUB > 4 ? U * SUB : 4, ZE = SUB == 1 ? 4 : 8;
  __shared__ __align__(16) char xs[2][OPS];
  __shared__ float sums[2][W4_NT];                         // SUMS of them, and what the other threads load again
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, l32 = lane & 31, half = lane >> 5;
  const int nblk = w4_blocks(a.K);
  const long long sets = (long long)((a.N + W4_WAVES * 32 - 1) / (W4_WAVES * 32)) * a.row_tiles;
  // The row tiles of a column tile run on one XCD, one after the other.
  const long long set = (long long)(blockIdx.x & 7) * a.per_xcd + (blockIdx.x >> 3);
  if (set >= sets) return;
  const int rt = (int)(set % a.row_tiles);
  const int n0 = ((int)(set / a.row_tiles) * W4_WAVES + __builtin_amdgcn_readfirstlane(wave)) * 32;
  const uint32_t len = (uint32_t)nblk * 8 * P * 1024;      // operands of a row tile
  const uint32_t slen = (uint32_t)nblk * SUB * 32;         // sums of a row tile
  const char* xop = a.xop + (size_t)rt * MT * len;
  const float* xsum = reinterpret_cast<const float*>(a.xsum) + (size_t)rt * MT * slen + (tid % SUMS / SROW * slen + tid % SROW);
  const W4Rows rows = w4_rows(a, n0, l32);

  W4Stage<NL> sr;
  // Chunk c's operands, ROW bytes of each row tile (behind the last chunk, the first again).
  auto stage_load = [&](W4Stage<NL>& g, int c) __attribute__((always_inline)) {
    const bool more = (uint32_t)c * ROW < len;
    const uint32_t at = more ? (uint32_t)c * ROW : 0u;
    g.sum = xsum[more ? (uint32_t)(c * KC * SUB & ~1) * 32 : 0u];
#pragma unroll
    for (int q = 0; q < NL; ++q) {
      const int o = (q * W4_NT + tid) * 16, m = o / ROW;
      g.v[q] = *reinterpret_cast<const u32x4*>(xop + at + ((uint32_t)m * len + o % ROW));
    }
  };
  auto stage_write = [&](const W4Stage<NL>& g, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NL; ++q) *reinterpret_cast<u32x4*>(xs[buf] + (q * W4_NT + tid) * 16) = g.v[q];
    sums[buf][tid] = g.sum;
  };
  auto fetch = [&](Wide& g, int b) __attribute__((always_inline)) {
    const uint8_t* w = a.w + rows.first * (size_t)(a.K / 2);
    const uint32_t row = rows.local * (uint32_t)(a.K / 2);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        g.w[u][j] = *reinterpret_cast<const u32x4*>(w + (row + (uint32_t)min((b + u) * 64 + j * 32 + half * 16, a.K / 2 - 16)));
  };

  // The scales and zero points in use, and the next ones, which are fetched a step after those were taken.
  struct Some { uint32_t s[SE * sizeof(ST) / 4], z[ZE / 4]; } now, next;
  auto fetch_scales = [&](int j) __attribute__((always_inline)) {
    if (a.gb == 1 && j + SE <= a.G) w4_fetch_scales<ST, SE, true>(a, next.s, rows, j);
    else w4_fetch_scales<ST, SE, false>(a, next.s, rows, j);
  };
  auto fetch_zeros = [&](int j) __attribute__((always_inline)) {
    if (a.gb == 1 && j + ZE <= a.G) w4_fetch_zeros<ZE, true>(a, next.z, rows, j);
    else w4_fetch_zeros<ZE, false>(a, next.z, rows, j);
  };
#pragma unroll
  for (int i = 0; i < ZE / 4; ++i) next.z[i] = 0;

  Wide ha, hb;
  fetch_scales(0);
  fetch_zeros(0);
  fetch(ha, 0);
  stage_load(sr, 0);

  f32x16 tot[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 16; ++r) tot[m][r] = 0.0f;

  // Block u of step q of the loop, times its rows of x (this lane's in x), onto tot.
  auto block = [&](const Wide& g, int q, int u, const char* x) __attribute__((always_inline)) {
    constexpr int TG = 8 / SUB;   // products of a group
#pragma unroll
    for (int sg = 0; sg < SUB; ++sg) {
      f32x16 blk[MT];
#pragma unroll
      for (int i = 0; i < TG; ++i) {
        const int t = sg * TG + i, j = t >> 2;
        uint32_t d;
        if constexpr (SUB == 4) {
          const auto pair = __builtin_amdgcn_permlane32_swap(g.w[u][j][2 * i], g.w[u][j][2 * i + 1], false, false);
          d = pair[sg & 1];
        } else {
          d = g.w[u][j][t & 3];
        }
        const bf16x8 wv = w4_expand(d);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int p = P - 1; p >= 0; --p) {
            const bf16x8 f = *reinterpret_cast<const bf16x8*>(x + m * ROW + (t * P + p) * 1024);
            if (i == 0 && p == P - 1) {
              f32x16 zero;
#pragma unroll
              for (int r = 0; r < 16; ++r) zero[r] = 0.0f;
              blk[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, wv, zero, 0, 0, 0);
            } else {
              blk[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, wv, blk[m], 0, 0, 0);
            }
          }
        }
      }
      const float scale = w4_get(now.s, (q * U + u) * SUB % SE + sg, (const ST*)nullptr);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int r = 0; r < 16; ++r) tot[m][r] = __builtin_fmaf(scale, blk[m][r], tot[m][r]);
        // Here and not in the next step, where the compiler would take them: blk's registers (164 instead of 128 with
        // groups of 128) would cost the CU its second workgroup.
        if (P == 1) asm volatile("" : "+v"(tot[m]));
      }
    }
  };

  // - sum s * z * X over a pair of entries (the ones at e), one to a half of the lanes, onto tot.  In float32: of a
  // product's 8 consecutive k, v_mfma_f32_32x32x16_bf16 cuts off what lies below the last bit of the largest, so that
  // X and s * z as bf16 parts side by side lost up to three such bits, always downwards.
  const uint32_t z_and = a.z ? 15u : 0u, z_or = a.z ? 0u : 8u;
  auto zero_points = [&](int e, const float* x) __attribute__((always_inline)) {
    const float lo = w4_get(now.s, e % SE, (const ST*)nullptr), hi = w4_get(now.s, e % SE + 1, (const ST*)nullptr);
    const uint32_t z = now.z[e % ZE >> 2] >> (8 * (e & 3) + 8 * half);
    const float t = (half ? hi : lo) * -(float)((z & z_and) | z_or);
#pragma unroll
    for (int m = 0; m < MT; ++m) tot[m] = __builtin_amdgcn_mfma_f32_32x32x2f32(x[m * SROW], t, tot[m], 0, 0, 0);
  };

  stage_write(sr, 0);
  __syncthreads();
  const int nsteps = nblk / U;
  // One step, q its place in the loop below.
  auto step = [&](const Wide& cur, Wide& nxt, int s, int q) __attribute__((always_inline)) {
    constexpr int NS = U * SUB;   // entries of a step
    const int b = s * U, c = b / KC;
    if (b % KC == 0) stage_load(sr, c + 1);
    if (q * NS % SE == 0) __builtin_memcpy(now.s, next.s, sizeof now.s);
    if (q * NS % ZE == 0) __builtin_memcpy(now.z, next.z, sizeof now.z);
    if (q * NS % ZE == NS % ZE) fetch_zeros(b * SUB - NS % ZE + ZE);
    if (q * NS % SE == NS % SE) fetch_scales(b * SUB - NS % SE + SE);
    fetch(nxt, min(b + U, nblk - U));
#pragma unroll
    for (int u = 0; u < U; ++u) block(cur, q, u, xs[c & 1] + (b % KC + u) * 8 * P * 1024 + lane * 16);
    if (NS >= 2) {
#pragma unroll
      for (int e = 0; e < NS; e += 2) zero_points(q * NS + e, sums[c & 1] + (b % KC * SUB + e) * 32 + lane);
    } else if (q % 2) {           // one entry a step: the pair of this step and the last
      zero_points(q - 1, sums[c & 1] + lane);
    }
    if ((b + U) % KC == 0) {
      stage_write(sr, (c + 1) & 1);
      __syncthreads();
    }
  };
  // Four steps or two, so that the scales and zero points of a step lie in the same place each time (Four where two
  // do: 18.5 us instead of 18.0 at R=40, K=512, N=3001, fp32 states, groups of 32.)
  for (int s = 0;;) {
    step(ha, hb, s, 0);
    if (U == 2 && s + 1 == nsteps) break;
    step(hb, ha, s + 1, 1);
    if ((s += 2) >= nsteps) break;
    if (U == 2 || SUB == 4) continue;
    step(ha, hb, s, 2);
    step(hb, ha, s + 1, 3);
    if ((s += 2) >= nsteps) break;
  }

  const int n = n0 + l32;
  if (n >= a.N) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = (rt * MT + m) * 32 + (r >> 2) * 8 + half * 4 + (r & 3);
      if (row >= a.R) continue;
      const size_t o = (size_t)row * a.N + n;
      if (a.out_bf16) store_out(reinterpret_cast<uint16_t*>(a.out) + o, tot[m][r]);
      else store_out(reinterpret_cast<float*>(a.out) + o, tot[m][r]);
    }
  }
}

}  // namespace sl
