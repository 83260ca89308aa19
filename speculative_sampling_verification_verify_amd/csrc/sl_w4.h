// Logits from a head of 4-bit weights with group scales:
//
//   out[r][n] = sum_g s[n][g] * sum_{k in g} (w[n][k] - z[n][g]) * x[r][k].
//
// The inner sums run on the matrix cores in bf16 with float32 accumulators,
// and nothing in them is rounded but the accumulators: a weight enters as the
// bf16 number 16 + w (16..31, exact: 0x4180 + 8 w, one shift and one and-or
// for two weights), and the 16 + z that is too much is taken out per group as
// (16 + z) * X_g with X_g = sum of the group's x, itself a product with ones.
// The scale multiplies the group's float32 sum.  fp32 hidden states are split
// into three bf16 parts (8 + 8 + 8 significand bits, truncated, so the parts
// add up to the value exactly) that take three products.
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

// The eight weights of a word as bf16 numbers 16 + w, in the order 0 4 1 5 2 6 3 7.
// The constants are kept in registers (one operand of an instruction may be a
// constant), so that a pair takes a shift and a v_and_or_b32.
__device__ __forceinline__ bf16x8 w4_expand(uint32_t w) {
  uint32_t mask = 0x00780078u, base = 0x41804180u;
  asm("" : "+s"(mask));
  asm("" : "+v"(base));
  u32x4 v;
  v.x = ((w << 3) & mask) | base;
  v.y = ((w >> 1) & mask) | base;
  v.z = ((w >> 5) & mask) | base;
  v.w = ((w >> 9) & mask) | base;
  return __builtin_bit_cast(bf16x8, v);
}

// Eight consecutive bf16 values in the same order.
__device__ __forceinline__ bf16x8 w4_order(uint4 a) {
  uint4 v;
  v.x = __builtin_amdgcn_perm(a.z, a.x, 0x05040100u);
  v.y = __builtin_amdgcn_perm(a.z, a.x, 0x07060302u);
  v.z = __builtin_amdgcn_perm(a.w, a.y, 0x05040100u);
  v.w = __builtin_amdgcn_perm(a.w, a.y, 0x07060302u);
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
  // The upper halves of eight words in the order 0 4 1 5 2 6 3 7.
  __device__ __forceinline__ static bf16x8 pack(const uint32_t (&u)[8]) {
    uint4 v;
    v.x = __builtin_amdgcn_perm(u[4], u[0], 0x07060302u);
    v.y = __builtin_amdgcn_perm(u[5], u[1], 0x07060302u);
    v.z = __builtin_amdgcn_perm(u[6], u[2], 0x07060302u);
    v.w = __builtin_amdgcn_perm(u[7], u[3], 0x07060302u);
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

// 16 + z of entry i.
__device__ __forceinline__ float w4_shift(const W4Args& a, const uint32_t* z, int i) {
  return 16.0f + (float)(a.z ? (z[i >> 2] >> (8 * (i & 3))) & 15u : 8u);
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

// COUNT scales and, with ZEROS, zeros of the lane's row from entry j on.
// TOGETHER: they lie side by side inside the row; else one by one, and entries
// behind the row's end repeat its last.
template <typename ST, int COUNT, bool ZEROS, bool TOGETHER, int SW, int ZW>
__device__ __forceinline__ void w4_fetch_scales(const W4Args& a, uint32_t (&sw)[SW], uint32_t (&zw)[ZW], const W4Rows& r,
                                                int j) {
  const ST* s = reinterpret_cast<const ST*>(a.s) + r.first * a.G;
  const uint8_t* z = a.z + r.first * a.G;
  const uint32_t row = r.local * (uint32_t)a.G;
  if (TOGETHER) {
    __builtin_memcpy(sw, s + (row + (uint32_t)j), COUNT * sizeof(ST));
    if (ZEROS && a.z) __builtin_memcpy(zw, z + (row + (uint32_t)j), COUNT);
  } else {
#pragma unroll
    for (int i = 0; i < SW; ++i) sw[i] = 0;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) w4_put(sw, i, s[row + w4_group(a, j + i)]);
    if (ZEROS && a.z) {
#pragma unroll
      for (int i = 0; i < ZW; ++i) zw[i] = 0;
#pragma unroll
      for (int i = 0; i < COUNT; ++i) zw[i >> 2] |= (uint32_t)z[row + w4_group(a, j + i)] << (8 * (i & 3));
    }
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
  if (a.gb == 1 && (b + U) * SUB <= a.G) w4_fetch_scales<ST, NS, true, true>(a, h.s, h.z, r, b * SUB);
  else w4_fetch_scales<ST, NS, true, false>(a, h.s, h.z, r, b * SUB);
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
    const float sc = w4_get(h.s, u * SUB + sg, (const ST*)nullptr), zz = w4_shift(a, h.z, u * SUB + sg);
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
// Here the 16 + z that a weight is too much costs more than it may: an
// operation for each result and group.  So it is taken out by a product of its
// own, tot = - sum_j t[n][j] * X[r][j] over the groups j, t = s * (16 + z): both
// sides float32, split into three bf16 parts each, of whose products the six
// above 2^-24 are formed -- 6 products for 16 groups, which have 32 to 128 of
// their own.
//
// R=320, K=4096, N=128256, groups of 128 with zeros: 380-389 us, 870 TFLOP/s, where
// the library's bf16 product of the same shape, with 4 times the weight bytes,
// takes 470 us (715) and its best on 8192^3 is 1198.  On the way: 16x16x32
// products with a shift of each group, 942 us; with the product above, 566; the
// checks out of the loop and the weights' pairs by two operations, 433; 32x32x16
// products, two column tiles a wavefront, 390; one column tile, which two
// workgroups of a CU then share, 380 (at N=32000 153 -> 117).  Leaving out, one
// at a time, the fetch of the weights, the LDS reads, the expansion or the
// scaling changed the 390 by less than 6%, and half as many workgroups on half
// the CUs took half the time: what bounds it is shared by the CUs.  Chunks of
// two blocks (403 us), two blocks ahead (451) and workgroups of four wavefronts
// (413) were slower.  Groups of 32: 573 us (16 scalings for 4 products).  R=64:
// 107 us, R=32: 83 us (3.4 TB/s, of which the first launch is 5 us): there a
// chunk's barrier and its wait for the weights.
// ---------------------------------------------------------------------------

// Blocks of 128 k in the workspace: an even number.
__host__ __device__ __forceinline__ int w4_blocks(int K) { return (K + 255) / 256 * 2; }

__device__ __forceinline__ void w4_split(float v, uint32_t (&o)[3]) {
  o[0] = __float_as_uint(v) & 0xFFFF0000u;
  const float r = v - __uint_as_float(o[0]);
  o[1] = __float_as_uint(r) & 0xFFFF0000u;
  o[2] = __float_as_uint(r - __uint_as_float(o[1])) & 0xFFFF0000u;
}

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
// ([h][row] 16 bytes), the rows' values; xsum: [row tile][16 entries][part] of
// 1 KB ([h][row] 8 entries), their sums over each 128 / SUB of k.  Rows beyond
// R, k beyond K and entries beyond the last are zeros, so that the product
// needs no checks: what it reads of the weights there meets zeros.
template <typename XT, int SUB>
__global__ __launch_bounds__(512) void w4_order_kernel(W4Args a) {
  constexpr int P = W4Hidden<XT>::PARTS;
  __shared__ float part[16][33];
  const int nblk = w4_blocks(a.K), n16 = (nblk * SUB + 15) / 16;
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
  // The block's entries, and behind the last block those up to the next 16.
  const int j1 = b + 1 == nblk ? n16 * 16 : (b + 1) * SUB;
  for (int q = threadIdx.x; q < (j1 - b * SUB) * 32; q += 512) {
    const int sg = q >> 5, rr = q & 31, j = b * SUB + sg;
    float t = 0.0f;
    if (sg < SUB) {
#pragma unroll
      for (int e = 0; e < 16 / SUB; ++e) t += part[sg * (16 / SUB) + e][rr];
    }
    uint32_t v[3];
    w4_split(t, v);
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<uint16_t*>(a.xsum + (((size_t)rt * n16 + (j >> 4)) * 3 + p) * 1024 + (((j >> 3) & 1) * 32 + rr) * 16 +
                                   (j & 7) * 2) = (uint16_t)(v[p] >> 16);
  }
}

template <int NL> struct W4Stage { u32x4 v[NL]; };

// What a wavefront fetches ahead of one column tile of 32: U blocks of 128 k.
template <typename ST, int SUB, int U>
struct W4Wide {
  static constexpr int NS = U * SUB;
  static constexpr int SW = (NS * (int)sizeof(ST) + 3) / 4;
  u32x4 w[U][2];
  uint32_t s[SW];
};

constexpr int W4_NT = 512;                 // threads per workgroup
constexpr int W4_WAVES = W4_NT / 64;

// MT * 32 rows by 32 columns a wavefront, eight wavefronts side by side.
// Operands of x come KC blocks at a time through two LDS buffers: the next
// chunk's are loaded into registers before this one is computed and written
// after it, one barrier a chunk.  Weights go from memory to registers, U
// blocks ahead.
template <typename XT, typename ST, int SUB, int MT, int U, int KC>
__global__ __launch_bounds__(W4_NT) __attribute__((amdgpu_waves_per_eu(2))) void w4_tile_kernel(W4Args a) {
  constexpr int P = W4Hidden<XT>::PARTS;
  constexpr int NT = 1;   // column tiles of 32 a wavefront; two take twice the registers, half the wavefronts
  constexpr int ROW = KC * 8 * P * 1024, OPS = MT * ROW;   // bytes of a chunk: one row tile's, all
  constexpr int NL = OPS / 16 / W4_NT;                     // 16-byte loads a thread
  static_assert(OPS % (16 * W4_NT) == 0 && KC % U == 0, "chunk does not fit the workgroup");
  typedef W4Wide<ST, SUB, U> Wide;
  __shared__ __align__(16) char xs[2][OPS];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, l32 = lane & 31, half = lane >> 5;
  const int nblk = w4_blocks(a.K);
  const long long sets = (long long)((a.N + W4_WAVES * NT * 32 - 1) / (W4_WAVES * NT * 32)) * a.row_tiles;
  // The row tiles of a column tile run on one XCD, one after the other.
  const long long set = (long long)(blockIdx.x & 7) * a.per_xcd + (blockIdx.x >> 3);
  if (set >= sets) return;
  const int rt = (int)(set % a.row_tiles);
  const int n0 = ((int)(set / a.row_tiles) * W4_WAVES + __builtin_amdgcn_readfirstlane(wave)) * NT * 32;
  const uint32_t len = (uint32_t)nblk * 8 * P * 1024;      // operands of a row tile
  const char* xop = a.xop + (size_t)rt * MT * len;
  W4Rows rows[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) rows[nt] = w4_rows(a, n0 + nt * 32, l32);

  W4Stage<NL> sr;
  // Chunk c's operands, ROW bytes of each row tile (behind the last chunk, the first again).
  auto stage_load = [&](W4Stage<NL>& g, int c) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NL; ++q) {
      const int o = (q * W4_NT + tid) * 16, m = o / ROW;
      const uint32_t at = (uint32_t)c * ROW < len ? (uint32_t)c * ROW : 0u;
      g.v[q] = *reinterpret_cast<const u32x4*>(xop + at + ((uint32_t)m * len + o % ROW));
    }
  };
  auto stage_write = [&](const W4Stage<NL>& g, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NL; ++q) *reinterpret_cast<u32x4*>(xs[buf] + (q * W4_NT + tid) * 16) = g.v[q];
  };
  auto fetch = [&](Wide (&g)[NT], int b) __attribute__((always_inline)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint8_t* w = a.w + rows[nt].first * (size_t)(a.K / 2);
      const uint32_t row = rows[nt].local * (uint32_t)(a.K / 2);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          g[nt].w[u][j] =
              *reinterpret_cast<const u32x4*>(w + (row + (uint32_t)min((b + u) * 64 + j * 32 + half * 16, a.K / 2 - 16)));
    }
    if (Wide::NS <= 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t none[1];
        w4_fetch_scales<ST, Wide::NS, false, false>(a, g[nt].s, none, rows[nt], b * SUB);
      }
    } else if (a.gb == 1 && (b + U) * SUB <= a.G) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t none[1];
        w4_fetch_scales<ST, Wide::NS, false, true>(a, g[nt].s, none, rows[nt], b * SUB);
      }
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t none[1];
        w4_fetch_scales<ST, Wide::NS, false, false>(a, g[nt].s, none, rows[nt], b * SUB);
      }
    }
  };

  Wide ha[NT], hb[NT];
  fetch(ha, 0);
  stage_load(sr, 0);

  // tot = - sum_j s * (16 + z) * X.
  f32x16 tot[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 16; ++r) tot[m][nt][r] = 0.0f;
  const int n16 = (nblk * SUB + 15) / 16;
  for (int j = 0; j < n16; ++j) {
    // The lane's eight entries of each column; behind the last they meet zeros.
    uint32_t sw[NT][8 * sizeof(ST) / 4], zw[NT][2];
    if (a.gb == 1 && (j + 1) * 16 <= a.G) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) w4_fetch_scales<ST, 8, true, true>(a, sw[nt], zw[nt], rows[nt], j * 16 + half * 8);
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) w4_fetch_scales<ST, 8, true, false>(a, sw[nt], zw[nt], rows[nt], j * 16 + half * 8);
    }
    bf16x8 t[NT][3];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t w[3][4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t v[3];
        w4_split(-w4_get(sw[nt], e, (const ST*)nullptr) * w4_shift(a, zw[nt], e), v);
#pragma unroll
        for (int p = 0; p < 3; ++p) w[p][e >> 1] = e & 1 ? w[p][e >> 1] | v[p] : v[p] >> 16;
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) t[nt][p] = __builtin_bit_cast(bf16x8, u32x4{w[p][0], w[p][1], w[p][2], w[p][3]});
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const char* xp = a.xsum + (((size_t)(rt * MT + m) * n16 + j) * 3) * 1024 + lane * 16;
      bf16x8 x[3];
#pragma unroll
      for (int p = 0; p < 3; ++p) x[p] = *reinterpret_cast<const bf16x8*>(xp + p * 1024);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f32x16 v = tot[m][nt];
        v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[0], t[nt][2], v, 0, 0, 0);
        v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[2], t[nt][0], v, 0, 0, 0);
        v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[1], t[nt][1], v, 0, 0, 0);
        v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[0], t[nt][1], v, 0, 0, 0);
        v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[1], t[nt][0], v, 0, 0, 0);
        v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[0], t[nt][0], v, 0, 0, 0);
        tot[m][nt] = v;
      }
    }
  }

  // Block u of what was fetched, times its rows of x (this lane's in x), onto tot.
  auto block = [&](const Wide (&g)[NT], int u, const char* x) __attribute__((always_inline)) {
    constexpr int TG = 8 / SUB;   // products of a group
#pragma unroll
    for (int sg = 0; sg < SUB; ++sg) {
      f32x16 blk[MT][NT];
#pragma unroll
      for (int q = 0; q < TG; ++q) {
        const int t = sg * TG + q, j = t >> 2;
        bf16x8 wv[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t d;
          if constexpr (SUB == 4) {
            const auto pair = __builtin_amdgcn_permlane32_swap(g[nt].w[u][j][2 * q], g[nt].w[u][j][2 * q + 1], false, false);
            d = pair[sg & 1];
          } else {
            d = g[nt].w[u][j][t & 3];
          }
          wv[nt] = w4_expand(d);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int p = P - 1; p >= 0; --p) {
            const bf16x8 f = *reinterpret_cast<const bf16x8*>(x + m * ROW + (t * P + p) * 1024);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (q == 0 && p == P - 1) {
                f32x16 zero;
#pragma unroll
                for (int r = 0; r < 16; ++r) zero[r] = 0.0f;
                blk[m][nt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, wv[nt], zero, 0, 0, 0);
              } else {
                blk[m][nt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, wv[nt], blk[m][nt], 0, 0, 0);
              }
            }
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float sc = w4_get(g[nt].s, u * SUB + sg, (const ST*)nullptr);
#pragma unroll
          for (int r = 0; r < 16; ++r) tot[m][nt][r] = __builtin_fmaf(sc, blk[m][nt][r], tot[m][nt][r]);
        }
    }
  };

  stage_write(sr, 0);
  __syncthreads();
  const int nsteps = nblk / U;
  auto step = [&](const Wide (&cur)[NT], Wide (&nxt)[NT], int s) __attribute__((always_inline)) {
    const int b = s * U, c = b / KC;
    fetch(nxt, min(b + U, nblk - U));
    if (b % KC == 0) stage_load(sr, c + 1);
#pragma unroll
    for (int u = 0; u < U; ++u) block(cur, u, xs[c & 1] + (b % KC + u) * 8 * P * 1024 + lane * 16);
    if ((b + U) % KC == 0) {
      stage_write(sr, (c + 1) & 1);
      __syncthreads();
    }
  };
  for (int s = 0;;) {
    step(ha, hb, s);
    if (U == 2 && s + 1 == nsteps) break;
    step(hb, ha, s + 1);
    if ((s += 2) >= nsteps) break;
  }

#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int n = n0 + nt * 32 + l32;
    if (n >= a.N) continue;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = (rt * MT + m) * 32 + (r >> 2) * 8 + half * 4 + (r & 3);
        if (row >= a.R) continue;
        const size_t o = (size_t)row * a.N + n;
        if (a.out_bf16) store_out(reinterpret_cast<uint16_t*>(a.out) + o, tot[m][nt][r]);
        else store_out(reinterpret_cast<float*>(a.out) + o, tot[m][nt][r]);
      }
    }
  }
}

}  // namespace sl
