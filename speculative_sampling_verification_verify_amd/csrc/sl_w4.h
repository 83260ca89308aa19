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
// v_mfma_f32_16x16x32_bf16: lane l holds row / column l % 16 of either operand
// at k = 8 * (l / 16) + 0..7, and rows 4 * (l / 16) + 0..3 of column l % 16 of
// the result.  Rows are rows of x, columns are rows of the weight matrix: a
// lane's results share one weight row, hence one scale.
#pragma once

#include "sl_common.h"

namespace sl {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct W4Args {
  const void* x;
  const uint8_t* w;
  const void* s;
  const uint8_t* z;   // or null
  void* out;
  int R, K, N;
  int G;              // groups per weight row
  int gb;             // 128-k blocks per group (1 where the group is 32 or 64)
  int row_tiles;      // tiles of MT * 16 rows
  int rp;             // rows staged of a tile (a power of two, 16 unless R is smaller)
  int kc;             // blocks of 128 k staged at a time
  int KS;             // wavefronts that share a column tile
  int per_xcd;        // workgroups of one XCD
  int out_bf16;
};

// The eight weights of a word as bf16 numbers 16 + w, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 w4_expand(uint32_t w) {
  uint4 v;
  v.x = ((w << 3) & 0x00780078u) | 0x41804180u;
  v.y = ((w >> 1) & 0x00780078u) | 0x41804180u;
  v.z = ((w >> 5) & 0x00780078u) | 0x41804180u;
  v.w = ((w >> 9) & 0x00780078u) | 0x41804180u;
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
  uint4 w[U];
  uint32_t s[SW], z[ZW];
};

__device__ __forceinline__ float w4_get(const uint32_t* w, int i, const uint16_t*) {
  return __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
}
__device__ __forceinline__ float w4_get(const uint32_t* w, int i, const float*) { return __uint_as_float(w[i]); }
__device__ __forceinline__ void w4_put(uint32_t* w, int i, uint16_t v) { w[i >> 1] |= (uint32_t)v << (16 * (i & 1)); }
__device__ __forceinline__ void w4_put(uint32_t* w, int i, float v) { w[i] = __float_as_uint(v); }

// Blocks b .. b + U - 1 of weight row `row` (those before block `end`; the
// others, and what lies beyond K, come as zeros).
template <typename ST, int SUB, int U>
__device__ __forceinline__ void w4_fetch(const W4Args& a, W4Ahead<ST, SUB, U>& h, int row, int quad, int b, int end) {
  typedef W4Ahead<ST, SUB, U> Ahead;
  const uint8_t* w = a.w + (size_t)row * (a.K / 2) + b * 64 + quad * 16;
  const size_t srow = (size_t)row * a.G;
  const ST* s = reinterpret_cast<const ST*>(a.s) + srow;
  const bool whole = b + U <= end && (b + U) * 128 <= a.K;
  if (whole) {
#pragma unroll
    for (int u = 0; u < U; ++u) h.w[u] = *reinterpret_cast<const uint4*>(w + u * 64);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = b + u < end && (b + u) * 128 + quad * 32 < a.K;
      h.w[u] = in ? *reinterpret_cast<const uint4*>(w + u * 64) : make_uint4(0, 0, 0, 0);
    }
  }
  if (whole && a.gb == 1) {
    __builtin_memcpy(h.s, s + b * SUB, Ahead::NS * sizeof(ST));
    if (a.z) __builtin_memcpy(h.z, a.z + srow + b * SUB, Ahead::NS);
  } else {
#pragma unroll
    for (int i = 0; i < Ahead::SW; ++i) h.s[i] = 0;
#pragma unroll
    for (int i = 0; i < Ahead::ZW; ++i) h.z[i] = 0;
#pragma unroll
    for (int i = 0; i < Ahead::NS; ++i) {
      const int g = min(a.gb == 1 ? b * SUB + i : (b + i) / a.gb, a.G - 1);
      w4_put(h.s, i, s[g]);
      if (a.z) h.z[i >> 2] |= (uint32_t)a.z[srow + g] << (8 * (i & 3));
    }
  }
}

// Block u of what was fetched, times the staged rows of block lb, onto tot.
template <typename XT, typename ST, int SUB, int MT, int NT, int U>
__device__ __forceinline__ void w4_block(const W4Args& a, const W4Ahead<ST, SUB, U> (&h)[NT], int u, int lb, const char* xs,
                                         const float* sums, int frag, int loff, int quad, f32x4 (&tot)[MT][NT]) {
  constexpr int P = W4Hidden<XT>::PARTS;
  uint32_t d[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    d[nt][0] = h[nt].w[u].x;
    d[nt][1] = h[nt].w[u].y;
    d[nt][2] = h[nt].w[u].z;
    d[nt][3] = h[nt].w[u].w;
    if (SUB > 1) w4_transpose(d[nt]);
  }
  f32x4 blk[MT][NT];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool begin = SUB == 4 || (SUB == 2 && !(i & 1)) || i == 0;
    const bool end = SUB == 4 || (SUB == 2 && (i & 1)) || i == 3;
    bf16x8 wv[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) wv[nt] = w4_expand(d[nt][i]);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int p = P - 1; p >= 0; --p) {
        const bf16x8 f = *reinterpret_cast<const bf16x8*>(xs + (((lb * 4 + i) * P + p) * MT + m) * frag + loff);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          blk[m][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              f, wv[nt], begin && p == P - 1 ? f32x4{0, 0, 0, 0} : blk[m][nt], 0, 0, 0);
      }
    }
    if (end) {
      const int sg = SUB == 4 ? i : SUB == 2 ? i >> 1 : 0, e = u * SUB + sg;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float sc = w4_get(h[nt].s, e, (const ST*)nullptr);
        const float zz = 16.0f + (float)(a.z ? (h[nt].z[e >> 2] >> (8 * (e & 3))) & 15u : 8u);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const f32x4 x4 = *reinterpret_cast<const f32x4*>(sums + ((lb * SUB + sg) * MT + m) * 16 + quad * 4);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            tot[m][nt][r] = __builtin_fmaf(sc, __builtin_fmaf(-zz, x4[r], blk[m][nt][r]), tot[m][nt][r]);
        }
      }
    }
  }
}

// Rows rt * MT * 16 .. of x, blocks b0 .. b1 - 1, into LDS as the products'
// operands: [block][i][part][MT][quad][rp] 16 bytes, and their sums per group
// (products with ones): [block][SUB][MT][16].  The caller has synchronised;
// the rows are ready when this returns.
template <typename XT, int SUB, int MT, int NTHR>
__device__ __forceinline__ void w4_stage(const W4Args& a, int rt, int b0, int b1, int rp, char* xs, float* sums) {
  constexpr int P = W4Hidden<XT>::PARTS;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, l16 = lane & 15, quad = lane >> 4;
  const int frag = 64 * rp, loff = (quad * rp + min(l16, rp - 1)) * 16;
  const bf16x8 ones = __builtin_bit_cast(bf16x8, make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u));
  const XT* x = reinterpret_cast<const XT*>(a.x);
  const int units = (b1 - b0) * 4 * MT * 4 * rp;
  for (int q = tid; q < units; q += NTHR) {
    const int r = q & (rp - 1), rest0 = q / rp, qd = rest0 & 3, rest = rest0 >> 2;
    const int m = rest % MT, i = rest / MT & 3, lb = rest / MT >> 2;
    const int k = (b0 + lb) * 128 + (SUB > 1 ? i * 32 + qd * 8 : qd * 32 + i * 8);
    const int row = min((rt * MT + m) * 16 + r, a.R - 1);
    bf16x8 f[P];
    if (k < a.K) {
      W4Hidden<XT>::load(x + (size_t)row * a.K + k, f);
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) f[p] = __builtin_bit_cast(bf16x8, make_uint4(0, 0, 0, 0));
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
      *reinterpret_cast<bf16x8*>(xs + (((lb * 4 + i) * P + p) * MT + m) * frag + (qd * rp + r) * 16) = f[p];
  }
  __syncthreads();
  for (int q = wave; q < (b1 - b0) * MT; q += NTHR / 64) {
    const int m = q % MT, lb = q / MT;
    f32x4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int p = P - 1; p >= 0; --p)
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            *reinterpret_cast<const bf16x8*>(xs + (((lb * 4 + i) * P + p) * MT + m) * frag + loff), ones, sum, 0, 0, 0);
      if (SUB == 4 || (SUB == 2 && (i & 1)) || i == 3) {
        const int sg = SUB == 4 ? i : SUB == 2 ? i >> 1 : 0;
        if (l16 == 0) *reinterpret_cast<f32x4*>(sums + ((lb * SUB + sg) * MT + m) * 16 + quad * 4) = sum;
        sum = f32x4{0, 0, 0, 0};
      }
    }
  }
  __syncthreads();
}

template <int MT, int NT>
__device__ __forceinline__ void w4_store(const W4Args& a, int rt, int n0, const f32x4 (&tot)[MT][NT]) {
  const int l16 = threadIdx.x & 15, quad = (threadIdx.x >> 4) & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int n = n0 + nt * 16 + l16;
    if (n >= a.N) continue;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = (rt * MT + m) * 16 + quad * 4 + r;
        if (row >= a.R) continue;
        const size_t o = (size_t)row * a.N + n;
        if (a.out_bf16) store_out(reinterpret_cast<uint16_t*>(a.out) + o, tot[m][nt][r]);
        else store_out(reinterpret_cast<float*>(a.out) + o, tot[m][nt][r]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows, all of them in LDS for the whole call: one workgroup per CU with a
// run of column tiles, whose blocks its 16 wavefronts share out evenly, U at a
// time.  A wavefront streams its share without a barrier, fetching one step
// ahead across tile borders; a tile that lies in several shares is added up at
// the end, in the order of the wavefronts.
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

  auto fetch = [&](W4Ahead<ST, SUB, U> (&h)[1]) {
    w4_fetch<ST, SUB, U>(a, h[0], min(ftile * 16 + l16, a.N - 1), quad, fstep * U, nblk);
    if (++fstep == steps) {
      fstep = 0;
      ++ftile;
    }
  };
  f32x4 tot[MT][1], head[MT][1];
#pragma unroll
  for (int m = 0; m < MT; ++m) tot[m][0] = head[m][0] = f32x4{0, 0, 0, 0};
  bool begun = step == 0;   // the current tile's first block is this wavefront's
  auto compute = [&](const W4Ahead<ST, SUB, U> (&h)[1]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (step * U + u < nblk) w4_block<XT, ST, SUB, MT, 1, U>(a, h, u, step * U + u, smem, sums, frag, loff, quad, tot);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (++step == steps) {
      if (begun) {
        w4_store<MT, 1>(a, 0, tile * 16, tot);
      } else {
#pragma unroll
        for (int m = 0; m < MT; ++m) head[m][0] = tot[m][0];
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) tot[m][0] = f32x4{0, 0, 0, 0};
      step = 0;
      ++tile;
      begun = true;
    }
  };

  W4Ahead<ST, SUB, U> ha[1], hb[1];
  const int n = last - first;
  if (n > 0) fetch(ha);
  w4_stage<XT, SUB, MT, W4S_NT>(a, 0, 0, nblk, rp, smem, sums);
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
    for (int m = 0; m < MT; ++m) head[m][0] = tot[m][0];
  }
  f32x4* part = reinterpret_cast<f32x4*>(smem);   // [wave][MT][lane], over the staged rows
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; ++m) part[(wave * MT + m) * 64 + lane] = head[m][0];
  __syncthreads();
  if (n > 0 && step > 0 && begun) {
    const long long end = (long long)(tile - t0 + 1) * steps;
    for (int w = wave + 1; w < W4S_WAVES && all * w / W4S_WAVES < end; ++w)
#pragma unroll
      for (int m = 0; m < MT; ++m) tot[m][0] += part[(w * MT + m) * 64 + lane];
    w4_store<MT, 1>(a, 0, tile * 16, tot);
  }
}

// ---------------------------------------------------------------------------
// More rows than that.
// ---------------------------------------------------------------------------
constexpr int W4_NT = 512;                 // threads per workgroup
constexpr int W4_WAVES = W4_NT / 64;
constexpr int W4_LDS = 64 * 1024;          // per workgroup: two fit a CU

// MT * 16 rows of x by NT * 16 columns a wavefront.  A workgroup stages its
// rows of x a chunk of K at a time and streams weights from memory into
// registers, fetching one step ahead.  KS wavefronts share a column tile, each
// with a part of K, and add up in LDS in a fixed order.
template <typename XT, typename ST, int SUB, int MT, int NT, int U>
__global__ __launch_bounds__(W4_NT) __attribute__((amdgpu_waves_per_eu(2))) void w4_tile_kernel(W4Args a) {
  constexpr int P = W4Hidden<XT>::PARTS;
  extern __shared__ __align__(16) char dsmem[];
  char* smem = dsmem;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l16 = lane & 15, quad = lane >> 4;
  constexpr int rp = 16, frag = 64 * rp;
  float* sums = reinterpret_cast<float*>(smem + a.kc * 4 * P * MT * frag);
  const int loff = (quad * rp + l16) * 16;
  const int nblk = (a.K + 127) / 128;
  const int ks = a.KS > 1 ? wave % a.KS : 0, wn = a.KS > 1 ? wave / a.KS : wave;
  const int cols = W4_WAVES / a.KS * NT * 16;
  const long long sets = (long long)((a.N + cols - 1) / cols) * a.row_tiles;
  const int chunks = (nblk + a.kc - 1) / a.kc;
  // The row tiles of a column tile run on one XCD, one after the other.
  const long long set = (long long)(blockIdx.x & 7) * a.per_xcd + (blockIdx.x >> 3);
  if (set >= sets) return;
  const int rt = (int)(set % a.row_tiles);
  const int n0 = (int)(set / a.row_tiles) * cols + wn * NT * 16;
  f32x4 tot[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) tot[m][nt] = f32x4{0, 0, 0, 0};

  for (int c = 0; c < chunks; ++c) {
    const int b0 = c * a.kc, b1 = min(nblk, b0 + a.kc);
    // This wavefront's blocks of the chunk.
    const int w0 = b0 + (b1 - b0) * ks / a.KS, w1 = b0 + (b1 - b0) * (ks + 1) / a.KS;
    auto fetch = [&](W4Ahead<ST, SUB, U> (&h)[NT], int b) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) w4_fetch<ST, SUB, U>(a, h[nt], min(n0 + nt * 16 + l16, a.N - 1), quad, b, w1);
    };
    auto compute = [&](const W4Ahead<ST, SUB, U> (&h)[NT], int b) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (b + u < w1) w4_block<XT, ST, SUB, MT, NT, U>(a, h, u, b + u - b0, smem, sums, frag, loff, quad, tot);
    };
    W4Ahead<ST, SUB, U> ha[NT], hb[NT];
    if (w0 < w1) fetch(ha, w0);
    __syncthreads();
    w4_stage<XT, SUB, MT, W4_NT>(a, rt, b0, b1, rp, smem, sums);
    for (int b = w0; b < w1; b += 2 * U) {
      if (b + U < w1) fetch(hb, b + U);
      compute(ha, b);
      if (b + U >= w1) break;
      if (b + 2 * U < w1) fetch(ha, b + 2 * U);
      compute(hb, b + U);
    }
  }

  if (a.KS > 1) {
    // [wave][MT][NT][lane] partial sums over the staged rows; the first
    // wavefront of a column tile adds them in order.
    f32x4* red = reinterpret_cast<f32x4*>(smem);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) red[((wave * MT + m) * NT + nt) * 64 + lane] = tot[m][nt];
    __syncthreads();
    if (ks != 0) return;
    for (int o = 1; o < a.KS; ++o)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) tot[m][nt] += red[(((wave + o) * MT + m) * NT + nt) * 64 + lane];
  }
  w4_store<MT, NT>(a, rt, n0, tot);
}

}  // namespace sl
