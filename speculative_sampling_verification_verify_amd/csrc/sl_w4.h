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
  int row_tiles;
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

__device__ __forceinline__ float w4_scale(const uint16_t* s, size_t i) { return __uint_as_float((uint32_t)s[i] << 16); }
__device__ __forceinline__ float w4_scale(const float* s, size_t i) { return s[i]; }

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

// One wavefront: 16 rows of x by 16 rows of the weight matrix, all of K in
// blocks of 128.  SUB: groups in a block (4, 2, or 1 where a group is one or
// more whole blocks).  A lane's 16-byte load holds 32 consecutive k; with more
// than one group in a block the words are transposed so that every product
// stays in one group.
template <typename XT, typename ST, typename OT, int SUB>
__global__ __launch_bounds__(256) void w4_kernel(W4Args a) {
  constexpr int P = W4Hidden<XT>::PARTS;
  const int lane = threadIdx.x & 63, l16 = lane & 15, quad = lane >> 4;
  const long long tile = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int rt = (int)(tile % a.row_tiles);
  const long long nt = tile / a.row_tiles;
  if (nt * 16 >= a.N) return;
  const int n = (int)nt * 16 + l16;
  const int nn = min(n, a.N - 1);
  const int row = min(rt * 16 + l16, a.R - 1);
  const XT* x = reinterpret_cast<const XT*>(a.x) + (size_t)row * a.K;
  const uint8_t* w = a.w + (size_t)nn * (a.K / 2);
  const ST* s = reinterpret_cast<const ST*>(a.s) + (size_t)nn * a.G;
  const uint8_t* z = a.z ? a.z + (size_t)nn * a.G : nullptr;
  const bf16x8 ones = __builtin_bit_cast(bf16x8, make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u));
  f32x4 tot = {0, 0, 0, 0}, blk = tot, sum = tot;
  const int nblk = (a.K + 127) / 128;
  int in_group = 0, g = 0;
  for (int b = 0; b < nblk; ++b) {
    uint32_t d[4] = {0, 0, 0, 0};
    const int kw = b * 128 + quad * 32;
    if (kw < a.K) {
      const uint4 v = *reinterpret_cast<const uint4*>(w + kw / 2);
      d[0] = v.x;
      d[1] = v.y;
      d[2] = v.z;
      d[3] = v.w;
    }
    if (SUB > 1) w4_transpose(d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int kx = SUB > 1 ? b * 128 + i * 32 + quad * 8 : b * 128 + quad * 32 + i * 8;
      bf16x8 f[P];
      if (kx < a.K) {
        W4Hidden<XT>::load(x + kx, f);
      } else {
#pragma unroll
        for (int p = 0; p < P; ++p) f[p] = __builtin_bit_cast(bf16x8, make_uint4(0, 0, 0, 0));
      }
      const bf16x8 wv = w4_expand(d[i]);
#pragma unroll
      for (int p = P - 1; p >= 0; --p) {
        blk = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[p], wv, blk, 0, 0, 0);
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[p], ones, sum, 0, 0, 0);
      }
      const bool end = SUB == 4 || (SUB == 2 && (i & 1)) || (SUB == 1 && i == 3 && (++in_group == a.gb || b + 1 == nblk));
      if (end && g < a.G) {
        const float sc = w4_scale(s, g), zz = 16.0f + (float)(z ? (z[g] & 15) : 8);
#pragma unroll
        for (int r = 0; r < 4; ++r) tot[r] = __builtin_fmaf(sc, __builtin_fmaf(-zz, sum[r], blk[r]), tot[r]);
        blk = sum = f32x4{0, 0, 0, 0};
        in_group = 0;
        ++g;
      }
    }
  }
  if (n < a.N) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int orow = rt * 16 + quad * 4 + r;
      if (orow < a.R) store_out(reinterpret_cast<OT*>(a.out) + (size_t)orow * a.N + n, tot[r]);
    }
  }
}

}  // namespace sl
