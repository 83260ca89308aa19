// Sampling and verifying with min-p, temperature, top-k and top-p.
//
// min-p keeps p(v) >= min_p * max p, which is z(v) >= zmax + T ln(min_p): a bound
// on the value, as top-k and top-p are.  It comes first (temperature, min-p,
// top-k, top-p), so that everything after it works on the few values that it
// keeps, and a row's processed distribution is its values >= thr, with one sum.
//
//   minp_cut_kernel       one workgroup per (logit row, row part): the part is
//                         read once, into registers; its maximum and the
//                         values that may be kept go to the workspace
//   minp_position_kernel  one workgroup per sequence, one wavefront per position:
//                         the kept values of the position's target and draft
//                         row, gathered in LDS, give p(x), q(x), the overlap
//                         and the draw as if the first rejection were there;
//                         then the acceptance
//   minp_row_kernel, minp_row_position_kernel, minp_finish_kernel
//                         the same from the logits, for rows without min-p and
//                         rows with more than the lists hold, one
//                         workgroup a row (a part's list is cut against the part's
//                         maximum: one flat part overflows it, also far below
//                         what the row keeps); where the caller says that there are
//                         none of the first, minp_left_kernel in place of the
//                         three, one workgroup a sequence
//
// Probabilities and normalisers are held in 64 bits, nucleus masses as multiples
// of 2^-42 of the largest value's (whole numbers, whose sum does not depend on
// its order): what decides is within V 2^-42 of its exact value.  (So is the
// normaliser behind a nucleus that minp_row_kernel or minp_left_kernel found: that
// mass.  From the lists it is a sum in float64.)
//
// What bounds it, at B = 256, V = 152064, 7 drafts, bf16 (1.17 GB of logits; all
// with min-p 0.05): the cut takes 173 of 193 us, 6.75 TB/s, which is what the
// memory gives to reads alone; the position kernel 17 us, most of it one chain of
// dependent steps, whose instructions are fetched from memory; the launch after it 4 us.
#pragma once

#include "sv_common.h"
#include "sv_finish.h"   // shfl_up_u64

namespace sv {

constexpr int MP_NT = 256;        // threads of a cut workgroup
constexpr int MP_WAVES = MP_NT / 64;
constexpr int MP_POS_NT = 512;    // threads of a position workgroup
constexpr int MP_POS_WAVES = MP_POS_NT / 64;
constexpr int MP_PART_CAP = 512;  // list entries of a row part
constexpr int MP_ROW_NT = 1024;   // threads of a row workgroup
constexpr int MP_ROW_GRID = 512;
constexpr int MP_LEFT_GRID = 256;
constexpr int MP_QUEUE = 128;
constexpr int MP_FEW_KEYS = 8192; // keys of one bin that a row workgroup holds
constexpr int MP_BINS = 256;      // bins of a row's masses, 1/8 wide in (zmax - z) / T; also a digit's
constexpr int MP_FIX = 42;        // fraction bits of a mass: at most 2^20 masses of at most 1

// Flags in a part's count.
constexpr uint32_t MP_BAD = 1u << 30;    // NaN or +inf
constexpr uint32_t MP_OVER = 1u << 31;   // more than MP_PART_CAP entries

// A row's processed distribution: its values with keys >= thr, exp((z - zmax) / T) / S each.
struct MinpRow {
  uint32_t thr;
  float zmax;
  double invS;
};

struct MinpArgs {
  Args a;                 // rows, parameters, outputs; a.pos the records, a.dense_count[0] the number of
                          // positions left to the row kernel, a.dense_list those positions; a.split
                          // rows to sample of a position workgroup
  const float* min_p;     // [B] or null (0)
  uint32_t* part_max;     // [rows][NP] largest key
  uint32_t* part_count;   // [rows][NP] entries, or flags
  void* part_list;        // [rows][NP][MP_PART_CAP] MinpEntry
  float* out_prob;        // sampler: [R] or null
  uint32_t* left;         // [B] 1: the row kernels finish the sequence
  MinpRow* rows;          // [B * (G + 1)][2] distributions of the positions left to the row kernels
};

template <typename ET> struct MinpEntry;
template <> struct MinpEntry<uint16_t> {
  typedef uint32_t type;   // bits, index in the part (a part has at most 2^14)
  __device__ __forceinline__ static type make(uint32_t bits, uint32_t i) { return bits << 16 | i; }
  __device__ __forceinline__ static uint32_t bits(type e) { return e >> 16; }
  __device__ __forceinline__ static uint32_t index(type e) { return e & 0xFFFFu; }
};
template <> struct MinpEntry<float> {
  typedef uint2 type;
  __device__ __forceinline__ static type make(uint32_t bits, uint32_t i) { return make_uint2(bits, i); }
  __device__ __forceinline__ static uint32_t bits(type e) { return e.x; }
  __device__ __forceinline__ static uint32_t index(type e) { return e.y; }
};

// How min-p treats sequence b.
enum { MP_INVALID = 0, MP_GREEDY = 1, MP_LIST = 2, MP_ROW = 3 };   // MP_ROW: min-p is off
struct MinpMode {
  Mode m;
  int kind, k;     // k: top-k, 0: off
  float mp;
};
__device__ __forceinline__ MinpMode minp_mode(const MinpArgs& ma, int b) {
  MinpMode r;
  r.m = seq_mode(ma.a, b);
  const int k = ma.a.topk ? ma.a.topk[b] : 0;
  r.k = k > 0 && k < ma.a.V ? k : 0;
  r.mp = ma.min_p ? ma.min_p[b] : 0.0f;
  const int gl = ma.a.gamma_len ? ma.a.gamma_len[b] : ma.a.G;
  const bool ok = r.m.mode != MODE_INVALID && r.m.tp == r.m.tp && r.mp <= 1.0f && (ma.a.sampler || (gl >= 1 && gl <= ma.a.G));
  r.kind = !ok ? MP_INVALID : r.m.mode == MODE_GREEDY ? MP_GREEDY : r.mp > 0.0f ? MP_LIST : MP_ROW;
  return r;
}

// ---------------------------------------------------------------------------
// Integers in the order of the values: of a bit pattern, pattern ^ (sign ?
// 0x7FF.. : 0), signed.  -0 comes right below +0.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int mp_order32(float f) {
  const int b = __float_as_int(f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
template <typename ET> __device__ __forceinline__ uint32_t mp_key_of_order(int o);
template <> __device__ __forceinline__ uint32_t mp_key_of_order<uint16_t>(int o) { return 0x8000u + (uint32_t)o + (o < 0 ? 1u : 0u); }
template <> __device__ __forceinline__ uint32_t mp_key_of_order<float>(int o) { return 0x80000000u + (uint32_t)o + (o < 0 ? 1u : 0u); }

// The smallest key whose value is not below c.
template <typename ET>
__device__ __forceinline__ uint32_t mp_key_from(double c) {
  if (!(c > -3.4028234663852886e38)) return Key<ET>::NEG_INF + 1;   // every finite value
  float f = (float)c;
  int o = mp_order32(f);
  if ((double)f < c) ++o;
  if (sizeof(ET) == 2) o = o >= 0 ? (int)(((uint32_t)o + 0xFFFFu) >> 16) : o >> 16;
  return mp_key_of_order<ET>(o);
}

// The smallest key that min-p keeps in a row whose largest is kmax.  (T = inf and min_p = 1: every finite value.)
template <typename ET>
__device__ __forceinline__ uint32_t mp_least_key(const MinpMode& mm, uint32_t kmax) {
  return min(mp_key_from<ET>((double)Key<ET>::value(kmax) + (double)mm.m.T * log((double)mm.mp)), kmax);
}

// exp(x) for x <= 0 in 64 bits: 2^k times the Taylor polynomial of degree 13 of exp on
// [-ln 2 / 2, ln 2 / 2]; the first term left out, r^14 / 14!, is at most 4.2e-18, below 2^-57.
__device__ __forceinline__ double mp_exp(double x) {
  x = fmax(x, -746.0);   // -inf, too: 2^-1076 and a bit, which ldexp rounds to 0
  const double k = rint(x * 1.4426950408889634);
  const double r = fma(k, -0x1.cf79abc9e3b3ap-40, fma(k, -0x1.62e42fefap-1, x));   // ln 2 in two parts, the first of 36 bits
  double p = 1.0 / 6227020800.0;
  p = fma(p, r, 1.0 / 479001600.0);
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return ldexp(p, (int)k);
}

// ---------------------------------------------------------------------------
// The cut: one workgroup per (row, part).  The whole part is in flight before its
// first value is used, and many workgroups a CU hide what then follows; a list is
// cut against the part's own maximum, so that no workgroup waits for another.
// (A row's true bound is higher: the position kernel skips parts whose maximum is
// below it.)
// ---------------------------------------------------------------------------

// Elements that a row begins behind a 16-byte boundary.
template <typename ET>
__device__ __forceinline__ int mp_lead(const ET* row) { return (int)((uintptr_t)row % 16 / sizeof(ET)); }

// The 16 bytes of a row from element e on; -inf before it and behind its end.
__device__ __forceinline__ u32x4 mp_load(const uint16_t* row, int e, int V) {
  u32x4 v = {0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u};
  if (e >= 0 && e + 8 <= V) {
    __builtin_memcpy(&v, row + e, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i >= 0 && e + i < V) v[i / 2] = i & 1 ? (v[i / 2] & 0xFFFFu) | (uint32_t)row[e + i] << 16 : (v[i / 2] & 0xFFFF0000u) | row[e + i];
  }
  return v;
}
__device__ __forceinline__ u32x4 mp_load(const float* row, int e, int V) {
  u32x4 v = {0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u};
  if (e >= 0 && e + 4 <= V) {
    __builtin_memcpy(&v, row + e, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e + i >= 0 && e + i < V) v[i] = __float_as_uint(row[e + i]);
  }
  return v;
}

typedef short s16x2 __attribute__((ext_vector_type(2)));

// Ordered integers of a 16-byte unit, in place, with their largest and smallest.
template <typename ET> struct MinpOrder;
template <> struct MinpOrder<uint16_t> {
  typedef s16x2 T;
  static constexpr int LOW = -32641;   // -inf
  static constexpr int HIGH = 32640;   // +inf
  __device__ __forceinline__ static T map(uint32_t x) {
    const s16x2 v = __builtin_bit_cast(s16x2, x);
    return v ^ ((v >> 15) & (short)0x7FFF);
  }
  __device__ __forceinline__ static T hi(T a, T b) { return __builtin_elementwise_max(a, b); }
  __device__ __forceinline__ static T lo(T a, T b) { return __builtin_elementwise_min(a, b); }
  __device__ __forceinline__ static int hi(T a) { return a.x > a.y ? a.x : a.y; }
  __device__ __forceinline__ static int lo(T a) { return a.x < a.y ? a.x : a.y; }
  __device__ __forceinline__ static int get(T a, int i) { return i ? a.y : a.x; }
  __device__ __forceinline__ static float value(int o) {
    return __uint_as_float((uint32_t)(o ^ ((o >> 31) & 0x7FFF)) << 16);
  }
  __device__ __forceinline__ static uint32_t bits(int o) { return (uint32_t)(o ^ ((o >> 31) & 0x7FFF)) & 0xFFFFu; }
  // No value >= f has a smaller integer than this.
  __device__ __forceinline__ static int floor_of(float f) { return mp_order32(f) >> 16; }
};
template <> struct MinpOrder<float> {
  typedef int T;
  static constexpr int LOW = (int)0x807FFFFFu;
  static constexpr int HIGH = 0x7F800000;
  __device__ __forceinline__ static T map(uint32_t x) { return (int)x ^ (((int)x >> 31) & 0x7FFFFFFF); }
  __device__ __forceinline__ static T hi(T a, T b) { return max(a, b); }
  __device__ __forceinline__ static T lo(T a, T b) { return min(a, b); }
  __device__ __forceinline__ static int get(T a, int) { return a; }
  __device__ __forceinline__ static float value(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7FFFFFFF)); }
  __device__ __forceinline__ static uint32_t bits(int o) { return (uint32_t)(o ^ ((o >> 31) & 0x7FFFFFFF)); }
  __device__ __forceinline__ static int floor_of(float f) { return mp_order32(f); }
};
template <typename ET> __device__ __forceinline__ int mp_hi(typename MinpOrder<ET>::T v) { return MinpOrder<ET>::hi(v); }
template <> __device__ __forceinline__ int mp_hi<float>(int v) { return v; }
template <typename ET> __device__ __forceinline__ int mp_lo(typename MinpOrder<ET>::T v) { return MinpOrder<ET>::lo(v); }
template <> __device__ __forceinline__ int mp_lo<float>(int v) { return v; }

__device__ __forceinline__ int wave_max_i32(int v) { return (int)(wave_max_dpp((uint32_t)v ^ 0x80000000u) ^ 0x80000000u); }
__device__ __forceinline__ int wave_min_i32(int v) { return (int)(wave_min_dpp((uint32_t)v ^ 0x80000000u) ^ 0x80000000u); }

template <typename ET, int VPL>
__global__ __launch_bounds__(MP_NT) void minp_cut_kernel(MinpArgs ma) {
  typedef MinpOrder<ET> O;
  typedef typename O::T T;
  typedef MinpEntry<ET> E;
  constexpr int VEC = Key<ET>::VEC, PER = 4 / sizeof(ET);   // values of a unit, of a word
  __shared__ int smax[MP_WAVES], smin[MP_WAVES];
  __shared__ uint32_t scnt[MP_WAVES];
  __shared__ typename E::type stage[MP_WAVES][MP_PART_CAP];
  const Args& a = ma.a;
  const long long unit = blockIdx.x;
  if (unit == 0 && threadIdx.x == 0) a.dense_count[0] = 0;   // the workspace needs no preparation
  const int part = (int)(unit % a.NP);
  const long long rowid = unit / a.NP;
  const int b = (int)(rowid / a.RS), slot = (int)(rowid % a.RS);
  const MinpMode mm = minp_mode(ma, b);
  const bool isP = slot <= a.G;
  const int pos = isP ? slot : slot - a.G - 1;
  if ((mm.kind != MP_LIST && mm.kind != MP_GREEDY) || pos > mm.m.g || (!isP && pos >= mm.m.g)) return;   // not used
  const ET* row = row_ptr<ET>(a, b, isP, pos);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  // Parts begin at a 16-byte boundary, the first one up to a unit before the row.
  const int e0 = part * a.PL - mp_lead(row), w0 = (wave * VPL * 64 + lane) * VEC;   // the lane's first value in the part
  u32x4 raw[VPL];
  if (e0 >= 0 && e0 + MP_NT * VPL * VEC <= a.V) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) raw[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + e0 + w0 + j * 64 * VEC));
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) raw[j] = mp_load(row, e0 + w0 + j * 64 * VEC, a.V);
  }
  T v[VPL][4], hi, lo;
#pragma unroll
  for (int j = 0; j < VPL; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[j][i] = O::map(raw[j][i]);
      hi = j + i == 0 ? v[j][i] : O::hi(hi, v[j][i]);
      lo = j + i == 0 ? v[j][i] : O::lo(lo, v[j][i]);
    }
  const int wh = wave_max_i32(mp_hi<ET>(hi)), wl = wave_min_i32(mp_lo<ET>(lo));
  if (lane == 0) {
    smax[wave] = wh;
    smin[wave] = wl;
  }
  __syncthreads();
  int top = smax[0], bot = smin[0];
#pragma unroll
  for (int i = 1; i < MP_WAVES; ++i) {
    top = max(top, smax[i]);
    bot = min(bot, smin[i]);
  }
  const bool bad = top >= O::HIGH || bot < O::LOW;
  // What may be kept: at least the part's maximum plus T ln(min_p), the sum
  // formed in 32 bits with room for its rounding.
  int t = top;
  if (mm.kind == MP_LIST) {
    const float z = O::value(top), d = mm.m.T * logf(mm.mp);
    const float c = z + d - 1e-5f * (fabsf(z) + fabsf(d)) - 1e-6f * mm.m.T;
    t = c > -3.4e38f ? O::floor_of(c) : O::LOW + 1;   // (also where T is infinite)
  }
  t = max(min(t, top), O::LOW + 1);
  if (t == 0) t = -1;   // -0 is not below +0
  uint32_t n = 0;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const T m = O::hi(O::hi(v[j][0], v[j][1]), O::hi(v[j][2], v[j][3]));
    const bool any = mp_hi<ET>(m) >= t;
    if (__ballot(any) == 0ull) continue;
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) c += O::get(v[j][i / PER], i % PER) >= t ? 1u : 0u;
    const uint32_t incl = wave_incl_scan_dpp(c);
    uint32_t at = n + incl - c;
    n += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int o = O::get(v[j][i / PER], i % PER);
      if (o >= t) {
        if (at < (uint32_t)MP_PART_CAP) stage[wave][at] = E::make(O::bits(o), (uint32_t)(w0 + j * 64 * VEC + i));
        ++at;
      }
    }
  }
  if (lane == 0) scnt[wave] = n;
  __syncthreads();
  uint32_t base = 0, total = 0;
#pragma unroll
  for (int i = 0; i < MP_WAVES; ++i) {
    if (i == wave) base = total;
    total += scnt[i];
  }
  typename E::type* out = reinterpret_cast<typename E::type*>(ma.part_list) + (size_t)unit * MP_PART_CAP;
  for (uint32_t i = lane; i < min(n, (uint32_t)MP_PART_CAP); i += 64)
    if (base + i < (uint32_t)MP_PART_CAP) out[base + i] = stage[wave][i];
  if (threadIdx.x == 0) {
    ma.part_max[unit] = mp_key_of_order<ET>(top);
    // Of equal maxima only the first counts where the token is the argmax.
    const bool over = total > (uint32_t)MP_PART_CAP && mm.kind != MP_GREEDY;
    ma.part_count[unit] = bad ? MP_BAD : over ? MP_OVER : min(total, (uint32_t)MP_PART_CAP);
  }
}

// ---------------------------------------------------------------------------
// Pieces for a group of NTHR threads: a workgroup, or (64) one wavefront of it,
// which needs no barrier.  `red` is NTHR / 64 slots.
// ---------------------------------------------------------------------------
template <int NTHR>
__device__ __forceinline__ void mp_sync() {
  if (NTHR == 64) wave_lds_sync();
  else __syncthreads();
}
template <int NTHR> __device__ __forceinline__ int mp_tid() { return (int)threadIdx.x & (NTHR - 1); }

// Every wavefront's value from its last lane, to all: fn(wavefront, value).
template <int NTHR, typename T, class F>
__device__ __forceinline__ void mp_gather_waves(T v, bool mine, T* red, F fn) {
  __syncthreads();
  if (mine) red[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NTHR / 64; ++i) fn(i, red[i]);
}
template <int NTHR>
__device__ __forceinline__ double mp_sum(double v, double* red) {
  v = wave_sum_dpp(v);
  if (NTHR == 64) return v;
  double r = 0.0;
  mp_gather_waves<NTHR>(v, (threadIdx.x & 63) == 0, red, [&](int, double x) { r += x; });
  return r;
}
// The exclusive prefix of v in thread order, and the total.
template <int NTHR>
__device__ __forceinline__ double mp_scan(double v, double* red, double* total) {
  const double incl = wave_incl_scan_f64(v);
  double base = 0.0, all = readlane_f64(incl, 63);
  if (NTHR > 64) {
    all = 0.0;
    mp_gather_waves<NTHR>(incl, (threadIdx.x & 63) == 63, red, [&](int i, double x) {
      if (i < (int)(threadIdx.x >> 6)) base += x;
      all += x;
    });
  }
  *total = all;
  return base + incl - v;
}
template <int NTHR>
__device__ __forceinline__ uint32_t mp_scan_u32(uint32_t v, uint32_t* red, uint32_t* total) {
  const uint32_t incl = wave_incl_scan_dpp(v);
  uint32_t base = 0, all = (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  if (NTHR > 64) {
    all = 0;
    mp_gather_waves<NTHR>(incl, (threadIdx.x & 63) == 63, red, [&](int i, uint32_t x) {
      if (i < (int)(threadIdx.x >> 6)) base += x;
      all += x;
    });
  }
  *total = all;
  return base + incl - v;
}
template <int NTHR, class Op>
__device__ __forceinline__ uint32_t mp_reduce_u32(uint32_t v, uint32_t neutral, uint32_t* red, Op op) {
  v = wave_reduce_dpp_u32(v, neutral, op);
  if (NTHR == 64) return v;
  uint32_t r = neutral;
  mp_gather_waves<NTHR>(v, (threadIdx.x & 63) == 0, red, [&](int, uint32_t x) { r = op(r, x); });
  return r;
}

struct MinpScratch {
  unsigned long long hist[MP_BINS];
  double red[MP_ROW_NT / 64];
  uint32_t red_u[MP_ROW_NT / 64];
  uint32_t bc[8];
};

// e in [0, 1] as a multiple of 2^-42, to the nearest: the fraction bits of 2^52 + e 2^42
// (a conversion to 64-bit integers takes ten instructions).
__device__ __forceinline__ unsigned long long mp_fixed(double e) {
  return (unsigned long long)__double_as_longlong(fma(e, (double)(1ull << MP_FIX), 0x1p52)) & ((1ull << 52) - 1);
}

// The largest key t with mass(key >= t) >= tau, of the keys that feed gives
// (with their masses; `above`: the mass of those it leaves out, all larger), a
// radix select from the top digit down; 0 if there is none.  *mass: mass(key >= t).
template <int LEVELS, int NTHR, class Feed>
__device__ __forceinline__ uint32_t mp_nucleus(Feed feed, unsigned long long above, double tau, MinpScratch& s, unsigned long long* mass) {
  uint32_t prefix = 0, pmask = 0;
  for (int lvl = 0; lvl < LEVELS; ++lvl) {
    const int shift = 8 * (LEVELS - 1 - lvl);
    mp_sync<NTHR>();
    for (int i = mp_tid<NTHR>(); i < 256; i += NTHR) s.hist[i] = 0ull;
    mp_sync<NTHR>();
    feed([&](uint32_t key, double e) {
      if ((key & pmask) == prefix) atomicAdd(&s.hist[(key >> shift) & 255u], mp_fixed(e));
    });
    mp_sync<NTHR>();
    if (mp_tid<NTHR>() < 64) {
      const int lane = threadIdx.x & 63, first = 255 - 4 * lane;   // four digits a lane, from the top
      unsigned long long c[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = s.hist[first - i];
        sum += c[i];
      }
      unsigned long long incl = sum;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const unsigned long long u = shfl_up_u64(incl, o);
        if (lane >= o) incl += u;
      }
      const unsigned long long reach = __ballot((double)(above + incl) >= tau);
      const int hit = reach ? __ffsll((long long)reach) - 1 : -1;
      if (lane == hit) {
        unsigned long long run = above + incl - sum;
        int d = 3;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          unsigned long long upto = run;
#pragma unroll
          for (int q = 0; q <= i; ++q) upto += c[q];
          if ((double)upto >= tau) d = i;
        }
        unsigned long long at = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q < d) run += c[q];
          if (q == d) at = c[q];
        }
        at += run;
        s.bc[0] = (uint32_t)(first - d);
        s.bc[1] = (uint32_t)run;
        s.bc[2] = (uint32_t)(run >> 32);
        s.bc[5] = (uint32_t)at;
        s.bc[6] = (uint32_t)(at >> 32);
      }
      if (lane == 0 && hit < 0) s.bc[0] = NONE;
    }
    mp_sync<NTHR>();
    const uint32_t d = s.bc[0];
    above = ((unsigned long long)s.bc[2] << 32) | s.bc[1];
    *mass = ((unsigned long long)s.bc[6] << 32) | s.bc[5];
    if (d == NONE) return 0;
    prefix |= d << shift;
    pmask |= 255u << shift;
  }
  return prefix;
}

// top-k, of the keys >= thr that feed gives (with any others below): raises thr.
template <typename ET, int NTHR, class Feed>
__device__ __forceinline__ void mp_top_k(Feed feed, const MinpMode& mm, MinpScratch& s, uint32_t* thr) {
  if (!mm.k) return;
  const auto some = [&](auto fn) { feed([&](uint32_t key) { fn(key >= *thr ? key : 0u); }); };
  uint32_t* hist = reinterpret_cast<uint32_t*>(s.hist);
  uint32_t t;
  mp_sync<NTHR>();
  if constexpr (NTHR == 64) t = wave_kth<Key<ET>::LEVELS>(some, (uint32_t)mm.k, hist);
  else t = block_kth_largest<Key<ET>::LEVELS, NTHR>(some, (uint32_t)mm.k, hist, s.bc);
  *thr = max(*thr, t);
}

// top-k and top-p of the keys that feed gives with their weights, the largest
// kmax; returns the sum of those >= thr.
template <typename ET, int NTHR, class Feed>
__device__ __forceinline__ double mp_filter(Feed feed, const MinpMode& mm, uint32_t kmax, MinpScratch& s, uint32_t* thr) {
  mp_top_k<ET, NTHR>([&](auto fn) { feed([&](uint32_t key, double) { fn(key); }); }, mm, s, thr);
  const bool nucleus = mm.m.tp < 1.0f && mm.m.tp > 0.0f;
  if (mm.m.tp <= 0.0f) *thr = kmax;
  double S = 0.0;
  unsigned long long mass;
#pragma unroll 1
  for (int pass = 0; pass < (nucleus ? 2 : 1); ++pass) {
    if (pass == 1) {
      const uint32_t t = mp_nucleus<Key<ET>::LEVELS, NTHR>([&](auto fn) {
        feed([&](uint32_t key, double e) {
          if (key >= *thr) fn(key, e);
        });
      }, 0ull, (double)mm.m.tp * S * (double)(1ull << MP_FIX), s, &mass);
      *thr = max(*thr, t);
    }
    double x = 0.0;
    feed([&](uint32_t key, double e) {
      if (key >= *thr) x += e;
    });
    S = mp_sum<NTHR>(x, s.red);
  }
  return S;
}

// ---------------------------------------------------------------------------
// One position from the logits, for rows without min-p or whose lists do not hold
// what is kept.  A pass over a row of 128255 takes 10 to 40 us of a workgroup, where it
// forms an exponential in 64 bits for each value; so what the passes form
// is what they need, once: two exponentials a value at most, fewer behind a nucleus.
// At 32 such sequences of up to 8 drafts (264 rows of 128255 in all, bf16): 120 us for
// the distributions, 93 us for the positions.  `few` holds `cap` keys.
// ---------------------------------------------------------------------------
template <typename ET>
__device__ __forceinline__ uint32_t mp_key_of(const u32x4& raw, int i) {   // of value i of a unit
  return Key<ET>::of_bits(sizeof(ET) == 2 ? (raw[i / 2] >> (16 * (i % 2))) & 0xFFFFu : raw[i]);
}

// fn(key, index) for a unit's values, a word at a time: 16 wavefronts hide what
// one copy of fn's code waits for, and eight copies neither fit the registers nor
// the instruction cache.
template <typename ET, class F>
__device__ __forceinline__ void mp_for_words(u32x4 raw, int e, F fn) {
#pragma unroll 1
  for (int w = 0; w < 4; ++w) {
    const uint32_t x = raw.x;
    raw = u32x4{raw.y, raw.z, raw.w, x};
    if (sizeof(ET) == 2) {
      fn(Key<ET>::of_bits(x & 0xFFFFu), e + 2 * w);
      fn(Key<ET>::of_bits(x >> 16), e + 2 * w + 1);
    } else {
      fn(Key<ET>::of_bits(x), e + w);
    }
  }
}

// fn(16 bytes, first element) for units `step` elements apart from e on, -inf
// behind the row's end; the next one is under way meanwhile.
template <typename ET, class F>
__device__ __forceinline__ void mp_for_units(const ET* row, int e, int end, int step, int V, F fn) {
  u32x4 next = {0, 0, 0, 0};
  if (e < end) next = mp_load(row, e, V);
#pragma unroll 1
  for (; e < end; e += step) {
    const u32x4 raw = next;
    if (e + step < end) next = mp_load(row, e + step, V);
    fn(raw, e);
  }
}

template <typename ET, int NTHR, class F>
__device__ __forceinline__ void mp_for_row(const ET* row, int V, F fn) {
  constexpr int VEC = Key<ET>::VEC;
  mp_for_units(row, (int)threadIdx.x * VEC, V, NTHR * VEC, V, [&](const u32x4& raw, int e) { mp_for_words<ET>(raw, e, fn); });
}

// A row's distribution; false: it has no valid one.  Passes over the row: its
// maximum; the sum, with the masses by bins of the value; the keys of the bin in
// which the nucleus ends.
template <typename ET, int NTHR>
__device__ __forceinline__ bool mp_row_stats(const ET* row, int V, const MinpMode& mm, MinpScratch& s, uint32_t* few, int cap, MinpRow* out) {
  constexpr int VEC = Key<ET>::VEC;
  const double invT = 1.0 / (double)mm.m.T;
  uint32_t kmax = 0, bad = 0;
  mp_for_units(row, (int)threadIdx.x * VEC, V, NTHR * VEC, V, [&](const u32x4& raw, int) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const uint32_t key = mp_key_of<ET>(raw, i);
      kmax = max(kmax, key);
      bad |= key_valid<ET>(key) ? 0u : 1u;
    }
  });
  kmax = mp_reduce_u32<NTHR>(kmax, 0u, s.red_u, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
  bad = mp_reduce_u32<NTHR>(bad, 0u, s.red_u, [](uint32_t x, uint32_t y) { return x | y; });
  if (bad || kmax <= Key<ET>::NEG_INF) return false;
  const float zmax = Key<ET>::value(kmax);
  const double z0 = (double)zmax;
  uint32_t thr = mm.mp > 0.0f ? mp_least_key<ET>(mm, kmax) : Key<ET>::NEG_INF + 1;
  const auto keys = [&](auto fn) { mp_for_row<ET, NTHR>(row, V, [&](uint32_t key, int) { fn(key); }); };
  const auto exponent = [&](uint32_t key) { return ((double)Key<ET>::value(key) - z0) * invT; };
  mp_top_k<ET, NTHR>(keys, mm, s, &thr);
  const bool nucleus = mm.m.tp < 1.0f && mm.m.tp > 0.0f;
  const auto bin = [](double x) { return (uint32_t)fmin(-8.0 * x, (double)(MP_BINS - 1)); };
  __syncthreads();
  for (int i = threadIdx.x; i < MP_BINS; i += NTHR) s.hist[i] = 0ull;
  __syncthreads();
  double sum = 0.0;
  if (mm.m.tp < 1.0f && !nucleus) thr = kmax;   // top_p <= 0
  keys([&](uint32_t key) {
    if (key >= thr) {
      const double x = exponent(key), e = mp_exp(x);
      sum += e;
      if (nucleus) atomicAdd(&s.hist[bin(x)], mp_fixed(e));
    }
  });
  double S = mp_sum<NTHR>(sum, s.red);   // (the bins are complete)
  if (nucleus) {
    const double tau = (double)mm.m.tp * S * (double)(1ull << MP_FIX);
    if (threadIdx.x < 64) {
      constexpr int PER = MP_BINS / 64;
      unsigned long long c = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) c += s.hist[threadIdx.x * PER + i];
      unsigned long long incl = c;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const unsigned long long u = shfl_up_u64(incl, o);
        if ((int)threadIdx.x >= o) incl += u;
      }
      const unsigned long long reach = __ballot((double)incl >= tau);
      if (reach == 0ull) {
        if (threadIdx.x == 0) s.bc[4] = NONE;
      } else if ((int)threadIdx.x == __ffsll((long long)reach) - 1) {
        unsigned long long run = incl - c;
        int i = 0;
        while (i < PER - 1 && (double)(run + s.hist[threadIdx.x * PER + i]) < tau) run += s.hist[threadIdx.x * PER + i++];
        s.bc[4] = threadIdx.x * PER + i;
        s.bc[5] = (uint32_t)run;
        s.bc[6] = (uint32_t)(run >> 32);
      }
      if (threadIdx.x == 0) s.bc[3] = 0;
    }
    __syncthreads();
    const uint32_t cross = s.bc[4];
    const unsigned long long above = ((unsigned long long)s.bc[6] << 32) | s.bc[5];
    if (cross != NONE) {   // (else rounding: everything is kept)
      const auto of_bin = [&](uint32_t key) { return key >= thr && bin(exponent(key)) == cross; };
      keys([&](uint32_t key) {
        if (of_bin(key)) {
          const uint32_t at = atomicAdd(&s.bc[3], 1u);
          if (at < (uint32_t)cap) few[at] = key;   // in any order: their masses are whole numbers
        }
      });
      __syncthreads();
      const uint32_t found = s.bc[3];
      uint32_t t;
      unsigned long long mass;
      if (found <= (uint32_t)cap) {
        t = mp_nucleus<Key<ET>::LEVELS, NTHR>([&](auto fn) {
          for (uint32_t j = threadIdx.x; j < found; j += NTHR) fn(few[j], mp_exp(exponent(few[j])));
        }, above, tau, s, &mass);
      } else {
        t = mp_nucleus<Key<ET>::LEVELS, NTHR>([&](auto fn) {
          keys([&](uint32_t key) {
            if (of_bin(key)) fn(key, mp_exp(exponent(key)));
          });
        }, above, tau, s, &mass);
      }
      if (t > thr) {   // what is kept has the mass found (another pass would take as long as the first)
        thr = t;
        S = (double)mass / (double)(1ull << MP_FIX);
      }
    }
  }
  out->thr = thr;
  out->zmax = zmax;
  out->invS = 1.0 / S;
  return true;
}

// The position's record from its two rows' distributions (the second is used
// where the position has a draft).  queue: MP_QUEUE entries a wavefront.
template <typename ET, int NTHR>
__device__ __forceinline__ PosRec mp_position_from_rows(const MinpArgs& ma, const MinpMode& mm, int b, int i, const MinpRow& r0,
                                                        const MinpRow& r1, MinpScratch& s, uint2* queue) {
  const Args& a = ma.a;
  const int V = a.V;
  const bool two = i < mm.m.g;
  PosRec rec{0.0, 0.0, 0.0, -1, 0u};
  const double invT = 1.0 / (double)mm.m.T;
  const ET* row[2] = {row_ptr<ET>(a, b, true, i), row_ptr<ET>(a, b, !two, i)};
  const MinpRow r[2] = {r0, two ? r1 : MinpRow{0xFFFFFFFFu, 0.0f, 0.0}};
  const auto prob = [&](int h, uint32_t key) {
    return key >= r[h].thr ? mp_exp(((double)Key<ET>::value(key) - (double)r[h].zmax) * invT) * r[h].invS : 0.0;
  };
  // A wavefront's run of consecutive ids: the draw then looks for its token in
  // one run.
  constexpr int NW = NTHR / 64, PER = Key<ET>::VEC;
  const int run = ((V + NW - 1) / NW + PER - 1) / PER * PER, wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  const int v1 = min(V, (wave + 1) * run);
  bool resid = two;
  double al = 0.0, z = 0.0;
  const auto weight = [&](uint32_t kp, uint32_t kq, double* overlap) {
    const double p = prob(0, kp);
    if (!(p > 0.0) || !resid) return p;
    const double q = prob(1, kq);
    *overlap += fmin(p, q);
    return fmax(p - q, 0.0);
  };
  // fn(key of the target's row, of the draft's, id) for the units at id v.
  const auto both = [&](const u32x4& raw, u32x4 other, int v, auto fn) {
    mp_for_words<ET>(raw, v, [&](uint32_t key, int id) {
      fn(key, mp_key_of<ET>(other, sizeof(ET) == 2 ? (id - v) & 1 : 0), id);
      if (sizeof(ET) == 4 || ((id - v) & 1)) other = u32x4{other.y, other.z, other.w, other.x};
    });
  };
  const ET* second = two ? row[1] : row[0];
  // The sums of the runs, in s.red, and their total.  Where a few values are kept,
  // these first go through a queue of the wavefront's, so that it forms their
  // probabilities 64 at a time.
  const bool few = r[0].thr > Key<ET>::NEG_INF + 1;
  const auto sums = [&]() {
    z = 0.0;
    uint2* mine = queue + wave * MP_QUEUE;
    int have = 0;
    u32x4 next0 = {0, 0, 0, 0}, next1 = {0, 0, 0, 0};
    const int e0 = wave * run;
    if (e0 + lane * PER < v1) {
      next0 = mp_load(row[0], e0 + lane * PER, V);
      next1 = mp_load(second, e0 + lane * PER, V);
    }
#pragma unroll 1
    for (int t = e0; t < v1; t += 64 * PER) {   // (runs end with a unit or the row)
      const int e = t + lane * PER;
      const bool in = e < v1;
      const u32x4 raw0 = next0, raw1 = next1;
      if (e + 64 * PER < v1) {
        next0 = mp_load(row[0], e + 64 * PER, V);
        next1 = mp_load(second, e + 64 * PER, V);
      }
      both(raw0, raw1, e, [&](uint32_t kp, uint32_t kq, int) {
        if (!few) {
          if (in) z += weight(kp, kq, &al);
          return;
        }
        const bool keep = in && kp >= r[0].thr;
        const unsigned long long mask = __ballot(keep);
        if (keep) mine[have + __popcll(mask & ((1ull << lane) - 1))] = make_uint2(kp, kq);
        have += __popcll(mask);
        if (have < 64) return;
        wave_lds_sync();
        const uint2 now = mine[lane], rest = mine[64 + lane];   // (MP_QUEUE entries)
        wave_lds_sync();
        mine[lane] = rest;
        have -= 64;
        z += weight(now.x, now.y, &al);
      });
    }
    wave_lds_sync();
    if (lane < have) z += weight(mine[lane].x, mine[lane].y, &al);
    return mp_sum<NTHR>(z, s.red);
  };
  double Z = sums();
  if (two && !(Z > 0.0)) {   // no residual is left: draw from p
    resid = false;
    Z = sums();
  }
  // min{v : C(v) > u Z}: first the run, then a tile of ids at a time; else the
  // last weight above 0.
  const double target = (double)a.u[(size_t)b * (a.G + 1) + a.G] * Z;
  double base = 0.0;
  int t0 = 0;
  for (int w = 0; w + 1 < NW && !(base + s.red[w] > target); ++w) {
    base += s.red[w];
    t0 += run;
  }
  rec.alpha = mp_sum<NTHR>(al, s.red);
  const int x = two ? a.draft[(size_t)b * a.G + i] : -1;
  if (x >= 0 && x < V) {
    rec.px = prob(0, Key<ET>::load_key(row[0], x));
    rec.qx = prob(1, Key<ET>::load_key(row[1], x));
  }
  uint32_t last = 0, hit = NONE;
  for (int again = 0; again < 2; ++again) {
    for (; t0 < V && hit == NONE; t0 += NTHR * PER) {
      const int v0 = t0 + (int)threadIdx.x * PER;
      double loc = 0.0, tot, none = 0.0;
      u32x4 raw = {0, 0, 0, 0}, other = raw;
      const bool some = v0 < V;
      if (some) {
        raw = mp_load(row[0], v0, V);
        other = mp_load(second, v0, V);
      }
      if (some) both(raw, other, v0, [&](uint32_t kp, uint32_t kq, int v) {
        const double w = weight(kp, kq, &none);
        loc += w;
        if (w > 0.0) last = (uint32_t)(v + 1);
      });
      double c = base + mp_scan<NTHR>(loc, s.red, &tot);
      uint32_t mine = NONE;
      if (some && c + loc > target) both(raw, other, v0, [&](uint32_t kp, uint32_t kq, int v) {
        const double w = weight(kp, kq, &none);
        c += w;
        if (mine == NONE && w > 0.0 && c > target) mine = (uint32_t)v;
      });
      hit = mp_reduce_u32<NTHR>(mine, NONE, s.red_u, [](uint32_t p, uint32_t q) { return p < q ? p : q; });
      base += tot;
    }
    last = mp_reduce_u32<NTHR>(last, 0u, s.red_u, [](uint32_t p, uint32_t q) { return p > q ? p : q; });
    if (hit != NONE || last != 0) break;
    t0 = 0;   // no weight from that run on: from the first id
    base = 0.0;
  }
  rec.tok = hit != NONE ? (int)hit : (int)last - 1;
  if (ma.a.sampler) rec.px = prob(0, Key<ET>::load_key(row[0], rec.tok));
  return rec;
}

// A sampled row's outputs, by one thread.
__device__ __forceinline__ void mp_put_sample(const MinpArgs& ma, int b, const PosRec& rec) {
  const Args& a = ma.a;
  const float u = a.u[b];
  const bool ok = rec.bad == 0u && u >= 0.0f && u < 1.0f;
  a.out_tokens[b] = ok ? rec.tok : -1;
  if (ma.out_prob) ma.out_prob[b] = ok ? (float)rec.px : __int_as_float(0x7FC00000);
}

// The positions that the position kernel left, in two launches: the distributions
// of their rows, one workgroup a row, then the positions.
template <typename ET>
__global__ __launch_bounds__(MP_ROW_NT) void minp_row_kernel(MinpArgs ma) {
  __shared__ MinpScratch s;
  __shared__ uint32_t few[MP_FEW_KEYS];
  const Args& a = ma.a;
  const uint32_t n = 2 * a.dense_count[0];
  for (uint32_t j = blockIdx.x; j < n; j += gridDim.x) {
    const int id = a.dense_list[j / 2], b = id / (a.G + 1), i = id % (a.G + 1), h = (int)(j & 1);
    const MinpMode mm = minp_mode(ma, b);
    if (h && i >= mm.m.g) continue;
    MinpRow r;
    const bool ok = mp_row_stats<ET, MP_ROW_NT>(row_ptr<ET>(a, b, !h, i), a.V, mm, s, few, MP_FEW_KEYS, &r);
    if (!ok) r.thr = 0;   // no key
    if (threadIdx.x == 0) ma.rows[2 * (size_t)id + h] = r;
    __syncthreads();
  }
}

template <typename ET>
__global__ __launch_bounds__(MP_ROW_NT) void minp_row_position_kernel(MinpArgs ma) {
  __shared__ MinpScratch s;
  __shared__ uint2 queue[MP_ROW_NT / 64 * MP_QUEUE];
  const Args& a = ma.a;
  const uint32_t n = a.dense_count[0];
  for (uint32_t j = blockIdx.x; j < n; j += gridDim.x) {
    const int id = a.dense_list[j], b = id / (a.G + 1), i = id % (a.G + 1);
    const MinpMode mm = minp_mode(ma, b);
    const MinpRow r0 = ma.rows[2 * (size_t)id], r1 = i < mm.m.g ? ma.rows[2 * (size_t)id + 1] : r0;
    PosRec rec{0.0, 0.0, 0.0, -1, 1u};
    if (r0.thr && r1.thr) rec = mp_position_from_rows<ET, MP_ROW_NT>(ma, mm, b, i, r0, r1, s, queue);
    if (threadIdx.x == 0) {
      if (a.sampler) mp_put_sample(ma, b, rec);
      else a.pos[id] = rec;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// One position from the lists, by a wavefront or a workgroup; PER entries of a
// row a thread.
// ---------------------------------------------------------------------------
template <int NTHR, int PER>
struct MinpSmem {
  static constexpr int CAP = NTHR * PER;
  MinpScratch s;
  uint32_t key[2][CAP], id[2][CAP];
  double w[2][CAP];      // weights, then probabilities
  int n[2];
  uint32_t base[NTHR];   // entries before each of some parts
};
typedef MinpSmem<64, 3> MinpWave;
typedef MinpSmem<MP_POS_NT, 2> MinpBlock;

enum { MP_OK = 0, MP_IS_BAD = 1, MP_TOO_LONG = 2 };

// A thread's part of a row: its maximum and count.
struct MinpPart {
  uint32_t top, count;
};
__device__ __forceinline__ MinpPart mp_part(const MinpArgs& ma, long long rowid, int p) {
  const long long at = rowid * ma.a.NP + p;
  return p < ma.a.NP ? MinpPart{ma.part_max[at], ma.part_count[at]} : MinpPart{0u, 0u};
}

// One row's processed distribution from its lists: the values that min-p keeps, in
// ascending id, into key[h], id[h] and w[h], exp((z - zmax) / T) each; then
// the probabilities of what top-k and top-p leave, 0 for the others.  first: the
// thread's part among the first NTHR.  (All of this is executed about once in a
// launch, from memory: its time is that of fetching the instructions, so there is
// one copy of it for both rows.)
template <typename ET, int NTHR, int PER>
__device__ __forceinline__ int mp_list_row(const MinpArgs& ma, const MinpMode& mm, long long rowid, const ET* row, int h, MinpPart first,
                                           MinpSmem<NTHR, PER>& s) {
  typedef MinpEntry<ET> E;
  constexpr int CAP = NTHR * PER;
  const int NP = ma.a.NP, tid = mp_tid<NTHR>();
  uint32_t kmax = first.top, flags = first.count;
#pragma unroll 1
  for (int p = NTHR + tid; p < NP; p += NTHR) {
    const MinpPart q = mp_part(ma, rowid, p);
    kmax = max(kmax, q.top);
    flags |= q.count;
  }
  kmax = mp_reduce_u32<NTHR>(kmax, 0u, s.s.red_u, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
  flags = mp_reduce_u32<NTHR>(flags, 0u, s.s.red_u, [](uint32_t x, uint32_t y) { return x | y; });
  if ((flags & MP_BAD) || kmax <= Key<ET>::NEG_INF) return MP_IS_BAD;
  if (flags & MP_OVER) return MP_TOO_LONG;
  const bool greedy = mm.kind == MP_GREEDY;
  const double z0 = (double)Key<ET>::value(kmax), invT = greedy ? 0.0 : 1.0 / (double)mm.m.T;
  // The smallest key that is kept.  (By its weight a value close to the border cannot be told from it.)
  const uint32_t least = greedy ? kmax : mp_least_key<ET>(mm, kmax);
  const int lead = mp_lead(row);
  int have = 0;
#pragma unroll 1
  for (int p0 = 0; p0 < NP; p0 += NTHR) {   // NTHR parts at a time
    uint32_t total;
    const MinpPart q = p0 == 0 ? first : mp_part(ma, rowid, p0 + tid);
    s.base[tid] = mp_scan_u32<NTHR>(q.top >= least ? q.count : 0u, s.s.red_u, &total);
    mp_sync<NTHR>();
    const int np = min(NP - p0, NTHR);
#pragma unroll 1
    for (uint32_t i0 = 0; i0 < total; i0 += NTHR) {
      const uint32_t i = i0 + (uint32_t)tid;
      uint32_t key = 0, id = 0;
      if (i < total) {
        int lo = 0, hi = np - 1;   // the last part whose base is at most i
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (s.base[mid] <= i) lo = mid;
          else hi = mid - 1;
        }
        const typename E::type e = reinterpret_cast<const typename E::type*>(ma.part_list)[((size_t)rowid * NP + p0 + lo) * MP_PART_CAP + (i - s.base[lo])];
        key = Key<ET>::of_bits(E::bits(e));
        id = (uint32_t)((p0 + lo) * ma.a.PL - lead) + E::index(e);
      }
      const double w = mp_exp(((double)Key<ET>::value(key) - z0) * invT);
      const bool keep = i < total && key >= least;
      uint32_t all, at = (uint32_t)have;
      if constexpr (NTHR == 64) {
        const unsigned long long mask = __ballot(keep);
        at += (uint32_t)__popcll(mask & ((1ull << tid) - 1));
        all = (uint32_t)__popcll(mask);
      } else {
        at += mp_scan_u32<NTHR>(keep ? 1u : 0u, s.s.red_u, &all);
      }
      if (keep && at < (uint32_t)CAP) {
        s.key[h][at] = key;
        s.id[h][at] = id;
        s.w[h][at] = w;
      }
      have += (int)all;
    }
    mp_sync<NTHR>();
  }
  if (greedy) have = 1;   // the lowest id
  if (have > CAP) return MP_TOO_LONG;
  if (tid == 0) s.n[h] = have;
  if (!greedy) {
    uint32_t thr = 0;
    const double S = mp_filter<ET, NTHR>([&](auto fn) {
#pragma unroll 1
      for (int j = tid; j < have; j += NTHR) fn(s.key[h][j], s.w[h][j]);
    }, mm, kmax, s.s, &thr);
#pragma unroll 1
    for (int j = tid; j < have; j += NTHR) s.w[h][j] = s.key[h][j] >= thr ? s.w[h][j] / S : 0.0;
  }
  mp_sync<NTHR>();
  return MP_OK;
}

// q(v) by v's place among the n ascending ids of row 1.
__device__ __forceinline__ double mp_find(const uint32_t* id, const double* w, int n, uint32_t v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (id[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  return lo < n && id[lo] == v ? w[lo] : 0.0;
}

// MP_OK: the record is the position's.
template <typename ET, int NTHR, int PER>
__device__ __forceinline__ int mp_position_from_lists(const MinpArgs& ma, const MinpMode& mm, int b, int i, MinpSmem<NTHR, PER>& s,
                                                      PosRec* out) {
  const Args& a = ma.a;
  const int tid = mp_tid<NTHR>();
  const bool two = i < mm.m.g;
  PosRec rec{0.0, 0.0, 0.0, -1, 1u};
  *out = rec;
  if (mm.kind == MP_INVALID) return MP_OK;
  if (mm.kind == MP_ROW) return MP_TOO_LONG;
  const long long rowid[2] = {(long long)b * a.RS + i, (long long)b * a.RS + (two ? a.G + 1 + i : i)};
  const MinpPart first[2] = {mp_part(ma, rowid[0], tid), mp_part(ma, rowid[1], tid)};
  const uint32_t x = two ? (uint32_t)a.draft[(size_t)b * a.G + i] : NONE;
  const float u = a.u[(size_t)b * (a.G + 1) + a.G];
#pragma unroll 1
  for (int h = 0; h < (two ? 2 : 1); ++h) {
    const int how = mp_list_row(ma, mm, h ? rowid[1] : rowid[0], row_ptr<ET>(a, b, !h, i), h, h ? first[1] : first[0], s);
    if (how == MP_IS_BAD) return MP_OK;
    if (how != MP_OK) return how;
  }
  rec.bad = 0u;
  const int n[2] = {s.n[0], two ? s.n[1] : 0};
  // A thread's run of consecutive entries of the target's row.
  const int per = (n[0] + NTHR - 1) / NTHR, j0 = tid * per;
  double al = 0.0, z = 0.0, px = 0.0, w[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    w[e] = 0.0;
    if (e < per && j0 + e < n[0]) {
      const double p = s.w[0][j0 + e], q = two ? mp_find(s.id[1], s.w[1], n[1], s.id[0][j0 + e]) : 0.0;
      al += fmin(p, q);
      w[e] = fmax(p - q, 0.0);
      if (s.id[0][j0 + e] == x) px = p;
    }
    z += w[e];
  }
  rec.alpha = mp_sum<NTHR>(al, s.s.red);
  rec.px = mp_sum<NTHR>(px, s.s.red);   // one thread's
  double Z, before = mp_scan<NTHR>(z, s.s.red, &Z);
  if (!(Z > 0.0)) {   // no residual is left: draw from p
    z = 0.0;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      w[e] = e < per && j0 + e < n[0] ? s.w[0][j0 + e] : 0.0;
      z += w[e];
    }
    before = mp_scan<NTHR>(z, s.s.red, &Z);
  }
  rec.qx = two ? mp_find(s.id[1], s.w[1], n[1], x) : 0.0;
  const double target = (double)u * Z;
  uint32_t mine = NONE, last = 0;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    before += w[e];
    if (w[e] > 0.0) {
      last = (uint32_t)(j0 + e + 1);
      if (mine == NONE && before > target) mine = (uint32_t)(j0 + e);
    }
  }
  uint32_t hit = mp_reduce_u32<NTHR>(mine, NONE, s.s.red_u, [](uint32_t p, uint32_t q) { return p < q ? p : q; });
  last = mp_reduce_u32<NTHR>(last, 0u, s.s.red_u, [](uint32_t p, uint32_t q) { return p > q ? p : q; });
  if (hit == NONE) hit = last - 1;
  rec.tok = (int)s.id[0][hit];
  if (a.sampler) rec.px = s.w[0][hit];
  *out = rec;
  return MP_OK;
}

// ---------------------------------------------------------------------------
// Acceptance of sequence b from its records, by one wavefront.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mp_finish(const MinpArgs& ma, int b, const Mode& m, const PosRec* rec) {
  const Args& a = ma.a;
  const int lane = threadIdx.x & 63, G = a.G, g = m.g;
  const float* ub = a.u + (size_t)b * (G + 1);
  PosRec r{0.0, 0.0, 0.0, -1, 0u};
  int32_t x = 0;
  float u = 0.5f;
  if (lane < g) {
    r = rec[lane];
    x = a.draft[(size_t)b * G + lane];
    u = ub[lane];
  }
  const float ures = ub[G], lv = a.lenience ? a.lenience[b] : 1.0f;
  const bool bad = lane < g && (x < 0 || x >= a.V || !(u >= 0.0f && u < 1.0f) || r.bad);
  const bool ok = lv >= 0.0f && lv <= 1.0f && ures >= 0.0f && ures < 1.0f && !rec[g].bad && __ballot(bad) == 0ull;
  // The first rejection; if there is none, the bonus position.
  const unsigned long long rejected = __ballot(lane < g && !((double)u * (double)lv * r.qx < r.px));
  const int n = rejected ? __ffsll((long long)rejected) - 1 : g;
  const int tok = rec[n].tok;
  const float qnan = __int_as_float(0x7FC00000);
  const auto value = [&](double v) { return ok ? (lane < g ? (float)v : 0.0f) : qnan; };
  for (int i = lane; i <= G; i += 64)
    a.out_tokens[(size_t)b * (G + 1) + i] = !ok || i > n ? -1 : i < n ? x : tok;   // (i < n <= 64: i is the lane)
  if (lane < G) {
    a.out_alpha[(size_t)b * G + lane] = value(r.alpha);
    if (a.out_pq) {
      a.out_pq[((size_t)b * G + lane) * 2] = value(r.px);
      a.out_pq[((size_t)b * G + lane) * 2 + 1] = value(r.qx);
    }
  }
  if (lane == 0) a.out_n[b] = ok ? n : -1;
}

// One workgroup per sequence, or per a.split rows to sample: 17 us for 256
// sequences of 7 drafts, 5 us for one row to sample.  A wavefront
// takes a position whose rows keep at most MinpWave::CAP values each; the whole
// workgroup takes the longer ones after that, up to MinpBlock::CAP; what then is
// left goes to other launches, which also finish the sequence: listed by
// position, or (WHOLE) by sequence, with REC_REDO in the records.  (Computed here,
// with the registers that takes, it made the kernel spill: 19 instead of 6 us for
// 1000 rows of 1000.)
template <typename ET, bool WHOLE>
__global__ __launch_bounds__(MP_POS_NT, 4) void minp_position_kernel(MinpArgs ma) {
  __shared__ union {
    MinpWave wave[MP_POS_WAVES];
    MinpBlock block;
  } s;
  __shared__ PosRec rec[SV_MAX_GAMMA + 1];
  __shared__ uint32_t later[SV_MAX_GAMMA + 1];
  const Args& a = ma.a;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int b0 = a.sampler ? (int)blockIdx.x * a.split : (int)blockIdx.x;
  const Mode m0 = seq_mode(ma.a, b0);
  const int count = a.sampler ? min(a.split, a.B - b0) : m0.g + 1;
  for (int j = wave; j < count; j += MP_POS_WAVES) {
    const int b = a.sampler ? b0 + j : b0, i = a.sampler ? 0 : j;
    PosRec r;
    const int how = mp_position_from_lists<ET>(ma, minp_mode(ma, b), b, i, s.wave[wave], &r);
    if (lane == 0) {
      rec[j] = r;
      later[j] = how != MP_OK;
    }
  }
  __syncthreads();
  bool left = false;
  for (int j = 0; j < count; ++j) {
    if (!later[j]) continue;
    const int b = a.sampler ? b0 + j : b0, i = a.sampler ? 0 : j;
    const MinpMode mm = minp_mode(ma, b);
    PosRec r;
    const int how = mp_position_from_lists<ET>(ma, mm, b, i, s.block, &r);
    __syncthreads();
    if (how != MP_OK) {
      if (!WHOLE && threadIdx.x == 0) a.dense_list[atomicAdd(&a.dense_count[0], 1u)] = b * (a.G + 1) + i;
      if (WHOLE && a.sampler && threadIdx.x == 0) a.dense_list[atomicAdd(&a.dense_count[0], 1u)] = b;
      left = true;
    }
    if (threadIdx.x == 0 && how == MP_OK) {
      later[j] = 0;
      rec[j] = r;
    }
    __syncthreads();
  }
  if (a.sampler) {
    if ((int)threadIdx.x < count && !later[threadIdx.x]) mp_put_sample(ma, b0 + (int)threadIdx.x, rec[threadIdx.x]);
    return;
  }
  if (threadIdx.x == 0) {
    if (WHOLE && left) a.dense_list[atomicAdd(&a.dense_count[0], 1u)] = b0;
    if (!WHOLE) ma.left[b0] = left;
  }
  if (left) {
    for (int j = threadIdx.x; j < count; j += MP_POS_NT) {
      if (later[j]) rec[j].bad = REC_REDO;
      if (WHOLE || !later[j]) a.pos[(size_t)b0 * (a.G + 1) + j] = rec[j];   // (else the row kernels write it)
    }
  } else if (wave == 0) {
    mp_finish(ma, b0, m0, rec);
  }
}

// The sequences (or rows to sample) that the position kernel left whole: one
// workgroup each (of 512 threads: 1024 do not get the registers that it needs).
template <typename ET>
__global__ __launch_bounds__(MP_POS_NT) void minp_left_kernel(MinpArgs ma) {
  __shared__ MinpScratch s;
  __shared__ __align__(8) uint32_t few[MP_FEW_KEYS];   // keys, then the queues
  static_assert(MP_POS_NT / 64 * MP_QUEUE * 2 <= MP_FEW_KEYS, "the queues");
  const Args& a = ma.a;
  const uint32_t n = a.dense_count[0];
  for (uint32_t j = blockIdx.x; j < n; j += gridDim.x) {
    const int b = a.dense_list[j];
    const MinpMode mm = minp_mode(ma, b);
    PosRec* pos = a.pos + (size_t)b * (a.G + 1);
    for (int i = 0; i <= (a.sampler ? 0 : mm.m.g); ++i) {
      if (!a.sampler && pos[i].bad != REC_REDO) continue;
      __syncthreads();
      MinpRow r0, r1;
      bool ok = mp_row_stats<ET, MP_POS_NT>(row_ptr<ET>(a, b, true, i), a.V, mm, s, few, MP_FEW_KEYS, &r0);
      __syncthreads();
      r1 = r0;
      if (ok && i < mm.m.g) ok = mp_row_stats<ET, MP_POS_NT>(row_ptr<ET>(a, b, false, i), a.V, mm, s, few, MP_FEW_KEYS, &r1);
      __syncthreads();
      PosRec rec{0.0, 0.0, 0.0, -1, 1u};
      if (ok) rec = mp_position_from_rows<ET, MP_POS_NT>(ma, mm, b, i, r0, r1, s, reinterpret_cast<uint2*>(few));
      __syncthreads();   // (everyone has read pos[i])
      if (threadIdx.x == 0) {
        if (a.sampler) mp_put_sample(ma, b, rec);
        else pos[i] = rec;
      }
    }
    __syncthreads();
    if (!a.sampler && threadIdx.x < 64) mp_finish(ma, b, mm.m, pos);
    __syncthreads();
  }
}

// The sequences that the position kernel did not finish: one wavefront each.
constexpr int MP_FIN_NT = 256;
__global__ __launch_bounds__(MP_FIN_NT) void minp_finish_kernel(MinpArgs ma) {
  const int b = (int)(blockIdx.x * (MP_FIN_NT / 64) + (threadIdx.x >> 6));
  if (b >= ma.a.B || !ma.left[b]) return;
  mp_finish(ma, b, seq_mode(ma.a, b), ma.a.pos + (size_t)b * (ma.a.G + 1));
}

}  // namespace sv
