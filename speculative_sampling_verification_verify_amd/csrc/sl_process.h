// Penalties, biases and masks on logits, and the token history behind them.
//
// Of a row's V values a step touches few: the tokens that the sequence holds,
// the drafts before the position and the biased ids.  Everything else is
// copied, or left alone in place, or set to -inf where the mask forbids it.
// So a workgroup first streams its piece of a row (copy and mask, 16 bytes a
// lane, nothing in place where the mask allows all), and then walks the lists:
// every touched token inside the piece is read again from the input and
// written once.  In place, the stream leaves allowed values as they are, so
// the second read still sees the input.
#pragma once

#include "sl_common.h"

namespace sl {

constexpr int PR_NT = 256;                                // threads per workgroup
constexpr int PR_SPECIAL = SL_MAX_DRAFT + SL_MAX_BIAS;    // drafts and biased ids of a row
constexpr int PR_HASH = 4096;                             // slots of their hash table
constexpr uint32_t IN_PROMPT = 0x80000000u;

struct ProcessArgs {
  const void* in;
  void* out;
  const uint32_t* counts;
  const int32_t* ids;
  const int32_t* num;
  const int32_t* slots;
  const int32_t* drafts;
  const float* rep;
  const float* pres;
  const float* freq;
  const int32_t* bias_ids;
  const float* bias_vals;
  const uint32_t* masks;
  const int32_t* mask_rows;
  const int32_t* rows;
  int S, draft_stride, first, NB, M, B, J, V;
  int W;        // words of a mask row
  int chunks;   // pieces per row
  int piece;    // elements per piece, a multiple of 32
  int wide;     // 1: the bases of in and out are 16-byte aligned
};

struct Penalty {
  float rep, pres, freq;
};

// One value after the penalties and the bias; no operation is contracted, so
// each is rounded by itself.
__device__ __forceinline__ float adjust(float z, bool seen, uint32_t count, const Penalty& p, float bias, bool biased) {
#pragma clang fp contract(off)
  if (seen) z = z > 0.0f ? z / p.rep : z * p.rep;
  const float f = p.freq * (float)count;
  z = z - f;
  z = z - (count ? p.pres : 0.0f);
  if (biased) z = z + bias;
  return z;
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

__device__ __forceinline__ uint32_t hash_of(uint32_t v) { return (v * 2654435761u) >> 20; }   // 12 bits

// The mask bits of the elements e .. e + 31 (as many as the table has).
__device__ __forceinline__ uint32_t mask_word(const uint32_t* m, int W, int e) {
  const int w = e >> 5, sh = e & 31;
  const uint32_t lo = m[w];
  if (!sh) return lo;
  const uint32_t hi = w + 1 < W ? m[w + 1] : 0u;
  return (lo >> sh) | (hi << (32 - sh));
}

template <typename ET> struct Elem;
template <> struct Elem<uint16_t> {
  static constexpr int VEC = 8;
  static constexpr uint16_t NEG_INF = 0xFF80u;
  static constexpr uint16_t QNAN = 0x7FC0u;
  // The 16 bytes with -inf where a bit is 0.
  __device__ __forceinline__ static uint4 mask(uint4 v, uint32_t bits) {
    return make_uint4(pair(v.x, bits), pair(v.y, bits >> 2), pair(v.z, bits >> 4), pair(v.w, bits >> 6));
  }
  __device__ __forceinline__ static uint32_t pair(uint32_t v, uint32_t bits) {
    const uint32_t lo = bits & 1u ? v & 0xFFFFu : 0xFF80u;
    const uint32_t hi = bits & 2u ? v & 0xFFFF0000u : 0xFF800000u;
    return lo | hi;
  }
};
template <> struct Elem<float> {
  static constexpr int VEC = 4;
  static constexpr uint32_t NEG_INF = 0xFF800000u;
  static constexpr uint32_t QNAN = 0x7FC00000u;
  __device__ __forceinline__ static uint4 mask(uint4 v, uint32_t bits) {
    return make_uint4(bits & 1u ? v.x : NEG_INF, bits & 2u ? v.y : NEG_INF, bits & 4u ? v.z : NEG_INF,
                      bits & 8u ? v.w : NEG_INF);
  }
};

template <typename ET> struct Raw;
template <> struct Raw<uint16_t> { typedef uint16_t type; };
template <> struct Raw<float> { typedef uint32_t type; };

// One workgroup per (row, piece).  Pieces start at whole 16-byte units of the
// row (after the `head` elements in front of its first one), so no two
// workgroups write into one unit.  With nothing to stream (in place, no mask)
// the pieces are shares of the lists instead.
template <typename ET>
__global__ __launch_bounds__(PR_NT) void process_kernel(ProcessArgs a) {
  typedef typename Raw<ET>::type RT;
  constexpr int VEC = Elem<ET>::VEC;
  __shared__ int32_t s_hash[PR_HASH];         // ids, -1 free
  __shared__ uint32_t s_twice[PR_HASH / 32];  // bit h: the id in slot h was listed more than once
  __shared__ int32_t s_spec[PR_SPECIAL];      // slot << 16 | entry that took it
  __shared__ int s_nspec;
  const int tid = threadIdx.x;
  const int c = (int)(blockIdx.x % (unsigned)a.chunks);
  const int row = (int)(blockIdx.x / (unsigned)a.chunks);
  const int b = row / a.J, j = row % a.J;
  if (a.rows && j >= a.rows[b]) return;
  const size_t base = (size_t)row * a.V;
  const RT* in = reinterpret_cast<const RT*>(a.in) + base;
  RT* out = reinterpret_cast<RT*>(a.out) + base;
  const bool copy = a.in != a.out;
  const bool shares = !copy && !a.mask_rows;
  const int head = a.wide ? min(a.V, (int)((16 - (base * sizeof(RT)) % 16) % 16 / sizeof(RT))) : 0;
  int lo = 0, hi = a.V;
  if (!shares) {
    if (c > 0) lo = min(a.V, head + c * a.piece);
    if (c + 1 < a.chunks) hi = min(a.V, head + (c + 1) * a.piece);
  }

  Penalty p;
  p.rep = a.rep ? a.rep[b] : 1.0f;
  p.pres = a.pres ? a.pres[b] : 0.0f;
  p.freq = a.freq ? a.freq[b] : 0.0f;
  const int mrow = a.mask_rows ? a.mask_rows[row] : -1;
  if (!(p.rep > 0.0f) || !finite(p.rep) || !finite(p.pres) || !finite(p.freq) || mrow < -1 || mrow >= a.M) {
    const int step = shares ? PR_NT * a.chunks : PR_NT;
    for (int e = lo + (shares ? c * PR_NT : 0) + tid; e < hi; e += step) out[e] = Elem<ET>::QNAN;
    return;
  }
  const uint32_t* mask = mrow >= 0 ? a.masks + (size_t)mrow * a.W : nullptr;
  const bool penal = p.rep != 1.0f || p.pres != 0.0f || p.freq != 0.0f;
  const int slot = a.counts && penal ? (a.slots ? a.slots[b] : b) : -1;
  const bool held = slot >= 0 && slot < a.S;
  const uint32_t* counts = held ? a.counts + (size_t)slot * a.V : nullptr;
  const int nd = a.drafts && penal ? a.first + j : 0;
  const int32_t* drafts = a.drafts + (size_t)b * a.draft_stride;
  const int32_t* bias_ids = a.bias_ids + (size_t)b * a.NB;
  const float* bias_vals = a.bias_vals + (size_t)b * a.NB;
  const int nlist = nd + a.NB;

  // The drafts and biased ids of this piece, each once.
  int hmask = 63;
  while (hmask + 1 < 2 * nlist) hmask = 2 * hmask + 1;
  if (nlist) {
    for (int i = tid; i <= hmask; i += PR_NT) s_hash[i] = -1;
    for (int i = tid; i < PR_HASH / 32; i += PR_NT) s_twice[i] = 0;
    if (tid == 0) s_nspec = 0;
    __syncthreads();
    for (int i = tid; i < nlist; i += PR_NT) {
      const int v = i < nd ? drafts[i] : bias_ids[i - nd];
      if (v < lo || v >= hi) continue;
      uint32_t h = hash_of(v) & hmask;
      for (;;) {   // the table has twice as many slots as there are ids
        const int old = atomicCAS(&s_hash[h], -1, v);
        if (old == -1) s_spec[atomicAdd(&s_nspec, 1)] = (int)(h << 16) | i;
        if (old == v) atomicOr(&s_twice[h >> 5], 1u << (h & 31));
        if (old == -1 || old == v) break;
        h = (h + 1) & hmask;
      }
    }
  }

  // Copy and mask.
  if (copy || mask) {
    const int start = c == 0 ? head : lo;
    const int units = a.wide ? (hi - start) / VEC : 0;
    constexpr uint32_t all = (1u << VEC) - 1u;
    for (int u = tid; u < units; u += PR_NT) {
      const int e = start + u * VEC;
      const uint32_t bits = mask ? mask_word(mask, a.W, e) & all : all;
      if (!copy && bits == all) continue;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (bits) v = *reinterpret_cast<const uint4*>(in + e);
      *reinterpret_cast<uint4*>(out + e) = Elem<ET>::mask(v, bits);
    }
    const int rest = start + units * VEC;
    const int before = c == 0 ? start : 0;   // elements in front of the row's first unit
    for (int i = tid; i < before + (hi - rest); i += PR_NT) {
      const int e = i < before ? i : rest + (i - before);
      const bool ok = !mask || (mask[e >> 5] >> (e & 31) & 1u);
      if (!ok || copy) out[e] = ok ? in[e] : (RT)Elem<ET>::NEG_INF;
    }
  }
  __syncthreads();

  // The listed ids.
  if (nlist) {
    const int ns = s_nspec;
    for (int k = tid; k < ns; k += PR_NT) {
      const int h = s_spec[k] >> 16, i = s_spec[k] & 0xFFFF;
      const int v = s_hash[h];
      if (shares && v % a.chunks != c) continue;
      if (mask && !(mask[v >> 5] >> (v & 31) & 1u)) continue;
      const uint32_t word = counts ? counts[v] : 0u;
      uint32_t count = word & ~IN_PROMPT;
      float bias = 0.0f;
      bool biased = false;
      if (s_twice[h >> 5] >> (h & 31) & 1u) {
        for (int d = 0; d < nd; ++d) count += drafts[d] == v;
        for (int d = 0; d < a.NB; ++d)
          if (bias_ids[d] == v) {
            bias = biased ? bias + bias_vals[d] : bias_vals[d];
            biased = true;
          }
      } else if (i < nd) {
        ++count;
      } else {
        bias = bias_vals[i - nd];
        biased = true;
      }
      store_out(reinterpret_cast<ET*>(out) + v,
                adjust(load_in(reinterpret_cast<const ET*>(in) + v), (word & IN_PROMPT) || count, count, p, bias, biased));
    }
  }

  // The tokens that the slot holds, other than those.
  if (held) {
    const int32_t* ids = a.ids + (size_t)slot * a.V;
    const int n = min(a.num[slot], a.V);
    const int step = shares ? PR_NT * a.chunks : PR_NT;
    for (int i = (shares ? c * PR_NT : 0) + tid; i < n; i += step) {
      const int v = ids[i];
      if (v < lo || v >= hi) continue;
      if (mask && !(mask[v >> 5] >> (v & 31) & 1u)) continue;
      if (nlist) {
        uint32_t h = hash_of(v) & hmask;
        int at;
        while ((at = s_hash[h]) != -1 && at != v) h = (h + 1) & hmask;
        if (at == v) continue;
      }
      const uint32_t word = counts[v];
      if (!word) continue;
      const uint32_t count = word & ~IN_PROMPT;
      store_out(reinterpret_cast<ET*>(out) + v,
                adjust(load_in(reinterpret_cast<const ET*>(in) + v), true, count, p, 0.0f, false));
    }
  }
}

// ---------------------------------------------------------------------------
// The token history.
// ---------------------------------------------------------------------------

struct HistoryArgs {
  uint32_t* counts;
  int32_t* ids;
  int32_t* num;
  const int32_t* slots;
  const int32_t* tokens;
  int S, V, B, T, prompt;
  int chunks;   // workgroups per sequence
};

constexpr int HA_NT = 256;

// One token a lane.  The atomic tells the one lane that finds a token new;
// a wavefront's new tokens take their places in the list with one atomic.
// The order of the list depends on the order of the wavefronts, the set that
// it holds and the counts do not.
__global__ __launch_bounds__(HA_NT) void history_append_kernel(HistoryArgs a) {
  const int b = (int)(blockIdx.x / (unsigned)a.chunks);
  const int i = (int)(blockIdx.x % (unsigned)a.chunks) * HA_NT + threadIdx.x;
  const int slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.S) return;
  const int v = i < a.T ? a.tokens[(size_t)b * a.T + i] : -1;
  bool fresh = false;
  if (v >= 0 && v < a.V) {
    uint32_t* c = a.counts + (size_t)slot * a.V + v;
    fresh = (a.prompt ? atomicOr(c, IN_PROMPT) : atomicAdd(c, 1u)) == 0u;
  }
  const unsigned long long who = __ballot(fresh);
  if (!who) return;
  const int lane = threadIdx.x & 63;
  int at = 0;
  if (lane == __ffsll((long long)who) - 1) at = atomicAdd(a.num + slot, __popcll(who));
  at = __shfl(at, __ffsll((long long)who) - 1) + __popcll(who & ((1ull << lane) - 1));
  if (fresh && at >= 0 && at < a.V) a.ids[(size_t)slot * a.V + at] = v;
}

constexpr int HR_NT = 1024;

// One workgroup per slot.
__global__ __launch_bounds__(HR_NT) void history_reset_kernel(HistoryArgs a) {
  const int slot = a.slots ? a.slots[blockIdx.x] : (int)blockIdx.x;
  if (slot < 0 || slot >= a.S) return;
  const int32_t* ids = a.ids + (size_t)slot * a.V;
  uint32_t* counts = a.counts + (size_t)slot * a.V;
  const int n = min(a.num[slot], a.V);
  for (int i = threadIdx.x; i < n; i += HR_NT) {
    const int v = ids[i];
    if (v >= 0 && v < a.V) counts[v] = 0u;
  }
  __syncthreads();
  if (threadIdx.x == 0) a.num[slot] = 0;
}

}  // namespace sl
