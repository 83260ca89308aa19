// Penalties, biases and masks on logits, and the token history behind them.
//
// Of a row's V values a step touches few: the tokens that the sequence holds,
// the drafts before the position and the biased ids.  Everything else is
// copied, or left alone in place, or set to -inf where the mask forbids it.
//
// Copying or masking (process_stream_kernel) is bound by the bytes of the
// logits.  A workgroup has a piece of the vocabulary, all rows of a sequence:
// it reads the history's list once and keeps the piece's touched ids, with
// their counts, in LDS.  Out of place, a row's piece goes through an LDS tile in
// which the touched values are adjusted between the load and the store, while
// the next row is being loaded: the logits are read and written once, in whole
// 16-byte units.  B=256, J=8, V=152064 with 2000 tokens held: 291 us, 4.3 TB/s
// (a plain copy by this kernel 249, by the library 233).  Writing the touched
// values again after a row was copied took 471 us, right behind each lane's own
// store 520: two more passes over scattered lines.  B=128, J=9, V=128256, ragged
// rows, a mask a row, 300 biases: 118 us, of which reading the lists, hashing
// the biased ids and the dependent loads before them are about half.  B=1000,
// J=5, V=1000 in fp32: 19.5 us, a chain of such loads in one round of workgroups.
// In place, only units that the mask changes are written, and then the touched
// values (B=64, J=5, V=128255, masks alone: 24 us; mixed masks touch nearly every
// unit, so 82 MB are read and written).  Without masks nothing is streamed: the
// lists are walked (process_lists_kernel; 97 us for the case above that takes
// 291 out of place).
#pragma once

#include "sl_common.h"

namespace sl {

constexpr int PR_NT = 256;                                // threads per workgroup
constexpr int PR_UNITS = 2;                               // 16-byte units that a lane has in flight
constexpr int PR_TILE = PR_NT * PR_UNITS;                 // units of the tile: one row's piece, or several rows'
constexpr int PR_ENTRIES = 1024;                          // touched ids of a piece kept in LDS; beyond, its list is walked per row
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
  int pieces;   // pieces of the vocabulary (stream), shares of the lists (lists)
  int piece;    // elements per piece, whole 16-byte units
  int groups;   // groups of rows of a sequence, each a workgroup's
  int wide;     // 1: the bases of in and out are 16-byte aligned
  int tile_off; // the tile's place in LDS
  int tile_rows; // rows that it holds
  int hmask;    // slots of the names' hash table - 1: at least one and a half times as many as there are names
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

// A unit that this call does not touch again goes past the caches.  B=128, J=9,
// V=128256 with masks, penalties and biases: stores 126 -> 101 us where the
// inputs of the last call are still in a cache, loads 125 -> 119 us on inputs
// that no cache holds.
__device__ __forceinline__ uint4 load_stream(const void* p) {
  typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ void store_stream(void* p, uint4 v) {
  typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(p));
}

// An id that drafts or biases name: the positions of the drafts that are it,
// and the sum of its biases.
struct Special {
  unsigned long long drafts;
  float bias;
  int biased;
};

// The ids that a sequence's drafts and biases name within [lo, hi), each once,
// in LDS: a hash table from id to entry.
struct Specials {
  int32_t* slot;      // [hmask + 1] ids, -1 free
  int32_t* entry;     // [hmask + 1] entry of the slot's id
  uint32_t* twice;    // [(hmask + 32) / 32] bit h: the id in slot h was named more than once
  Special* entries;
  int32_t* source;    // per entry: its slot
  int n;              // names: drafts and biases
  int hmask;

  static __host__ __device__ int bytes(int names, int hmask) {
    return names ? (hmask + 1) * 8 + (hmask + 32) / 32 * 4 + names * ((int)sizeof(Special) + 4) : 0;
  }

  // Builds the table; returns the number of entries.  Every thread calls it.
  __device__ __forceinline__ int build(char* smem, int* count, const int32_t* drafts, int nd, const int32_t* bias_ids,
                                       const float* bias_vals, int nb, int hm, int lo, int hi) {
    n = nd + nb;
    hmask = hm;
    if (!n) return 0;
    entries = reinterpret_cast<Special*>(smem);
    slot = reinterpret_cast<int32_t*>(entries + n);
    entry = slot + hmask + 1;
    source = entry + hmask + 1;
    twice = reinterpret_cast<uint32_t*>(source + n);
    const int tid = threadIdx.x;
    // The first names are loaded before the table is cleared.
    int v[PR_UNITS];
    float val[PR_UNITS];
    auto names = [&](int i0) {
#pragma unroll
      for (int k = 0; k < PR_UNITS; ++k) {
        const int i = i0 + k * PR_NT;
        v[k] = i < n ? i < nd ? drafts[i] : bias_ids[i - nd] : -1;
        val[k] = i >= nd && i < n ? bias_vals[i - nd] : 0.0f;
      }
    };
    names(tid);
    for (int i = tid; i <= hmask; i += PR_NT) slot[i] = -1;
    for (int i = tid; i < (hmask + 32) / 32; i += PR_NT) twice[i] = 0;
    if (tid == 0) *count = 0;
    __syncthreads();
    for (int i0 = tid;;) {
#pragma unroll
      for (int k = 0; k < PR_UNITS; ++k) {
        const int i = i0 + k * PR_NT;
        if (v[k] < lo || v[k] >= hi) continue;
        uint32_t h = hash_of(v[k]) & hmask;
        for (;;) {
          const int old = atomicCAS(&slot[h], -1, v[k]);
          if (old == -1) {
            const int e = atomicAdd(count, 1);
            entry[h] = e;
            source[e] = (int)h;
            entries[e] = i < nd ? Special{1ull << i, 0.0f, 0} : Special{0ull, val[k], 1};
          }
          if (old == v[k]) atomicOr(&twice[h >> 5], 1u << (h & 31));
          if (old == -1 || old == v[k]) break;
          h = (h + 1) & hmask;
        }
      }
      if ((i0 += PR_UNITS * PR_NT) >= n) break;
      names(i0);
    }
    __syncthreads();
    const int ne = *count;
    for (int e = tid; e < ne; e += PR_NT) {   // those named more than once, in the order of their names
      const int h = source[e];
      if (!(twice[h >> 5] >> (h & 31) & 1u)) continue;
      Special s = {0ull, 0.0f, 0};
      for (int d = 0; d < nd; ++d)
        if (drafts[d] == slot[h]) s.drafts |= 1ull << d;
      for (int d = 0; d < nb; ++d)
        if (bias_ids[d] == slot[h]) {
          s.bias = s.biased ? s.bias + bias_vals[d] : bias_vals[d];
          s.biased = 1;
        }
      entries[e] = s;
    }
    __syncthreads();
    return ne;
  }
  // The entry of id v, or -1.
  __device__ __forceinline__ int find(int v) const {
    uint32_t h = hash_of(v) & hmask;
    int at;
    while ((at = slot[h]) != -1 && at != v) h = (h + 1) & hmask;
    return at == v ? entry[h] : -1;
  }
  __device__ __forceinline__ int id(int e) const { return slot[source[e]]; }
};

// Adjusts one value of row j in place of what out holds there; nothing where
// the row does not touch it.
template <typename ET>
__device__ __forceinline__ void touch(const ET* in, ET* out, uint32_t word, const Special& s, int first, int j, const Penalty& p) {
  const int sees = first + j;
  const uint32_t count = (word & ~IN_PROMPT) + (uint32_t)__popcll(sees < 64 ? s.drafts & ((1ull << sees) - 1) : s.drafts);
  const bool seen = (word & IN_PROMPT) || count;
  if (!seen && !s.biased) return;
  store_out(out, adjust(load_in(in), seen, count, p, s.bias, s.biased != 0));
}

// What the kernels know of a sequence.
struct Sequence {
  Penalty p;
  bool bad;                // a penalty out of range: its rows become NaN
  const uint32_t* counts;  // of its slot, or null
  const int32_t* ids;
  int held;                // ids listed
  int nd;                  // drafts that its last row sees
  int rows;                // rows used
};
__device__ __forceinline__ Sequence sequence(const ProcessArgs& a, int b) {
  Sequence q;
  q.p.rep = a.rep ? a.rep[b] : 1.0f;
  q.p.pres = a.pres ? a.pres[b] : 0.0f;
  q.p.freq = a.freq ? a.freq[b] : 0.0f;
  q.bad = !(q.p.rep > 0.0f) || !finite(q.p.rep) || !finite(q.p.pres) || !finite(q.p.freq);
  const bool penal = !q.bad && (q.p.rep != 1.0f || q.p.pres != 0.0f || q.p.freq != 0.0f);
  const int slot = a.counts && penal ? (a.slots ? a.slots[b] : b) : -1;
  const bool held = slot >= 0 && slot < a.S;
  q.counts = held ? a.counts + (size_t)slot * a.V : nullptr;
  q.ids = held ? a.ids + (size_t)slot * a.V : nullptr;
  q.held = held ? max(0, min(a.num[slot], a.V)) : 0;
  q.nd = a.drafts && penal ? a.first + a.J - 1 : 0;
  q.rows = a.rows ? min(a.rows[b], a.J) : a.J;
  return q;
}

// One workgroup per (sequence, piece, group of rows).  Pieces start at whole
// 16-byte units of the sequence's first row; where a row's units lie otherwise
// (V odd), its `head` elements in front of its first unit move the piece, so
// that no two workgroups write into one unit.
// LISTS: the call has a history, drafts or biases.
template <typename ET, bool LISTS>
__global__ __launch_bounds__(PR_NT) void process_stream_kernel(ProcessArgs a) {
  typedef typename Raw<ET>::type RT;
  constexpr int VEC = Elem<ET>::VEC;
  constexpr uint32_t ALL = (1u << VEC) - 1u;
  extern __shared__ __align__(16) char smem[];
  __shared__ int s_special, s_listed;
  const int tid = threadIdx.x;
  const int c = (int)(blockIdx.x % (unsigned)a.pieces);
  const int rest = (int)(blockIdx.x / (unsigned)a.pieces);
  const int grp = rest % a.groups, b = rest / a.groups;
  const Sequence q = sequence(a, b);
  const int per = (a.J + a.groups - 1) / a.groups;
  const int j0 = grp * per, j1 = min(j0 + per, q.rows);
  if (j0 >= j1) return;
  const bool copy = a.in != a.out;
  const size_t seq = (size_t)b * a.J * a.V;

  const int lo = c * a.piece;

  // Row j: where its piece lies, and its mask.
  struct Row {
    const RT* in;
    RT* out;
    int head, from, to, start, units;
    const uint32_t* mask;
    bool bad;
  };
  auto place = [&](int j) {
    Row r;
    const size_t base = seq + (size_t)j * a.V;
    r.in = reinterpret_cast<const RT*>(a.in) + base;
    r.out = reinterpret_cast<RT*>(a.out) + base;
    r.head = a.wide ? min(a.V, (int)((16 - (base * sizeof(RT)) % 16) % 16 / sizeof(RT))) : 0;
    r.from = c == 0 ? 0 : min(a.V, lo + r.head);
    r.to = c + 1 == a.pieces ? a.V : min(a.V, lo + a.piece + r.head);
    r.start = c == 0 ? r.head : r.from;   // the first unit; in front of it, elements of the row's head
    r.units = a.wide ? (r.to - r.start) / VEC : 0;
    return r;
  };
  auto row_of = [&](int j) {
    Row r = place(j);
    const int m = a.mask_rows ? a.mask_rows[(size_t)b * a.J + j] : -1;
    r.bad = q.bad || m < -1 || m >= a.M;
    r.mask = m >= 0 && m < a.M ? a.masks + (size_t)m * a.W : nullptr;
    return r;
  };

  // Through the tile: `rows` rows a pass, each with VEC elements in front of its
  // first unit (for its head) and as many behind its last.
  const bool lists = LISTS && (q.held || q.nd || (a.NB && !q.bad));
  const int upr = a.piece / VEC, rows = min(a.tile_rows, j1 - j0), stride = a.piece + 2 * VEC;
  uint4 nv[PR_UNITS];
  auto load = [&](int j) {
#pragma unroll
    for (int k = 0; k < PR_UNITS; ++k) {
      const int f = tid + k * PR_NT, rr = rows > 1 ? f / upr : 0, u = f - rr * upr;
      nv[k] = make_uint4(0, 0, 0, 0);
      if (rr < rows && j + rr < j1) {
        const Row r = place(j + rr);
        if (u < r.units) nv[k] = load_stream(r.in + (r.start + u * VEC));
      }
    }
  };
  if (copy && lists) load(j0);   // while the lists are read

  // Touched ids of [lo, hi): the piece, and the VEC elements behind it that a row's head may add.
  const int hi = c + 1 == a.pieces ? a.V : min(a.V, lo + a.piece + VEC);
  int2* entries = reinterpret_cast<int2*>(smem);   // (id, count word), other than the specials
  Specials sp;
  int ne = 0, listed = 0;
  bool kept = true;
  if (lists) {
    // The first ids and their counts are under way while the names are sorted out.
    int v[PR_UNITS];
    uint32_t word[PR_UNITS];
    auto ids = [&](int i0) {
#pragma unroll
      for (int k = 0; k < PR_UNITS; ++k) v[k] = i0 + k * PR_NT < q.held ? q.ids[i0 + k * PR_NT] : -1;
#pragma unroll
      for (int k = 0; k < PR_UNITS; ++k) word[k] = v[k] >= lo && v[k] < hi ? q.counts[v[k]] : 0u;
    };
    ids(tid);
    if (tid == 0) s_listed = 0;
    ne = sp.build(smem + PR_ENTRIES * sizeof(int2), &s_special, a.drafts + (size_t)b * a.draft_stride, q.nd,
                  a.bias_ids + (size_t)b * a.NB, a.bias_vals + (size_t)b * a.NB, a.NB, a.hmask, lo, hi);
    __syncthreads();
    for (int i = tid;;) {
#pragma unroll
      for (int k = 0; k < PR_UNITS; ++k) {
        if (v[k] < lo || v[k] >= hi || (ne && sp.find(v[k]) >= 0)) continue;
        const int at = atomicAdd(&s_listed, 1);
        if (at < PR_ENTRIES) entries[at] = make_int2(v[k], (int)word[k]);
      }
      if ((i += PR_TILE) >= q.held) break;
      ids(i);
    }
    __syncthreads();
    kept = s_listed <= PR_ENTRIES;
    listed = kept ? s_listed : q.held;
  }
  const bool tile = LISTS && copy && (ne || listed);

  auto allowed = [&](const uint32_t* mask, int v) { return !mask || (mask[v >> 5] >> (v & 31) & 1u); };
  // The i-th touched id (i < ne + listed) in [from, to), its count word and its names; or -1.
  auto touched = [&](int i, int from, int to, uint32_t& word, Special& s) {
    int v;
    s = Special{0ull, 0.0f, 0};
    if (i < ne) {
      v = sp.id(i);
      if (v < from || v >= to) return -1;
      s = sp.entries[i];
      word = q.counts ? q.counts[v] : 0u;
    } else if (kept) {
      v = entries[i - ne].x;
      if (v < from || v >= to) return -1;
      word = (uint32_t)entries[i - ne].y;
    } else {
      v = q.ids[i - ne];
      if (v < from || v >= to || (ne && sp.find(v) >= 0)) return -1;
      word = q.counts[v];
    }
    return v;
  };
  auto fill_nan = [&](const Row& r) {
    for (int e = r.from + tid; e < r.to; e += PR_NT) r.out[e] = Elem<ET>::QNAN;
  };

  if (!tile) {
    for (int j = j0; j < j1; ++j) {
      const Row r = row_of(j);
      if (r.bad) {
        fill_nan(r);
        continue;
      }
      if (copy || r.mask) {
        for (int u = tid; u < r.units; u += PR_TILE) {
          uint4 v[PR_UNITS];
          uint32_t ok[PR_UNITS];
#pragma unroll
          for (int k = 0; k < PR_UNITS; ++k) {
            const int e = r.start + (u + k * PR_NT) * VEC;
            ok[k] = u + k * PR_NT < r.units ? r.mask ? mask_word(r.mask, a.W, e) & ALL : ALL : 0u;
            v[k] = make_uint4(0, 0, 0, 0);
            if (ok[k] && (copy || ok[k] != ALL)) v[k] = *reinterpret_cast<const uint4*>(r.in + e);
          }
#pragma unroll
          for (int k = 0; k < PR_UNITS; ++k) {
            RT* o = r.out + (r.start + (u + k * PR_NT) * VEC);
            if (u + k * PR_NT >= r.units || !(copy || ok[k] != ALL)) continue;
            if (copy) store_stream(o, Elem<ET>::mask(v[k], ok[k]));
            else *reinterpret_cast<uint4*>(o) = Elem<ET>::mask(v[k], ok[k]);
          }
        }
        const int tail = r.start + r.units * VEC, before = r.start - r.from;
        for (int i = tid; i < before + (r.to - tail); i += PR_NT) {
          const int e = i < before ? r.from + i : tail + (i - before);
          const bool ok = allowed(r.mask, e);
          if (!ok || copy) r.out[e] = ok ? r.in[e] : (RT)Elem<ET>::NEG_INF;
        }
      }
    }
    if (!LISTS || copy || !(ne || listed)) return;
    __syncthreads();   // in place: the touched values, which the masks left as they were
    for (int j = j0; j < j1; ++j) {
      const Row r = row_of(j);
      if (r.bad) continue;
      for (int i = tid; i < ne + listed; i += PR_NT) {
        uint32_t word;
        Special s;
        const int v = touched(i, r.from, r.to, word, s);
        if (v >= 0 && allowed(r.mask, v))
          touch(reinterpret_cast<const ET*>(r.in) + v, reinterpret_cast<ET*>(r.out) + v, word, s, a.first, j, q.p);
      }
    }
    return;
  }

  ET* buf = reinterpret_cast<ET*>(smem + a.tile_off);
  for (int j = j0; j < j1; j += rows) {
    const int n = min(rows, j1 - j);
#pragma unroll
    for (int k = 0; k < PR_UNITS; ++k) {
      const int f = tid + k * PR_NT, rr = rows > 1 ? f / upr : 0, u = f - rr * upr;
      // (Only the row's units: what lies behind them in the tile are elements that other lanes write below.)
      if (rr < n && u < place(j + rr).units) *reinterpret_cast<uint4*>(buf + (rr * stride + VEC + u * VEC)) = nv[k];
    }
    for (int rr = 0; rr < n; ++rr) {
      const Row r = row_of(j + rr);
      if (r.bad) continue;
      const int tail = r.start + r.units * VEC, before = r.start - r.from;
      for (int i = tid; i < before + (r.to - tail); i += PR_NT) {
        const int e = i < before ? r.from + i : tail + (i - before);
        reinterpret_cast<RT*>(buf)[rr * stride + VEC + (e - r.start)] = r.in[e];
      }
    }
    __syncthreads();
    if (j + rows < j1) load(j + rows);
    for (int rr = 0; rr < n; ++rr) {
      const Row r = row_of(j + rr);
      for (int i = tid; i < ne + listed; i += PR_NT) {
        uint32_t word;
        Special s;
        const int v = touched(i, r.from, r.to, word, s);
        ET* z = buf + (rr * stride + VEC + (v - r.start));
        if (v >= 0) touch(z, z, word, s, a.first, j + rr, q.p);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PR_UNITS; ++k) {
      const int f = tid + k * PR_NT, rr = rows > 1 ? f / upr : 0, u = f - rr * upr;
      if (rr >= n) continue;
      const Row r = row_of(j + rr);
      if (r.bad || u >= r.units) continue;
      const int e = r.start + u * VEC;
      const uint4 v = *reinterpret_cast<const uint4*>(buf + (rr * stride + VEC + u * VEC));
      store_stream(r.out + e, Elem<ET>::mask(v, r.mask ? mask_word(r.mask, a.W, e) & ALL : ALL));
    }
    for (int rr = 0; rr < n; ++rr) {
      const Row r = row_of(j + rr);
      if (r.bad) {
        fill_nan(r);
        continue;
      }
      const int tail = r.start + r.units * VEC, before = r.start - r.from;
      for (int i = tid; i < before + (r.to - tail); i += PR_NT) {
        const int e = i < before ? r.from + i : tail + (i - before);
        r.out[e] = allowed(r.mask, e) ? reinterpret_cast<const RT*>(buf)[rr * stride + VEC + (e - r.start)] : (RT)Elem<ET>::NEG_INF;
      }
    }
    // The next rows' units lie otherwise: nobody may fill the tile while another lane still reads these.
    if (j + rows < j1) __syncthreads();
  }
}

// In place, without masks: one workgroup per (sequence, share of the lists,
// group of rows); a lane takes a listed id of a row.
template <typename ET>
__global__ __launch_bounds__(PR_NT) void process_lists_kernel(ProcessArgs a) {
  typedef typename Raw<ET>::type RT;
  extern __shared__ __align__(16) char smem[];
  __shared__ int s_count;
  const int tid = threadIdx.x;
  const int c = (int)(blockIdx.x % (unsigned)a.pieces);
  const int rest = (int)(blockIdx.x / (unsigned)a.pieces);
  const int grp = rest % a.groups, b = rest / a.groups;
  const Sequence q = sequence(a, b);
  const int per = (a.J + a.groups - 1) / a.groups;
  const int j0 = grp * per, nj = min(j0 + per, q.rows) - j0;
  if (nj <= 0) return;
  ET* z = reinterpret_cast<ET*>(a.out) + ((size_t)b * a.J + j0) * a.V;
  if (q.bad) {
    RT* o = reinterpret_cast<RT*>(z);
    for (size_t e = (size_t)c * PR_NT + tid; e < (size_t)nj * a.V; e += (size_t)PR_NT * a.pieces) o[e] = Elem<ET>::QNAN;
    return;
  }
  Specials sp;
  const int ne = sp.build(smem, &s_count, a.drafts + (size_t)b * a.draft_stride, q.nd, a.bias_ids + (size_t)b * a.NB,
                          a.bias_vals + (size_t)b * a.NB, a.NB, a.hmask, 0, a.V);
  const Special none = {0ull, 0.0f, 0};
  for (int r0 = 0; r0 < nj; r0 += 16) {   // 16 rows at a time: the items fit 32 bits
    const unsigned m = (unsigned)min(16, nj - r0);
    // (The table's order differs between workgroups: they share its ids out by their values.)
    for (unsigned i = tid; i < ne * m; i += PR_NT) {
      const int e = (int)(i / m), j = r0 + (int)(i % m), v = sp.id(e);
      if (v % a.pieces != c) continue;
      ET* at = z + (size_t)j * a.V + v;
      touch(at, at, q.counts ? q.counts[v] : 0u, sp.entries[e], a.first, j0 + j, q.p);
    }
    for (unsigned i = c * PR_NT + tid; i < q.held * m; i += PR_NT * a.pieces) {
      const int j = r0 + (int)(i % m), v = q.ids[i / m];
      if (v < 0 || v >= a.V || (ne && sp.find(v) >= 0)) continue;
      ET* at = z + (size_t)j * a.V + v;
      touch(at, at, q.counts[v], none, a.first, j0 + j, q.p);
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

// Both history kernels are a few dependent memory accesses long: append takes
// 3.1 us for 256 x 8 tokens and 3.9 us for 8 x 4096, reset 2.7 us for 256 slots
// of 500 tokens and 5 us for 8 of 3000, less than it takes to launch them.

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
