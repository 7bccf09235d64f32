// Drawing one token per row of logits: temperature, top-k, top-p and min-p,
// from a given uniform number (beside greedy and typical acceptance, whose next
// token is the argmax).  For a row x with maximum m:
//   w_v = exp((x_v - m) / temperature);
//   order the tokens by (larger x, lower index) and keep the shortest of
//     the first top_k,
//     those with (mass of the tokens before) < top_p * (mass of the first top_k),
//     those with w_v >= min_p   (the first token always);
//   the token is the first in vocab order at which the kept mass exceeds
//   u * (whole kept mass).
// Every filter keeps a prefix of that order, so together they are one cut: a
// value, how many tokens equal to it stay (the lowest indices), and a smallest
// value for min-p.
//
// A cluster of CTAs holds a row in shared memory: the logits are read from memory
// once (by every pass, where a slice does not fit).  Weights are integers (2^44 for
// the maximum), so every sum is the same in any order; each is good to about 1e-9 of
// itself (the exponent as a sum of two floats, a 128-entry table, a short polynomial)
// before it is cut to a whole number, which costs up to 2^-44 of the maximum.  That
// matters because a draw compares u against up to 10^5 borders: with weights good to
// 6e-8 about one row in a thousand of a flat distribution would draw a neighbour of
// the token that its definition gives; and with 32 bits a cut by top_p near 1 missed
// a long flat tail altogether.
// The cut is found by a histogram of counts and masses over 64 bins of
// (m - x) / temperature, half a power of two each, and then among the tokens of
// the one bin that the cut falls in: by histograms over their keys, 6 bits at a
// time, until at most 128 are left, which are ranked, or a single value.  A
// histogram is kept a column per lane, so that 32 lanes never meet in a bank.
// The CTAs meet in distributed shared memory: each reads all sums and lists and
// searches by itself, so a pass costs one cluster barrier.
//
// What it costs (cycles of one of two CTAs of an SM with 32k tokens of bf16): 9k for
// the load, 5k for a histogram of counts, 17k with masses, 7k to 16k for a pass over
// the tokens of a bin, 5k for a meeting of the cluster with its search, 12k to 16k
// for the last pass over the weights, 8k for the walk to the token; few rows are
// bound by the chain of meetings, many by the instructions.  The weights are worked
// out two at a time, in instructions for pairs.
// One row of 32000 fp32 logits: 14.2 us.  64 rows of 128000 bf16 logits with
// parameters of their own: 57 us, which is the longest row's chain of passes.  256
// rows of 32000 fp16 logits without filters: 19.8 us.
#include <cooperative_groups.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "serve.cuh"

namespace cg = cooperative_groups;

namespace mt {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 64;           // 6 bits a pass
constexpr int kList = 128;          // tokens that are ranked directly, four threads each
constexpr int kMaxCluster = 8;
constexpr int kWBits = 44;          // weight of the maximum: 2^44 * kSampleMaxVocab < 2^63

// Monotone 32-bit key of a float (-0 as +0).
__device__ __forceinline__ uint32_t ord_of(float v) {
  const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_ord(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// Low key bits that are the same for every value of a 16-bit type.
template <typename T> struct KeyShift { static constexpr int v = 0; };
template <> struct KeyShift<__half> { static constexpr int v = 13; };
template <> struct KeyShift<__nv_bfloat16> { static constexpr int v = 16; };

// The value of a shifted key.
template <int KS>
__device__ __forceinline__ float value_of_key(uint32_t key) {
  const uint32_t o = key << KS;
  return of_ord((o & 0x80000000u) ? o : o | ((1u << KS) - 1u));
}

struct Scale {
  float m;         // the row's maximum
  float ref;       // what the weights refer to: m, or a little more (reference below)
  float hi, lo;    // log2(e) / temperature as a sum
};

// For 16-bit values: their maximum m, unless it is so much smaller than the values that
// matter (|x| up to |m| + 31 t: weights above 2^-44) that 24 bits do not hold every x - m,
// as with log-probabilities of a nearly certain token.  Then 0, or for m > 0 a power of
// two of at least m and at most 0.016 t: within 2^13 of all of those, so that a difference
// is exact where |x| is the larger, as it is with m otherwise.
__device__ __forceinline__ float reference(float m, float t) {
  const float r = t * (31.f / 4095.f);
  if (!(fabsf(m) < r) || !(r < 1e30f)) return m;
  return m > 0.f ? __uint_as_float((__float_as_uint(r) + 0x7fffffu) & 0xff800000u) : 0.f;
}

constexpr unsigned kTable = 128;

struct Table {  // entry k: 2^(30 + (127 - k)/128)
  int v[kTable];
};

// floor(2^64 f) for f in [0, 1): exact but for bits below 2^-64.
__device__ __forceinline__ unsigned long long fraction64(float f) {
  const uint32_t b = __float_as_uint(f);
  const int up = (int)(b >> 23) - 127 + 41;  // the 24-bit significand's place
  const unsigned long long m = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
  return up >= 0 ? m << up : up > -24 ? m >> -up : 0ull;
}

// Two fp32 in one register pair, for the instructions that take both at once.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2_of(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2_of(float a) { return f2_of(a, a); }
__device__ __forceinline__ float f2_get(F2 x, int i) { return __uint_as_float((uint32_t)(i ? x >> 32 : x)); }
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 f2_sub(F2 a, F2 b) { return f2_fma(b, f2_of(-1.f), a); }

// Weights of two values: 2^44 exp((x - ref) / t), cut to a whole number.
// 2^e with e = n/128 + r, |r| <= 1/256:  2^(30 + (n mod 128)/128) * (1 + q) *
// 2^(n div 128 - 30), q = 2^r - 1.  -n (>= 0) is read off the low bits of
// -e * 128 + 1.5 * 2^23; with 127 added, its low 7 bits are the table's index and the
// others the shift.  The product with q is a 32-bit high product of the table's
// 2^30 .. 2^31 and q * 2^32 (the only conversion).  -inf shifts everything out.
// TWO: the rounding error of x - ref by the form for any two floats; 16-bit values
// need only the form for |x| <= |ref|, because elsewhere their difference is exact.
template <bool TWO>
__device__ __forceinline__ void weights(float x0, float x1, const Scale& s, const int* table, unsigned long long (&w)[2]) {
  const F2 x = f2_of(x0, x1), m = f2_of(s.ref), hi = f2_of(s.hi);
  F2 d = f2_sub(x, m);
  d = f2_of(fminf(f2_get(d, 0), 0.f), fminf(f2_get(d, 1), 0.f));  // 0 for x = m = +inf, too
  const F2 minus_p = f2_mul(d, f2_of(-s.hi));
  F2 err;
  if (TWO) {
    const F2 bb = f2_sub(d, x);
    err = f2_add(f2_sub(x, f2_sub(d, bb)), f2_sub(f2_of(-s.ref), bb));
  } else {
    err = f2_sub(x, f2_add(d, m));
  }
  const F2 e = f2_add(f2_fma(d, hi, minus_p), f2_fma(d, f2_of(s.lo), f2_mul(err, hi)));
  const F2 z = f2_fma(minus_p, f2_of(128.f), f2_of(12582912.f));
  const F2 minus_r = f2_fma(f2_add(z, f2_of(-12582912.f)), f2_of(-0.0078125f), minus_p);
  const F2 r = f2_sub(e, minus_r);
  constexpr float k32 = 4294967296.f;
  F2 q = f2_fma(r, f2_of(5.5504109e-2f * k32), f2_of(2.4022651e-1f * k32));  // ln2^3/6, ln2^2/2
  q = f2_mul(f2_fma(r, q, f2_of(6.9314718e-1f * k32)), r);                   // ln2
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const unsigned n = __float_as_uint(f2_get(z, i)) - (0x4B400000u - (kTable - 1));
    const int t = table[n & (kTable - 1)];
    const unsigned v = (unsigned)(t + __mulhi(t, __float2int_rn(f2_get(q, i))));
    w[i] = ((unsigned long long)v << (kWBits - 30)) >> min(n / kTable, 63u);
  }
}
template <bool TWO>
__device__ __forceinline__ unsigned long long weight(float x, const Scale& s, const int* table) {
  unsigned long long w[2];
  weights<TWO>(x, x, s, table, w);
  return w[0];
}

// A histogram: counts, and the sums of the low 21 bits of the weights and of what is
// above them, a column per lane.  A column has at most 2^11 tokens, so neither sum
// overflows where a weight is below 2^42; the larger ones, of the first kCoarse bins of
// (m - x) / temperature, are added in units of 8, 2^-38 of themselves.  (Sums of 64 bits
// took 59 us for 60 of 128k bf16 tokens with top-p 0.9 where these take 56.)
constexpr int kCoarse = 5;
struct Hist {
  unsigned cnt[kBins][32], lo[kBins][32], hi[kBins][32];
};

struct Found {  // a bin of a histogram of the whole cluster
  unsigned in;              // tokens in the bin
  unsigned cnt;             // tokens before it
  unsigned long long mass;  // their mass
  unsigned long long own;   // the bin's
};

struct Cut {  // the last token that is kept
  uint32_t key;             // its shifted key
  int idx;                  // its index, or -1: the first `stay` tokens of that key
  unsigned stay;
  unsigned long long mass;  // mass up to it
};

struct __align__(16) Smem {
  Hist hist;
  int table[kTable];
  // read by the cluster:
  unsigned long long best;
  unsigned bin_cnt[2][kBins];            // this CTA's sums of a histogram, by turns
  unsigned long long bin_mass[2][kBins];
  unsigned list_n[2];                    // this CTA's tokens of a range, one list for each cut
  uint32_t list_key[2][kList];
  int list_idx[2][kList];
  unsigned long long tot_mass;           // this CTA's kept mass and tokens equal to the cut
  unsigned tot_ties;
  // this CTA's own:
  unsigned long long key[kWarps];
  unsigned part_cnt[kMaxCluster][kBins];
  unsigned long long part_mass[kMaxCluster][kBins];
  Found bins[kBins];
  unsigned long long unit[kBins];        // a token's mass, where a bin is one value
  unsigned long long whole;
  unsigned long long rank_key[kList], rank_mass[kList];
  Cut cut;
  unsigned long long run_mass[kWarps];
  unsigned run_ties[kWarps];
  double ln_min_p;
  float x_min;
};

// NaN as -inf, in a packed vector.
template <typename T>
__device__ __forceinline__ uint4 no_nan(uint4 r) {
  if constexpr (sizeof(T) == 4) {
    float v[4];
    memcpy(v, &r, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = fmaxf(v[e], -INFINITY);
    memcpy(&r, v, 16);
  } else if constexpr (std::is_same<T, __half>::value) {
    __half2 v[4];
    memcpy(v, &r, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __hmax2(v[e], __half2half2(__ushort_as_half(0xfc00)));
    memcpy(&r, v, 16);
  } else {
    __nv_bfloat162 v[4];
    memcpy(v, &r, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __hmax2(v[e], __bfloat162bfloat162(__ushort_as_bfloat16(0xff80)));
    memcpy(&r, v, 16);
  }
  return r;
}

// Largest element of a packed vector without NaN.
template <typename T>
__device__ __forceinline__ float vec_max(const uint4& r) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
  } else if constexpr (std::is_same<T, __half>::value) {
    __half2 v[4];
    memcpy(v, &r, 16);
    const __half2 m = __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3]));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    __nv_bfloat162 v[4];
    memcpy(v, &r, 16);
    const __nv_bfloat162 m = __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
}

// A CTA's part of a row, staged in shared memory by the first pass over it (or,
// where it does not fit, read again by every pass).  Warp w holds a contiguous
// run of 16-byte vectors and lane l a contiguous part of it, so that sums by lane
// are sums in vocab order.  NaN counts as -inf, and so do the places of a ragged
// first or last vector that lie outside the row.
template <typename T, bool STAGED>
struct Slice {
  static constexpr int EPV = 16 / (int)sizeof(T);
  const T* row;
  uint4* stage;
  int V, beg, end, mis;  // this CTA's vectors; vector v holds elements v * EPV - mis and on
  int per_lane;          // vectors of a lane
  int lbeg, lend;        // this lane's vectors

  __device__ __forceinline__ void init(const T* row_, int V_, uint4* stage_, unsigned rank, unsigned C) {
    row = row_;
    V = V_;
    stage = stage_;
    mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int nvec = (V + mis + EPV - 1) / EPV;
    const int per = (nvec + (int)C - 1) / (int)C;
    beg = min(nvec, (int)rank * per);
    end = min(nvec, beg + per);
    per_lane = (end - beg + kThreads - 1) / kThreads;
    lbeg = min(end, beg + (int)threadIdx.x * per_lane);
    lend = min(end, lbeg + per_lane);
  }
  __device__ __forceinline__ uint4 load(int v) const {
    const int e0 = v * EPV - mis;
    if (e0 >= 0 && e0 + EPV <= V) return no_nan<T>(__ldg(reinterpret_cast<const uint4*>(row + e0)));
    T t[EPV];
#pragma unroll
    for (int e = 0; e < EPV; ++e) {
      const int i = e0 + e;
      t[e] = i >= 0 && i < V ? row[i] : Act<T>::from_f(-INFINITY);
    }
    uint4 r;
    memcpy(&r, t, 16);
    return no_nan<T>(r);
  }
  // Where vector beg + i is staged: lanes that read their own parts (four
  // vectors each, mostly) then hit distinct banks.
  static __device__ __forceinline__ int place(int i) { return (i & ~3) | ((i & 3) ^ ((i >> 3) & 3)); }
  __device__ __forceinline__ uint4 get(int v) const { return STAGED ? stage[place(v - beg)] : load(v); }
  __device__ __forceinline__ int index(int v, int e) const { return v * EPV - mis + e; }
  __device__ __forceinline__ bool in_row(int v, int e) const { return (unsigned)index(v, e) < (unsigned)V; }
  // f(x, e) over the elements of a vector
  template <class F>
  static __device__ __forceinline__ void vec(const uint4& r, F f) {
    T t[EPV];
    memcpy(t, &r, 16);
#pragma unroll
    for (int e = 0; e < EPV; ++e) f(Act<T>::to_f(t[e]), e);
  }
  // f(x0, x1, v, e) over the pairs of elements (e and e + 1) of this lane's vectors;
  // vectors whose elements are all below `least` may be left out.  Those that reach
  // out of the row go to g(x, v, e) instead, element by element, without what lies
  // outside.
  template <class F, class G>
  __device__ __forceinline__ void pairs(float least, F f, G g) const {
#pragma unroll 1
    for (int v = lbeg; v < lend; ++v) {
      const uint4 r = get(v);
      if (vec_max<T>(r) < least) continue;
      if (index(v, 0) >= 0 && index(v, EPV) <= V) {
        T t[EPV];
        memcpy(t, &r, 16);
#pragma unroll
        for (int e = 0; e < EPV; e += 2) f(Act<T>::to_f(t[e]), Act<T>::to_f(t[e + 1]), v, e);
      } else {
#pragma unroll 1
        for (int e = 0; e < EPV; ++e)
          if (in_row(v, e)) g(fmaxf(Act<T>::to_f(row[index(v, e)]), -INFINITY), v, e);
      }
    }
  }
  // f(x, v, e) over this lane's elements; vectors whose elements are all below
  // `least` may be left out
  template <class F>
  __device__ __forceinline__ void each(float least, F f) const {
#pragma unroll 1
    for (int v = lbeg; v < lend; ++v) {
      const uint4 r = get(v);
      if (!(vec_max<T>(r) < least)) vec(r, [&](float x, int e) { f(x, v, e); });
    }
  }
  // The first pass, in whole lines: the row into shared memory; the largest value
  // and its lowest index (a thread's indices rise) as a key, 0 where there is
  // nothing above -inf.
  __device__ __forceinline__ unsigned long long first() const {
    constexpr int U = 4;  // vectors in flight
    float best = -INFINITY;
    int bi = 0;
#pragma unroll 1
    for (int v0 = beg + (int)threadIdx.x; v0 < end; v0 += U * kThreads) {
      uint4 r[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (v0 + j * kThreads < end) r[j] = load(v0 + j * kThreads);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int v = v0 + j * kThreads;
        if (v >= end) continue;
        if (STAGED) stage[place(v - beg)] = r[j];
        const float m = vec_max<T>(r[j]);
        if (m > best) {  // then search the vector
          T t[EPV];
          memcpy(t, &r[j], 16);
#pragma unroll
          for (int e = EPV - 1; e >= 0; --e)
            if (Act<T>::to_f(t[e]) == m) bi = index(v, e);
          best = m;
        }
      }
    }
    return best > -INFINITY ? ((unsigned long long)ord_of(best) << 32) | (0xffffffffu - (unsigned)bi) : 0ull;
  }
};

__device__ __forceinline__ unsigned long long shfl_up64(unsigned long long v, int o) {
  return __shfl_up_sync(0xffffffffu, v, o);
}

__device__ __forceinline__ void clear(Hist& h) {
  uint4* p = reinterpret_cast<uint4*>(&h);
  for (int i = threadIdx.x; i < (int)(sizeof(Hist) / 16); i += kThreads) p[i] = make_uint4(0, 0, 0, 0);
}

// The cluster's histogram in sm.bins, each bin with what lies before it (base_cnt
// and base_mass included).  The histogram is left zero; turn: which of the two
// places the sums pass through; coarse: how many bins' masses are in units of 8; units:
// the masses are counts times sm.unit.
__device__ __noinline__ void meet(Smem& sm, int turn, unsigned base_cnt, unsigned long long base_mass, int coarse, bool units) {
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, C = (int)cl.num_blocks();
  __syncthreads();
  {  // eight threads a bin, four columns each
    const int b = tid >> 3, c = tid & 7;
    unsigned n = 0;
    unsigned long long m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      n += sm.hist.cnt[b][c + 8 * j];
      m += sm.hist.lo[b][c + 8 * j] + ((unsigned long long)sm.hist.hi[b][c + 8 * j] << 21);
      sm.hist.cnt[b][c + 8 * j] = sm.hist.lo[b][c + 8 * j] = sm.hist.hi[b][c + 8 * j] = 0;
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      n += __shfl_xor_sync(0xffffffffu, n, o);
      m += __shfl_xor_sync(0xffffffffu, m, o);
    }
    if (c == 0) {
      sm.bin_cnt[turn][b] = n;
      sm.bin_mass[turn][b] = units ? n * sm.unit[b] : b < coarse ? m << 3 : m;
    }
  }
  cl.sync();
  const int r = tid / kBins, b = tid % kBins;  // a thread per CTA and bin
  if (r < C) {
    const Smem* p = cl.map_shared_rank(&sm, r);
    sm.part_cnt[r][b] = p->bin_cnt[turn][b];
    sm.part_mass[r][b] = p->bin_mass[turn][b];
  }
  __syncthreads();
  if (tid < 32) {  // two bins a lane
    unsigned n[2] = {0, 0};
    unsigned long long m[2] = {0, 0};
    for (int q = 0; q < C; ++q)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        n[j] += sm.part_cnt[q][2 * lane + j];
        m[j] += sm.part_mass[q][2 * lane + j];
      }
    unsigned ni = n[0] + n[1];
    unsigned long long mi = m[0] + m[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, ni, o);
      const unsigned long long y = shfl_up64(mi, o);
      if (lane >= o) {
        ni += x;
        mi += y;
      }
    }
    ni += base_cnt;
    mi += base_mass;
    sm.bins[2 * lane] = Found{n[0], ni - n[0] - n[1], mi - m[0] - m[1], m[0]};
    sm.bins[2 * lane + 1] = Found{n[1], ni - n[1], mi - m[1], m[1]};
    if (lane == 31) sm.whole = mi;
  }
  __syncthreads();
}

// The bin of sm.bins at which the running count reaches want_cnt or, where that is
// 0, the running mass want_mass; every warp for itself.
__device__ __forceinline__ int find(const Smem& sm, unsigned want_cnt, unsigned long long want_mass) {
  int at = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const Found f = sm.bins[32 * j + (threadIdx.x & 31)];
    at += __popc(__ballot_sync(0xffffffffu, want_cnt ? f.cnt + f.in < want_cnt : f.mass + f.own < want_mass));
  }
  return min(at, kBins - 1);
}

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams a, const __grid_constant__ Table table) {
  using S = Slice<T, STAGED>;
  constexpr int EPV = S::EPV;
  constexpr int KS = KeyShift<T>::v;
  constexpr bool TWO = sizeof(T) == 4;
  extern __shared__ uint4 dyn[];  // Smem, then the staged slice
  static_assert(sizeof(Smem) % 16 == 0, "the slice is aligned");
  Smem& sm = *reinterpret_cast<Smem*>(dyn);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int n = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < (int)kTable) sm.table[tid] = table.v[tid];
  if (tid < 2) sm.list_n[tid] = 0;
  clear(sm.hist);
  pdl_wait();
  const int src = a.row_index ? a.row_index[n] : n;
  if (src < 0 || src >= a.rows) {  // the same for the whole cluster
    if (src >= a.rows && rank == 0 && tid == 0) a.tokens[n] = -1;
    return;
  }
  const float temp = a.temperature ? a.temperature[n] : 1.f;
  int want_k = a.top_k ? a.top_k[n] : 0;
  const float top_p = a.top_p ? a.top_p[n] : 1.f;
  const float min_p = a.min_p ? a.min_p[n] : 0.f;
  const float u = a.uniforms[n];
  if (min_p > 1.f) want_k = 1;  // no weight reaches it: the first token alone
  // the one thing that takes 64-bit floats (two results a clock and SM), by one thread
  if (tid == 0) sm.ln_min_p = min_p > 0.f ? log((double)min_p) : 0.0;

  S s;
  s.init(static_cast<const T*>(a.logits) + src * a.row_stride, a.V, dyn + sizeof(Smem) / 16, (unsigned)rank, (unsigned)C);

  // ---- maximum and its lowest index ----
  {
    unsigned long long key = s.first();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
      key = k > key ? k : key;
    }
    if (lane == 0) sm.key[warp] = key;
    __syncthreads();
    if (warp == 0) {
      key = lane < kWarps ? sm.key[lane] : 0ull;
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) {
        const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
        key = k > key ? k : key;
      }
      if (lane == 0) sm.best = key;
    }
  }
  cl.sync();
  unsigned long long best = lane < C ? cl.map_shared_rank(&sm, lane)->best : 0ull;
#pragma unroll
  for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
    const unsigned long long k = __shfl_xor_sync(0xffffffffu, best, o);
    best = k > best ? k : best;
  }
  best = __shfl_sync(0xffffffffu, best, 0);
  if (!(temp > 0.f) || best == 0ull) {  // greedy, or a row of nothing but -inf
    if (rank == 0 && tid == 0) a.tokens[n] = best == 0ull ? -1 : (int)(0xffffffffu - (unsigned)best);
    cl.sync();  // no CTA leaves while others read it
    return;
  }
  Scale sc;
  sc.m = of_ord((uint32_t)(best >> 32));
  sc.ref = TWO ? sc.m : reference(sc.m, temp);
  {
    // log2(e) / t as the sum of two floats
    const float h = 1.44269502f, l = 1.92596303e-8f;  // log2(e)
    sc.hi = h / temp;
    sc.lo = (fmaf(-sc.hi, temp, h) + l) / temp;
    if (!(sc.hi < 1e30f)) {
      sc.hi = 1e30f;
      sc.lo = 0.f;
    }
  }
  // smallest value that min-p keeps: x >= m + t ln(min_p), the next float up
  if (tid == 0)
    sm.x_min = min_p > 0.f ? fminf(__double2float_ru((double)sc.m + (double)temp * sm.ln_min_p), sc.m) : -INFINITY;

  // ---- the cut ----
  const bool use_k = want_k > 0 && want_k < a.V, use_p = top_p < 1.f;
  Cut cut{0u, -1, 0u, 0ull};
  if (use_k || use_p) {
    const float width = sc.hi * 2.f;
    auto bin_of = [&](float x) {  // rounded, so that no conversion is needed; it never falls as x falls
      const float z = fminf((sc.m - x) * width, (float)(kBins - 1)) + 12582912.f;
      return x == sc.m ? 0 : __float_as_int(z) - 0x4B400000;
    };
    // a weight as the histograms hold it; coarse: its token's bin is one of the first
    auto weight_of = [&](float x, bool coarse) {
      const unsigned long long w = weight<TWO>(x, sc, sm.table);
      return coarse ? w & ~7ull : w;
    };
    auto add_mass = [&](int b, unsigned long long w, bool coarse) {
      w >>= coarse ? 3 : 0;
      atomicAdd(&sm.hist.lo[b][lane], (unsigned)w & 0x1fffffu);
      atomicAdd(&sm.hist.hi[b][lane], (unsigned)(w >> 21));
    };
    auto add = [&](int b, float x, bool coarse) {
      atomicAdd(&sm.hist.cnt[b][lane], 1u);
      if (use_p) add_mass(b, weight<TWO>(x, sc, sm.table), coarse);
    };
    auto add_one = [&](float x, int, int) {
      const int b = bin_of(x);
      add(b, x, b < kCoarse);
    };
    if (use_p) {
      s.pairs(-INFINITY, [&](float x0, float x1, int, int) {
        const int b0 = bin_of(x0), b1 = bin_of(x1);
        unsigned long long w[2];
        weights<TWO>(x0, x1, sc, sm.table, w);
        atomicAdd(&sm.hist.cnt[b0][lane], 1u);
        add_mass(b0, w[0], b0 < kCoarse);
        atomicAdd(&sm.hist.cnt[b1][lane], 1u);
        add_mass(b1, w[1], b1 < kCoarse);
      }, add_one);
    } else {
      s.pairs(-INFINITY, [&](float x0, float x1, int, int) {
        atomicAdd(&sm.hist.cnt[bin_of(x0)][lane], 1u);
        atomicAdd(&sm.hist.cnt[bin_of(x1)][lane], 1u);
      }, add_one);
    }
    int turn = 0;
    meet(sm, turn, 0u, 0ull, kCoarse, false);
    unsigned long long whole = sm.whole;
    const int bin_k = use_k ? find(sm, (unsigned)want_k, 0ull) : 0;
    Found in_k = sm.bins[bin_k];
    // sm.bins is written again by the first cut's passes: what the second may need
    // of it is kept by each warp, two bins a lane
    const Found mine0 = sm.bins[lane], mine1 = sm.bins[32 + lane];
    __syncthreads();

    // from the bin that a count or mass falls in to the last token kept
    auto refine = [&](int bin, Found f, int which, unsigned want_cnt, unsigned long long want_mass) {
      const bool coarse = bin < kCoarse;
      // the bin's keys, with room for rounding on both sides
      const float xh = sc.m - ((float)bin - 0.5f) / width, xl = sc.m - ((float)bin + 0.5f) / width;
      uint32_t hi = bin == 0 ? 0xffffffffu >> KS : ord_of(xh + 1e-5f * (fabsf(sc.m) + fabsf(xh)) + 1e-30f) >> KS;
      uint32_t lo = bin == kBins - 1 ? 0u : ord_of(xl - 1e-5f * (fabsf(sc.m) + fabsf(xl)) - 1e-30f) >> KS;
      if (!(fabsf(sc.m) < INFINITY)) {
        hi = 0xffffffffu >> KS;
        lo = 0;
      }
      hi = min(hi, (uint32_t)(best >> 32) >> KS);
      for (int pass = 0; pass < 7; ++pass) {  // 6 of at most 32 bits each, then one value or a list
        // whole vectors below the range are passed over (keys below -inf's are no numbers)
        const float least = lo <= ord_of(-INFINITY) >> KS ? -INFINITY : value_of_key<KS>(lo), most = value_of_key<KS>(hi);
        if (f.in <= kList) {
          // few tokens: listed, and ranked by (key, lower index) by four threads each
          s.each(least, [&](float x, int v, int e) {
            if (x < least || x > most || bin_of(x) != bin || !s.in_row(v, e)) return;
            const uint32_t k = ord_of(x) >> KS;
            const unsigned at = atomicAdd(&sm.list_n[which], 1u);
            if (at < kList) {  // f.in says so
              sm.list_key[which][at] = k;
              sm.list_idx[which][at] = s.index(v, e);
            }
          });
          cl.sync();
          const int c = lane < C ? (int)cl.map_shared_rank(&sm, lane)->list_n[which] : 0;
          int ci = c;
#pragma unroll
          for (int o = 1; o < kMaxCluster; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, ci, o);
            if (lane >= o) ci += x;
          }
          const int total = min(__shfl_sync(0xffffffffu, ci, kMaxCluster - 1), kList);
          int from = 0;
#pragma unroll
          for (int r = 0; r < kMaxCluster - 1; ++r) from += tid >= __shfl_sync(0xffffffffu, ci, r);
          const int before = __shfl_sync(0xffffffffu, ci - c, from);  // (from < 8: lists before this thread's)
          if (tid < total) {
            const Smem* p = cl.map_shared_rank(&sm, from);
            const uint32_t k = p->list_key[which][tid - before];
            sm.rank_key[tid] = ((unsigned long long)k << 32) | (0xffffffffu - (unsigned)p->list_idx[which][tid - before]);
            sm.rank_mass[tid] = use_p ? weight_of(value_of_key<KS>(k), coarse) : 0ull;
          }
          __syncthreads();
          const int t = tid >> 2;
          const unsigned long long k = t < total ? sm.rank_key[t] : ~0ull;
          unsigned cnt = 0;
          unsigned long long m = 0;
#pragma unroll 4
          for (int j = tid & 3; j < total; j += 4) {
            const bool before = sm.rank_key[j] > k;
            cnt += before;
            m += before ? sm.rank_mass[j] : 0ull;
          }
          cnt += __shfl_xor_sync(0xffffffffu, cnt, 1);
          m += __shfl_xor_sync(0xffffffffu, m, 1);
          cnt += __shfl_xor_sync(0xffffffffu, cnt, 2);
          m += __shfl_xor_sync(0xffffffffu, m, 2);
          cnt += f.cnt;
          m += f.mass;
          if (t < total && (tid & 3) == 0) {
            const unsigned long long w = sm.rank_mass[t];
            if (want_cnt ? cnt + 1 == want_cnt : m < want_mass && want_mass <= m + w)
              sm.cut = Cut{(uint32_t)(k >> 32), (int)(0xffffffffu - (unsigned)k), 0u, m + w};
          }
          __syncthreads();
          cut = sm.cut;
          __syncthreads();
          return;
        }
        if (hi == lo) break;
        const int shift = max(0, 32 - __clz(hi - lo) - 6);
        s.each(least, [&](float x, int v, int e) {
          if (x < least || x > most || bin_of(x) != bin || !s.in_row(v, e)) return;
          const uint32_t k = ord_of(x) >> KS;
          if (shift) add((int)((hi - k) >> shift), x, coarse);
          else atomicAdd(&sm.hist.cnt[hi - k][lane], 1u);
        });
        // a bin of one value needs no masses: the rare lanes in the range would hold up
        // every warp for them (64 rows of 128k bf16, top-p 0.9: 69 -> 63 us)
        if (shift == 0 && use_p && tid < kBins) sm.unit[tid] = hi >= (unsigned)tid ? weight_of(value_of_key<KS>(hi - tid), coarse) : 0ull;
        turn ^= 1;
        meet(sm, turn, f.cnt, f.mass, coarse ? kBins : 0, shift == 0 && use_p);
        const int b = find(sm, want_cnt, want_mass);
        f = sm.bins[b];
        __syncthreads();
        hi -= (uint32_t)b << shift;
        const uint32_t span = (1u << shift) - 1u;
        lo = max(lo, hi > span ? hi - span : 0u);
      }
      // one value, of many tokens: the first `stay` of them
      const unsigned long long w = use_p ? weight_of(value_of_key<KS>(hi), coarse) : 0ull;
      const unsigned stay = want_cnt ? want_cnt - f.cnt : w ? (unsigned)((want_mass - f.mass + w - 1) / w) : f.in;
      cut = Cut{hi, -1, stay, f.mass + stay * w};
    };
    if (use_k) {
      refine(bin_k, in_k, 0, (unsigned)want_k, 0ull);
      whole = cut.mass;
    }
    if (use_p) {
      // kept: mass before < top_p * whole, a whole number's comparison with the
      // next whole number at or above the product
      unsigned long long want = 1;
      if (top_p > 0.f) {
        const unsigned long long f = fraction64(top_p);
        want = max(__umul64hi(whole, f) + (whole * f != 0), 1ull);
      }
      if (want > whole) want = whole;
      const int b = min(__popc(__ballot_sync(0xffffffffu, mine0.mass + mine0.own < want)) +
                            __popc(__ballot_sync(0xffffffffu, mine1.mass + mine1.own < want)),
                        kBins - 1);
      Found f;
      f.in = __shfl_sync(0xffffffffu, b < 32 ? mine0.in : mine1.in, b & 31);
      f.cnt = __shfl_sync(0xffffffffu, b < 32 ? mine0.cnt : mine1.cnt, b & 31);
      f.mass = __shfl_sync(0xffffffffu, b < 32 ? mine0.mass : mine1.mass, b & 31);
      f.own = __shfl_sync(0xffffffffu, b < 32 ? mine0.own : mine1.own, b & 31);
      refine(b, f, 1, 0u, want);
    }
  }
  const bool cuts = use_k || use_p;
  __syncthreads();
  const float x_min = sm.x_min;
  // the smallest value that is kept, and whether of its tokens only some are
  const float cut_x = cuts ? value_of_key<KS>(cut.key) : -INFINITY;
  const float least = fmaxf(x_min, cut_x);
  const bool some = cuts && cut_x >= x_min;
  auto kind = [&](float x, int v, int e) {  // 2: kept, 1: equal to the cut, 0: not kept
    if (x < least) return 0;
    if (x > least || !some) return 2;
    return cut.idx >= 0 ? (s.index(v, e) <= cut.idx ? 2 : 0) : s.in_row(v, e) ? 1 : 0;
  };

  // ---- kept mass of each lane's part, in vocab order; of the tokens equal to the
  // cut the first `stay` count ----
  unsigned long long lane_mass = 0;
  unsigned lane_ties = 0;
  if (!cuts && x_min == -INFINITY) {
    s.pairs(-INFINITY, [&](float x0, float x1, int, int) {
      unsigned long long w[2];
      weights<TWO>(x0, x1, sc, sm.table, w);
      lane_mass += w[0] + w[1];
    }, [&](float x, int, int) { lane_mass += weight<TWO>(x, sc, sm.table); });
  } else {
    s.pairs(least, [&](float x0, float x1, int v, int e) {
      bool in0 = x0 > least, in1 = x1 > least;
      if (x0 == least || x1 == least) {
        const int k0 = kind(x0, v, e), k1 = kind(x1, v, e + 1);
        in0 = k0 == 2;
        in1 = k1 == 2;
        lane_ties += (k0 == 1) + (k1 == 1);
      }
      if (in0 || in1) {
        unsigned long long w[2];
        weights<TWO>(x0, x1, sc, sm.table, w);
        lane_mass += (in0 ? w[0] : 0ull) + (in1 ? w[1] : 0ull);
      }
    }, [&](float x, int v, int e) {
      const int k = kind(x, v, e);
      if (k == 2) lane_mass += weight<TWO>(x, sc, sm.table);
      lane_ties += k == 1;
    });
  }
  {
    unsigned long long m = lane_mass;
    unsigned t = lane_ties;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m += __shfl_xor_sync(0xffffffffu, m, o);
      t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    if (lane == 0) {
      sm.run_mass[warp] = m;
      sm.run_ties[warp] = t;
    }
    __syncthreads();
    if (warp == 0) {
      m = lane < kWarps ? sm.run_mass[lane] : 0ull;
      t = lane < kWarps ? sm.run_ties[lane] : 0u;
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) {
        m += __shfl_xor_sync(0xffffffffu, m, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
      }
      if (lane == 0) {
        sm.tot_mass = m;
        sm.tot_ties = t;
      }
    }
  }
  cl.sync();
  // ---- the CTA, the warp, the lane and the token that the draw falls in ----
  const unsigned long long wt = cuts && cut.idx < 0 ? weight<TWO>(value_of_key<KS>(cut.key), sc, sm.table) : 0ull;
  // From each lane's (mass, ties) to running values: `run` and `ties` become what
  // lies before the lane (added to base_*), and the lane's mass with its share of
  // the ties is returned.
  auto running = [&](unsigned long long m, unsigned t, unsigned long long base_mass, unsigned base_ties,
                     unsigned long long& run, unsigned& ties) {
    unsigned ti = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, ti, o);
      if (lane >= o) ti += x;
    }
    ties = base_ties + ti - t;
    m += (ties >= cut.stay ? 0u : min(t, cut.stay - ties)) * wt;
    unsigned long long mi = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = shfl_up64(mi, o);
      if (lane >= o) mi += x;
    }
    run = base_mass + mi - m;
    return m;
  };
  unsigned long long run, m;
  unsigned ties;
  m = running(lane < C ? cl.map_shared_rank(&sm, lane)->tot_mass : 0ull,
              lane < C ? cl.map_shared_rank(&sm, lane)->tot_ties : 0u, 0ull, 0u, run, ties);
  const unsigned long long whole = __shfl_sync(0xffffffffu, run + m, 31);
  // the kept mass must exceed u * whole: a whole number at or below it
  const unsigned long long target = u >= 1.f ? whole - 1 : u > 0.f ? __umul64hi(whole, fraction64(u)) : 0ull;
  unsigned hit = __ballot_sync(0xffffffffu, run <= target && target < run + m);
  if (hit && __ffs(hit) - 1 == rank) {
    const unsigned long long cta_run = __shfl_sync(0xffffffffu, run, rank);
    const unsigned cta_ties = __shfl_sync(0xffffffffu, ties, rank);
    m = running(lane < kWarps ? sm.run_mass[lane] : 0ull, lane < kWarps ? sm.run_ties[lane] : 0u, cta_run, cta_ties, run, ties);
    hit = __ballot_sync(0xffffffffu, run <= target && target < run + m);
    if (hit && __ffs(hit) - 1 == warp) {
      const unsigned long long warp_run = __shfl_sync(0xffffffffu, run, warp);
      const unsigned warp_ties = __shfl_sync(0xffffffffu, ties, warp);
      m = running(lane_mass, lane_ties, warp_run, warp_ties, run, ties);
      hit = __ballot_sync(0xffffffffu, run <= target && target < run + m);
      if (hit) {
        // that lane's elements, 32 at a time
        const int l = __ffs(hit) - 1;
        unsigned long long r = __shfl_sync(0xffffffffu, run, l);
        unsigned t = __shfl_sync(0xffffffffu, ties, l);
        const int v0 = __shfl_sync(0xffffffffu, s.lbeg, l), v1 = __shfl_sync(0xffffffffu, s.lend, l);
        for (int v = v0; v < v1; v += 32 / EPV) {
          const int vv = v + lane / EPV, e = lane % EPV;
          unsigned long long w = 0;
          unsigned tie = 0;
          if (vv < v1) {
            const uint4 raw = s.get(vv);
            float x = 0.f;
            S::vec(raw, [&](float y, int j) {
              if (j == e) x = y;
            });
            const int k = kind(x, vv, e);
            if (k == 2) w = weight<TWO>(x, sc, sm.table);
            tie = k == 1;
          }
          m = running(w, tie, r, t, run, ties);
          hit = __ballot_sync(0xffffffffu, run <= target && target < run + m);
          if (hit) {
            if (lane == __ffs(hit) - 1) a.tokens[n] = s.index(vv, e);
            break;
          }
          r = __shfl_sync(0xffffffffu, run + m, 31);
          t = __shfl_sync(0xffffffffu, ties + tie, 31);
        }
      }
    }
  }
  cl.sync();  // no CTA leaves while others read it
}

// Largest staged slice.  Up to about 74 KB of it two CTAs fit an SM beside their Smem of
// 39 KB; above (fp32 rows of 153k to 196k tokens, 16-bit ones of twice that) one.
constexpr int kStageMax = 96 * 1024;
constexpr int kMaxDevices = 64;

Table make_table() {
  Table t;
  for (int j = 0; j < (int)kTable; ++j) t.v[kTable - 1 - j] = (int)(std::exp2(30.0 + j / 128.0) + 0.5);
  return t;
}

template <typename T, bool STAGED>
cudaError_t launch_s(const SampleParams& a, int C, size_t smem, cudaStream_t stream) {
  static std::atomic<bool> opted[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !opted[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(sample_kernel<T, STAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(Smem) + kStageMax);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) opted[dev].store(true, std::memory_order_release);
  }
  static const Table table = make_table();
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.N * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem) + smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, STAGED>, a, table);
}

// CTAs per row: enough that a lane has at most eight vectors of a slice, and, when
// rows are few, until the grid is about one resident wave (two CTAs per SM) or a
// lane has less than one vector.  One wave, because a row's chain of meetings is
// what a second wave would repeat: before the weights went in pairs, 64 rows of 128k
// bf16, top-p, took 73 us with 4 CTAs a row and 90 with 8; 256 rows of 32k fp16,
// unfiltered, 20 with 1 and 26 with 2.
template <typename T>
cudaError_t launch_t(const SampleParams& a, cudaStream_t stream) {
  constexpr int EPV = 16 / (int)sizeof(T);
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int nvec = (a.V + EPV - 1) / EPV + 1;
  int C = 1;
  while (C < kMaxCluster && (nvec / C > 8 * kThreads || (2LL * a.N * C < 3 * sms && nvec / C > kThreads))) C *= 2;
  const size_t bytes = 16 * (size_t)(((nvec + C - 1) / C + 3) / 4 * 4);  // Slice::place permutes within four
  if (bytes <= (size_t)kStageMax) return launch_s<T, true>(a, C, bytes, stream);
  return launch_s<T, false>(a, C, 0, stream);
}

}  // namespace

cudaError_t launch_sample(const SampleParams& a, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case 0: return launch_t<float>(a, stream);
    case 1: return launch_t<__half>(a, stream);
    default: return launch_t<__nv_bfloat16>(a, stream);
  }
}

}  // namespace mt
