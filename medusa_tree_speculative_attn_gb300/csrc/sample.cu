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
// A cluster of CTAs holds a row in registers: the logits are read from memory
// once.  Weights are integers (2^44 for the maximum), so every sum is exact and
// the same in any order; each weight is good to about 1e-9 of itself (the
// exponent as a sum of two floats, a 128-entry table, a short polynomial).  That
// matters because a draw compares u against up to 10^5 borders: with weights
// good to 6e-8 about one row in a thousand of a flat distribution would draw a
// neighbour of the token that its definition gives.
// The cut is found by a histogram of counts (and masses) over 512 bins of
// (m - x) / temperature, 1/16 of a power of two each, and then among the tokens
// of the one bin that the cut falls in: ranked directly if they are at most 512,
// else by histograms over their keys, 9 bits at a time, until a single value is
// left.  The CTAs meet in distributed shared memory: each reads all histograms
// and lists and searches by itself, so a pass costs one cluster barrier.
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
constexpr int kBins = kThreads;     // a thread per bin in the search
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
  float hi, lo;    // log2(e) / temperature as a sum
};

constexpr int kTable = 128;

struct Table {  // 2^(30 + j/128)
  int v[kTable];
};

// floor(2^64 f) for f in [0, 1): exact but for bits below 2^-64.
__device__ __forceinline__ unsigned long long fraction64(float f) {
  const uint32_t b = __float_as_uint(f);
  const int up = (int)(b >> 23) - 127 + 41;  // the 24-bit significand's place
  const unsigned long long m = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
  return up >= 0 ? m << up : up > -24 ? m >> -up : 0ull;
}

// Weight of x: 2^44 exp((x - m) / t), cut to a whole number.
// 2^e with e = n/128 + r, |r| <= 1/256:  table[n mod 128] * (1 + q) * 2^(n div 128),
// q = 2^r - 1.  n is read off the low bits of e * 128 + 1.5 * 2^23; the product
// with q is a 32-bit high product of the table's 2^30 .. 2^31 and q * 2^32 (the
// only conversion), and the power of two a 32-bit shift and a 64-bit product.
// TWO: the rounding error of x - m by the form for any two floats; 16-bit values
// need only the form for |x| <= |m|, because elsewhere their difference is exact.
template <bool TWO>
__device__ __forceinline__ unsigned long long weight(float x, const Scale& s, const int* table) {
  const float d = x - s.m;
  const float p = d * s.hi;
  // below one unit (-inf too); d is no number only where x = m = +inf
  if (!(p > -45.f)) return x == s.m ? 1ull << kWBits : 0ull;
  float err;
  if (TWO) {
    const float bb = d - x;
    err = (x - (d - bb)) + (-s.m - bb);
  } else {
    err = x - (d + s.m);
  }
  const float e = fmaf(d, s.hi, -p) + fmaf(d, s.lo, err * s.hi);
  const float z = fmaf(p, 128.f, 12582912.f);
  const int n = __float_as_int(z) - 0x4B400000;
  const float r = fmaf(z - 12582912.f, -0.0078125f, p) + e;
  constexpr float k32 = 4294967296.f;
  float q = fmaf(r, 5.5504109e-2f * k32, 2.4022651e-1f * k32);  // ln2^3/6, ln2^2/2
  q = fmaf(r, q, 6.9314718e-1f * k32) * r;                      // ln2
  const int t = table[n & (kTable - 1)];
  const unsigned w = (unsigned)(t + __mulhi(t, __float2int_rn(q)));
  const int up = (kWBits - 30) + (n >> 7);  // n <= 0
  return (unsigned long long)(w >> max(0, -up)) * (1u << max(0, up));
}

struct Hist {
  unsigned cnt[kBins], lo[kBins], hi[kBins];  // count; low and high 16 bits of the 32-bit weights, summed
};

constexpr int kList = kThreads;  // tokens of one bin that are ranked directly, a thread each

struct List {
  unsigned n;
  uint32_t key[kList];
  int idx[kList];
};

struct Found {  // where a search ended
  int bin;
  unsigned cnt;             // tokens before the bin
  unsigned long long mass;  // their mass (2^32 for the maximum)
};

struct Smem {
  Hist hist[3];  // the bins; two for the bin that is searched further
  int table[kTable];
  unsigned long long key[kWarps];        // block reduction of (value, index)
  unsigned long long best;               // this CTA's, read by the cluster
  unsigned wc[kWarps];                   // scans
  unsigned long long wm[kWarps];
  unsigned long long whole;
  double ln_min_p;
  float x_min;
  Found found;
  List list[2];                          // this CTA's tokens of a bin, read by the cluster
  uint32_t mkey[kList];                  // the cluster's
  int midx[kList];
  unsigned long long mw[kList];
  uint32_t cut_key;
  int cut_idx;
  unsigned long long cut_mass;
  unsigned long long run_mass[kWarps];   // each warp's kept mass and tokens equal to the cut
  unsigned run_ties[kWarps];
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
// run of 16-byte vectors, lane l every 32nd of them.  NaN counts as -inf, and so
// do the places of a ragged first or last vector that lie outside the row (an
// index outside [0, V) is never drawn: its weight is 0 and it is below every cut
// but that of a row without enough tokens above -inf, where it adds nothing).
template <typename T, bool STAGED>
struct Slice {
  static constexpr int EPV = 16 / (int)sizeof(T);
  const T* row;
  uint4* stage;
  int V, beg, mis;  // this CTA's first vector; vector v holds elements v * EPV - mis and on
  int wbeg, wend;   // this warp's vectors

  __device__ __forceinline__ void init(const T* row_, int V_, uint4* stage_, unsigned rank, unsigned C) {
    row = row_;
    V = V_;
    stage = stage_;
    mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int nvec = (V + mis + EPV - 1) / EPV;
    const int per = (nvec + (int)C - 1) / (int)C;
    beg = min(nvec, (int)rank * per);
    const int end = min(nvec, beg + per);
    const int run = ((end - beg + kWarps - 1) / kWarps + 31) / 32 * 32;
    wbeg = min(end, beg + (int)(threadIdx.x >> 5) * run);
    wend = min(end, wbeg + run);
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
  __device__ __forceinline__ uint4 get(int v) const { return STAGED ? stage[v - beg] : load(v); }
  __device__ __forceinline__ int index(int v, int e) const { return v * EPV - mis + e; }
  // f(x, e) over the elements of a vector
  template <class F>
  static __device__ __forceinline__ void vec(const uint4& r, F f) {
    T t[EPV];
    memcpy(t, &r, 16);
#pragma unroll
    for (int e = 0; e < EPV; ++e) f(Act<T>::to_f(t[e]), e);
  }
  // f(x, v, e) over this thread's elements
  template <class F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll 1
    for (int v = wbeg + (int)(threadIdx.x & 31); v < wend; v += 32) vec(get(v), [&](float x, int e) { f(x, v, e); });
  }
  // The first pass: the row into shared memory; the largest value and its
  // lowest index (a thread's indices rise) as a key, 0 where there is nothing
  // above -inf.
  __device__ __forceinline__ unsigned long long first() const {
    constexpr int U = 4;  // vectors in flight
    float best = -INFINITY;
    int bi = 0;
#pragma unroll 1
    for (int v0 = wbeg + (int)(threadIdx.x & 31); v0 < wend; v0 += U * 32) {
      uint4 r[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (v0 + j * 32 < wend) r[j] = load(v0 + j * 32);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int v = v0 + j * 32;
        if (v >= wend) continue;
        if (STAGED) stage[v - beg] = r[j];
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

// A histogram summed over the cluster, a thread per bin: the bin's count and
// mass, and what lies before it.
struct Prefix {
  unsigned cnt, before_cnt;
  unsigned long long mass, before_mass;

  __device__ void sum(Smem& sm, int buf, cg::cluster_group& cl, unsigned base_cnt, unsigned long long base_mass) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cnt = 0;
    mass = 0;
#pragma unroll 4
    for (unsigned r = 0; r < cl.num_blocks(); ++r) {
      const Hist* p = &cl.map_shared_rank(&sm, r)->hist[buf];
      cnt += p->cnt[tid];
      mass += p->lo[tid] + ((unsigned long long)p->hi[tid] << 16);
    }
    unsigned ci = cnt;
    unsigned long long mi = mass;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned cv = __shfl_up_sync(0xffffffffu, ci, o);
      const unsigned long long mv = shfl_up64(mi, o);
      if (lane >= o) {
        ci += cv;
        mi += mv;
      }
    }
    if (lane == 31) {
      sm.wc[warp] = ci;
      sm.wm[warp] = mi;
    }
    __syncthreads();
    before_cnt = base_cnt + ci - cnt;
    before_mass = base_mass + mi - mass;
    for (int w = 0; w < warp; ++w) {
      before_cnt += sm.wc[w];
      before_mass += sm.wm[w];
    }
    if (tid == kThreads - 1) sm.whole = before_mass + mass;
    __syncthreads();
  }
  // The bin at which the running count reaches want_cnt or, where that is 0, the
  // running mass want_mass.  Every CTA finds the same.
  __device__ Found find(Smem& sm, unsigned want_cnt, unsigned long long want_mass) const {
    const bool here = want_cnt ? before_cnt < want_cnt && want_cnt <= before_cnt + cnt
                               : before_mass < want_mass && want_mass <= before_mass + mass;
    if (here) sm.found = Found{(int)threadIdx.x, before_cnt, before_mass};
    __syncthreads();
    const Found f = sm.found;
    __syncthreads();
    return f;
  }
};

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams a, const __grid_constant__ Table table) {
  using S = Slice<T, STAGED>;
  extern __shared__ uint4 stage[];
  constexpr int EPV = S::EPV;
  constexpr int KS = KeyShift<T>::v;
  constexpr bool TWO = sizeof(T) == 4;
  __shared__ Smem sm;
  cg::cluster_group cl = cg::this_cluster();
  const unsigned C = cl.num_blocks(), rank = cl.block_rank();
  const int n = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kTable) sm.table[tid] = table.v[tid];
  if (tid < 2) sm.list[tid].n = 0;
  for (int b = 0; b < 3; ++b) sm.hist[b].cnt[tid] = sm.hist[b].lo[tid] = sm.hist[b].hi[tid] = 0;
  pdl_wait();
  const int src = a.row_index ? a.row_index[n] : n;
  if (src < 0 || src >= a.rows) {  // the same for the whole cluster
    if (src >= a.rows && rank == 0 && tid == 0) a.tokens[n] = -1;
    return;
  }
  const float temp = a.temperature ? a.temperature[n] : 1.f;
  int want_k = a.top_k ? a.top_k[n] : 0;
  const float top_p = a.top_p ? a.top_p[n] : 1.f;
  float min_p = a.min_p ? a.min_p[n] : 0.f;
  const float u = a.uniforms[n];
  if (min_p > 1.f) want_k = 1;  // no weight reaches it: the first token alone
  // the one thing that takes 64-bit floats (two results a clock and SM), by one thread
  if (tid == 0) sm.ln_min_p = min_p > 0.f ? log((double)min_p) : 0.0;

  S s;
  s.init(static_cast<const T*>(a.logits) + src * a.row_stride, a.V, stage, rank, C);

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
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) key = sm.key[w] > key ? sm.key[w] : key;
      sm.best = key;
    }
  }
  cl.sync();  // (histograms are zero, too)
  unsigned long long best = 0;
  for (unsigned r = 0; r < C; ++r) {
    const unsigned long long k = cl.map_shared_rank(&sm, r)->best;
    best = k > best ? k : best;
  }
  if (!(temp > 0.f) || best == 0ull) {  // greedy, or a row of nothing but -inf
    if (rank == 0 && tid == 0) a.tokens[n] = best == 0ull ? -1 : (int)(0xffffffffu - (unsigned)best);
    cl.sync();  // no CTA leaves while others read it
    return;
  }
  Scale sc;
  sc.m = of_ord((uint32_t)(best >> 32));
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
  bool cut = false;
  uint32_t cut_key = 0;       // ord >> KS
  int cut_idx = -1;           // the last token of that value that is kept,
  unsigned stay = 0;          // or how many are (where the index is not known)
  if (use_k || use_p) {
    const float width = sc.hi * 16.f;
    auto bin_of = [&](float x) { return x == sc.m ? 0 : min(kBins - 1, __float2int_rz((sc.m - x) * width)); };
    auto weight_of = [&](float x) {  // 2^32 for the maximum
      return (weight<TWO>(x, sc, sm.table) + (1u << (kWBits - 33))) >> (kWBits - 32);
    };
    auto add = [&](Hist& h, int b, float x) {
      if (use_k) atomicAdd(&h.cnt[b], 1u);
      if (use_p) {
        const unsigned long long w = weight_of(x);
        const unsigned l = (unsigned)w & 0xffffu, g = (unsigned)(w >> 16);
        if (l) atomicAdd(&h.lo[b], l);
        if (g) atomicAdd(&h.hi[b], g);
      }
    };
    s.each([&](float x, int v, int e) {
      if ((unsigned)s.index(v, e) < (unsigned)a.V) add(sm.hist[0], bin_of(x), x);
    });
    cl.sync();
    int buf = 1;  // the next pass's histogram, zero at this point and read by nobody
    unsigned long long cut_mass = 0;  // mass up to the cut
    int which = 0, listed = -1;       // the next list; the bin whose tokens are merged
    unsigned nlist = 0;
    // from the bin that a count or mass falls in to the last token kept
    auto refine = [&](Found f, unsigned want_cnt, unsigned long long want_mass) {
      const int bin = f.bin;
      // the bin's tokens, ranked directly if they are few (they mostly are)
      if (bin != listed) {
        List& mine = sm.list[which];
        s.each([&](float x, int v, int e) {
          const int i = s.index(v, e);
          if (bin_of(x) != bin || (unsigned)i >= (unsigned)a.V) return;
          const unsigned at = atomicAdd(&mine.n, 1u);
          if (at < kList) {
            mine.key[at] = ord_of(x) >> KS;
            mine.idx[at] = i;
          }
        });
        cl.sync();
        nlist = 0;
        bool fits = true;
        int from = -1, at = 0;
        for (unsigned r = 0; r < C; ++r) {
          const unsigned c = cl.map_shared_rank(&sm, r)->list[which].n;
          if (from < 0 && (unsigned)tid < nlist + c) {
            from = (int)r;
            at = tid - (int)nlist;
          }
          fits = fits && c <= kList;
          nlist += c;
        }
        fits = fits && nlist <= kList;
        if (fits && tid < (int)nlist) {
          const List* l = &cl.map_shared_rank(&sm, from)->list[which];
          sm.mkey[tid] = l->key[at];
          sm.midx[tid] = l->idx[at];
          sm.mw[tid] = use_p ? weight_of(value_of_key<KS>(l->key[at])) : 0ull;
        }
        __syncthreads();
        which ^= 1;
        listed = fits ? bin : -1;
      }
      if (listed == bin) {
        if (tid < (int)nlist) {
          const uint32_t k = sm.mkey[tid];
          const int i = sm.midx[tid];
          const unsigned long long w = sm.mw[tid];
          unsigned c = f.cnt;
          unsigned long long m = f.mass;
          for (unsigned j = 0; j < nlist; ++j)
            if (sm.mkey[j] > k || (sm.mkey[j] == k && sm.midx[j] < i)) {
              ++c;
              m += sm.mw[j];
            }
          if (want_cnt ? c + 1 == want_cnt : m < want_mass && want_mass <= m + w) {
            sm.cut_key = k;
            sm.cut_idx = i;
            sm.cut_mass = m + w;
          }
        }
        __syncthreads();
        cut = true;
        cut_key = sm.cut_key;
        cut_idx = sm.cut_idx;
        cut_mass = sm.cut_mass;
        __syncthreads();
        return;
      }
      // the bin's keys, with room for rounding on both sides
      const float xh = sc.m - (float)bin / width, xl = sc.m - (float)(bin + 1) / width;
      uint32_t hi = ord_of(xh + 1e-5f * (fabsf(sc.m) + fabsf(xh)) + 1e-30f) >> KS;
      uint32_t lo = bin == kBins - 1 ? 0u : ord_of(xl - 1e-5f * (fabsf(sc.m) + fabsf(xl)) - 1e-30f) >> KS;
      if (!(fabsf(sc.m) < INFINITY)) {
        hi = 0xffffffffu >> KS;
        lo = 0;
      }
      while (true) {
        const int bits = 32 - __clz(hi - lo);
        const int shift = max(0, bits - 9);
        Hist& h = sm.hist[buf];
        s.each([&](float x, int v, int e) {
          const uint32_t k = ord_of(x) >> KS;
          if (k >= lo && k <= hi && bin_of(x) == bin && (unsigned)s.index(v, e) < (unsigned)a.V) add(h, (int)((hi - k) >> shift), x);
        });
        cl.sync();
        // past this barrier nobody reads the other buffer any more
        Hist& o = sm.hist[3 - buf];
        o.cnt[tid] = o.lo[tid] = o.hi[tid] = 0;
        Prefix sub;
        sub.sum(sm, buf, cl, f.cnt, f.mass);
        f = sub.find(sm, want_cnt, want_mass);  // ends in a block barrier
        buf = 3 - buf;
        hi -= (uint32_t)f.bin << shift;
        if (shift == 0) break;
        const uint32_t span = (1u << shift) - 1u;
        lo = max(lo, hi > span ? hi - span : 0u);
      }
      cut = true;
      cut_key = hi;
      cut_idx = -1;
      const unsigned long long w = use_p ? weight_of(value_of_key<KS>(hi)) : 0ull;
      stay = want_cnt ? want_cnt - f.cnt : (unsigned)((want_mass - f.mass + w - 1) / w);
      cut_mass = f.mass + stay * w;
    };
    Prefix bins;
    bins.sum(sm, 0, cl, 0u, 0ull);
    unsigned long long whole = sm.whole;
    if (use_k) {
      refine(bins.find(sm, (unsigned)want_k, 0ull), (unsigned)want_k, 0ull);
      whole = cut_mass;
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
      refine(bins.find(sm, 0u, want), 0u, want);
    }
  }
  __syncthreads();
  const float x_min = sm.x_min;
  auto kind = [&](float x, int i) {  // 2: kept, 1: equal to the cut, 0: not kept
    if (x < x_min) return 0;
    if (!cut) return 2;
    const uint32_t k = ord_of(x) >> KS;
    if (k != cut_key) return k > cut_key ? 2 : 0;
    return cut_idx < 0 ? ((unsigned)i < (unsigned)a.V ? 1 : 0) : i <= cut_idx ? 2 : 0;
  };

  // ---- kept mass of each warp's run, in vocab order ----
  {
    unsigned long long mass = 0;
    unsigned ties = 0;
    s.each([&](float x, int v, int e) {
      const int k = kind(x, s.index(v, e));
      if (k == 2) mass += weight<TWO>(x, sc, sm.table);
      ties += k == 1;
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mass += __shfl_xor_sync(0xffffffffu, mass, o);
      ties += __shfl_xor_sync(0xffffffffu, ties, o);
    }
    if (lane == 0) {
      sm.run_mass[warp] = mass;
      sm.run_ties[warp] = ties;
    }
  }
  cl.sync();
  // ---- the run that the draw falls in: every warp looks at all of them (a lane
  // per run, CTA by CTA), and the one that holds it goes on.  Of the tokens equal
  // to the cut the first `stay` in vocab order count.
  const unsigned long long wt = cut && cut_idx < 0 ? weight<TWO>(value_of_key<KS>(cut_key), sc, sm.table) : 0ull;
  const int nruns = (int)C * kWarps;  // at most 128
  unsigned long long mass[4];
  unsigned long long whole = 0, mine0 = 0, mine = 0;
  unsigned tb = 0, ties0 = 0;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int run = g * 32 + lane;
    mass[g] = 0;
    unsigned t = 0;
    if (run < nruns) {
      const Smem* p = cl.map_shared_rank(&sm, (unsigned)(run / kWarps));
      mass[g] = p->run_mass[run % kWarps];
      t = p->run_ties[run % kWarps];
    }
    unsigned ti = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, ti, o);
      if (lane >= o) ti += x;
    }
    const unsigned before = tb + ti - t;
    mass[g] += (before >= stay ? 0u : min(t, stay - before)) * wt;
    unsigned long long mi = mass[g];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = shfl_up64(mi, o);
      if (lane >= o) mi += x;
    }
    const int me = (int)rank * kWarps + warp;
    if (me / 32 == g) {
      ties0 = __shfl_sync(0xffffffffu, before, me % 32);
      mine = __shfl_sync(0xffffffffu, mass[g], me % 32);
      mine0 = whole + __shfl_sync(0xffffffffu, mi, me % 32) - mine;
    }
    whole += __shfl_sync(0xffffffffu, mi, 31);
    tb += __shfl_sync(0xffffffffu, ti, 31);
  }
  // the kept mass must exceed u * whole: a whole number at or below it
  const unsigned long long target = u >= 1.f ? whole - 1 : u > 0.f ? __umul64hi(whole, fraction64(u)) : 0ull;
  if (mine0 <= target && target < mine0 + mine) {
    unsigned long long run = mine0;
    unsigned trun = ties0;
    for (int v0 = s.wbeg; v0 < s.wend; v0 += 32) {  // 32 vectors at a time
      const int v = v0 + lane;
      unsigned long long w[EPV], sum = 0;
      unsigned tie = 0;  // bit e: element e equals the cut
#pragma unroll
      for (int e = 0; e < EPV; ++e) w[e] = 0;
      if (v < s.wend) {
        S::vec(s.get(v), [&](float x, int e) {
          const int k = kind(x, s.index(v, e));
          if (k == 2) w[e] = weight<TWO>(x, sc, sm.table);
          if (k == 1) tie |= 1u << e;
        });
      }
      const unsigned nt = __popc(tie);
      unsigned ti = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, ti, o);
        if (lane >= o) ti += x;
      }
      unsigned t = trun + ti - nt;
#pragma unroll
      for (int e = 0; e < EPV; ++e) {
        if (((tie >> e) & 1u) && t++ < stay) w[e] = wt;
        sum += w[e];
      }
      unsigned long long wi = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = shfl_up64(wi, o);
        if (lane >= o) wi += x;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, run + wi > target);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          unsigned long long at = run + wi - sum;
          int tok = -1;
#pragma unroll
          for (int e = 0; e < EPV; ++e) {
            at += w[e];
            if (tok < 0 && at > target) tok = s.index(v, e);
          }
          a.tokens[n] = tok;
        }
        break;
      }
      run += __shfl_sync(0xffffffffu, wi, 31);
      trun += __shfl_sync(0xffffffffu, ti, 31);
    }
  }
  cl.sync();  // no CTA leaves while others read it
}

constexpr int kStageMax = 96 * 1024;  // two CTAs per SM
constexpr int kMaxDevices = 64;

Table make_table() {
  Table t;
  for (int j = 0; j < kTable; ++j) t.v[j] = (int)(std::exp2(30.0 + j / (double)kTable) + 0.5);
  return t;
}

template <typename T, bool STAGED>
cudaError_t launch_s(const SampleParams& a, int C, size_t smem, cudaStream_t stream) {
  static std::atomic<bool> opted[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !opted[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(sample_kernel<T, STAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageMax);
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
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, STAGED>, a, table);
}

// CTAs per row: enough that a slice is at most four vectors a thread, and,
// when rows are few, until the grid fills the GPU twice or a thread has less
// than one vector.
template <typename T>
cudaError_t launch_t(const SampleParams& a, cudaStream_t stream) {
  constexpr int EPV = 16 / (int)sizeof(T);
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int nvec = (a.V + EPV - 1) / EPV + 1;
  int C = 1;
  while (C < kMaxCluster && (nvec / C > 4 * kThreads || ((long long)a.N * C < 2 * sms && nvec / C > kThreads))) C *= 2;
  const size_t bytes = 16 * (size_t)((nvec + C - 1) / C);
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
