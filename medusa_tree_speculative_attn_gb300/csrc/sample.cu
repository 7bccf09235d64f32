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
// once.  Weights are integers (2^40 for the maximum), so every sum is exact and
// the same in any order; each weight is good to about 5e-10 of itself (the
// exponent as a sum of two floats, a 32-entry table, a short polynomial).  That
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

#include "serve.cuh"

namespace cg = cooperative_groups;

namespace mt {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;     // a thread per bin in the search
constexpr int kMaxCluster = 8;
constexpr int kMaxChunks = 512;     // warp-wide vectors per CTA: kSampleMaxVocab / kMaxCluster / (32 lanes * 4 fp32)
constexpr int kWBits = 40;          // weight of the maximum

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

struct Scale {
  float m;         // the row's maximum
  float hi, lo;    // log2(e) / temperature as a sum
};

// Weight of x: 2^40 exp((x - m) / t), rounded to a whole number.
// 2^e with e = n/32 + r, |r| <= 1/64:  table[n mod 32] * (1 + r * p(r)) * 2^(n div 32),
// n read off the low bits of e * 32 + 1.5 * 2^23, the correction r * p(r) as a
// 32-bit integer of 2^-37 (the only conversion instruction).
__device__ __forceinline__ unsigned long long weight(float x, const Scale& s, const unsigned long long* table) {
  const float d = x - s.m;
  const float p = d * s.hi;
  // below half a unit (-inf too); d is no number only where x = m = +inf
  if (!(p > -41.f)) return x == s.m ? 1ull << kWBits : 0ull;
  const float bb = d - x;
  const float err = (x - (d - bb)) + (-s.m - bb);  // x - m = d + err exactly
  const float e = fmaf(d, s.hi, -p) + fmaf(d, s.lo, err * s.hi);
  const float z = fmaf(p, 32.f, 12582912.f);
  const int n = __float_as_int(z) - 0x4B400000;
  const float r = fmaf(z - 12582912.f, -0.03125f, p) + e;
  constexpr float k37 = 137438953472.f;
  float q = fmaf(r, 9.618129e-3f * k37, 5.5504109e-2f * k37);  // ln2^4/24, ln2^3/6
  q = fmaf(r, q, 2.4022651e-1f * k37);                         // ln2^2/2
  q = fmaf(r, q, 6.9314718e-1f * k37) * r;                     // ln2
  const unsigned long long t = table[n & 31];
  const unsigned long long w = t + (((long long)(int)(t >> 10) * __float2int_rn(q)) >> 27);
  const int sh = -(n >> 5);
  return (w + ((1ull << sh) >> 1)) >> sh;
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
  unsigned long long table[32];
  unsigned long long key[kWarps];        // block reduction of (value, index)
  unsigned long long best;               // this CTA's, read by the cluster
  unsigned wc[kWarps];                   // scans
  unsigned long long wm[kWarps];
  Found found;
  List list[2];                          // this CTA's tokens of a bin, read by the cluster
  uint32_t mkey[kList];                  // the cluster's
  int midx[kList];
  unsigned long long mw[kList];
  uint32_t cut_key;
  int cut_idx;
  unsigned long long cut_mass;
  unsigned long long chunk_mass[kMaxChunks];
  unsigned chunk_ties[kMaxChunks];
  unsigned long long tot_mass;           // this CTA's kept mass (2^40 units), read by the cluster
  unsigned tot_ties;
};

// A CTA's part of a row, staged in shared memory by the first pass over it (or,
// where it does not fit, read again by every pass).
template <typename T, bool STAGED>
struct Slice {
  static constexpr int EPV = 16 / (int)sizeof(T);
  const T* row;
  uint4* stage;
  int V, beg, end, mis;  // this CTA's vectors [beg, end); vector v holds elements v * EPV - mis and on

  __device__ __forceinline__ uint4 load(int v) const {
    const int e0 = v * EPV - mis;
    if (e0 >= 0 && e0 + EPV <= V) return __ldg(reinterpret_cast<const uint4*>(row + e0));
    T t[EPV];  // a row's ragged first or last vector
#pragma unroll
    for (int e = 0; e < EPV; ++e) {
      const int i = e0 + e;
      t[e] = i >= 0 && i < V ? row[i] : Act<T>::from_f(-INFINITY);
    }
    uint4 r;
    memcpy(&r, t, 16);
    return r;
  }
  __device__ __forceinline__ uint4 get(int v) const { return STAGED ? stage[v - beg] : load(v); }
  // f(x, e) over the elements of vector v that lie in the row; NaN counts as -inf
  template <class F>
  __device__ __forceinline__ void vec(const uint4& r, int v, F f) const {
    T t[EPV];
    memcpy(t, &r, 16);
    const int e0 = v * EPV - mis;
#pragma unroll
    for (int e = 0; e < EPV; ++e) {
      const float x = Act<T>::to_f(t[e]);
      if ((unsigned)(e0 + e) < (unsigned)V) f(x == x ? x : -INFINITY, e);
    }
  }
  // f(x, index) over this thread's elements
  template <class F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll 1
    for (int v = beg + (int)threadIdx.x; v < end; v += kThreads)
      vec(get(v), v, [&](float x, int e) { f(x, v * EPV - mis + e); });
  }
  // the first pass: every element as f(x, index), the row into shared memory
  template <class F>
  __device__ __forceinline__ void first(F f) const {
    constexpr int U = 4;  // vectors in flight
#pragma unroll 1
    for (int v0 = beg + (int)threadIdx.x; v0 < end; v0 += U * kThreads) {
      uint4 r[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (v0 + j * kThreads < end) r[j] = load(v0 + j * kThreads);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int v = v0 + j * kThreads;
        if (v < end) {
          if (STAGED) stage[v - beg] = r[j];
          vec(r[j], v, [&](float x, int e) { f(x, v * EPV - mis + e); });
        }
      }
    }
  }
};

__device__ __forceinline__ unsigned long long shfl_up64(unsigned long long v, int o) {
  return __shfl_up_sync(0xffffffffu, v, o);
}

// Sums the cluster's histograms (a thread per bin) and finds the bin at which
// the running count reaches `want_cnt` or, where that is 0, the running mass
// reaches want_mass; base_* is what lies before the first bin.  Every CTA finds
// the same.  *whole: the mass of all bins and what lies before them.
__device__ Found search(Smem& sm, int buf, cg::cluster_group& cl, unsigned base_cnt, unsigned long long base_mass,
                        unsigned want_cnt, unsigned long long want_mass) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned c = 0;
  unsigned long long lo = 0;
  for (unsigned r = 0; r < cl.num_blocks(); ++r) {
    const Hist* p = &cl.map_shared_rank(&sm, r)->hist[buf];
    c += p->cnt[tid];
    lo += p->lo[tid];
    lo += (unsigned long long)p->hi[tid] << 16;
  }
  unsigned ci = c;
  unsigned long long mi = lo;
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
  unsigned cb = base_cnt;
  unsigned long long mb = base_mass;
  for (int w = 0; w < warp; ++w) {
    cb += sm.wc[w];
    mb += sm.wm[w];
  }
  const unsigned c0 = cb + ci - c;
  const unsigned long long m0 = mb + mi - lo;
  const bool here = want_cnt ? c0 < want_cnt && want_cnt <= c0 + c : m0 < want_mass && want_mass <= m0 + lo;
  if (here) sm.found = Found{tid, c0, m0};
  __syncthreads();
  const Found f = sm.found;
  __syncthreads();
  return f;
}

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(SampleParams a) {
  using S = Slice<T, STAGED>;
  extern __shared__ uint4 stage[];
  constexpr int EPV = S::EPV;
  constexpr int KS = KeyShift<T>::v;
  __shared__ Smem sm;
  cg::cluster_group cl = cg::this_cluster();
  const unsigned C = cl.num_blocks(), rank = cl.block_rank();
  const int n = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 32) sm.table[tid] = (unsigned long long)(exp2(tid * (1.0 / 32)) * (double)(1ull << kWBits) + 0.5);
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

  S s;
  s.row = static_cast<const T*>(a.logits) + src * a.row_stride;
  s.V = a.V;
  s.mis = (int)((reinterpret_cast<uintptr_t>(s.row) & 15) / sizeof(T));
  const int nvec = (a.V + s.mis + EPV - 1) / EPV;
  const int per = (nvec + (int)C - 1) / (int)C;
  s.beg = min(nvec, (int)rank * per);
  s.end = min(nvec, s.beg + per);
  s.stage = stage;

  // ---- maximum and its lowest index ----
  {
    float best = -INFINITY;
    int bi = 0x7fffffff;
    s.first([&](float x, int i) {  // a thread's indices rise
      if (x > best) {
        best = x;
        bi = i;
      }
    });
    unsigned long long key = bi == 0x7fffffff ? 0ull : ((unsigned long long)ord_of(best) << 32) | (0xffffffffu - (unsigned)bi);
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
    double k = 1.4426950408889634074 / (double)temp;
    k = k > 1e30 ? 1e30 : k;
    sc.hi = (float)k;
    sc.lo = (float)(k - (double)sc.hi);
  }

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
      return (weight(x, sc, sm.table) + (1u << (kWBits - 33))) >> (kWBits - 32);
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
    s.each([&](float x, int) { add(sm.hist[0], bin_of(x), x); });
    cl.sync();
    int buf = 1;  // the next pass's histogram, zero at this point and read by nobody
    unsigned long long cut_mass = 0;  // mass up to the cut
    int which = 0, listed = -1;       // the next list; the bin whose tokens are merged
    unsigned nlist = 0;
    auto value_of = [&](uint32_t key) {  // the value of a key
      const uint32_t o = key << KS;
      return of_ord((o & 0x80000000u) ? o : o | ((1u << KS) - 1u));
    };
    // from the bin that a count or mass falls in to the last token kept
    auto refine = [&](Found f, unsigned want_cnt, unsigned long long want_mass) {
      const int bin = f.bin;
      // the bin's tokens, ranked directly if they are few (they mostly are)
      if (bin != listed) {
        List& mine = sm.list[which];
        s.each([&](float x, int i) {
          if (bin_of(x) != bin) return;
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
          sm.mw[tid] = use_p ? weight_of(value_of(l->key[at])) : 0ull;
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
        s.each([&](float x, int) {
          const uint32_t k = ord_of(x) >> KS;
          if (k >= lo && k <= hi && bin_of(x) == bin) add(h, (int)((hi - k) >> shift), x);
        });
        cl.sync();
        // past this barrier nobody reads the other buffer any more
        Hist& o = sm.hist[3 - buf];
        o.cnt[tid] = o.lo[tid] = o.hi[tid] = 0;
        f = search(sm, buf, cl, f.cnt, f.mass, want_cnt, want_mass);  // ends in a block barrier
        buf = 3 - buf;
        hi -= (uint32_t)f.bin << shift;
        if (shift == 0) break;
        const uint32_t span = (1u << shift) - 1u;
        lo = max(lo, hi > span ? hi - span : 0u);
      }
      cut = true;
      cut_key = hi;
      cut_idx = -1;
      const unsigned long long w = use_p ? weight_of(value_of(hi)) : 0ull;
      stay = want_cnt ? want_cnt - f.cnt : (unsigned)((want_mass - f.mass + w - 1) / w);
      cut_mass = f.mass + stay * w;
    };
    unsigned long long whole;
    if (use_k) {
      const Found f = search(sm, 0, cl, 0u, 0ull, (unsigned)want_k, 0ull);
      refine(f, (unsigned)want_k, 0ull);
      whole = cut_mass;
    } else {
      whole = 0;
      // the mass of every bin: the search below wants a mass, so sum first
      unsigned long long mine = 0;
      for (unsigned r = 0; r < C; ++r) {
        const Hist* p = &cl.map_shared_rank(&sm, r)->hist[0];
        mine += p->lo[tid] + ((unsigned long long)p->hi[tid] << 16);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
      if (lane == 0) sm.wm[warp] = mine;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) whole += sm.wm[w];
      __syncthreads();
    }
    if (use_p) {
      // kept: mass before < top_p * whole, a whole number's comparison with the
      // next whole number at or above the product
      const double pz = ceil((double)top_p * (double)whole);
      unsigned long long want = pz > 1.0 ? (unsigned long long)pz : 1ull;
      if (want > whole) want = whole;
      const Found f = search(sm, 0, cl, 0u, 0ull, 0u, want);
      refine(f, 0u, want);
    }
  }
  // smallest value that min-p keeps: x >= m + t ln(min_p), the next float up
  float x_min = -INFINITY;
  if (min_p > 0.f) {
    x_min = fminf(__double2float_ru((double)sc.m + (double)temp * log((double)min_p)), sc.m);
  }

  // ---- kept mass of each warp-wide vector, in vocab order ----
  auto kind = [&](float x, int i) {  // 2: kept, 1: equal to the cut, 0: not kept
    if (x < x_min) return 0;
    if (!cut) return 2;
    const uint32_t k = ord_of(x) >> KS;
    if (k != cut_key) return k > cut_key ? 2 : 0;
    return cut_idx < 0 ? 1 : i <= cut_idx ? 2 : 0;
  };
  const int nch = (s.end - s.beg + 31) / 32;  // chunks of 32 vectors, 32 * EPV elements each
  {
#pragma unroll 1
    for (int v = s.beg + tid; v - lane < s.end; v += kThreads) {
      unsigned long long mass = 0;
      unsigned ties = 0;
      if (v < s.end)
        s.vec(s.get(v), v, [&](float x, int e) {
          const int k = kind(x, v * EPV - s.mis + e);
          if (k == 2) mass += weight(x, sc, sm.table);
          ties += k == 1;
        });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        mass += __shfl_xor_sync(0xffffffffu, mass, o);
        ties += __shfl_xor_sync(0xffffffffu, ties, o);
      }
      if (lane == 0) {
        const int c = (v - s.beg) / 32;
        sm.chunk_mass[c] = mass;
        sm.chunk_ties[c] = ties;
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    unsigned long long mass = 0;
    unsigned ties = 0;
    for (int c = lane; c < nch; c += 32) {
      mass += sm.chunk_mass[c];
      ties += sm.chunk_ties[c];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mass += __shfl_xor_sync(0xffffffffu, mass, o);
      ties += __shfl_xor_sync(0xffffffffu, ties, o);
    }
    if (lane == 0) {
      sm.tot_mass = mass;
      sm.tot_ties = ties;
    }
  }
  cl.sync();
  if (warp == 0) {
    // every CTA's kept mass; the first `stay` ties in vocab order count
    const uint32_t co = cut_key << KS;
    const float cx = of_ord((co & 0x80000000u) ? co : co | ((1u << KS) - 1u));
    const unsigned long long wt = cut ? weight(cx, sc, sm.table) : 0ull;
    unsigned long long whole = 0, mine0 = 0, mine = 0;
    unsigned ties = 0, ties0 = 0;
    for (unsigned r = 0; r < C; ++r) {
      const Smem* p = cl.map_shared_rank(&sm, r);
      const unsigned t = p->tot_ties;
      const unsigned take = ties >= stay ? 0u : min(t, stay - ties);
      const unsigned long long w = p->tot_mass + take * wt;
      if (r == rank) {
        mine0 = whole;
        mine = w;
        ties0 = ties;
      }
      whole += w;
      ties += t;
    }
    // the kept mass must exceed u * whole: a whole number at or below it
    const double tu = (double)whole * (double)u;
    unsigned long long target = tu > 0.0 ? (unsigned long long)tu : 0ull;
    if (target >= whole) target = whole - 1;
    if (mine0 <= target && target < mine0 + mine) {
      // the chunk: 32 at a time
      unsigned long long run = mine0;
      unsigned trun = ties0;
      int c0 = 0;
      unsigned long long m = 0;
      unsigned t = 0;
      for (;; c0 += 32) {
        const int c = c0 + lane;
        m = c < nch ? sm.chunk_mass[c] : 0ull;
        t = c < nch ? sm.chunk_ties[c] : 0u;
        unsigned ti = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned x = __shfl_up_sync(0xffffffffu, ti, o);
          if (lane >= o) ti += x;
        }
        const unsigned tb = trun + ti - t;  // ties before this chunk
        unsigned long long w = m + (tb >= stay ? 0u : min(t, stay - tb)) * wt;
        unsigned long long wi = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long x = shfl_up64(wi, o);
          if (lane >= o) wi += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, run + wi > target);
        if (hit || c0 + 32 >= nch) {
          const int l = hit ? __ffs(hit) - 1 : min(31, nch - 1 - c0);
          run += __shfl_sync(0xffffffffu, wi - w, l);
          trun = __shfl_sync(0xffffffffu, tb, l);
          c0 += l;
          break;
        }
        run += __shfl_sync(0xffffffffu, wi, 31);
        trun += __shfl_sync(0xffffffffu, ti, 31);
      }
      // the element: this lane's vector of the chunk
      const int v = s.beg + c0 * 32 + lane;
      unsigned long long w[EPV], sum = 0;
      unsigned char tie[EPV];
      unsigned nt = 0;
#pragma unroll
      for (int e = 0; e < EPV; ++e) {
        w[e] = 0;
        tie[e] = 0;
      }
      if (v < s.end) {
        s.vec(s.get(v), v, [&](float x, int e) {
          const int k = kind(x, v * EPV - s.mis + e);
          if (k == 2) w[e] = weight(x, sc, sm.table);
          tie[e] = k == 1;
          nt += k == 1;
        });
      }
      unsigned ti = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, ti, o);
        if (lane >= o) ti += x;
      }
      unsigned tb = trun + ti - nt;
#pragma unroll
      for (int e = 0; e < EPV; ++e) {
        if (tie[e] && tb++ < stay) w[e] = wt;
        sum += w[e];
      }
      unsigned long long wi = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = shfl_up64(wi, o);
        if (lane >= o) wi += x;
      }
      unsigned long long at = run + wi - sum;
      const unsigned hit = __ballot_sync(0xffffffffu, run + wi > target);
      if (hit && lane == __ffs(hit) - 1) {
        int tok = -1;
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
          at += w[e];
          if (tok < 0 && at > target) tok = v * EPV - s.mis + e;
        }
        a.tokens[n] = tok;
      }
    }
  }
  cl.sync();  // no CTA leaves while others read it
}

constexpr int kStageMax = 96 * 1024;  // two CTAs per SM
constexpr int kMaxDevices = 64;

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
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, STAGED>, a);
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
