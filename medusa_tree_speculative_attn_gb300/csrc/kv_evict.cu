// Eviction: of each sequence and KV head, the slots worth keeping go to new pages, in their
// order, until a budget is met: the first `sinks`, the last `recent`, and of those between
// the ones of largest weight (lower slots first among equals).
//
// Into new pages and not in place, so that a prompt's pages that other sequences share stay
// whole, no row waits for another to be read, and a call that is repeated gives the same.
//
// Two kernels, and one that does both for few short rows.  select: a CTA per (sequence, KV head)
// finds the weight that the cut falls on by a radix select over order-preserving keys (11, 11 and
// 10 bits), which lie in shared memory where all of a row's fit, and are read again for each pass
// where not, and lists the kept slots; every warp has a contiguous range of slots, so their order
// costs one scan over warps.  move: a warp per (new page, KV head)
// gathers the page's 16 keys and values, all in flight together, and their weights.  A
// block-scaled page takes the largest of its rows' scales; a row from a page of a smaller one
// is encoded again, value / new scale, rounded once; between powers of two that loses only codes
// that underflow.
//
// Bound by memory: every kept row is read and written once, the weights are read once.  64
// sequences of 3000 to 4224 slots back to 4096, 8 heads of 128 columns in block-scaled codes:
// 160 us for 966 MB, 6.0 TB/s (88 % of a copy), of which select takes 17 and move, at a copy's
// rate, 142; 16 prompts of 4000 to 16384 to 2048 slots of a 16-bit cache: 60 us, select 18 for
// 128 CTAs of up to 16k keys, which three passes of a digit and two of counting go over; one
// sequence of 4224: 10.5 us, a chain of passes.  (A slot a thread and 512 threads:
// select 37 us for the prompts.)  Rows of 64 bytes: 55 % of a copy, two pages a warp no faster.
#include <atomic>
#include <cmath>

#include "serve.cuh"

namespace mt {

namespace {

constexpr int kP = 16;
constexpr int kMaxDevices = 64;
constexpr int kBins = 2048;
constexpr int kMaxKeys = 53248, kManyKeys = 24576;  // in shared memory: for one CTA an SM, and for two

// Keys in the order of the weights: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (!(w == w)) return 0u;
  const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The slots of (sequence b, KV head h) that stay, by a block of THREADS threads: keep(i, slot)
// is called for every place i of the first min(L, budget), by some thread.  L: the sequence's
// slots, within the table.  s_keys: [max_keys / 4], four slots each.
template <int THREADS, typename Keep>
__device__ __forceinline__ void select_slots(const EvictParams& p, int b, int h, int L, uint4* s_keys, int max_keys, Keep keep) {
  constexpr int WARPS = THREADS / 32, PER = kBins / THREADS;
  __shared__ unsigned s_bins[kBins];
  __shared__ int s_warp[WARPS], s_warp2[WARPS];
  __shared__ unsigned s_bin;
  __shared__ int s_left;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_bin = 0;
    s_left = 0;
  }
  if (L <= p.budget) {
    for (int i = tid; i < L; i += THREADS) keep(i, i);
    return;
  }
  // the slots between, lo .. hi - 1, and how many of them stay
  const int lo = p.sinks, hi = L - p.recent, stay = p.budget - p.sinks - p.recent;
  const int quads = (hi + 3) / 4, q_lo = lo / 4;
  const int* bt = p.block_tables + (size_t)b * p.max_blocks;
  auto keys_of = [&](int page, int q) {
    if (page < 0 || page >= p.num_pages) return make_uint4(0, 0, 0, 0);  // reported by whoever moves it
    const float4 w = *reinterpret_cast<const float4*>(p.weights + ((size_t)page * p.Hkv + h) * kP + q % 4 * 4);
    return make_uint4(key_of(w.x), key_of(w.y), key_of(w.z), key_of(w.w));
  };
  const bool held = quads * 4 <= max_keys;
  if (held) {
    for (int q0 = q_lo + tid; q0 < quads; q0 += 4 * THREADS) {  // four pages' numbers, then their weights on their way
      int page[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) page[e] = q0 + e * THREADS < quads ? bt[(q0 + e * THREADS) / 4] : -1;
      uint4 k[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = keys_of(page[e], q0 + e * THREADS);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (q0 + e * THREADS < quads) s_keys[q0 + e * THREADS] = k[e];
    }
  }
  // the keys of slots 4 q .. 4 q + 3, and which of them are between
  auto quad = [&](int q, uint32_t (&k)[4]) {
    const uint4 v = held ? s_keys[q] : keys_of(bt[q / 4], q);
    k[0] = v.x;
    k[1] = v.y;
    k[2] = v.z;
    k[3] = v.w;
    unsigned in = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) in |= (4 * q + e >= lo && 4 * q + e < hi ? 1u : 0u) << e;
    return in;
  };
  auto scan = [&](unsigned v) {  // of a warp, inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  auto before_warp = [&](const int* x) {  // sum of the warps before this one
    return __reduce_add_sync(0xffffffffu, lane < warp ? (unsigned)x[lane] : 0u);
  };
  // the key of the last that stays, by digits; `left`: how many of its equals stay
  uint32_t cut = 0;
  int left = stay;
  if (stay > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += THREADS) s_bins[i] = 0;
      __syncthreads();  // (the keys are there, too)
      for (int q = q_lo + tid; q < quads; q += THREADS) {
        uint32_t k[4];
        const unsigned in = quad(q, k);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((in >> e & 1u) && (pass == 0 || (k[e] >> (shift + bits)) == (cut >> (shift + bits))))
            atomicAdd(&s_bins[(k[e] >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      // bins from the top: a thread has PER neighbours, thread 0 the highest
      unsigned c[PER], sum = 0;
#pragma unroll
      for (int e = 0; e < PER; ++e) sum += c[e] = s_bins[kBins - 1 - PER * tid - e];
      const unsigned incl = scan(sum);
      if (lane == 31) s_warp[warp] = (int)incl;
      __syncthreads();
      unsigned before = incl - sum + before_warp(s_warp);
      if (before < (unsigned)left && before + sum >= (unsigned)left) {
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          if (before < (unsigned)left && before + c[e] >= (unsigned)left) {
            s_bin = kBins - 1 - PER * tid - e;
            s_left = left - (int)before;
          }
          before += c[e];
        }
      }
      __syncthreads();
      cut |= s_bin << shift;
      left = s_left;
    }
  }
  // which stay: every warp counts those of its range above the cut and on it
  const int per = ((quads - q_lo + WARPS - 1) / WARPS + 31) / 32 * 32;
  const int i0 = min(q_lo + warp * per, quads), i1 = min(i0 + per, quads);
  int above = 0, equal = 0;
  if (stay > 0) {
    for (int q = i0 + lane; q < i1; q += 32) {
      uint32_t k[4];
      const unsigned in = quad(q, k);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        above += (in >> e & 1u) && k[e] > cut;
        equal += (in >> e & 1u) && k[e] == cut;
      }
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
  }
  __syncthreads();  // everybody has read s_warp
  if (lane == 0) {
    s_warp[warp] = above;
    s_warp2[warp] = equal;
  }
  __syncthreads();
  // places: the sinks first, then what is above the cut and the first `left` on it
  int eq_before = (int)before_warp(s_warp2);
  int at = p.sinks + (int)before_warp(s_warp) + min(eq_before, left);
  if (stay > 0) {
    for (int q0 = i0; q0 < i1; q0 += 32) {
      uint32_t k[4] = {0, 0, 0, 0};
      const unsigned in = q0 + lane < i1 ? quad(q0 + lane, k) : 0u;
      unsigned eq = 0, gt = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        gt |= ((in >> e & 1u) && k[e] > cut ? 1u : 0u) << e;
        eq |= ((in >> e & 1u) && k[e] == cut ? 1u : 0u) << e;
      }
      // equals in the lanes before, then places: two counts in one scan each
      const int n = (int)scan(__popc(eq));
      const int eq_all = __shfl_sync(0xffffffffu, n, 31);
      int rank = eq_before + n - __popc(eq);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (eq >> e & 1u) gt |= (rank++ < left ? 1u : 0u) << e;  // from here on: all that stay
      const int m = (int)scan(__popc(gt));
      int to = at + m - __popc(gt);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (gt >> e & 1u) {
          // (always: but where the weights lie in memory only, somebody may change them meanwhile)
          if (to < p.budget - p.recent) keep(to, 4 * (q0 + lane) + e);
          ++to;
        }
      at += __shfl_sync(0xffffffffu, m, 31);
      eq_before += eq_all;
    }
  }
  for (int i = tid; i < p.sinks; i += THREADS) keep(i, i);
  for (int i = tid; i < p.recent; i += THREADS) keep(p.budget - p.recent + i, L - p.recent + i);
}

// THREADS: 256, 512 or 1024.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(const EvictParams p, int max_keys) {
  extern __shared__ uint4 s_keys[];
  const int h = blockIdx.x % p.Hkv, b = blockIdx.x / p.Hkv;
  pdl_wait();
  const int L = p.seq_lens[b];
  if (L < 0) return;
  if ((long long)L > (long long)p.max_blocks * kP) {
    if (threadIdx.x == 0) set_status(p.status, kStPages);
    return;
  }
  int* kept = p.kept + ((size_t)b * p.Hkv + h) * p.budget;
  select_slots<THREADS>(p, b, h, L, s_keys, max_keys, [&](int i, int slot) { kept[i] = slot; });
  for (int i = L + threadIdx.x; i < p.budget; i += THREADS) kept[i] = -1;
}

// A code's value times from / to, for the rounding to a code that follows: exactly as that product
// would be rounded.  Of codes with 4 bits and scales with 24 the product is on the border between two
// codes (5 bits), or 2^-29 of itself and more from it; hi and lo, the ratio in two parts, are off by
// 2^-48; so the product's 32 bits, with the last one set towards the side that they are off to, round
// as it would.
__device__ __forceinline__ float times(float x, float hi, float lo) {
  const float rest = x * lo, y = fmaf(x, hi, rest), off = fmaf(x, hi, -y) + rest;
  if (!(fabsf(off) > 0x1p-36f * fabsf(y))) return copysignf(y, x);  // a NaN, too; -0 stays one
  const uint32_t bits = __float_as_uint(y);
  return __uint_as_float((bits - ((__float_as_uint(off) ^ bits) >> 31)) | 1u);
}

// The rows that move_page has moved, encoded again with all care: under scales that differ by more
// than a power of two its products are rounded on the way to a code.  Apart from it, and from the old
// rows again, so that pages whose scales are powers of two, as the appends write them, pay nothing
// (the same at once, for all: one sequence of 4224 slots 13.4 us, not 11).
template <int RB>
__device__ __noinline__ void encode_exactly(const uint8_t* cache, uint8_t* to, int block, int at, int n, float from, float top) {
  constexpr int LPR = RB / 16, RPS = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const float hi = from / top, lo = fmaf(-hi, top, from) / top;
#pragma unroll 1
  for (int first = 0; first < kP; first += RPS) {
    const int row = first + lane / LPR, r = row & 15;  // row < kP: RPS divides it
    const int b = __shfl_sync(0xffffffffu, block, r), a = __shfl_sync(0xffffffffu, at, r);
    const float h = __shfl_sync(0xffffffffu, hi, r), l = __shfl_sync(0xffffffffu, lo, r);
    if (row >= n || (h == 1.f && l == 0.f)) continue;
    const int off = lane % LPR * 16;
    uint4 c = *reinterpret_cast<const uint4*>(cache + ((size_t)b * kP + a) * RB + off);
    float x[8], y[8];
    e4m3x8_to_f(make_uint2(c.x, c.y), x);
    e4m3x8_to_f(make_uint2(c.z, c.w), y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = times(x[e], h, l);
      y[e] = times(y[e], h, l);
    }
    const uint2 u = e4m3x8_of(x), v = e4m3x8_of(y);
    *reinterpret_cast<uint4*>(to + (size_t)row * RB + off) = make_uint4(u.x, u.y, v.x, v.y);
  }
}

constexpr int kMoveWarps = 4;

// New page j of (sequence b, KV head h), by a warp.  RB: bytes of a row.  L: the sequence's
// slots; kept: where the page's rows come from.
template <int RB, bool SCALED>
__device__ __forceinline__ void move_page(const EvictParams& p, int b, int h, int j, int L, const int* kept) {
  constexpr int LPR = RB / 16;                       // lanes per row (16-byte words), at most 32
  constexpr int RPS = 32 / LPR, STEPS = kP / RPS;    // rows a step
  const int lane = threadIdx.x & 31;
  const int n = min(L, p.budget) - j * kP;  // rows of this page
  if (n <= 0) return;
  // lane r < 16: where row r comes from
  const int r = lane & 15;
  int slot = r < n ? kept[r] : 0;
  const bool stray = slot < 0 || slot >= L;  // not as select leaves it
  if (stray) slot = 0;
  const int to = p.new_tables[(size_t)b * p.new_blocks + j];
  const int from = p.block_tables[(size_t)b * p.max_blocks + slot / kP];
  if (__any_sync(0xffffffffu, stray || (r < n && (from < 0 || from >= p.num_pages)) || to < 0 || to >= p.num_pages)) {
    if (lane == 0) set_status(p.status, kStPages);
    return;
  }
  const int src = r < n ? from * p.Hkv + h : 0;  // (page, head); below 2^27
  const int dst = to * p.Hkv + h;
  float ks = 0.f, vs = 0.f, w = 0.f;
  if (r < n) {
    if (SCALED) {
      ks = p.k_scales[src];
      vs = p.v_scales[src];
    }
    w = p.weights[(size_t)src * kP + slot % kP];
  }
  uint4 k[STEPS], v[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int row = s * RPS + lane / LPR;
    const int block = __shfl_sync(0xffffffffu, src, row & 15), at = __shfl_sync(0xffffffffu, slot % kP, row & 15);
    const size_t off = ((size_t)block * kP + at) * RB + (lane % LPR) * 16;
    k[s] = v[s] = make_uint4(0, 0, 0, 0);
    if (row < n) {
      k[s] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k_cache) + off));
      v[s] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.v_cache) + off));
    }
  }
  float kf = 1.f, vf = 1.f, km = ks, vm = vs;
  if (SCALED) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
      vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
    }
    kf = ks / km;
    vf = vs / vm;
    if (lane == 0) {
      p.k_scales[dst] = km;
      p.v_scales[dst] = vm;
    }
  }
  if (lane < n && lane < kP) p.weights[(size_t)dst * kP + lane] = w;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int row = s * RPS + lane / LPR;
    const size_t off = ((size_t)dst * kP + row) * RB + (lane % LPR) * 16;
    if (SCALED) {
      const float fk = __shfl_sync(0xffffffffu, kf, row & 15), fv = __shfl_sync(0xffffffffu, vf, row & 15);
      auto again = [](uint4& c, float f) {
        if (f == 1.f) return;
        float x[8], y[8];
        e4m3x8_to_f(make_uint2(c.x, c.y), x);
        e4m3x8_to_f(make_uint2(c.z, c.w), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= f;
          y[e] *= f;
        }
        const uint2 lo = e4m3x8_of(x), hi = e4m3x8_of(y);
        c = make_uint4(lo.x, lo.y, hi.x, hi.y);
      };
      again(k[s], fk);
      again(v[s], fv);
    }
    if (row < n) {
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.k_cache) + off) = k[s];
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.v_cache) + off) = v[s];
    }
  }
  if (SCALED) {
    auto odd = [](float from, float top) { return ((__float_as_uint(from) ^ __float_as_uint(top)) & 0x7fffffu) != 0; };
    if (__any_sync(0xffffffffu, r < n && (odd(ks, km) || odd(vs, vm)))) {
      uint8_t* kc = static_cast<uint8_t*>(p.k_cache);
      uint8_t* vc = static_cast<uint8_t*>(p.v_cache);
      const size_t page = (size_t)dst * kP * RB;
      encode_exactly<RB>(kc, kc + page, src, slot % kP, n, ks, km);
      encode_exactly<RB>(vc, vc + page, src, slot % kP, n, vs, vm);
    }
  }
}

template <int RB, bool SCALED>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(const EvictParams p, int pages_out, long long items) {
  const long long item = (long long)blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  if (item >= items) return;
  pdl_wait();
  const int h = (int)(item % p.Hkv), j = (int)(item / p.Hkv % pages_out), b = (int)(item / p.Hkv / pages_out);
  const int L = p.seq_lens[b];
  if (L < 0 || (long long)L > (long long)p.max_blocks * kP) return;
  move_page<RB, SCALED>(p, b, h, j, L, p.kept + ((size_t)b * p.Hkv + h) * p.budget + j * kP);
}

// Both in one launch, where the rows are few and their pages too: `parts` CTAs a (sequence, KV
// head) select, each for itself (SMs would idle otherwise), and move a part of the pages.  One
// sequence of 4224 slots, 8 heads: 10.5 us against 11.7 in two launches (with 1024 threads
// 11.4), and 2.7 us less of the host; 15 of up to 7812, 8 heads: 20.3 against 17.3, two of
// 32441, two heads: 79 against 38.
constexpr int kBothPages = 32;    // of a part, at most
constexpr int kBothSlots = 6144;  // the widest table
constexpr int kBothThreads = 512;

template <int RB, bool SCALED>
__global__ void __launch_bounds__(kBothThreads) evict_both_kernel(const EvictParams p, int max_keys, int parts, int part_pages) {
  extern __shared__ uint4 s_keys[];
  __shared__ int s_kept[kBothPages * kP];
  const int h = blockIdx.x % p.Hkv, part = blockIdx.x / p.Hkv % parts, b = blockIdx.x / p.Hkv / parts;
  pdl_wait();
  const int L = p.seq_lens[b];
  if (L < 0) return;
  if ((long long)L > (long long)p.max_blocks * kP) {
    if (threadIdx.x == 0) set_status(p.status, kStPages);
    return;
  }
  int* kept = p.kept + ((size_t)b * p.Hkv + h) * p.budget;
  const int first = part * part_pages * kP, last = min(first + part_pages * kP, p.budget);
  select_slots<kBothThreads>(p, b, h, L, s_keys, max_keys, [&](int i, int slot) {
    if (i < first || i >= last) return;
    s_kept[i - first] = slot;
    kept[i] = slot;
  });
  for (int i = max(L, first) + threadIdx.x; i < last; i += kBothThreads) kept[i] = -1;
  __syncthreads();
  for (int j = threadIdx.x >> 5; j < part_pages; j += kBothThreads / 32)
    move_page<RB, SCALED>(p, b, h, part * part_pages + j, L, s_kept + j * kP);
}

// Launches evict_both_kernel if it is its case.
template <int RB, bool SCALED>
cudaError_t launch_both(const EvictParams& p, int sms, bool* done, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.Hkv, slots = (long long)p.max_blocks * kP;
  const int pages_out = (p.budget + kP - 1) / kP;
  *done = false;
  if (slots > kBothSlots) return cudaSuccess;
  // a page a warp if SMs are left for that
  long long parts = (pages_out + kBothThreads / 32 - 1) / (kBothThreads / 32);
  if (parts > 2LL * sms / rows) parts = 2LL * sms / rows;
  if (parts < 1 || (pages_out + parts - 1) / parts > kBothPages) return cudaSuccess;
  const int part_pages = (int)((pages_out + parts - 1) / parts);
  parts = (pages_out + part_pages - 1) / part_pages;
  *done = true;
  return launch_pdl(evict_both_kernel<RB, SCALED>, dim3((unsigned)(rows * parts)), dim3(kBothThreads), (size_t)slots * 4,
                    stream, p, (int)slots, (int)parts, part_pages);
}

template <int RB, bool SCALED>
cudaError_t launch_move(const EvictParams& p, cudaStream_t stream) {
  const int pages_out = (p.budget + kP - 1) / kP;
  const long long items = (long long)p.B * pages_out * p.Hkv, blocks = (items + kMoveWarps - 1) / kMoveWarps;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  return launch_pdl(evict_move_kernel<RB, SCALED>, dim3((unsigned)blocks), dim3(kMoveWarps * 32), 0, stream, p, pages_out,
                    items);
}

}  // namespace

cudaError_t launch_kv_evict(const EvictParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.Hkv;
  if (rows >= (1ll << 31)) return cudaErrorInvalidValue;
  static std::atomic<int> sms_of[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev >= 0 && dev < kMaxDevices ? sms_of[dev].load(std::memory_order_acquire) : 0;
  if (!sms) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(evict_select_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize, kManyKeys * 4);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(evict_select_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) sms_of[dev].store(sms, std::memory_order_release);
  }
  bool done = false;
  if (p.k_scales)
    e = p.row_bytes == 64 ? launch_both<64, true>(p, sms, &done, stream) : launch_both<128, true>(p, sms, &done, stream);
  else if (p.row_bytes == 64)
    e = launch_both<64, false>(p, sms, &done, stream);
  else if (p.row_bytes == 128)
    e = launch_both<128, false>(p, sms, &done, stream);
  else if (p.row_bytes == 256)
    e = launch_both<256, false>(p, sms, &done, stream);
  else
    e = launch_both<512, false>(p, sms, &done, stream);
  if (done || e != cudaSuccess) return e;
  // few rows: as many threads and as much shared memory as there are for each; many: all rows
  // at once, or nearly, with fewer threads for short tables
  const long long slots = (long long)p.max_blocks * kP, most = rows <= sms ? kMaxKeys : kManyKeys;
  const int keys = (int)(slots < most ? slots : most);
  if (rows <= 2LL * sms)
    e = launch_pdl(evict_select_kernel<1024>, dim3((unsigned)rows), dim3(1024), (size_t)keys * 4, stream, p, keys);
  else if (slots > 2048)
    e = launch_pdl(evict_select_kernel<512>, dim3((unsigned)rows), dim3(512), (size_t)keys * 4, stream, p, keys);
  else
    e = launch_pdl(evict_select_kernel<256>, dim3((unsigned)rows), dim3(256), (size_t)keys * 4, stream, p, keys);
  if (e != cudaSuccess) return e;
  if (p.k_scales) return p.row_bytes == 64 ? launch_move<64, true>(p, stream) : launch_move<128, true>(p, stream);
  switch (p.row_bytes) {
    case 64: return launch_move<64, false>(p, stream);
    case 128: return launch_move<128, false>(p, stream);
    case 256: return launch_move<256, false>(p, stream);
    default: return launch_move<512, false>(p, stream);
  }
}

}  // namespace mt
