// Eviction: of each sequence and KV head, the slots worth keeping go to new pages, in their
// order, until a budget is met: the first `sinks`, the last `recent`, and of those between
// the ones of largest weight (lower slots first among equals).
//
// Into new pages and not in place, so that a prompt's pages that other sequences share stay
// whole, no row waits for another to be read, and a call that is repeated gives the same.
//
// Two kernels.  select: a CTA per (sequence, KV head) finds the weight that the cut falls on
// by a radix select over order-preserving keys (11, 11 and 10 bits), which lie in shared
// memory as far as they fit, and lists the kept slots; every warp has a contiguous range of
// slots, so their order costs one scan over warps.  move: a warp per (new page, KV head)
// gathers the page's 16 keys and values, all in flight together, and their weights.  A
// block-scaled page takes the largest of its rows' scales; a row from a page of a smaller one
// is encoded again, value / new scale, which loses only codes that underflow.
//
// Bound by memory: every kept row is read and written once, the weights are read once.
#include <cmath>

#include "serve.cuh"

namespace mt {

namespace {

constexpr int kP = 16;
constexpr int kSelWarps = 16;
constexpr int kSelThreads = kSelWarps * 32;
constexpr int kBins = 2048;
constexpr int kMaxKeys = 40960;  // in shared memory

// Keys in the order of the weights: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (!(w == w)) return 0u;
  const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p, int max_keys) {
  extern __shared__ uint32_t s_keys[];  // [max_keys]
  __shared__ unsigned s_bins[kBins];
  __shared__ int s_warp[kSelWarps], s_warp2[kSelWarps];
  __shared__ unsigned s_bin;
  __shared__ int s_left;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.Hkv, b = blockIdx.x / p.Hkv;
  pdl_wait();
  const int L = p.seq_lens[b];
  if (L < 0) return;
  if ((long long)L > (long long)p.max_blocks * kP) {
    if (tid == 0) set_status(p.status, kStPages);
    return;
  }
  int* kept = p.kept + ((size_t)b * p.Hkv + h) * p.budget;
  if (L <= p.budget) {
    for (int i = tid; i < p.budget; i += kSelThreads) kept[i] = i < L ? i : -1;
    return;
  }
  // the slots between: count of them, and how many stay
  const int lo = p.sinks, count = L - p.recent - lo, stay = p.budget - p.sinks - p.recent;
  const int* bt = p.block_tables + (size_t)b * p.max_blocks;
  auto fetch = [&](int i) {
    const int slot = lo + i, page = bt[slot / kP];
    if (page < 0 || page >= p.num_pages) return 0u;  // reported by whoever moves it or its neighbours
    return key_of(p.weights[((size_t)page * p.Hkv + h) * kP + slot % kP]);
  };
  const bool held = count <= max_keys;
  if (held) {
#pragma unroll 4
    for (int i = tid; i < count; i += kSelThreads) s_keys[i] = fetch(i);
  }
  auto key = [&](int i) { return held ? s_keys[i] : fetch(i); };
  // the key of the last that stays, by digits; `left`: how many of its equals stay
  uint32_t cut = 0;
  int left = stay;
  if (stay > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kSelThreads) s_bins[i] = 0;
      __syncthreads();
      for (int i = tid; i < count; i += kSelThreads) {
        const uint32_t k = key(i);
        if (pass == 0 || (k >> (shift + bits)) == (cut >> (shift + bits)))
          atomicAdd(&s_bins[(k >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      // bins from the top: a thread has four neighbours, thread 0 the highest
      unsigned c[4], sum = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += c[e] = s_bins[kBins - 1 - 4 * tid - e];
      unsigned incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) s_warp[warp] = (int)incl;
      __syncthreads();
      unsigned before = incl - sum;
      for (int w = 0; w < warp; ++w) before += (unsigned)s_warp[w];
      if (before < (unsigned)left && before + sum >= (unsigned)left) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (before < (unsigned)left && before + c[e] >= (unsigned)left) {
            s_bin = kBins - 1 - 4 * tid - e;
            s_left = left - (int)before;
          }
          before += c[e];
        }
      }
      __syncthreads();
      cut |= s_bin << shift;
      left = s_left;
      __syncthreads();
    }
  }
  // which stay: every warp counts those of its range above the cut and on it
  const int per = ((count + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int i0 = min(warp * per, count), i1 = min(i0 + per, count);
  int above = 0, equal = 0;
  if (stay > 0) {
    for (int i = i0 + lane; i < i1; i += 32) {
      const uint32_t k = key(i);
      above += k > cut;
      equal += k == cut;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
  }
  if (lane == 0) {
    s_warp[warp] = above;
    s_warp2[warp] = equal;
  }
  __syncthreads();
  int eq_before = 0, at = p.sinks;  // places: the sinks first
  for (int w = 0; w < warp; ++w) {
    at += s_warp[w] + max(min(s_warp2[w], left - eq_before), 0);
    eq_before += s_warp2[w];
  }
  if (stay > 0) {
    for (int i = i0; i < i1; i += 32) {
      const bool in = i + lane < i1;
      const uint32_t k = in ? key(i + lane) : 0u;
      const unsigned eq = __ballot_sync(0xffffffffu, in && k == cut), below = (1u << lane) - 1u;
      const bool stays = in && (k > cut || (k == cut && eq_before + __popc(eq & below) < left));
      const unsigned all = __ballot_sync(0xffffffffu, stays);
      if (stays) kept[at + __popc(all & below)] = lo + i + lane;
      at += __popc(all);
      eq_before += __popc(eq);
    }
  }
  for (int i = tid; i < p.sinks; i += kSelThreads) kept[i] = i;
  for (int i = tid; i < p.recent; i += kSelThreads) kept[p.budget - p.recent + i] = L - p.recent + i;
}

constexpr int kMoveWarps = 4;

// RB: bytes of a row.
template <int RB, bool SCALED>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(const EvictParams p, int pages_out, long long items) {
  constexpr int LPR = RB / 16;                       // lanes per row (16-byte words), at most 32
  constexpr int RPS = 32 / LPR, STEPS = kP / RPS;    // rows a step
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  if (item >= items) return;
  pdl_wait();
  const int h = (int)(item % p.Hkv), j = (int)(item / p.Hkv % pages_out), b = (int)(item / p.Hkv / pages_out);
  const int L = p.seq_lens[b];
  if (L < 0 || (long long)L > (long long)p.max_blocks * kP) return;
  const int n = min(L, p.budget) - j * kP;  // rows of this page
  if (n <= 0) return;
  // lane r < 16: where row r comes from
  const int r = lane & 15;
  const int slot = r < n ? p.kept[((size_t)b * p.Hkv + h) * p.budget + j * kP + r] : 0;
  const int to = p.new_tables[(size_t)b * p.new_blocks + j];
  const int from = p.block_tables[(size_t)b * p.max_blocks + slot / kP];
  if (__any_sync(0xffffffffu, (r < n && (from < 0 || from >= p.num_pages)) || to < 0 || to >= p.num_pages)) {
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
  float kf = 1.f, vf = 1.f;
  if (SCALED) {
    float km = ks, vm = vs;
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
  const long long slots = (long long)p.max_blocks * kP - p.sinks - p.recent;
  const int keys = (int)(slots < 0 ? 0 : slots < kMaxKeys ? slots : kMaxKeys);
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4);
  if (e != cudaSuccess) return e;
  e = launch_pdl(evict_select_kernel, dim3((unsigned)rows), dim3(kSelThreads), (size_t)keys * 4, stream, p, keys);
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
