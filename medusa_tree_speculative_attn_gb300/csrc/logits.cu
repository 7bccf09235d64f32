// Logits before a draw or an acceptance: penalties for repeated tokens, biases, grammar
// masks.  For a row x of sequence b, with seen_v: v is in the sequence's history or on the
// row's tree path, and c_v: how often v was generated (history from output_starts on, path):
//   x_v = x_v > 0 ? x_v / repetition : x_v * repetition   where seen_v
//   x_v = x_v - frequency * c_v - presence                 where c_v > 0
//   x_v = x_v + bias of v's last entry
//   x_v = -inf                                             where the row's mask says no
// in 32 bits with one rounding to the logits' type; other entries keep their bits.
//
// Few entries change, and the rest is a copy: a CTA takes a slice of the vocabulary and some
// of a sequence's rows.  It counts the slice's tokens of the history in shared memory (integer
// atomics: any order gives the same counts) and lists the tokens that matter as it first meets
// them, once for all rows (the list's order is any, and no result depends on it).  Then a warp
// takes a part of a row at a time through shared memory: brought asynchronously while the one
// before is worked on, the tokens that matter changed where they lie, written in 16-byte
// vectors with -inf where the mask says so.  In place, a row without a mask is not copied; its
// listed tokens alone are read and written.  A node's path is a bit mask of its ancestors, and
// a tree token has the bit mask of the nodes that hold it, so its count in a row is a
// population count.
//
// 16 trees of 64 nodes, 32000 bf16 logits, histories of 2048 to 4096 tokens, a third of the
// rows under a mask: 33 us for 133 MB, 4.0 TB/s (59 % of a copy): 3 for the lists, 25 for the
// copy, the rest instructions of the 1600 tokens a row that change.  Listed by a look at every
// word of the slice it took 36, with the changes made in global memory behind the copy 42, with
// eight rows a thread on their way 47.  One row of 32000 fp32 logits: 3.5 us, a launch and three
// dependent trips to memory.  Single rows of many sequences: a slice's chain of steps.
#include <atomic>
#include <cmath>

#include "serve.cuh"

namespace mt {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSlice = 6144;  // 120 rows of 102136, fp16: 2048 31 us, 4096 22, 6144 18 (three CTAs an SM), 8192 21
constexpr int kMaxDevices = 64;
constexpr int kCtas = 4;      // per SM, by registers
constexpr int kMaxRows = 64;  // of a CTA
constexpr unsigned kSeen = 0x80000000u;    // in a slice's count word: in the history
constexpr unsigned kInTree = 0x40000000u;  // a tree token: listed apart
constexpr unsigned kCount = 0x3fffffffu;
constexpr int kBiased = 1 << 16;           // in a token's place: it has a bias
constexpr int kPartBytes = 2048;           // of a row, that a warp takes at a time: four 16-byte vectors a lane
constexpr int kPlace = kPartBytes + 16;    // its place in shared memory

template <typename T> struct Lowest;
template <> struct Lowest<float> { static constexpr uint32_t word = 0xff800000u, one = 0xff800000u; };
template <> struct Lowest<__half> { static constexpr uint32_t word = 0xfc00fc00u, one = 0xfc00u; };
template <> struct Lowest<__nv_bfloat16> { static constexpr uint32_t word = 0xff80ff80u, one = 0xff80u; };

template <typename T>
__device__ __forceinline__ T minus_inf() {
  const uint32_t bits = Lowest<T>::one;
  T v;
  memcpy(&v, &bits, sizeof(T));
  return v;
}

// N mask bits from token v on (N <= 8): the word behind is looked at only where they reach.
template <int N>
__device__ __forceinline__ unsigned mask_bits(const int* mask, int v) {
  const int w = v >> 5, s = v & 31;
  unsigned bits = (unsigned)__ldg(mask + w) >> s;
  if (s + N > 32) bits |= (unsigned)__ldg(mask + w + 1) << (32 - s);
  return bits & ((1u << N) - 1u);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtas) logits_kernel(const LogitsParams p, int slice, int slices, int groups, int group_rows) {
  constexpr int N = 16 / (int)sizeof(T), kPart = kPartBytes / (int)sizeof(T);  // tokens of a vector, of a part
  constexpr int K = kPartBytes / 512;  // vectors of a part per lane
  constexpr unsigned kAll = (1u << N) - 1u;
  extern __shared__ __align__(16) uint8_t smem[];  // the warps' parts
  unsigned* s_count = reinterpret_cast<unsigned*>(smem + kWarps * 2 * kPlace);  // [slice]
  unsigned* s_entry = s_count + slice;                                          // [slice] bias entry + 1 (with biases)
  uint16_t* s_list = reinterpret_cast<uint16_t*>(s_count + (p.num_bias ? 2 : 1) * slice);  // [slice]
  __shared__ int s_listed, s_trees;
  __shared__ int s_which[kMaxRows];
  __shared__ int s_tok[kMaxTree], s_par[kMaxTree], s_at[kMaxTree];
  __shared__ unsigned long long s_anc[kMaxTree], s_nodes[kMaxTree];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = blockIdx.x % slices * slice, group = blockIdx.x / slices % groups, b = blockIdx.x / slices / groups;
  const int n = min(slice, p.V - v0);
  const int t0 = group * group_rows, rows = min(group_rows, p.T - t0);
  pdl_wait();
  int len = 0, start = 0;
  if (p.history_lens) {
    len = min(p.history_lens[b], p.history_width);
    if (len < 0) return;  // no sequence
    start = p.output_starts ? p.output_starts[b] : 0;
  }
  const T* in = static_cast<const T*>(p.logits) + (size_t)b * p.stride[0] + (size_t)t0 * p.stride[1] + v0;
  T* out = static_cast<T*>(p.out) + (size_t)b * p.out_stride[0] + (size_t)t0 * p.out_stride[1] + v0;
  const bool in_place = p.logits == p.out;
  const int words = (p.V + 31) / 32;

  // ---- the slice's tokens that matter ----
  for (int i = tid; i < (p.num_bias ? 2 : 1) * slice / 4; i += kThreads)
    reinterpret_cast<uint4*>(s_count)[i] = make_uint4(0, 0, 0, 0);
  if (tid < rows) {  // each row's mask: -1 for none, num_masks for one past the last, which allows nothing
    const int row = b * p.T + t0 + tid;
    s_which[tid] = !p.mask ? -1 : p.mask_index ? min(max(p.mask_index[row], -1), p.num_masks) : row;
  }
  if (tid == 0) s_listed = s_trees = 0;
  if (p.tree_tokens && tid < p.T) {
    s_tok[tid] = p.tree_tokens[(size_t)b * p.T + tid];
    const int par = p.tree_parents ? p.tree_parents[(size_t)b * p.T + tid] : tid - 1;
    const bool ok = tid == 0 ? par == -1 : (par >= 0 && par < tid);
    if (!ok) set_status(p.status, kStTree);
    s_par[tid] = ok ? par : -1;
  }
  const int* history = p.history + (size_t)b * p.history_width;
  int tok[16];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int i = i0 + e * kThreads + tid;
      tok[e] = i < len ? history[i] : -1;
    }
  };
  fetch(0);
  __syncthreads();
  // The rows go through shared memory where they are copied or masked, a warp a part of a row at
  // a time, the next one on its way: element i of a part lies at its place as it lies to a
  // 16-byte boundary in memory.
  const int per = (n + kPart - 1) / kPart, items = rows * per;
  uint8_t* place = smem + warp * (2 * kPlace);
  const uint32_t place_u = static_cast<uint32_t>(__cvta_generic_to_shared(place));
  auto bring = [&](int item, int turn) {
    if (item < items) {
      const int t = item / per, c0 = item % per * kPart, m = min(kPart, n - c0), which = s_which[t];
      if (!(in_place && which < 0) && !(which >= 0 && which == p.num_masks)) {
        const T* src = in + (size_t)t * p.stride[1] + c0;
        const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(src) & 15);
        const int head = min(m, (int)((16 - off) & 15) / (int)sizeof(T)), vecs = (m - head) / N;
        const uint32_t to = place_u + turn * kPlace + off + head * (int)sizeof(T);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int i = k * 32 + lane;
          if (i < vecs) cp_async16(to + i * 16, src + head + i * N);
        }
        T* x = reinterpret_cast<T*>(place + turn * kPlace + off);
        for (int i = lane; i < head; i += 32) x[i] = src[i];
        for (int i = head + vecs * N + lane; i < m; i += 32) x[i] = src[i];
      }
    }
    cp_commit();
  };
  bring(warp, 0);
  if (p.tree_tokens && tid < p.T) {
    unsigned long long anc = 0, nodes = 0;
    for (int a = tid; a >= 0; a = s_par[a]) anc |= 1ull << a;  // parents are earlier: at most T steps
    s_anc[tid] = anc;
    const unsigned at = (unsigned)s_tok[tid] - (unsigned)v0;
    if (s_tok[tid] >= 0 && at < (unsigned)n) {
      for (int a = 0; a < p.T; ++a)
        if (s_tok[a] == s_tok[tid]) nodes |= 1ull << a;
      if (__ffsll((long long)nodes) - 1 == tid) {  // the first of the nodes that hold it
        const int k = atomicAdd(&s_trees, 1);
        s_at[k] = (int)at;
        s_nodes[k] = nodes;
        atomicOr(&s_count[at], kInTree);
      }
    }
  }
  if (p.tree_tokens) __syncthreads();
#pragma unroll 1
  for (int i0 = 0; i0 < len; i0 += 16 * kThreads) {
    if (i0) fetch(i0);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if (i0 + e * kThreads >= len) break;
      const unsigned at = (unsigned)tok[e] - (unsigned)v0;
      if (tok[e] >= 0 && at < (unsigned)n) {
        const unsigned was = i0 + e * kThreads + tid >= start ? atomicAdd(&s_count[at], 1u) : atomicOr(&s_count[at], kSeen);
        if (was == 0) s_list[atomicAdd(&s_listed, 1)] = (uint16_t)at;  // its first
      }
    }
  }
  if (p.num_bias) __syncthreads();
  for (int i = tid; i < p.num_bias; i += kThreads) {
    const int token = p.bias_tokens[(size_t)b * p.num_bias + i];
    const unsigned at = (unsigned)token - (unsigned)v0;
    if (token >= 0 && at < (unsigned)n && atomicMax(&s_entry[at], (unsigned)i + 1u) == 0 && s_count[at] == 0)
      s_list[atomicAdd(&s_listed, 1)] = (uint16_t)at;
  }
  const float rep = p.repetition ? p.repetition[b] : 1.f, pres = p.presence ? p.presence[b] : 0.f;
  const float freq = p.frequency ? p.frequency[b] : 0.f;
  const float* bias = p.bias_values + (size_t)b * p.num_bias;

  __syncthreads();  // the list is whole
  const int listed = s_listed, entries = listed + s_trees;
  // One of the tokens that matter: its place in the slice (-1: none), what it is, what is
  // taken off for its count, its bias.  A tree token's count is the row's.
  struct Token {
    int at;
    unsigned what;  // kSeen, and the count that is not a path's; kInTree: and a path's
    float sub, add;
  };
  auto token = [&](int e) {
    Token k{-1, 0u, 0.f, 0.f};
    if (e >= entries) return k;
    k.at = e < listed ? (int)s_list[e] : s_at[e - listed];
    k.what = s_count[k.at];
    k.sub = __fmul_rn(freq, (float)(k.what & kCount));
    const unsigned entry = p.num_bias ? s_entry[k.at] : 0u;
    if (entry) k.add = bias[entry - 1];
    if (entry) k.at |= kBiased;
    return k;
  };
  // Its new value in row t; false: as it was.
  auto change = [&](const Token& k, int e, int t, float& y) {
    unsigned c = k.what & ~kInTree;
    float sub = k.sub;
    if (k.what & kInTree) {
      const unsigned path = (unsigned)__popcll(s_anc[t0 + t] & s_nodes[e - listed]);
      c += path;
      sub = __fmul_rn(freq, (float)(c & kCount));
    }
    if (rep != 1.f && c) y = y > 0.f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
    if (c & kCount) y = __fsub_rn(__fsub_rn(y, sub), pres);
    if (k.at & kBiased) y = __fadd_rn(y, k.add);
    return c || (k.at & kBiased);
  };
  // The first of them stay with their lanes for all rows.
  constexpr int kHeld = 2;
  Token held[kHeld];
#pragma unroll
  for (int q = 0; q < kHeld; ++q) held[q] = token(q * 32 + lane);
  // All of them that lie in tokens c0 .. c0 + m - 1 of row t, from `x` to `y`.
  auto change_all = [&](int t, int c0, int m, const T* x, T* y) {
    auto one = [&](const Token& k, int e) {
      const int at = k.at < 0 ? -1 : (k.at & ~kBiased) - c0;
      if (at < 0 || at >= m) return;
      float v = Act<T>::to_f(x[at]);
      if (change(k, e, t, v)) y[at] = Act<T>::from_f(v);
    };
#pragma unroll
    for (int q = 0; q < kHeld; ++q) one(held[q], q * 32 + lane);
    for (int e = kHeld * 32 + lane; e < entries; e += 32) one(token(e), e);
  };
  int turn = 0;
#pragma unroll 1
  for (int item = warp; item < items; item += kWarps, turn ^= 1) {
    bring(item + kWarps, turn ^ 1);
    const int t = item / per, c0 = item % per * kPart, m = min(kPart, n - c0), which = s_which[t];
    const T* src = in + (size_t)t * p.stride[1] + c0;
    T* dst = out + (size_t)t * p.out_stride[1] + c0;
    if (in_place && which < 0) {  // nothing but those tokens
      change_all(t, c0, m, src, dst);
      continue;
    }
    const bool none = which >= 0 && which == p.num_masks;
    const int* mask = which >= 0 && !none ? p.mask + (size_t)which * words : nullptr;
    const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(src) & 15);
    T* x = reinterpret_cast<T*>(place + turn * kPlace + off);
    const int first = v0 + c0;
    const int head = min(m, (int)((16 - off) & 15) / (int)sizeof(T)), vecs = (m - head) / N;
    unsigned yes[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = k * 32 + lane;
      yes[k] = none ? 0u : mask && i < vecs ? mask_bits<N>(mask, first + head + i * N) : kAll;
    }
    cp_wait<1>();
    __syncwarp();
    if (!none) {
      change_all(t, c0, m, x, x);
      __syncwarp();
    }
    auto one = [&](int i) {
      dst[i] = none || (mask && !(mask_bits<1>(mask, first + i) & 1u)) ? minus_inf<T>() : x[i];
    };
    if ((reinterpret_cast<uintptr_t>(dst) & 15) == off) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = k * 32 + lane;
        if (i >= vecs) continue;
        constexpr uint32_t low = Lowest<T>::word;
        uint4 w = make_uint4(low, low, low, low);
        if (yes[k] != 0u) w = *reinterpret_cast<const uint4*>(x + head + i * N);
        if (yes[k] != 0u && yes[k] != kAll) {
          T e[N];
          memcpy(e, &w, 16);
#pragma unroll
          for (int q = 0; q < N; ++q)
            if (!(yes[k] >> q & 1u)) e[q] = minus_inf<T>();
          memcpy(&w, e, 16);
        }
        *reinterpret_cast<uint4*>(dst + head + i * N) = w;
      }
      for (int i = lane; i < head; i += 32) one(i);
      for (int i = head + vecs * N + lane; i < m; i += 32) one(i);
    } else {
      for (int i = lane; i < m; i += 32) one(i);
    }
    __syncwarp();  // the place is filled again
  }
  cp_wait<0>();
}

template <typename T>
cudaError_t launch_t(const LogitsParams& p, cudaStream_t stream) {
  static std::atomic<int> sms_of[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev >= 0 && dev < kMaxDevices ? sms_of[dev].load(std::memory_order_acquire) : 0;
  if (!sms) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(logits_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kWarps * 2 * kPlace + (kMaxSlice + 64) * 10);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) sms_of[dev].store(sms, std::memory_order_release);
  }
  // Rows are shared out where even the smallest slices, a warp's part, would leave SMs without
  // work; then a sequence's slices, so many that the CTAs fill the SMs once.  With few rows a
  // slice is as long as shared memory allows: every slice goes over the whole history.
  constexpr int kPart = kPartBytes / (int)sizeof(T);
  int groups = (p.T + kMaxRows - 1) / kMaxRows;
  const int parts = (p.V + kPart - 1) / kPart;
  while ((long long)p.B * parts * groups < 2LL * sms && groups < p.T) groups = groups * 2 < p.T ? groups * 2 : p.T;
  const int group_rows = (p.T + groups - 1) / groups;
  groups = (p.T + group_rows - 1) / group_rows;
  const int least = group_rows >= kWarps ? parts : (p.V + kMaxSlice - 1) / kMaxSlice;
  const long long fill = (long long)kCtas * sms / ((long long)p.B * groups);
  int slices = (int)(fill < least ? least : fill > 2 * parts ? 2 * parts : fill);
  const int slice = ((p.V + slices - 1) / slices + 63) / 64 * 64;
  slices = (p.V + slice - 1) / slice;
  const long long blocks = (long long)p.B * groups * slices;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  const size_t smem = kWarps * 2 * kPlace + (size_t)slice * ((p.num_bias ? 8 : 4) + 2);
  return launch_pdl(logits_kernel<T>, dim3((unsigned)blocks), dim3(kThreads), smem, stream, p, slice, slices, groups,
                    group_rows);
}

}  // namespace

cudaError_t launch_logits(const LogitsParams& p, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case 0: return launch_t<float>(p, stream);
    case 1: return launch_t<__half>(p, stream);
    default: return launch_t<__nv_bfloat16>(p, stream);
  }
}

}  // namespace mt
