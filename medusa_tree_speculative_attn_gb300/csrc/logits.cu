// Logits before a draw or an acceptance: penalties for repeated tokens, biases, grammar
// masks.  For a row x of sequence b, with seen_v: v is in the sequence's history or on the
// row's tree path, and c_v: how often v was generated (history from output_starts on, path):
//   x_v = x_v > 0 ? x_v / repetition : x_v * repetition   where seen_v
//   x_v = x_v - frequency * c_v - presence                 where c_v > 0
//   x_v = x_v + bias of v's last entry
//   x_v = -inf                                             where the row's mask says no
// in 32 bits with one rounding to the logits' type; other entries keep their bits.
//
// Bound by memory, and few entries change: a CTA takes a slice of the vocabulary and some of
// a sequence's rows.  It counts the slice's tokens of the history in shared memory (integer
// atomics: any order gives the same counts), lists the tokens that matter once, and then
//   - goes over the rows in 16-byte vectors where something has to be copied or masked (in
//     place, a row without a mask is not touched, and whole vectors of masked tokens are
//     written without being read);
//   - changes the listed tokens of every row, a warp a row.
// A node's path is a bit mask of its ancestors, and a tree token has the bit mask of the
// nodes that hold it, so its count in a row is a population count.
#include <cmath>

#include "serve.cuh"

namespace mt {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSlice = 4096;
constexpr unsigned kSeen = 0x80000000u;    // in a slice's count word: in the history
constexpr unsigned kInTree = 0x40000000u;  // a tree token: listed apart
constexpr unsigned kCount = 0x3fffffffu;

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

template <typename T>
__global__ void __launch_bounds__(kThreads) logits_kernel(const LogitsParams p, int slice, int slices, int groups, int group_rows) {
  constexpr int N = 16 / (int)sizeof(T);  // of a vector
  extern __shared__ unsigned s_count[];                                     // [slice]
  unsigned* s_entry = s_count + slice;                                      // [slice] bias entry + 1 (with biases)
  uint16_t* s_list = reinterpret_cast<uint16_t*>(s_count + (p.num_bias ? 2 : 1) * slice);  // [slice]
  __shared__ int s_listed, s_trees;
  __shared__ int s_tok[kMaxTree], s_par[kMaxTree], s_at[kMaxTree];
  __shared__ unsigned long long s_anc[kMaxTree], s_nodes[kMaxTree];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = blockIdx.x % slices * slice, group = blockIdx.x / slices % groups, b = blockIdx.x / slices / groups;
  const int n = min(slice, p.V - v0);
  const int t0 = group * group_rows, t1 = min(t0 + group_rows, p.T);
  pdl_wait();
  int len = 0, start = 0;
  if (p.history_lens) {
    len = min(p.history_lens[b], p.history_width);
    if (len < 0) return;  // no sequence
    start = p.output_starts ? p.output_starts[b] : 0;
  }
  for (int i = tid; i < (p.num_bias ? 2 : 1) * slice; i += kThreads) s_count[i] = 0;
  if (tid == 0) s_listed = s_trees = 0;
  if (p.tree_tokens && tid < p.T) {
    s_tok[tid] = p.tree_tokens[(size_t)b * p.T + tid];
    const int par = p.tree_parents ? p.tree_parents[(size_t)b * p.T + tid] : tid - 1;
    const bool ok = tid == 0 ? par == -1 : (par >= 0 && par < tid);
    if (!ok) set_status(p.status, kStTree);
    s_par[tid] = ok ? par : -1;
  }
  __syncthreads();
  const int* history = p.history + (size_t)b * p.history_width;
#pragma unroll 4
  for (int i = tid; i < len; i += kThreads) {
    const unsigned at = (unsigned)(history[i] - v0);
    if (at < (unsigned)n) {
      if (i >= start) atomicAdd(&s_count[at], 1u);
      else atomicOr(&s_count[at], kSeen);
    }
  }
  for (int i = tid; i < p.num_bias; i += kThreads) {
    const unsigned at = (unsigned)(p.bias_tokens[(size_t)b * p.num_bias + i] - v0);
    if (at < (unsigned)n) atomicMax(&s_entry[at], (unsigned)i + 1u);
  }
  if (p.tree_tokens && tid < p.T) {
    unsigned long long anc = 0, nodes = 0;
    for (int a = tid; a >= 0; a = s_par[a]) anc |= 1ull << a;  // parents are earlier: at most T steps
    s_anc[tid] = anc;
    const unsigned at = (unsigned)(s_tok[tid] - v0);
    if (at < (unsigned)n) {
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
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const unsigned c = s_count[i];
    if (!(c & kInTree) && (c || (p.num_bias && s_entry[i]))) s_list[atomicAdd(&s_listed, 1)] = (uint16_t)i;
  }
  const T* in = static_cast<const T*>(p.logits) + (size_t)b * p.stride[0] + v0;
  T* out = static_cast<T*>(p.out) + (size_t)b * p.out_stride[0] + v0;
  const bool in_place = p.logits == p.out;
  const int words = (p.V + 31) / 32;
  // a row's mask: -1 for none, num_masks for one past the last, which allows nothing
  auto mask_of = [&](int t) {
    if (!p.mask) return -1;
    const int row = b * p.T + t;
    return p.mask_index ? min(max(p.mask_index[row], -1), p.num_masks) : row;
  };
  for (int t = t0; t < t1; ++t) {
    const int which = mask_of(t);
    if (in_place && which < 0) continue;
    const bool none = which == p.num_masks && which >= 0;
    const int* mask = which >= 0 ? p.mask + (size_t)which * words : nullptr;
    const T* src = in + (size_t)t * p.stride[1];
    T* dst = out + (size_t)t * p.out_stride[1];
    // elements up to the first 16-byte boundary of both, whole vectors, the rest
    const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(dst) & 15);
    int head = (int)((16 - off) & 15) / (int)sizeof(T), vecs = 0;
    if ((reinterpret_cast<uintptr_t>(src) & 15) == off && head < n) vecs = (n - head) / N;
    else head = n;
    auto one = [&](int i) {
      const bool no = none || (mask && !(mask_bits<1>(mask, v0 + i) & 1u));
      if (no) dst[i] = minus_inf<T>();
      else if (!in_place) dst[i] = src[i];
    };
    for (int i = tid; i < head; i += kThreads) one(i);
    for (int i = head + vecs * N + tid; i < n; i += kThreads) one(i);
#pragma unroll 4
    for (int i = tid; i < vecs; i += kThreads) {
      const int at = head + i * N;
      const unsigned yes = none ? 0u : mask ? mask_bits<N>(mask, v0 + at) : (1u << N) - 1u;
      uint4* d = reinterpret_cast<uint4*>(dst + at);
      constexpr uint32_t low = Lowest<T>::word;
      if (yes == 0) {
        *d = make_uint4(low, low, low, low);
      } else if (yes != (1u << N) - 1u || !in_place) {
        T x[N];
        const uint4 w = *reinterpret_cast<const uint4*>(src + at);
        memcpy(x, &w, 16);
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (!(yes >> e & 1u)) x[e] = minus_inf<T>();
        uint4 y;
        memcpy(&y, x, 16);
        *d = y;
      }
    }
  }
  __syncthreads();  // the list is whole, and the rows are copied
  const float rep = p.repetition ? p.repetition[b] : 1.f, pres = p.presence ? p.presence[b] : 0.f;
  const float freq = p.frequency ? p.frequency[b] : 0.f;
  const float* bias = p.bias_values + (size_t)b * p.num_bias;
  const int listed = s_listed, trees = s_trees;
  for (int t = t0 + warp; t < t1; t += kWarps) {
    const int which = mask_of(t);
    if (which >= 0 && which == p.num_masks) continue;
    const int* mask = which >= 0 ? p.mask + (size_t)which * words : nullptr;
    const T* src = in + (size_t)t * p.stride[1];
    T* dst = out + (size_t)t * p.out_stride[1];
    auto change = [&](int at, bool seen, unsigned count) {
      if (mask && !(mask_bits<1>(mask, v0 + at) & 1u)) return;
      float x = Act<T>::to_f(src[at]);
      if (seen) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
      if (count) x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, (float)count)), pres);
      if (p.num_bias && s_entry[at]) x = __fadd_rn(x, bias[s_entry[at] - 1]);
      dst[at] = Act<T>::from_f(x);
    };
#pragma unroll 2
    for (int i = lane; i < listed; i += 32) {
      const int at = s_list[i];
      const unsigned c = s_count[at];
      change(at, c != 0, c & kCount);
    }
    if (trees) {
      const unsigned long long anc = s_anc[t];
      for (int i = lane; i < trees; i += 32) {
        const int at = s_at[i];
        const unsigned c = s_count[at] & ~kInTree, path = (unsigned)__popcll(anc & s_nodes[i]);
        const unsigned count = (c & kCount) + path;
        if (c || path || (p.num_bias && s_entry[at])) change(at, c || path, count);
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const LogitsParams& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int slice = kMaxSlice, groups = 1;
  auto slices = [&] { return (p.V + slice - 1) / slice; };
  auto ctas = [&] { return (long long)p.B * slices() * groups; };
  while (ctas() < 4LL * sms && groups < p.T) groups = groups * 2 < p.T ? groups * 2 : p.T;
  while (ctas() < 2LL * sms && slice > 1024) slice /= 2;
  const int group_rows = (p.T + groups - 1) / groups;
  groups = (p.T + group_rows - 1) / group_rows;
  const long long blocks = ctas();
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  const size_t smem = (size_t)slice * ((p.num_bias ? 8 : 4) + 2);
  return launch_pdl(logits_kernel<T>, dim3((unsigned)blocks), dim3(kThreads), smem, stream, p, slice, slices(), groups,
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
