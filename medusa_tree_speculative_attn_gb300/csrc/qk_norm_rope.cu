// Root-mean-square norms of every query and key head and the position
// rotation, in one pass.  For one head row x of D elements, in fp32:
//   y = x * rsqrt(mean(x^2) + eps) * w      (skipped without weights)
//   lo' = lo*c - hi*s,  hi' = hi*c + lo*s   (skipped without a RoPE table;
//                                            each product and sum rounded)
// and one rounding to the act dtype at the end.  The same rotation, in the
// same arithmetic, as the tree attention applies by itself
// (TensorRT-LLM issue 1946, position offsets for Medusa tokens).
//
// Bound by memory: each row is read and written once.  A row is D/16 lanes of
// two 16-byte chunks (columns [8k, 8k + 8) and the same of the upper half), so
// the rotation's pairs sit in one lane and the norm's sum takes log2(D/16)
// shuffles.  A warp takes kSteps times that many heads of one token, whose
// (cos, sin) pairs are loaded once for all of them, and then the same heads of
// further tokens (its weights stay in registers): the next token's rows and
// pairs, and the position of the one after, are in flight while a token is
// worked on.
//
// 32 query and 8 KV heads of 128 columns, bf16, views of one projection: 16384
// tokens 55 us (344 MB, 6.2 TB/s, 92 % of a copy), 1024 tokens 5.1 us, half of it
// the launch and the first loads' latency.
#include <atomic>

#include "serve.cuh"

namespace mt {

namespace {

constexpr int kWarps = 4;
constexpr int kSteps = 2;

// The (cos, sin) pairs of one token that a lane rotates with.
struct Pairs {
  float4 t[4];  // pairs 2e and 2e + 1
  __device__ __forceinline__ void load(const NormRopeParams& a, int pos, int D, int c) {
    if (!a.rope || pos < 0 || pos >= a.max_pos) return;
    const float4* p = reinterpret_cast<const float4*>(a.rope + (size_t)pos * (D / 2) + 8 * c);
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = p[e];
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_kernel(NormRopeParams a) {
  constexpr int LPR = D / 16;    // lanes per row
  constexpr int RPS = 32 / LPR;  // rows per step
  constexpr int HPW = RPS * kSteps;
  const int lane = threadIdx.x & 31, sub = lane / LPR, c = lane % LPR;
  const int nq = (a.Hq + HPW - 1) / HPW, parts = nq + (a.Hkv + HPW - 1) / HPW;
  const long long warps = (long long)gridDim.x * kWarps;
  const long long gw = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  // neighbouring warps take the parts of one token; a warp keeps its part
  const long long stride = warps / parts;
  long long tok = gw / parts;
  if (tok >= stride || tok >= a.N) return;
  int part = (int)(gw - tok * parts);
  pdl_wait();
  const bool is_q = part < nq;
  if (!is_q) part -= nq;
  const int H = is_q ? a.Hq : a.Hkv, h0 = part * HPW + sub;
  const long long st0 = is_q ? a.q_st[0] : a.k_st[0], st1 = is_q ? a.q_st[1] : a.k_st[1];
  const long long so0 = is_q ? a.qo_st[0] : a.ko_st[0], so1 = is_q ? a.qo_st[1] : a.ko_st[1];
  const T* src = static_cast<const T*>(is_q ? a.q : a.k) + h0 * st1 + 8 * c;
  T* dst = static_cast<T*>(is_q ? a.q_out : a.k_out) + h0 * so1 + 8 * c;
  const T* w = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
  auto load_rows = [&](long long t, Row8<T>(&lo)[kSteps], Row8<T>(&hi)[kSteps]) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (h0 + s * RPS < H) {
        const T* p = src + t * st0 + s * RPS * st1;
        lo[s].load_stream(p);
        hi[s].load_stream(p + D / 2);
      } else {
        lo[s].zero();
        hi[s].zero();
      }
    }
  };
  auto position = [&](long long t) { return t < a.N && a.positions ? a.positions[t] : 0; };
  Row8<T> lo[kSteps], hi[kSteps], nlo[kSteps], nhi[kSteps], wl, wh;
  Pairs cs, ncs;
  int pos = position(tok), npos = position(tok + stride);
  load_rows(tok, lo, hi);
  if (w) {
    wl.load(w + 8 * c);
    wh.load(w + D / 2 + 8 * c);
  }
  cs.load(a, pos, D, c);
  while (true) {
    const long long next = tok + stride;
    const bool more = next < a.N;
    const int nnpos = position(next + stride);
    if (more) {
      load_rows(next, nlo, nhi);
      ncs.load(a, npos, D, c);
    }
    const bool past = a.rope && pos >= a.max_pos;
    if (past && lane == 0) set_status(a.status, kStPosition);
    if (pos >= 0 && !past) {  // else: no token here, its rows are left as they were
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        float xl[8], xh[8];
        lo[s].to_f(xl);
        hi[s].to_f(xh);
        if (w) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(xl[e], xl[e], fmaf(xh[e], xh[e], ss));
#pragma unroll
          for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          const float inv = rsqrtf(ss * (1.f / D) + a.eps);
          float fl[8], fh[8];
          wl.to_f(fl);
          wh.to_f(fh);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            xl[e] = xl[e] * inv * fl[e];
            xh[e] = xh[e] * inv * fh[e];
          }
        }
        if (a.rope) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float4 t = cs.t[e / 2];
            float l0, h0v, l1, h1v;
            rope_pair(xl[e], xh[e], t.x, t.y, l0, h0v);
            rope_pair(xl[e + 1], xh[e + 1], t.z, t.w, l1, h1v);
            xl[e] = l0;
            xh[e] = h0v;
            xl[e + 1] = l1;
            xh[e + 1] = h1v;
          }
        }
        if (h0 + s * RPS < H) {
          T* p = dst + tok * so0 + s * RPS * so1;
          lo[s].from_f(xl);
          hi[s].from_f(xh);
          lo[s].store(p);
          hi[s].store(p + D / 2);
        }
      }
    }
    if (!more) break;
    tok = next;
    pos = npos;
    npos = nnpos;
    cs = ncs;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      lo[s] = nlo[s];
      hi[s] = nhi[s];
    }
  }
}

constexpr int kMaxDevices = 64;

template <typename T, int D>
cudaError_t launch_t(const NormRopeParams& a, cudaStream_t stream) {
  constexpr int HPW = 32 / (D / 16) * kSteps;
  // one resident wave at most, looked up once per device
  static std::atomic<int> resident[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int wave = dev >= 0 && dev < kMaxDevices ? resident[dev].load(std::memory_order_relaxed) : 0;
  if (wave <= 0) {
    int per_sm = 0, sms = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, norm_rope_kernel<T, D>, kWarps * 32, 0);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    wave = (per_sm < 1 ? 1 : per_sm) * sms;
    if (dev >= 0 && dev < kMaxDevices) resident[dev].store(wave, std::memory_order_relaxed);
  }
  const long long parts = (a.Hq + HPW - 1) / HPW + (a.Hkv + HPW - 1) / HPW;
  long long blocks = (a.N * parts + kWarps - 1) / kWarps;
  const long long least = (parts + kWarps - 1) / kWarps;  // a whole token's parts
  if (blocks > wave) blocks = wave > least ? wave : least;
  return launch_pdl(norm_rope_kernel<T, D>, dim3((unsigned)blocks), dim3(kWarps * 32), 0, stream, a);
}

template <typename T>
cudaError_t launch_d(const NormRopeParams& a, cudaStream_t stream) {
  return a.D == 64 ? launch_t<T, 64>(a, stream) : launch_t<T, 128>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& a, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case 0: return launch_d<float>(a, stream);
    case 1: return launch_d<__half>(a, stream);
    default: return launch_d<__nv_bfloat16>(a, stream);
  }
}

}  // namespace mt
