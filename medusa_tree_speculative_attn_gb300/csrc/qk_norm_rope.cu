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
// shuffles.  A warp takes kSteps times that many heads of one token: the
// token's (cos, sin) pairs are loaded once for all of them, and all rows are in
// flight before the first is used.
#include "serve.cuh"

namespace mt {

namespace {

constexpr int kWarps = 8;
constexpr int kSteps = 2;

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_kernel(NormRopeParams a) {
  constexpr int LPR = D / 16;    // lanes per row
  constexpr int RPS = 32 / LPR;  // rows per step
  constexpr int HPW = RPS * kSteps;
  const int lane = threadIdx.x & 31, sub = lane / LPR, c = lane % LPR;
  const int nq = (a.Hq + HPW - 1) / HPW, nk = (a.Hkv + HPW - 1) / HPW;
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long tok = item / (nq + nk);
  if (tok >= a.N) return;
  pdl_wait();
  int part = (int)(item - tok * (nq + nk));
  const bool is_q = part < nq;
  if (!is_q) part -= nq;
  const int H = is_q ? a.Hq : a.Hkv;
  const long long* st = is_q ? a.q_st : a.k_st;
  const T* src = static_cast<const T*>(is_q ? a.q : a.k) + tok * st[0];
  const int pos = a.positions ? a.positions[tok] : 0;
  Row8<T> lo[kSteps], hi[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int h = part * HPW + s * RPS + sub;
    if (h < H) {
      const T* p = src + h * st[1] + 8 * c;
      lo[s].load_stream(p);
      hi[s].load_stream(p + D / 2);
    } else {
      lo[s].zero();
      hi[s].zero();
    }
  }
  if (pos < 0) return;  // no token here: its rows are left as they were
  float4 cs[4];
  if (a.rope) {
    if (pos >= a.max_pos) {
      if (lane == 0) set_status(a.status, kStPosition);
      return;
    }
    const float4* t = reinterpret_cast<const float4*>(a.rope + (size_t)pos * (D / 2) + 8 * c);
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = t[e];
  }
  const T* w = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
  Row8<T> wl, wh;
  if (w) {
    wl.load(w + 8 * c);
    wh.load(w + D / 2 + 8 * c);
  }
  const long long* so = is_q ? a.qo_st : a.ko_st;
  T* dst = static_cast<T*>(is_q ? a.q_out : a.k_out) + tok * so[0];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int h = part * HPW + s * RPS + sub;
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
        const float4 t = cs[e / 2];  // (cos, sin) of pairs e and e + 1
        float l0, h0, l1, h1;
        rope_pair(xl[e], xh[e], t.x, t.y, l0, h0);
        rope_pair(xl[e + 1], xh[e + 1], t.z, t.w, l1, h1);
        xl[e] = l0;
        xh[e] = h0;
        xl[e + 1] = l1;
        xh[e + 1] = h1;
      }
    }
    if (h < H) {
      T* p = dst + h * so[1] + 8 * c;
      lo[s].from_f(xl);
      hi[s].from_f(xh);
      lo[s].store(p);
      hi[s].store(p + D / 2);
    }
  }
}

template <typename T, int D>
cudaError_t launch_t(const NormRopeParams& a, cudaStream_t stream) {
  constexpr int HPW = 32 / (D / 16) * kSteps;
  const long long items = (long long)a.N * ((a.Hq + HPW - 1) / HPW + (a.Hkv + HPW - 1) / HPW);
  const long long blocks = (items + kWarps - 1) / kWarps;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
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
