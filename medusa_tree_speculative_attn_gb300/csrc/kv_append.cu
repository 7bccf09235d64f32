// Appending new keys and values to the paged cache, with the position rotation
// of the keys on the way (the other half of vLLM issue 1171's "update block
// tables": how a prompt's or an accepted path's rows get into the pages).
//
// Sequence b's new rows go to logical slots seq_lens[b] + i; a row's key is
// rotated at its slot (rounded once to the act dtype, the same arithmetic as
// the tree attention's own rotation).  The cache holds the act dtype, E4M3
// codes under one scale, or E4M3 codes with a scale for each block, one page
// (16 slots) of one KV head:
//   scale = block_scale(largest magnitude of the rows), and a page whose first
//   slot is older keeps the larger of its scale and the new rows'; when that
//   grows, the page's older codes are re-encoded under the new scale.
//
// Bound by memory: every row is read once and written once.  One warp owns one
// (page, KV head) with both its K and its V: the block's maximum is a warp
// reduction, nothing is shared between warps, and all 16 rows' loads are in
// flight together.  Warps of neighbouring heads sit in one CTA, so the page's
// (cos, sin) rows come from L1 after the first.
//
// Which page a warp takes, without a prefix over the batch: with row offsets o,
// sequence b touches at most floor(o[b+1]/16) - floor(o[b]/16) + 2 pages (n new
// rows span at most floor((n + 30) / 16)), so items floor(o[b]/16) + 2b and on
// are its own, and b is found by bisection.
#include "serve.cuh"

namespace mt {

namespace {

constexpr int kWarps = 8;
constexpr int kP = 16;  // slots per page

// What one (page, head, K or V) does with its rows in registers: the block's
// maximum and scale, the older rows' codes, the new rows' codes.
template <typename T, int D, int STEPS>
__device__ __forceinline__ void store_rows(const AppendParams& a, Row8<T> (&lo)[STEPS], Row8<T> (&hi)[STEPS], int sub,
                                           int c, int r0, int r1, long long block, void* cache, float* scales,
                                           float one_scale) {
  constexpr int RPS = 16 / STEPS;
  const size_t base = (size_t)block * kP * D;  // the (page, head)'s 16 rows
  if (a.mode == kCacheAct) {
    T* dst = static_cast<T*>(cache) + base;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = s * RPS + sub;
      if (r >= r0 && r < r1) {
        lo[s].store(dst + r * D + 8 * c);
        hi[s].store(dst + r * D + D / 2 + 8 * c);
      }
    }
    return;
  }
  uint8_t* dst = static_cast<uint8_t*>(cache) + base;
  float scale = one_scale;
  if (a.mode == kCacheBlock8) {
    float amax = 0.f;  // rows outside [r0, r1) are zero; fmaxf passes a NaN over
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      float xl[8], xh[8];
      lo[s].to_f(xl);
      hi[s].to_f(xh);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(xl[e]), fabsf(xh[e])));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    scale = block_scale(amax);
    if (r0 > 0) {
      const float old = scales[block];
      if (old >= scale) {
        scale = old;
      } else {
        const float f = old / scale;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const int r = s * RPS + sub;
          if (r < r0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint2* p = reinterpret_cast<uint2*>(dst + r * D + h * (D / 2) + 8 * c);
              float x[8];
              e4m3x8_to_f(*p, x);
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] *= f;
              *p = e4m3x8_of(x);
            }
          }
        }
      }
    }
    __syncwarp();  // every lane has read the old scale
    if (sub == 0 && c == 0) scales[block] = scale;
  }
  // a power of two divides exactly by its inverse; another scale (a cache's own)
  // takes the division that the tree attention's writes take
  const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0u;
  const float inv = 1.f / scale;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = s * RPS + sub;
    if (r < r0 || r >= r1) continue;
    float x[8];
    lo[s].to_f(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = pow2 ? x[e] * inv : x[e] / scale;
    *reinterpret_cast<uint2*>(dst + r * D + 8 * c) = e4m3x8_of(x);
    hi[s].to_f(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = pow2 ? x[e] * inv : x[e] / scale;
    *reinterpret_cast<uint2*>(dst + r * D + D / 2 + 8 * c) = e4m3x8_of(x);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(AppendParams a, long long items) {
  constexpr int LPR = D / 16;    // lanes per row
  constexpr int RPS = 32 / LPR;  // rows per step
  constexpr int STEPS = kP / RPS;
  const long long gw = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long item = gw / a.Hkv;
  const int head = (int)(gw - item * a.Hkv);
  if (item >= items) return;
  pdl_wait();
  const int lane = threadIdx.x & 31, sub = lane / LPR, c = lane % LPR;

  // malformed offsets are reported even where no item falls on them
  if (a.row_offsets && gw < a.B && lane == 0) {
    const int o0 = a.row_offsets[gw], o1 = a.row_offsets[gw + 1];
    if (o0 < 0 || o1 < o0 || o1 > a.N) set_status(a.status, kStPages);
  }

  // the item's sequence, its rows and its page
  int b, pg;  // pg: the item's page counted from the first one written
  long long first_row = 0;
  int n;
  if (a.row_offsets) {
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.row_offsets[mid] / kP + 2LL * mid <= item) lo = mid; else hi = mid - 1;
    }
    b = lo;
    const int o0 = a.row_offsets[b], o1 = a.row_offsets[b + 1];
    if (o0 < 0 || o1 < o0 || o1 > a.N) return;
    pg = (int)(item - (o0 / kP + 2LL * b));
    if (pg < 0) return;  // offsets that start above 0: items before the first sequence
    first_row = o0;
    n = o1 - o0;
  } else {
    const int per = (a.max_depth + 1 + kP - 1) / kP + 1;
    b = (int)(item / per);
    pg = (int)(item - (long long)b * per);
    n = a.accept_len[b] + 1;
    if (n < 1 || n > a.max_depth + 1) {
      if (lane == 0 && a.seq_lens[b] >= 0) set_status(a.status, kStPages);
      return;
    }
  }
  const int len = a.seq_lens[b];
  if (len < 0 || n == 0) return;  // no sequence here, or nothing new
  if ((long long)len + n > (long long)a.max_blocks * kP) {
    if (lane == 0) set_status(a.status, kStPages);
    return;
  }
  pg += len / kP;
  if (pg > (len + n - 1) / kP) return;
  const int r0 = max(len - pg * kP, 0), r1 = min(len + n - pg * kP, kP);
  const int page = a.block_tables[(size_t)b * a.max_blocks + pg];
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) set_status(a.status, kStPages);
    return;
  }
  if (a.rope && pg * kP + r1 > a.max_pos) {
    if (lane == 0) set_status(a.status, kStPosition);
    return;
  }

  // all rows' loads first
  Row8<T> kl[STEPS], kh[STEPS], vl[STEPS], vh[STEPS];
  bool bad = false;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = s * RPS + sub;
    bool live = r >= r0 && r < r1;
    long long row = 0;
    if (live) {
      const int i = pg * kP + r - len;
      if (a.row_offsets) {
        row = first_row + i;
      } else {
        const int node = a.accept_path[(size_t)b * (a.max_depth + 1) + i];
        live = node >= 0 && node < a.T;
        bad = bad || !live;
        row = (long long)b * a.T + node;
      }
    }
    if (live) {
      const T* kp = static_cast<const T*>(a.k) + row * a.k_st[0] + head * a.k_st[1] + 8 * c;
      const T* vp = static_cast<const T*>(a.v) + row * a.v_st[0] + head * a.v_st[1] + 8 * c;
      kl[s].load_stream(kp);
      kh[s].load_stream(kp + D / 2);
      vl[s].load_stream(vp);
      vh[s].load_stream(vp + D / 2);
    } else {
      kl[s].zero();
      kh[s].zero();
      vl[s].zero();
      vh[s].zero();
    }
  }
  if (__any_sync(0xffffffffu, bad)) {  // a node outside the tree: the page is left alone
    if (lane == 0) set_status(a.status, kStPages);
    return;
  }
  if (a.rope) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = s * RPS + sub;
      if (r < r0 || r >= r1) continue;
      const float4* cs = reinterpret_cast<const float4*>(a.rope + (size_t)(pg * kP + r) * (D / 2) + 8 * c);
      float xl[8], xh[8];
      kl[s].to_f(xl);
      kh[s].to_f(xh);
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
      kl[s].from_f(xl);
      kh[s].from_f(xh);
    }
  }
  const long long block = (long long)page * a.Hkv + head;
  store_rows<T, D, STEPS>(a, kl, kh, sub, c, r0, r1, block, a.k_cache, a.k_scales, a.k_scale);
  store_rows<T, D, STEPS>(a, vl, vh, sub, c, r0, r1, block, a.v_cache, a.v_scales, a.v_scale);
}

template <typename T, int D>
cudaError_t launch_t(const AppendParams& a, cudaStream_t stream) {
  const long long items = a.row_offsets ? (long long)a.N / kP + 2LL * a.B
                                        : (long long)a.B * ((a.max_depth + 1 + kP - 1) / kP + 1);
  const long long blocks = (items * a.Hkv + kWarps - 1) / kWarps;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  return launch_pdl(append_kernel<T, D>, dim3((unsigned)blocks), dim3(kWarps * 32), 0, stream, a, items);
}

template <typename T>
cudaError_t launch_d(const AppendParams& a, cudaStream_t stream) {
  return a.D == 64 ? launch_t<T, 64>(a, stream) : launch_t<T, 128>(a, stream);
}

}  // namespace

cudaError_t launch_append(const AppendParams& a, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case 0: return launch_d<float>(a, stream);
    case 1: return launch_d<__half>(a, stream);
    default: return launch_d<__nv_bfloat16>(a, stream);
  }
}

}  // namespace mt
