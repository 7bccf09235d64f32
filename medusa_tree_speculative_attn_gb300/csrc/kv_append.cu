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
// Bound by memory: every row is read once and written once.  One warp owns the
// keys or the values of one (page, KV head): the block's maximum is a warp
// reduction, nothing is shared between warps, all 16 rows' loads are in flight
// together, and they are asked for before the page's number is known.  Warps of
// neighbouring heads sit in one CTA, so the page's (cos, sin) rows come from L1
// after the first.
//
// Which page a warp takes, without a prefix over the batch: with row offsets o,
// sequence b touches at most floor(o[b+1]/16) - floor(o[b]/16) + 2 pages (n new
// rows span at most floor((n + 30) / 16)), so items floor(o[b]/16) + 2b and on
// are its own, and b is found by a 32-wide search.
//
// 8 sequences of 512 to 1500 tokens, 32 heads of 128 columns, fp16 to an fp16
// cache: 48 us (306 MB, 6.3 TB/s, 93 % of a copy).  16 of 100 to 4000, 8 heads,
// bf16 to block scales: 44 us (239 MB, 5.4 TB/s, 79 %): a warp has to hold a whole
// block before it can write the first code.  64 single tokens: 3.2 us, a launch.
#include "serve.cuh"

namespace mt {

namespace {

constexpr int kWarps = 4;
constexpr int kP = 16;  // slots per page

// What one (page, head, K or V) does with its rows in registers: the block's
// maximum and scale, the older rows' codes, the new rows' codes.
template <typename T, int D, int STEPS, int MODE>
__device__ __forceinline__ void store_rows(Row8<T> (&lo)[STEPS], Row8<T> (&hi)[STEPS], int sub, int c, int r0, int r1,
                                           long long block, void* cache, float* scales, float one_scale, float old) {
  constexpr int RPS = 16 / STEPS;
  const size_t base = (size_t)block * kP * D;  // the (page, head)'s 16 rows
  if (MODE == kCacheAct) {
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
  if (MODE == kCacheBlock8) {
    AbsMax<T> top;  // rows outside [r0, r1) are zero
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      top.add(lo[s]);
      top.add(hi[s]);
    }
    float amax = top.get();
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    scale = block_scale(amax);
    if (r0 > 0) {
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
    if (sub == 0 && c == 0) scales[block] = scale;
  }
  // a power of two divides exactly by its inverse; a scale that is none takes
  // the division that the tree attention's writes take
  const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0u;
  const float inv = 1.f / scale;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = s * RPS + sub;
    if (r < r0 || r >= r1) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[8];
      if (h) hi[s].to_f(x); else lo[s].to_f(x);
      if (pow2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] /= scale;
      }
      *reinterpret_cast<uint2*>(dst + r * D + h * (D / 2) + 8 * c) = e4m3x8_of(x);
    }
  }
}

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 4 ? 5 : 7) append_kernel(AppendParams a, long long items) {
  constexpr int LPR = D / 16;    // lanes per row
  constexpr int RPS = 32 / LPR;  // rows per step
  constexpr int STEPS = kP / RPS;
  const long long gw = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long item = gw / (2 * a.Hkv);
  if (item >= items) return;
  const int unit = (int)(gw - item * (2 * a.Hkv));
  const bool is_v = unit >= a.Hkv;
  const int head = is_v ? unit - a.Hkv : unit;
  pdl_wait();
  const int lane = threadIdx.x & 31, sub = lane / LPR, c = lane % LPR;

  // malformed offsets are reported even where no item falls on them
  if (a.row_offsets && gw < a.B && lane == 0) {
    const int o0 = a.row_offsets[gw], o1 = a.row_offsets[gw + 1];
    if (o0 < 0 || o1 < o0 || o1 > a.N) set_status(a.status, kStPages);
  }

  // the item's sequence, its rows and its page.  The search is 32 wide: each
  // lane looks at one sequence, so that up to 32 sequences take one round trip
  // to memory (the length comes with it), up to 1024 two.
  int b = 0, pg;  // pg: the item's page counted from the first one written
  long long first_row = 0;
  int n, len;
  if (a.row_offsets) {
    int lo = 0, step = 1;
    while (step * 32 < a.B) step *= 32;
    int o0 = 0, o1 = 0, l = 0;
    for (; step > 0; step /= 32) {
      const int mine = lo + lane * step;
      bool at = false;
      if (mine < a.B) {
        o0 = a.row_offsets[mine];
        if (step == 1) {
          o1 = a.row_offsets[mine + 1];
          l = a.seq_lens[mine];
        }
        at = o0 / kP + 2LL * mine <= item;
      }
      // the last lane of the leading ones (lane 0 where even it is past)
      const unsigned yes = __ballot_sync(0xffffffffu, at);
      const int last = max(__ffs(~yes) - 2, yes == 0xffffffffu ? 31 : 0);
      lo += last * step;
      if (step == 1) {
        o0 = __shfl_sync(0xffffffffu, o0, last);
        o1 = __shfl_sync(0xffffffffu, o1, last);
        l = __shfl_sync(0xffffffffu, l, last);
      }
    }
    b = lo;
    len = l;
    if (o0 < 0 || o1 < o0 || o1 > a.N) return;
    const long long at = item - (o0 / kP + 2LL * b);
    if (at < 0) return;  // offsets that start above 0: items before the first sequence
    pg = (int)at;
    first_row = o0;
    n = o1 - o0;
  } else {
    const int per = (a.max_depth + 1 + kP - 1) / kP + 1;
    b = (int)(item / per);
    pg = (int)(item - (long long)b * per);
    n = a.accept_len[b] + 1;
    len = a.seq_lens[b];
    // a node outside the tree anywhere on the path (of 64 at most), and nothing is written
    const int* path = a.accept_path + (size_t)b * (a.max_depth + 1);
    const unsigned n0 = lane < n && lane <= a.max_depth ? (unsigned)path[lane] : 0u;
    const unsigned n1 = lane + 32 < n && lane + 32 <= a.max_depth ? (unsigned)path[lane + 32] : 0u;
    const bool stray = max(n0, n1) >= (unsigned)a.T;
    if (n < 1 || n > a.max_depth + 1 || __any_sync(0xffffffffu, stray)) {
      if (lane == 0 && len >= 0) set_status(a.status, kStPages);
      return;
    }
  }
  if (len < 0 || n == 0) return;  // no sequence here, or nothing new
  if ((long long)len + n > (long long)a.max_blocks * kP) {
    if (lane == 0) set_status(a.status, kStPages);
    return;
  }
  pg += len / kP;
  if (pg > (len + n - 1) / kP) return;
  const int r0 = max(len - pg * kP, 0), r1 = min(len + n - pg * kP, kP);
  const int page = a.block_tables[(size_t)b * a.max_blocks + pg];

  // all rows' loads, before the page is known
  const T* src = static_cast<const T*>(is_v ? a.v : a.k);
  const long long st0 = is_v ? a.v_st[0] : a.k_st[0], st1 = is_v ? a.v_st[1] : a.k_st[1];
  Row8<T> lo[STEPS], hi[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = s * RPS + sub;
    const bool live = r >= r0 && r < r1;
    long long row = 0;
    if (live) {
      const int i = pg * kP + r - len;
      if (a.row_offsets) row = first_row + i;
      else row = (long long)b * a.T + a.accept_path[(size_t)b * (a.max_depth + 1) + i];
    }
    if (live) {
      const T* p = src + row * st0 + head * st1 + 8 * c;
      lo[s].load_stream(p);
      hi[s].load_stream(p + D / 2);
    } else {
      lo[s].zero();
      hi[s].zero();
    }
  }
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) set_status(a.status, kStPages);
    return;
  }
  if (a.rope && pg * kP + r1 > a.max_pos) {
    if (lane == 0) set_status(a.status, kStPosition);
    return;
  }
  const long long block = (long long)page * a.Hkv + head;
  float* scales = is_v ? a.v_scales : a.k_scales;
  const float old = MODE == kCacheBlock8 && r0 > 0 ? scales[block] : 0.f;
  if (a.rope && !is_v) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = s * RPS + sub;
      if (r < r0 || r >= r1) continue;
      const float4* cs = reinterpret_cast<const float4*>(a.rope + (size_t)(pg * kP + r) * (D / 2) + 8 * c);
      float xl[8], xh[8];
      lo[s].to_f(xl);
      hi[s].to_f(xh);
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
      lo[s].from_f(xl);
      hi[s].from_f(xh);
    }
  }
  __syncwarp();  // every lane has read the old scale
  store_rows<T, D, STEPS, MODE>(lo, hi, sub, c, r0, r1, block, is_v ? a.v_cache : a.k_cache, scales,
                                is_v ? a.v_scale : a.k_scale, old);
}

template <typename T, int D, int MODE>
cudaError_t launch_t(const AppendParams& a, cudaStream_t stream) {
  const long long items = a.row_offsets ? (long long)a.N / kP + 2LL * a.B
                                        : (long long)a.B * ((a.max_depth + 1 + kP - 1) / kP + 1);
  const long long blocks = (items * 2 * a.Hkv + kWarps - 1) / kWarps;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  return launch_pdl(append_kernel<T, D, MODE>, dim3((unsigned)blocks), dim3(kWarps * 32), 0, stream, a, items);
}

template <typename T, int D>
cudaError_t launch_m(const AppendParams& a, cudaStream_t stream) {
  switch (a.mode) {
    case kCacheAct: return launch_t<T, D, kCacheAct>(a, stream);
    case kCacheE4m3: return launch_t<T, D, kCacheE4m3>(a, stream);
    default: return launch_t<T, D, kCacheBlock8>(a, stream);
  }
}

template <typename T>
cudaError_t launch_d(const AppendParams& a, cudaStream_t stream) {
  return a.D == 64 ? launch_m<T, 64>(a, stream) : launch_m<T, 128>(a, stream);
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
