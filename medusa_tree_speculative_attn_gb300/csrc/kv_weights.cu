// The attention weight that every cached slot of a block-scaled cache has received: what
// eviction goes by.  For slot s of sequence b under KV head h, with the query rows r of the
// call (all new tokens', or the accepted path's) and lse_r as the attention returned it,
//   out[s] = decay * weights[s] (0 for a slot that is new) + sum_r exp(q_r . k_s * scale - lse_r).
//
// A row's weights need its softmax sum, so they cannot fall out of the attention's own pass;
// with the sum given, one pass over the keys is enough and no two CTAs share a slot: no
// atomics, the same bits in every run.
//
// As in attn_block8.cu the keys are the 16-row side of m16n8k16 products in fp16 (every E4M3
// code is exact there, and a query scaled to a power of two keeps its bits), converted in
// registers; a lane takes 16 consecutive bytes of a key row as four k-steps, and the queries
// lie in shared memory in that order, one 16-byte read for two k-steps.  A warp takes pages
// of its own, four in flight, and a slot's sum over rows is two shuffles at the end.
#include <cmath>

#include "serve.cuh"

namespace mt {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kP = 16;
constexpr int kFlight = 4;     // pages a warp keeps in flight
constexpr int kMaxRows = 256;  // query rows in shared memory at a time

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t r;
  memcpy(&r, &h, 4);
  return r;
}

// A page as one lane holds it: 16-byte chunks ch * 4 + tig of rows gid and gid + 8, and (of
// the lanes with tig 0) those slots' weights before the call.
template <int D>
struct Page {
  uint4 k[D / 64][2];
  float old[2];
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv_weights_kernel(const WeightsParams p, int chunks, int per_warp) {
  constexpr int NC = D / 64;
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* s_q = reinterpret_cast<uint4*>(smem);  // [tile of 8 rows][chunk][half][lane]
  const int most = min(kMaxRows, (p.rows + 7) & ~7);
  float2* s_row = reinterpret_cast<float2*>(smem + (size_t)most * D * 2);  // score -> base 2, lse in base 2
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  const int h = blockIdx.x % p.Hkv, chunk = blockIdx.x / p.Hkv % chunks, b = blockIdx.x / p.Hkv / chunks;
  pdl_wait();
  const int L = p.seq_lens[b];
  if ((long long)L > (long long)p.max_blocks * kP) {
    if (chunk == 0 && threadIdx.x == 0) set_status(p.status, kStPages);
    return;
  }
  const int npages = (max(L, 0) + kP - 1) / kP;
  const int first = chunk * per_warp * kWarps + warp;  // this warp's pages: first, first + 4, ...
  if (chunk * per_warp * kWarps >= npages) return;
  int nodes = p.T;
  const int* path = nullptr;
  if (p.accept_path) {
    path = p.accept_path + (size_t)b * (p.max_depth + 1);
    nodes = p.accept_len[b] + 1;
    bool stray = nodes < 1 || nodes > p.max_depth + 1;
    if (!stray)
      for (int i = lane; i < nodes; i += 32) stray = stray || (unsigned)path[i] >= (unsigned)p.T;
    if (__any_sync(0xffffffffu, stray)) {  // the same in every warp
      if (threadIdx.x == 0) set_status(p.status, kStPages);
      return;
    }
  }
  const int rows = nodes * p.g;
  const int mine = min(per_warp, (npages - first + kWarps - 1) / kWarps);  // perhaps below 1
  const int* bt = p.block_tables + (size_t)b * p.max_blocks;
  const int prev = p.prev_lens ? p.prev_lens[b] : L;

  for (int r0 = 0; r0 < rows; r0 += kMaxRows) {
    const int n = min(kMaxRows, rows - r0), tiles = (n + 7) / 8;
    const float* before = r0 == 0 ? p.weights : p.out;  // later rows add to what the earlier ones left
    const float decay = r0 == 0 ? p.decay : 1.f;
    // ids and key scales of 32 pages, a lane each (per_warp <= 32)
    const int id = lane < mine ? bt[first + lane * kWarps] : -1;
    const bool good = id >= 0 && id < p.num_pages;
    const float ks = good ? __ldg(p.k_scales + (size_t)id * p.Hkv + h) : 0.f;
    if (lane < mine && !good) set_status(p.status, kStPages);
    auto load = [&](Page<D>& x, int i) {
      const int pg = __shfl_sync(0xffffffffu, good ? id : -1, i & 31);
      if (i >= mine || pg < 0) return;
      const size_t at = (size_t)pg * p.Hkv + h;
      const uint8_t* k = static_cast<const uint8_t*>(p.k_cache) + at * kP * D;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          x.k[c][r] = __ldg(reinterpret_cast<const uint4*>(k + (gid + 8 * r) * D + (c * 4 + tig) * 16));
      if (tig == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int slot = (first + i * kWarps) * kP + gid + 8 * r;
          x.old[r] = slot < (r0 == 0 ? prev : L) ? before[at * kP + gid + 8 * r] * decay : 0.f;
        }
      }
    };
    Page<D> ring[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) load(ring[u], u);
    // the queries: a warp a row of 8, lanes as they multiply
    if (r0 > 0) __syncthreads();
    for (int t = warp; t < tiles; t += kWarps) {
      const int row = t * 8 + gid;
      Row8<T> raw[2 * NC];
#pragma unroll
      for (int x = 0; x < 2 * NC; ++x) raw[x].zero();
      float l2 = INFINITY;
      if (row < n) {
        const int at = (r0 + row) / p.g, node = path ? path[at] : at, head = h * p.g + (r0 + row) % p.g;
        const size_t q = ((size_t)b * p.T + node) * p.Hq + head;
#pragma unroll
        for (int x = 0; x < 2 * NC; ++x)
          raw[x].load(static_cast<const T*>(p.q) + q * D + (x / 2) * 64 + tig * 16 + (x % 2) * 8);
        l2 = p.lse[q] * 1.4426950408889634f;
      }
      AbsMax<T> top;
#pragma unroll
      for (int x = 0; x < 2 * NC; ++x) top.add(raw[x]);
      float amax = top.get();
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^8 <= scaled maximum < 2^9: a bf16 keeps its bits down to 2^-25 of it, an fp16 to 2^-22
      const int ex = amax > 0.f ? (int)(__float_as_uint(amax) >> 23) - 127 : 0;
      const int k = min(max(8 - ex, -120), 120);
      const float f2 = __uint_as_float((uint32_t)(127 + k) << 23);
      const float c = amax < INFINITY ? p.scale_log2 * __uint_as_float((uint32_t)(127 - k) << 23)
                                      : __int_as_float(0x7fffffff);
      if (tig == 0) s_row[row] = make_float2(row < n ? c : 0.f, l2);
#pragma unroll
      for (int x = 0; x < 2 * NC; ++x) {  // 8 columns: two k-steps of four
        float f[8];
        raw[x].to_f(f);
        s_q[(t * 2 * NC + x) * 32 + lane] = make_uint4(pack_h2(f[0] * f2, f[1] * f2), pack_h2(f[2] * f2, f[3] * f2),
                                                       pack_h2(f[4] * f2, f[5] * f2), pack_h2(f[6] * f2, f[7] * f2));
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int i0 = 0; i0 < mine; i0 += kFlight) {
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int i = i0 + u;
        if (i >= mine) break;
        const int pg = __shfl_sync(0xffffffffu, good ? id : -1, i);
        const float scale = __shfl_sync(0xffffffffu, ks, i);
        uint32_t a[NC][4][4];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const uint4 w0 = ring[u].k[c][0], w1 = ring[u].k[c][1];
          const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            a[c][x][0] = e4m3x2_to_h2(x0[x] & 0xffffu);
            a[c][x][1] = e4m3x2_to_h2(x1[x] & 0xffffu);
            a[c][x][2] = e4m3x2_to_h2(x0[x] >> 16);
            a[c][x][3] = e4m3x2_to_h2(x1[x] >> 16);
          }
        }
        const float old[2] = {ring[u].old[0], ring[u].old[1]};
        load(ring[u], i + kFlight);
        float sum[2] = {0.f, 0.f};
#pragma unroll 2
        for (int t = 0; t < tiles; ++t) {
          float s[4] = {0.f, 0.f, 0.f, 0.f};
          const float4 rc = *reinterpret_cast<const float4*>(s_row + t * 8 + 2 * tig);
#pragma unroll
          for (int x = 0; x < 2 * NC; ++x) {
            const uint4 q = s_q[(t * 2 * NC + x) * 32 + lane];
            mma(s, a[x / 2][2 * (x % 2)], q.x, q.y);
            mma(s, a[x / 2][2 * (x % 2) + 1], q.z, q.w);
          }
          // element e: row 2 tig + (e & 1), key gid + 8 (e >> 1)
          const float c0 = rc.x * scale, c1 = rc.z * scale;
          sum[0] += fast_exp2(fmaf(s[0], c0, -rc.y)) + fast_exp2(fmaf(s[1], c1, -rc.w));
          sum[1] += fast_exp2(fmaf(s[2], c0, -rc.y)) + fast_exp2(fmaf(s[3], c1, -rc.w));
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
          sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
          const int slot = (first + i * kWarps) * kP + gid + 8 * r;
          if (tig == 0 && pg >= 0 && slot < L) p.out[((size_t)pg * p.Hkv + h) * kP + gid + 8 * r] = old[r] + sum[r];
        }
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_t(const WeightsParams& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int per_warp = 32;
  auto chunks = [&] { return (p.max_blocks + per_warp * kWarps - 1) / (per_warp * kWarps); };
  while (per_warp > 1 && (long long)p.B * p.Hkv * chunks() < 16LL * sms) per_warp /= 2;
  const long long blocks = (long long)p.B * p.Hkv * chunks();
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  const int most = p.rows < kMaxRows ? (p.rows + 7) & ~7 : kMaxRows;
  const size_t smem = (size_t)most * (D * 2 + sizeof(float2));
  e = cudaFuncSetAttribute(kv_weights_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kMaxRows * (D * 2 + (int)sizeof(float2)));
  if (e != cudaSuccess) return e;
  return launch_pdl(kv_weights_kernel<T, D>, dim3((unsigned)blocks), dim3(kThreads), smem, stream, p, chunks(), per_warp);
}

}  // namespace

cudaError_t launch_kv_weights(const WeightsParams& p, int dtype, cudaStream_t stream) {
  if (p.D == 64)
    return dtype == 1 ? launch_t<__half, 64>(p, stream) : launch_t<__nv_bfloat16, 64>(p, stream);
  return dtype == 1 ? launch_t<__half, 128>(p, stream) : launch_t<__nv_bfloat16, 128>(p, stream);
}

}  // namespace mt
