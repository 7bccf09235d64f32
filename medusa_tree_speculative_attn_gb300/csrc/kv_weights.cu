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
// lie in shared memory in that order, one 16-byte read for two k-steps.  Persistent CTAs walk
// the balanced schedule of 64-slot tiles; a warp takes a page of each and brings the pages,
// with their old weights, into a ring of its own.  A slot's sum over rows is two shuffles.
// Up to 48 rows a KV head: beyond, the tensor-core path (kv_weights_tc.cu).
//
// Bound by the keys' bytes: 64 sequences of 256 to 8192 tokens, one query each, 32 query and 8
// KV heads: 54 us for 291 MB, 5.4 TB/s (79 % of a copy; six pages in flight instead of four 57,
// with fewer CTAs 62); accepted paths of 1 to 5 nodes, 16 sequences: 25 us; one sequence of
// 4096: 5.5 us.
#include <atomic>
#include <cmath>

#include "serve.cuh"

namespace mt {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kP = 16;
constexpr int kMaxRows = 48;  // query rows of a KV head: more go to the tensor-core path
constexpr int kMaxDevices = 64;

template <int D>
struct Cfg {
  static constexpr int CTAS = 4;   // per SM
  static constexpr int DEPTH = 4;  // pages a warp has in its ring
  static constexpr int kKeys = kP * D;
  static constexpr int kSlot = kKeys + kP * 4;  // a page's keys and old weights
  static constexpr int kRing = kWarps * DEPTH * kSlot;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// Byte offset of 16-byte chunk ch of key row r in a slot: permuted so that the fragment
// reads (eight lanes a phase: two rows of four chunks) hit distinct banks.
template <int D>
__device__ __forceinline__ int k_off(int r, int ch) {
  return r * D + ((D == 128 ? ch ^ ((r & 1) << 2) : ch) << 4);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, Cfg<D>::CTAS) kv_weights_kernel(const WeightsParams p, const Sched sched) {
  using C = Cfg<D>;
  constexpr int NC = D / 64, DEPTH = C::DEPTH;
  extern __shared__ __align__(128) uint8_t smem[];
  const int most = (p.rows + 7) & ~7;
  uint4* s_q = reinterpret_cast<uint4*>(smem + C::kRing);                   // [tile of 8 rows][chunk][half][lane]
  float2* s_row = reinterpret_cast<float2*>(smem + C::kRing + most * D * 2);  // score -> base 2, lse in base 2
  int* s_pfx = reinterpret_cast<int*>(s_row + most);                        // [B + 1]
  __shared__ int s_warp[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  pdl_wait();
  AttnParams a{};  // the tiles of the cached slots alone
  a.B = p.B;
  a.T = 0;
  a.max_blocks = p.max_blocks;
  a.seq_lens = p.seq_lens;
  a.status = p.status;
  const int total = block8_prefix<kWarps>(a, s_pfx, s_warp, blockIdx.x == 0);
  Sched sc = sched;
  sc.tile_pfx = s_pfx;
  __shared__ PieceRec s_pieces[kMaxPieceRecs];
  __shared__ int s_npieces;
  if (warp == 0) {
    const int n = list_pieces(sc, total, s_pieces, p.seq_lens);
    if (lane == 0) s_npieces = n;
  }
  __syncthreads();
  PieceSrc it;
  it.init(s_pieces, s_npieces, sc, blockIdx.x, p.seq_lens);
  int L = 0;
  uint8_t* ring = smem + warp * (DEPTH * C::kSlot);
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  Piece pc;
  while (it.next(pc, L)) {  // every thread walks with the same values
    const int b = pc.b, h = pc.kvh;
    const int npages = (L + kP - 1) / kP;
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
        continue;
      }
    }
    const int rows = nodes * p.g, prev = p.prev_lens ? p.prev_lens[b] : L;
    // this warp's pages: first + 4 i
    const int first = 4 * pc.tile_begin + warp;
    const int mine = min(pc.tile_end - pc.tile_begin, max(0, (npages - first + kWarps - 1) / kWarps));
    const int* bt = p.block_tables + (size_t)b * p.max_blocks;
    const int tiles = (rows + 7) / 8;
    // page ids and scales of 32 pages, a lane each; the next 32 ids are fetched while
    // these are used, their scales half way
    auto fetch_id = [&](int i) { return i < mine ? bt[first + 4 * i] : -1; };
    auto fetch_scale = [&](int id) {
      return id >= 0 && id < p.num_pages ? __ldg(p.k_scales + (size_t)id * p.Hkv + h) : 0.f;
    };
    int id_cur = fetch_id(lane), id_nxt = -1, id_iss = id_cur, iss_base = 0;
    float ks_cur = fetch_scale(id_cur), ks_nxt = 0.f;
    auto issue = [&](int i) {
      if (i < mine) {
        if (i - iss_base >= 32) {
          iss_base += 32;
          id_iss = id_nxt;
        }
        const int id = __shfl_sync(0xffffffffu, id_iss, i - iss_base);
        if (id >= 0 && id < p.num_pages) {
          const size_t page = (size_t)id * p.Hkv + h;
          const uint8_t* src = static_cast<const uint8_t*>(p.k_cache) + page * C::kKeys;
          const uint32_t dst = ring_u + (i % DEPTH) * C::kSlot;
          constexpr int CPR = D / 16;  // chunks per row
#pragma unroll
          for (int x = 0; x < kP * CPR / 32; ++x) {
            const int q = x * 32 + lane;
            cp_async16(dst + k_off<D>(q / CPR, q % CPR), src + q * 16);
          }
          if (lane < 4 && (first + 4 * i) * kP < prev) cp_async16(dst + C::kKeys + lane * 16, p.weights + page * kP + lane * 4);
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) issue(i);
    // the queries: a warp eight rows, lanes as they multiply
    __syncthreads();  // those of the piece before are no longer read
    for (int t = warp; t < tiles; t += kWarps) {
      const int row = t * 8 + gid;
      Row8<T> raw[2 * NC];
#pragma unroll
      for (int x = 0; x < 2 * NC; ++x) raw[x].zero();
      float l2 = INFINITY;
      if (row < rows) {
        const int at = row / p.g, node = path ? path[at] : at, head = h * p.g + row % p.g;
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
      if (tig == 0) s_row[row] = make_float2(row < rows ? c : 0.f, l2);
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
    for (int i = 0; i < mine; ++i) {
      const int at = i & 31;
      if (at == 0) {
        if (i > 0) {
          id_cur = id_nxt;
          ks_cur = ks_nxt;
        }
        id_nxt = fetch_id(i + 32 + lane);
      } else if (at == 16) {
        ks_nxt = fetch_scale(id_nxt);
      }
      issue(i + DEPTH - 1);
      cp_wait<DEPTH - 1>();
      __syncwarp();
      const uint8_t* kp = ring + (i % DEPTH) * C::kSlot;
      const int pg = __shfl_sync(0xffffffffu, id_cur, at);
      const float scale = __shfl_sync(0xffffffffu, ks_cur, at);
      uint32_t k[NC][4][4];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint4 w0 = *reinterpret_cast<const uint4*>(kp + k_off<D>(gid, c * 4 + tig));
        const uint4 w1 = *reinterpret_cast<const uint4*>(kp + k_off<D>(gid + 8, c * 4 + tig));
        const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          k[c][x][0] = e4m3x2_to_h2(x0[x] & 0xffffu);
          k[c][x][1] = e4m3x2_to_h2(x1[x] & 0xffffu);
          k[c][x][2] = e4m3x2_to_h2(x0[x] >> 16);
          k[c][x][3] = e4m3x2_to_h2(x1[x] >> 16);
        }
      }
      float sum[2] = {0.f, 0.f};
#pragma unroll 2
      for (int t = 0; t < tiles; ++t) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const float4 rc = *reinterpret_cast<const float4*>(s_row + t * 8 + 2 * tig);
#pragma unroll
        for (int x = 0; x < 2 * NC; ++x) {
          const uint4 q = s_q[(t * 2 * NC + x) * 32 + lane];
          mma(s, k[x / 2][2 * (x % 2)], q.x, q.y);
          mma(s, k[x / 2][2 * (x % 2) + 1], q.z, q.w);
        }
        // element e: row 2 tig + (e & 1), key gid + 8 (e >> 1)
        const float c0 = score_factor(rc.x, scale), c1 = score_factor(rc.z, scale);
        sum[0] += fast_exp2(fmaf(s[0], c0, -rc.y)) + fast_exp2(fmaf(s[1], c1, -rc.w));
        sum[1] += fast_exp2(fmaf(s[2], c0, -rc.y)) + fast_exp2(fmaf(s[3], c1, -rc.w));
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
      }
      // lanes 0 .. 15: a slot each
      const float lo = __shfl_sync(0xffffffffu, sum[0], 4 * (lane & 7)), hi = __shfl_sync(0xffffffffu, sum[1], 4 * (lane & 7));
      const int slot = (first + 4 * i) * kP + lane;
      if (lane < kP && slot < L) {
        if (pg >= 0 && pg < p.num_pages) {
          const float old = slot < prev ? reinterpret_cast<const float*>(kp + C::kKeys)[lane] * p.decay : 0.f;
          p.out[((size_t)pg * p.Hkv + h) * kP + lane] = old + (lane < 8 ? lo : hi);
        } else {
          set_status(p.status, kStPages);
        }
      }
      __syncwarp();  // every lane has read the slot before it is filled again
    }
    cp_wait<0>();
    __syncwarp();
  }
}

template <typename T, int D>
cudaError_t launch_t(const WeightsParams& p, cudaStream_t stream) {
  using C = Cfg<D>;
  static std::atomic<int> sms_of[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev >= 0 && dev < kMaxDevices ? sms_of[dev].load(std::memory_order_acquire) : 0;
  if (!sms) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kv_weights_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kRing + kMaxRows * (D * 2 + (int)sizeof(float2)) + 4 * (8192 + 1));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) sms_of[dev].store(sms, std::memory_order_release);
  }
  const int most = (p.rows + 7) & ~7;
  const size_t smem = C::kRing + (size_t)most * (D * 2 + sizeof(float2)) + 4 * ((size_t)p.B + 1);
  int per_sm = (int)(232448 / (smem + 2304));  // and 1280 bytes of static memory, and the system's 1024
  per_sm = per_sm < 1 ? 1 : per_sm < C::CTAS ? per_sm : C::CTAS;
  // no more CTAs than tiles that the tables can hold
  const long long tiles = (long long)p.B * p.Hkv * ((p.max_blocks + 3) / 4);
  Sched s{};
  s.B = p.B;
  s.T = 0;
  s.Hkv = p.Hkv;
  s.nrg = 1;
  s.G = (int)(tiles < (long long)per_sm * sms ? tiles : (long long)per_sm * sms);
  s.splits = 0;
  s.seg_cost = 4;
  return launch_pdl(kv_weights_kernel<T, D>, dim3(s.G), dim3(kThreads), smem, stream, p, s);
}

}  // namespace

cudaError_t launch_kv_weights(const WeightsParams& p, int dtype, cudaStream_t stream) {
  // Here against there, in us, cold caches, 8 KV heads of 128 columns, bf16: 64 sequences of 256 to
  // 4096 slots, 48 rows 47 against 52, 64 55 against 53; 16 of 512 to 8192, 48 rows 29 against 29, 64
  // 33 against 29; 8 of 4000, 40 rows 22.5 against 22.6, 48 24.6 against 23.0.  Short work has its
  // start, which is longer there: 4 of 2000, 48 rows 14.3 against 16.5, 64 15.0 against 16.8, 128 20.5
  // against 19.1; but what a sequence holds is not known here, and the table may be much wider.
  if (p.rows > kMaxRows) return launch_kv_weights_tc(p, dtype, stream);
  if (p.D == 64)
    return dtype == 1 ? launch_t<__half, 64>(p, stream) : launch_t<__nv_bfloat16, 64>(p, stream);
  return dtype == 1 ? launch_t<__half, 128>(p, stream) : launch_t<__nv_bfloat16, 128>(p, stream);
}

}  // namespace mt
