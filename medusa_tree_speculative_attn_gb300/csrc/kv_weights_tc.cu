// Tensor-core path of the slots' attention weights (kv_weights.cu), for calls with more query
// rows than the register-fragment kernel serves well: trees and chunks of a prompt.
//
// A slot's weight is a sum over query rows, so the keys are the M side: a tile of 128 slots
// (eight pages) by up to 256 query rows, S^T = K Q^T, has a key per TMEM lane, and the thread
// that owns the lane adds up its row of exp2(S * scale - lse) in registers, with no reduction
// between threads.  What belongs to a column (the query's scale and its lse) comes from shared
// memory, the same address for all lanes; what belongs to a key (its page's scale) is the
// thread's own.
//
// Operands stay in 8 bits (kind::f8f6f4): key codes go by TMA straight into the tile, and a
// query row enters as the sum of two (bf16) or three (fp16) E4M3 parts, as in block8_prep.cu,
// worked out by the CTA when it takes up a segment and kept for all of its tiles.  Roles: a
// warp issues the copies (a lane per page), one the products, eight add up, four of them the
// even tiles and four the odd ones, each set with a 256-column accumulator of its own.  Every
// mbarrier wait is bounded (as in attn_block8_tc.cu), and the sums' warps meet by mbarriers
// too, so that a timeout leaves nobody waiting.
//
// More than 256 query rows of a KV head are taken in passes over the segment's tiles.
#include <cudaTypedefs.h>

#include <atomic>
#include <climits>

#include "serve.cuh"
#include "tc_ptx.cuh"

namespace mt {

namespace {

constexpr int kP = 16;
constexpr int kPages = 8;  // of a tile
constexpr int kTile = kPages * kP;
constexpr int kCols = 256;  // query rows at a time
constexpr int kSmemLimit = 232448;
constexpr int kMaxDevices = 64;
constexpr int kSumWarps = 8, kCopyWarp = 8, kMmaWarp = 9, kThreads = 10 * 32;

template <int D, int NP>
struct Cfg {
  static constexpr int kQPart = kCols * D;
  static constexpr int kQ = NP * kQPart;
  static constexpr int kStage = kTile * D;
  static constexpr int kMeta = 1024 + kCols * 8;  // barriers, columns
  static constexpr int kFit = (kSmemLimit - 1024 - kMeta - kQ - 4 * (8192 + 4)) / kStage;
  static constexpr int STAGES = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = 1024 + kQ + STAGES * kStage + kMeta;  // and the prefix
  static_assert(STAGES >= 3, "shared memory budget");
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 lanes x 32 bits, 32 consecutive columns per thread; and the wait, through which the
// registers pass so that no use of them can move ahead of it.
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :
               : "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}

// Two fp32 in one register pair, for the instructions that take both at once.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2_of(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float f2_lo(F2 x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float f2_hi(F2 x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// D[tmem] (+)= A[smem] * B[smem]: E4M3 both, K-major, fp32 accumulator.
template <bool ACC>
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  if (ACC) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.eq.u32 p, 1, 1;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc)
        : "memory");
  } else {
    asm volatile(
        "{\n.reg .pred p;\nsetp.eq.u32 p, 1, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc)
        : "memory");
  }
}

// Instruction descriptor of kind::f8f6f4 with E4M3 operands (format 0), both
// K-major, fp32 accumulator (1 at bits 4-5), N >> 3 at bit 17, M >> 4 at bit 24.
__device__ __forceinline__ uint32_t idesc_f8(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// K-major matrix of rows of D bytes, swizzled over 128 (D = 128) or 64 bytes: eight-row
// groups D * 8 bytes apart; swizzle mode at bits 61-63 (2: 128, 4: 64).
template <int D>
__device__ __forceinline__ uint64_t desc_rows8(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)((8 * D) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(D == 128 ? 2 : 4) << 61;
  return d;
}

// Byte offset of 16-byte chunk ch of row r in such a matrix.
template <int D>
__device__ __forceinline__ int row_off(int r, int ch) {
  return r * D + ((D == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3)) << 4);
}

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, int* status,
                                       uint64_t limit) {
  return tc::mbar_wait(bar, parity, abort, status, limit);
}

// Waits that ignore the abort flag (copies and MMAs in flight at the end).
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, int* status) {
  const uint64_t t0 = tc::global_timer_ns();
  while (!tc::mbar_try_wait(bar, parity)) {
    if (tc::global_timer_ns() - t0 > tc::kDrainLimitNs) {
      set_status(status, kStTimeout);
      return;
    }
  }
}

// Eight lanes (D / 16) a row: 16 columns c of query row `row` of this pass as E4M3 parts in
// their places; returns the row's scale (scores of the parts -> base 2).
template <typename T, int D, int NP>
__device__ __forceinline__ float place_query(const T* src, float scale_log2, uint8_t* sq, int row, int c) {
  Row8<T> r0, r1;
  r0.zero();
  r1.zero();
  if (src) {
    r0.load(src + 16 * c);
    r1.load(src + 16 * c + 8);
  }
  float x[16];
  {
    float t[8];
    r0.to_f(t);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = t[e];
    r1.to_f(t);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[8 + e] = t[e];
  }
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
  for (int off = 1; off < D / 16; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  const float scale = block_scale(amax), inv = 1.f / scale;
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] *= inv;
#pragma unroll
  for (int part = 0; part < NP; ++part) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = e4m3x2_of(x[4 * i], x[4 * i + 1]), hi = e4m3x2_of(x[4 * i + 2], x[4 * i + 3]);
      w[i] = lo | hi << 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // what the part leaves, exactly
        const uint32_t h2 = e4m3x2_to_h2(h ? hi : lo);
        __half2 v;
        memcpy(&v, &h2, 4);
        const float2 f = __half22float2(v);
        x[4 * i + 2 * h] -= f.x;
        x[4 * i + 2 * h + 1] -= f.y;
      }
    }
    *reinterpret_cast<uint4*>(sq + part * (kCols * D) + row_off<D>(row, c)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  // an infinity has no parts: the row's weights become NaN, as they would be
  return amax < INFINITY ? scale * scale_log2 : __int_as_float(0x7fffffff);
}

template <typename T, int D, int NP>
__global__ void __launch_bounds__(kThreads, 1)
    kv_weights_tc_kernel(const __grid_constant__ CUtensorMap map_k, const WeightsParams p, const Sched sched) {
  using C = Cfg<D, NP>;
  constexpr int S = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;             // [part][256 rows] swizzled
  uint8_t* sK = sQ + C::kQ;       // [stage][128 rows] swizzled
  float4* s_col = reinterpret_cast<float4*>(sK + S * C::kStage);  // of two columns: their scales, minus their lse
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_col + kCols / 2);
  uint64_t* full = bars;           // [S] a tile's codes have landed
  uint64_t* empty = full + S;      // [S] and are multiplied
  uint64_t* acc_full = empty + S;  // [2] a tile's scores are there
  uint64_t* acc_empty = acc_full + 2;  // [2] and read out
  uint64_t* idle = acc_empty + 2;      // the sums' warps have left the pass before
  uint64_t* q_full = idle + 1;         // the pass's queries are in place
  uint64_t* fin = q_full + 1;          // every product done
  uint64_t* never = fin + 1;           // nothing arrives here (timeout test hook)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * 6 + 8) * 8 + 8 <= 1024, "barrier area");
  int* s_pfx = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 1024);  // [B + 1]
  __shared__ int s_warp[kThreads / 32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&acc_full[s], 1);
      tc::mbar_init(&acc_empty[s], 4);
    }
    tc::mbar_init(idle, kSumWarps);
    tc::mbar_init(q_full, kSumWarps);
    tc::mbar_init(fin, 1);
    tc::mbar_init(never, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  if (warp == kCopyWarp && lane == 0) tc::prefetch_tmap(&map_k);
  pdl_wait();
  AttnParams a{};  // the tiles of the cached slots alone
  a.B = p.B;
  a.T = 0;
  a.max_blocks = p.max_blocks;
  a.seq_lens = p.seq_lens;
  a.status = p.status;
  tc::tc_fence_before();
  block8_prefix<kThreads / 32, false, kPages>(a, s_pfx, s_warp, blockIdx.x == 0);  // (ends in a barrier)
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Sched sc = sched;
  sc.tile_pfx = s_pfx;
  PieceIter it;
  it.init(sc, blockIdx.x);
  Piece pc;
  bool ok = true;
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    const bool r = tc::mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_flag, p.status, p.wait_limit_ns);
    ok = __all_sync(0xffffffffu, r) && ok;
  };
  // The query rows of a piece's sequence, 0 for one whose path is out of range: every role
  // finds the same.
  auto rows_of = [&](int b) {
    int nodes = p.T;
    if (p.accept_path) {
      const int* path = p.accept_path + (size_t)b * (p.max_depth + 1);
      nodes = p.accept_len[b] + 1;
      bool stray = nodes < 1 || nodes > p.max_depth + 1;
      if (!stray)
        for (int i = lane; i < nodes; i += 32) stray = stray || (unsigned)path[i] >= (unsigned)p.T;
      if (__any_sync(0xffffffffu, stray)) nodes = 0;
    }
    return nodes * p.g;
  };

  if (warp == kCopyWarp) {
    // -------------------------------------------------------------- copies
    const uint64_t policy = tc::policy_evict_first();
    const int oob_row = p.num_pages * p.Hkv * kP;  // past the cache: TMA fills zeros
    uint32_t pos = 0;
    while (ok && it.next(pc)) {
      const int rows = rows_of(pc.b), npages = (p.seq_lens[pc.b] + kP - 1) / kP;
      const int* bt = p.block_tables + (size_t)pc.b * p.max_blocks;
      for (int r0 = 0; ok && r0 < rows; r0 += kCols) {
        // page ids of 32 pages (four tiles) at a time, a lane each, the next 32 in flight
        auto fetch = [&](int q) { return q < npages ? __ldg(bt + q) : -1; };
        int base = pc.tile_begin * kPages;
        int id0 = fetch(base + lane), id1 = fetch(base + 32 + lane);
        for (int j = pc.tile_begin; j < pc.tile_end; ++j, ++pos) {
          if (j * kPages - base >= 32) {
            base += 32;
            id0 = id1;
            id1 = fetch(base + 32 + lane);
          }
          const uint32_t st = pos % S;
          const int id = __shfl_sync(0xffffffffu, id0, (j * kPages - base) + (lane & 7));
          if (pos >= (uint32_t)S) wait_all(&empty[st], ((pos / S) - 1) & 1);
          if (!ok) break;
          if (lane == 0) tc::mbar_arrive_expect_tx(&full[st], C::kStage);
          __syncwarp();
          if (lane < kPages)
            tc::tma_load_2d(sK + st * C::kStage + lane * kP * D, &map_k, 0,
                            id >= 0 && id < p.num_pages ? (id * p.Hkv + pc.kvh) * kP : oob_row, &full[st], policy);
          __syncwarp();
        }
      }
    }
    // no TMA load may still be writing shared memory when the CTA exits
    if (lane == 0)
      for (uint32_t t = pos > (uint32_t)S ? pos - S : 0; t < pos; ++t) drain_wait(&full[t % S], (t / S) & 1, p.status);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    const uint32_t sQ_u = tc::smem_u32(sQ), sK_u = tc::smem_u32(sK);
    uint32_t pos = 0, pass = 0;
    if (p.test_stall) wait_all(never, 0);  // test hook: a wait that can only time out
    while (ok && it.next(pc)) {
      const int rows = rows_of(pc.b);
      for (int r0 = 0; ok && r0 < rows; r0 += kCols, ++pass) {
        const int n = (min(kCols, rows - r0) + 31) / 32 * 32;
        const uint32_t idesc = idesc_f8(kTile, n);
        wait_all(q_full, pass & 1);
        for (int j = pc.tile_begin; ok && j < pc.tile_end; ++j, ++pos) {
          const uint32_t st = pos % S, buf = pos & 1;
          wait_all(&full[st], (pos / S) & 1);
          if (pos >= 2) wait_all(&acc_empty[buf], ((pos / 2) - 1) & 1);
          if (!ok) break;
          tc::tc_fence_after();
          const uint64_t kd = desc_rows8<D>(sK_u + st * C::kStage);
          if (tc::elect_one()) {
#pragma unroll
            for (int part = 0; part < NP; ++part) {
              const uint64_t qd = desc_rows8<D>(sQ_u + part * C::kQPart);
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) {  // 32 codes: 2 descriptor units
                if (part == 0 && kk == 0) mma_f8_ss<false>(tmem + buf * kCols, kd, qd, idesc);
                else mma_f8_ss<true>(tmem + buf * kCols, kd + (uint64_t)(kk * 2), qd + (uint64_t)(kk * 2), idesc);
              }
            }
            tc::mma_commit(&empty[st]);
            tc::mma_commit(&acc_full[buf]);
          }
          __syncwarp();
        }
      }
    }
    if (tc::elect_one()) tc::mma_commit(fin);
    __syncwarp();
    if (lane == 0) drain_wait(fin, 0, p.status);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- sums
    const int set = warp >> 2, quad = warp & 3;  // tiles of this parity; TMEM lanes 32 quad ...
    const int key = quad * 32 + lane;            // of the tile
    const uint32_t addr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(set * kCols);
    uint32_t pos = 0, pass = 0;
    while (ok && it.next(pc)) {
      const int b = pc.b, h = pc.kvh, rows = rows_of(b);
      if (rows == 0 && threadIdx.x == 0) set_status(p.status, kStPages);
      const int L = p.seq_lens[b], prev = p.prev_lens ? p.prev_lens[b] : L;
      const int* path = p.accept_path ? p.accept_path + (size_t)b * (p.max_depth + 1) : nullptr;
      const int* bt = p.block_tables + (size_t)b * p.max_blocks;
      const int tiles = pc.tile_end - pc.tile_begin;
      for (int r0 = 0; ok && r0 < rows; r0 += kCols, ++pass, pos += (uint32_t)tiles) {
        // the queries and the columns' constants, once nobody uses the pass before's
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(idle);
        wait_all(idle, pass & 1);
        if (!ok) break;
        const int n = min(kCols, rows - r0), cols = (n + 31) / 32 * 32;
        constexpr int LPR = D / 16, RPW = 32 / LPR;
        for (int q0 = warp * RPW; q0 < cols; q0 += kSumWarps * RPW) {
          const int row = q0 + lane / LPR;
          const T* src = nullptr;
          float l2 = INFINITY;  // a column past the rows gives 2^-inf
          if (row < n) {
            const int at = (r0 + row) / p.g, node = path ? path[at] : at, head = h * p.g + (r0 + row) % p.g;
            const size_t q = ((size_t)b * p.T + node) * p.Hq + head;
            src = static_cast<const T*>(p.q) + q * D;
            l2 = p.lse[q] * 1.4426950408889634f;
          }
          const float c = place_query<T, D, NP>(src, p.scale_log2, sQ, row, lane % LPR);
          if (lane % LPR == 0) {
            float* col = reinterpret_cast<float*>(s_col + row / 2) + (row & 1);
            col[0] = row < n ? c : 0.f;
            col[2] = -l2;
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(q_full);
        // this thread's keys: page id two of its tiles ahead, scale and old weight one
        const float* before = r0 == 0 ? p.weights : p.out;
        const int had = r0 == 0 ? prev : L;
        const float decay = r0 == 0 ? p.decay : 1.f;
        auto fetch_id = [&](int j) {
          const int slot = (pc.tile_begin + j) * kTile + key;
          return j < tiles && slot < L ? bt[slot / kP] : INT_MIN;
        };
        auto fetch = [&](int j, int id, float& ks, float& old) {
          ks = old = 0.f;
          if (id < 0 || id >= p.num_pages) return;
          const size_t page = (size_t)id * p.Hkv + h;
          ks = __ldg(p.k_scales + page);
          if ((pc.tile_begin + j) * kTile + key < had) old = before[page * kP + key % kP];
        };
        int j = (int)((set ^ pos) & 1);  // this set's first tile
        int id = fetch_id(j), id_next = fetch_id(j + 2);
        float ks, old;
        fetch(j, id, ks, old);
        wait_all(q_full, pass & 1);
        for (; ok && j < tiles; j += 2) {
          float ks_next, old_next;
          fetch(j + 2, id_next, ks_next, old_next);
          const int id_after = fetch_id(j + 4);
          const uint32_t at = (pos + (uint32_t)j) / 2;
          wait_all(&acc_full[set], at & 1);
          if (!ok) break;
          tc::tc_fence_after();
          const F2 k2 = f2_of(ks, ks);
          F2 sum0 = f2_of(0.f, 0.f), sum1 = sum0;
          uint32_t s0[32], s1[32];
          auto add = [&](uint32_t (&s)[32], int col) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 u = s_col[(col + i) / 2], v = s_col[(col + i) / 2 + 1];
              const F2 x = f2_fma(f2_mul(f2_of(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), k2), f2_of(u.x, u.y),
                                  f2_of(u.z, u.w));
              const F2 y = f2_fma(f2_mul(f2_of(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), k2),
                                  f2_of(v.x, v.y), f2_of(v.z, v.w));
              sum0 = f2_add(sum0, f2_of(fast_exp2(f2_lo(x)), fast_exp2(f2_hi(x))));
              sum1 = f2_add(sum1, f2_of(fast_exp2(f2_lo(y)), fast_exp2(f2_hi(y))));
            }
          };
          tmem_ld_x32(addr, s0);
          tmem_ld_wait(s0);
#pragma unroll 1
          for (int col = 0; col < cols; col += 64) {  // 32 columns in flight while 32 are added
            if (col + 32 < cols) tmem_ld_x32(addr + col + 32, s1);
            add(s0, col);
            if (col + 32 < cols) {
              tmem_ld_wait(s1);
              if (col + 64 < cols) tmem_ld_x32(addr + col + 64, s0);
              add(s1, col + 32);
              if (col + 64 < cols) tmem_ld_wait(s0);
            }
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&acc_empty[set]);
          const float sum = (f2_lo(sum0) + f2_hi(sum0)) + (f2_lo(sum1) + f2_hi(sum1));
          if (id >= 0 && id < p.num_pages) p.out[((size_t)id * p.Hkv + h) * kP + key % kP] = fmaf(old, decay, sum);
          else if (id != INT_MIN) set_status(p.status, kStPages);
          id = id_next;
          id_next = id_after;
          ks = ks_next;
          old = old_next;
        }
      }
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

template <typename T, int D, int NP>
cudaError_t launch_t(const WeightsParams& p, cudaStream_t stream) {
  using C = Cfg<D, NP>;
  static std::atomic<int> sms_of[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev >= 0 && dev < kMaxDevices ? sms_of[dev].load(std::memory_order_acquire) : 0;
  if (!sms) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kv_weights_tc_kernel<T, D, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem + 4 * (8192 + 1));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) sms_of[dev].store(sms, std::memory_order_release);
  }
  auto enc = get_encode();
  if (!enc) return cudaErrorInvalidValue;
  alignas(64) CUtensorMap map;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)p.num_pages * p.Hkv * kP};
  const cuuint64_t strides[1] = {(cuuint64_t)D};
  const cuuint32_t box[2] = {(cuuint32_t)D, kP};
  const cuuint32_t es[2] = {1, 1};
  if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p.k_cache), dims, strides, box, es,
          CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const long long tiles = (long long)p.B * p.Hkv * ((p.max_blocks + kPages - 1) / kPages);
  Sched s{};
  s.B = p.B;
  s.T = 0;
  s.Hkv = p.Hkv;
  s.nrg = 1;
  s.G = (int)(tiles < sms ? tiles : sms);
  s.splits = 0;
  s.seg_cost = 3;
  return launch_pdl(kv_weights_tc_kernel<T, D, NP>, dim3(s.G), dim3(kThreads), (size_t)C::kSmem + 4 * ((size_t)p.B + 1),
                    stream, map, p, s);
}

}  // namespace

cudaError_t launch_kv_weights_tc(const WeightsParams& p, int dtype, cudaStream_t stream) {
  if (p.D == 64) return dtype == 1 ? launch_t<__half, 64, 3>(p, stream) : launch_t<__nv_bfloat16, 64, 2>(p, stream);
  return dtype == 1 ? launch_t<__half, 128, 3>(p, stream) : launch_t<__nv_bfloat16, 128, 2>(p, stream);
}

}  // namespace mt
