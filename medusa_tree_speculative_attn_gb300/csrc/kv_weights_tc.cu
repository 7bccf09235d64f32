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
// worked out by the CTA when it takes up a segment and kept for all of its tiles.
//
// Roles: a warp issues the copies (a lane per page), one the products, sixteen add up.  A
// constant from shared memory costs a 16-byte read for every two columns and warp, so a thread
// takes a key of two tiles at once: a unit is two tiles by 128 columns, two units fill TMEM,
// and each has a group of eight warps, 64 columns a warp.  The sums of a pair of tiles meet in
// shared memory.  Every mbarrier wait is bounded (as in attn_block8_tc.cu), and the sums'
// warps meet by mbarriers too, so that a timeout leaves nobody waiting.
//
// More than 256 query rows of a KV head are taken in passes over the segment's tiles.
//
// Bound by a unit's chain, products (16 of 100 cycles) then sums (2800 cycles with both groups
// at work, of which the exponentials' unit is busy 2050), one accumulator a group.  Chunks of
// 64 tokens for 8 sequences of 4096 to 16384, 32 query and 8 KV heads, bf16: 69 us, 39 % of the
// products' rate; 4.0 of 5.2 thousand cycles a pair of tiles for the chain, 8000 cycles to
// begin and 7000 to change a segment.  A tile at a time with eight warps took 80 us, with
// sixteen 75; four groups of 64 columns 81 (a product of 64 columns takes 80 cycles).
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
constexpr int kInfo = 32;  // tiles whose pages' numbers and scales are kept: more than the roles are ever apart
constexpr int kSmemLimit = 232448;
constexpr int kMaxDevices = 64;
constexpr int kNone = INT_MIN;  // no page
constexpr int kUnit = 128;  // query rows of a unit: an accumulator has them for two tiles
constexpr int kAcc = 2;     // accumulators, each of a group of eight warps
constexpr int kSumWarps = 16, kCopyWarp = 16, kMmaWarp = 17, kThreads = 18 * 32;

template <int D, int NP>
struct Cfg {
  static constexpr int kQPart = kCols * D;
  static constexpr int kQ = NP * kQPart;
  static constexpr int kStage = kTile * D;
  static constexpr int kPart = kAcc * 4 * 2 * kTile * 4;
  static constexpr int kMeta = 1024 + kCols * 8 + kPart + kInfo * kPages * 8 +
                               kMaxPieceRecs * (int)sizeof(PieceRec);  // barriers, columns, parts of sums, pages, pieces
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

// 32 lanes x 32 bits, eight consecutive columns per thread of two accumulators; and the
// wait, through which the registers pass so that no use of them can move ahead of it.
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[8], uint32_t (&s)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(s[0]), "+r"(s[1]), "+r"(s[2]), "+r"(s[3]), "+r"(s[4]), "+r"(s[5]), "+r"(s[6]), "+r"(s[7])
               :
               : "memory");
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

// A query row's 16 columns of one lane (D / 16 lanes a row).
template <typename T>
struct QueryPart {
  Row8<T> r0, r1;
  __device__ __forceinline__ void load(const T* src) {
    r0.zero();
    r1.zero();
    if (src) {
      r0.load(src);
      r1.load(src + 8);
    }
  }
};

// Columns 16 c .. 16 c + 15 of query row `row` of this pass as E4M3 parts in their places;
// returns the row's scale (scores of the parts -> base 2).  Scaled to 448 at most, an fp16
// holds all of a query's bits above 2^-24, far below the last part's smallest step (2^-9).
template <typename T, int D, int NP>
__device__ __forceinline__ float place_query(const QueryPart<T>& q, float scale_log2, uint8_t* sq, int row, int c) {
  AbsMax<T> top;
  top.add(q.r0);
  top.add(q.r1);
  float amax = top.get();
#pragma unroll
  for (int off = 1; off < D / 16; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  const float scale = block_scale(amax), inv = 1.f / scale;
  __half2 x[8];
  {
    float t[8];
    q.r0.to_f(t);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __floats2half2_rn(t[2 * e] * inv, t[2 * e + 1] * inv);
    q.r1.to_f(t);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 + e] = __floats2half2_rn(t[2 * e] * inv, t[2 * e + 1] * inv);
  }
#pragma unroll
  for (int part = 0; part < NP; ++part) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t bits;
      memcpy(&bits, &x[e], 4);
      uint16_t code;
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(code) : "r"(bits));
      if (e & 1) w[e / 2] |= (uint32_t)code << 16; else w[e / 2] = code;
      if (part + 1 < NP) {  // what the part leaves, exactly
        const uint32_t h = e4m3x2_to_h2(code);
        __half2 v;
        memcpy(&v, &h, 4);
        x[e] = __hsub2(x[e], v);
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
  float* s_part = reinterpret_cast<float*>(s_col + kCols / 2);  // [pair's turn][half unit][tile][key]
  int2* s_page = reinterpret_cast<int2*>(s_part + C::kPart / 4);  // [kInfo][8] a tile's pages: number, scale
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_page + kInfo * kPages);
  uint64_t* full = bars;           // [S] a tile's codes have landed
  uint64_t* empty = full + S;      // [S] and are multiplied
  uint64_t* acc_full = empty + S;         // [kAcc] a unit's scores are there
  uint64_t* acc_empty = acc_full + kAcc;  // [kAcc] and read out
  uint64_t* parts = acc_empty + kAcc;     // [kAcc] the units' sums of a pair are there
  uint64_t* parts_read = parts + kAcc;    // [kAcc] and read
  uint64_t* idle = parts_read + kAcc;     // the sums' warps have left the pass before
  uint64_t* q_full = idle + 1;         // the pass's queries are in place
  uint64_t* fin = q_full + 1;          // every product done
  uint64_t* never = fin + 1;           // nothing arrives here (timeout test hook)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * 6 + 4 * kAcc + 4) * 8 + 8 <= 1024, "barrier area");
  PieceRec* s_pieces = reinterpret_cast<PieceRec*>(reinterpret_cast<uint8_t*>(bars) + 1024);
  int* s_pfx = reinterpret_cast<int*>(s_pieces + kMaxPieceRecs);  // [B + 1]
  __shared__ int s_warp[kThreads / 32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kAcc; ++s) {
      tc::mbar_init(&acc_full[s], 2);  // the products, and their issuer itself (below)
      tc::mbar_init(&acc_empty[s], kSumWarps / kAcc);
      tc::mbar_init(&parts[s], kSumWarps);
      tc::mbar_init(&parts_read[s], kSumWarps);
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
  const int total = block8_prefix<kThreads / 32, false, kPages>(a, s_pfx, s_warp, blockIdx.x == 0);
  Sched sc = sched;
  sc.tile_pfx = s_pfx;
  // this CTA's pieces, listed once by a warp (the walk's divisions are slow in 64 bits)
  __shared__ int s_npieces;
  if (warp == kCopyWarp) {
    const int n = list_pieces(sc, total, s_pieces, p.seq_lens);
    if (lane == 0) s_npieces = n;
  }
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PieceSrc it;
  it.init(s_pieces, s_npieces, sc, blockIdx.x, p.seq_lens);
  Piece pc;
  int L = 0;
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
    while (ok && it.next(pc, L)) {
      const int rows = rows_of(pc.b), npages = (L + kP - 1) / kP;
      const int* bt = p.block_tables + (size_t)pc.b * p.max_blocks;
      for (int r0 = 0; ok && r0 < rows; r0 += kCols) {
        // page ids of 32 pages (four tiles) at a time, a lane each, the next 64 in flight
        // (their scales with them): kNone behind the last
        auto fetch = [&](int q) { return q < npages ? max(__ldg(bt + q), -1) : kNone; };
        auto fetch_scale = [&](int id) {
          return id >= 0 && id < p.num_pages ? __ldg(p.k_scales + (size_t)id * p.Hkv + pc.kvh) : 0.f;
        };
        int base = pc.tile_begin * kPages;
        int id0 = fetch(base + lane), id1 = fetch(base + 32 + lane), id2 = fetch(base + 64 + lane);
        float ks0 = fetch_scale(id0), ks1 = fetch_scale(id1);
        for (int j = pc.tile_begin; j < pc.tile_end; ++j, ++pos) {
          if (j * kPages - base >= 32) {
            base += 32;
            id0 = id1;
            ks0 = ks1;
            id1 = id2;
            ks1 = fetch_scale(id1);
            id2 = fetch(base + 64 + lane);
          }
          const uint32_t st = pos % S;
          const int id = __shfl_sync(0xffffffffu, id0, (j * kPages - base) + (lane & 7));
          const float ks = __shfl_sync(0xffffffffu, ks0, (j * kPages - base) + (lane & 7));
          if (pos >= (uint32_t)S) wait_all(&empty[st], ((pos / S) - 1) & 1);
          if (!ok) break;
          // (the place is free: the products of the tile S before are done, so every group has
          // left the pair eight before that tile's, which holds tiles after the one kInfo back)
          if (lane < kPages) s_page[pos % kInfo * kPages + lane] = make_int2(id, __float_as_int(ks));
          __syncwarp();
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
    uint32_t pos = 0, unit = 0, pass = 0;
    if (p.test_stall) wait_all(never, 0);  // test hook: a wait that can only time out
    while (ok && it.next(pc, L)) {
      const int rows = rows_of(pc.b);
      for (int r0 = 0; ok && r0 < rows; r0 += kCols, ++pass) {
        const int cols = (min(kCols, rows - r0) + 31) / 32 * 32;
        wait_all(q_full, pass & 1);
        for (int j = pc.tile_begin; ok && j < pc.tile_end; j += 2) {
          const int two = min(2, pc.tile_end - j);
          for (int x = 0; x < two; ++x) wait_all(&full[(pos + x) % S], ((pos + x) / S) & 1);
          for (int c0 = 0; ok && c0 < cols; c0 += kUnit, ++unit) {
            const uint32_t buf = unit % kAcc;
            if (unit >= kAcc) wait_all(&acc_empty[buf], ((unit / kAcc) - 1) & 1);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t idesc = idesc_f8(kTile, min(kUnit, cols - c0));
#pragma unroll 1
            for (int x = 0; x < two; ++x) {
              const uint64_t kd = desc_rows8<D>(sK_u + (pos + x) % S * C::kStage);
              const uint32_t d = tmem + buf * (2 * kUnit) + x * kUnit;
              if (tc::elect_one()) {
#pragma unroll
                for (int part = 0; part < NP; ++part) {
                  const uint64_t qd = desc_rows8<D>(sQ_u + part * C::kQPart + c0 * D);
#pragma unroll
                  for (int kk = 0; kk < D / 32; ++kk) {  // 32 codes: 2 descriptor units
                    if (part == 0 && kk == 0) mma_f8_ss<false>(d, kd, qd, idesc);
                    else mma_f8_ss<true>(d, kd + (uint64_t)(kk * 2), qd + (uint64_t)(kk * 2), idesc);
                  }
                }
                if (c0 + kUnit >= cols) tc::mma_commit(&empty[(pos + x) % S]);
                if (x == two - 1) tc::mma_commit(&acc_full[buf]);
              }
              __syncwarp();
            }
            // passes on what this warp acquired with the tiles: their pages
            if (lane == 0) tc::mbar_arrive(&acc_full[buf]);
            __syncwarp();
          }
          pos += (uint32_t)two;
        }
      }
    }
    if (tc::elect_one()) tc::mma_commit(fin);
    __syncwarp();
    if (lane == 0) drain_wait(fin, 0, p.status);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- sums
    const int quad = warp & 3, half = warp >> 2 & 1;  // TMEM lanes 32 quad ..; 64 columns of a unit
    const uint32_t group = warp >> 3;                 // units of this number modulo kAcc
    const int key = quad * 32 + lane;                 // of a tile
    const uint32_t addr = tmem + ((uint32_t)(quad * 32) << 16) + group * (2 * kUnit) + (uint32_t)(half * 64);
    const float inv_g = 1.f / (float)p.g;
    uint32_t unit = 0, pair = 0, pos = 0, pass = 0;
    while (ok && it.next(pc, L)) {
      const int b = pc.b, h = pc.kvh, rows = rows_of(b);
      if (rows == 0 && threadIdx.x == 0) set_status(p.status, kStPages);
      const int prev = p.prev_lens ? p.prev_lens[b] : L;
      const int* path = p.accept_path ? p.accept_path + (size_t)b * (p.max_depth + 1) : nullptr;
      const int tiles = pc.tile_end - pc.tile_begin;
      for (int r0 = 0; ok && r0 < rows; r0 += kCols, ++pass) {
        // the queries and the columns' constants, asked for together, and put in their places
        // once nobody uses the pass before's
        const int n = min(kCols, rows - r0), cols = (n + 31) / 32 * 32;
        constexpr int LPR = D / 16, RPW = 32 / LPR, IT = kCols / (kSumWarps * RPW);
        QueryPart<T> raw[IT];
        float l2[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int row = (i * kSumWarps + warp) * RPW + lane / LPR;
          l2[i] = INFINITY;  // a column past the rows gives 2^-inf
          const T* src = nullptr;
          if (row < n) {
            // (exact: rows are below 2^20)
            const int at = (int)(((float)(r0 + row) + 0.5f) * inv_g), node = path ? path[at] : at;
            const int head = h * p.g + (r0 + row) - at * p.g;
            const size_t q = ((size_t)b * p.T + node) * p.Hq + head;
            src = static_cast<const T*>(p.q) + q * D + 16 * (lane % LPR);
            l2[i] = p.lse[q];
          }
          raw[i].load(src);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(idle);
        wait_all(idle, pass & 1);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int row = (i * kSumWarps + warp) * RPW + lane / LPR;
          if ((i * kSumWarps + warp) * RPW >= cols) break;  // the same for the warp
          const float c = place_query<T, D, NP>(raw[i], p.scale_log2, sQ, row, lane % LPR);
          if (lane % LPR == 0) {
            float* col = reinterpret_cast<float*>(s_col + row / 2) + (row & 1);
            col[0] = row < n ? c : 0.f;
            col[2] = -l2[i] * 1.4426950408889634f;
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(q_full);
        const float* before = r0 == 0 ? p.weights : p.out;  // later rows add to what the earlier ones left
        const int had = r0 == 0 ? prev : L;
        const float decay = r0 == 0 ? p.decay : 1.f;
        wait_all(q_full, pass & 1);
        // A pair's sums: a unit's group leaves its own, and when all are there each warp writes
        // one page's (a half-warp adds a unit's), a pair later, so that nobody waits.
        const int units = (cols + kUnit - 1) / kUnit;
        size_t at = 0;
        bool writes = false, known = false;
        float old = 0.f;
        int last_j = 0;
        uint32_t last_pos = 0;
        // What this warp writes of the pair that begins with tile j, and the old weight.  The
        // pair's pages may be looked at by who has seen its scores, or the others' sums of it.
        auto look = [&](int j, uint32_t ps) {
          const int x = warp >> 3, id = j + x < tiles ? s_page[(ps + x) % kInfo * kPages + (warp & 7)].x : kNone;
          const int slot = (pc.tile_begin + j + x) * kTile + (warp & 7) * kP + (lane & 15);
          const bool good = id >= 0 && id < p.num_pages;
          writes = good && lane < kP && slot < L;
          at = ((size_t)(good ? id : 0) * p.Hkv + h) * kP + (lane & 15);
          old = writes && slot < had ? before[at] : 0.f;
          if (id != kNone && !good && lane == 0) set_status(p.status, kStPages);
        };
        auto finish = [&](uint32_t pr) {
          const uint32_t side = pr % kAcc;
          wait_all(&parts[side], (pr / kAcc) & 1);
          if (!ok) return;
          if (!known) look(last_j, last_pos);
          const float* part = s_part + (size_t)((side * 4 + (lane >> 4) * 2) * 2 + (warp >> 3)) * kTile + (warp & 7) * kP + (lane & 15);
          const int first = (lane >> 4) * 2;
          float all = first < 2 * units ? part[0] + part[2 * kTile] : 0.f;
          all += __shfl_xor_sync(0xffffffffu, all, 16);
          if (lane == 0) tc::mbar_arrive(&parts_read[side]);
          if (writes) p.out[at] = fmaf(old, decay, all);
        };
        for (int j = 0; ok && j < tiles; j += 2, ++pair, unit += (uint32_t)units) {
          const uint32_t side = pair % kAcc;
          const int u = (int)((group - unit) % kAcc);  // the pair's unit that is this group's, if there is one
          if (u < units) {
            F2 k[2], sum[2][2];
            wait_all(&acc_full[group], ((unit + (uint32_t)u) / kAcc) & 1);
            if (!ok) break;
            tc::tc_fence_after();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float ks = __int_as_float(s_page[(pos + x) % kInfo * kPages + key / kP].y);
              k[x] = f2_of(ks, ks);
              sum[x][0] = sum[x][1] = f2_of(0.f, 0.f);
            }
            const int c0 = u * kUnit + half * 64, steps = max(0, min(8, (cols - c0) / 8));  // whole fours: cols are
            const float4* col = s_col + c0 / 2;
            uint32_t s[2][2][8];  // [turn][tile]: eight columns are added while eight are on their way
            auto load = [&](int y, int turn) {  // (no second tile: what is left over there, and not used)
              tmem_ld_x8(addr + y * 8, s[turn][0]);
              tmem_ld_x8(addr + kUnit + y * 8, s[turn][1]);
            };
            auto add = [&](int y, int turn) {
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                const float4 c = col[y * 4 + i / 2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const uint32_t* v = s[turn][x] + i;
                  const F2 z = f2_fma(f2_mul(f2_of(__uint_as_float(v[0]), __uint_as_float(v[1])), k[x]), f2_of(c.x, c.y),
                                      f2_of(c.z, c.w));
                  sum[x][i / 2 & 1] = f2_add(sum[x][i / 2 & 1], f2_of(fast_exp2(f2_lo(z)), fast_exp2(f2_hi(z))));
                }
              }
            };
            if (steps > 0) load(0, 0);
#pragma unroll 1
            for (int y = 0; y < steps; y += 2) {
              tmem_ld_wait(s[0][0], s[0][1]);
              load(y + 1, 1);
              add(y, 0);
              tmem_ld_wait(s[1][0], s[1][1]);
              if (y + 2 < steps) load(y + 2, 0);
              add(y + 1, 1);
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&acc_empty[group]);
            if (pair >= kAcc) wait_all(&parts_read[side], ((pair / kAcc) - 1) & 1);
            if (!ok) break;
#pragma unroll
            for (int x = 0; x < 2; ++x)
              s_part[((side * 4 + u * 2 + half) * 2 + x) * kTile + key] =
                  (f2_lo(sum[x][0]) + f2_hi(sum[x][0])) + (f2_lo(sum[x][1]) + f2_hi(sum[x][1]));
          } else if (pair >= kAcc) {
            wait_all(&parts_read[side], ((pair / kAcc) - 1) & 1);
            if (!ok) break;
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&parts[side]);
          if (j > 0) finish(pair - 1);
          known = u < units;
          if (known) look(j, pos);
          last_j = j;
          last_pos = pos;
          pos += (uint32_t)min(2, tiles - j);
        }
        if (ok) finish(pair - 1);
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
