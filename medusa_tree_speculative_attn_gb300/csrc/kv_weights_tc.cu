// Tensor-core path of the slots' attention weights (kv_weights.cu), for calls with more query
// rows than the register-fragment kernel serves well: trees and chunks of a prompt.
//
// A slot's weight is a sum over query rows, so the keys are the M side: a tile of 128 slots
// (eight pages) by up to 256 query rows, S^T = K Q^T, has a key per TMEM lane, and the thread
// that owns the lane adds up its row of exp2(S * scale - lse) in registers, with no reduction
// between threads.  What belongs to a column (its lse, and the query's scale) comes from shared
// memory, the same address for all lanes; what belongs to a key (its page's scale) is the
// thread's own.
//
// Operands stay in 8 bits (kind::f8f6f4): key codes go by TMA straight into the tile, and a
// query row enters as the sum of three (bf16) or four (fp16) E5M2 parts, worked out by the CTA
// when it takes up a segment and kept for all of its tiles.  They hold an element's every bit down
// to 2^-23 (bf16) or 2^-20 (fp16) of its row's largest, and leave at most 2^-31 of that of a smaller
// one, so that keys that miss a query's dominant channel get their scores in 32 bits, too.  Two E4M3
// and E5M2 parts of a bf16 are quicker (60 us for the chunks below) but lose bits from 2^-14 of the
// largest on.
//
// Roles: a warp issues the copies (a lane per page), one the products, sixteen add up, two
// write the weights.  Two accumulators of 256 columns fill TMEM, for even and odd tiles; each
// has a group of eight summing warps, 128 columns a warp, whose two sums of a key meet in
// shared memory, and a writing warp.  Every mbarrier wait is bounded (as in attn_block8_tc.cu),
// and the warps of a role meet by mbarriers too, so that a timeout leaves nobody waiting.
//
// More than 256 query rows of a KV head are taken in passes over the segment's tiles.
//
// Bound by turns: an accumulator is filled, then read out, and two of them are not enough to keep
// either the products or the sums at work all the time.  Chunks of 64 tokens for 8 sequences of 4096
// to 16384, 32 query and 8 KV heads, bf16: 64 us (up to 73 in some processes), 41 % of the products'
// rate; counters: tensor pipe 45 % active, issue 40 %, shared memory's load path 38 % (a column's
// constant is an address common to a warp, but every lane gets its copy), the exponentials' unit
// 30 %.  7000 cycles to begin and 10000 to take up a segment's queries are 14 of them.
// Measured and worse, against 60 us with two parts: a unit of two tiles by 128 columns (68: half
// the constants' reads, but both tiles wait for one another), tile by tile (67); a scale for every
// 16 columns (66), for every column (79); the weights written by the summing warps (69).
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
constexpr int kAcc = 2;  // accumulators, each of a group of eight warps: even and odd tiles
constexpr int kSumWarps = 16, kCopyWarp = 16, kMmaWarp = 17, kWriteWarp = 18, kThreads = 20 * 32;

template <int D, int NP>
struct Cfg {
  static constexpr int kWhole = NP == 3 ? 9 : 6;  // elements of 2^-kWhole and more keep all bits in their parts
  static constexpr int kQPart = kCols * D;
  static constexpr int kQ = NP * kQPart;
  static constexpr int kStage = kTile * D;
  static constexpr int kPart = kAcc * 2 * kTile * 4;
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

// 32 lanes x 32 bits, 16 consecutive columns per thread; and the wait, through which the
// registers pass so that no use of them can move ahead of it.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
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
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// D[tmem] (+)= A[smem] * B[smem]: 8 bits both, K-major, fp32 accumulator.
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

// Instruction descriptor of kind::f8f6f4 with A in E4M3 (format 0 at bits 7-9), B in E5M2 (format 1
// at bits 10-12), both K-major, fp32 accumulator (1 at bits 4-5), N >> 3 at bit 17, M >> 4 at bit 24.
__device__ __forceinline__ uint32_t idesc_f8(int M, int N) {
  return (1u << 4) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
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

// The largest magnitude of a row, NaN left out.
template <typename T, int D>
__device__ __forceinline__ float row_max(const QueryPart<T>& q) {
  AbsMax<T> top;
  top.add(q.r0);
  top.add(q.r1);
  float amax = top.get();
#pragma unroll
  for (int off = 1; off < D / 16; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  return amax;
}

// Biased exponent (in 32 bits) of the smallest magnitude above 0 of a lane's 16 columns, at least
// 255 where there is none.
template <typename T>
__device__ __forceinline__ int least_exponent(const QueryPart<T>& q) {
  const uint4 w0 = q.r0.w[0], w1 = q.r1.w[0];
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint32_t least = 0xffffffffu;  // of both halves, less 1: zeros are largest
#pragma unroll
  for (int e = 0; e < 8; ++e) least = __vminu2(least, __vsub2(w[e] & 0x7fff7fffu, 0x00010001u));
  const uint32_t bits = min(least & 0xffffu, least >> 16) + 1;
  if (bits > 0x7fffu) return 255;
  const uint16_t half = (uint16_t)bits;
  T v;
  memcpy(&v, &half, 2);
  return (int)(__float_as_uint(Act<T>::to_f(v)) >> 23);
}

// A row's scale: the smallest power of two under which its largest magnitude is 57344 = 1.75 * 2^15
// at most, the largest E5M2 (down to 2^-120: it and its inverse are normal numbers).
__device__ __forceinline__ float query_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int k = (int)(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 15 : 14);
  return __uint_as_float((uint32_t)(max(k, -120) + 127) << 23);
}

// Columns 16 c .. 16 c + 15 of query row `row` of this pass, divided by `scale`, as E5M2 parts in
// their places.  A part is the nearest of 3 bits to what the ones before it leave, so NP of them
// hold 3 NP bits: an element's 8 (bf16, 3 parts) or 11 (fp16, 4 parts), all of them, down to a last
// bit of 2^-16, the smallest E5M2.  What they leave of smaller elements is 2^-17 at most.
template <typename T, int D, int NP>
__device__ __forceinline__ void place_query(const QueryPart<T>& q, float scale, uint8_t* sq, int row, int c) {
  const float inv = 1.f / scale;
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
      asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(code) : "r"(bits));
      if (e & 1) w[e / 2] |= (uint32_t)code << 16; else w[e / 2] = code;
      if (part + 1 < NP) {  // what the part leaves, exactly: an E5M2 is the upper byte of an fp16
        const uint32_t h = __byte_perm((uint32_t)code, 0u, 0x1404);
        __half2 v;
        memcpy(&v, &h, 4);
        x[e] = __hsub2(x[e], v);
      }
    }
    *reinterpret_cast<uint4*>(sq + part * (kCols * D) + row_off<D>(row, c)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
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
  float* s_minus = reinterpret_cast<float*>(sK + S * C::kStage);  // [256] of a column: minus its lse
  float* s_scale = s_minus + kCols;                               // [256] its scale (scores of the parts -> base 2)
  float* s_part = s_scale + kCols;  // [accumulator][half of the columns][key]
  int2* s_page = reinterpret_cast<int2*>(s_part + C::kPart / 4);  // [kInfo][8] a tile's pages: number, scale
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_page + kInfo * kPages);
  uint64_t* full = bars;           // [S] a tile's codes have landed
  uint64_t* empty = full + S;      // [S] and are multiplied
  uint64_t* acc_full = empty + S;         // [kAcc] a tile's scores are there
  uint64_t* acc_empty = acc_full + kAcc;  // [kAcc] and read out
  uint64_t* parts = acc_empty + kAcc;     // [kAcc] the sums of a tile are there
  uint64_t* parts_read = parts + kAcc;    // [kAcc] and read
  uint64_t* idle = parts_read + kAcc;     // the warps of sums and weights have left the pass before
  uint64_t* q_full = idle + 1;         // the pass's queries are in place
  uint64_t* fin = q_full + 1;          // every product done
  uint64_t* never = fin + 1;           // nothing arrives here (timeout test hook)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * 6 + 4 * kAcc + 4) * 8 + 8 <= 1024, "barrier area");
  __shared__ int2 s_span[2 * kSumWarps];  // largest and smallest exponent of each warp's query rows, by pass
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
      tc::mbar_init(&parts[s], kSumWarps / kAcc);
      tc::mbar_init(&parts_read[s], 1);
    }
    tc::mbar_init(idle, kSumWarps + 2);
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
          // (the place is free: the products of the tile S before are done, so the sums' groups have
          // left the tiles of their accumulators before it, and the writers of a group the one
          // before that, or the whole pass before: fewer than kInfo tiles back)
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
    uint32_t pos = 0, pass = 0, uses[kAcc] = {};
    static_assert(kAcc == 2, "accumulators");
    if (p.test_stall) wait_all(never, 0);  // test hook: a wait that can only time out
    while (ok && it.next(pc, L)) {
      const int rows = rows_of(pc.b);
      for (int r0 = 0; ok && r0 < rows; r0 += kCols, ++pass) {
        const int cols = (min(kCols, rows - r0) + 31) / 32 * 32;
        wait_all(q_full, pass & 1);
        const uint32_t idesc = idesc_f8(kTile, cols);
        for (int j = pc.tile_begin; j < pc.tile_end; ++j, ++pos) {
          const uint32_t st = pos % S, buf = j & 1, use = buf ? uses[1]++ : uses[0]++;
          wait_all(&full[st], (pos / S) & 1);
          if (use >= 1) wait_all(&acc_empty[buf], (use - 1) & 1);
          if (!ok) break;
          tc::tc_fence_after();
          const uint64_t kd = desc_rows8<D>(sK_u + st * C::kStage);
          const uint32_t d = tmem + buf * kCols;
          if (tc::elect_one()) {
            // the smallest parts first: the accumulator cuts what an addition leaves over, and a small
            // sum loses less (the weights' error 5.0e-7 of the norm with the largest first)
#pragma unroll
            for (int part = NP - 1; part >= 0; --part) {
              const uint64_t qd = desc_rows8<D>(sQ_u + part * C::kQPart);
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) {  // 32 codes: 2 descriptor units
                if (part == NP - 1 && kk == 0) mma_f8_ss<false>(d, kd, qd, idesc);
                else mma_f8_ss<true>(d, kd + (uint64_t)(kk * 2), qd + (uint64_t)(kk * 2), idesc);
              }
            }
            tc::mma_commit(&empty[st]);
            tc::mma_commit(&acc_full[buf]);
          }
          __syncwarp();
          // passes on what this warp acquired with the tile: its pages
          if (lane == 0) tc::mbar_arrive(&acc_full[buf]);
          __syncwarp();
        }
      }
    }
    if (tc::elect_one()) tc::mma_commit(fin);
    __syncwarp();
    if (lane == 0) drain_wait(fin, 0, p.status);
    __syncwarp();
  } else if (warp >= kWriteWarp) {
    // -------------------------------------------------------------- weights
    // A warp writes the tiles of one group, a lane every 32nd slot.  In every pass over a segment
    // a slot is the same thread's, which reads back what it wrote.
    const int x = warp - kWriteWarp;
    uint32_t pos = 0, use = 0, pass = 0;
    while (ok && it.next(pc, L)) {
      const int rows = rows_of(pc.b), prev = p.prev_lens ? p.prev_lens[pc.b] : L;
      for (int r0 = 0; ok && r0 < rows; r0 += kCols, ++pass) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(idle);
        wait_all(idle, pass & 1);
        if (!ok) break;
        const float* before = r0 == 0 ? p.weights : p.out;  // later rows add to what the earlier ones left
        const int had = r0 == 0 ? prev : L;
        const float decay = r0 == 0 ? p.decay : 1.f;
        for (int j = pc.tile_begin; j < pc.tile_end; ++j, ++pos) {
          if ((j & 1) != x) continue;
          wait_all(&parts[x], use & 1);
          if (!ok) break;
          ++use;
          float all[kTile / 32], old[kTile / 32];
          size_t at[kTile / 32];
          bool writes[kTile / 32];
#pragma unroll
          for (int i = 0; i < kTile / 32; ++i) {
            const int key = i * 32 + lane, slot = j * kTile + key;
            const int id = s_page[pos % kInfo * kPages + key / kP].x;
            const bool good = id >= 0 && id < p.num_pages;
            writes[i] = good && slot < L;
            at[i] = ((size_t)(good ? id : 0) * p.Hkv + pc.kvh) * kP + key % kP;
            old[i] = writes[i] && slot < had ? before[at[i]] : 0.f;
            if (id != kNone && !good) set_status(p.status, kStPages);
            all[i] = s_part[x * 2 * kTile + key] + s_part[(x * 2 + 1) * kTile + key];
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&parts_read[x]);
#pragma unroll
          for (int i = 0; i < kTile / 32; ++i)
            if (writes[i]) p.out[at[i]] = fmaf(old[i], decay, all[i]);
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- sums
    const int quad = warp & 3, half = warp >> 2 & 1;  // TMEM lanes 32 quad ..; half of the columns
    const int group = warp >> 3;                      // tiles of this parity
    const int key = quad * 32 + lane;                 // of a tile
    const uint32_t addr = tmem + ((uint32_t)(quad * 32) << 16) + group * kCols;
    const float inv_g = 1.f / (float)p.g;
    uint32_t pos = 0, use = 0, pass = 0;
    while (ok && it.next(pc, L)) {
      const int b = pc.b, h = pc.kvh, rows = rows_of(b);
      if (rows == 0 && threadIdx.x == 0) set_status(p.status, kStPages);
      const int* path = p.accept_path ? p.accept_path + (size_t)b * (p.max_depth + 1) : nullptr;
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
        // each row's scale is a power of two of its own, unless all elements keep their bits under
        // the largest one
        float amax[IT];
        int top = INT_MIN, low = INT_MAX;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          amax[i] = row_max<T, D>(raw[i]);
          low = min(low, least_exponent(raw[i]));
          if (amax[i] > 0.f) top = max(top, (int)(__float_as_uint(query_scale(amax[i])) >> 23));
          if (!(amax[i] < INFINITY)) low = -1000;
        }
        top = __reduce_max_sync(0xffffffffu, top);
        low = __reduce_min_sync(0xffffffffu, low);
        if (lane == 0) s_span[(pass & 1) * kSumWarps + warp] = make_int2(top, low);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(idle);
        wait_all(idle, pass & 1);
        if (!ok) break;
        {
          const int2 span = s_span[(pass & 1) * kSumWarps + (lane & (kSumWarps - 1))];
          top = __reduce_max_sync(0xffffffffu, span.x);
          low = __reduce_min_sync(0xffffffffu, span.y);
        }
        // (no row above 0: any scale)
        const float shared = top == INT_MIN ? 1.f : __uint_as_float((uint32_t)top << 23);
        const bool same = top == INT_MIN || top - low <= C::kWhole;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int row = (i * kSumWarps + warp) * RPW + lane / LPR;
          if ((i * kSumWarps + warp) * RPW >= cols) break;  // the same for the warp
          const float scale = same ? shared : query_scale(amax[i]);
          place_query<T, D, NP>(raw[i], scale, sQ, row, lane % LPR);
          if (lane % LPR == 0) {
            s_minus[row] = -l2[i] * 1.4426950408889634f;
            // an infinity has no parts: the row's weights become NaN, as they would be
            s_scale[row] = row >= n ? 0.f : amax[i] < INFINITY ? scale * p.scale_log2 : __int_as_float(0x7fffffff);
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(q_full);
        wait_all(q_full, pass & 1);
        const int c0 = half * (cols / 2), steps = cols / 32;  // sixteens of a half
        const uint32_t from = addr + c0;
        for (int j = pc.tile_begin; j < pc.tile_end; ++j, ++pos) {
          if ((j & 1) != group) continue;
          wait_all(&acc_full[group], use & 1);
          if (!ok) break;
          tc::tc_fence_after();
          const float ks = __int_as_float(s_page[pos % kInfo * kPages + key / kP].y);
          F2 sum0 = f2_of(0.f, 0.f), sum1 = sum0;
          uint32_t s[2][16];  // sixteen columns are added while sixteen are on their way
          auto walk = [&](auto add16) {
            tmem_ld_x16(from, s[0]);
#pragma unroll 1
            for (int y = 0; y < steps; y += 2) {
              tmem_ld_wait(s[0]);
              if (y + 1 < steps) tmem_ld_x16(from + (y + 1) * 16, s[1]);
              add16(s[0], y);
              if (y + 1 == steps) break;
              tmem_ld_wait(s[1]);
              if (y + 2 < steps) tmem_ld_x16(from + (y + 2) * 16, s[0]);
              add16(s[1], y + 1);
            }
          };
          auto take = [&](F2 z, F2& to) { to = f2_add(to, f2_of(fast_exp2(f2_lo(z)), fast_exp2(f2_hi(z)))); };
          auto two = [](const uint32_t* v) { return f2_of(__uint_as_float(v[0]), __uint_as_float(v[1])); };
          const float4* minus = reinterpret_cast<const float4*>(s_minus + c0);
          if (same) {
            const float k1 = score_factor(shared * p.scale_log2, ks);
            const F2 k = f2_of(k1, k1);
            walk([&](const uint32_t (&v)[16], int y) {
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 c = minus[y * 4 + i / 4];
                take(f2_fma(two(v + i), k, f2_of(c.x, c.y)), sum0);
                take(f2_fma(two(v + i + 2), k, f2_of(c.z, c.w)), sum1);
              }
            });
          } else {
            const float4* scale = reinterpret_cast<const float4*>(s_scale + c0);
            walk([&](const uint32_t (&v)[16], int y) {
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 c = minus[y * 4 + i / 4], e = scale[y * 4 + i / 4];
                take(f2_fma(two(v + i), f2_of(score_factor(e.x, ks), score_factor(e.y, ks)), f2_of(c.x, c.y)), sum0);
                take(f2_fma(two(v + i + 2), f2_of(score_factor(e.z, ks), score_factor(e.w, ks)), f2_of(c.z, c.w)), sum1);
              }
            });
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&acc_empty[group]);
          if (use >= 1) wait_all(&parts_read[group], (use - 1) & 1);
          if (!ok) break;
          ++use;
          s_part[(group * 2 + half) * kTile + key] = (f2_lo(sum0) + f2_hi(sum0)) + (f2_lo(sum1) + f2_hi(sum1));
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&parts[group]);
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
  s.seg_cost = 5;
  return launch_pdl(kv_weights_tc_kernel<T, D, NP>, dim3(s.G), dim3(kThreads), (size_t)C::kSmem + 4 * ((size_t)p.B + 1),
                    stream, map, p, s);
}

}  // namespace

cudaError_t launch_kv_weights_tc(const WeightsParams& p, int dtype, cudaStream_t stream) {
  if (p.D == 64) return dtype == 1 ? launch_t<__half, 64, 4>(p, stream) : launch_t<__nv_bfloat16, 64, 3>(p, stream);
  return dtype == 1 ? launch_t<__half, 128, 4>(p, stream) : launch_t<__nv_bfloat16, 128, 3>(p, stream);
}

}  // namespace mt
