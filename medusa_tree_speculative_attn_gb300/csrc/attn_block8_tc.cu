// Tensor-core path of the block-scaled attention (sm_103a: tcgen05 + TMEM +
// TMA), for calls with more query rows than the register-fragment kernel
// serves well (attn_block8.cu; the choice is block8_plan's).
//
// The structure is the 16-bit kernel's (attn_tc.cu): persistent CTAs, one per
// SM, walk the balanced schedule; a CTA holds up to MT * 128 query rows of one
// (sequence, KV head) and streams 64-slot tiles of four pages.  What differs is
// how 8-bit operands reach the tensor cores:
//   S = Q K^T  stays in 8 bits (kind::f8f6f4): the cache's key codes go by TMA
//              straight into the operand tile, and a query row enters as the
//              sum of two (bf16) or three (fp16) E4M3 parts (block8_prep.cu),
//              which multiply the same key tile one after the other into the
//              same accumulator.  An 8-bit step covers 32 of the D products in
//              the time that a 16-bit step takes for 16, so two parts cost what
//              a 16-bit product costs, and no key is ever converted;
//   O = P V    needs softmax weights over a wider range than 8 bits hold, so it
//              runs in fp16: four warps convert value codes to fp16 (exact, one
//              instruction for two codes) on the way into the tile.
// Scales: a page's key scale multiplies its 16 columns of S in the softmax's
// exponent (no extra operation); its value scale 2^lv joins the exponent, so the
// running maximum is that of (score + lv), P = 2^(score + lv - max + 3) fits
// fp16, and the row's sum takes each page's part times 2^-lv.
//
// Warps: 4 * MT softmax warps (one thread per query row), one issuing Q K^T, one
// issuing P V, two issuing the copies (a lane per page of a tile) and four
// converting (a page each).  Issuing and converting are apart because each is a
// chain of short steps that one warp cannot overlap: in one warp they took 2250
// cycles a tile, more than the softmax (stamps in a copy of the kernel).  A ring
// slot is one tile (keys in 8 bits, value codes, values in fp16) or one part of an
// M tile's queries, copied to TMEM.  Every mbarrier wait is bounded; on a timeout
// MT_ERR_TIMEOUT is recorded, the other roles stop, the copies and MMAs in flight
// are waited for and TMEM is freed.
//
// Bound by the roles' chains of steps, not by a unit: with 256 rows a tile takes
// about 1950 cycles, of which the tensor cores work 1070 and the schedulers issue
// half.  8 sequences of 32768 keys, 26 nodes, 64 query and 8 KV heads: 228 us, 53 % of
// the products' floor (238 called with other inputs each time); 16 sequences of 512 to
// 8192 keys, 64 nodes, 32 query and 8 KV heads: 95 us; 64 sequences of 256 to 8192 keys,
// 32 rows a head: 176 us, 47 % of a copy of the cache.
#include <cudaTypedefs.h>

#include <atomic>
#include <climits>

#include "serve.cuh"
#include "tc_ptx.cuh"

namespace mt {

namespace {

constexpr int kSmemLimit = 232448;  // opt-in dynamic shared memory per CTA
constexpr int kMaxDevices = 64;
constexpr int kPages = kTileKeys / 16;  // of a tile

template <int D, int MT, int NP>
struct Cfg {
  static constexpr int NH = D / 64;                   // 64-column halves of an fp16 value row
  static constexpr int kPTile = 128 * kTileKeys * 2;  // P of one M tile: 128 rows x 128 B
  // P tiles of an M tile, by turns: with two, P does not wait for the P V of the tile
  // before.  8 sequences of 208 rows and 32768 keys 240 -> 229 us; with MT = 1 the ring
  // slot that it takes costs more (64 sequences of 32 rows 181 -> 186, fp16 184 -> 198).
  static constexpr int PB = MT == 2 ? 2 : 1;
  static constexpr int kPBytes = MT * PB * kPTile;
  static constexpr int kKTile = kTileKeys * D;        // key codes, swizzled rows of D bytes
  static constexpr int kHalf = kTileKeys * 128;       // 64 values of 64 columns
  static constexpr int kVTile = NH * kHalf;
  static constexpr int kV8 = kKTile;                  // value codes, plain rows
  static constexpr int kStage = kKTile + kVTile + kV8;  // >= 128 * D: one part of an M tile's queries
  static constexpr int kMetaBytes = 4096;  // barriers, scales, piece list
  static constexpr int kFit = (kSmemLimit - 1024 - kMetaBytes - kPBytes) / kStage;
  static constexpr int STAGES = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = 1024 + kPBytes + STAGES * kStage + kMetaBytes;
  static constexpr int kSoftmaxWarps = 4 * MT;
  static constexpr int kQkWarp = kSoftmaxWarps;
  static constexpr int kPvWarp = kSoftmaxWarps + 1;
  static constexpr int kCopyWarp = kSoftmaxWarps + 2;
  // One copy warp was busy for 1700 cycles a tile: 64 sequences of 32 rows took 199 us
  // (fp16 204) against 184 (187) with two, 8 of 208 rows 241 against 238.
  static constexpr int kCopyWarps = 2;
  static constexpr int kConvert0 = kCopyWarp + kCopyWarps;
  static constexpr int kThreads = (kConvert0 + kPages) * 32;
  static constexpr int kQSlots = MT * NP;  // ring slots of a piece's queries
  // TMEM: O (D fp32 columns per M tile), S (64), Q (D / 4 columns of four codes per part)
  static constexpr int kTmemUsed = MT * (D + kTileKeys + NP * (D / 4));
  static constexpr int kTmemCols = kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static_assert(kTmemUsed <= 512, "TMEM budget");
  static_assert(STAGES >= 3 && kStage >= 128 * D, "shared memory budget");
  __device__ static constexpr uint32_t o_col(int m) { return (uint32_t)(m * D); }
  __device__ static constexpr uint32_t s_col(int m) { return (uint32_t)(MT * D + m * kTileKeys); }
  __device__ static constexpr uint32_t q_col(int m, int part) {
    return (uint32_t)(MT * (D + kTileKeys) + (m * NP + part) * (D / 4));
  }
};

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

// 32 lanes x 32 bits, 32 consecutive columns per thread; and the wait, through which
// the registers pass so that no use of them can move ahead of it.
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
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// D[tmem] (+)= A[tmem] * B[smem]: E4M3 both, fp32 accumulator; A is M x 32, one
// row per lane, four consecutive codes per 32-bit column.
template <bool ACC>
__device__ __forceinline__ void mma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc) {
  if (ACC) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.eq.u32 p, 1, 1;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc)
        : "memory");
  } else {
    asm volatile(
        "{\n.reg .pred p;\nsetp.eq.u32 p, 1, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc)
        : "memory");
  }
}

// Instruction descriptor of kind::f8f6f4 with E4M3 operands (format 0), both
// K-major, fp32 accumulator (1 at bits 4-5), N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// K-major matrix of rows of D bytes, swizzled over 128 (D = 128) or 64 bytes:
// eight-row groups D * 8 bytes apart; swizzle mode at bits 61-63 (2: 128, 4: 64).
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

// What a wait does when its first try fails, out of line: the roles share the
// instruction caches (1.5% with MT = 1).
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

// Visibility of the 64 columns of tile j: cached slot s < L, or a new token of
// the row's ancestor mask.  Columns are pages: npre cached ones, then the new
// tokens' blocks, so new token t sits at column npre * 16 + t.
__device__ __forceinline__ unsigned long long visible(int L, int npre, int k0, unsigned long long anc) {
  const int pre = L - k0, base = npre * 16 - k0;
  unsigned long long see = pre >= 64 ? ~0ull : pre <= 0 ? 0ull : (1ull << pre) - 1ull;
  if (base < 64) see |= base >= 0 ? anc << base : base > -64 ? anc >> -base : 0ull;
  return see;
}

// Whether 16 codes hold a NaN; those that do become 0.
__device__ __forceinline__ bool drop_nan(uint4& c) {
  uint32_t w[4] = {c.x, c.y, c.z, c.w};
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
    nan = nan || m != 0u;
    w[i] &= ~m;
  }
  c = make_uint4(w[0], w[1], w[2], w[3]);
  return nan;
}

// Columns of tile j (from k0) that are cached pages'.
__device__ __forceinline__ unsigned long long cached(int npre, int k0) { return Reach::below64(npre * 16 - k0); }

// REACH: with a window and sinks, and the rows' log-sum-exp.  Only the visible pages are
// streamed.  A value row of the window's edge, which not every node sees, must not bring a
// NaN to those that do not: its NaN codes are 0 in the products, and each row that sees it
// looks for them itself at its end (a CTA that has met one).  16 sequences of 512 to 32768
// keys under a window of 4096, 64 nodes, 32 query and 8 KV heads: 88 us, 40 % of the
// products' rate, as without a window.
template <typename T, int D, int MT, int NP, bool REACH>
__global__ void __launch_bounds__(Cfg<D, MT, NP>::kThreads, 1)
    attn_block8_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                          const __grid_constant__ CUtensorMap map_kn, const __grid_constant__ CUtensorMap map_vn,
                          const __grid_constant__ CUtensorMap map_q, const Block8Params p) {
  using C = Cfg<D, MT, NP>;
  constexpr int S = C::STAGES, PB = C::PB;
  constexpr uint32_t kIdescQK = idesc_f8(128, kTileKeys);
  // Rows of an M tile: whole nodes.  Where g does not divide 128 the rest of a tile's rows are what
  // was left in their place; no row's result depends on another's.
  const int RT = REACH ? p.a.rows_per_group / MT : 128;
  constexpr uint32_t kIdescPV = tc::idesc_f16(false, true, 128, D);
  const AttnParams& a = p.a;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sP = smem;                       // [m] P tiles, 128-byte swizzled, K-major
  uint8_t* sKV = sP + C::kPBytes;           // [stage] keys, values, value codes
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + S * C::kStage);
  uint64_t* land = bars;                    // [S] a tile's codes, or query rows, have landed
  uint64_t* full = land + S;                // [S] a tile's values are converted (tiles only)
  uint64_t* empty = full + S;               // [S] consumed by the MMAs (or copied to TMEM) and by the four converters
  uint64_t* s_full = empty + S;             // [MT] S computed
  uint64_t* p_full = s_full + MT;           // [MT][PB] P written (and O rescaled)
  uint64_t* pv_done = p_full + MT * C::PB;  // [MT][PB] O += P V done
  uint64_t* s_free = pv_done + MT * C::PB;  // [MT] S read out
  uint64_t* o_free = s_free + MT;           // O of the previous piece read out
  uint64_t* fin = o_free + 1;               // [2] every MMA of each issuer done
  uint64_t* never = fin + 2;                // nothing arrives here (timeout test hook)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_npieces = const_cast<int*>(abort_flag + 1);
  volatile int* s_nan = s_npieces + 1;  // REACH: a value row of the window's edge had a NaN
  static_assert((3 * 8 + 8 * 2 + 4) * 8 + 16 <= 1024, "barrier area");
  // per stage: key scales, log2 and inverse of the value scales, and how many rows
  // of each page hold keys of the sequence
  float* s_scale = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + 1024);  // [S][4][4]
  static_assert(8 * 16 * 4 <= 1024, "metadata");
  PieceRec* s_pieces = reinterpret_cast<PieceRec*>(reinterpret_cast<uint8_t*>(bars) + 2048);
  static_assert(2048 + kMaxPieceRecs * sizeof(PieceRec) <= C::kMetaBytes, "piece list");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nnew = (a.T + 15) / 16;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&land[s], 1);
      tc::mbar_init(&full[s], kPages);
      tc::mbar_init(&empty[s], 1 + kPages);
    }
    for (int m = 0; m < MT; ++m) {
      tc::mbar_init(&s_full[m], 2);  // the MMAs, and the issuer itself (below)
      for (int i = 0; i < C::PB; ++i) {
        tc::mbar_init(&p_full[m * C::PB + i], 4);
        tc::mbar_init(&pv_done[m * C::PB + i], 1);
      }
      tc::mbar_init(&s_free[m], 4);
    }
    tc::mbar_init(o_free, C::kSoftmaxWarps);
    tc::mbar_init(&fin[0], 1);
    tc::mbar_init(&fin[1], 1);
    tc::mbar_init(never, 1);
    *abort_flag = 0;
    *s_nan = 0;
    tc::fence_barrier_init();
  }
  if (warp == C::kQkWarp) {
    tc::tmem_alloc(tmem_slot, C::kTmemCols);
    tc::tmem_relinquish();
  }
  if (warp == C::kCopyWarp && lane == 0) {
    tc::prefetch_tmap(&map_k);
    tc::prefetch_tmap(&map_v);
    tc::prefetch_tmap(&map_kn);
    tc::prefetch_tmap(&map_vn);
    tc::prefetch_tmap(&map_q);
  }
  pdl_wait();  // everything above overlaps the preparation's end
  if (warp == C::kPvWarp) {
    // this CTA's pieces: the first four records with the count, the rest (rare) after
    const int* src = p.pieces + piece_rec_offset(a.sched.G) + (size_t)blockIdx.x * kMaxPieceRecs * 8;
    const int first = src[lane];
    const int n = p.pieces[blockIdx.x];
    int* dst = reinterpret_cast<int*>(s_pieces);
    dst[lane] = first;
    if (lane == 0) *s_npieces = n;
    for (int e = 32 + lane; e < (n > 0 ? n : 0) * 8; e += 32) dst[e] = src[e];
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sKV_u = tc::smem_u32(sKV), sP_u = tc::smem_u32(sP);
  bool ok = true;
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    const bool r = tc::mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_flag, a.status, a.wait_limit_ns);
    ok = __all_sync(0xffffffffu, r) && ok;
  };
  PieceSrc pi;
  pi.init(s_pieces, *s_npieces, a.sched, blockIdx.x, a.seq_lens);
  Piece pc;
  int L = 0;

  if (warp >= C::kCopyWarp && warp < C::kCopyWarp + C::kCopyWarps) {
    // -------------------------------------------------------------- copies
    // The two warps share the ring by slots, odd and even: a slot's every `empty`
    // phase is then waited for by one warp, in order.  (By positions, a warp could
    // come to a slot whose last phase but one is still open, and a wait by parity
    // would take that for the last: the other warp's position is two phases back,
    // and queries are consumed ahead of the tiles before them.)
    const uint32_t turn = warp - C::kCopyWarp;
    const uint64_t policy = tc::policy_evict_first();
    const uint64_t q_policy = tc::policy_evict_last();
    const int oob_row = a.num_pages * a.Hkv * 16;  // past the cache: TMA fills zeros
    uint32_t pos = 0;                              // ring position
    while (ok && pi.next(pc, L)) {
      // the piece's queries: part `part` of M tile m per ring slot
      for (int s = 0; s < C::kQSlots && ok; ++s, ++pos) {
        const uint32_t st = pos % S;
        if (st % C::kCopyWarps != turn) continue;
        if (pos >= (uint32_t)S) wait_all(&empty[st], ((pos / S) - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          const int m = s / NP, part = s % NP;
          tc::mbar_arrive_expect_tx(&land[st], RT * D);
          tc::tma_load_3d(sKV + st * C::kStage, &map_q, 0, pc.kvh * a.g,
                          (part * a.B + pc.b) * a.T + (pc.rg * a.rows_per_group + m * RT) / a.g, &land[st], q_policy);
        }
        __syncwarp();
      }
      if (!ok) break;
      // page ids and scales of 32 pages of the table at a time, a lane each; ids
      // are fetched two windows ahead of use, scales one
      const Reach reach(L, REACH ? p.window : INT_MAX, REACH ? p.sinks : 0);
      const int npre = REACH ? reach.npre : (L + 15) / 16;
      const int* bt = a.block_tables + (size_t)pc.b * a.max_blocks;
      const size_t nb0 = ((size_t)pc.b * a.Hkv + pc.kvh) * nnew;  // the new tokens' blocks
      auto fetch_id = [&](int q) { return q < npre ? __ldg(bt + (REACH ? reach.page(q) : q)) : -1; };
      auto fetch_scale = [&](const float* sc, int id) {
        return id >= 0 && id < a.num_pages ? __ldg(sc + (size_t)id * a.Hkv + pc.kvh) : 1.f;
      };
      // value scales are positive; a smaller one (or one that is no number) would
      // leave the exponent's range
      auto clamp = [](float v) { return fmaxf(v, 5.421010862427522e-20f); };
      int base = pc.tile_begin * 4;
      int id0 = fetch_id(base + lane), id1 = fetch_id(base + 32 + lane), id2 = fetch_id(base + 64 + lane);
      float ks0 = fetch_scale(p.k_scales, id0), vs0 = clamp(fetch_scale(p.v_scales, id0));
      float ks1 = fetch_scale(p.k_scales, id1), vs1 = fetch_scale(p.v_scales, id1);
      float lv0 = log2f(vs0), iv0 = 1.f / vs0;
      for (int j = pc.tile_begin; j < pc.tile_end; ++j, ++pos) {
        if (j * 4 - base >= 32) {  // windows are whole tiles
          base += 32;
          id0 = id1;
          ks0 = ks1;
          vs0 = clamp(vs1);
          lv0 = log2f(vs0);
          iv0 = 1.f / vs0;
          id1 = id2;
          ks1 = fetch_scale(p.k_scales, id1);
          vs1 = fetch_scale(p.v_scales, id1);
          id2 = fetch_id(base + 64 + lane);
        }
        const uint32_t st = pos % S;
        if (st % C::kCopyWarps != turn) continue;
        // lane l < 4 has page l of the tile
        const int pg = j * 4 + (lane & 3);
        const int id = __shfl_sync(0xffffffffu, id0, pg - base);
        float ks = __shfl_sync(0xffffffffu, ks0, pg - base), lv = __shfl_sync(0xffffffffu, lv0, pg - base);
        float iv = __shfl_sync(0xffffffffu, iv0, pg - base);
        int row = oob_row, rows = 0;
        const bool from_new = pg >= npre && pg - npre < nnew;
        if (pg < npre) {
          if (id >= 0 && id < a.num_pages) {
            row = (id * a.Hkv + pc.kvh) * 16;
            // REACH: the rows that some node sees, and those that not every node sees
            if (REACH) {
              rows = (int)reach.see16(pg * 16, 0);
              rows |= (rows & ~(int)reach.see16(pg * 16, a.T - 1)) << 16;
            } else {
              rows = min(16, L - pg * 16);
            }
          } else if (lane < kPages) {
            set_status(a.status, kStPages);
          }
        } else if (from_new) {
          row = (int)((nb0 + pg - npre) * 16);
          rows = REACH ? 0xffff : 16;
          ks = __ldg(p.k_block_scales + nb0 + pg - npre);
          const float vs = clamp(__ldg(p.v_block_scales + nb0 + pg - npre));
          lv = log2f(vs);
          iv = 1.f / vs;
        }
        if (pos >= (uint32_t)S) wait_all(&empty[st], ((pos / S) - 1) & 1);
        if (!ok) break;
        if (lane < kPages) {
          float* sc = s_scale + st * 16 + lane;
          sc[0] = ks;
          sc[4] = lv;
          sc[8] = iv;
          sc[12] = __int_as_float(rows);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_expect_tx(&land[st], 2 * C::kKTile);
        __syncwarp();
        if (lane < kPages) {
          uint8_t* stage = sKV + st * C::kStage + lane * 16 * D;
          tc::tma_load_2d(stage, from_new ? &map_kn : &map_k, 0, row, &land[st], policy);
          tc::tma_load_2d(stage + C::kKTile + C::kVTile, from_new ? &map_vn : &map_v, 0, row, &land[st], policy);
        }
        __syncwarp();
      }
    }
    // no TMA load of this warp's may still be writing shared memory when the CTA exits
    if (lane == 0)
      for (uint32_t t = pos > (uint32_t)S ? pos - S : 0; t < pos; ++t)
        if (t % S % C::kCopyWarps == turn) drain_wait(&land[t % S], (t / S) & 1, a.status);
    __syncwarp();
  } else if (warp >= C::kConvert0) {
    // ---------------------------------------------------------- conversion
    // Warp pid turns page pid's value codes into fp16: 16-byte chunks of codes,
    // consecutive lanes on consecutive chunks, become two 8-column chunks of the
    // 128-byte-swizzled rows.  The slot is the warp's once the codes have landed
    // (they were asked for after its last use).
    const int pid = warp - C::kConvert0;
    uint32_t pos = 0;
    while (ok && pi.next(pc, L)) {
      // The queries' slots too are waited for and given back: a wait by parity must
      // neither skip a phase nor come two late.
      for (int s = 0; s < C::kQSlots && ok; ++s, ++pos) {
        wait_all(&land[pos % S], (pos / S) & 1);
        if (lane == 0) tc::mbar_arrive(&empty[pos % S]);
        __syncwarp();
      }
      if (!ok) break;
      for (int j = pc.tile_begin; j < pc.tile_end; ++j, ++pos) {
        const uint32_t st = pos % S;
        wait_all(&land[st], (pos / S) & 1);
        if (!ok) break;
        uint8_t* stage = sKV + st * C::kStage;
        const uint8_t* codes = stage + C::kKTile + C::kVTile + pid * 16 * D;
        const int rows = __float_as_int(s_scale[st * 16 + 12 + pid]);
        constexpr int CPR = D / 16;
#pragma unroll
        for (int i = 0; i < 16 * CPR / 32; ++i) {
          const int q = i * 32 + lane;
          const int r = q / CPR, col = (q % CPR) * 16;
          uint4 c = *reinterpret_cast<const uint4*>(codes + q * 16);
          // rows that hold no key of the sequence may hold anything (NaN codes
          // too): their weights are 0 and so are their values
          if (REACH ? !(rows >> r & 1) : r >= rows) c = make_uint4(0, 0, 0, 0);
          if (REACH && (rows >> (16 + r) & 1) && drop_nan(c)) *s_nan = 1;
          const int row = pid * 16 + r, c0 = (col % 64) / 8;
          uint8_t* dst = stage + C::kKTile + (col / 64) * C::kHalf + row * 128;
          const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<uint4*>(dst + (((c0 + h) ^ (row & 7)) << 4)) =
                make_uint4(e4m3x2_to_h2(w[2 * h] & 0xffffu), e4m3x2_to_h2(w[2 * h] >> 16),
                           e4m3x2_to_h2(w[2 * h + 1] & 0xffffu), e4m3x2_to_h2(w[2 * h + 1] >> 16));
        }
        tc::fence_proxy_async_smem();  // read by the tensor core; the codes' place is refilled by TMA
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&full[st]);
          tc::mbar_arrive(&empty[st]);
        }
        __syncwarp();
      }
    }
  } else if (warp == C::kQkWarp) {
    // ---------------------------------------------------------- QK issuer
    uint32_t it = 0, pos = 0;  // tiles so far; ring position
    uint32_t phase = 0;        // bit s: parity of slot s's next tile (queries leave `full` alone)
    if (a.test_stall) wait_all(never, 0);  // test hook: a wait that can only time out
    while (ok && pi.next(pc, L)) {
      // the queries in TMEM give way once the products that read them are done
      if (it >= 1)
        for (int m = 0; m < MT; ++m) wait_all(&s_full[m], (it - 1) & 1);
#pragma unroll 1  // unrolled, its code costs the fp16 kernel up to 12% (the roles share the instruction caches)
      for (int s = 0; s < C::kQSlots && ok; ++s) {
        const uint32_t st = (pos + s) % S;
        wait_all(&land[st], ((pos + s) / S) & 1);
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t qd = desc_rows8<D>(sKV_u + st * C::kStage);
        const uint32_t col = tmem + C::q_col(s / NP, s % NP);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)  // 32 codes: 2 descriptor units, 8 columns
          if (tc::elect_one()) tc::tmem_cp_128x256b(col + kk * 8, qd + (uint64_t)(kk * 2));
        if (tc::elect_one()) tc::mma_commit(&empty[st]);
        __syncwarp();
      }
      if (!ok) break;
      pos += C::kQSlots;
      for (int j = pc.tile_begin; j < pc.tile_end; ++j, ++it, ++pos) {
        const uint32_t st = pos % S;
        wait_all(&full[st], (phase >> st) & 1);
        phase ^= 1u << st;
        if (!ok) break;
        const uint64_t kd = desc_rows8<D>(sKV_u + st * C::kStage);
#pragma unroll 1  // (short code: 2% with MT = 2)
        for (int m = 0; m < MT; ++m) {
          if (it >= 1) {
            wait_all(&s_free[m], (it - 1) & 1);
            if (!ok) break;
          }
          tc::tc_fence_after();
          if (tc::elect_one()) {
#pragma unroll
            for (int part = 0; part < NP; ++part)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) {
                const uint32_t q = tmem + C::q_col(m, part) + kk * 8;
                if (part == 0 && kk == 0) mma_f8_ts<false>(tmem + C::s_col(m), q, kd, kIdescQK);
                else mma_f8_ts<true>(tmem + C::s_col(m), q, kd + (uint64_t)(kk * 2), kIdescQK);
              }
            tc::mma_commit(&s_full[m]);
          }
          __syncwarp();
          // passes on what this warp acquired with the tile: the softmax reads the
          // page scales without a wait of its own on `land` (4% of the 32k workload)
          if (lane == 0) tc::mbar_arrive(&s_full[m]);
          __syncwarp();
        }
        if (!ok) break;
      }
    }
    if (tc::elect_one()) tc::mma_commit(&fin[0]);
    __syncwarp();
    if (lane == 0) drain_wait(&fin[0], 0, a.status);
    __syncwarp();
  } else if (warp == C::kPvWarp) {
    // ---------------------------------------------------------- PV issuer
    uint32_t it = 0, npieces = 0, pos = 0;
    while (ok && pi.next(pc, L)) {
      pos += C::kQSlots;
      for (int j = pc.tile_begin; j < pc.tile_end; ++j, ++it, ++pos) {
        const uint32_t st = pos % S;
        const bool first = j == pc.tile_begin;
        if (first && npieces > 0) {
          wait_all(o_free, (npieces - 1) & 1);
          if (!ok) break;
        }
        const uint32_t v_u = sKV_u + st * C::kStage + C::kKTile;
        const uint64_t vd = tc::smem_desc(v_u, C::kHalf, 1024);
#pragma unroll 1
        for (int m = 0; m < MT; ++m) {
          wait_all(&p_full[m * PB + it % PB], (it / PB) & 1);
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t d_t = tmem + C::o_col(m);
          const uint64_t pd = tc::smem_desc(sP_u + (m * PB + it % PB) * C::kPTile, 16, 1024);
          if (first) {
            if (tc::elect_one()) tc::mma_f16_ss<false>(d_t, pd, vd, kIdescPV);
          } else {
            if (tc::elect_one()) tc::mma_f16_ss<true>(d_t, pd, vd, kIdescPV);
          }
#pragma unroll
          for (int kk = 1; kk < kTileKeys / 16; ++kk)  // next 16 keys: P +32 B, V +2048 B
            if (tc::elect_one()) tc::mma_f16_ss<true>(d_t, pd + (uint64_t)(kk * 2), vd + (uint64_t)(kk * 128), kIdescPV);
          if (tc::elect_one()) tc::mma_commit(&pv_done[m * PB + it % PB]);
          __syncwarp();
        }
        if (!ok) break;
        if (tc::elect_one()) tc::mma_commit(&empty[st]);
        __syncwarp();
      }
      ++npieces;
    }
    if (tc::elect_one()) tc::mma_commit(&fin[1]);
    __syncwarp();
    if (lane == 0) drain_wait(&fin[1], 0, a.status);
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    const int m = warp >> 2;              // M tile of this warpgroup
    const int quad = warp & 3;            // TMEM lane quadrant
    const int r = quad * 32 + lane;       // row within the M tile
    const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
    uint32_t it = 0, pos = 0;
    while (ok && pi.next(pc, L)) {
      pos += C::kQSlots;
      const int row = pc.rg * a.rows_per_group + m * RT + r;
      const bool row_ok = row < a.rows && r < RT;
      const int node = row_ok ? row / a.g : 0, h = pc.kvh * a.g + (row_ok ? row % a.g : 0);
      const unsigned long long anc = p.anc[(size_t)pc.b * a.T + node];
      const float qs = p.q_scale[((size_t)pc.b * a.T + node) * a.Hq + h];
      const Reach reach(L, REACH ? p.window : INT_MAX, REACH ? p.sinks : 0);
      const int npre = REACH ? reach.npre : (L + 15) / 16;
      const int depth = REACH ? p.depth[(size_t)pc.b * a.T + node] : 0;
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = pc.tile_begin; j < pc.tile_end; ++j, ++it, ++pos) {
        wait_all(&s_full[m], it & 1);
        if (!ok) break;
        tc::tc_fence_after();
        uint32_t sr[64];
        tc::tmem_ld_x64(tmem + lane_addr + C::s_col(m), sr);
        const uint32_t st = pos % S;
        const float4 ks = *reinterpret_cast<const float4*>(s_scale + st * 16);
        const float4 lv = *reinterpret_cast<const float4*>(s_scale + st * 16 + 4);
        const float4 iv = *reinterpret_cast<const float4*>(s_scale + st * 16 + 8);
        float c4[4] = {ks.x * qs, ks.y * qs, ks.z * qs, ks.w * qs};
        const float l4[4] = {lv.x, lv.y, lv.z, lv.w}, i4[4] = {iv.x, iv.y, iv.z, iv.w};
        tc::tmem_ld_wait();
        // the scores are in registers: S may take the next tile's scores
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&s_free[m]);
        const int k0 = j * kTileKeys;
        if (REACH ? reach.partial(k0, kTileKeys, a.T - 1) : k0 + kTileKeys > L) {
          const unsigned long long see = REACH ? (visible(reach.Lv, npre, k0, anc) & ~cached(npre, k0)) | reach.see64(k0, depth)
                                               : visible(L, npre, k0, anc);
#pragma unroll
          for (int hw = 0; hw < 2; ++hw) {
            const uint32_t bits = (uint32_t)(see >> (32 * hw));
            if (bits == 0xffffffffu) continue;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((bits >> c) & 1u)) sr[32 * hw + c] = 0xff800000u;  // -inf
          }
          // -inf comes through the factor: of a page that the row does not see, any will do
          if (REACH) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if (!((uint32_t)(see >> (16 * g)) & 0xffffu)) c4[g] = 1.f;
          }
        }
        // maximum of score + lv: per page of the raw products, then scaled
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          // three inputs an instruction, two chains
          float x0 = __uint_as_float(sr[16 * g]), x1 = __uint_as_float(sr[16 * g + 1]);
#pragma unroll
          for (int c = 2; c < 14; c += 4) {
            x0 = fmaxf(fmaxf(x0, __uint_as_float(sr[16 * g + c])), __uint_as_float(sr[16 * g + c + 1]));
            x1 = fmaxf(fmaxf(x1, __uint_as_float(sr[16 * g + c + 2])), __uint_as_float(sr[16 * g + c + 3]));
          }
          x0 = fmaxf(fmaxf(x0, __uint_as_float(sr[16 * g + 14])), __uint_as_float(sr[16 * g + 15]));
          mx = fmaxf(mx, fmaf(fmaxf(x0, x1), c4[g], l4[g]));
        }
        // O is rescaled only when the maximum grows by more than 8: P <= 2^11
        const bool grow = mx > m_run + 8.f;
        const bool need_o = grow && m_run != -INFINITY;
        const float m_new = grow ? mx : m_run;
        const float sc = need_o ? fast_exp2(m_run - m_new) : 1.f;
        const float off = m_new == -INFINITY ? 0.f : 3.f - m_new;
        uint32_t pk[32];
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float o = off + l4[g];
          const F2 c2 = f2_of(c4[g], c4[g]), o2 = f2_of(o, o);
          F2 s2 = f2_of(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const F2 x = f2_fma(f2_of(__uint_as_float(sr[16 * g + 2 * c]), __uint_as_float(sr[16 * g + 2 * c + 1])), c2, o2);
            const float p0 = fast_exp2(f2_lo(x)), p1 = fast_exp2(f2_hi(x));
            s2 = f2_add(s2, f2_of(p0, p1));
            pk[8 * g + c] = pack_h2(p0, p1);
          }
          sum = fmaf(f2_lo(s2) + f2_hi(s2), i4[g], sum);
        }
        // P once the P.V that read its place last is done: row r is
        // 128 B (64 keys), 16-byte chunk c at c ^ (r % 8)
        if (it >= (uint32_t)PB) {
          wait_all(&pv_done[m * PB + it % PB], (it / PB - 1) & 1);
          if (!ok) break;
        }
        uint8_t* prow = sP + (m * PB + it % PB) * C::kPTile + (r >> 3) * 1024 + (r & 7) * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(prow + ((c ^ (r & 7)) << 4)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        tc::fence_proxy_async_smem();
        if (__any_sync(0xffffffffu, need_o)) {
          if (PB > 1 && it >= 1) {  // O of the tile before
            wait_all(&pv_done[m * PB + (it - 1) % PB], ((it - 1) / PB) & 1);
            if (!ok) break;
          }
          tc::tc_fence_after();
#pragma unroll 1
          for (int hh = 0; hh < D / 64; ++hh) {
            uint32_t o[64];
            tc::tmem_ld_x64(tmem + lane_addr + C::o_col(m) + 64 * hh, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 64; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * sc);
            tc::tmem_st_x64(tmem + lane_addr + C::o_col(m) + 64 * hh, o);
          }
        }
        tc::tmem_st_wait();
        l_run = fmaf(l_run, sc, sum);
        m_run = m_new;
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_full[m * PB + it % PB]);
      }
      if (!ok) break;
      // epilogue, once the piece's last P.V is done: O / l to the output, or the
      // piece's own O / l with its maximum and sum to a partial slot
      wait_all(&pv_done[m * PB + (it - 1) % PB], ((it - 1) / PB) & 1);
      if (!ok) break;
      tc::tc_fence_after();
      const int seg_row = m * RT + r;
      // NaN values at the window's edge, for the columns col .. col + 31 of a row that sees them
      auto edge_nan = [&](uint32_t (&o)[32], int col) {
        const int last = min(reach.edge + a.T - 1, min(reach.Lv, pc.tile_end * kTileKeys));
        for (int c = max(max(reach.edge, 0), pc.tile_begin * kTileKeys); c < last; ++c) {
          if (!(reach.see16(c & ~15, depth) >> (c & 15) & 1u)) continue;
          const int id = a.block_tables[(size_t)pc.b * a.max_blocks + reach.page(c >> 4)];
          if (id < 0 || id >= a.num_pages) continue;
          const uint8_t* v = static_cast<const uint8_t*>(a.v_cache) + (((size_t)id * a.Hkv + pc.kvh) * 16 + (c & 15)) * D + col;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if ((v[i] & 0x7f) == 0x7f) o[i] = 0x7fffffffu;
        }
      };
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;  // a NaN sum makes the row NaN
#pragma unroll 1  // 32 columns at a time: with 64 the code is long enough to slow the other roles (fp16 12%)
      for (int col = 0; col < D; col += 32) {
        uint32_t o[32];
        tmem_ld_x32(tmem + lane_addr + C::o_col(m) + col, o);
        tmem_ld_wait(o);
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * inv);
        if (REACH && row_ok && *s_nan) edge_nan(o, col);
        if (row_ok && pc.slot < 0) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (((size_t)pc.b * a.T + node) * a.Hq + h) * D + col);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            T v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = Act<T>::from_f(__uint_as_float(o[8 * c + e]));
            uint4 w;
            memcpy(&w, v, 16);
            dst[c] = w;
          }
        } else if (row_ok) {
          uint4* dst = reinterpret_cast<uint4*>(a.part_o) + ((size_t)pc.slot * (D / 4) + col / 4) * a.part_rows + seg_row;
#pragma unroll
          for (int c = 0; c < 8; ++c) dst[(size_t)c * a.part_rows] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
      }
      if (row_ok && pc.slot >= 0) a.part_ml[(size_t)pc.slot * a.part_rows + seg_row] = make_float2(m_run, l_run);
      if (REACH && row_ok && pc.slot < 0 && p.lse)
        p.lse[((size_t)pc.b * a.T + node) * a.Hq + h] = row_lse(m_run, l_run);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(o_free);
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == C::kQkWarp) tc::tmem_dealloc(tmem, C::kTmemCols);
}

// Merges a split segment's pieces, each left as O / l in fp32 with its maximum and
// sum: a block per 32 rows of a segment, a lane per row, a warp per eight columns of
// every 64, four pieces in flight.  (In the act dtype the pieces cost a second
// rounding, 1.4 times the whole error.)
constexpr int kCombineWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kCombineWarps * 32) block8_combine_kernel(const AttnParams a, float* lse) {
  constexpr int U = 4, N = D / 64;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Sched& s = a.sched;
  const int HR = s.Hkv * s.nrg, blocks = (a.part_rows + 31) / 32;
  const int seg = blockIdx.x / blocks, r = blockIdx.x % blocks * 32 + lane;
  const int b = seg / HR, kvh = seg % HR / s.nrg, rg = seg % s.nrg;
  pdl_wait();
  const int nt = s.tile_pfx[b + 1] - s.tile_pfx[b];
  if (nt == 0) return;
  const long long X = sched_total_cost(s), t0 = (long long)s.tile_pfx[b] * HR + (long long)(seg - b * HR) * nt;
  const int c0 = sched_cta_of(sched_tile_cost(s, t0, seg), X, s.G);
  const int c1 = sched_cta_of(sched_tile_cost(s, t0 + nt - 1, seg), X, s.G);
  const int row = rg * a.rows_per_group + r;
  if (c0 == c1 || r >= a.part_rows || row >= a.rows) return;  // one piece has written the output
  float M = -INFINITY, l = 0.f, acc[N][8] = {};
  const float4* part = reinterpret_cast<const float4*>(a.part_o);
#pragma unroll 1
  for (int k0 = c0; k0 <= c1; k0 += U) {
    float2 ml[U];
    float4 v[U][N][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // a CTA between the first and the last may hold no tile, and has written
      // nothing then
      const int cta = k0 + u;
      ml[u] = make_float2(-INFINITY, 0.f);
      if (cta > c1 || !(cta == c0 || cta == c1 || X * (cta + 1) / s.G != X * cta / s.G)) continue;
      const size_t slot = (size_t)seg + cta;
      ml[u] = a.part_ml[slot * a.part_rows + r];
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[u][n][h] = part[(slot * (D / 4) + 16 * n + 2 * warp + h) * a.part_rows + r];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (ml[u].y == 0.f) continue;  // no piece, or one that saw no key of the row (a NaN goes on)
      const float m = fmaxf(M, ml[u].x);
      const float fo = fast_exp2(M - m), fn = fast_exp2(ml[u].x - m) * ml[u].y;
      l = fmaf(l, fo, fn);
      M = m;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float* o = acc[n] + 4 * h;
          const float4 x = v[u][n][h];
          o[0] = fmaf(x.x, fn, o[0] * fo);
          o[1] = fmaf(x.y, fn, o[1] * fo);
          o[2] = fmaf(x.z, fn, o[2] * fo);
          o[3] = fmaf(x.w, fn, o[3] * fo);
        }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int node = row / a.g, h = kvh * a.g + row % a.g;
  const size_t at = ((size_t)b * a.T + node) * a.Hq + h;
  if (lse && warp == 0) lse[at] = row_lse(M, l);
  T* out = static_cast<T*>(a.out) + at * D + 8 * warp;
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[n][e] *= inv;
    Row8<T> w;
    w.from_f(acc[n]);
    w.store(out + 64 * n);
  }
}

template <typename T, int D>
cudaError_t launch_combine_t(const AttnParams& a, float* lse, cudaStream_t stream) {
  const long long blocks = (long long)a.B * a.sched.Hkv * a.sched.nrg * ((a.part_rows + 31) / 32);
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  return launch_pdl(block8_combine_kernel<T, D>, dim3((unsigned)blocks), dim3(kCombineWarps * 32), 0, stream, a, lse);
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

// Rows of D codes in boxes of 16 rows (one page or block of one KV head), zeros
// past the end; keys swizzled as the tensor cores read them, values plain.
bool map_pages(CUtensorMap* map, const void* base, long long rows, int D, bool keys) {
  auto enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)D};
  const cuuint32_t box[2] = {(cuuint32_t)D, 16};
  const cuuint32_t es[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             !keys ? CU_TENSOR_MAP_SWIZZLE_NONE : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query parts [parts * B * T][Hq][D]: boxes of one M tile (128 / g nodes x g heads).
bool map_queries(CUtensorMap* map, const void* base, long long nodes, int Hq, int g, int D) {
  auto enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)nodes};
  const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)Hq * D};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)g, (cuuint32_t)(128 / g)};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int MT, int NP, bool REACH>
cudaError_t launch_r(const Block8Params& p, cudaStream_t stream) {
  using C = Cfg<D, MT, NP>;
  const AttnParams& a = p.a;
  static std::atomic<bool> opted[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !opted[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(attn_block8_tc_kernel<T, D, MT, NP, REACH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) opted[dev].store(true, std::memory_order_release);
  }
  alignas(64) CUtensorMap k, v, kn, vn, q;
  const long long rows = (long long)a.num_pages * a.Hkv * 16, nrows = (long long)a.B * a.Hkv * ((a.T + 15) / 16) * 16;
  if (!map_pages(&k, a.k_cache, rows, D, true) || !map_pages(&v, a.v_cache, rows, D, false) ||
      !map_pages(&kn, p.k_blocks, nrows, D, true) || !map_pages(&vn, p.v_blocks, nrows, D, false) ||
      !map_queries(&q, p.q8, (long long)NP * a.B * a.T, a.Hq, a.g, D))
    return cudaErrorInvalidValue;
  return launch_pdl(attn_block8_tc_kernel<T, D, MT, NP, REACH>, dim3(a.sched.G), dim3(C::kThreads), (size_t)C::kSmem,
                    stream, k, v, kn, vn, q, p);
}

template <typename T, int D, int MT, int NP>
cudaError_t launch_t(const Block8Params& p, cudaStream_t stream) {
  return p.window > 0 ? launch_r<T, D, MT, NP, true>(p, stream) : launch_r<T, D, MT, NP, false>(p, stream);
}

template <int D>
cudaError_t launch_d(const Block8Params& p, int dtype, cudaStream_t stream) {
  if (dtype == 1) return launch_t<__half, D, 1, 3>(p, stream);
  if (p.a.rows_per_group <= 128) return launch_t<__nv_bfloat16, D, 1, 2>(p, stream);
  return launch_t<__nv_bfloat16, D, 2, 2>(p, stream);
}

}  // namespace

cudaError_t launch_attn_block8_tc(const Block8Params& p, int dtype, cudaStream_t stream) {
  return p.a.D == 64 ? launch_d<64>(p, dtype, stream) : launch_d<128>(p, dtype, stream);
}

cudaError_t launch_block8_combine(const Block8Params& p, int dtype, cudaStream_t stream) {
  if (p.a.D == 64)
    return dtype == 1 ? launch_combine_t<__half, 64>(p.a, p.lse, stream) : launch_combine_t<__nv_bfloat16, 64>(p.a, p.lse, stream);
  return dtype == 1 ? launch_combine_t<__half, 128>(p.a, p.lse, stream) : launch_combine_t<__nv_bfloat16, 128>(p.a, p.lse, stream);
}

}  // namespace mt
