// Tree attention over a paged cache of E4M3 codes with one scale for each
// (page, KV head), fp16/bf16 activations.
//
// The T new tokens of a sequence (T = 1: a decoding step) attend to its L
// cached slots and to their own tree ancestors (the Medusa tree mask, vLLM
// issue 1171); the cache is only read.  The new keys and values are seen as the
// append encodes them, in blocks of 16 new tokens, each block of a KV head under
// its own power-of-two scale.  Stored, an accepted token shares its page's scale
// with other rows: a power of two changes no code's value but by underflow.
//
// With few query rows (T * g for g query heads per KV head) the cache's bytes
// bound the work, so the codes go from memory to the matrix instructions with
// as few steps as possible: each warp owns a page at a time, brings its 16 keys
// and values into a ring of its own (cp.async, no barrier between warps), reads
// them as fragments and converts in registers (one instruction for two codes;
// every E4M3 value is exact in fp16).  Both products are m16n8k16 fp16 with fp32
// accumulators, with the cache on the 16-row side and the query rows on the
// 8-column side, so that eight rows (a decoding step of eight heads a KV head)
// waste nothing:
//   S^T = K Q^T: any order of the D products is the same sum, so a lane takes 16
//     consecutive bytes of a key row as four k-steps of four, and Q is held in
//     the same order;
//   O^T = V^T P^T: a lane takes 8 or 16 consecutive columns of four value rows
//     (row i of tile t is column i * (D/8) + 2t, row i + 8 the one after), a byte
//     permute pairs two rows' codes before the conversion, and P^T is S^T's
//     fragment after an 8x8 transposition.
// Queries are scaled to a power of two per row (exact; a bf16 query keeps all
// its bits in fp16).  Softmax in base 2; the maximum of a row moves only when a
// score exceeds it by more than 8, which one vote per page finds, so the common
// page has no reduction.  A page's value scale 2^lv joins the exponent: the
// maximum is that of score + lv, P = 2^(score + lv - max + 3) is what a value's
// code is multiplied with, and the row's sum takes P * 2^-lv.  So the fp16 of P is
// spent on what a key adds to the output, 2^11 down to 2^-24, whatever the scales
// and the weights of the pages before it (scaled by the largest value scale so far,
// a page of a large scale and next to no weight left the others no bits).
//
// The batch's 64-slot tiles (four pages, one a warp) are dealt out evenly over
// persistent CTAs (common.cuh's balanced schedule, its prefix computed by every
// CTA from the lengths).  A split segment's pieces leave O / l in fp32 with their
// maximum and sum; the one that completes the segment's tile count merges them, so
// a call is one launch.
//
// Bound by the cache's bytes: 64 sequences of 256 to 8192 tokens, 32 query and 8 KV
// heads of 128 columns, one query each: 95 to 97 us for 549 MB, 5.7 TB/s (84 % of a copy).
// A call for one sequence of 2048 tokens takes 12.4 us, all of it latency: the
// prefix, the first page ids, the first pages, one merge.
#include <atomic>
#include <climits>
#include <cmath>

#include "serve.cuh"

namespace mt {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kP = 16;
constexpr int kMaxDevices = 64;

// NT: 8-row tiles of query rows a CTA holds.
template <int D, int NT>
struct Cfg {
  static constexpr int ROWS = 8 * NT;
  // per SM, by registers.  NT = 1: four CTAs of 128 registers and three pages a warp
  // were slower, 100 us against 97 at the size named above, and spilled.
  static constexpr int CTAS = NT <= 2 ? 3 : 2;
  static constexpr int DEPTH = NT <= 2 ? 4 : 6;  // pages a warp keeps in flight
  static constexpr int kPage = 16 * D;           // bytes of a page's K or V
  static constexpr int kRing = kWarps * DEPTH * 2 * kPage;
  static constexpr int LDO = D + 4;                            // merge rows, in floats
  static constexpr int kMerge = kWarps * 8 * LDO * 4;
  static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
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

// The 8x8 transposition of 16-bit values held two a lane, row i in lanes 4i .. 4i + 3.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2 and inverse of a page's value scale.  One below 2^-64 (or one that is no number)
// would leave the exponent's range: it counts as 2^-64.
__device__ __forceinline__ void log2_scale(float vs, float& lv, float& iv) {
  vs = fmaxf(vs, 5.421010862427522e-20f);
  lv = log2f(vs);
  iv = 1.f / vs;
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t r;
  memcpy(&r, &h, 4);
  return r;
}

// Adds to a segment's tile count and returns the count before: acquire-release at
// GPU scope, so that the piece that completes it sees what the others wrote.
__device__ __forceinline__ unsigned count_tiles(unsigned* counter, unsigned n) {
  unsigned old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(counter), "r"(n) : "memory");
  return old;
}

// Byte offset of 16-byte chunk ch of row r in a page's K or V: chunks are
// permuted within a row so that the fragment reads (eight lanes a phase: K two
// rows of four chunks, V four even or odd rows of two) hit distinct banks.
template <int D>
__device__ __forceinline__ int k_off(int r, int ch) {
  return r * D + ((D == 128 ? ch ^ ((r & 1) << 2) : ch) << 4);
}
template <int D>
__device__ __forceinline__ int v_off(int r, int ch) {
  return r * D + ((D == 128 ? ch ^ (((r >> 1) & 3) << 1) : ch ^ ((r >> 1) & 3)) << 4);
}

// One warp's running result for NT * 8 query rows.  Lane (gid, tig) holds query
// row gid of each tile as an operand, and rows 2 tig and 2 tig + 1 of the results.
template <int D, int NT>
struct State {
  uint32_t q[NT][D / 16][2];
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];  // l is this lane's part
  float c[NT][2];            // score -> base-2 units, without the page's scale

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][t][e] = 0.f;
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
    }
  }
};

// Which of a page's 16 keys a row sees: every one, those before a limit, or
// those of an ancestor mask.
enum : int { kSeeAll, kSeeLimit, kSeeMask };

// Folds one page (codes in shared memory) into the running result; lv, iv: log2 and
// inverse of its value scale.
template <int D, int NT, int SEE>
__device__ __forceinline__ void page_step(State<D, NT>& st, const uint8_t* kp, const uint8_t* vp, float ks, float lv,
                                          float iv, int limit, const unsigned (&see)[NT][2]) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  float s[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll
  for (int ch = 0; ch < D / 64; ++ch) {  // 16-byte chunks of a key row per lane
    const uint4 w0 = *reinterpret_cast<const uint4*>(kp + k_off<D>(gid, ch * 4 + tig));
    const uint4 w1 = *reinterpret_cast<const uint4*>(kp + k_off<D>(gid + 8, ch * 4 + tig));
    const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t a[4] = {e4m3x2_to_h2(x0[x] & 0xffffu), e4m3x2_to_h2(x1[x] & 0xffffu), e4m3x2_to_h2(x0[x] >> 16),
                             e4m3x2_to_h2(x1[x] >> 16)};
#pragma unroll
      for (int i = 0; i < NT; ++i) mma(s[i], a, st.q[i][ch * 4 + x][0], st.q[i][ch * 4 + x][1]);
    }
  }
  // scores in base-2 units + lv; element e: row 2 tig + (e & 1), key gid + 8 (e >> 1)
  bool over = false;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[i][e] = fmaf(s[i][e], st.c[i][e & 1] * ks, lv);
      if (SEE != kSeeAll) {
        const int key = gid + 8 * (e >> 1);
        if (!(SEE == kSeeLimit ? key < limit : ((see[i][e & 1] >> key) & 1u))) s[i][e] = -INFINITY;
      }
      over = over || s[i][e] > st.m[i][e & 1] + 8.f;
    }
  }
  if (__any_sync(0xffffffffu, over)) {  // a maximum grows by more than 2^8: O moves
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float f[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = fmaxf(s[i][r], s[i][2 + r]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        f[r] = 1.f;
        if (mx > st.m[i][r] + 8.f) {
          f[r] = fast_exp2(st.m[i][r] - mx);  // 0 from -inf
          st.l[i][r] *= f[r];
          st.m[i][r] = mx;
        }
      }
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[i][t][e] *= f[e & 1];
    }
  }
  uint32_t pb[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float m = st.m[i][e & 1];
      s[i][e] = fast_exp2(s[i][e] + (m == -INFINITY ? 0.f : 3.f - m));
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) st.l[i][r] = fmaf(s[i][r] + s[i][2 + r], iv, st.l[i][r]);
#pragma unroll
    for (int h = 0; h < 2; ++h) pb[i][h] = transpose8(pack_h2(s[i][2 * h], s[i][2 * h + 1]));
  }
  // values: rows 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9, columns gid * D/8 ...
  constexpr int NW = D / 32;  // 4-byte words of a row per lane
  uint32_t v[4][NW];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = 2 * tig + (r & 1) + (r >> 1) * 8;
    if (D == 128) {
      const uint4 w = *reinterpret_cast<const uint4*>(vp + v_off<D>(row, gid));
      v[r][0] = w.x;
      v[r][1] = w.y;
      v[r][NW - 2] = w.z;
      v[r][NW - 1] = w.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(vp + v_off<D>(row, gid >> 1) + (gid & 1) * 8);
      v[r][0] = w.x;
      v[r][1] = w.y;
    }
  }
#pragma unroll
  for (int w = 0; w < NW; ++w) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // bytes 2h and 2h + 1 of both rows, paired by byte
      const uint32_t sel = h ? 0x7362 : 0x5140;
      const uint32_t p0 = __byte_perm(v[0][w], v[1][w], sel), p1 = __byte_perm(v[2][w], v[3][w], sel);
      const uint32_t a[4] = {e4m3x2_to_h2(p0 & 0xffffu), e4m3x2_to_h2(p0 >> 16), e4m3x2_to_h2(p1 & 0xffffu),
                             e4m3x2_to_h2(p1 >> 16)};
#pragma unroll
      for (int i = 0; i < NT; ++i) mma(st.o[i][2 * w + h], a, pb[i][0], pb[i][1]);
    }
  }
}

// Folds a page that not every row sees whole.  Value rows that no row sees may hold
// anything, NaN codes too: they are made 0, as their weights are.  Those that only the
// shallower nodes see, at the window's edge, lose their NaN codes for the step and give
// them back to the columns of the rows that do see them; `values`: where the codes came
// from.
template <int D, int NT>
__device__ __forceinline__ void partial_step(State<D, NT>& st, const uint8_t* kp, uint8_t* vp, float ks, float lv,
                                             float iv, const Reach& reach, int c0, const AttnParams& a,
                                             const int* s_depth, int row0, const uint8_t* values) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const unsigned any = reach.see16(c0, 0), all = reach.see16(c0, a.T - 1);
  constexpr int CPR = D / 16;
  bool odd = false;
  for (int e = lane; e < 16 * CPR; e += 32) {
    const int r = e / CPR;
    uint4* w = reinterpret_cast<uint4*>(vp + e * 16);  // a row's chunks, in whatever order
    if (!(any >> r & 1u)) {
      *w = make_uint4(0, 0, 0, 0);
    } else if (!(all >> r & 1u)) {
      uint32_t x[4] = {w->x, w->y, w->z, w->w};
      bool nan = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t m = __vcmpeq4(x[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        nan = nan || m != 0u;
        x[i] &= ~m;
      }
      if (nan) *w = make_uint4(x[0], x[1], x[2], x[3]);
      odd = odd || nan;
    }
  }
  odd = __any_sync(0xffffffffu, odd);
  __syncwarp();  // page_step's lanes read rows that other lanes have changed; a vote orders no memory
  unsigned see[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + i * 8 + 2 * tig + r;
      see[i][r] = row < a.rows ? reach.see16(c0, s_depth[row / a.g]) : 0u;
    }
  page_step<D, NT, kSeeMask>(st, kp, vp, ks, lv, iv, kP, see);
  if (odd && values) {
#pragma unroll 1
    for (unsigned left = any & ~all; left; left &= left - 1) {
      const int r = __ffs(left) - 1;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint8_t code = values[r * D + gid * (D / 8) + 2 * t + (e >> 1)];
            if ((see[i][e & 1] >> r & 1u) && (code & 0x7f) == 0x7f) st.o[i][t][e] = __int_as_float(0x7fffffff);
          }
    }
  }
}

// One block of up to 16 new tokens of K or V as codes in shared memory (rows
// past T are zero); returns the block's scale.  odd: which tokens have an element that is
// not finite, added to by the call for the values and then the one for the keys.
template <typename T, int D>
__device__ __forceinline__ float quantise_new(const T* src, size_t row_stride, int rows, uint8_t* dst, bool keys,
                                              unsigned& odd) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, STEPS = 16 / RPS;
  const int lane = threadIdx.x & 31, sub = lane / LPR, c = lane % LPR;
  Row8<T> lo[STEPS], hi[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = s * RPS + sub;
    lo[s].zero();
    hi[s].zero();
    if (r < rows) {
      lo[s].load(src + r * row_stride + 8 * c);
      hi[s].load(src + r * row_stride + D / 2 + 8 * c);
    }
  }
  float amax = largest_bits<T, STEPS>(lo, hi);
  if (!(amax < INFINITY)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      odd |= odd_rows<RPS>(not_finite(lo[s]) || not_finite(hi[s])) << (s * RPS);
      drop_odd(lo[s]);
      drop_odd(hi[s]);
    }
    amax = largest_bits<T, STEPS>(lo, hi);
  }
  const float scale = block_scale(amax), inv = 1.f / scale;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = s * RPS + sub;
    float x[2][8];
    lo[s].to_f(x[0]);
    hi[s].to_f(x[1]);
    if (keys && (odd >> r & 1u)) x[0][0] = __int_as_float(0x7fffffff);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = h * (D / 2) + 8 * c;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[h][e] *= inv;
      const int off = (keys ? k_off<D>(r, col >> 4) : v_off<D>(r, col >> 4)) + (col & 8);
      *reinterpret_cast<uint2*>(dst + off) = e4m3x8_of(x[h]);
    }
  }
  return scale;
}

// Merges the pieces that CTAs c0 .. c1 left of a segment, by the block of the last
// one: 16 threads a row, eight columns each.  Each thread brings its own part of up
// to 4 * DEPTH pieces into the idle rings at once, so that a round costs one trip to
// L2 (0.33 us a piece one after the other).  X: the schedule's total cost.
template <typename T, int D, int NT, bool REACH>
__device__ __forceinline__ void merge_pieces(const Block8Params& p, const Piece& done, int c0, int c1, long long X,
                                             uint8_t* ring) {
  constexpr int U = 4 * Cfg<D, NT>::DEPTH;  // pieces of eight rows that the rings hold
  __shared__ float2 s_ml[U][8];
  const AttnParams& a = p.a;
  const int tid = threadIdx.x, rr = tid >> 4, c8 = tid & 15, G = a.sched.G;
  const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + (rr * (D / 8) + c8) * 16;
#pragma unroll 1
  for (int i = 0; i < NT; ++i) {
    const int row = done.rg * (8 * NT) + i * 8 + rr;
    const bool live = row < a.rows && c8 < D / 8;
    float M = -INFINITY, l = 0.f, acc[8] = {};
#pragma unroll 1
    for (int k0 = c0; k0 <= c1; k0 += U) {
      const int n = min(U, c1 - k0 + 1);
      for (int x = tid; x < n * 8; x += kThreads) {
        const int cta = k0 + (x >> 3), r = i * 8 + (x & 7);
        float2 v = make_float2(-INFINITY, 0.f);
        // a CTA between the first and the last may hold no tile, and has written
        // nothing then
        if (done.rg * (8 * NT) + r < a.rows && (cta == c0 || cta == c1 || X * (cta + 1) / G != X * cta / G))
          v = __ldcg(a.part_ml + (size_t)(done.seg + cta) * a.part_rows + r);
        s_ml[x >> 3][x & 7] = v;
      }
      if (live) {
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
          const float* o = p.frag_o + ((size_t)(done.seg + k0 + k) * a.part_rows + i * 8 + rr) * D + c8 * 8;
          cp_async16(mine + k * 32 * D, o);
          cp_async16(mine + k * 32 * D + 16 * D, o + 4);
        }
      }
      cp_commit();
      cp_wait<0>();
      __syncthreads();
      if (live) {
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
          const float2 ml = s_ml[k][rr];
          if (ml.y == 0.f) continue;  // no piece, or one that saw no key of the row (a NaN goes on)
          const float4* o = reinterpret_cast<const float4*>(ring + k * 32 * D) + rr * (D / 8) + c8;
          const float4 x = o[0], y = o[D];
          const float m = fmaxf(M, ml.x);
          const float fo = fast_exp2(M - m), fn = fast_exp2(ml.x - m) * ml.y;
          const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(v[e], fn, acc[e] * fo);
          l = fmaf(l, fo, fn);
          M = m;
        }
      }
      __syncthreads();  // the rings and s_ml are filled again
    }
    if (!live) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= inv;
    const int node = row / a.g, h = done.kvh * a.g + row % a.g;
    const size_t at = ((size_t)done.b * a.T + node) * a.Hq + h;
    Row8<T> v;
    v.from_f(acc);
    v.store(static_cast<T*>(a.out) + at * D + c8 * 8);
    if (REACH && c8 == 0 && p.lse) p.lse[at] = row_lse(M, l);
  }
}

// REACH: with a window and sinks, and the rows' log-sum-exp.  A page that some row sees in
// part takes the masked step; 64 sequences of 256 to 100000 tokens under a window of 4096,
// one query each, 32 query and 8 KV heads: 92 us for 533 MB, 5.8 TB/s (85 % of a copy), the
// rate of the whole cache's instance.
template <typename T, int D, int NT, bool REACH>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::CTAS) attn_block8_kernel(const Block8Params p) {
  using C = Cfg<D, NT>;
  constexpr int RG = C::ROWS;
  extern __shared__ __align__(128) uint8_t smem[];
  int* s_pfx = reinterpret_cast<int*>(smem + C::kSmem);  // [B + 1]
  __shared__ int s_warp[kWarps];
  __shared__ int s_par[kMaxTree];
  __shared__ unsigned long long s_anc[kMaxTree];
  __shared__ int s_depth[REACH ? kMaxTree : 1];
  __shared__ float s_m[kWarps][RG], s_l[kWarps][RG];
  __shared__ int s_last;
  const AttnParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gid = lane >> 2, tig = lane & 3;
  const int nnew = (a.T + kP - 1) / kP;
  pdl_wait();

  // every CTA: tiles of each sequence and their prefix
  block8_prefix<kWarps, REACH>(a, s_pfx, s_warp, blockIdx.x == 0, p.window, p.sinks);
  // One warp walks the pieces: the cursor and the schedule's 64-bit arithmetic stay out
  // of everybody's registers.  Its lanes do so together, with the same values: where one
  // thread did, its loops and divisions left it apart from its warp in an instance that
  // fills its registers, and the warp then came to each barrier twice.
  __shared__ long long s_cur, s_end;
  __shared__ Piece s_piece;
  __shared__ int s_bcur, s_more;
  Sched sc = a.sched;
  sc.tile_pfx = s_pfx;
  sc.splits = 0;
  if (warp == 0) {
    PieceIter it;
    it.init(sc, blockIdx.x);
    s_cur = it.cur;
    s_end = it.end;
    s_bcur = it.bcur;
    __syncwarp();
  }
  uint8_t* ring = smem + warp * (C::DEPTH * 2 * C::kPage);
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const uint8_t* kc = static_cast<const uint8_t*>(a.k_cache);
  const uint8_t* vc = static_cast<const uint8_t*>(a.v_cache);

  while (true) {
    if (warp == 0) {
      PieceIter it;
      it.s = sc;
      it.cta = blockIdx.x;
      it.cur = s_cur;
      it.end = s_end;
      it.bcur = s_bcur;
      Piece next;
      const bool more = it.next(next);
      __syncwarp();  // every lane has read the cursor
      s_cur = it.cur;
      s_bcur = it.bcur;
      s_piece = next;
      s_more = more;
      __syncwarp();
    }
    __syncthreads();
    if (!s_more) break;
    const Piece pc = s_piece;
    const int b = pc.b, kvh = pc.kvh;
    const Reach reach(a.seq_lens[b], REACH ? p.window : INT_MAX, REACH ? p.sinks : 0);
    const int L = REACH ? reach.Lv : a.seq_lens[b];  // cached slots, or the visible pages' columns
    const int npre = (L + kP - 1) / kP;
    const int row0 = pc.rg * RG;
    const bool has_new = pc.tile_end * 4 > npre;
    // the rows' depths: where the window's edge lies in these tiles
    const bool has_edge = REACH && reach.partial(pc.tile_begin * 64, (pc.tile_end - pc.tile_begin) * 64, a.T - 1);
    if (has_new || has_edge) {
      // ancestors of every node, by walking up (a chain without parents)
      if (tid < a.T) {
        const int par = p.parents ? p.parents[(size_t)b * a.T + tid] : tid - 1;
        const bool ok = tid == 0 ? par == -1 : (par >= 0 && par < tid);
        if (!ok) set_status(a.status, kStTree);
        s_par[tid] = ok ? par : -1;
      }
      __syncthreads();
      if (tid < a.T) {
        unsigned long long anc = 0;
        for (int n = tid; n >= 0; n = s_par[n]) anc |= 1ull << n;  // parents are earlier: at most T steps
        if (REACH) anc = seen_ancestors(anc, tid, s_par, a.seq_lens[b], p.window, p.sinks, s_depth[tid]);
        s_anc[tid] = anc;
      }
      __syncthreads();
    }
    // this warp's pages: 4 * (tile_begin + i) + warp, the cached ones first
    const int tiles = pc.tile_end - pc.tile_begin;
    const int first = 4 * pc.tile_begin + warp;
    const int npages = min(tiles, max(0, (npre - first + 3) / 4));
    const int* bt = a.block_tables + (size_t)b * a.max_blocks;
    // page ids and scales of 32 pages, a lane each; the next 32 ids are fetched
    // while these are used, their scales half way
    auto fetch_id = [&](int i) {
      if (i >= npages) return -1;
      return bt[REACH ? reach.page(first + 4 * i) : first + 4 * i];
    };
    auto fetch_scale = [&](const float* sc_, int id) {
      return id >= 0 && id < a.num_pages ? __ldg(sc_ + (size_t)id * a.Hkv + kvh) : 0.f;
    };
    int id_cur = fetch_id(lane), id_nxt = -1;
    float ks_cur = fetch_scale(p.k_scales, id_cur), vs_nxt = fetch_scale(p.v_scales, id_cur);
    float ks_nxt = 0.f, lv_cur, iv_cur;
    log2_scale(vs_nxt, lv_cur, iv_cur);
    int id_iss = id_cur, iss_base = 0;  // the issuing side runs ahead of the computing side
    bool bad = false;
    auto issue = [&](int i) {
      if (i < npages) {
        if (i - iss_base >= 32) {
          iss_base += 32;
          id_iss = id_nxt;
        }
        const int id = __shfl_sync(0xffffffffu, id_iss, i - iss_base);
        if (id >= 0 && id < a.num_pages) {
          const size_t src = ((size_t)id * a.Hkv + kvh) * C::kPage;
          const uint32_t dst = ring_u + (i % C::DEPTH) * 2 * C::kPage;
          constexpr int CPR = D / 16;  // chunks per row
#pragma unroll
          for (int x = 0; x < 16 * CPR / 32; ++x) {
            const int q = x * 32 + lane, r = q / CPR, ch = q % CPR;
            cp_async16(dst + k_off<D>(r, ch), kc + src + q * 16);
            cp_async16(dst + C::kPage + v_off<D>(r, ch), vc + src + q * 16);
          }
        } else {
          bad = true;
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < C::DEPTH - 1; ++i) issue(i);

    // queries: this lane's columns of row gid of each tile, scaled to fp16
    State<D, NT> st;
    st.clear();
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int row = row0 + i * 8 + gid;
      Row8<T> raw[D / 32];
#pragma unroll
      for (int x = 0; x < D / 32; ++x) raw[x].zero();
      if (row < a.rows) {
        const int node = row / a.g, h = kvh * a.g + row % a.g;
        const T* q = static_cast<const T*>(a.q_rot) + (((size_t)b * a.T + node) * a.Hq + h) * D + tig * 16;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) raw[x].load(q + (x / 2) * 64 + (x % 2) * 8);
      }
      AbsMax<T> top;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) top.add(raw[x]);
      float amax = top.get();
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^8 <= scaled maximum < 2^9: a bf16 keeps its bits down to 2^-25 of it, an fp16 to 2^-22
      const int ex = amax > 0.f ? (int)(__float_as_uint(amax) >> 23) - 127 : 0;
      const int k = min(max(8 - ex, -120), 120);
      const float f2 = __uint_as_float((uint32_t)(127 + k) << 23);
      // an infinity makes every score NaN (of its products alone, keys of one sign would
      // give -inf throughout, and with that a sum of 0)
      const float c = amax < INFINITY ? a.scale_log2 * __uint_as_float((uint32_t)(127 - k) << 23)
                                      : __int_as_float(0x7fffffff);
      st.c[i][0] = __shfl_sync(0xffffffffu, c, 8 * tig);  // rows 2 tig and 2 tig + 1
      st.c[i][1] = __shfl_sync(0xffffffffu, c, 8 * tig + 4);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        float f[8];
        raw[x].to_f(f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // four columns: k-step 2x + e
          st.q[i][2 * x + e][0] = pack_h2(f[4 * e] * f2, f[4 * e + 1] * f2);
          st.q[i][2 * x + e][1] = pack_h2(f[4 * e + 2] * f2, f[4 * e + 3] * f2);
        }
      }
    }

    const unsigned none[NT][2] = {};
#pragma unroll 1
    for (int i = 0; i < npages; ++i) {
      const int at = i & 31;
      if (at == 0) {
        if (i > 0) {
          id_cur = id_nxt;
          ks_cur = ks_nxt;
          log2_scale(vs_nxt, lv_cur, iv_cur);
        }
        id_nxt = fetch_id(i + 32 + lane);
      } else if (at == 16) {
        ks_nxt = fetch_scale(p.k_scales, id_nxt);
        vs_nxt = fetch_scale(p.v_scales, id_nxt);
      }
      issue(i + C::DEPTH - 1);
      cp_wait<C::DEPTH - 1>();
      __syncwarp();
      uint8_t* kp = ring + (i % C::DEPTH) * 2 * C::kPage;
      uint8_t* vp = kp + C::kPage;
      const float ks = __shfl_sync(0xffffffffu, ks_cur, at), lv = __shfl_sync(0xffffffffu, lv_cur, at);
      const float iv = __shfl_sync(0xffffffffu, iv_cur, at);
      const int c0 = (first + 4 * i) * kP;
      const int limit = L - c0;
      if (REACH ? !reach.partial(c0, kP, a.T - 1) : limit >= kP) {
        page_step<D, NT, kSeeAll>(st, kp, vp, ks, lv, iv, kP, none);
      } else if (REACH) {
        const int id = __shfl_sync(0xffffffffu, id_cur, at);
        const uint8_t* values = id >= 0 && id < a.num_pages ? vc + ((size_t)id * a.Hkv + kvh) * C::kPage : nullptr;
        partial_step<D, NT>(st, kp, vp, ks, lv, iv, reach, c0, a, s_depth, row0, values);
      } else {
        // the sequence ends in this page: rows past it may hold anything, NaN
        // codes too; their weights are 0 and their values are made 0
        for (int e = lane; e < (kP - limit) * (D / 16); e += 32)
          *reinterpret_cast<uint4*>(vp + limit * D + e * 16) = make_uint4(0, 0, 0, 0);
        __syncwarp();
        page_step<D, NT, kSeeLimit>(st, kp, vp, ks, lv, iv, limit, none);
      }
      __syncwarp();  // every lane has read the slot before it is filled again
    }
    cp_wait<0>();
    __syncwarp();
    if (bad && lane == 0) set_status(a.status, kStPages);

    // the new tokens' block that falls to this warp, if any
    const int pn = first + 4 * npages - npre;
    if (npages < tiles && pn >= 0 && pn < nnew) {
      const size_t rs = (size_t)a.Hkv * D;
      const size_t src = ((size_t)b * a.T + pn * kP) * rs + (size_t)kvh * D;
      const int rows = min(kP, a.T - pn * kP);
      float ks = 0.f, vs = 0.f;
      unsigned odd = 0;
#pragma unroll 1  // one after the other: both at once take more registers than there are
      for (int x = 0; x < 2; ++x) {
        vs = ks;
        ks = quantise_new<T, D>(static_cast<const T*>(x ? p.k_new : p.v_new) + src, rs, rows, ring + (1 - x) * C::kPage, x == 1, odd);
      }
      __syncwarp();
      unsigned see[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = row0 + i * 8 + 2 * tig + r;
          see[i][r] = row < a.rows ? (unsigned)(s_anc[row / a.g] >> (pn * kP)) & 0xffffu : 0u;
        }
      float lv, iv;
      log2_scale(vs, lv, iv);
      page_step<D, NT, kSeeMask>(st, ring, ring + C::kPage, ks, lv, iv, kP, see);
    }

    // ---- join the four warps and write the piece ----
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float l = st.l[i][r];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (gid == 0) {
          s_m[warp][i * 8 + 2 * tig + r] = st.m[i][r];
          s_l[warp][i * 8 + 2 * tig + r] = l;
        }
      }
    float* s_o = reinterpret_cast<float*>(smem);  // [warp][8][LDO]
    // Rows 8i .. 8i + 7 from the four warps' parts in s_m, s_l and s_o: to the output,
    // or to the piece's slot.
    auto join = [&](int i, int slot) {
      const int rr = tid >> 4, rg_row = i * 8 + rr, row = row0 + rg_row, c8 = tid & 15;  // 16 threads a row
      if (row >= a.rows || c8 >= D / 8) return;
      float M = -INFINITY, f[kWarps], l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][rg_row]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        f[w] = s_m[w][rg_row] == -INFINITY ? 0.f : fast_exp2(s_m[w][rg_row] - M);
        l += f[w] * s_l[w][rg_row];
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float acc[8] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4* o = reinterpret_cast<const float4*>(s_o + (w * 8 + rr) * C::LDO + c8 * 8);
        const float4 x = o[0], y = o[1];
        const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(f[w], v[e], acc[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= inv;
      if (slot < 0) {
        Row8<T> v;
        v.from_f(acc);
        const int node = row / a.g, h = kvh * a.g + row % a.g;
        const size_t at = ((size_t)b * a.T + node) * a.Hq + h;
        v.store(static_cast<T*>(a.out) + at * D + c8 * 8);
        if (REACH && c8 == 0 && p.lse) p.lse[at] = row_lse(M, l);
      } else {
        float4* d = reinterpret_cast<float4*>(p.frag_o + ((size_t)slot * a.part_rows + rg_row) * D + c8 * 8);
        d[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        d[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (c8 == 0) a.part_ml[(size_t)slot * a.part_rows + rg_row] = make_float2(M, l);
      }
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      __syncthreads();  // rings (or the previous tile's rows) are no longer read
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float* o = s_o + (warp * 8 + 2 * tig + r) * C::LDO + gid * (D / 8);
#pragma unroll
        for (int t = 0; t < D / 16; t += 2)
          *reinterpret_cast<float4*>(o + 2 * t) =
              make_float4(st.o[i][t][r], st.o[i][t][2 + r], st.o[i][t + 1][r], st.o[i][t + 1][2 + r]);
      }
      __syncthreads();
      join(i, pc.slot);
    }
    if (pc.slot >= 0) {
      // the piece that brings the segment's tiles to their number merges it: the
      // others' results are visible to it through the counter, which is that of
      // the segment's first CTA (a CTA's run crosses into at most one segment that
      // another CTA goes on with)
      const int nt = s_pfx[b + 1] - s_pfx[b];
      const int HR = sc.Hkv * sc.nrg;
      const long long X = sched_total_cost(sc);
      const long long t0 = (long long)s_pfx[b] * HR + (long long)(pc.seg - b * HR) * nt;
      const int c0 = sched_cta_of(sched_tile_cost(sc, t0, pc.seg), X, sc.G);
      __syncthreads();
      if (tid == 0) {
        unsigned* counter = p.frag_tiles + c0;
        s_last = count_tiles(counter, (unsigned)tiles) + (unsigned)tiles == (unsigned)nt;
        if (s_last) *counter = 0;  // left at zero for the next call
      }
      __syncthreads();
      if (s_last) {
        const int c1 = sched_cta_of(sched_tile_cost(sc, t0 + nt - 1, pc.seg), X, sc.G);
        merge_pieces<T, D, NT, REACH>(p, pc, c0, c1, X, smem);
      }
    }
    __syncthreads();  // the rings are filled again by the next piece
  }
}

template <typename T, int D, int NT, bool REACH>
cudaError_t launch_r(const Block8Params& p, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  const size_t smem = (size_t)C::kSmem + sizeof(int) * (size_t)(p.a.B + 1);
  static std::atomic<bool> opted[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !opted[dev].load(std::memory_order_acquire)) {
    // the largest batch's prefix included
    e = cudaFuncSetAttribute(attn_block8_kernel<T, D, NT, REACH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem + 4 * (8192 + 1));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) opted[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(attn_block8_kernel<T, D, NT, REACH>, dim3(p.a.sched.G), dim3(kThreads), smem, stream, p);
}

template <typename T, int D, int NT>
cudaError_t launch_t(const Block8Params& p, cudaStream_t stream) {
  return p.window > 0 ? launch_r<T, D, NT, true>(p, stream) : launch_r<T, D, NT, false>(p, stream);
}

template <typename T, int D>
cudaError_t launch_n(const Block8Params& p, cudaStream_t stream) {
  switch (p.a.rows_per_group) {
    case 8: return launch_t<T, D, 1>(p, stream);
    case 16: return launch_t<T, D, 2>(p, stream);
    default: return launch_t<T, D, 4>(p, stream);
  }
}

template <typename T>
cudaError_t launch_d(const Block8Params& p, cudaStream_t stream) {
  return p.a.D == 64 ? launch_n<T, 64>(p, stream) : launch_n<T, 128>(p, stream);
}

}  // namespace

Block8Plan block8_plan(int batch, int kv_heads, int rows, int g, int max_blocks, int tree_size, int dtype, bool windowed,
                       int sms) {
  Block8Plan p{};
  // Up to 16 rows the register-fragment kernel, which wastes no rows; from 17 on the
  // tensor-core kernel, whose tile has 128 (256) rows.  64 sequences of 256 to 8192
  // tokens, 8 KV heads: 16 rows 107 us against 177, 24 rows 195 against 177, 32 rows
  // 205 against 177; 4 sequences of 2000: 20.9 against 21.9, and 32.8 against 22.6.
  // The latter's tiles are built for g that divides 128; for any other g the former
  // takes every count, and streams a KV head's cache once per 32 rows: 16 sequences of
  // 512 to 8192 tokens, 64 nodes, 24, 28 and 40 query heads for 8, 4 and 8 KV heads 321,
  // 348 and 518 us, where 32 for 8 take 95.  fp16 queries fill three operand parts, and
  // with those two tiles do not fit in TMEM: the same trees 119 us.
  // Under a window the tiles take any g, with 128 / g * g rows: whole nodes.  Trees of 64 nodes as
  // above, up to 32768 tokens, window 4096, 24 and 56 heads for 8: 86 and 151 us, the
  // register-fragment kernel 352 and 759; 18 rows of 4 sequences, window 1024, 19 against 26.
  if (rows > 16 && (tc_supported(128, g) || (windowed && g <= 128))) {
    const int tile = 128 / g * g;
    p.tc = true;
    p.parts = dtype == 1 ? 3 : 2;
    p.rows_per_group = p.parts == 2 && rows > tile ? 2 * tile : tile;
    p.ctas = sms;
    p.seg_cost = 5;  // 16 sequences of 64 nodes: 3 98 us, 5 95, 8 97, 12 100
  } else {
    p.rows_per_group = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
    p.ctas = sms * (rows <= 8 ? Cfg<128, 1>::CTAS : rows <= 16 ? Cfg<128, 2>::CTAS : Cfg<128, 4>::CTAS);
    // starting and leaving a piece costs as much as twelve tiles: 64 sequences of one
    // query and of 16 rows, and 16 of 16 rows, take 95, 107 and 51 us with 8, 95, 106
    // and 50 with 12, 96, 113 and 53 with 24 (with 2, an earlier kernel took 107 us
    // for the first against 100 with 8).  Not measured with few sequences, whose pieces
    // are few
    p.seg_cost = 12;
  }
  p.nrg = (rows + p.rows_per_group - 1) / p.rows_per_group;
  if (!p.tc) {
    // Few segments: a piece of t tiles takes about t / 2 us and the merge about
    // 0.1 us a piece, so a segment of n tiles is best cut into about sqrt(5 n)
    // pieces (n from the block table's width, which is all the host knows: under a
    // table of 131072 slots one sequence of 2048 tokens, 32/8 heads, takes 16.2 us
    // against 12.2 under one of 2048; with 32 KV heads 12.9 and 12.8).
    const double n = max_blocks / 4.0 + (tree_size + 63) / 64;
    const double most = (double)batch * kv_heads * p.nrg * std::ceil(std::sqrt(5.0 * n));
    if (most < p.ctas) p.ctas = (int)most;
  }
  return p;
}

cudaError_t launch_attn_block8(const Block8Params& p, int dtype, cudaStream_t stream) {
  return dtype == 1 ? launch_d<__half>(p, stream) : launch_d<__nv_bfloat16>(p, stream);
}

}  // namespace mt
