// Parameter blocks, launchers and device helpers of the serving operators
// around the verify step (internal to the library): norms with rotation, cache
// append, block-scaled 8-bit attention, sampling.
#pragma once

#include "kernels.cuh"

namespace mt {

enum : int { kStPosition = -7 };  // matches MT_ERR_POSITION

// ---------------------------------------------------------------------------
// 8 consecutive act-dtype elements as 16-byte words.
// ---------------------------------------------------------------------------
template <typename T>
struct Row8 {
  static constexpr int kWords = 8 * (int)sizeof(T) / 16;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = reinterpret_cast<const uint4*>(p)[k];
  }
  __device__ __forceinline__ void load_stream(const T* p) {  // read once
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = __ldcs(reinterpret_cast<const uint4*>(p) + k);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) reinterpret_cast<uint4*>(p)[k] = w[k];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void to_f(float (&x)[8]) const {
    T v[8];
    memcpy(v, w, sizeof(v));
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = Act<T>::to_f(v[e]);
  }
  __device__ __forceinline__ void from_f(const float (&x)[8]) {
    T v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = Act<T>::from_f(x[e]);
    memcpy(w, v, sizeof(v));
  }
};

// Largest magnitude of rows held as packed act-dtype words: 16-bit types stay
// packed (half the instructions, and no widened copy for the compiler to keep in
// registers).  A NaN is passed over.
template <typename T>
struct AbsMax {
  typedef __half2 V2;
  V2 m;
  __device__ __forceinline__ AbsMax() { m = __float2half2_rn(0.f); }
  __device__ __forceinline__ void add(const Row8<T>& r) {
    V2 v[4];
    memcpy(v, r.w, sizeof(v));
#pragma unroll
    for (int e = 0; e < 4; ++e) m = __hmax2(m, __habs2(v[e]));
  }
  __device__ __forceinline__ float get() const { return fmaxf(__low2float(m), __high2float(m)); }
};
template <>
struct AbsMax<__nv_bfloat16> {
  typedef __nv_bfloat162 V2;
  V2 m;
  __device__ __forceinline__ AbsMax() { m = __float2bfloat162_rn(0.f); }
  __device__ __forceinline__ void add(const Row8<__nv_bfloat16>& r) {
    V2 v[4];
    memcpy(v, r.w, sizeof(v));
#pragma unroll
    for (int e = 0; e < 4; ++e) m = __hmax2(m, __habs2(v[e]));
  }
  __device__ __forceinline__ float get() const { return fmaxf(__low2float(m), __high2float(m)); }
};
template <>
struct AbsMax<float> {
  float m = 0.f;
  __device__ __forceinline__ void add(const Row8<float>& r) {
    float v[8];
    memcpy(v, r.w, sizeof(v));
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
  }
  __device__ __forceinline__ float get() const { return m; }
};

// ---------------------------------------------------------------------------
// E4M3 codes and block scales.
// ---------------------------------------------------------------------------

// Two values as codes (nearest even, saturated to +-448), a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_of(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ uint2 e4m3x8_of(const float (&x)[8]) {
  return make_uint2(e4m3x2_of(x[0], x[1]) | e4m3x2_of(x[2], x[3]) << 16,
                    e4m3x2_of(x[4], x[5]) | e4m3x2_of(x[6], x[7]) << 16);
}

// Two codes (low 16 bits) as two fp16 values: exact, fp16 holds every E4M3 value.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t pair) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)pair));
  return r;
}

__device__ __forceinline__ void e4m3x8_to_f(uint2 c, float (&x)[8]) {
  const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e4m3x2_to_h2(w[i]);
    __half2 v;
    memcpy(&v, &h, 4);
    const float2 f = __half22float2(v);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Scale of a block whose largest magnitude is amax: the smallest power of two
// 2^k, k in [-64, 119], with amax <= 448 * 2^k = 1.75 * 2^(k + 8).  A power of
// two costs no precision (E4M3's steps are relative, so another scale in the
// same octave gives steps of the same size), makes code -> value exact in
// every act dtype, and lets a block's codes move to a larger scale without
// drift: only codes that fall below the smallest E4M3 step are rounded.  The
// range keeps the scale, its inverse and 448 times it normal fp32 numbers.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int k = (int)(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
  k = min(max(k, -64), 119);
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

// ---------------------------------------------------------------------------
// Per-head norms of queries and keys, with the rotation in the same pass.
// ---------------------------------------------------------------------------
struct NormRopeParams {
  int N, Hq, Hkv, D;
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  long long q_st[2], k_st[2], qo_st[2], ko_st[2];  // (token, head) strides in elements
  const int* positions;  // [N] or null
  const void* q_weight;  // [D] act, or null: no norm
  const void* k_weight;
  float eps;
  const float2* rope;  // null: no rotation
  int max_pos;
  int* status;
};
cudaError_t launch_norm_rope(const NormRopeParams& a, int dtype, cudaStream_t stream);

// ---------------------------------------------------------------------------
// Appending keys and values to a paged cache.
// ---------------------------------------------------------------------------
enum : int { kCacheAct = 0, kCacheE4m3 = 1, kCacheBlock8 = 2 };

struct AppendParams {
  int B, N, Hkv, D, max_blocks, num_pages, mode;
  const void* k;
  const void* v;
  long long k_st[2], v_st[2];  // (row, head) strides in elements
  void* k_cache;
  void* v_cache;
  float* k_scales;  // [num_pages][Hkv] (block-scaled caches)
  float* v_scales;
  float k_scale, v_scale;  // one scale for the whole cache (kCacheE4m3)
  const int* block_tables;
  const int* seq_lens;
  const int* row_offsets;  // [B + 1], or null: the accepted path's rows
  const int* accept_path;  // [B][max_depth + 1]
  const int* accept_len;   // [B]
  int T, max_depth;
  const float2* rope;  // null: keys are stored as given
  int max_pos;
  int* status;
};
cudaError_t launch_append(const AppendParams& a, int dtype, cudaStream_t stream);

// ---------------------------------------------------------------------------
// Tree attention over a block-scaled 8-bit cache.
// ---------------------------------------------------------------------------
constexpr int kMaxFragCtas = 4096;

struct Block8Params {
  AttnParams a;           // q_rot: the queries as they attend; part_o, part_ml, sched, out, status, ...
  const float* k_scales;  // [num_pages][Hkv]
  const float* v_scales;
  const void* k_new;      // [B][T][Hkv][D] act, as they attend
  const void* v_new;
  const int* parents;     // [B][T], or null: a chain
  // the register-fragment kernel's split segments, merged by their last piece:
  float* frag_o;          // [slots][rows per slot][D] each piece's O / l
  unsigned* frag_tiles;   // [kMaxFragCtas] tiles done of the segment that a CTA starts and another ends
  // the tensor-core path, written by its preparation:
  int* tile_pfx;          // [B + 1], for the combine
  int parts;              // E4M3 parts of a query row: 2 (bf16) or 3 (fp16)
  uint8_t* q8;            // [parts][B][T][Hq][D]
  float* q_scale;         // [B][T][Hq] scale of the row's parts times the softmax scale times log2(e)
  uint8_t* k_blocks;      // [B][Hkv][ceil(T / 16)][16][D] the new tokens' codes
  uint8_t* v_blocks;
  float* k_block_scales;  // [B][Hkv][ceil(T / 16)]
  float* v_block_scales;
  unsigned long long* anc;  // [B][T]
  int* pieces;            // piece table (common.cuh)
};

// Largest magnitude of a warp's rows of 16-bit values, by their bits, so that an infinity
// or a NaN is larger than any number.
template <typename T, int STEPS>
__device__ __forceinline__ float largest_bits(const Row8<T> (&lo)[STEPS], const Row8<T> (&hi)[STEPS]) {
  unsigned top = 0;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const uint4 a = lo[s].w[0], b = hi[s].w[0];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
  }
  const uint16_t bits = (uint16_t)__reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xffffu));
  T v;
  memcpy(&v, &bits, 2);
  return Act<T>::to_f(v);
}

// Whether a packed 16-bit row has a NaN or an infinity.
template <typename T>
__device__ __forceinline__ bool not_finite(const Row8<T>& r) {
  typename AbsMax<T>::V2 v[4];
  memcpy(v, r.w, sizeof(v));
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __habs2(v[e]);
  const auto m = __hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3]));
  return !(__low2float(m) < INFINITY && __high2float(m) < INFINITY);
}

// A new token that holds a NaN or an infinity makes NaN of the nodes that see it and must
// leave the others alone.  But a NaN value would reach those too, as 0 * NaN in the matrix
// products, and an infinity by way of its block's scale, under which every other code of
// the block is 0.  So neither enters a scale, both get codes of 0, and a code of the
// token's key is NaN: its scores are NaN where it is seen and are replaced where it is not.
// Of R rows in a warp, 32 / R lanes each: bit i says that row i has one.
template <int R>
__device__ __forceinline__ unsigned odd_rows(bool odd) {
  const unsigned lanes = __ballot_sync(0xffffffffu, odd);
  unsigned rows = 0;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (lanes >> (i * (32 / R)) & ((1u << (32 / R)) - 1u)) rows |= 1u << i;
  return rows;
}
template <typename T>
__device__ __forceinline__ void drop_odd(Row8<T>& r) {
  float x[8];
  r.to_f(x);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = fabsf(x[e]) < INFINITY ? x[e] : 0.f;
  r.from_f(x);
}

// Tiles of each sequence (cached pages, then the new tokens' blocks, four to a
// tile; none for seq_lens < 0) and their exclusive prefix in pfx[0 .. B], by a
// block of W warps; returns the total.  A length past the block table has no
// tiles and is recorded by the block that says so.
template <int W>
__device__ __forceinline__ int block8_prefix(const AttnParams& a, int* pfx, int* s_warp, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nnew = (a.T + 15) / 16;
  int carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += W * 32) {
    const int b = b0 + tid;
    int n = 0;
    if (b < a.B) {
      const int L = a.seq_lens[b];
      if ((long long)L > (long long)a.max_blocks * 16) {
        if (report) set_status(a.status, kStPages);
      } else if (L >= 0) {
        n = ((L + 15) / 16 + nnew + 3) / 4;
      }
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int off = carry;
    for (int w = 0; w < W; ++w) {
      if (w < warp) off += s_warp[w];
      carry += s_warp[w];
    }
    if (b < a.B) pfx[b] = off + incl - n;
    __syncthreads();
  }
  if (tid == 0) pfx[a.B] = carry;
  __syncthreads();
  return carry;
}

// How a call runs: the tensor-core kernel or the register-fragment kernel, its
// row group, row groups per KV head, persistent CTAs, and the cost of starting a
// piece (in 64-slot tiles).
struct Block8Plan {
  bool tc;
  int rows_per_group, nrg, ctas, seg_cost, parts;
};
Block8Plan block8_plan(int batch, int kv_heads, int rows, int g, int max_blocks, int tree_size, int dtype, int sms);
cudaError_t launch_attn_block8(const Block8Params& p, int dtype, cudaStream_t stream);
cudaError_t launch_block8_prep(const Block8Params& p, int dtype, cudaStream_t stream);
cudaError_t launch_block8_combine(const Block8Params& p, int dtype, cudaStream_t stream);
cudaError_t launch_attn_block8_tc(const Block8Params& p, int dtype, cudaStream_t stream);

// ---------------------------------------------------------------------------
// Sampling.
// ---------------------------------------------------------------------------
// Largest vocab: that many weights of 2^44 (the maximum's) stay below 2^63, and an
// eighth of it (a CTA's slice) leaves a lane at most 2^11 tokens of 16 warps, which the
// histograms' columns rely on.
constexpr int kSampleMaxVocab = 500000;

struct SampleParams {
  int N, V, rows;  // rows to draw, vocab, rows of logits
  long long row_stride;
  const void* logits;
  const int* row_index;  // [N] or null
  const float* uniforms;
  const float* temperature;  // each [N] or null
  const int* top_k;
  const float* top_p;
  const float* min_p;
  int* tokens;
};
cudaError_t launch_sample(const SampleParams& a, int dtype, cudaStream_t stream);

}  // namespace mt
