// Preparation of the block-scaled attention's tensor-core path: everything the
// attention kernel wants laid out before it streams the cache.
//   - each query row as E4M3 parts: scaled by a power of two so that its
//     largest magnitude is at most 448, then x = hi + lo (+ lo2 for fp16), each
//     part the code nearest to what is left.  A part takes 4 significant bits,
//     so two hold a bf16's 8 and three an fp16's 11; what falls below the last
//     part's smallest step is under 2^-17 of the row's maximum;
//   - the new tokens' keys and values as blocks of codes with their scales, in
//     the page layout [b][KV head][block][16][D];
//   - each node's ancestor mask (the Medusa tree mask, vLLM issue 1171);
//   - the schedule: tiles per sequence, their prefix, every CTA's pieces.
// Latency matters more than bytes here: the rows are a few MB at most.
#include "serve.cuh"

namespace mt {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kP = 16;

template <typename T, int D>
__device__ __forceinline__ void split_query(const Block8Params& p, long long row, int c) {
  const AttnParams& a = p.a;
  Row8<T> r0, r1;
  const T* src = static_cast<const T*>(a.q_rot) + row * D + 16 * c;
  r0.load(src);
  r1.load(src + 8);
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
  const long long nrows = (long long)a.B * a.T * a.Hq;
  for (int part = 0; part < p.parts; ++part) {
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
    *reinterpret_cast<uint4*>(p.q8 + (part * nrows + row) * D + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  // an infinity has no parts: the row's scores become NaN, as they would be
  if (c == 0) p.q_scale[row] = amax < INFINITY ? scale * a.scale_log2 : __int_as_float(0x7fffffff);
}

// One block of up to 16 new tokens of V, or of K (then `values` are their values).
template <typename T, int D>
__device__ __forceinline__ void quantise_block(const T* src, const T* values, size_t row_stride, int rows, uint8_t* dst,
                                               float* scale_out) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, STEPS = 16 / RPS;
  const int lane = threadIdx.x & 31, sub = lane / LPR, c = lane % LPR;
  Row8<T> lo[STEPS], hi[STEPS], vlo[STEPS], vhi[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = s * RPS + sub;
    lo[s].zero();
    hi[s].zero();
    vlo[s].zero();
    vhi[s].zero();
    if (r < rows) {
      lo[s].load(src + r * row_stride + 16 * c);
      hi[s].load(src + r * row_stride + 16 * c + 8);
      if (values) {  // asked for with the rest
        vlo[s].load(values + r * row_stride + 16 * c);
        vhi[s].load(values + r * row_stride + 16 * c + 8);
      }
    }
  }
  unsigned odd = 0;  // the tokens that have an element that is not finite
  if (values && !(largest_bits<T, STEPS>(vlo, vhi) < INFINITY)) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) odd |= odd_rows<RPS>(not_finite(vlo[s]) || not_finite(vhi[s])) << (s * RPS);
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
    float x[8], y[8];
    lo[s].to_f(x);
    hi[s].to_f(y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] *= inv;
      y[e] *= inv;
    }
    if (values && (odd >> r & 1u)) x[0] = __int_as_float(0x7fffffff);
    const uint2 u = e4m3x8_of(x), v = e4m3x8_of(y);
    *reinterpret_cast<uint4*>(dst + r * D + 16 * c) = make_uint4(u.x, u.y, v.x, v.y);
  }
  if (lane == 0) *scale_out = scale;
}

// Whether the piece walk's products fit in 32 bits (the balanced schedule's
// total cost times G + 1).
__device__ __forceinline__ bool fits_int(const Sched& s, int total) {
  const long long HR = (long long)s.Hkv * s.nrg;
  return ((long long)total * HR + (long long)s.seg_cost * s.B * HR) * (s.G + 1) < (1LL << 31);
}

template <typename I>
__device__ void list_pieces(const Block8Params& p, const Sched& sc) {
  PieceRec* recs = reinterpret_cast<PieceRec*>(p.pieces + piece_rec_offset(sc.G));
  for (int c = threadIdx.x; c < sc.G; c += kThreads) {
    PieceIterT<I> it;
    it.init(sc, c);
    Piece pc;
    int n = 0;
    while (it.next(pc)) {
      if (n == kMaxPieceRecs) {
        n = -1;
        break;
      }
      PieceRec r;
      r.b = pc.b; r.kvh = pc.kvh; r.rg = pc.rg; r.seg = pc.seg;
      r.tile_begin = pc.tile_begin; r.tile_end = pc.tile_end; r.slot = pc.slot;
      r.L = p.a.seq_lens[pc.b];
      recs[(size_t)c * kMaxPieceRecs + n] = r;
      ++n;
    }
    p.pieces[c] = n;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) block8_prep_kernel(Block8Params p) {
  const AttnParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nnew = (a.T + kP - 1) / kP;
  pdl_wait();
  if (blockIdx.x == 0) {
    extern __shared__ int s_pfx[];  // [B + 1]
    __shared__ int s_warp[kWarps];
    const int total = block8_prefix<kWarps>(a, s_pfx, s_warp, true);
    for (int b = tid; b <= a.B; b += kThreads) p.tile_pfx[b] = s_pfx[b];
    Sched sc = a.sched;
    sc.tile_pfx = s_pfx;
    if (fits_int(sc, total)) list_pieces<int>(p, sc);
    else list_pieces<long long>(p, sc);
    return;
  }
  const long long nw = (long long)(gridDim.x - 1) * kWarps;
  const long long gw = (long long)(blockIdx.x - 1) * kWarps + warp;
  // new tokens' blocks: K, then V
  const long long nblk = (long long)a.B * a.Hkv * nnew;
  const size_t rs = (size_t)a.Hkv * D;
  for (long long u = gw; u < 2 * nblk; u += nw) {
    const bool is_v = u >= nblk;
    const long long blk = is_v ? u - nblk : u;
    const int j = (int)(blk % nnew), h = (int)(blk / nnew % a.Hkv), b = (int)(blk / nnew / a.Hkv);
    const size_t at = ((size_t)b * a.T + j * kP) * rs + (size_t)h * D;
    const T* values = static_cast<const T*>(p.v_new) + at;
    quantise_block<T, D>(is_v ? values : static_cast<const T*>(p.k_new) + at, is_v ? nullptr : values, rs, min(kP, a.T - j * kP), (is_v ? p.v_blocks : p.k_blocks) + (size_t)blk * kP * D,
                         (is_v ? p.v_block_scales : p.k_block_scales) + blk);
  }
  // ancestor masks: a warp per sequence, lane l for nodes l and l + 32
  __shared__ int s_par[kWarps][kMaxTree];
  for (long long b = gw; b < a.B; b += nw) {
    bool ok = true;
    for (int i = lane; i < a.T; i += 32) {
      const int par = p.parents ? p.parents[(size_t)b * a.T + i] : i - 1;
      const bool fine = i == 0 ? par == -1 : (par >= 0 && par < i);
      ok = ok && fine;
      s_par[warp][i] = fine ? par : -1;
    }
    if (!__all_sync(0xffffffffu, ok) && lane == 0 && a.seq_lens[b] >= 0) set_status(a.status, kStTree);
    __syncwarp();
    for (int i = lane; i < a.T; i += 32) {
      unsigned long long anc = 0;
      for (int n = i; n >= 0; n = s_par[warp][n]) anc |= 1ull << n;  // parents are earlier: at most T steps
      p.anc[(size_t)b * a.T + i] = anc;
    }
    __syncwarp();
  }
  // queries
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  const long long nrows = (long long)a.B * a.T * a.Hq;
  for (long long r0 = gw * RPW; r0 < nrows; r0 += nw * RPW) {
    const long long row = r0 + lane / LPR;
    split_query<T, D>(p, row < nrows ? row : nrows - 1, lane % LPR);  // the last row again, with the same result
  }
}

template <typename T, int D>
cudaError_t launch_t(const Block8Params& p, cudaStream_t stream) {
  const AttnParams& a = p.a;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.B * a.T * a.Hq;
  long long blocks = (rows * (D / 16) + kThreads - 1) / kThreads + 1;
  const long long wave = 4LL * sms;
  if (blocks > wave) blocks = wave;
  if (blocks < 2) blocks = 2;
  return launch_pdl(block8_prep_kernel<T, D>, dim3((unsigned)blocks), dim3(kThreads), sizeof(int) * (size_t)(a.B + 1),
                    stream, p);
}

template <typename T>
cudaError_t launch_d(const Block8Params& p, cudaStream_t stream) {
  return p.a.D == 64 ? launch_t<T, 64>(p, stream) : launch_t<T, 128>(p, stream);
}

}  // namespace

cudaError_t launch_block8_prep(const Block8Params& p, int dtype, cudaStream_t stream) {
  return dtype == 1 ? launch_d<__half>(p, stream) : launch_d<__nv_bfloat16>(p, stream);
}

}  // namespace mt
