// C ABI of the serving operators around the verify step: host-side validation,
// workspace layout and launches.
#include <climits>
#include <cmath>

#include "api_common.cuh"
#include "serve.cuh"

namespace {

using namespace mt;

bool act_dtype(int dt) { return dt == MT_F32 || dt == MT_F16 || dt == MT_BF16; }

int act_bytes(int dt) { return dt == MT_F32 ? 4 : 2; }

// Whole 16-byte steps between tokens and between heads.
bool strides_ok(const long long (&st)[2], int elem) {
  return st[0] >= 0 && st[1] >= 0 && st[0] * elem % 16 == 0 && st[1] * elem % 16 == 0;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// A table made for this head size on the current device.
int check_rope(const mt_rope* rope, int head_dim) {
  int dev = 0;
  if (rope->head_dim != head_dim) return MT_ERR_INVALID_ARG;
  if (cudaGetDevice(&dev) != cudaSuccess) return MT_ERR_CUDA;
  return dev == rope->device ? MT_OK : MT_ERR_INVALID_ARG;
}

int check_block8(const mt_attn_desc* d) {
  if (!d) return MT_ERR_INVALID_ARG;
  if (d->batch < 1 || d->batch > kMaxBatch) return MT_ERR_INVALID_ARG;
  if (d->tree_size < 1 || d->tree_size > kMaxTree) return MT_ERR_UNSUPPORTED;
  if (d->num_kv_heads < 1 || d->num_q_heads < 1 || d->num_q_heads % d->num_kv_heads) return MT_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return MT_ERR_UNSUPPORTED;
  if (d->page_size != 16) return MT_ERR_UNSUPPORTED;
  if (d->max_blocks_per_seq < 1 || d->num_pages < 1) return MT_ERR_INVALID_ARG;
  if ((long long)d->num_pages * d->num_kv_heads * d->page_size >= (1ll << 31) ||
      (long long)d->max_blocks_per_seq * d->page_size >= (1ll << 31) - 4096)
    return MT_ERR_UNSUPPORTED;
  if (d->dtype != MT_F16 && d->dtype != MT_BF16) return MT_ERR_UNSUPPORTED;
  if (d->cache_dtype != MT_E4M3) return MT_ERR_UNSUPPORTED;
  if (!(d->sm_scale >= 0.f) || std::isinf(d->sm_scale)) return MT_ERR_INVALID_ARG;
  return MT_OK;
}

struct Block8Ws {
  size_t ml, o, counters, pfx, anc, pieces, q8, q_scale, k_blocks, v_blocks, block_scales, depth, total;
  int rows, nrg, part_rows, G;
  Block8Plan plan;
};

// visible_blocks: the most pages that a sequence's new tokens see; reach: with a window or a log-sum-exp
int block8_ws(const mt_attn_desc* d, int visible_blocks, bool windowed, bool reach, Block8Ws* w) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MT_ERR_CUDA;
  const long long rows = (long long)d->tree_size * (d->num_q_heads / d->num_kv_heads);
  if (rows > (1 << 20)) return MT_ERR_UNSUPPORTED;
  w->rows = (int)rows;
  w->plan = block8_plan(d->batch, d->num_kv_heads, w->rows, d->num_q_heads / d->num_kv_heads, visible_blocks, d->tree_size,
                        d->dtype, windowed, sms);
  w->nrg = w->plan.nrg;
  w->part_rows = w->rows < w->plan.rows_per_group ? w->rows : w->plan.rows_per_group;
  w->G = w->plan.ctas;
  if (!w->plan.tc && w->G > kMaxFragCtas) return MT_ERR_UNSUPPORTED;
  const long long nslots = (long long)d->batch * d->num_kv_heads * w->nrg + w->G;
  if (nslots > (1ll << 30)) return MT_ERR_INVALID_ARG;
  size_t off = kAlign;  // status word and padding
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes);
    return at;
  };
  // the one part that has to be zero between calls comes first, at the same place
  // for every descriptor, so that a workspace serves any that it is large enough for
  w->counters = take(kMaxFragCtas * sizeof(unsigned));
  const size_t part = (size_t)nslots * w->part_rows;
  w->ml = take(part * sizeof(float2));
  w->o = take(part * d->head_dim * sizeof(float));
  if (w->plan.tc) {
    const size_t nodes = (size_t)d->batch * d->tree_size, qrows = nodes * d->num_q_heads;
    const size_t blocks = (size_t)d->batch * d->num_kv_heads * ((d->tree_size + 15) / 16);
    if ((long long)blocks * 16 >= (1ll << 31)) return MT_ERR_UNSUPPORTED;
    w->pfx = take(sizeof(int) * (size_t)(d->batch + 1));
    w->anc = take(nodes * sizeof(unsigned long long));
    w->pieces = take(sizeof(int) * (size_t)piece_rec_offset(w->G) + sizeof(PieceRec) * kMaxPieceRecs * (size_t)w->G);
    w->q8 = take(qrows * d->head_dim * w->plan.parts);
    w->q_scale = take(qrows * sizeof(float));
    w->k_blocks = take(blocks * 16 * d->head_dim);
    w->v_blocks = take(blocks * 16 * d->head_dim);
    w->block_scales = take(2 * blocks * sizeof(float));
    w->depth = reach ? take(nodes * sizeof(int)) : 0;
  }
  w->total = off;
  return MT_OK;
}

// window 0: the whole cache is visible and there is no lse (the kernels without either)
int attn_block8(const mt_attn_desc* d, int window, int sinks, const void* q, const void* k_new, const void* v_new,
                const void* k_cache, const void* v_cache, const float* k_scales, const float* v_scales,
                const int32_t* block_tables, const int32_t* seq_lens, const int32_t* tree_parents, void* out,
                float* lse, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  int st = check_block8(d);
  if (st != MT_OK) return st;
  if (!q || !k_new || !v_new || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables || !seq_lens || !out ||
      !workspace)
    return MT_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(out) || reinterpret_cast<uintptr_t>(workspace) % kAlign ||
      !aligned4(k_scales, v_scales, block_tables, seq_lens, tree_parents, lse))
    return MT_ERR_INVALID_ARG;
  // the output is written while other blocks still read the inputs
  const size_t tokens = (size_t)d->batch * d->tree_size, q_bytes = tokens * d->num_q_heads * d->head_dim * 2;
  const size_t new_bytes = tokens * d->num_kv_heads * d->head_dim * 2;
  if (overlap(out, q_bytes, q, q_bytes) || overlap(out, q_bytes, k_new, new_bytes) ||
      overlap(out, q_bytes, v_new, new_bytes))
    return MT_ERR_INVALID_ARG;
  if (lse) {
    const size_t lse_bytes = tokens * d->num_q_heads * 4;
    if (overlap(lse, lse_bytes, q, q_bytes) ||
        overlap(lse, lse_bytes, k_new, new_bytes) || overlap(lse, lse_bytes, v_new, new_bytes) ||
        overlap(lse, lse_bytes, out, q_bytes))
      return MT_ERR_INVALID_ARG;
  }
  // sinks in whole pages, and a window that starts and ends inside two
  long long blocks = d->max_blocks_per_seq;
  if (window > 0 && ((long long)sinks + 15) / 16 + ((long long)window + 15) / 16 + 1 < blocks)
    blocks = ((long long)sinks + 15) / 16 + ((long long)window + 15) / 16 + 1;
  Block8Ws w;
  // (a log-sum-exp alone leaves the output as the call without one has it, so with its kernel)
  st = block8_ws(d, (int)blocks, window > 0 && window < INT_MAX, window > 0, &w);
  if (st != MT_OK) return st;
  if (ws_bytes < w.total) return MT_ERR_INVALID_ARG;
  char* ws = static_cast<char*>(workspace);
  Block8Params p{};
  AttnParams& a = p.a;
  a.B = d->batch; a.T = d->tree_size; a.Hq = d->num_q_heads; a.Hkv = d->num_kv_heads;
  a.D = d->head_dim; a.P = d->page_size; a.max_blocks = d->max_blocks_per_seq; a.num_pages = d->num_pages;
  a.g = d->num_q_heads / d->num_kv_heads;
  a.rows = w.rows; a.rows_per_group = w.plan.rows_per_group; a.part_rows = w.part_rows;
  const float scale = d->sm_scale > 0.f ? d->sm_scale : (float)(1.0 / std::sqrt((double)d->head_dim));
  a.scale_log2 = scale * 1.4426950408889634f;
  a.q_rot = q; a.k_cache = k_cache; a.v_cache = v_cache;
  a.block_tables = block_tables; a.seq_lens = seq_lens;
  a.out = out; a.status = reinterpret_cast<int*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.sched.B = d->batch; a.sched.T = d->tree_size; a.sched.Hkv = d->num_kv_heads;
  a.sched.nrg = w.nrg; a.sched.G = w.G; a.sched.splits = 0; a.sched.seg_cost = w.plan.seg_cost;
  p.k_scales = k_scales; p.v_scales = v_scales;
  p.k_new = k_new; p.v_new = v_new; p.parents = tree_parents;
  p.window = window; p.sinks = sinks; p.lse = lse;
  if (!w.plan.tc) {
    p.frag_o = reinterpret_cast<float*>(ws + w.o);
    p.frag_tiles = reinterpret_cast<unsigned*>(ws + w.counters);
    return cuda_status(launch_attn_block8(p, d->dtype, stream));
  }
  a.part_o = ws + w.o;
  p.tile_pfx = reinterpret_cast<int*>(ws + w.pfx);
  a.sched.tile_pfx = p.tile_pfx;
  p.parts = w.plan.parts;
  p.q8 = reinterpret_cast<uint8_t*>(ws + w.q8);
  p.q_scale = reinterpret_cast<float*>(ws + w.q_scale);
  p.k_blocks = reinterpret_cast<uint8_t*>(ws + w.k_blocks);
  p.v_blocks = reinterpret_cast<uint8_t*>(ws + w.v_blocks);
  p.k_block_scales = reinterpret_cast<float*>(ws + w.block_scales);
  p.v_block_scales = p.k_block_scales + (size_t)d->batch * d->num_kv_heads * ((d->tree_size + 15) / 16);
  p.anc = reinterpret_cast<unsigned long long*>(ws + w.anc);
  p.depth = window > 0 ? reinterpret_cast<int*>(ws + w.depth) : nullptr;
  p.pieces = reinterpret_cast<int*>(ws + w.pieces);
  wait_bound(&a.wait_limit_ns, &a.test_stall);
  st = cuda_status(launch_block8_prep(p, d->dtype, stream));
  if (st == MT_OK) st = cuda_status(launch_attn_block8_tc(p, d->dtype, stream));
  if (st != MT_OK) return st;
  return cuda_status(launch_block8_combine(p, d->dtype, stream));
}

int append(const mt_append_desc* d, AppendParams& a, const void* k, const void* v, const mt_rope* rope, void* k_cache,
           void* v_cache, float* k_scales, float* v_scales, const int32_t* block_tables, const int32_t* seq_lens,
           void* status_ws, cudaStream_t stream) {
  if (d->batch < 1 || d->batch > kMaxBatch || d->num_rows < 0 || d->num_kv_heads < 1 || d->max_blocks_per_seq < 1 ||
      d->num_pages < 1)
    return MT_ERR_INVALID_ARG;
  if (!act_dtype(d->dtype) || (d->cache_dtype != 0 && d->cache_dtype != MT_E4M3)) return MT_ERR_UNSUPPORTED;
  if (d->head_dim != 64 && d->head_dim != 128) return MT_ERR_UNSUPPORTED;
  if (d->page_size != 16) return MT_ERR_UNSUPPORTED;
  if ((long long)d->num_pages * d->num_kv_heads * d->page_size >= (1ll << 31) ||
      (long long)d->max_blocks_per_seq * d->page_size >= (1ll << 31) - 4096)
    return MT_ERR_UNSUPPORTED;
  if ((k_scales == nullptr) != (v_scales == nullptr) || (k_scales && d->cache_dtype != MT_E4M3))
    return MT_ERR_INVALID_ARG;
  if (d->num_rows == 0) return MT_OK;  // nothing new
  if (!k || !v || !k_cache || !v_cache || !block_tables || !seq_lens || !status_ws) return MT_ERR_INVALID_ARG;
  const int eb = act_bytes(d->dtype);
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(status_ws) ||
      !strides_ok(d->k_stride, eb) || !strides_ok(d->v_stride, eb) ||
      !aligned4(k_scales, v_scales, block_tables, seq_lens, a.row_offsets, a.accept_path, a.accept_len))
    return MT_ERR_INVALID_ARG;
  a.mode = d->cache_dtype == 0 ? kCacheAct : k_scales ? kCacheBlock8 : kCacheE4m3;
  if (a.mode == kCacheE4m3 && (!(d->k_scale > 0.f) || std::isinf(d->k_scale) || !(d->v_scale > 0.f) ||
                               std::isinf(d->v_scale)))
    return MT_ERR_INVALID_ARG;
  if (rope) {
    const int st = check_rope(rope, d->head_dim);
    if (st != MT_OK) return st;
    a.rope = rope->table;
    a.max_pos = rope->max_pos;
  }
  a.B = d->batch; a.N = d->num_rows; a.Hkv = d->num_kv_heads; a.D = d->head_dim;
  a.max_blocks = d->max_blocks_per_seq; a.num_pages = d->num_pages;
  a.k = k; a.v = v;
  for (int i = 0; i < 2; ++i) {
    a.k_st[i] = d->k_stride[i];
    a.v_st[i] = d->v_stride[i];
  }
  a.k_cache = k_cache; a.v_cache = v_cache; a.k_scales = k_scales; a.v_scales = v_scales;
  a.k_scale = d->k_scale; a.v_scale = d->v_scale;
  a.block_tables = block_tables; a.seq_lens = seq_lens;
  a.status = static_cast<int*>(status_ws);
  return cuda_status(launch_append(a, d->dtype, stream));
}

}  // namespace

extern "C" {

int mt_qk_norm_rope(const mt_norm_rope_desc* d, const void* q, const void* k, const int32_t* positions,
                    const void* q_weight, const void* k_weight, const mt_rope* rope, void* q_out, void* k_out,
                    void* status_ws, cudaStream_t stream) {
  const mt_call_range range("mt_qk_norm_rope");
  if (!d || d->num_tokens < 0 || d->num_q_heads < 1 || d->num_kv_heads < 1) return MT_ERR_INVALID_ARG;
  if (!act_dtype(d->dtype) || (d->head_dim != 64 && d->head_dim != 128)) return MT_ERR_UNSUPPORTED;
  if ((q_weight == nullptr) != (k_weight == nullptr) || (!q_weight && !rope)) return MT_ERR_INVALID_ARG;
  if (q_weight && (!(d->eps >= 0.f) || std::isinf(d->eps))) return MT_ERR_INVALID_ARG;
  if (d->num_tokens == 0) return MT_OK;
  if (!q || !k || !q_out || !k_out || !status_ws || (rope && !positions)) return MT_ERR_INVALID_ARG;
  const int eb = act_bytes(d->dtype);
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(status_ws) ||
      !aligned16(q_weight) || !aligned16(k_weight) || !strides_ok(d->q_stride, eb) || !strides_ok(d->k_stride, eb) ||
      !strides_ok(d->q_out_stride, eb) || !strides_ok(d->k_out_stride, eb) || !aligned4(positions))
    return MT_ERR_INVALID_ARG;
  NormRopeParams a{};
  if (rope) {
    const int st = check_rope(rope, d->head_dim);
    if (st != MT_OK) return st;
    a.rope = rope->table;
    a.max_pos = rope->max_pos;
  }
  a.N = d->num_tokens; a.Hq = d->num_q_heads; a.Hkv = d->num_kv_heads; a.D = d->head_dim;
  a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
  for (int i = 0; i < 2; ++i) {
    a.q_st[i] = d->q_stride[i];
    a.k_st[i] = d->k_stride[i];
    a.qo_st[i] = d->q_out_stride[i];
    a.ko_st[i] = d->k_out_stride[i];
  }
  a.positions = positions;
  a.q_weight = q_weight; a.k_weight = k_weight; a.eps = d->eps;
  a.status = static_cast<int*>(status_ws);
  return cuda_status(launch_norm_rope(a, d->dtype, stream));
}

int mt_kv_append_paged(const mt_append_desc* d, const void* k, const void* v, const int32_t* row_offsets,
                       const mt_rope* rope, void* k_cache, void* v_cache, float* k_scales, float* v_scales,
                       const int32_t* block_tables, const int32_t* seq_lens, void* status_ws, cudaStream_t stream) {
  const mt_call_range range("mt_kv_append_paged");
  if (!d || !row_offsets) return MT_ERR_INVALID_ARG;
  AppendParams a{};
  a.row_offsets = row_offsets;
  return append(d, a, k, v, rope, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, status_ws, stream);
}

int mt_kv_append_accepted(const mt_append_desc* d, int tree_size, int max_depth, const void* k, const void* v,
                          const int32_t* accept_path, const int32_t* accept_len, const mt_rope* rope, void* k_cache,
                          void* v_cache, float* k_scales, float* v_scales, const int32_t* block_tables,
                          const int32_t* seq_lens, void* status_ws, cudaStream_t stream) {
  const mt_call_range range("mt_kv_append_accepted");
  if (!d || !accept_path || !accept_len) return MT_ERR_INVALID_ARG;
  if (tree_size < 1 || tree_size > kMaxTree) return MT_ERR_UNSUPPORTED;
  if (max_depth < 0 || max_depth >= kMaxTree || d->batch < 1 || d->batch > kMaxBatch ||
      d->num_rows != d->batch * tree_size)
    return MT_ERR_INVALID_ARG;
  AppendParams a{};
  a.accept_path = accept_path;
  a.accept_len = accept_len;
  a.T = tree_size;
  a.max_depth = max_depth;
  return append(d, a, k, v, rope, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, status_ws, stream);
}

size_t mt_tree_attn_block8_workspace_size(const mt_attn_desc* d) {
  Block8Ws w, r;  // of either form (without a window or a log-sum-exp the nodes' depths are not needed)
  if (check_block8(d) != MT_OK || block8_ws(d, d->max_blocks_per_seq, false, true, &w) != MT_OK ||
      block8_ws(d, d->max_blocks_per_seq, true, true, &r) != MT_OK)
    return 0;
  return w.total > r.total ? w.total : r.total;
}

int mt_tree_attn_paged_block8(const mt_attn_desc* d, const void* q, const void* k_new, const void* v_new,
                              const void* k_cache, const void* v_cache, const float* k_scales, const float* v_scales,
                              const int32_t* block_tables, const int32_t* seq_lens, const int32_t* tree_parents,
                              void* out, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  const mt_call_range range("mt_tree_attn_paged_block8");
  return attn_block8(d, 0, 0, q, k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens,
                     tree_parents, out, nullptr, workspace, ws_bytes, stream);
}

int mt_tree_attn_paged_block8_window(const mt_attn_desc* d, int window, int sinks, const void* q, const void* k_new,
                                     const void* v_new, const void* k_cache, const void* v_cache,
                                     const float* k_scales, const float* v_scales, const int32_t* block_tables,
                                     const int32_t* seq_lens, const int32_t* tree_parents, void* out, float* lse,
                                     void* workspace, size_t ws_bytes, cudaStream_t stream) {
  const mt_call_range range("mt_tree_attn_paged_block8_window");
  if (window < 0 || sinks < 0) return MT_ERR_INVALID_ARG;
  return attn_block8(d, window ? window : INT_MAX, sinks, q, k_new, v_new, k_cache, v_cache, k_scales, v_scales,
                     block_tables, seq_lens, tree_parents, out, lse, workspace, ws_bytes, stream);
}

int mt_kv_attn_weights(const mt_attn_desc* d, int max_depth, float decay, const void* q, const float* lse,
                       const void* k_cache, const float* k_scales, const int32_t* block_tables,
                       const int32_t* seq_lens, const int32_t* prev_lens, const int32_t* accept_path,
                       const int32_t* accept_len, const float* weights, float* out, void* status_ws,
                       cudaStream_t stream) {
  const mt_call_range range("mt_kv_attn_weights");
  const int st = check_block8(d);
  if (st != MT_OK) return st;
  if (!q || !lse || !k_cache || !k_scales || !block_tables || !seq_lens || !weights || !out || !status_ws)
    return MT_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(weights) || !aligned16(out) || !aligned16(status_ws) ||
      !aligned4(lse, k_scales, block_tables, seq_lens, prev_lens, accept_path, accept_len))
    return MT_ERR_INVALID_ARG;
  if ((accept_path == nullptr) != (accept_len == nullptr)) return MT_ERR_INVALID_ARG;
  if (accept_path && (max_depth < 0 || max_depth >= kMaxTree)) return MT_ERR_INVALID_ARG;
  if (!(decay >= 0.f) || std::isinf(decay)) return MT_ERR_INVALID_ARG;
  const size_t bytes = (size_t)d->num_pages * d->num_kv_heads * 16 * sizeof(float);
  if (out != weights && overlap(out, bytes, weights, bytes)) return MT_ERR_INVALID_ARG;
  WeightsParams p{};
  p.B = d->batch; p.T = d->tree_size; p.Hq = d->num_q_heads; p.Hkv = d->num_kv_heads; p.D = d->head_dim;
  p.max_blocks = d->max_blocks_per_seq; p.num_pages = d->num_pages;
  p.g = d->num_q_heads / d->num_kv_heads;
  const long long rows = (long long)(accept_path ? max_depth + 1 : d->tree_size) * p.g;
  if (rows > (1 << 20)) return MT_ERR_UNSUPPORTED;
  p.rows = (int)rows;
  p.q = q; p.lse = lse; p.k_cache = k_cache; p.k_scales = k_scales;
  p.block_tables = block_tables; p.seq_lens = seq_lens; p.prev_lens = prev_lens;
  p.accept_path = accept_path; p.accept_len = accept_len; p.max_depth = max_depth;
  const float scale = d->sm_scale > 0.f ? d->sm_scale : (float)(1.0 / std::sqrt((double)d->head_dim));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.decay = decay;
  p.weights = weights; p.out = out;
  p.status = static_cast<int*>(status_ws);
  wait_bound(&p.wait_limit_ns, &p.test_stall);
  return cuda_status(launch_kv_weights(p, d->dtype, stream));
}

int mt_kv_evict(const mt_attn_desc* d, int new_blocks_per_seq, int budget, int sinks, int recent, void* k_cache,
                void* v_cache, float* k_scales, float* v_scales, float* weights, const int32_t* block_tables,
                const int32_t* seq_lens, const int32_t* new_tables, int32_t* kept, void* status_ws,
                cudaStream_t stream) {
  const mt_call_range range("mt_kv_evict");
  if (!d || d->batch < 1 || d->batch > kMaxBatch || d->num_kv_heads < 1 || d->max_blocks_per_seq < 1 || d->num_pages < 1)
    return MT_ERR_INVALID_ARG;
  if (!act_dtype(d->dtype) || (d->cache_dtype != 0 && d->cache_dtype != MT_E4M3)) return MT_ERR_UNSUPPORTED;
  if (d->head_dim != 64 && d->head_dim != 128) return MT_ERR_UNSUPPORTED;
  if (d->page_size != 16) return MT_ERR_UNSUPPORTED;
  if ((long long)d->num_pages * d->num_kv_heads * d->page_size >= (1ll << 31) ||
      (long long)d->max_blocks_per_seq * d->page_size >= (1ll << 31) - 4096)
    return MT_ERR_UNSUPPORTED;
  if (budget < 1 || sinks < 0 || recent < 0 || (long long)sinks + recent > budget || new_blocks_per_seq < 1 ||
      (long long)new_blocks_per_seq * 16 < budget)
    return MT_ERR_INVALID_ARG;
  if ((k_scales == nullptr) != (v_scales == nullptr) || (k_scales && d->cache_dtype != MT_E4M3))
    return MT_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !weights || !block_tables || !seq_lens || !new_tables || !kept || !status_ws)
    return MT_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(weights) || !aligned16(status_ws) ||
      !aligned4(k_scales, v_scales, block_tables, seq_lens, new_tables, kept))
    return MT_ERR_INVALID_ARG;
  EvictParams p{};
  p.B = d->batch; p.Hkv = d->num_kv_heads; p.max_blocks = d->max_blocks_per_seq; p.new_blocks = new_blocks_per_seq;
  p.num_pages = d->num_pages;
  p.row_bytes = d->head_dim * (d->cache_dtype == MT_E4M3 ? 1 : act_bytes(d->dtype));
  p.budget = budget; p.sinks = sinks; p.recent = recent;
  p.k_cache = k_cache; p.v_cache = v_cache; p.k_scales = k_scales; p.v_scales = v_scales; p.weights = weights;
  p.block_tables = block_tables; p.seq_lens = seq_lens; p.new_tables = new_tables;
  p.kept = kept;
  p.status = static_cast<int*>(status_ws);
  return cuda_status(launch_kv_evict(p, stream));
}

int mt_process_logits(const mt_logits_desc* d, const void* logits, void* out, const int32_t* history,
                      const int32_t* history_lens, const int32_t* output_starts, const float* repetition,
                      const float* presence, const float* frequency, const int32_t* bias_tokens,
                      const float* bias_values, const int32_t* mask, const int32_t* mask_index,
                      const int32_t* tree_tokens, const int32_t* tree_parents, void* status_ws, cudaStream_t stream) {
  const mt_call_range range("mt_process_logits");
  if (!d || d->batch < 0 || d->tree_size < 0 || d->vocab < 1 || d->history_width < 0 || d->num_bias < 0 ||
      d->num_masks < 0 || d->history_width >= (1 << 30))
    return MT_ERR_INVALID_ARG;
  if (!act_dtype(d->dtype) || d->vocab > (1 << 30)) return MT_ERR_UNSUPPORTED;
  const long long rows = (long long)d->batch * d->tree_size;
  if (rows > (1 << 24)) return MT_ERR_INVALID_ARG;
  for (const long long s : {d->stride[0], d->stride[1], d->out_stride[0], d->out_stride[1]})
    if (s < 0 || s > (1ll << 38)) return MT_ERR_INVALID_ARG;  // (their sums over 2^24 rows fit)
  if ((history && !history_lens) || (history_lens && !history && d->history_width > 0) || (output_starts && !history_lens))
    return MT_ERR_INVALID_ARG;
  if ((bias_tokens == nullptr) != (bias_values == nullptr) || (mask_index && !mask) || (tree_parents && !tree_tokens))
    return MT_ERR_INVALID_ARG;
  if (mask && !mask_index && d->num_masks < rows) return MT_ERR_INVALID_ARG;
  if (tree_tokens && d->tree_size > kMaxTree) return MT_ERR_UNSUPPORTED;
  if (rows == 0) return MT_OK;
  const size_t eb = (size_t)act_bytes(d->dtype);
  if (!logits || !out || !status_ws || reinterpret_cast<uintptr_t>(logits) % eb ||
      reinterpret_cast<uintptr_t>(out) % eb || !aligned16(status_ws) ||
      !aligned4(history, history_lens, output_starts, repetition, presence, frequency, bias_tokens, bias_values, mask,
                mask_index, tree_tokens, tree_parents))
    return MT_ERR_INVALID_ARG;
  // rows of `out` apart from one another, and `out` the logits themselves or apart from them
  const long long b1 = d->batch - 1, t1 = d->tree_size - 1, v = d->vocab;
  const long long* st = d->out_stride;
  if ((t1 && st[1] < v) || (b1 && st[0] < v) ||
      (t1 && b1 && st[0] < t1 * st[1] + v && st[1] < b1 * st[0] + v))
    return MT_ERR_INVALID_ARG;
  const size_t in_bytes = (size_t)(b1 * d->stride[0] + t1 * d->stride[1] + v) * eb;
  const size_t out_bytes = (size_t)(b1 * st[0] + t1 * st[1] + v) * eb;
  const bool same = logits == out && (!b1 || d->stride[0] == st[0]) && (!t1 || d->stride[1] == st[1]);
  if (!same && overlap(logits, in_bytes, out, out_bytes)) return MT_ERR_INVALID_ARG;
  LogitsParams p{};
  p.B = d->batch; p.T = d->tree_size; p.V = d->vocab;
  p.logits = logits; p.out = out;
  for (int i = 0; i < 2; ++i) {
    p.stride[i] = d->stride[i];
    p.out_stride[i] = d->out_stride[i];
  }
  p.history = history; p.history_lens = history_lens; p.history_width = history ? d->history_width : 0;
  p.output_starts = output_starts;
  p.repetition = repetition; p.presence = presence; p.frequency = frequency;
  p.bias_tokens = bias_tokens; p.bias_values = bias_values; p.num_bias = bias_tokens ? d->num_bias : 0;
  p.mask = mask; p.num_masks = mask ? d->num_masks : 0; p.mask_index = mask_index;
  p.tree_tokens = tree_tokens; p.tree_parents = tree_parents;
  p.status = static_cast<int*>(status_ws);
  return cuda_status(launch_logits(p, d->dtype, stream));
}

int mt_sample_tokens(int num_rows, int vocab, mt_dtype logits_dtype, const void* logits, int num_logit_rows,
                     long long row_stride, const int32_t* row_index, const float* uniforms, const float* temperature,
                     const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens,
                     cudaStream_t stream) {
  const mt_call_range range("mt_sample_tokens");
  if (num_rows < 0 || num_rows > (1 << 24) || vocab < 1 || num_logit_rows < 0 || row_stride < 0)
    return MT_ERR_INVALID_ARG;
  if (!act_dtype(logits_dtype) || vocab > kSampleMaxVocab) return MT_ERR_UNSUPPORTED;
  if (!row_index && num_logit_rows != num_rows) return MT_ERR_INVALID_ARG;
  if (num_rows == 0) return MT_OK;
  if ((!logits && num_logit_rows > 0) || !uniforms || !tokens ||
      reinterpret_cast<uintptr_t>(logits) % act_bytes(logits_dtype) ||
      !aligned4(row_index, uniforms, temperature, top_k, top_p, min_p, tokens))
    return MT_ERR_INVALID_ARG;
  SampleParams a{};
  a.N = num_rows; a.V = vocab; a.rows = num_logit_rows; a.row_stride = row_stride;
  a.logits = logits; a.row_index = row_index; a.uniforms = uniforms;
  a.temperature = temperature; a.top_k = top_k; a.top_p = top_p; a.min_p = min_p;
  a.tokens = tokens;
  return cuda_status(launch_sample(a, logits_dtype, stream));
}

}  // extern "C"
