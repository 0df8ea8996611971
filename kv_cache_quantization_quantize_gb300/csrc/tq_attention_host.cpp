// Entry points of the exact paged cache and of cross attention: argument checks and launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include <cudaTypedefs.h>

#include "tq_attention.cuh"

namespace tq {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)
                                                                : nullptr;
  }();
  return encode;
}

cudaError_t encode_map(CUtensorMap* m, int dtype, int rank, void* base, const cuuint64_t* dims, const cuuint64_t* strides,
                       const cuuint32_t* box) {
  const auto encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = encode(m, dtype == TQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                            base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t attn_tensor_map(const tq_kv& kv, bool values, int box_tokens, CUtensorMap* m) {
  const int64_t* st = values ? kv.v_strides : kv.k_strides;
  void* base = values ? kv.v : kv.k;
  const cuuint64_t d = (cuuint64_t)kv.head_dim;
  // an empty dimension is given as one (no request has tokens there), a stride that is never taken as any valid one
  const cuuint64_t tokens = (cuuint64_t)std::max(kv.tokens, 1), outer = (cuuint64_t)std::max(kv.outer, 1);
  const cuuint64_t dims[4] = {d, tokens, (cuuint64_t)kv.n_kv_heads, outer};
  auto bytes = [&](cuuint64_t n, int64_t stride) { return n > 1 ? (cuuint64_t)stride * 2 : d * 2; };
  const cuuint64_t strides[3] = {bytes(tokens, st[1]), bytes(dims[2], st[2]), bytes(outer, st[0])};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_tokens, 1, 1};
  return encode_map(m, kv.dtype, 4, base, dims, strides, box);
}

cudaError_t query_tensor_map(const tq_queries& q, int head_dim, int dtype, int G, CUtensorMap* m) {
  const cuuint64_t d = (cuuint64_t)head_dim;
  const cuuint64_t dims[3] = {d, (cuuint64_t)q.n_q_heads, (cuuint64_t)q.n_rows};
  auto bytes = [&](cuuint64_t n, int64_t stride) { return n > 1 ? (cuuint64_t)stride * 2 : d * 2; };
  const cuuint64_t strides[2] = {bytes(dims[1], q.q_strides[1]), bytes(dims[2], q.q_strides[0])};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(128 / G)};
  return encode_map(m, dtype, 3, const_cast<void*>(q.q), dims, strides, box);
}

}  // namespace tq

namespace {

tq_status fail(tq_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return tq::set_error(st, buf);
}

tq_status done(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return tq::set_error(TQ_OK, "");
}

// SMs of the current device (asked once per device).
cudaError_t sm_count(int* out) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*out = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev].store(*out, std::memory_order_relaxed);
  return e;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

tq_status check_map(const int32_t* table, int max_seqs, int max_pages, int64_t stride, const int32_t* free_ids,
                    int n_blocks, const int32_t* n_free, const int32_t* ids, int batch) {
  if (!table || !free_ids || !n_free || (!ids && batch > 0)) return fail(TQ_ERR_INVALID_ARG, "NULL array");
  if (max_seqs < 1 || max_pages < 1 || max_pages > (1 << 20))
    return fail(TQ_ERR_INVALID_ARG, "max_seqs %d, max_pages %d: at least 1, at most 2^20 pages", max_seqs, max_pages);
  if (stride < max_pages) return fail(TQ_ERR_INVALID_ARG, "table_stride %lld below max_pages", (long long)stride);
  if (n_blocks < 1 || n_blocks > (1 << 24) - 1) return fail(TQ_ERR_INVALID_ARG, "n_blocks %d: 1 to 2^24 - 1", n_blocks);
  if (batch < 0) return fail(TQ_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (batch > 4096) return fail(TQ_ERR_UNSUPPORTED, "batch %d: at most 4096", batch);
  return TQ_OK;
}

tq_status check_kv(const tq_kv* kv, bool map) {
  if (!kv) return fail(TQ_ERR_INVALID_ARG, "kv is NULL");
  if (kv->head_dim != 64 && kv->head_dim != 128 && kv->head_dim != 256)
    return fail(TQ_ERR_UNSUPPORTED, "head_dim %d: supported 64, 128, 256", kv->head_dim);
  if (kv->dtype != TQ_BF16 && kv->dtype != TQ_F16) return fail(TQ_ERR_UNSUPPORTED, "cache type %d: bf16 or f16", kv->dtype);
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 65535 || kv->outer < 0 || kv->tokens < 0)
    return fail(TQ_ERR_INVALID_ARG, "n_kv_heads %d, outer %d, tokens %d", kv->n_kv_heads, kv->outer, kv->tokens);
  if (!kv->outer || !kv->tokens) return TQ_OK;  // no element
  if (!kv->k || !kv->v) return fail(TQ_ERR_INVALID_ARG, "k or v is NULL");
  if (!map) return TQ_OK;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return fail(TQ_ERR_INVALID_ARG, "k and v have to be 16-byte aligned");
  const int size[3] = {kv->outer, kv->tokens, kv->n_kv_heads};
  for (int i = 0; i < 3; ++i)
    for (const int64_t st : {kv->k_strides[i], kv->v_strides[i]})
      if (size[i] > 1 && (st < 1 || st % 8 || st >= (int64_t)1 << 38))
        return fail(TQ_ERR_INVALID_ARG, "stride %lld of k or v: a positive multiple of 8 elements", (long long)st);
  return TQ_OK;
}

tq_status check_queries(const tq_queries* q, const tq_kv* kv) {
  if (!q) return fail(TQ_ERR_INVALID_ARG, "queries are NULL");
  if (q->batch < 0 || q->n_rows < 0 || q->max_q < 0 || q->max_kv < 0)
    return fail(TQ_ERR_INVALID_ARG, "batch %d, n_rows %d, max_q %d, max_kv %d: none below 0", q->batch, q->n_rows,
                q->max_q, q->max_kv);
  if (q->batch > 65535) return fail(TQ_ERR_UNSUPPORTED, "batch %d: at most 65535", q->batch);
  if (q->n_q_heads < 1 || q->n_q_heads % kv->n_kv_heads)
    return fail(TQ_ERR_INVALID_ARG, "n_q_heads %d not a multiple of n_kv_heads %d", q->n_q_heads, kv->n_kv_heads);
  if (q->n_q_heads / kv->n_kv_heads > 1024)
    return fail(TQ_ERR_UNSUPPORTED, "%d query heads per KV head: at most 1024", q->n_q_heads / kv->n_kv_heads);
  if ((int64_t)q->n_rows * q->n_q_heads >= (int64_t)1 << 31)
    return fail(TQ_ERR_UNSUPPORTED, "n_rows x n_q_heads: below 2^31");
  if (std::isnan(q->softmax_scale) || std::isinf(q->softmax_scale))
    return fail(TQ_ERR_INVALID_ARG, "softmax_scale is not finite");
  if (!q->batch || !q->n_rows) return TQ_OK;
  if (!q->q || !q->out || !q->d_q_starts) return fail(TQ_ERR_INVALID_ARG, "q, out or d_q_starts is NULL");
  if (!aligned(q->q, 16) || !aligned(q->out, 16)) return fail(TQ_ERR_INVALID_ARG, "q and out have to be 16-byte aligned");
  const int size[2] = {q->n_rows, q->n_q_heads};  // the stride of a size of 1 is never taken
  for (int i = 0; i < 2; ++i)
    if (size[i] > 1 && (q->q_strides[i] % 8 || q->out_strides[i] % 8))
      return fail(TQ_ERR_INVALID_ARG, "strides of q and out: multiples of 8 elements");
  return TQ_OK;
}

// Requests of up to 32 rows (queries x query heads per KV head) take the rows kernel, others the tensor cores. Measured
// with 4 query heads per KV head, head_dim 128: 32 rows, rows kernel against tensor cores: 19.8 against 26.9 us over
// 8192 tokens, 56 against 61 us over 65536; 64 rows, which would be two tiles: 22.8 against 27.0 us over 8192 tokens, but
// 83 against 63 us over 65536, and 28 against 22 us for 16 requests of 512.
tq::AttnPlan plan_of(const tq_queries& q, const tq_kv& kv, int sms) {
  tq::AttnPlan p;
  const int64_t rows = (int64_t)(q.max_q > 0 ? std::min(q.max_q, q.n_rows) : q.n_rows) * (q.n_q_heads / kv.n_kv_heads);
  const bool tc = rows > 32;
  static_cast<tq::AttnShape&>(p) = tc ? tq::attn_tc_shape(kv.head_dim, sms) : tq::attn_rows_shape(kv.head_dim, rows, sms);
  p.tc = tc;
  p.max_rows = rows;
  p.ctas = std::min(p.ctas, tq::kMaxAttnCtas);
  if (q.max_kv > 0) {  // no more CTAs than the most work there can be feeds: one tile of 64 tokens takes one
    const double tiles = (double)q.batch * kv.n_kv_heads * ((rows + p.tile_rows - 1) / p.tile_rows);
    const double most = tiles * ((double)q.max_kv * 64 / p.unit + 64 + p.cost);
    if (most < (double)p.ctas * p.least) p.ctas = std::max(1, (int)std::ceil(most / p.least));
  }
  p.bytes = p.ctas * p.cta_bytes;
  return p;
}

tq_status attend(const tq_queries* q, const tq_kv* kv_in, tq::AttnArgs& a, void* ws, size_t ws_bytes,
                 uint32_t* status, tq_stream_t stream) {
  if (!q->batch || !q->n_rows) return tq::set_error(TQ_OK, "");
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return done(e, "device");
  const tq::AttnPlan p = plan_of(*q, *kv_in, sms);
  if (!ws || ws_bytes < p.bytes || !aligned(ws, 256))
    return fail(TQ_ERR_INVALID_ARG, "workspace: %zu bytes, 256-byte aligned, are needed (got %zu)", p.bytes, ws_bytes);
  tq_kv kv = *kv_in;
  if (!kv.outer || !kv.tokens) {  // nothing to read: the tensor maps need an address all the same
    kv.k = kv.v = const_cast<void*>(q->q);
    kv.outer = kv.tokens = 0;
    for (int i = 0; i < 3; ++i) kv.k_strides[i] = kv.v_strides[i] = kv.head_dim;  // an empty tensor's may be anything
  }
  a.q = q->q;
  a.out = q->out;
  a.q_row = q->q_strides[0];
  a.q_head = q->q_strides[1];
  a.o_row = q->out_strides[0];
  a.o_head = q->out_strides[1];
  a.q_starts = q->d_q_starts;
  a.status = status;
  a.part = ws;
  const double scale = q->softmax_scale > 0.f ? (double)q->softmax_scale : 1.0 / std::sqrt((double)kv.head_dim);
  a.scale_log2 = (float)(scale * 1.4426950408889634);
  if (!std::isfinite(a.scale_log2)) return fail(TQ_ERR_INVALID_ARG, "softmax_scale %g is too large", scale);
  a.n_rows = q->n_rows;
  a.batch = q->batch;
  a.hq = q->n_q_heads;
  a.hkv = kv.n_kv_heads;
  a.G = a.hq / a.hkv;
  a.div_g.set((uint32_t)a.G);
  a.outer = kv.outer;
  a.tokens = kv.tokens;
  a.max_rows = (int)p.max_rows;
  // Costs are 64ths of a unit >> shift. The line's length is below tiles x (the longest tile's cost); the shift keeps
  // that below 2^30. Launches that need one have lines of more than 2^30 / 64 units, and costs that much coarser.
  const double slope = a.causal ? std::max(1, p.tile_rows * 64 / (a.G * p.unit)) : 0;
  const double tiles = ((double)a.n_rows * a.G / p.tile_rows + a.batch) * a.hkv;
  const double longest = (double)a.most_kv * 64 / p.unit + p.cost + 2 + slope * ((double)p.max_rows / p.tile_rows + 2);
  a.shift = 0;
  while (a.shift < 30 && tiles * (std::ldexp(longest, -a.shift) + 1) >= 1073741824.0) ++a.shift;
  if (tiles * (std::ldexp(longest, -a.shift) + 1) >= 1073741824.0)
    return fail(TQ_ERR_UNSUPPORTED, "batch x heads x rows: too many tiles for one launch");
  a.slope = (int)slope >> a.shift;
  tq::AttnMaps m = {};
  e = tq::attn_tensor_map(kv, false, p.unit, &m.k);
  if (e == cudaSuccess) e = tq::attn_tensor_map(kv, true, p.unit, &m.v);
  // Queries by TMA: a tile's 128 rows are whole queries where the group's size divides 128, with strides that TMA takes.
  // At head_dim 64 the softmax threads' own loads are faster (8 ragged prompts 38.2 against 41.2 us); at 128 and 256
  // TMA is (long cross attention 257 against 268 us, a mixed batch 69 against 75 us).
  auto fits = [](int64_t n, int64_t stride) { return n <= 1 || (stride > 0 && stride < (int64_t)1 << 38); };
  if (p.tc && kv.head_dim > 64 && 128 % a.G == 0 && fits(a.hq, a.q_head) && fits(a.n_rows, a.q_row)) {
    a.q_tma = 1;
    if (e == cudaSuccess) e = tq::query_tensor_map(*q, kv.head_dim, kv.dtype, a.G, &m.q);
  }
  if (e == cudaSuccess)
    e = p.tc ? tq::launch_attn_tc(a, m, p, kv.head_dim, kv.dtype, (cudaStream_t)stream)
             : tq::launch_attn_rows(a, m, p, kv.head_dim, kv.dtype, (cudaStream_t)stream);
  return done(e, "attention launch");
}

}  // namespace

extern "C" {

tq_status tq_blocks_release(int32_t* d_table, int max_seqs, int max_pages, int64_t table_stride, int32_t* d_free,
                            int n_blocks, int32_t* d_n_free, const int32_t* d_seq_ids, const int32_t* d_keep,
                            int batch, uint32_t* d_status, tq_stream_t stream) {
  const tq::NvtxRange nvtx_range("tq_blocks_release");
  const tq_status st = check_map(d_table, max_seqs, max_pages, table_stride, d_free, n_blocks, d_n_free, d_seq_ids, batch);
  if (st != TQ_OK) return st;
  if (!batch) return tq::set_error(TQ_OK, "");
  tq::BlockMap m = {};
  m.table = d_table;
  m.stride = table_stride;
  m.free = d_free;
  m.n_free = d_n_free;
  m.ids = d_seq_ids;
  m.lens = d_keep;
  m.status = d_status;
  m.max_seqs = max_seqs;
  m.max_pages = max_pages;
  m.n_blocks = n_blocks;
  m.batch = batch;
  return done(tq::launch_blocks_release(m, (cudaStream_t)stream), "tq_blocks_release");
}

tq_status tq_blocks_map(int32_t* d_table, int max_seqs, int max_pages, int64_t table_stride, const int32_t* d_free,
                        int n_blocks, int32_t* d_n_free, const int32_t* d_seq_ids, const int32_t* d_lens,
                        const int32_t* d_n_new, int batch, int32_t* d_starts, int32_t* d_totals, int32_t* d_slots,
                        int max_tokens, uint32_t* d_status, tq_stream_t stream) {
  const tq::NvtxRange nvtx_range("tq_blocks_map");
  const tq_status st = check_map(d_table, max_seqs, max_pages, table_stride, d_free, n_blocks, d_n_free, d_seq_ids, batch);
  if (st != TQ_OK) return st;
  if (!d_starts || (batch > 0 && (!d_lens || !d_n_new || !d_totals)) || (max_tokens > 0 && !d_slots))
    return fail(TQ_ERR_INVALID_ARG, "NULL array");
  if (max_tokens < 0 || max_tokens > (1 << 30)) return fail(TQ_ERR_INVALID_ARG, "max_tokens %d: 0 to 2^30", max_tokens);
  tq::BlockMap m = {};
  m.table = d_table;
  m.stride = table_stride;
  m.free = const_cast<int32_t*>(d_free);
  m.n_free = d_n_free;
  m.ids = d_seq_ids;
  m.lens = d_lens;
  m.n_new = d_n_new;
  m.starts = d_starts;
  m.totals = d_totals;
  m.slots = d_slots;
  m.status = d_status;
  m.max_seqs = max_seqs;
  m.max_pages = max_pages;
  m.n_blocks = n_blocks;
  m.batch = batch;
  m.max_tokens = max_tokens;
  return done(tq::launch_blocks_map(m, (cudaStream_t)stream), "tq_blocks_map");
}

tq_status tq_paged_append(const tq_kv* pool, const void* k, const void* v, tq_dtype dt, const int64_t* k_strides,
                          const int64_t* v_strides, const int32_t* d_slots, int n_tokens, uint32_t* d_status,
                          tq_stream_t stream) {
  const tq::NvtxRange nvtx_range("tq_paged_append");
  const tq_status st = check_kv(pool, false);
  if (st != TQ_OK) return st;
  if (pool->tokens != tq::kPage || pool->outer < 1 || pool->outer > (1 << 24) - 1)
    return fail(TQ_ERR_INVALID_ARG, "a pool has 1 to 2^24 - 1 blocks of 128 tokens (got %d of %d)", pool->outer, pool->tokens);
  if (dt != TQ_BF16 && dt != TQ_F16 && dt != TQ_F32) return fail(TQ_ERR_INVALID_ARG, "dtype %d", (int)dt);
  if (n_tokens < 0) return fail(TQ_ERR_INVALID_ARG, "n_tokens %d < 0", n_tokens);
  if (!n_tokens) return tq::set_error(TQ_OK, "");
  if (!k || !v || !k_strides || !v_strides || !d_slots) return fail(TQ_ERR_INVALID_ARG, "NULL array");
  const size_t esz = dt == TQ_F32 ? 4 : 2;
  if (!aligned(k, esz) || !aligned(v, esz) || !aligned(pool->k, 2) || !aligned(pool->v, 2))
    return fail(TQ_ERR_INVALID_ARG, "an address is not a multiple of its element's size");
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return done(e, "device");
  return done(tq::launch_paged_append(*pool, k, v, (int)dt, k_strides, v_strides, d_slots, n_tokens, d_status, sms,
                                      (cudaStream_t)stream),
              "tq_paged_append");
}

size_t tq_attention_workspace_bytes(const tq_queries* q, const tq_kv* kv) {
  int sms = 0;
  if (check_kv(kv, false) != TQ_OK || !q || q->batch < 1 || q->n_rows < 1 || q->max_q < 0 || q->n_q_heads < 1 ||
      q->n_q_heads % kv->n_kv_heads || sm_count(&sms) != cudaSuccess)
    return 0;
  return plan_of(*q, *kv, sms).bytes;
}

tq_status tq_paged_attention(const tq_queries* q, const tq_kv* kv, const int32_t* d_table, int max_seqs,
                             int max_pages, int64_t table_stride, const int32_t* d_seq_ids, const int32_t* d_kv_lens,
                             int causal, void* d_workspace, size_t workspace_bytes, uint32_t* d_status,
                             tq_stream_t stream) {
  const tq::NvtxRange nvtx_range("tq_paged_attention");
  tq_status st = check_kv(kv, true);
  if (st == TQ_OK) st = check_queries(q, kv);
  if (st != TQ_OK) return st;
  if (kv->tokens != tq::kPage || kv->outer < 1 || kv->outer > (1 << 24) - 1)
    return fail(TQ_ERR_INVALID_ARG, "a pool has 1 to 2^24 - 1 blocks of 128 tokens (got %d of %d)", kv->outer, kv->tokens);
  if (max_seqs < 1 || max_pages < 1 || max_pages > (1 << 20) || table_stride < max_pages)
    return fail(TQ_ERR_INVALID_ARG, "max_seqs %d, max_pages %d (at most 2^20), table_stride %lld", max_seqs, max_pages,
                (long long)table_stride);
  if (causal != 0 && causal != 1) return fail(TQ_ERR_INVALID_ARG, "causal %d: 0 or 1", causal);
  if (q->batch && q->n_rows && (!d_table || !d_kv_lens)) return fail(TQ_ERR_INVALID_ARG, "d_table or d_kv_lens is NULL");
  if (!d_seq_ids && q->batch > max_seqs) return fail(TQ_ERR_INVALID_ARG, "batch %d above max_seqs %d", q->batch, max_seqs);
  tq::AttnArgs a = {};
  a.mode = tq::kKvPaged;
  a.causal = causal;
  a.kv_lens = d_kv_lens;
  a.seq_ids = d_seq_ids;
  a.table = d_table;
  a.table_stride = table_stride;
  a.max_seqs = max_seqs;
  a.most_kv = max_pages * tq::kPage;
  return attend(q, kv, a, d_workspace, workspace_bytes, d_status, stream);
}

tq_status tq_cross_attention(const tq_queries* q, const tq_kv* kv, const int32_t* d_kv_starts,
                             const int32_t* d_kv_lens, void* d_workspace, size_t workspace_bytes, uint32_t* d_status,
                             tq_stream_t stream) {
  const tq::NvtxRange nvtx_range("tq_cross_attention");
  tq_status st = check_kv(kv, true);
  if (st == TQ_OK) st = check_queries(q, kv);
  if (st != TQ_OK) return st;
  if ((d_kv_starts != nullptr) == (d_kv_lens != nullptr) && q->batch && q->n_rows)
    return fail(TQ_ERR_INVALID_ARG, "d_kv_starts (packed states) or d_kv_lens (padded states), one of the two");
  if (d_kv_starts && kv->outer != 1) return fail(TQ_ERR_INVALID_ARG, "packed states have outer 1 (got %d)", kv->outer);
  if (d_kv_lens && kv->outer < q->batch) return fail(TQ_ERR_INVALID_ARG, "outer %d below batch %d", kv->outer, q->batch);
  tq::AttnArgs a = {};
  a.mode = d_kv_starts ? tq::kKvPacked : tq::kKvPadded;
  a.kv_lens = d_kv_lens;
  a.kv_starts = d_kv_starts;
  a.max_seqs = kv->outer;
  a.most_kv = kv->tokens;  // packed: the most that one request can have
  return attend(q, kv, a, d_workspace, workspace_bytes, d_status, stream);
}

}  // extern "C"
