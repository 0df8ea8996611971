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

cudaError_t attn_tensor_map8(const tq_kv& kv, bool values, int channels, int box_tokens, bool swizzle, CUtensorMap* m) {
  const auto encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  const int64_t* st = values ? kv.v_strides : kv.k_strides;
  const cuuint64_t dims[4] = {(cuuint64_t)kv.head_dim, (cuuint64_t)kv.tokens, (cuuint64_t)kv.n_kv_heads, (cuuint64_t)kv.outer};
  auto bytes = [&](cuuint64_t n, int64_t stride) { return n > 1 ? (cuuint64_t)stride : dims[0]; };  // a stride that is never taken: any
  const cuuint64_t strides[3] = {bytes(dims[1], st[1]), bytes(dims[2], st[2]), bytes(dims[3], st[0])};
  const cuuint32_t box[4] = {(cuuint32_t)channels, (cuuint32_t)box_tokens, 1, 1}, estr[4] = {1, 1, 1, 1};
  // L2 fetches what a token's head has and not the next head's: 32 requests of 4096 to 8192 tokens of 8 heads of 128, heads
  // of a token together, 75.5 us against 87 with 256 bytes
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, values ? kv.v : kv.k, dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE,
                            !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : channels == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                            kv.head_dim == 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
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

// `scaled`: a pool of 8 bits.
tq_status check_kv(const tq_kv* kv, bool map, bool scaled = false) {
  if (!kv) return fail(TQ_ERR_INVALID_ARG, "kv is NULL");
  if (kv->head_dim != 64 && kv->head_dim != 128 && kv->head_dim != 256)
    return fail(TQ_ERR_UNSUPPORTED, "head_dim %d: supported 64, 128, 256", kv->head_dim);
  if (scaled && kv->dtype != TQ_E4M3) return fail(TQ_ERR_UNSUPPORTED, "cache type %d: with scales, e4m3", kv->dtype);
  if (!scaled && kv->dtype != TQ_BF16 && kv->dtype != TQ_F16) return fail(TQ_ERR_UNSUPPORTED, "cache type %d: bf16 or f16", kv->dtype);
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 65535 || kv->outer < 0 || kv->tokens < 0)
    return fail(TQ_ERR_INVALID_ARG, "n_kv_heads %d, outer %d, tokens %d", kv->n_kv_heads, kv->outer, kv->tokens);
  if (!kv->outer || !kv->tokens) return TQ_OK;  // no element
  if (!kv->k || !kv->v) return fail(TQ_ERR_INVALID_ARG, "k or v is NULL");
  if (!map) return TQ_OK;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return fail(TQ_ERR_INVALID_ARG, "k and v have to be 16-byte aligned");
  const int size[3] = {kv->outer, kv->tokens, kv->n_kv_heads};
  for (int i = 0; i < 3; ++i)
    for (const int64_t st : {kv->k_strides[i], kv->v_strides[i]})
      if (size[i] > 1 && (st < 1 || st % (scaled ? 16 : 8) || st >= (int64_t)1 << 38))
        return fail(TQ_ERR_INVALID_ARG, "stride %lld of k or v: a positive multiple of %d elements", (long long)st, scaled ? 16 : 8);
  return TQ_OK;
}

tq_status check_scales(const tq_scales* s, const tq_kv* kv) {
  if (!s || !s->k || !s->v || !aligned(s->k, 4) || !aligned(s->v, 4))
    return fail(TQ_ERR_INVALID_ARG, "scales of k and v: two arrays of floats");
  if (kv->outer > 1 && (s->k_block < kv->n_kv_heads || s->v_block < kv->n_kv_heads))
    return fail(TQ_ERR_INVALID_ARG, "scales: %lld and %lld entries from block to block for %d heads", (long long)s->k_block,
                (long long)s->v_block, kv->n_kv_heads);
  return TQ_OK;
}

tq_status check_pool(const tq_kv* kv) {
  if (kv->tokens != tq::kPage || kv->outer < 1 || kv->outer > (1 << 24) - 1)
    return fail(TQ_ERR_INVALID_ARG, "a pool has 1 to 2^24 - 1 blocks of 128 tokens (got %d of %d)", kv->outer, kv->tokens);
  return TQ_OK;
}

tq_status check_table(int max_seqs, int max_pages, int64_t stride) {
  if (max_seqs < 1 || max_pages < 1 || max_pages > (1 << 20) || stride < max_pages)
    return fail(TQ_ERR_INVALID_ARG, "max_seqs %d, max_pages %d (at most 2^20), table_stride %lld", max_seqs, max_pages,
                (long long)stride);
  return TQ_OK;
}

// rot as the kernels take it (NULL: none), for heads of head_dim channels.
tq_status check_rotary(const tq_rotary* rot, int head_dim, tq::Rotation* r) {
  *r = {};
  if (!rot) return TQ_OK;
  if (rot->rotary_dim < 8 || rot->rotary_dim % 8 || rot->rotary_dim > head_dim)
    return fail(TQ_ERR_UNSUPPORTED, "rotary_dim %d: a multiple of 8, at most head_dim %d", rot->rotary_dim, head_dim);
  if (rot->interleaved != 0 && rot->interleaved != 1) return fail(TQ_ERR_INVALID_ARG, "interleaved %d: 0 or 1", rot->interleaved);
  if (!std::isfinite(rot->factor)) return fail(TQ_ERR_INVALID_ARG, "factor is not finite");
  if (!rot->d_turns || !aligned(rot->d_turns, 8)) return fail(TQ_ERR_INVALID_ARG, "d_turns: 8-byte aligned device memory");
  r->turns = rot->d_turns;
  r->pairs = rot->rotary_dim / 2;
  r->interleaved = rot->interleaved;
  r->factor = rot->factor;
  return TQ_OK;
}

constexpr int kMostRows = 0x7fffff00;  // of rotations and rotated appends: the last CTA counts some rows past them in 32 bits

bool known_type(int dt) { return dt == TQ_BF16 || dt == TQ_F16 || dt == TQ_F32; }

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
// 83 against 63 us over 65536, and 28 against 22 us for 16 requests of 512. Over 8 bits 64 against 76 us for 16 requests of 8
// drafts over 4096 to 8192; there the rows kernel, in tiles of 32 rows, is also the faster one for little work, which its many
// small parts spread better: where the tensor cores' tiles would be few (kRowsEach rows for each SM; 32 heads on 8 of 128, 16 queries
// over 1000 tokens 12.5 against 18.8 us, over 16000 32.6 against 38.9; 16 heads on 4 of 256 12.3 against 26.9 and 30.2 against
// 43.9; but 8 requests of 128 34.8 against 19.5) and each CTA gets kUnitsEach units at most (120 queries over 4000 tokens, 13 units:
// 46.8 against 40.3). The rule counts padded rows, so near its edge it loses some: two prompts of 100 tokens, 32 heads on 8 of 128, 18.5 us
// so and 15.0 with the other kernel, 4 requests of 16 after 2000 27.4 and 24.7, one of 200 after 30 22.1 and 20.8; two
// of 64 after 1000 at 64 channels 5 %.
constexpr int kRowsEach = 32, kUnitsEach = 8;
tq::AttnPlan plan_of(const tq_queries& q, const tq_kv& kv, int sms) {
  tq::AttnPlan p;
  const int64_t rows = (int64_t)(q.max_q > 0 ? std::min(q.max_q, q.n_rows) : q.n_rows) * (q.n_q_heads / kv.n_kv_heads);
  const bool e4m3 = kv.dtype == TQ_E4M3;
  bool tc = rows > 32;
  if (tc && e4m3 && q.max_kv > 0) {
    auto tiles = [&](int of) { return (double)q.batch * kv.n_kv_heads * ((rows + of - 1) / of); };
    const tq::AttnShape few = tq::attn8_rows_shape(kv.head_dim, rows, sms);
    const int wide = tq::attn8_tc_shape(kv.head_dim, sms).tile_rows;
    tc = tiles(wide) * wide > kRowsEach * (double)sms || tiles(few.tile_rows) * (((int64_t)q.max_kv + few.unit - 1) / few.unit) > kUnitsEach * (double)few.ctas;
  }
  static_cast<tq::AttnShape&>(p) = tc ? (e4m3 ? tq::attn8_tc_shape(kv.head_dim, sms) : tq::attn_tc_shape(kv.head_dim, sms))
                                      : (e4m3 ? tq::attn8_rows_shape : tq::attn_rows_shape)(kv.head_dim, rows, sms);
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

// q_dtype: of queries and outputs; the cache's own, unless that has 8 bits.
tq_status attend(const tq_queries* q, int q_dtype, const tq_kv* kv_in, tq::AttnArgs& a, void* ws, size_t ws_bytes,
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
  if (kv.dtype == TQ_E4M3) {
    const int channels = p.tc ? kv.head_dim : std::min(kv.head_dim, 128);  // the rows kernel reads what TMA wrote, in the swizzle
    e = tq::attn_tensor_map8(kv, false, channels, p.unit, !p.tc, &m.k);
    if (e == cudaSuccess) e = tq::attn_tensor_map8(kv, true, channels, p.unit, !p.tc, &m.v);
    if (e == cudaSuccess)
      e = (p.tc ? tq::launch_attn8_tc : tq::launch_attn8_rows)(a, m, p, kv.head_dim, q_dtype, (cudaStream_t)stream);
    return done(e, "attention launch");
  }
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
  if (check_pool(pool) != TQ_OK) return TQ_ERR_INVALID_ARG;
  if (!known_type(dt)) return fail(TQ_ERR_INVALID_ARG, "dtype %d", (int)dt);
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

tq_status tq_rotate(const tq_rotary* rot, const void* x, void* out, tq_dtype dt, const int64_t* x_strides,
                    const int64_t* out_strides, const int32_t* d_positions, int n_tokens, int n_heads, int head_dim,
                    int inverse, tq_stream_t stream) {
  const tq::NvtxRange nvtx_range("tq_rotate");
  if (!rot) return fail(TQ_ERR_INVALID_ARG, "rot is NULL");
  if (head_dim < 8 || head_dim % 8 || head_dim > 1024)
    return fail(TQ_ERR_UNSUPPORTED, "head_dim %d: a multiple of 8, at most 1024", head_dim);
  tq::Rotation r;
  const tq_status st = check_rotary(rot, head_dim, &r);
  if (st != TQ_OK) return st;
  if (!known_type(dt)) return fail(TQ_ERR_INVALID_ARG, "dtype %d", (int)dt);
  if (inverse != 0 && inverse != 1) return fail(TQ_ERR_INVALID_ARG, "inverse %d: 0 or 1", inverse);
  if (n_tokens < 0 || n_heads < 0) return fail(TQ_ERR_INVALID_ARG, "n_tokens %d, n_heads %d: none below 0", n_tokens, n_heads);
  if (n_tokens > kMostRows || n_heads > 65535)
    return fail(TQ_ERR_UNSUPPORTED, "n_tokens %d, n_heads %d: at most %d and 65535", n_tokens, n_heads, kMostRows);
  if (!n_tokens || !n_heads) return tq::set_error(TQ_OK, "");
  if (!x || !out || !x_strides || !out_strides || !d_positions) return fail(TQ_ERR_INVALID_ARG, "NULL array");
  const size_t esz = dt == TQ_F32 ? 4 : 2;
  if (!aligned(x, esz) || !aligned(out, esz)) return fail(TQ_ERR_INVALID_ARG, "an address is not a multiple of its element's size");
  r.inverse = inverse;
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return done(e, "device");
  return done(tq::launch_rotate(r, x, out, (int)dt, x_strides, out_strides, d_positions, n_tokens, n_heads, head_dim, sms,
                                (cudaStream_t)stream),
              "tq_rotate");
}

tq_status tq_paged_extend(const tq_kv* pool, const tq_scales* scales, const tq_new_rows* rows, const tq_rotary* rot,
                          const int32_t* d_table, int max_seqs, int max_pages, int64_t table_stride,
                          const int32_t* d_seq_ids, const int32_t* d_starts, const int32_t* d_totals, int batch,
                          uint32_t* d_status, tq_stream_t stream) {
  const tq::NvtxRange nvtx_range("tq_paged_extend");
  tq_status st = check_kv(pool, scales != nullptr, scales != nullptr);
  if (st == TQ_OK) st = check_pool(pool);
  if (st == TQ_OK && scales) st = check_scales(scales, pool);
  tq::Rotation r;
  if (st == TQ_OK) st = check_rotary(rot, pool->head_dim, &r);
  if (st == TQ_OK) st = check_table(max_seqs, max_pages, table_stride);
  if (st != TQ_OK) return st;
  if (!rows) return fail(TQ_ERR_INVALID_ARG, "rows are NULL");
  if (!known_type(rows->dtype)) return fail(TQ_ERR_INVALID_ARG, "dtype %d", rows->dtype);
  if (rows->n_rows < 0 || batch < 0 || rows->n_q_heads < 0 || rows->n_q_heads > 65535)
    return fail(TQ_ERR_INVALID_ARG, "n_rows %d, batch %d, n_q_heads %d (at most 65535): none below 0", rows->n_rows, batch, rows->n_q_heads);
  if (batch > 65535) return fail(TQ_ERR_UNSUPPORTED, "batch %d: at most 65535", batch);
  if (rows->n_rows > kMostRows) return fail(TQ_ERR_UNSUPPORTED, "n_rows %d: at most %d", rows->n_rows, kMostRows);
  if (rows->q && !rot) return fail(TQ_ERR_INVALID_ARG, "q without rot: nothing to do");
  if (!batch || !rows->n_rows) return tq::set_error(TQ_OK, "");
  const bool queries = rows->q && rows->n_q_heads;
  if (!rows->k || !rows->v || (queries && !rows->q_out) || !d_table || !d_starts || !d_totals)
    return fail(TQ_ERR_INVALID_ARG, "NULL array");
  if (!d_seq_ids && batch > max_seqs) return fail(TQ_ERR_INVALID_ARG, "batch %d above max_seqs %d", batch, max_seqs);
  const size_t esz = rows->dtype == TQ_F32 ? 4 : 2;
  if (!aligned(rows->k, esz) || !aligned(rows->v, esz) || (queries && (!aligned(rows->q, esz) || !aligned(rows->q_out, esz))) ||
      !aligned(pool->k, 2) || !aligned(pool->v, 2))
    return fail(TQ_ERR_INVALID_ARG, "an address is not a multiple of its element's size");
  tq::StepMap m = {d_table, table_stride, d_seq_ids, d_starts, d_totals, max_seqs, max_pages, batch, rows->n_rows};
  tq_new_rows n = *rows;
  if (!queries) n.q = nullptr;
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return done(e, "device");
  return done(tq::launch_paged_extend(*pool, scales, n, r, m, d_status, sms, (cudaStream_t)stream), "tq_paged_extend");
}

size_t tq_attention_workspace_bytes(const tq_queries* q, const tq_kv* kv) {
  int sms = 0;
  if (!kv || check_kv(kv, false, kv->dtype == TQ_E4M3) != TQ_OK || !q || q->batch < 1 || q->n_rows < 1 || q->max_q < 0 || q->n_q_heads < 1 ||
      q->n_q_heads % kv->n_kv_heads || sm_count(&sms) != cudaSuccess)
    return 0;
  return plan_of(*q, *kv, sms).bytes;
}

// tq_paged_attention, and with scales tq_paged_attention8
static tq_status paged_attention(const tq_queries* q, int q_dtype, const tq_kv* kv, const tq_scales* scales, const int32_t* d_table,
                                 int max_seqs, int max_pages, int64_t table_stride, const int32_t* d_seq_ids,
                                 const int32_t* d_kv_lens, int causal, void* d_workspace, size_t workspace_bytes,
                                 uint32_t* d_status, tq_stream_t stream) {
  tq_status st = check_queries(q, kv);
  if (st != TQ_OK) return st;
  if (check_pool(kv) != TQ_OK || check_table(max_seqs, max_pages, table_stride) != TQ_OK) return TQ_ERR_INVALID_ARG;
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
  if (scales) {
    a.k_scale = scales->k;
    a.v_scale = scales->v;
    a.ks_block = scales->k_block;
    a.vs_block = scales->v_block;
  }
  return attend(q, q_dtype, kv, a, d_workspace, workspace_bytes, d_status, stream);
}

tq_status tq_paged_attention(const tq_queries* q, const tq_kv* kv, const int32_t* d_table, int max_seqs,
                             int max_pages, int64_t table_stride, const int32_t* d_seq_ids, const int32_t* d_kv_lens,
                             int causal, void* d_workspace, size_t workspace_bytes, uint32_t* d_status,
                             tq_stream_t stream) {
  const tq::NvtxRange nvtx_range("tq_paged_attention");
  const tq_status st = check_kv(kv, true);
  if (st != TQ_OK) return st;
  return paged_attention(q, kv->dtype, kv, nullptr, d_table, max_seqs, max_pages, table_stride, d_seq_ids, d_kv_lens, causal,
                         d_workspace, workspace_bytes, d_status, stream);
}

tq_status tq_paged_attention8(const tq_queries* q, tq_dtype q_dtype, const tq_kv* kv, const tq_scales* scales,
                              const int32_t* d_table, int max_seqs, int max_pages, int64_t table_stride,
                              const int32_t* d_seq_ids, const int32_t* d_kv_lens, int causal, void* d_workspace,
                              size_t workspace_bytes, uint32_t* d_status, tq_stream_t stream) {
  const tq::NvtxRange nvtx_range("tq_paged_attention8");
  tq_status st = check_kv(kv, true, true);
  if (st == TQ_OK) st = check_scales(scales, kv);
  if (st != TQ_OK) return st;
  if (q_dtype != TQ_BF16 && q_dtype != TQ_F16) return fail(TQ_ERR_UNSUPPORTED, "queries of type %d: bf16 or f16", (int)q_dtype);
  return paged_attention(q, q_dtype, kv, scales, d_table, max_seqs, max_pages, table_stride, d_seq_ids, d_kv_lens, causal,
                         d_workspace, workspace_bytes, d_status, stream);
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
  return attend(q, kv->dtype, kv, a, d_workspace, workspace_bytes, d_status, stream);
}

}  // extern "C"
