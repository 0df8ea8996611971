// Attention of new tokens over an exact cache or an encoder's states: arguments, and what both kernels share.
#pragma once

#include <cuda.h>

#include "tq_device.cuh"

namespace tq {

constexpr int kMaxAttnCtas = 1024;  // of a launch

enum KvMode { kKvPaged = 0, kKvPadded = 1, kKvPacked = 2 };

// x / d for 0 <= x < 2^31 and a d that does not change in a launch: (mulhi(x, m) + x) >> s (Granlund and Montgomery,
// Division by invariant integers using multiplication, 1994).
struct FastDiv {
  uint32_t m, s;
  void set(uint32_t d) {
    s = 0;
    while ((1ull << s) < d) ++s;
    m = (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ int operator()(int x) const { return (int)((__umulhi((uint32_t)x, m) + (uint32_t)x) >> s); }
};

struct AttnArgs {
  const void* q;
  void* out;
  int64_t q_row, q_head, o_row, o_head;  // strides in elements
  const int32_t* q_starts;
  const int32_t* kv_lens;    // paged, padded
  const int32_t* kv_starts;  // packed
  const int32_t* seq_ids;    // paged; NULL: row b
  const int32_t* table;      // paged
  int64_t table_stride;
  uint32_t* status;
  void* part;                // workspace (tq_attention_line.cuh)
  float scale_log2;          // softmax scale * log2(e)
  int n_rows, batch, hq, hkv, G;
  FastDiv div_g;             // by G
  int max_seqs, outer, tokens;   // max_seqs: padded: the outer size
  int most_kv;               // paged, padded: tokens of a request at most
  int q_tma;                 // tensor-core kernel: queries come by TMA (their map is valid)
  int slope, shift;          // cost that each tile of a causal request has over the one before, and the scale of costs
                             // (tq_attention_line.cuh)
  int mode, causal;
  const float *k_scale, *v_scale;  // a cache of 8 bits: entry (block, KV head) at block * ks_block + head
  int64_t ks_block, vs_block;
  int max_rows;              // rows (query, head of the group) of a request and KV head at most
};

// One request as its CTA sees it. Bad arrays give an empty request and status bits.
struct Request {
  int q0, n_q, kv;  // first row, queries, tokens to attend to
  int row, base;    // paged: table row; padded: outer index; packed: base = first token
};

__device__ __forceinline__ Request find_request(const AttnArgs& a, int b, uint32_t& err) {
  // the loads first, so that they overlap
  const bool packed = a.mode == kKvPacked;
  const int32_t* lens = packed ? a.kv_starts : a.kv_lens;
  const int q0 = a.q_starts[b], q1 = a.q_starts[b + 1], x = lens[b];
  const int y = packed ? a.kv_starts[b + 1] : a.seq_ids ? a.seq_ids[b] : b;
  const bool bad_q = q0 < 0 || q1 < q0 || q1 > a.n_rows;
  Request r;
  r.q0 = bad_q ? 0 : q0;
  r.n_q = bad_q ? 0 : q1 - q0;
  bool bad_kv, bad_id = false;
  if (packed) {
    bad_kv = x < 0 || y < x || y > a.tokens;
    r.kv = y - x;
    r.base = x;
    r.row = 0;
  } else {
    bad_kv = x < 0 || x > a.most_kv;
    bad_id = y < 0 || y >= a.max_seqs;
    r.kv = x;
    r.base = 0;
    r.row = bad_id ? 0 : y;
  }
  if (bad_kv || bad_id) r.kv = 0;
  err |= (bad_q || bad_kv ? TQ_DEV_ERR_LENGTH : 0u) | (bad_id ? TQ_DEV_ERR_SEQ_ID : 0u);
  return r;
}

// Tokens that query i of the request sees.
__device__ __forceinline__ int seen(const AttnArgs& a, const Request& r, int i) {
  return a.causal ? max(0, r.kv - r.n_q + i + 1) : r.kv;
}

// Where the block of tokens [128 page, 128 page + 128) of a request starts in the K and V tensors: outer index
// and token. A page without a block is past the last outer index, where copies read zeros.
__device__ __forceinline__ int2 page_place(const AttnArgs& a, const Request& r, int page, uint32_t& err) {
  if (a.mode == kKvPaged) {
    int blk = a.table[(int64_t)r.row * a.table_stride + page];
    if (blk < 0 || blk >= a.outer) {
      err |= TQ_DEV_ERR_BLOCK;
      blk = a.outer;
    }
    return make_int2(blk, 0);
  }
  return make_int2(r.row, r.base + page * kPage);
}

// The rows of a request and KV head are f = query * G + (head of the group); tiles take kTile consecutive ones.
// Tokens that any row of a tile sees.
__device__ __forceinline__ int tile_kv(const AttnArgs& a, const Request& r, int tile, int tile_rows) {
  const int last = min((tile + 1) * tile_rows, r.n_q * a.G) - 1;
  return last < 0 ? 0 : seen(a, r, a.div_g(last));
}

// The scales of a unit of tokens in a cache of 8 bits: of its keys; of its values their logarithm and inverse.
struct UnitScale {
  float k, log_v, inv_v;
};
__device__ __forceinline__ UnitScale unit_scale(const AttnArgs& a, int block, int head) {
  UnitScale r = {1.f, 0.f, 1.f};
  if (block < a.outer) {
    r.k = clamp_scale(a.k_scale[block * a.ks_block + head]);
    const float v = clamp_scale(a.v_scale[block * a.vs_block + head]);
    const uint32_t u = __float_as_uint(v);
    r.log_v = u & 0x7fffffu ? log2f(v) : (float)((int)(u >> 23) - 127);
    r.inv_v = 1.f / v;
  }
  return r;
}
// Two e4m3 numbers, which f16 holds exactly: the low half's and the high half's of a word.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(x));
  return r;
}
// The power of two that takes a bf16 row to f16 with its largest value in [2^7, 2^8), by the bits of that value (sign
// off): bf16 numbers stay exact down to 2^-25 of it. And its inverse.
__device__ __forceinline__ float to_f16_by(uint32_t top) { return __uint_as_float((261u - max(top >> 7, 8u)) << 23); }
__device__ __forceinline__ float to_f16_back(uint32_t top) { return __uint_as_float((max(top >> 7, 8u) - 7u) << 23); }
// Two bf16 values times `by`, in f16.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t x, float by) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(x & 0xffff0000u) * by), "f"(__uint_as_float(x << 16) * by));
  return r;
}

// 2^x as the special function unit gives it (relative error about 2^-22, 0 for -inf).
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats rounded to the cache's type, the first in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two results in the queries' type. A result is an average of values, so over a cache of f16 a finite one past f16's largest
// number is there by the rounding of weights alone (up to 2^-11 of it, and what the sums add; the next number is already
// infinite): up to 2^-8 past it is that number. A cache of 8 bits can hold more, and results behind that are infinite.
template <bool BF16>
__device__ __forceinline__ uint32_t result2(float lo, float hi) {
  if constexpr (!BF16) {
    constexpr float kMost = 65504.f, kNear = 65504.f * (1.f + 1.f / 256.f);
    if (fabsf(lo) > kMost && fabsf(lo) <= kNear) lo = copysignf(kMost, lo);
    if (fabsf(hi) > kMost && fabsf(hi) <= kNear) hi = copysignf(kMost, hi);
  }
  return pack2<BF16>(lo, hi);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// ---- launchers ----
struct AttnMaps {
  CUtensorMap k, v, q;  // q: with AttnArgs::q_tma
};
// Tensor map of K or V for boxes of 64 channels x box_tokens tokens of one head, 128-byte swizzle: dimensions
// {head_dim, tokens, heads, outer}.
cudaError_t attn_tensor_map(const tq_kv& kv, bool values, int box_tokens, CUtensorMap* m);
// Of a pool of 8 bits, for boxes of `channels` bytes x box_tokens tokens of one head: 128-byte swizzle (64-byte at head_dim
// 64) or none.
cudaError_t attn_tensor_map8(const tq_kv& kv, bool values, int channels, int box_tokens, bool swizzle, CUtensorMap* m);
// Tensor map of the queries for boxes of 64 channels x the G heads of a group x 128 / G queries: 128 rows of a tile.
cudaError_t query_tensor_map(const tq_queries& q, int head_dim, int dtype, int G, CUtensorMap* m);
// A kernel's tiles and launch: rows (query, head of the group) of a tile, tokens of a unit, CTAs at most, bytes of
// workspace per CTA; a tile's fixed cost and the least work of a CTA (tq_attention_line.cuh).
struct AttnShape {
  int tile_rows, unit, ctas;
  size_t cta_bytes;
  int cost, least;
};
struct AttnPlan : AttnShape {
  bool tc;           // tensor-core kernel (tq_attention_tc.cu), else the rows kernel (tq_attention_rows.cu)
  int64_t max_rows;  // rows of a request and KV head at most
  size_t bytes;      // of workspace
};
AttnShape attn_rows_shape(int d, int64_t rows, int sms);
AttnShape attn_tc_shape(int d, int sms);
AttnShape attn8_rows_shape(int d, int64_t rows, int sms);
AttnShape attn8_tc_shape(int d, int sms);
cudaError_t launch_attn_rows(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, int dtype, cudaStream_t s);
cudaError_t launch_attn_tc(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, int dtype, cudaStream_t s);
// Over a pool of 8 bits; dtype: of the queries.
cudaError_t launch_attn8_rows(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, int dtype, cudaStream_t s);
cudaError_t launch_attn8_tc(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, int dtype, cudaStream_t s);

}  // namespace tq
