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

// Two results in the cache's type. A result is an average of values, so a finite one past f16's largest number is there
// by the rounding of weights alone (up to 2^-11 of it; the next number is already infinite): it is that number.
template <bool BF16>
__device__ __forceinline__ uint32_t result2(float lo, float hi) {
  if constexpr (!BF16) {
    constexpr float kMost = 65504.f;
    if (fabsf(lo) > kMost && fabsf(lo) < INFINITY) lo = copysignf(kMost, lo);
    if (fabsf(hi) > kMost && fabsf(hi) < INFINITY) hi = copysignf(kMost, hi);
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
cudaError_t launch_attn_rows(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, int dtype, cudaStream_t s);
cudaError_t launch_attn_tc(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, int dtype, cudaStream_t s);

}  // namespace tq
