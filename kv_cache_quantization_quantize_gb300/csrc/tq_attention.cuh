// Attention of new tokens over an exact cache or an encoder's states: arguments, and what both kernels share.
#pragma once

#include <cuda.h>

#include "tq_device.cuh"

namespace tq {

constexpr int kMaxAttnSplits = 128;

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
  float* part;               // partials of the splits (see part_slot)
  float scale_log2;          // softmax scale * log2(e)
  int n_rows, batch, hq, hkv, G;
  FastDiv div_g;             // by G
  int max_seqs, max_pages, outer, tokens;
  int mode, causal;
  int n_splits, max_rows;    // max_rows: rows (query, head of the group) of a request and KV head at most
  int tiles;                 // rows kernel: tiles of every request
};

// One request as its CTA sees it. Bad arrays give an empty request and status bits.
struct Request {
  int q0, n_q, kv;  // first row, queries, tokens to attend to
  int row, base;    // paged: table row; padded: outer index; packed: base = first token
};

__device__ __forceinline__ Request find_request(const AttnArgs& a, int b, uint32_t& err) {
  Request r;
  r.q0 = a.q_starts[b];
  const int q1 = a.q_starts[b + 1];
  r.n_q = q1 - r.q0;
  if (r.q0 < 0 || q1 < r.q0 || q1 > a.n_rows) {
    err |= TQ_DEV_ERR_LENGTH;
    r.q0 = r.n_q = 0;
  }
  r.row = b;
  r.base = 0;
  if (a.mode == kKvPacked) {
    r.base = a.kv_starts[b];
    const int k1 = a.kv_starts[b + 1];
    r.kv = k1 - r.base;
    r.row = 0;
    if (r.base < 0 || k1 < r.base || k1 > a.tokens) {
      err |= TQ_DEV_ERR_LENGTH;
      r.kv = 0;
    }
  } else {
    r.kv = a.kv_lens[b];
    const int64_t most = a.mode == kKvPaged ? (int64_t)a.max_pages * kPage : a.tokens;
    if (r.kv < 0 || r.kv > most) {
      err |= TQ_DEV_ERR_LENGTH;
      r.kv = 0;
    }
    if (a.mode == kKvPaged) {
      if (a.seq_ids) r.row = a.seq_ids[b];
      if (r.row < 0 || r.row >= a.max_seqs) {
        err |= TQ_DEV_ERR_SEQ_ID;
        r.row = 0;
        r.kv = 0;
      }
    }
  }
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
  return last < 0 ? 0 : seen(a, r, last / a.G);
}

// Splits of a range of `units`: split s takes units [s * per, min(units, (s + 1) * per)).
__device__ __forceinline__ int units_per_split(int units, int n_splits) { return (units + n_splits - 1) / n_splits; }

// Partial of (row of q, query head) and split s: {m, l} and D floats of the weighted sum; weights are
// exp2(score * scale_log2 - m) and l their sum. All {m, l} come first.
__device__ __forceinline__ size_t part_slot(const AttnArgs& a, int row, int head, int s) {
  return ((size_t)row * a.hq + head) * a.n_splits + s;
}
__device__ __forceinline__ float2* part_ml(const AttnArgs& a) { return reinterpret_cast<float2*>(a.part); }
__device__ __forceinline__ float* part_o(const AttnArgs& a) {
  // n_rows * hq * n_splits pairs, rounded up to 16 bytes
  return a.part + (((size_t)a.n_rows * a.hq * a.n_splits * 2 + 3) & ~(size_t)3);
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
  CUtensorMap k, v;
};
// Tensor map of K or V for boxes of 64 channels x box_tokens tokens of one head, 128-byte swizzle: dimensions
// {head_dim, tokens, heads, outer}.
cudaError_t attn_tensor_map(const tq_kv& kv, bool values, int box_tokens, CUtensorMap* m);
// One launch plan: which kernel, its tiles and splits, and the bytes of partials it needs.
struct AttnPlan {
  int unit;          // tokens of a unit: splits take whole units
  int tile_rows;     // rows kernel: rows (query, head of the group) of a tile
  int n_splits;      // rows kernel
  int64_t max_rows;  // rows (query, head of the group) of a request and KV head at most
  int64_t tiles;     // rows kernel: tiles of one KV head over all requests
  bool tc;           // tensor-core kernel
  int ctas;          // its CTAs
  size_t bytes;
};
// Tensor-core kernel (tq_attention_tc.cu): its workspace, its unit of tokens, and the launch.
size_t attn_tc_bytes(int d, int ctas);
int attn_tc_unit(int d);
cudaError_t launch_attn_tc(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, int dtype, cudaStream_t s);
AttnPlan attn_plan(const tq_queries& q, const tq_kv& kv, int64_t max_tokens, int sms);
cudaError_t launch_attention(const AttnArgs& a, const tq_kv& kv, const AttnPlan& p, cudaStream_t s);

}  // namespace tq
