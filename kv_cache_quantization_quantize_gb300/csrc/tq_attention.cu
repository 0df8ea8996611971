// Attention of few new tokens per request (single tokens, drafts) over an exact cache or an encoder's states, and
// the join of split sequences. See tq_paged_attention and tq_cross_attention in tq.h for the operation.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "tq_attention.cuh"

namespace tq {
namespace {

// =============================================================================================
// k_attn_rows: one CTA takes a tile of up to 16 MT rows (query, head of the group) of one request and KV head, and
// one split of its tokens. Every K and V byte is used by all rows of the tile, and is read once from DRAM, which
// bounds the kernel. A producer warp keeps STAGES units of 64 tokens of K and V in flight with TMA; each of four
// consumer warps takes 16 tokens of a unit, with softmax statistics and sums of its own, so that nothing in the
// loop waits for another warp; the warps' sums are joined once at the end. Scores and sums run on mma.sync
// m16n8k16: at 16 rows the tensor pipe has a few percent of its work, and its register operands need no copies.
// =============================================================================================
constexpr int kUnit = 64;
constexpr int kRowsThreads = 160;  // four consumer warps, one producer warp

template <int D>
struct RowsShape {
  static constexpr int kTile = kUnit * D * 2;                  // bytes of K or V of one unit
  static constexpr int kStages = D == 64 ? 6 : 3;              // 96 KB (192 KB at head_dim 256) in flight
  static constexpr int kCtas = D == 256 ? 1 : 2;               // CTAs per SM
  static constexpr int smem(int rows) { return 1024 + kStages * 2 * kTile + rows * D * 2 + 1280; }
};

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Byte offset of 16-byte chunk `chunk` of row `row` in a tile of `rows` rows kept as 64-channel blocks of
// 128-byte rows in the 128-byte swizzle (as TMA writes it).
__device__ __forceinline__ uint32_t sw_off(int rows, int row, int chunk) {
  return (uint32_t)(((chunk >> 3) * rows + row) * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

template <int D, int MT, bool BF16>
__global__ void __launch_bounds__(kRowsThreads, RowsShape<D>::kCtas)
    k_attn_rows(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v) {
  constexpr int R = 16 * MT, ST = RowsShape<D>::kStages, KS = D / 16;
  constexpr uint32_t kTile = RowsShape<D>::kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sq = smem + ST * 2 * kTile;
  uint64_t* full = reinterpret_cast<uint64_t*>(sq + R * D * 2);
  uint64_t* empty = full + ST;
  float2* ml = reinterpret_cast<float2*>(empty + ST);  // [4][R] (16-byte aligned: 2 ST barriers)
  __shared__ int gave_up;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    gave_up = 0;
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  pdl_wait();
  if (a.n_splits > 1) pdl_launch();  // the join may be scheduled; it waits for this kernel's end
  uint32_t err = 0;
  int x = blockIdx.x;
  const int split = x % a.n_splits;
  x /= a.n_splits;
  const int h = x % a.hkv, b = x / a.hkv / a.tiles, tile = x / a.hkv % a.tiles;
  const Request r = find_request(a, b, err);
  if (r.n_q * (int64_t)a.G > a.max_rows) err |= TQ_DEV_ERR_SPLITS;
  const int rows = err & TQ_DEV_ERR_SPLITS ? 0 : r.n_q * a.G;
  const int f0 = tile * R;
  const int kv = tile_kv(a, r, tile, R);
  const int units = (kv + kUnit - 1) / kUnit, per = units_per_split(units, a.n_splits);
  const int u0 = split * per, u1 = min(units, u0 + per);
  const bool direct = units <= per;  // one split has it all
  if (threadIdx.x == 0 && err && a.status) atomicOr(a.status, err);
  if (f0 >= rows || (u0 >= u1 && split > 0)) return;

  // queries into shared memory; rows past the last are zero
  for (int i = threadIdx.x; i < R * (D / 8); i += kRowsThreads) {
    const int row = i / (D / 8), c = i % (D / 8), f = f0 + row;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (f < rows) {
      const int qi = f / a.G, g = f - qi * a.G;
      v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (int64_t)(r.q0 + qi) * a.q_row +
                                          (int64_t)(h * a.G + g) * a.q_head + c * 8);
    }
    *reinterpret_cast<uint4*>(sq + sw_off(R, row, c)) = v;
  }
  __syncthreads();

  if (warp == 4) {
    // ---- producer ----
    int2 place = make_int2(0, 0);
    bool ok = true;
    int issued = 0;
    for (int u = u0; u < u1; ++u) {
      const int k = u - u0, st = k % ST;
      if ((k & 31) == 0 && u + lane < u1) {
        place = page_place(a, r, (u + lane) >> 1, err);
        place.y += ((u + lane) & 1) * kUnit;
      }
      const int w = __shfl_sync(0xffffffffu, place.x, k & 31), y = __shfl_sync(0xffffffffu, place.y, k & 31);
      if (lane == 0) {
        if (k >= ST) ok = mbar_wait(&empty[st], ((k / ST) - 1) & 1);
        if (ok) {
          uint8_t* dst = smem + st * 2 * kTile;
          mbar_expect_tx(&full[st], 2 * kTile);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            tma_load_4d(dst + c * (kUnit * 128), &map_k, c * 64, y, h, w, &full[st]);
            tma_load_4d(dst + kTile + c * (kUnit * 128), &map_v, c * 64, y, h, w, &full[st]);
          }
          issued = k + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
    }
    if (lane == 0) {
      // leave only when every copy has landed (they have, unless a wait gave up)
      bool landed = ok;
      for (int k = max(0, issued - ST); k < issued; ++k) landed &= mbar_wait(&full[k % ST], (k / ST) & 1);
      if (!landed) {
        err |= TQ_DEV_ERR_TIMEOUT;
        atomicExch(&gave_up, 1);
      }
    }
    if (err && a.status) atomicOr(a.status, err);
    __syncthreads();
    return;
  }

  // ---- consumers ----
  const int g = lane >> 2, c2 = (lane & 3) * 2, mi = lane >> 3, ri = lane & 7;
  const uint32_t base = smem_u32(smem), qbase = smem_u32(sq);
  float o[MT][D / 8][4];
  float m[MT][2], l[MT][2];
  int lim[MT][2];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[t][e] = -INFINITY;
      l[t][e] = 0.f;
      const int f = f0 + t * 16 + g + e * 8;
      lim[t][e] = f < rows ? seen(a, r, f / a.G) : 0;
    }
  }
  constexpr bool kHoldQ = D * MT <= 128;  // the query fragments stay in registers
  uint32_t aq[kHoldQ ? MT : 1][kHoldQ ? KS : 1][4];
  if constexpr (kHoldQ) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) ldsm4(aq[t][ks], qbase + sw_off(R, t * 16 + (mi & 1) * 8 + ri, ks * 2 + (mi >> 1)));
  }
  bool ok = true;
  for (int u = u0; u < u1; ++u) {
    const int k = u - u0, st = k % ST;
    ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (k / ST) & 1));
    if (!ok) break;
    const int t0 = u * kUnit + warp * 16;
    if (t0 < kv) {
      const uint32_t kt = base + st * 2 * kTile, vt = kt + kTile;
      float s[MT][2][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < 2; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t bk[4];
        ldsm4(bk, kt + sw_off(kUnit, warp * 16 + (mi >> 1) * 8 + ri, ks * 2 + (mi & 1)));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          uint32_t af[4];
          if constexpr (kHoldQ) {
#pragma unroll
            for (int i = 0; i < 4; ++i) af[i] = aq[t][ks][i];
          } else {
            ldsm4(af, qbase + sw_off(R, t * 16 + (mi & 1) * 8 + ri, ks * 2 + (mi >> 1)));
          }
          mma16816<BF16>(s[t][0], af, bk[0], bk[1]);
          mma16816<BF16>(s[t][1], af, bk[2], bk[3]);
        }
      }
      // masked scores are selected away, not added to: what stands behind a sequence can be NaN
      uint32_t p[MT][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = t0 + n * 8 + c2 + (e & 1);
            s[t][n][e] = tok < lim[t][e >> 1] ? s[t][n][e] * a.scale_log2 : -INFINITY;
            top[e >> 1] = fmaxf(top[e >> 1], s[t][n][e]);
          }
        float alpha[2], mu[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
          top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
          const float mn = fmaxf(m[t][e], top[e]);
          mu[e] = mn == -INFINITY ? 0.f : mn;
          alpha[e] = exp2_fast(m[t][e] - mu[e]);
          m[t][e] = mn;
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][n][e] = exp2_fast(s[t][n][e] - mu[e >> 1]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          l[t][e] = l[t][e] * alpha[e] + (s[t][0][2 * e] + s[t][0][2 * e + 1] + s[t][1][2 * e] + s[t][1][2 * e + 1]);
        p[t][0] = pack2<BF16>(s[t][0][0], s[t][0][1]);
        p[t][1] = pack2<BF16>(s[t][0][2], s[t][0][3]);
        p[t][2] = pack2<BF16>(s[t][1][0], s[t][1][1]);
        p[t][3] = pack2<BF16>(s[t][1][2], s[t][1][3]);
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[t][i][0] *= alpha[0];
            o[t][i][1] *= alpha[0];
            o[t][i][2] *= alpha[1];
            o[t][i][3] *= alpha[1];
          }
        }
      }
      // a chunk that the sequence ends in: V rows behind it are zeroed (0 x NaN is NaN)
      uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
      if (t0 + 16 > kv) {
        const int n0 = kv - (t0 + c2), n1 = n0 - 8;
        keep0 = n0 >= 2 ? 0xffffffffu : n0 == 1 ? 0x0000ffffu : 0u;
        keep1 = n1 >= 2 ? 0xffffffffu : n1 == 1 ? 0x0000ffffu : 0u;
      }
#pragma unroll
      for (int np = 0; np < D / 16; ++np) {
        uint32_t bv[4];
        ldsm4t(bv, vt + sw_off(kUnit, warp * 16 + (mi & 1) * 8 + ri, np * 2 + (mi >> 1)));
        bv[0] &= keep0;
        bv[1] &= keep1;
        bv[2] &= keep0;
        bv[3] &= keep1;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          mma16816<BF16>(o[t][2 * np], p[t], bv[0], bv[1]);
          mma16816<BF16>(o[t][2 * np + 1], p[t], bv[2], bv[3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
  if (!ok && lane == 0) {
    atomicExch(&gave_up, 1);
    if (a.status) atomicOr(a.status, TQ_DEV_ERR_TIMEOUT);
  }
  __syncthreads();
  if (*(volatile int*)&gave_up) return;

  // ---- join of the four warps, through the stages' memory ----
  constexpr int kPad = D + 4;
  float* so = reinterpret_cast<float*>(smem);  // [4][R][kPad]
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = l[t][e];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      const int row = warp * R + t * 16 + g + e * 8;
      if ((lane & 3) == 0) ml[row] = make_float2(m[t][e], v);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(so + row * kPad + i * 8 + c2) = make_float2(o[t][i][2 * e], o[t][i][2 * e + 1]);
    }
  named_barrier(1, 128);
  for (int i = threadIdx.x; i < R * (D / 4); i += 128) {
    const int row = i / (D / 4), c = (i % (D / 4)) * 4, f = f0 + row;
    if (f >= rows) continue;
    float2 w[4];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = ml[j * R + row];
      top = fmaxf(top, w[j].x);
    }
    const float mu = top == -INFINITY ? 0.f : top;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float wt = exp2_fast(w[j].x - mu);
      const float4 v = *reinterpret_cast<const float4*>(so + (j * R + row) * kPad + c);
      sum += wt * w[j].y;
      acc.x += wt * v.x;
      acc.y += wt * v.y;
      acc.z += wt * v.z;
      acc.w += wt * v.w;
    }
    const int qi = f / a.G, head = h * a.G + f - qi * a.G;
    if (direct) {
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      uint2 out;
      out.x = pack2<BF16>(acc.x * inv, acc.y * inv);
      out.y = pack2<BF16>(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (int64_t)(r.q0 + qi) * a.o_row +
                                (int64_t)head * a.o_head + c) = out;
    } else {
      const size_t slot = part_slot(a, r.q0 + qi, head, split);
      *reinterpret_cast<float4*>(part_o(a) + slot * D + c) = acc;
      if (c == 0) part_ml(a)[slot] = make_float2(top, sum);
    }
  }
}

// =============================================================================================
// k_attn_join: o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the splits of one row. One CTA per row of a tile
// (`rows` of each); its threads take D / 4 columns x 512 / D groups of splits.
// =============================================================================================
template <int D, bool BF16>
__global__ void __launch_bounds__(128)
    k_attn_join(const __grid_constant__ AttnArgs a, int tile_rows, int rows, int unit) {
  constexpr int kCols = D / 4, kGroups = 128 / kCols;
  __shared__ float2 sml[kMaxAttnSplits];
  __shared__ float4 sacc[kGroups][kCols];
  pdl_wait();
  int x = blockIdx.x;
  const int in_tile = x % rows;
  x /= rows;
  const int h = x % a.hkv;
  const int b = x / a.hkv / a.tiles, tile = x / a.hkv % a.tiles;
  uint32_t err = 0;
  const Request r = find_request(a, b, err);
  const int f = tile * tile_rows + in_tile;
  if (f >= r.n_q * (int64_t)a.G || r.n_q * (int64_t)a.G > a.max_rows) return;
  const int row = r.q0 + f / a.G, head = h * a.G + f % a.G;
  const int kv = tile_kv(a, r, tile, tile_rows);
  const int units = (kv + unit - 1) / unit, per = units_per_split(units, a.n_splits);
  if (units <= per) return;  // its kernel has written the result
  const int live = (units + per - 1) / per;
  const size_t slot = part_slot(a, row, head, 0);
  for (int s = threadIdx.x; s < live; s += 128) sml[s] = part_ml(a)[slot + s];
  __syncthreads();
  float top = -INFINITY;
  for (int s = 0; s < live; ++s) top = fmaxf(top, sml[s].x);
  const float mu = top == -INFINITY ? 0.f : top;
  const int c = threadIdx.x % kCols, grp = threadIdx.x / kCols;
  const float4* po = reinterpret_cast<const float4*>(part_o(a) + slot * D) + c;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int s = grp; s < live; s += kGroups) {
    const float w = exp2_fast(sml[s].x - mu);
    const float4 v = po[(size_t)s * kCols];
    acc.x += w * v.x;
    acc.y += w * v.y;
    acc.z += w * v.z;
    acc.w += w * v.w;
  }
  for (int s = 0; s < live; ++s) sum += exp2_fast(sml[s].x - mu) * sml[s].y;
  sacc[grp][c] = acc;
  __syncthreads();
  if (grp > 0) return;
#pragma unroll
  for (int i = 1; i < kGroups; ++i) {
    acc.x += sacc[i][c].x;
    acc.y += sacc[i][c].y;
    acc.z += sacc[i][c].z;
    acc.w += sacc[i][c].w;
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  uint2 out;
  out.x = pack2<BF16>(acc.x * inv, acc.y * inv);
  out.y = pack2<BF16>(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (int64_t)row * a.o_row + (int64_t)head * a.o_head + c * 4) =
      out;
}

template <int D, int MT, bool BF16>
cudaError_t launch_rows_as(const AttnArgs& a, const AttnMaps& m, cudaStream_t s) {
  constexpr int R = 16 * MT;
  constexpr int smem = RowsShape<D>::smem(R);
  cudaError_t e = cudaFuncSetAttribute(k_attn_rows<D, MT, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_attn_rows<D, MT, BF16>, dim3((unsigned)(a.batch * a.tiles) * a.hkv * a.n_splits),
                    dim3(kRowsThreads), smem, s, a, m.k, m.v);
}

template <bool BF16>
cudaError_t launch_rows(const AttnArgs& a, const AttnMaps& m, int d, int tile_rows, cudaStream_t s) {
  if (d == 64) return tile_rows == 16 ? launch_rows_as<64, 1, BF16>(a, m, s) : launch_rows_as<64, 2, BF16>(a, m, s);
  if (d == 128) return tile_rows == 16 ? launch_rows_as<128, 1, BF16>(a, m, s) : launch_rows_as<128, 2, BF16>(a, m, s);
  return launch_rows_as<256, 1, BF16>(a, m, s);
}

template <int D>
cudaError_t launch_join(const AttnArgs& a, const AttnPlan& p, int dtype, cudaStream_t s) {
  const int rows = (int)std::min<int64_t>(p.tile_rows, p.max_rows);
  const dim3 grid((unsigned)(p.tiles * a.hkv * rows));
  return dtype == TQ_BF16 ? launch_pdl(k_attn_join<D, true>, grid, dim3(128), 0, s, a, p.tile_rows, rows, p.unit)
                          : launch_pdl(k_attn_join<D, false>, grid, dim3(128), 0, s, a, p.tile_rows, rows, p.unit);
}

}  // namespace

cudaError_t attn_tensor_map(const tq_kv& kv, bool values, int box_tokens, CUtensorMap* m) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)
                                                                : nullptr;
  }();
  if (!encode) return cudaErrorNotSupported;
  const int64_t* st = values ? kv.v_strides : kv.k_strides;
  void* base = values ? kv.v : kv.k;
  const cuuint64_t d = (cuuint64_t)kv.head_dim;
  // an empty dimension is given as one (no request has tokens there), a stride that is never taken as any valid one
  const cuuint64_t tokens = (cuuint64_t)std::max(kv.tokens, 1), outer = (cuuint64_t)std::max(kv.outer, 1);
  const cuuint64_t dims[4] = {d, tokens, (cuuint64_t)kv.n_kv_heads, outer};
  auto bytes = [&](cuuint64_t n, int64_t stride) { return n > 1 ? (cuuint64_t)stride * 2 : d * 2; };
  const cuuint64_t strides[3] = {bytes(tokens, st[1]), bytes(dims[2], st[2]), bytes(outer, st[0])};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_tokens, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = encode(m, kv.dtype == TQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                            base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

AttnPlan attn_plan(const tq_queries& q, const tq_kv& kv, int64_t max_tokens, int sms) {
  AttnPlan p;
  const int G = q.n_q_heads / kv.n_kv_heads, d = kv.head_dim;
  const int64_t rows = (int64_t)(q.max_q > 0 ? std::min(q.max_q, q.n_rows) : q.n_rows) * G;
  p.max_rows = rows;
  p.tc = rows > (d == 256 ? 16 : 32);
  p.ctas = std::min(sms, 1024);  // one per SM
  p.tiles = 1;
  p.tile_rows = p.n_splits = 1;
  if (p.tc) {
    p.unit = attn_tc_unit(d);
    p.bytes = attn_tc_bytes(d, p.ctas);
    return p;
  }
  p.tile_rows = rows <= 16 ? 16 : 32;
  p.unit = kUnit;
  p.tiles = q.batch;
  int64_t tokens = max_tokens;
  if (q.max_kv > 0) tokens = std::min<int64_t>(tokens, q.max_kv);
  const int64_t units = std::max<int64_t>(1, (tokens + p.unit - 1) / p.unit);
  const int64_t base = p.tiles * kv.n_kv_heads;
  const int64_t slots = (int64_t)sms * (d == 256 ? 1 : 2);
  // the fewest splits within 3 % of the least cost: waves of CTAs x (units of a CTA + about 4 for its start and end)
  const int most = (int)std::min<int64_t>(units, kMaxAttnSplits);
  auto cost = [&](int n) {
    const int64_t per = (units + n - 1) / n, live = (units + per - 1) / per;
    return (double)((base * live + slots - 1) / slots) * (double)(per + 4);
  };
  double best = cost(1);
  for (int n = 2; n <= most; ++n) best = std::min(best, cost(n));
  p.n_splits = 1;
  while (cost(p.n_splits) > 1.03 * best) ++p.n_splits;
  p.bytes = 0;
  if (p.n_splits > 1) {
    const size_t slots_n = (size_t)q.n_rows * q.n_q_heads * p.n_splits;
    p.bytes = ((slots_n * 2 + 3) & ~(size_t)3) * 4 + slots_n * kv.head_dim * 4;
  }
  return p;
}

cudaError_t launch_attention(const AttnArgs& a, const tq_kv& kv, const AttnPlan& p, cudaStream_t s) {
  AttnMaps m;
  cudaError_t e = attn_tensor_map(kv, false, p.unit, &m.k);
  if (e == cudaSuccess) e = attn_tensor_map(kv, true, p.unit, &m.v);
  if (e != cudaSuccess) return e;
  e = p.tc                  ? launch_attn_tc(a, m, p, kv.head_dim, kv.dtype, s)
      : kv.dtype == TQ_BF16 ? launch_rows<true>(a, m, kv.head_dim, p.tile_rows, s)
                          : launch_rows<false>(a, m, kv.head_dim, p.tile_rows, s);
  if (e != cudaSuccess || p.tc || p.n_splits == 1) return e;
  return kv.head_dim == 64    ? launch_join<64>(a, p, kv.dtype, s)
         : kv.head_dim == 128 ? launch_join<128>(a, p, kv.dtype, s)
                              : launch_join<256>(a, p, kv.dtype, s);
}

}  // namespace tq
