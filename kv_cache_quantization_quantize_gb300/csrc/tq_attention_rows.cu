// Attention of few new tokens per request (single tokens, drafts) over an exact cache or an encoder's states.
#include "tq_attention_rows.cuh"

namespace tq {
namespace {

// =============================================================================================
// k_attn_rows: a CTA takes its part of the line (tq_attention_line.cuh) in tiles of up to 16 MT rows (query, head of
// the group) of one request and KV head. Every K and V byte is used by all rows of the tile and read once, which
// bounds the kernel: DRAM. A producer warp walks the parts and keeps a ring of K and V tiles in flight
// with TMA, over the ends of parts. Four consumer warps share each unit: for the scores each takes a quarter of its
// tokens, for the sums each takes D / 4 channels of all of them, with the weights handed over through shared memory. So no warp holds more
// than D / 4 channels of the sums and nothing has to be joined at the end; one barrier per unit hands over the weights
// and tells whether a maximum outgrew its range (kLazy), which is rare after a tile's first unit. Scores and sums run
// on mma.sync m16n8k16: at 16 or 32 rows the tensor pipe has a fifth of its time's work, and its register operands
// need no copies.
// Measured (GB300, 32 query heads on 8 KV heads, head_dim 128, bf16, with the join): 4 x 32768 tokens 86 us, 6.2 TB/s, 93 %
// of a measured copy (the kernel alone 84 us); one sequence of 131072 tokens 88 us; of 32768 30 to 34 us, of which about 4 us
// are the way to the first load, 4 us the join and 20 us the bytes. A unit takes 930 cycles of a CTA, its bytes 2900 of an
// SM's share of DRAM.
// =============================================================================================
template <int D, int MT>
struct RowsShape {
  static constexpr int R = 16 * MT;
  static constexpr int U = D == 64 ? 128 : 64;    // tokens of a unit: 16 KB of K and as much of V (32 at head_dim 256)
  static constexpr int kEntry = U * D * 2;        // bytes of K or V of one unit
  // Bytes in flight: 64 KB of each of two CTAs on an SM (head_dim 128), 48 KB of each of three or two (64), 128 KB
  // (256). More only queue up: with 5 and 6 entries at head_dim 128, 16 sequences of 4096 to 8192 tokens took 65.2 and
  // 67.2 us instead of 63.7. At head_dim 64 a third CTA hides the shorter units' latencies: 64 x 4096 tokens took 126 us
  // with two CTAs, 105 us with three.
  static constexpr int kCtas = D == 256 ? 1 : D == 64 && MT == 1 ? 3 : 2;  // CTAs per SM
  static constexpr int kEntries = D == 64 ? 3 : 4;
  static constexpr int kQRow = D * 2 + 16;  // bytes of a query row: 16 more than it has, so that ldmatrix meets no conflicts
  static constexpr int kQ = R * kQRow;
  static constexpr int kP = R * U * 2;  // weights of one unit
  static constexpr int kSmem = 1024 + kEntries * kEntry + 2 * kQ + 2 * kP;
};

template <int D, int MT, bool BF16>
__global__ void __launch_bounds__(kRowsThreads, RowsShape<D, MT>::kCtas)
    k_attn_rows(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v) {
  using Sh = RowsShape<D, MT>;
  using W = Walk<Sh::R, Sh::U, kTileCost, 0>;
  constexpr int U = Sh::U, TW = U / 4, NS = TW / 8;  // tokens of a warp, tiles of 8 of them
  constexpr int R = Sh::R, ST = Sh::kEntries, KS = D / 16, NP = D / 64;  // NP: pairs of 8-channel tiles of a warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sp = smem + ST * Sh::kEntry;
  uint8_t* sq = sp + 2 * Sh::kP;
  __shared__ alignas(8) uint64_t full[ST], empty[ST], q_full[2], q_empty[2], part_full[kParts], part_empty[kParts];
  __shared__ Part parts[kParts];
  __shared__ LineStart first;
  __shared__ int warp_sums[kRowsThreads / 32];
  __shared__ float sx[4][R];  // row maxima or sums of each warp
  __shared__ int gave_up;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 32) {
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  if (threadIdx.x == 0) {
    gave_up = 0;
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 4);
    }
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&part_full[i], 1);
      mbar_init(&part_empty[i], 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  pdl_wait();
  pdl_launch();  // the join may be scheduled; it waits for this kernel's end
  find_start<W, kRowsThreads>(a, kMinPart, first, warp_sums);
  bool ok = true;

  if (warp == 4) {
    // ---- producer: the parts, their queries, and for every unit ring entry e with K and entry e + 1 with V ----
    W w;
    w.start(a, first);
    CutTile cut = {};
    uint32_t err = 0;
    int e = 0, issued = 0, q_used = 0;
    for (int at = 0;; ++at) {
      Part g = {};
      const bool more = w.next(a, g, cut);
      const int i = at % kParts;
      if (at >= kParts) ok = warp_wait(&part_empty[i], (at / kParts - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        parts[i] = g;
        mbar_arrive(&part_full[i]);
      }
      if (!more) break;
      if (g.n_all > 0) {
        const int buf = q_used & 1, n = min(R, g.rows - g.f0);
        if (q_used >= 2) ok = warp_wait(&q_empty[buf], (q_used / 2 - 1) & 1);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&q_full[buf], (uint32_t)n * (D * 2));
        __syncwarp();
        for (int j = lane; j < n; j += 32) {  // rows past the last hold anything: their results are not written
          const int f = g.f0 + j, qi = a.div_g(f), head = g.h * a.G + f - qi * a.G;
          bulk_g2s(sq + buf * Sh::kQ + j * Sh::kQRow,
                   static_cast<const uint16_t*>(a.q) + (int64_t)(g.q0 + qi) * a.q_row + (int64_t)head * a.q_head, D * 2,
                   &q_full[buf]);
        }
        ++q_used;
      }
      Request r;
      r.row = g.row;
      r.base = g.base;
      int2 place = make_int2(0, 0);
      for (int k = 0; k < g.n_all && ok; ++k, e += 2) {
        if ((k & 31) == 0 && k + lane < g.n_all) {
          const int tok = (g.u0 + k + lane) * U;
          place = page_place(a, r, tok / kPage, err);
          place.y += tok % kPage;
        }
        const int pw = __shfl_sync(0xffffffffu, place.x, k & 31), py = __shfl_sync(0xffffffffu, place.y, k & 31);
        if (lane == 0) {
#pragma unroll
          for (int which = 0; which < 2; ++which) {
            const int st = (e + which) % ST;
            if (ok && e + which >= ST) ok = mbar_wait(&empty[st], ((e + which) / ST - 1) & 1);
            if (!ok) break;
            uint8_t* dst = smem + st * Sh::kEntry;
            mbar_expect_tx(&full[st], Sh::kEntry);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_4d(dst + c * (U * 128), which ? &map_v : &map_k, c * 64, py, g.h, pw, &full[st]);
            issued = e + which + 1;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (!ok) break;
    }
    if (lane == 0) {
      cut_tiles(a)[blockIdx.x] = cut;
      // leave only when every copy has landed (they have, unless a wait gave up)
      for (int i = max(0, issued - ST); i < issued; ++i) ok &= mbar_wait(&full[i % ST], (i / ST) & 1);
      for (int i = max(0, q_used - 2); i < q_used; ++i) ok &= mbar_wait(&q_full[i & 1], (i / 2) & 1);
      if (!ok) err |= TQ_DEV_ERR_TIMEOUT;
    }
    if (err && a.status) atomicOr(a.status, err);
    return;
  }

  // ---- consumers. A wait that gives up is made known at the next barrier, where all four warps leave together ----
  const int g8 = lane >> 2, c2 = (lane & 3) * 2, mi = lane >> 3, ri = lane & 7;
  const uint32_t ring = smem_u32(smem), pbase = smem_u32(sp), qbase = smem_u32(sq);
  int e = 0, q_used = 0, unit = 0;
  auto give_up = [&] {
    if (!ok) gave_up = 1;
  };
  for (int at = 0;; ++at) {
    const int pi = at % kParts;
    ok = ok && warp_wait(&part_full[pi], (at / kParts) & 1);
    Part g = {};
    if (ok) g = parts[pi];
    give_up();
    if (consumers_any(!ok)) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(&part_empty[pi]);
    if (g.n_all < 0) break;
    Request r;
    r.n_q = g.n_q;
    r.kv = g.r_kv;
    float o[MT][2 * NP][4], m[MT][2], l[MT][2];
    int lim[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int i = 0; i < 2 * NP; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[t][x] = 0.f;
        const int f = g.f0 + t * 16 + g8 + x * 8;
        lim[t][x] = f < g.rows ? seen(a, r, a.div_g(f)) : 0;
        m[t][x] = f < g.rows ? -INFINITY : INFINITY;  // a row past the last, of any scores, never outgrows its maximum
      }
    }
    const int lim_all = seen(a, r, a.div_g(g.f0));  // what every row of the tile sees needs no mask
    constexpr bool kHoldQ = D * MT <= 128 || (D == 256 && MT == 1);  // the query fragments stay in registers
    uint32_t aq[kHoldQ ? MT : 1][kHoldQ ? KS : 1][4];
    const uint32_t qb = qbase + (q_used & 1) * Sh::kQ + ((mi & 1) * 8 + ri) * Sh::kQRow + (mi >> 1) * 16;
    if (g.n_all > 0) {
      ok = warp_wait(&q_full[q_used & 1], (q_used / 2) & 1);
      if constexpr (kHoldQ) {
        if (ok) {
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) ldsm4(aq[t][ks], qb + t * 16 * Sh::kQRow + ks * 32);
        }
      }
    }
    bool left = false;
    for (int k = 0; k < g.n_all; ++k, e += 2, ++unit) {
      const int base = (g.u0 + k) * U, t0 = base + warp * TW;
      const uint32_t pb = pbase + (unit & 1) * Sh::kP;
      float s[MT][NS][4], top[MT][2];
      // scores of this warp's tokens
      {
        const int st = e % ST;
        ok = ok && warp_wait(&full[st], (e / ST) & 1);
        const uint32_t kt = ring + st * Sh::kEntry;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int n = 0; n < NS; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
        if (ok && t0 < g.kv) {
          // at 16 tokens per warp the odd steps have sums of their own: half the chain of dependent products
          constexpr int kChains = NS == 2 ? 2 : 1;
          float s2[kChains == 2 ? MT : 1][2][4] = {};
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2) {
            uint32_t bk[2][NS / 2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int n = 0; n < NS / 2; ++n)
                ldsm4(bk[x][n], kt + sw_off(U, warp * TW + n * 16 + (mi >> 1) * 8 + ri, (ks + x) * 2 + (mi & 1)));
#pragma unroll
            for (int t = 0; t < MT; ++t) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t af[4];
                if constexpr (kHoldQ) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) af[i] = aq[t][ks + x][i];
                } else {
                  ldsm4(af, qb + t * 16 * Sh::kQRow + (ks + x) * 32);
                }
#pragma unroll
                for (int n = 0; n < NS / 2; ++n) {
                  if constexpr (kChains == 2) {
                    mma16816<BF16>(x ? s2[t][0] : s[t][0], af, bk[x][n][0], bk[x][n][1]);
                    mma16816<BF16>(x ? s2[t][1] : s[t][1], af, bk[x][n][2], bk[x][n][3]);
                  } else {
                    mma16816<BF16>(s[t][2 * n], af, bk[x][n][0], bk[x][n][1]);
                    mma16816<BF16>(s[t][2 * n + 1], af, bk[x][n][2], bk[x][n][3]);
                  }
                }
              }
            }
          }
          if constexpr (kChains == 2) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[t][n][i] += s2[t][n][i];
          }
        }
      }
      // masked scores are selected away, not added to: what stands behind a sequence can be NaN
      bool need = false;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        top[t][0] = top[t][1] = -INFINITY;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& x = s[t][n][i];
            x *= a.scale_log2;
            if (base + U > lim_all) x = t0 + n * 8 + c2 + (i & 1) < lim[t][i >> 1] ? x : -INFINITY;
            top[t][i >> 1] = fmaxf(top[t][i >> 1], x);
          }
        need |= top[t][0] - m[t][0] > kLazy || top[t][1] - m[t][1] > kLazy;  // a sum m + kLazy could round to more
      }
      float sum[MT][2];
      for (;;) {  // twice where a maximum outgrew its range: the code is not doubled, since a cold path costs its fetches
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const float mu[2] = {m[t][0] == -INFINITY ? 0.f : m[t][0], m[t][1] == -INFINITY ? 0.f : m[t][1]};
          sum[t][0] = sum[t][1] = 0.f;
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[i] = BF16 ? exp2_fast(s[t][n][i] - mu[i >> 1]) : exp2_fast((s[t][n][i] - mu[i >> 1]) + kLift);
              sum[t][i >> 1] += w[i];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
              asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(pb + sw_off(R, t * 16 + g8 + x * 8, warp * NS + n) + c2 * 2),
                           "r"(pack2<BF16>(w[2 * x], w[2 * x + 1]))
                           : "memory");
          }
        }
        give_up();
        if (!consumers_any(need || !ok)) break;
        if (*(volatile int*)&gave_up) {
          left = true;
          break;
        }
        // new maxima for all rows, from all four warps
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            top[t][x] = fmaxf(top[t][x], __shfl_xor_sync(0xffffffffu, top[t][x], 1));
            top[t][x] = fmaxf(top[t][x], __shfl_xor_sync(0xffffffffu, top[t][x], 2));
            if ((lane & 3) == 0) sx[warp][t * 16 + g8 + x * 8] = top[t][x];
          }
        consumers_any(false);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          float alpha[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int row = t * 16 + g8 + x * 8;
            const float mn = fmaxf(m[t][x], fmaxf(fmaxf(sx[0][row], sx[1][row]), fmaxf(sx[2][row], sx[3][row])));
            alpha[x] = mn == -INFINITY ? 1.f : exp2_fast(m[t][x] - mn);
            m[t][x] = mn;
            l[t][x] *= alpha[x];
          }
          if (k > 0) {
#pragma unroll
            for (int i = 0; i < 2 * NP; ++i) {
              o[t][i][0] *= alpha[0];
              o[t][i][1] *= alpha[0];
              o[t][i][2] *= alpha[1];
              o[t][i][3] *= alpha[1];
            }
          }
        }
        need = false;  // no weight is above 1 now
      }
      if (left) break;
      if (lane == 0) mbar_arrive(&empty[e % ST]);  // K: the weights that were made of it were stored before the barrier
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        l[t][0] += sum[t][0];
        l[t][1] += sum[t][1];
      }
      // sums of D / 4 channels over all tokens of the unit
      {
        const int st = (e + 1) % ST;
        ok = warp_wait(&full[st], ((e + 1) / ST) & 1);
        const uint32_t vt = ring + st * Sh::kEntry;
        if (ok) {
          constexpr int kGroup = D * MT <= 128 ? 4 : 2;  // steps of 16 tokens whose operands are loaded together
#pragma unroll
          for (int k0 = 0; k0 < U / 16; k0 += kGroup) {
            uint32_t ap[kGroup][MT][4], bv[kGroup][NP][4];
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
              const int ks = k0 + j;
#pragma unroll
              for (int t = 0; t < MT; ++t) ldsm4(ap[j][t], pb + sw_off(R, t * 16 + (mi & 1) * 8 + ri, ks * 2 + (mi >> 1)));
#pragma unroll
              for (int np = 0; np < NP; ++np)
                ldsm4t(bv[j][np], vt + sw_off(U, ks * 16 + (mi & 1) * 8 + ri, (warp * NP + np) * 2 + (mi >> 1)));
            }
            if (g.kv < base + U) {  // the unit that the sequence ends in: V rows behind it are zeroed (0 x NaN is NaN)
#pragma unroll
              for (int j = 0; j < kGroup; ++j) {
                const int n0 = g.kv - (base + (k0 + j) * 16 + c2), n1 = n0 - 8;
                const uint32_t keep0 = n0 >= 2 ? 0xffffffffu : n0 == 1 ? 0x0000ffffu : 0u;
                const uint32_t keep1 = n1 >= 2 ? 0xffffffffu : n1 == 1 ? 0x0000ffffu : 0u;
#pragma unroll
                for (int np = 0; np < NP; ++np) {
                  bv[j][np][0] &= keep0;
                  bv[j][np][1] &= keep1;
                  bv[j][np][2] &= keep0;
                  bv[j][np][3] &= keep1;
                }
              }
            }
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
#pragma unroll
              for (int np = 0; np < NP; ++np)
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                  mma16816<BF16>(o[t][2 * np], ap[j][t], bv[j][np][0], bv[j][np][1]);
                  mma16816<BF16>(o[t][2 * np + 1], ap[j][t], bv[j][np][2], bv[j][np][3]);
                }
          }
        }
        uint32_t used = 0;
#pragma unroll
        for (int t = 0; t < MT; ++t) used |= bits_of(o[t]);
        __syncwarp();
        if (ok && lane == 0) give_back(&empty[st], used, a.batch);
      }
    }
    if (left) break;
    if (g.n_all > 0) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[q_used & 1]);
      ++q_used;
    }
    // the row sums of the four warps
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float v = l[t][x];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if ((lane & 3) == 0) sx[warp][t * 16 + g8 + x * 8] = v;
      }
    give_up();
    if (consumers_any(!ok)) break;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = t * 16 + g8 + x * 8, f = g.f0 + row;
        if (f >= g.rows) continue;
        const float sum = sx[0][row] + sx[1][row] + sx[2][row] + sx[3][row];
        if (g.direct) {
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          const int qi = a.div_g(f), head = g.h * a.G + f - qi * a.G;
          uint16_t* dst = static_cast<uint16_t*>(a.out) + (int64_t)(g.q0 + qi) * a.o_row + (int64_t)head * a.o_head +
                          warp * (D / 4) + c2;
#pragma unroll
          for (int i = 0; i < 2 * NP; ++i)
            *reinterpret_cast<uint32_t*>(dst + i * 8) = result2<BF16>(o[t][i][2 * x] * inv, o[t][i][2 * x + 1] * inv);
        } else {
          float* po = cut_o<R, D>(a, gridDim.x, blockIdx.x, g.slot) + row * D + warp * (D / 4) + c2;
#pragma unroll
          for (int i = 0; i < 2 * NP; ++i)
            *reinterpret_cast<float2*>(po + i * 8) = make_float2(o[t][i][2 * x], o[t][i][2 * x + 1]);
          if (warp == 0 && (lane & 3) == 0)
            cut_ml<R>(a, gridDim.x, blockIdx.x, g.slot)[row] = make_float2(m[t][x], sum);
        }
      }
  }
  if (!ok && lane == 0 && a.status) atomicOr(a.status, TQ_DEV_ERR_TIMEOUT);
}

template <int D, int MT, bool BF16>
cudaError_t launch_as(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, cudaStream_t s) {
  using Sh = RowsShape<D, MT>;
  static std::atomic<uint64_t> known{0};
  cudaError_t e = allow_smem(k_attn_rows<D, MT, BF16>, Sh::kSmem, known);
  if (e == cudaSuccess)
    e = launch_pdl(k_attn_rows<D, MT, BF16>, dim3(p.ctas), dim3(kRowsThreads), Sh::kSmem, s, a, m.k, m.v);
  if (e != cudaSuccess) return e;
  return launch_join<D, Sh::R, BF16>(a, p.ctas, p.max_rows, s);
}

template <bool BF16>
cudaError_t launch_type(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, cudaStream_t s) {
  if (d == 64) return p.tile_rows == 16 ? launch_as<64, 1, BF16>(a, m, p, s) : launch_as<64, 2, BF16>(a, m, p, s);
  if (d == 128) return p.tile_rows == 16 ? launch_as<128, 1, BF16>(a, m, p, s) : launch_as<128, 2, BF16>(a, m, p, s);
  return p.tile_rows == 16 ? launch_as<256, 1, BF16>(a, m, p, s) : launch_as<256, 2, BF16>(a, m, p, s);
}

}  // namespace

AttnShape attn_rows_shape(int d, int64_t rows, int sms) {
  const int tile = rows <= 16 ? 16 : 32;
  const int ctas = sms * (d == 256 ? RowsShape<256, 1>::kCtas : d == 64 && tile == 16 ? RowsShape<64, 1>::kCtas : 2);
  return {tile, d == 64 ? RowsShape<64, 1>::U : RowsShape<128, 1>::U, ctas, cta_bytes(tile, d), kTileCost, kMinPart};
}
cudaError_t launch_attn_rows(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, int dtype, cudaStream_t s) {
  return dtype == TQ_BF16 ? launch_type<true>(a, m, p, d, s) : launch_type<false>(a, m, p, d, s);
}

}  // namespace tq
