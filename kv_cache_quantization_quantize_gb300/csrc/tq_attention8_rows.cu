// Attention of few new tokens per request (single tokens, drafts) over a paged cache of 8 bits.
#include "tq_attention_rows.cuh"

namespace tq {
namespace {

// =============================================================================================
// k_attn8_rows: the division of work of k_attn_rows (tq_attention_rows.cu) over e4m3 pages, whose bytes bound it. Numbers of
// e4m3 are exact in f16, so the products are m16n8k16 in f16 on numbers that each warp takes from e4m3 to f16 behind
// shared memory, two to an instruction:
//   - K: a thread's 16 bytes are 16 channels of one token, four to a product step; the order of channels within a step is
//     free, as long as the queries' fragments have the same.
//   - V: ldmatrix moves pairs of neighbouring channels as one 16-bit element, transposed; a byte permutation then parts
//     the even channels from the odd ones, which go to products of their own.
// Scales: with p = 2^(s - m + log2 vs - m'), where m + m' is a maximum of s + log2 vs, the sums are of p times the number and the statistic
// is of p / vs, so scales cost nothing per element but an addition, and weights are rounded to f16 relative to what they are
// multiplied with, however far apart the scales of pages are.
// Measured: 32 single tokens over 4096 to 8192, 32 heads on 8 of 128, 71.0 us, 5.4 TB/s (79 % of a copy: a unit's chain of
// products, maximum and products is not all hidden by two CTAs); one over 32768 21.9 us, of which some 8 are the way to the
// first load and the join; 16 requests of 8 drafts, tiles of 32 rows, 65 us (42 %, the chain). At head_dim 64 a unit has half the bytes
// and the same chain, exponentials and barrier: 64 single tokens over 4096 to 8192, 16 heads on 4, 52 us (57 %). 64 short
// requests of 100 to 1000 tokens, 32 heads on 8 of 128, 28 us (35 %).
// =============================================================================================
constexpr int k8TileCost = 64;   // start and end of a tile, as one unit
constexpr int k8MinPart = 64;    // no CTA gets less than that (2 requests of 100 to 1000 tokens: 15.2 us with 128, 10.9 so)

template <int D, int MT>
struct Rows8Shape {
  static constexpr int R = 16 * MT;
  // Consumers: for the sums each has D / kWarps channels, 16 at least. With 8 at head_dim 128 two CTAs leave 96 registers (32
  // requests of 4096 to 8192 tokens 93 us, with 4 72); at 256 8 are faster (16 requests of 8 drafts each 62.7 against 68.5).
  static constexpr int kWarps = D == 256 ? 8 : 4;
  static constexpr int kThreads = 32 * kWarps + 32;
  static constexpr int U = kPage;  // tokens of a unit: a page, which has one scale
  static constexpr int kEntry = U * D;          // bytes of K or V of one unit
  static constexpr int kCtas = D == 256 ? 1 : D == 64 && MT == 1 ? 3 : 2;  // CTAs per SM
  static constexpr int kEntries = D == 64 ? 6 : 4;
  static constexpr int kQRow = D * 2 + 16;  // bytes of a query row
  static constexpr int kQ = R * kQRow;
  static constexpr int kP = R * U * 2;  // weights of one unit
  static constexpr int kSmem = 1024 + kEntries * kEntry + 2 * kQ + 2 * kP;
};

// Byte offset of 16-byte chunk `chunk` of token `row` in a tile of U tokens as TMA writes it: blocks of 128-byte rows in the
// 128-byte swizzle, or 64-byte rows in the 64-byte one.
template <int D, int U>
__device__ __forceinline__ uint32_t raw_off(int row, int chunk) {
  if constexpr (D == 64) return (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
  else return (uint32_t)((chunk >> 3) * (U * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}
// Barrier over the consumer warps; true for all where the predicate is true for one.
template <int WARPS>
__device__ __forceinline__ bool any_of(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(32 * WARPS)
      : "memory");
  return r != 0;
}
// Token that column (or row) x of a group of 8 stands for: with rows of 128 bytes, neighbours are four apart, so that the loads of K,
// of two tokens by eight lanes, meet no bank conflict.
template <int D>
__device__ __forceinline__ int tok8(int x) {
  return D == 64 ? x : (x >> 1) | ((x & 1) << 2);
}

template <int D, int MT, bool BF16>
__global__ void __launch_bounds__(Rows8Shape<D, MT>::kThreads, Rows8Shape<D, MT>::kCtas)
    k_attn8_rows(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v) {
  using Sh = Rows8Shape<D, MT>;
  using W = Walk<Sh::R, Sh::U, k8TileCost, 0>;
  constexpr int NW = Sh::kWarps, U = Sh::U, TW = U / NW, NS = TW / 8;  // tokens of a warp, tiles of 8 of them
  constexpr int R = Sh::R, ST = Sh::kEntries, KS = D / 16, NC = D / (16 * NW);  // NC: 16-channel chunks of a warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sp = smem + ST * Sh::kEntry;
  uint8_t* sq = sp + 2 * Sh::kP;
  __shared__ alignas(8) uint64_t full[ST], empty[ST], q_full[2], q_empty[2], part_full[kParts], part_empty[kParts];
  __shared__ Part parts[kParts];
  __shared__ LineStart first;
  __shared__ int warp_sums[Sh::kThreads / 32];
  __shared__ float sx[NW][R];  // row maxima or sums of each warp
  __shared__ UnitScale scales[ST];  // of unit e / 2
  __shared__ float q_back[2][R];  // what a row's scores are multiplied with
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
      mbar_init(&empty[i], NW);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], NW);
    }
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&part_full[i], 1);
      mbar_init(&part_empty[i], NW);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  pdl_wait();
  pdl_launch();  // the join may be scheduled; it waits for this kernel's end
  find_start<W, Sh::kThreads>(a, k8MinPart, first, warp_sums);
  bool ok = true;

  if (warp == NW) {
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
      UnitScale us = {};
      for (int k = 0; k < g.n_all && ok; ++k, e += 2) {
        if ((k & 31) == 0 && k + lane < g.n_all) {
          const int tok = (g.u0 + k + lane) * U;
          place = page_place(a, r, tok / kPage, err);
          place.y += tok % kPage;
          us = unit_scale(a, place.x, g.h);
        }
        const int pw = __shfl_sync(0xffffffffu, place.x, k & 31), py = __shfl_sync(0xffffffffu, place.y, k & 31);
        const UnitScale u1 = {__shfl_sync(0xffffffffu, us.k, k & 31), __shfl_sync(0xffffffffu, us.log_v, k & 31),
                              __shfl_sync(0xffffffffu, us.inv_v, k & 31)};
        if (lane == 0) {
#pragma unroll
          for (int which = 0; which < 2; ++which) {
            const int st = (e + which) % ST;
            if (ok && e + which >= ST) ok = mbar_wait(&empty[st], ((e + which) / ST - 1) & 1);
            if (!ok) break;
            if (which == 0) scales[e / 2 % ST] = u1;  // read by all before they give the entry back
            uint8_t* dst = smem + st * Sh::kEntry;
            mbar_expect_tx(&full[st], Sh::kEntry);
#pragma unroll
            for (int c = 0; c < (D + 127) / 128; ++c)
              tma_load_4d(dst + c * (U * 128), which ? &map_v : &map_k, c * 128, py, g.h, pw, &full[st]);
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

  // ---- consumers. A wait that gives up is made known at the next barrier, where all of them leave together ----
  const int g8 = lane >> 2, j4 = lane & 3, mi = lane >> 3, ri = lane & 7;
  const int tk0 = tok8<D>(2 * j4), tk1 = tok8<D>(2 * j4 + 1);  // tokens of this thread's two columns of a group of 8
  const uint32_t ring = smem_u32(smem), pbase = smem_u32(sp);
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
    if (any_of<NW>(!ok)) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(&part_empty[pi]);
    if (g.n_all < 0) break;
    Request r;
    r.n_q = g.n_q;
    r.kv = g.r_kv;
    const int qbuf = q_used & 1;
    if (g.n_all > 0) {
      ok = warp_wait(&q_full[qbuf], (q_used / 2) & 1);
      if constexpr (BF16) {  // the queries to f16, each row by a power of two
        if (ok) {
          constexpr int kWords = D / 64;
          for (int row = warp; row < min(R, g.rows - g.f0); row += NW) {
            uint32_t* p = reinterpret_cast<uint32_t*>(sq + qbuf * Sh::kQ + row * Sh::kQRow) + lane;
            uint32_t v[kWords], top = 0;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
              v[i] = p[32 * i];
              top = max(top, max(v[i] & 0x7fffu, (v[i] >> 16) & 0x7fffu));
            }
            top = __reduce_max_sync(0xffffffffu, top);
            const float by = to_f16_by(top);
#pragma unroll
            for (int i = 0; i < kWords; ++i) p[32 * i] = bf16x2_to_f16x2(v[i], by);
            if (lane == 0) q_back[qbuf][row] = to_f16_back(top);
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");  // the buffer's next queries come by bulk copies
        }
        give_up();
        if (any_of<NW>(!ok)) break;
      }
    }
    float o[MT][2 * NC][4], m[MT][2], mv[MT][2], l[MT][2], back[MT][2];  // m, mv: of scores, of values' scales
    int lim[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int i = 0; i < 2 * NC; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[t][x] = mv[t][x] = 0.f;
        const int row = t * 16 + g8 + x * 8, f = g.f0 + row;
        lim[t][x] = f < g.rows ? seen(a, r, a.div_g(f)) : 0;
        m[t][x] = f < g.rows ? -INFINITY : INFINITY;  // a row past the last, of any scores, never outgrows its maximum
        back[t][x] = a.scale_log2 * (BF16 && f < g.rows && g.n_all > 0 ? q_back[qbuf][row] : 1.f);
      }
    }
    const int lim_all = seen(a, r, a.div_g(g.f0));  // what every row of the tile sees needs no mask
    constexpr bool kHoldQ = D * MT <= 128 || (D == 256 && MT == 1);  // the query fragments stay in registers
    uint32_t aq[kHoldQ ? MT : 1][kHoldQ ? KS : 1][4];
    const uint8_t* qrow = sq + qbuf * Sh::kQ + g8 * Sh::kQRow + j4 * 32;
    // step 4 c + s holds channels 64 c + 16 j + 4 s .. + 3 of lane j of each four, as the loads of K have them
    auto query = [&](int t, int ks, uint32_t (&f)[4]) {
      const uint8_t* p = qrow + t * 16 * Sh::kQRow + (ks >> 2) * 128 + (ks & 3) * 8;
      const uint2 x = *reinterpret_cast<const uint2*>(p), y = *reinterpret_cast<const uint2*>(p + 8 * Sh::kQRow);
      f[0] = x.x;
      f[1] = y.x;
      f[2] = x.y;
      f[3] = y.y;
    };
    if constexpr (kHoldQ) {
      if (g.n_all > 0 && ok) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) query(t, ks, aq[t][ks]);
      }
    }
    bool left = false;
    for (int k = 0; k < g.n_all; ++k, e += 2, ++unit) {
      const int base = (g.u0 + k) * U, t0 = base + warp * TW;
      const uint32_t pb = pbase + (unit & 1) * Sh::kP;
      float s[MT][NS][4], top[MT][2];
      UnitScale us = {1.f, 0.f, 1.f};
      // scores of this warp's tokens
      {
        const int st = e % ST;
        ok = ok && warp_wait(&full[st], (e / ST) & 1);
        const uint8_t* kt = smem + st * Sh::kEntry;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int n = 0; n < NS; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
        if (ok) us = scales[e / 2 % ST];
        if (ok && t0 < g.kv) {
          // at 16 tokens per warp the odd steps have sums of their own: half the chain of dependent products
          constexpr int kChains = NS == 2 ? 2 : 1;
          float s2[kChains == 2 ? MT : 1][2][4] = {};
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint4 raw[NS];
#pragma unroll
            for (int n = 0; n < NS; ++n)
              raw[n] = *reinterpret_cast<const uint4*>(kt + raw_off<D, U>(warp * TW + n * 8 + tok8<D>(g8), c * 4 + j4));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t af[MT][4];
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                if constexpr (kHoldQ) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) af[t][i] = aq[t][4 * c + x][i];
                } else {
                  query(t, 4 * c + x, af[t]);
                }
              }
#pragma unroll
              for (int n = 0; n < NS; ++n) {
                const uint32_t w = x == 0 ? raw[n].x : x == 1 ? raw[n].y : x == 2 ? raw[n].z : raw[n].w;
                const uint32_t b0 = e4m3_lo(w), b1 = e4m3_hi(w);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                  if constexpr (kChains == 2) mma16816<false>(x & 1 ? s2[t][n] : s[t][n], af[t], b0, b1);
                  else mma16816<false>(s[t][n], af[t], b0, b1);
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
        const float by[2] = {back[t][0] * us.k, back[t][1] * us.k};
        top[t][0] = top[t][1] = -INFINITY;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& x = s[t][n][i];
            x *= by[i >> 1];
            if (base + U > lim_all) x = t0 + n * 8 + (i & 1 ? tk1 : tk0) < lim[t][i >> 1] ? x : -INFINITY;
            top[t][i >> 1] = fmaxf(top[t][i >> 1], x);
          }
        // (apart: far scores have no room for the logarithm)
        need |= (top[t][0] - m[t][0]) + (us.log_v - mv[t][0]) > kLazy || (top[t][1] - m[t][1]) + (us.log_v - mv[t][1]) > kLazy;
        need |= us.log_v - fmaxf(mv[t][0], mv[t][1]) < kThin;
      }
      float sum[MT][2];
      for (;;) {  // twice where a maximum or a scale left its range: the code is not doubled, since a cold path costs its fetches
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const float mu[2] = {m[t][0] == -INFINITY ? 0.f : m[t][0], m[t][1] == -INFINITY ? 0.f : m[t][1]};
          float above[2] = {(us.log_v - mv[t][0]) + kLift, (us.log_v - mv[t][1]) + kLift};
          sum[t][0] = sum[t][1] = 0.f;
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[i] = exp2_fast((s[t][n][i] - mu[i >> 1]) + above[i >> 1]);
              sum[t][i >> 1] += w[i];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
              asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(pb + sw_off(R, t * 16 + g8 + x * 8, warp * NS + n) + j4 * 4),
                           "r"(pack2<false>(w[2 * x], w[2 * x + 1]))
                           : "memory");
          }
        }
        give_up();
        if (!any_of<NW>(need || !ok)) break;
        if (*(volatile int*)&gave_up) {
          left = true;
          break;
        }
        // new references for all rows, from all warps
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            top[t][x] = fmaxf(top[t][x], __shfl_xor_sync(0xffffffffu, top[t][x], 1));
            top[t][x] = fmaxf(top[t][x], __shfl_xor_sync(0xffffffffu, top[t][x], 2));
            if ((lane & 3) == 0) sx[warp][t * 16 + g8 + x * 8] = top[t][x];
          }
        any_of<NW>(false);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          float alpha[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int row = t * 16 + g8 + x * 8;
            float mx = sx[0][row];
#pragma unroll
            for (int i = 1; i < NW; ++i) mx = fmaxf(mx, sx[i][row]);
            alpha[x] = 1.f;
            const float by = (m[t][x] - mx) + (mv[t][x] - us.log_v);
            if (by < 0.f) {
              alpha[x] = exp2_fast(by);
              m[t][x] = mx;
              mv[t][x] = us.log_v;
              l[t][x] = rescaled(l[t][x], by);
            }
          }
          if (k > 0) {
#pragma unroll
            for (int i = 0; i < 2 * NC; ++i) {
              o[t][i][0] *= alpha[0];
              o[t][i][1] *= alpha[0];
              o[t][i][2] *= alpha[1];
              o[t][i][3] *= alpha[1];
            }
          }
        }
        bool thin = false;
#pragma unroll
        for (int t = 0; t < MT; ++t) thin |= us.log_v - fmaxf(mv[t][0], mv[t][1]) < kThin;
        if (thin) {  // the unit's part of the statistic by exponentials of its own
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float mu = m[t][i >> 1];
                l[t][i >> 1] += exp2_fast((s[t][n][i] - (mu == -INFINITY ? 0.f : mu)) + (kLift - mv[t][i >> 1]));
              }
          us.inv_v = 0.f;  // and nothing from the weights
        }
        need = false;  // no weight is above 1 now
      }
      if (left) break;
      if (lane == 0) mbar_arrive(&empty[e % ST]);  // K: the weights that were made of it were stored before the barrier
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        l[t][0] += sum[t][0] * us.inv_v;
        l[t][1] += sum[t][1] * us.inv_v;
      }
      // sums of D / NW channels over all tokens of the unit
      {
        const int st = (e + 1) % ST;
        ok = warp_wait(&full[st], ((e + 1) / ST) & 1);
        const uint32_t vt = ring + st * Sh::kEntry;
        if (ok) {
          constexpr int kGroup = D * MT <= 128 ? 4 : 2;  // steps of 16 tokens whose operands are loaded together
#pragma unroll
          for (int k0 = 0; k0 < U / 16; k0 += kGroup) {
            uint32_t ap[kGroup][MT][4], bv[kGroup][NC][2];  // [2]: the step's first and second 8 tokens
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
#pragma unroll
              for (int t = 0; t < MT; ++t)
                ldsm4(ap[j][t], pb + sw_off(R, t * 16 + (mi & 1) * 8 + ri, (k0 + j) * 2 + (mi >> 1)));
            if constexpr (NC == 1) {  // two steps to a load
#pragma unroll
              for (int j = 0; j < kGroup; j += 2) {
                uint32_t v[4];
                ldsm4t(v, vt + raw_off<D, U>((k0 + j + (mi >> 1)) * 16 + (mi & 1) * 8 + tok8<D>(ri), warp));
                bv[j][0][0] = v[0], bv[j][0][1] = v[1], bv[j + 1][0][0] = v[2], bv[j + 1][0][1] = v[3];
              }
            } else {  // two chunks of 16 channels to a load
#pragma unroll
              for (int j = 0; j < kGroup; ++j)
#pragma unroll
                for (int c = 0; c < NC; c += 2) {
                  uint32_t v[4];
                  ldsm4t(v, vt + raw_off<D, U>((k0 + j) * 16 + (mi & 1) * 8 + tok8<D>(ri), warp * NC + c + (mi >> 1)));
                  bv[j][c][0] = v[0], bv[j][c][1] = v[1], bv[j][c + 1][0] = v[2], bv[j][c + 1][1] = v[3];
                }
            }
            if (g.kv < base + U) {  // the unit that the sequence ends in: V rows behind it are zeroed (0 x NaN is NaN)
#pragma unroll
              for (int j = 0; j < kGroup; ++j) {
                const int n0 = g.kv - (base + (k0 + j) * 16);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const uint32_t keep = (8 * x + tk0 < n0 ? 0x0000ffffu : 0u) | (8 * x + tk1 < n0 ? 0xffff0000u : 0u);
#pragma unroll
                  for (int c = 0; c < NC; ++c) bv[j][c][x] &= keep;
                }
              }
            }
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
#pragma unroll
              for (int c = 0; c < NC; ++c) {
                // {token 0: channels 2 p, 2 p + 1; token 1: the same} -> {2 p: both tokens; 2 p + 1: both}
                const uint32_t x = __byte_perm(bv[j][c][0], 0, 0x3120), y = __byte_perm(bv[j][c][1], 0, 0x3120);
                const uint32_t x0 = e4m3_lo(x), y0 = e4m3_lo(y), x1 = e4m3_hi(x), y1 = e4m3_hi(y);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                  mma16816<false>(o[t][2 * c], ap[j][t], x0, y0);
                  mma16816<false>(o[t][2 * c + 1], ap[j][t], x1, y1);
                }
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
    // the row sums of the warps
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
    if (any_of<NW>(!ok)) break;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = t * 16 + g8 + x * 8, f = g.f0 + row;
        if (f >= g.rows) continue;
        float sum = sx[0][row];
#pragma unroll
        for (int i = 1; i < NW; ++i) sum += sx[i][row];
        const float2 part = part_reference(m[t][x], mv[t][x], sum);
        const int ch = warp * (D / NW) + j4 * 4;  // channels 4 j .. 4 j + 3 of each chunk: even, odd, even, odd
        if (g.direct) {
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          const int qi = a.div_g(f), head = g.h * a.G + f - qi * a.G;
          uint16_t* dst = static_cast<uint16_t*>(a.out) + (int64_t)(g.q0 + qi) * a.o_row + (int64_t)head * a.o_head + ch;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            *reinterpret_cast<uint2*>(dst + c * 16) =
                make_uint2(result2<BF16>(o[t][2 * c][2 * x] * inv, o[t][2 * c + 1][2 * x] * inv),
                           result2<BF16>(o[t][2 * c][2 * x + 1] * inv, o[t][2 * c + 1][2 * x + 1] * inv));
        } else {
          float* po = cut_o<R, D>(a, gridDim.x, blockIdx.x, g.slot) + row * D + ch;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            *reinterpret_cast<float4*>(po + c * 16) =
                make_float4(o[t][2 * c][2 * x] * part.y, o[t][2 * c + 1][2 * x] * part.y, o[t][2 * c][2 * x + 1] * part.y, o[t][2 * c + 1][2 * x + 1] * part.y);
          if (warp == 0 && (lane & 3) == 0)
            cut_ml<R>(a, gridDim.x, blockIdx.x, g.slot)[row] = make_float2(part.x, sum * part.y);
        }
      }
  }
  if (!ok && lane == 0 && a.status) atomicOr(a.status, TQ_DEV_ERR_TIMEOUT);
}

template <int D, int MT, bool BF16>
cudaError_t launch_as(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, cudaStream_t s) {
  using Sh = Rows8Shape<D, MT>;
  static std::atomic<uint64_t> known{0};
  cudaError_t e = allow_smem(k_attn8_rows<D, MT, BF16>, Sh::kSmem, known);
  if (e == cudaSuccess)
    e = launch_pdl(k_attn8_rows<D, MT, BF16>, dim3(p.ctas), dim3(Sh::kThreads), Sh::kSmem, s, a, m.k, m.v);
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

namespace {
template <int D, int MT>
AttnShape rows8_shape(int sms) {
  using Sh = Rows8Shape<D, MT>;
  return {Sh::R, Sh::U, sms * Sh::kCtas, cta_bytes(Sh::R, D), k8TileCost, k8MinPart};
}
}  // namespace

AttnShape attn8_rows_shape(int d, int64_t rows, int sms) {
  if (d == 64) return rows <= 16 ? rows8_shape<64, 1>(sms) : rows8_shape<64, 2>(sms);
  if (d == 128) return rows <= 16 ? rows8_shape<128, 1>(sms) : rows8_shape<128, 2>(sms);
  return rows <= 16 ? rows8_shape<256, 1>(sms) : rows8_shape<256, 2>(sms);
}
cudaError_t launch_attn8_rows(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, int dtype, cudaStream_t s) {
  return dtype == TQ_BF16 ? launch_type<true>(a, m, p, d, s) : launch_type<false>(a, m, p, d, s);
}

}  // namespace tq
