// Attention of chunks of new tokens over a paged cache of 8 bits, on the tensor cores (tcgen05).
#include "tq_attention_tc.cuh"

namespace tq {
namespace {

// =============================================================================================
// k_attn8_tc: the division of work of k_attn_tc (tq_attention_tc.cu) over e4m3 pages. A warpgroup of its own takes each
// K and V tile from the ring that TMA fills, brings its numbers to f16 (which holds every one of them) in the 128-byte swizzle that
// the products read, with zeros behind the sequence, and hands it on; so the products, in f16, and the softmax are those of
// the exact cache. The scales are the softmax's: with p = 2^(s - m + log2 vs - m'), where m + m' is a maximum of s + log2 vs, O sums p times
// the numbers and the statistic p / vs: one constant of the exponent and one product per unit and row. Queries in bf16 are brought to
// f16 by a power of two for each row on their way into shared memory (or TMEM), which the scores' scale takes out again.
// 2048 queries after 30720 tokens, 32 heads on 8 of 128, take 744 us, 1.43 PFLOP/s (75 % of the library's products). The tensor pipe
// is active 61 % of that time and issue slots 49 %: a tile's chain of scores, softmax and products is not all hidden by the
// other tile's. Without the conversions' work it would be 701 us, for they take issue slots from the softmax. Some registers are
// spilled (152 to 200 bytes a thread at D = 64 and 128, 52 at 256); whether inside the loop has not been measured.
// =============================================================================================
constexpr uint32_t kTmemQ = 128;  // kPair: the queries are an operand in TMEM, in these columns
constexpr int kScales = 16;       // ring of units' scales: more units than are between TMA and the softmax

template <int D>
struct Tc8Shape {
  static constexpr int kNT = D == 256 ? 1 : 2;     // tiles of 128 rows: TMEM holds S and O of two up to D = 128
  static constexpr int kBN = D == 256 ? 64 : 128;  // tokens of a K or V tile
  static constexpr int kTile = kBN * D * 2;        // its bytes in f16
  static constexpr int kRaw = kBN * D;             // and in e4m3
  static constexpr int kStages = D == 64 ? 6 : D == 128 ? 3 : 4;
  static constexpr int kRawStages = kStages;
  // One tile's softmax is shared by two warpgroups that take its units in turn, each with a buffer of S and P of its own:
  // with one warp per scheduler it would be the bound, as it is of the exact kernel (10 % there).
  static constexpr bool kPair = kNT == 1;
  static constexpr int kThreads = 512;
  // Start and end of a tile, in 64ths of a unit: 7 units of 128 tokens, 10 of 64 (4096 x 4096 causal, 16 query heads on 4 at
  // D = 256 218 us with 5 units, 191 with 7, 178 with 10, 179 with 13; 16 requests of up to 700 on up to 4000 tokens, 32 heads on
  // 8 of 128, 244 with 3, 231 with 5, 212 with 7, 207 with 9, but 4096 x 4096 161 with 7 and 164 with 9).
  static constexpr int kTileCost = D == 256 ? 640 : 448;
  // No CTA gets less than this, or short work would be in more parts than it is worth joining (16 queries of a request of 8000
  // tokens at D = 256: 46.2 us with 128, 39.9 so; at 64 38.2 and 24.9) or leave CTAs idle (4 requests of 16 to 64 on up to 1000 tokens
  // at D = 128: 30.7 us with 384, 22.4 so).
  static constexpr int kMinPart = D == 256 ? 384 : D == 128 ? 128 : 320;
  static constexpr int kQ = kPair ? 0 : 128 * D * 2;   // bytes of a tile's queries
  static constexpr int kOutRow = D == 64 ? 128 : 64;  // bytes of each row of results that pass shared memory at a time
  static constexpr int kStage = 32 * kOutRow;          // of a softmax warp, for its results on their way out
  static constexpr int kSmem =
      1024 + kNT * kQ + kStages * kTile + kRawStages * kRaw + 8 * kStage + (kPair ? 1024 : 0) + 512;
  // TMEM columns: S_t at t * 128, P_t at kP + t * kPStep, O_t at kO + t * D. At D = 128 they fill all 512 columns
  // with P_t over S_t, so that the next S_t waits for P_t's product, and so they do at D = 256 with the queries; at
  // D = 64 P_t has a place of its own, and the next S_t is made while the softmax works on this one.
  static constexpr bool kOwnP = D == 64;
  static constexpr uint32_t kP = kOwnP ? 256 : 0, kPStep = kOwnP ? 64 : 128;
  // At D = 256 one tile has to hide its own softmax: S and P are doubled, so that the scores of the next unit are made
  // before this one's products, and weights can be written while the last ones are used.
  static constexpr int kBufs = D == 256 ? 2 : 1;
  static constexpr uint32_t kBuf = 64;  // columns from one buffer of S and P to the next
  static constexpr uint32_t kO = D == 64 ? 384 : 256;
  // At D = 128 the tiles' softmaxes take turns: left alone they fall into step, share the special function units and
  // then leave the tensor pipe idle together (2048 queries after 14336 tokens, 32 heads on 8: 388 us, without turns 461).
  // At D = 64 the softmax is the bound and turns only add waits (the same with 16 heads on 4: 148 us, with turns 182).
  static constexpr bool kTurns = D == 128;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(Tc8Shape<D>::kThreads, 1)
    k_attn8_tc(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v) {
  using Sh = Tc8Shape<D>;
  constexpr int NT = Sh::kNT, BN = Sh::kBN, ST = Sh::kStages, T = 128 * NT;
  using W = Walk<T, BN, Sh::kTileCost, NT>;
  constexpr int SR = Sh::kRawStages;
  constexpr uint32_t kTile = Sh::kTile;
  constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | (8u << 24);  // f16 operands, fp32 sums
  constexpr uint32_t kIdescO =
      (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* skv = smem + NT * Sh::kQ;
  uint8_t* sraw = skv + ST * kTile;
  uint8_t* sout = sraw + SR * Sh::kRaw;
  uint64_t* full = reinterpret_cast<uint64_t*>(sout + 8 * Sh::kStage + (Sh::kPair ? 1024 : 0));
  uint64_t* empty = full + ST;
  uint64_t* raw_full = empty + ST;
  uint64_t* raw_empty = raw_full + SR;
  uint64_t* q_full = raw_empty + SR;   // per tile: queries are in shared memory
  // per tile and buffer of S and P (one barrier each, so that none is ever two phases ahead of a waiting warp):
  constexpr int NB = NT * Sh::kBufs;
  uint64_t* s_full = q_full + NT;      // scores are in TMEM
  uint64_t* p_full = s_full + NB;      // and half of the unit: weights are in TMEM, O is rescaled
  uint64_t* o_full = p_full + 2 * NB;  // the product with V is done
  uint64_t* s_free = o_full + NB;      // the softmax has read the scores (kOwnP)
  uint64_t* turn = s_free + NB;        // per tile: the other tile's warps have made their weights
  uint64_t* part_full = turn + NT;     // ring of parts
  uint64_t* part_empty = part_full + kParts;
  uint64_t* drained = part_empty + kParts;
  // kPair, per warpgroup and warp: the row maxima after a unit, and the row sums, can be read; the part is written out
  uint64_t* m_full = drained + 1;
  uint64_t* l_full = m_full + 8;
  uint64_t* written = l_full + 8;
  uint64_t* q_tmem = written + 8;  // the queries are in TMEM
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(Sh::kPair ? q_tmem + 1 : drained + 1);
  __shared__ alignas(8) uint64_t scale_full[kScales];
  __shared__ UnitScale scales[kScales];
  __shared__ int warp_sums[Sh::kThreads / 32];
  __shared__ Part parts[kParts];
  __shared__ LineStart first;

  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  constexpr int kMmaWarp = 8, kTmaWarp = 9, kWalkWarp = 10, kMmaWarp1 = 11, kConvert = 12;
  if (threadIdx.x == 32) {
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 4);    // the converting warps
      mbar_init(&empty[i], NT);  // a commit by each warp that uses the entry
    }
    for (int i = 0; i < SR; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < kScales; ++i) mbar_init(&scale_full[i], 1);
    for (int i = 0; i < NT; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&turn[i], 4);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&s_free[i], 4);
    }
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&part_full[i], 1);
      mbar_init(&part_empty[i], 8 + 3 + 4);
    }
    mbar_init(drained, 2);
    for (int i = 0; Sh::kPair && i < 24; ++i) mbar_init(&m_full[i], 1);
    if constexpr (Sh::kPair) mbar_init(q_tmem, 8);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  pdl_wait();
  pdl_launch();  // the join may be scheduled; it waits for this kernel's end
  uint32_t err = 0;

  tc_fence_before();
  find_start<W, Sh::kThreads>(a, Sh::kMinPart, first, warp_sums);
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_base);
  // unit j of a tile uses buffer j % kBufs for the (j / kBufs)-th time
  auto buf_of = [](int j) { return j % Sh::kBufs; };
  auto turn_of = [](int j) { return (j / Sh::kBufs) & 1; };
  bool ok = true;
  int at = 0;  // parts taken from the ring
  // the next part of the ring into registers; false: no more (or a wait gave up)
  auto take = [&](Part& g) {
    const int i = at % kParts;
    ok = ok && warp_wait(&part_full[i], (at / kParts) & 1);
    if (!ok) return false;
    g = parts[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&part_empty[i]);
    ++at;
    return g.n_all >= 0;
  };
  // The softmax threads hold a row of scores: they take registers from the other warps (256 x 208 + 256 x 48 = 512 x 128,
  // what the block was launched with).
  if (warp >= kMmaWarp) {
    set_regs_dec<48>();
    if (warp == kTmaWarp) {
      // ---- K and V tiles as they lie: for every unit, ring entry e holds K and entry e + 1 its V ----
      int e = 0, issued = 0;
      UnitScale us = {};
      Part g;
      while (ok && take(g)) {
        Request r;
        r.row = g.row;
        r.base = g.base;
        int2 place = make_int2(0, 0);
        for (int k = 0; k < g.n_all && ok; ++k, e += 2) {
          if ((k & 31) == 0 && k + lane < g.n_all) {
            const int tok = (g.u0 + k + lane) * BN;
            place = page_place(a, r, tok / kPage, err);
            place.y += tok % kPage;
            us = unit_scale(a, place.x, g.h);
          }
          const UnitScale u1 = {__shfl_sync(0xffffffffu, us.k, k & 31), __shfl_sync(0xffffffffu, us.log_v, k & 31),
                                __shfl_sync(0xffffffffu, us.inv_v, k & 31)};
          const int pw = __shfl_sync(0xffffffffu, place.x, k & 31), py = __shfl_sync(0xffffffffu, place.y, k & 31);
          if (lane == 0) {
#pragma unroll
            for (int which = 0; which < 2; ++which) {
              const int st = (e + which) % SR;
              if (ok && e + which >= SR) ok = mbar_wait(&raw_empty[st], ((e + which) / SR - 1) & 1);
              if (!ok) break;
              if (which == 0) {
                scales[(e / 2) % kScales] = u1;
                mbar_arrive(&scale_full[(e / 2) % kScales]);
              }
              mbar_expect_tx(&raw_full[st], Sh::kRaw);
              tma_load_4d(sraw + st * Sh::kRaw, which ? &map_v : &map_k, 0, py, g.h, pw, &raw_full[st]);
              issued = e + which + 1;
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
      }
      // leave only when every copy has landed (they have, unless a wait gave up)
      if (lane == 0) {
        for (int i = max(0, issued - SR); i < issued; ++i) ok &= mbar_wait(&raw_full[i % SR], (i / SR) & 1);
        if (!ok) err |= TQ_DEV_ERR_TIMEOUT;
      }
      if (err && a.status) atomicOr(a.status, err);
    } else if (warp == kMmaWarp || warp == kMmaWarp1) {
      // ---- products of tile t, or of one tile its scores and its sums ----
      const int t = NT == 2 && warp == kMmaWarp1;
      const bool does_s = NT == 2 || warp == kMmaWarp, does_o = NT == 2 || warp == kMmaWarp1;
      const bool leader = elect_one();
      const uint32_t q_lo = umma_desc_sw128_lo(smem_u32(smem)) + t * (Sh::kQ >> 4), kv_lo = smem_u32(skv) >> 4;
      const uint32_t sd = tmem + t * 128, pa = tmem + Sh::kP + t * Sh::kPStep, od = tmem + Sh::kO + t * D;
      int e = 0;       // ring entry of the unit's K
      int made = 0;    // units whose products are issued
      int loaded = 0;  // query tiles taken
      // S_t = Q_t K^T of unit j from ring entry `entry`, or nothing; the entry is given back either way, once it has been
      // filled. Where S_t goes, the scores of unit j - kBufs have been read, and with P_t over them, used.
      auto scores = [&](int entry, bool wanted, int j) {
        const int st = entry % ST, before = j - Sh::kBufs;
        ok = ok && warp_wait(&full[st], (entry / ST) & 1);
        if (wanted && before >= 0)
          ok = ok && warp_wait((Sh::kOwnP ? s_free : o_full) + t * Sh::kBufs + buf_of(before), turn_of(before));
        if (!ok) return;
        tc_fence_after();
        if (leader) {
          if (wanted) {
            const uint32_t ka = kv_lo + st * (kTile >> 4) + (1u << 16);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const uint32_t step = (i & 3) * 2;
              const uint32_t kb = ka + (i >> 2) * (BN * 128 >> 4) + step;
              if constexpr (Sh::kPair) umma_ts_lo(sd + buf_of(j) * Sh::kBuf, tmem + kTmemQ + i * 8, kb, kIdescS, i > 0);
              else umma_bf16_lo(sd, q_lo + (i >> 2) * 1024 + step, kb, kIdescS, i > 0);
            }
            umma_commit(&s_full[t * Sh::kBufs + buf_of(j)]);
          }
          umma_commit(&empty[st]);
        }
      };
      Part g;
      while (ok && take(g)) {
        const int n_all = uniform(g.n_all), n = uniform(t == 0 ? g.n_of[0] : g.n_of[NT - 1]);
        const int kv = uniform(g.kv), u0 = uniform(g.u0);
        if (n_all == 0) continue;
        if (does_s) {
          if (n > 0) {
            ok = warp_wait(Sh::kPair ? q_tmem : &q_full[t], loaded & 1);
            ++loaded;
          }
          scores(e, n > 0, made);
        }
        for (int k = 0; k < n_all && ok; ++k, e += 2) {
          if ((Sh::kOwnP || Sh::kPair) && does_s && k + 1 < n_all) scores(e + 2, k + 1 < n, made + 1);
          if (!does_o) {
            made += k < n;
            continue;
          }
          const int vs = (e + 1) % ST;
          ok = ok && warp_wait(&full[vs], ((e + 1) / ST) & 1);
          if (!ok) break;
          // the unit that the sequence ends in: the steps of 16 tokens behind it are left out
          const int valid = min(BN, kv - (u0 + k) * BN), steps = (valid + 15) / 16;
          if (k < n) {
            // MN-major operand: 64-channel blocks BN x 128 bytes apart, 8-token groups 1024 bytes apart
            const uint32_t va = kv_lo + vs * (kTile >> 4) + ((uint32_t)(BN * 128 >> 4) << 16);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              ok = ok && warp_wait(&p_full[2 * (t * Sh::kBufs + buf_of(made)) + half], turn_of(made));
              if (!ok) break;
              tc_fence_after();
              if (leader) {
#pragma unroll
                for (int i = half * (BN / 32); i < (half + 1) * (BN / 32); ++i)
                  if (i < steps) umma_ts_lo(od, pa + buf_of(made) * Sh::kBuf + i * 8, va + i * (2048 >> 4), kIdescO, k > 0 || i > 0);
              }
            }
            if (!ok) break;
            if (leader) umma_commit(&o_full[t * Sh::kBufs + buf_of(made)]);
            ++made;
          }
          if (leader) umma_commit(&empty[vs]);
          if (!Sh::kOwnP && !Sh::kPair && k + 1 < n_all) scores(e + 2, k + 1 < n, made);
        }
      }
      // leave only when every product is done
      if (leader) umma_commit(drained);
      const bool done = warp_wait(drained, 0);
      if ((!ok || !done) && lane == 0 && a.status) atomicOr(a.status, TQ_DEV_ERR_TIMEOUT);
    } else if (warp == kWalkWarp && lane == 0) {
      // ---- the parts of this CTA, in order ----
      W w;
      w.start(a, first);
      CutTile cut = {};
      for (bool more = true; more;) {
        Part g = {};
        more = w.next(a, g, cut);
        const int i = at % kParts;
        if (at >= kParts) ok = mbar_wait(&part_empty[i], (at / kParts - 1) & 1);
        if (!ok) break;
        parts[i] = g;
        mbar_arrive(&part_full[i]);
        ++at;
      }
      cut_tiles(a)[blockIdx.x] = cut;
      if (!ok && a.status) atomicOr(a.status, TQ_DEV_ERR_TIMEOUT);
    } else if (warp >= kConvert) {
      // ---- e4m3 to f16: a thread takes 16 channels of a token at a time ----
      constexpr int kPer = D / 16, kTake = Sh::kRaw / 16 / 128, kRows = 128 / kPer;  // rows of one step of all threads
      const int id = threadIdx.x - kConvert * 32, c = id % kPer;
      const int to = (c >> 2) * (BN * 128) + id / kPer * 128;  // steps are multiples of 8 rows: one place in the swizzle
      // lanes of every second 64 channels write their second half first: no bank conflicts
      const bool odd = (c >> 2) & 1;
      const uint32_t x_at = ((((c & 3) * 2 + odd) ^ (id / kPer)) & 7) << 4;
      int e = 0;
      Part g;
      while (ok && take(g)) {
        for (int k = 0; k < g.n_all && ok; ++k) {
          const int valid = g.kv - (g.u0 + k) * BN;
#pragma unroll 1
          for (int which = 0; which < 2; ++which, ++e) {
            const int rs = e % SR, fs = e % ST;
            ok = warp_wait(&raw_full[rs], (e / SR) & 1);
            if (ok && e >= ST) ok = warp_wait(&empty[fs], (e / ST - 1) & 1);
            if (!ok) break;
            const uint8_t* src = sraw + rs * Sh::kRaw + id * 16;
            uint8_t* dst = skv + fs * kTile + to;
#pragma unroll
            for (int i0 = 0; i0 < kTake; i0 += 4) {  // loads in flight
              uint4 v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(src + (i0 + i) * 2048);
              if (which && valid < BN) {  // rows behind the sequence: 0 x NaN is NaN
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (id / kPer + (i0 + i) * kRows >= valid) v[i] = make_uint4(0, 0, 0, 0);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t x0 = odd ? v[i].z : v[i].x, x1 = odd ? v[i].w : v[i].y;
                const uint32_t y0 = odd ? v[i].x : v[i].z, y1 = odd ? v[i].y : v[i].w;
                uint8_t* p = dst + (i0 + i) * (kRows * 128);
                *reinterpret_cast<uint4*>(p + x_at) = make_uint4(e4m3_lo(x0), e4m3_hi(x0), e4m3_lo(x1), e4m3_hi(x1));
                *reinterpret_cast<uint4*>(p + (x_at ^ 16)) = make_uint4(e4m3_lo(y0), e4m3_hi(y0), e4m3_lo(y1), e4m3_hi(y1));
              }
            }
            fence_async_smem();
            __syncwarp();
            // The raw entry is given back here and not behind its loads: those had been issued, but not all had returned, when
            // TMA wrote the next tile there (a tile in 50 had rows of the next one).
            if (lane == 0) {
              mbar_arrive(&raw_empty[rs]);
              mbar_arrive(&full[fs]);
            }
          }
        }
      }
      if (!ok && lane == 0 && a.status) atomicOr(a.status, TQ_DEV_ERR_TIMEOUT);
    }
  } else {
    set_regs_inc<208>();
    // ---- softmax of tile t: a thread per row (kPair: of every other unit) ----
    constexpr bool kPair = Sh::kPair;
    const int wg = warp >> 2, t = kPair ? 0 : wg, row_t = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const uint32_t ts = tmem + t * 128 + lanes, tp = tmem + Sh::kP + t * Sh::kPStep + lanes;
    const uint32_t to = tmem + Sh::kO + t * D + lanes;
    int made = 0;
    int turns = 0;  // units that both tiles have made
    Part g = {};
    // a part's queries, a row per thread, in f16 with a power of two taken out of each bf16 row, into shared memory as a
    // K-major operand, with zeros in rows past the last; with kPair into TMEM, half of the channels by each warpgroup
    float back = a.scale_log2;  // what the scores are multiplied with
    auto load_q = [&] {
      if ((t == 0 ? g.n_of[0] : g.n_of[NT - 1]) == 0) return;
      const int f = g.f0 + t * 128 + row_t, fq = min(f, g.rows - 1), qi = a.div_g(fq), head = g.h * a.G + fq - qi * a.G;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (int64_t)(g.q0 + qi) * a.q_row +
                                                        (int64_t)head * a.q_head);
      float by = 1.f;
      if constexpr (BF16) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint4 v = __ldg(src + i);
          top = max(max(top, max(v.x & 0x7fffu, (v.x >> 16) & 0x7fffu)), max(v.y & 0x7fffu, (v.y >> 16) & 0x7fffu));
          top = max(max(top, max(v.z & 0x7fffu, (v.z >> 16) & 0x7fffu)), max(v.w & 0x7fffu, (v.w >> 16) & 0x7fffu));
        }
        by = to_f16_by(top);
        back = a.scale_log2 * to_f16_back(top);
      }
      auto chunk = [&](int i) {
        uint4 v = __ldg(src + i);
        if constexpr (BF16)
          v = make_uint4(bf16x2_to_f16x2(v.x, by), bf16x2_to_f16x2(v.y, by), bf16x2_to_f16x2(v.z, by), bf16x2_to_f16x2(v.w, by));
        return v;
      };
      if constexpr (kPair) {
#pragma unroll 1
        for (int x = wg * (D / 128); x < (wg + 1) * (D / 128); ++x) {  // 64 channels
          uint32_t r[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 v = chunk(x * 8 + i);
            r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
          }
          tmem_st32(tmem + lanes + kTmemQ + x * 32, r);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_tmem);
      } else {
#pragma unroll 8
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<uint4*>(smem + t * Sh::kQ + (i >> 3) * 16384 + row_t * 128 + (((i & 7) ^ (row_t & 7)) << 4)) =
              f < g.rows ? chunk(i) : make_uint4(0, 0, 0, 0);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
      }
    };
    // kPair: the other warpgroup has the same rows in its warp of the same rank. A unit's maxima go from one to the other
    // (through their owner's stage, which is free until the part is written out), so that O has one scale; the sums
    // stay apart until the part's end.
    const int mine8 = warp, other8 = warp ^ 4;
    float2* const m_own = reinterpret_cast<float2*>(sout + warp * Sh::kStage) + lane;
    const float2* const m_other = reinterpret_cast<const float2*>(sout + other8 * Sh::kStage) + lane;
    float* const l_all = reinterpret_cast<float*>(sout + 8 * Sh::kStage) + row_t;  // [2][128]
    int ends = 0;   // parts written out
    int units = 0;  // units of the parts before
    bool have = take(g);
    if (have) load_q();
    while (have && ok) {
      if (kPair && ends > 0) {  // O can be written again, and what the warpgroups exchange
        ok = warp_wait(&written[other8], (ends - 1) & 1);
        if (!ok) break;
        tc_fence_after();
      }
      const int n = t == 0 ? g.n_of[0] : g.n_of[NT - 1];
      const int f = g.f0 + t * 128 + row_t;
      const bool mine = f < g.rows;
      const int qi = mine ? a.div_g(f) : 0;
      Request r;
      r.n_q = g.n_q;
      r.kv = g.r_kv;
      const int lim = mine ? seen(a, r, qi) : 0;
      // what every row of the tile sees needs no mask; rows past the last may hold anything
      const int lim_all = seen(a, r, a.div_g(min(g.f0 + t * 128, g.rows - 1)));
      const int u0 = g.u0;
      const int both = Sh::kTurns ? min(g.n_of[0], g.n_of[NT - 1]) : 0;
      float m = mine ? -INFINITY : kFarLifted, l = 0.f;  // a row past the last never outgrows its maximum (or does so for nothing)
      float mv = 0.f;            // m's part of the values' scale: weights are 2^(s - m + log2 vs - mv)
      float ml = m, mlv = 0.f;   // what l is relative to (kPair; else m)
      for (int k = kPair ? (made ^ wg) & 1 : 0; k < n; k += kPair ? 2 : 1) {
        const int j = made + k, bi = t * Sh::kBufs + buf_of(j);
        ok = warp_wait(&s_full[bi], turn_of(j)) && warp_wait(&scale_full[(units + k) % kScales], ((units + k) / kScales) & 1);
        if (!ok) break;
        const UnitScale us = scales[(units + k) % kScales];
        const float scale = fmaxf(back * us.k, 1.17549435e-38f);  // above 0: times -inf it is that
        tc_fence_after();
        // the other tile's weights are made: now this one has the special function units, and that one the tensor pipe
        if (k < both && (t == 1 || turns > 0)) {
          ok = warp_wait(&turn[t], (t == 1 ? turns : turns - 1) & 1);
          if (!ok) break;
        }
        float s[BN];
#pragma unroll
        for (int c = 0; c < BN; c += 32) tmem_ld32_async(ts + buf_of(j) * Sh::kBuf + c, s + c);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < BN; c += 32) tie32(s + c);
        if constexpr (Sh::kOwnP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[bi]);
        }
        const int base = (u0 + k) * BN;
        if (base + BN > lim_all) {
          const int left = lim - base;
#pragma unroll
          for (int c = 0; c < BN; ++c) s[c] = c < left ? s[c] : -INFINITY;
        }
        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < BN - 4; c += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) top[i] = max3(top[i], s[c + i], s[c + 4 + i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], s[BN - 4 + i]);
        const float mx = fmaxf(max3(top[0], top[1], top[2]), top[3]) * scale;
        if (kPair && k > 0) {
          ok = warp_wait(&m_full[other8], turn_of(j - 1));
          if (!ok) break;
          m = m_other->x;
          mv = m_other->y;
        }
        // the sum of both maxima's parts may outgrow theirs; far scores have no room for the logarithm, so it stays apart
        const bool more = (mx - m) + (us.log_v - mv) > kLazy;  // also where m is -inf and mx is not
        const float mn = more ? mx : m, mvn = more ? us.log_v : mv;
        if constexpr (kPair) {
          *m_own = make_float2(mn, mvn);
          __syncwarp();
          if (lane == 0) mbar_arrive(&m_full[mine8]);
          if (mn != ml || mvn != mlv) l = rescaled(l, (ml - mn) + (mlv - mvn));
          ml = mn;
          mlv = mvn;
        }
        const bool grew = more && m != -INFINITY;
        const float mu = mn == -INFINITY ? 0.f : mn, own = us.log_v - mvn, held = least_above(own, mx - mn), above = held + kLift;
        const float inv_v = held == own ? us.inv_v : exp2_fast(-(held + mvn));
        const bool far = fabsf(mu) > kFarLifted;
        const bool special = __any_sync(0xffffffffu, grew || far);
        // O_t is whole before it is rescaled, and P_t has been used before it is written again
        const int last = special ? j - 1 : Sh::kOwnP ? j - Sh::kBufs : -1;
        if (last >= 0) {
          ok = warp_wait(&o_full[t * Sh::kBufs + buf_of(last)], turn_of(last));
          if (!ok) break;
          tc_fence_after();
        }
        if (special) {
          if (__any_sync(0xffffffffu, grew)) {
            const float by = grew ? (m - mn) + (mv - mvn) : 0.f, alpha = exp2_fast(by);
            if constexpr (!kPair) l = rescaled(l, by);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(to + c, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(to + c, o);
            }
          }
        }
        // s * scale - mu in one rounding is off by what mu was rounded by, the same for all tokens of the row. Past kFarLifted it would
        // leave the weights' range: there the scores are rounded as mu was, and then taken from it.
        const bool by_steps = special && __any_sync(0xffffffffu, far);
        if (by_steps) {
#pragma unroll
          for (int c = 0; c < BN; ++c) s[c] = __fsub_rn(__fmul_rn(s[c], scale), mu) + above;
        }
        m = mn;
        mv = mvn;
        const float from = by_steps ? 0.f : above - mu;
        const float by = by_steps ? 1.f : scale;
        const float2 sc = make_float2(by, by), off = make_float2(from, from);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // the product with the first half of V starts while the second is made
#pragma unroll
          for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 y = fma2(make_float2(s[c + 2 * i], s[c + 2 * i + 1]), sc, off);
              y.x = exp2_fast(y.x);
              y.y = exp2_fast(y.y);
              sum[i & 1] = add2(sum[i & 1], y);
              p[i] = pack2<false>(y.x, y.y);
            }
            tmem_st16(tp + buf_of(j) * Sh::kBuf + c / 2, p);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * bi + half]);
        }
        if (k < both) {
          if (lane == 0) mbar_arrive(&turn[1 - t]);
          ++turns;
        }
        const float2 all = add2(sum[0], sum[1]);
        l += (all.x + all.y) * inv_v;
      }
      if (!ok) break;
      made += n;
      units += g.n_all;
      if constexpr (kPair) {  // for parts without a unit too: a barrier must not run ahead of the other's wait by two phases
        if (n > 0 && ((made - 1) & 1) != wg) {
          ok = warp_wait(&m_full[other8], turn_of(made - 1));
          if (!ok) break;
          tc_fence_after();
          m = m_other->x;
          mv = m_other->y;
          if (m != ml || mv != mlv) l = rescaled(l, (ml - m) + (mlv - mv));
        }
        l_all[wg * 128] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_full[mine8]);
        ok = warp_wait(&l_full[other8], ends & 1);
        if (!ok) break;
        l = l_all[0] + l_all[128];
      }
      // where this part's result goes; then the next tile's queries, so that its scores are made under the end of
      // this one
      const bool direct = g.direct;
      const float2 part = part_reference(m, mv, l);
      const float inv = direct ? (l > 0.f ? 1.f / l : 0.f) : part.y;
      // the rows of the warp's 32 that go out by this lane: 16 bytes of each piece of row (i 32 + lane) / kLanes
      constexpr int kLanes = Sh::kOutRow / 16;
      int64_t to_row[kLanes];
      uint32_t rows_out = 0;
#pragma unroll
      for (int i = 0; i < kLanes; ++i) {
        const int row = (warp & 3) * 32 + (i * 32 + lane) / kLanes, fr = g.f0 + t * 128 + row;
        if (fr < g.rows) rows_out |= 1u << i;
        const int q = a.div_g(min(fr, g.rows - 1));
        to_row[i] = direct ? (int64_t)(g.q0 + q) * a.o_row + (int64_t)(g.h * a.G + min(fr, g.rows - 1) - q * a.G) * a.o_head
                           : (int64_t)(t * 128 + row) * D;
      }
      float* po = cut_o<T, D>(a, gridDim.x, blockIdx.x, g.slot);
      if (!direct && (!kPair || wg == 0)) cut_ml<T>(a, gridDim.x, blockIdx.x, g.slot)[t * 128 + row_t] = make_float2(part.x, l * inv);
      have = take(g);
      if (!ok) break;
      if (have) load_q();
      if (!ok) break;
      if (n > 0) {
        ok = warp_wait(&o_full[t * Sh::kBufs + buf_of(made - 1)], turn_of(made - 1));
        if (!ok) break;
        tc_fence_after();
      }
      // Through shared memory, kOutRow bytes of each row at a time, so that a store of the warp covers whole pieces of rows.
      uint8_t* stage = sout + warp * Sh::kStage;
      auto piece = [&](const uint4 (&v)[kLanes], int c) {  // columns from c on: 16-bit results, fp32 sums
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kLanes; ++i)
          *reinterpret_cast<uint4*>(stage + lane * Sh::kOutRow + ((i ^ (lane * kLanes / 8 & (kLanes - 1))) << 4)) = v[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kLanes; ++i) {
          const int row = (i * 32 + lane) / kLanes, j = lane % kLanes;
          const uint4 x = *reinterpret_cast<const uint4*>(stage + row * Sh::kOutRow + ((j ^ (row * kLanes / 8 & (kLanes - 1))) << 4));
          if (!(rows_out >> i & 1)) continue;
          if (direct) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + to_row[i] + c + j * 8) = x;
          else *reinterpret_cast<uint4*>(po + to_row[i] + c + j * 4) = x;
        }
      };
      constexpr int kStep = Sh::kOutRow / 2;  // columns of 16-bit results in a piece
#pragma unroll 1
      for (int c = kPair ? wg * (D / 2) : 0; c < (kPair ? (wg + 1) * (D / 2) : D); c += kStep) {
        uint4 v[kLanes];
#pragma unroll
        for (int x = 0; x < kStep / 32; ++x) {
          float o[32];
          __syncwarp();
          if (n > 0) {
            tmem_ld32_async(to + c + 32 * x, o);
            tmem_wait_ld();
            tie32(o);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = n > 0 ? o[i] * inv : 0.f;
          if (direct) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[4 * x + i] = make_uint4(result2<BF16>(o[8 * i], o[8 * i + 1]), result2<BF16>(o[8 * i + 2], o[8 * i + 3]),
                                        result2<BF16>(o[8 * i + 4], o[8 * i + 5]), result2<BF16>(o[8 * i + 6], o[8 * i + 7]));
          } else {
#pragma unroll
            for (int h = 0; h < 8 / kLanes; ++h) {
#pragma unroll
              for (int i = 0; i < kLanes; ++i) {
                const float* p = o + (h * kLanes + i) * 4;
                v[i] = make_uint4(__float_as_uint(p[0]), __float_as_uint(p[1]), __float_as_uint(p[2]), __float_as_uint(p[3]));
              }
              piece(v, c + 32 * x + h * kLanes * 4);
            }
          }
        }
        if (direct) piece(v, c);
      }
      tc_fence_before();
      if constexpr (kPair) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&written[mine8]);
        ++ends;
      }
    }
    if (!ok && lane == 0 && a.status) atomicOr(a.status, TQ_DEV_ERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
  }
}

template <int D, bool BF16>
cudaError_t launch_tc8_as(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, cudaStream_t s) {
  using Sh = Tc8Shape<D>;
  static std::atomic<uint64_t> known{0};
  cudaError_t e = allow_smem(k_attn8_tc<D, BF16>, Sh::kSmem, known);
  if (e == cudaSuccess)
    e = launch_pdl(k_attn8_tc<D, BF16>, dim3(p.ctas), dim3(Sh::kThreads), Sh::kSmem, s, a, m.k, m.v);
  if (e != cudaSuccess) return e;
  return launch_join<D, 128 * Sh::kNT, BF16>(a, p.ctas, p.max_rows, s);
}

template <int D>
AttnShape tc8_shape(int sms) {
  using Sh = Tc8Shape<D>;
  return {128 * Sh::kNT, Sh::kBN, sms, cta_bytes(128 * Sh::kNT, D), Sh::kTileCost, Sh::kMinPart};
}

}  // namespace

AttnShape attn8_tc_shape(int d, int sms) { return d == 64 ? tc8_shape<64>(sms) : d == 128 ? tc8_shape<128>(sms) : tc8_shape<256>(sms); }

cudaError_t launch_attn8_tc(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, int dtype, cudaStream_t s) {
  if (dtype == TQ_BF16)
    return d == 64    ? launch_tc8_as<64, true>(a, m, p, s)
           : d == 128 ? launch_tc8_as<128, true>(a, m, p, s)
                      : launch_tc8_as<256, true>(a, m, p, s);
  return d == 64    ? launch_tc8_as<64, false>(a, m, p, s)
         : d == 128 ? launch_tc8_as<128, false>(a, m, p, s)
                    : launch_tc8_as<256, false>(a, m, p, s);
}

}  // namespace tq
