// Attention of chunks of new tokens over an exact cache or an encoder's states, on the tensor cores (tcgen05).
#include "tq_attention_tc.cuh"

namespace tq {
namespace {

// =============================================================================================
// k_attn_tc: a CTA takes its part of the line; at a time NT tiles of 128 rows (query, head of the group) of one request
// and KV head, over their tokens or the part of them that is its own. The rows of a group share K and V, so a tile is full at any group size.
//   - a TMA warp keeps a ring of K and V tiles (BN tokens) in flight, in the 128-byte swizzle;
//   - two MMA warps issue S_t = Q_t K^T into TMEM, and O_t += P_t V with P_t read from TMEM and V taken as it lies
//     (tokens x channels, the MN-major operand form): one per tile, or where there is one tile, one for the scores and
//     one for the sums, so that one's waits do not hold up the other's products;
//   - a warpgroup per tile reads S_t (a thread per row, so row sums need no exchange), writes P_t = 2^(s - m) in 16
//     bits over it, and rescales O_t only where a row's maximum grew by more than 2^8: the weights stay below
//     2^8, far inside fp32 and f16, and the final division takes the factor out.
// The two tiles alternate: while one's softmax runs, the tensor pipe works for the other. One tile has both warpgroups:
// they take its units in turn and hand each row's maximum on through shared memory; row sums meet at the end.
// Measured (GB300, bf16, calls back to back on one input of random values; the ranges are of several boxes), 32 query heads
// on 8 KV heads, head_dim 128: 8192 queries on 8192 tokens without a mask 618 to 632 us, 1740 to 1780 TFLOP/s (91 to 93 % of
// a measured cuBLAS burst); causal 338 to 368 us, 1495 to 1628; 2048 queries after 30720 tokens 629 to 646 us, 1650 to 1695
// (708 us where keys have strong channels and inputs change from call to call). A unit of both tiles takes 2500 cycles
// there, its four products 2048. Head_dim 64 is bound by the softmax, at 2 warps per scheduler: a unit takes 2290 cycles, its
// products 1024 (8192 x 8192, 16 heads: 254 us, 1083 TFLOP/s without a mask; causal 144.5 us, 951). Head_dim 256 is bound by
// K and V, which pass shared memory for 128 rows only: 64 KB a unit, whose products take 1024 cycles and which takes about
// 1750 (4096 x 4096, 16 heads on 4: 204 us, 1350 TFLOP/s without a mask; causal 123 to 126 us, 1090 to 1120; 2048 queries
// after 14336 tokens 345 to 372 us, 1385 to 1490).
// =============================================================================================
// kPair: the queries are an operand in TMEM, in these columns. From shared memory, 64 tokens' scores would read 64 KB of
// them in 512 cycles, beside 32 KB of K, 32 KB of V and 64 KB that arrive (2048 queries after 14336 tokens: 376 us with
// the queries there, 345 so).
constexpr uint32_t kTmemQ = 128;
template <int D>
struct TcShape {
  static constexpr int kNT = D == 256 ? 1 : 2;     // tiles of 128 rows: TMEM holds S and O of two up to D = 128
  static constexpr int kBN = D == 256 ? 64 : 128;  // tokens of a K or V tile
  static constexpr int kTile = kBN * D * 2;        // its bytes
  static constexpr int kStages = D == 64 ? 8 : 4;  // 128 KB of K and V in flight
  // One tile's softmax is shared by two warpgroups that take its units in turn, each with a buffer of S and P of its own:
  // with one warp per scheduler it was the bound (2048 queries after 14336 tokens: 413 us, with two 376).
  static constexpr bool kPair = kNT == 1;
  static constexpr int kThreads = 384;
  // Start and end of a tile, in 64ths of a unit: 3 units of 128 tokens, 5 of 64 (4096 x 4096 causal at D = 256: 138 us
  // with 3 units, 123 with 5, 126 with 7). No CTA gets less than a tile of one unit costs: short work takes fewer CTAs.
  static constexpr int kTileCost = D == 256 ? 320 : 192;
  static constexpr int kMinPart = kTileCost + 64;
  static constexpr int kQ = 128 * D * 2;           // bytes of a tile's queries
  static constexpr int kStage = 4096;              // of a softmax warp, for its results on their way out
  static constexpr int kSmem = 1024 + kNT * kQ + kStages * kTile + 8 * kStage + (kPair ? 1024 : 0) + 512;
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
  // then leave the tensor pipe idle together (2900 cycles per unit against 2500; the SMs differed by 30 %). At D = 64
  // the softmax is the bound and turns only add waits (2290 cycles per unit without them, 2900 with).
  static constexpr bool kTurns = D == 128;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(TcShape<D>::kThreads, 1)
    k_attn_tc(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_q) {
  using Sh = TcShape<D>;
  constexpr int NT = Sh::kNT, BN = Sh::kBN, ST = Sh::kStages, T = 128 * NT;
  using W = Walk<T, BN, Sh::kTileCost, NT>;
  constexpr uint32_t kTile = Sh::kTile;
  constexpr uint32_t kType = BF16 ? 1u : 0u;
  constexpr uint32_t kIdescS = (1u << 4) | (kType << 7) | (kType << 10) | ((uint32_t)(BN >> 3) << 17) | (8u << 24);
  constexpr uint32_t kIdescO =
      (1u << 4) | (kType << 7) | (kType << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* skv = smem + NT * Sh::kQ;
  uint8_t* sout = skv + ST * kTile;
  uint64_t* full = reinterpret_cast<uint64_t*>(sout + 8 * Sh::kStage + (Sh::kPair ? 1024 : 0));
  uint64_t* empty = full + ST;
  uint64_t* q_full = empty + ST;       // per tile: queries are in shared memory
  uint64_t* q_empty = q_full + NT;     // per tile: their last scores are made (q_tma)
  // per tile and buffer of S and P (one barrier each, so that none is ever two phases ahead of a waiting warp):
  constexpr int NB = NT * Sh::kBufs;
  uint64_t* s_full = q_empty + NT;     // scores are in TMEM
  uint64_t* p_full = s_full + NB;      // and half of the unit: weights are in TMEM, O is rescaled
  uint64_t* o_full = p_full + 2 * NB;  // the product with V is done
  uint64_t* s_free = o_full + NB;      // the softmax has read the scores (kOwnP)
  uint64_t* v_clean = s_free + NB;     // per ring entry: V rows behind the sequence are zeroed
  uint64_t* turn = v_clean + ST;       // per tile: the other tile's warps have made their weights
  uint64_t* part_full = turn + NT;     // ring of parts
  uint64_t* part_empty = part_full + kParts;
  uint64_t* drained = part_empty + kParts;
  // kPair, per warpgroup and warp: the row maxima after a unit, and the row sums, can be read; the part is written out
  uint64_t* m_full = drained + 1;
  uint64_t* l_full = m_full + 8;
  uint64_t* written = l_full + 8;
  uint64_t* q_tmem = written + 8;  // the queries are in TMEM
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(Sh::kPair ? q_tmem + 1 : drained + 1);
  __shared__ int warp_sums[Sh::kThreads / 32];
  __shared__ Part parts[kParts];
  __shared__ LineStart first;

  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  constexpr int kMmaWarp = 8, kTmaWarp = 9, kWalkWarp = 10, kMmaWarp1 = 11;
  if (threadIdx.x == 32) {
    prefetch_map(&map_k);
    prefetch_map(&map_v);
    if (a.q_tma) prefetch_map(&map_q);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], NT);  // a commit by each warp that uses the entry
      mbar_init(&v_clean[i], 1);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(&q_full[i], a.q_tma ? 1 : 4);
      mbar_init(&q_empty[i], Sh::kPair ? 8 : 1);
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
      mbar_init(&part_empty[i], 8 + 3);
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
  // The softmax threads hold a row of scores: they take registers from the other warps (8 x 32 x 216 + 4 x 32 x 72 =
  // 384 x 168, what the block was launched with).
  if (warp >= kMmaWarp) {
    set_regs_dec<72>();
    if (warp == kTmaWarp) {
      // ---- K and V tiles: for every unit, ring entry e holds K and entry e + 1 its V ----
      int e = 0, issued = 0;
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
          }
          const int pw = __shfl_sync(0xffffffffu, place.x, k & 31), py = __shfl_sync(0xffffffffu, place.y, k & 31);
          if (lane == 0) {
#pragma unroll
            for (int which = 0; which < 2; ++which) {
              const int st = (e + which) % ST;
              if (ok && e + which >= ST) ok = mbar_wait(&empty[st], ((e + which) / ST - 1) & 1);
              if (!ok) break;
              uint8_t* dst = skv + st * kTile;
              mbar_expect_tx(&full[st], kTile);
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(dst + c * (BN * 128), which ? &map_v : &map_k, c * 64, py, g.h, pw, &full[st]);
              issued = e + which + 1;
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
      }
      // leave only when every copy has landed (they have, unless a wait gave up)
      if (lane == 0) {
        for (int i = max(0, issued - ST); i < issued; ++i) ok &= mbar_wait(&full[i % ST], (i / ST) & 1);
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
      uint32_t cleaned = 0;  // parities of v_clean: an entry is cleaned again only after this warp gave it back
      // S_t = Q_t K^T of unit j from ring entry `entry`, or nothing; the entry is given back either way, once it has been
      // filled. Where S_t goes, the scores of unit j - kBufs have been read, and with P_t over them, used.
      auto scores = [&](int entry, bool wanted, int j, bool last) {
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
            if (!Sh::kPair && last && a.q_tma) umma_commit(&q_empty[t]);
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
          scores(e, n > 0, made, n == 1);
        }
        for (int k = 0; k < n_all && ok; ++k, e += 2) {
          if ((Sh::kOwnP || Sh::kPair) && does_s && k + 1 < n_all) scores(e + 2, k + 1 < n, made + 1, k + 2 == n);
          if (!does_o) {
            made += k < n;
            continue;
          }
          const int vs = (e + 1) % ST;
          ok = ok && warp_wait(&full[vs], ((e + 1) / ST) & 1);
          if (!ok) break;
          // the unit that the sequence ends in: V rows behind it are zeroed up to the next step of 16 (0 x NaN is
          // NaN), and the steps behind them are left out
          const int valid = min(BN, kv - (u0 + k) * BN), steps = (valid + 15) / 16;
          if (valid & 15) {
            if (t == 0) {
              const int rows16 = (16 - (valid & 15)) * (D / 8);
              for (int i = lane; i < rows16; i += 32) {
                const int c = i % (D / 8), row = valid + i / (D / 8);
                *reinterpret_cast<uint4*>(skv + vs * kTile + (c >> 3) * (BN * 128) + row * 128 + (c & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
              }
              fence_async_smem();
              __syncwarp();
              if (NT == 2 && lane == 0) mbar_arrive(&v_clean[vs]);
            } else {
              ok = warp_wait(&v_clean[vs], (cleaned >> vs) & 1);
              cleaned ^= 1u << vs;
            }
          }
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
          if (!Sh::kOwnP && !Sh::kPair && k + 1 < n_all) scores(e + 2, k + 1 < n, made, k + 2 == n);
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
      int loads[NT] = {};
      for (bool more = true; more;) {
        Part g = {};
        more = w.next(a, g, cut);
        const int i = at % kParts;
        if (at >= kParts) ok = mbar_wait(&part_empty[i], (at / kParts - 1) & 1);
        if (!ok) break;
        parts[i] = g;
        mbar_arrive(&part_full[i]);
        ++at;
        // its queries, once the last scores with the ones before them are made; rows past the last are other requests'
        // or zeros: their results are not written
        if (more && a.q_tma) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (g.n_of[t] == 0) continue;
            if (loads[t] > 0) ok = ok && mbar_wait(&q_empty[t], (loads[t] - 1) & 1);
            if (!ok) break;
            mbar_expect_tx(&q_full[t], Sh::kQ);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(smem + t * Sh::kQ + c * 16384, &map_q, c * 64, g.h * a.G, g.q0 + a.div_g(g.f0 + t * 128), &q_full[t]);
            ++loads[t];
          }
          if (!ok) break;
        }
      }
      // leave only when every copy has landed
      for (int t = 0; t < NT; ++t)
        if (loads[t] > 0) ok &= mbar_wait(&q_full[t], (loads[t] - 1) & 1);
      cut_tiles(a)[blockIdx.x] = cut;
      if (!ok && a.status) atomicOr(a.status, TQ_DEV_ERR_TIMEOUT);
    }
  } else {
    set_regs_inc<216>();
    // ---- softmax of tile t: a thread per row (kPair: of every other unit) ----
    constexpr bool kPair = Sh::kPair;
    constexpr float kPast = BF16 ? kFar : kFarLifted;
    const int wg = warp >> 2, t = kPair ? 0 : wg, row_t = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const uint32_t ts = tmem + t * 128 + lanes, tp = tmem + Sh::kP + t * Sh::kPStep + lanes;
    const uint32_t to = tmem + Sh::kO + t * D + lanes;
    int made = 0;
    int turns = 0;  // units that both tiles have made
    Part g = {};
    // a part's queries into shared memory, as a K-major operand, where they do not come by TMA (group sizes such as 3 or
    // 6), with zeros in rows past the last; with kPair into TMEM, from either place, where such rows repeat the last one
    // or hold what TMA brought
    int loaded = 0;  // query tiles in TMEM
    auto load_q = [&] {
      if constexpr (kPair) {  // each warpgroup half of the channels, from where TMA put them or from memory, into TMEM
        if (g.n_of[0] == 0) return;
        if (a.q_tma) ok = warp_wait(&q_full[0], loaded & 1);
        if (!ok) return;
        const int f = g.f0 + row_t, qi = a.div_g(min(f, g.rows - 1)), head = g.h * a.G + min(f, g.rows - 1) - qi * a.G;
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(g.q0 + qi) * a.q_row + (int64_t)head * a.q_head;
#pragma unroll 1
        for (int x = wg * (D / 128); x < (wg + 1) * (D / 128); ++x) {  // 64 channels
          uint32_t r[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 v = a.q_tma ? *reinterpret_cast<const uint4*>(smem + x * 16384 + row_t * 128 + ((i ^ (row_t & 7)) << 4))
                                    : __ldg(reinterpret_cast<const uint4*>(src + x * 64 + i * 8));
            r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
          }
          tmem_st32(tmem + lanes + kTmemQ + x * 32, r);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (a.q_tma) mbar_arrive(&q_empty[0]);
          mbar_arrive(q_tmem);
        }
        ++loaded;
        return;
      }
      if (a.q_tma || (t == 0 ? g.n_of[0] : g.n_of[NT - 1]) == 0) return;
      constexpr int kBatch = D == 64 ? 8 : 16;
      constexpr int kChunks = D / 8, kRowsStep = 128 / kChunks;  // 16-byte chunks of a row; rows of one step
      const int c = row_t % kChunks;
      for (int r0 = row_t / kChunks; r0 < 128; r0 += kBatch * kRowsStep) {
        uint4 v[kBatch];  // loads in flight
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int f = g.f0 + t * 128 + r0 + j * kRowsStep;
          v[j] = make_uint4(0, 0, 0, 0);
          if (f < g.rows) {
            const int qi = a.div_g(f), head = g.h * a.G + f - qi * a.G;
            v[j] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                        (int64_t)(g.q0 + qi) * a.q_row + (int64_t)head * a.q_head + c * 8));
          }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int row = r0 + j * kRowsStep;
          *reinterpret_cast<uint4*>(smem + t * Sh::kQ + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v[j];
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[t]);
    };
    // kPair: the other warpgroup has the same rows in its warp of the same rank. A unit's maxima go from one to the other
    // (through their owner's stage, which is free until the part is written out), so that O has one scale; the sums
    // stay apart until the part's end.
    const int mine8 = warp, other8 = warp ^ 4;
    float* const m_own = reinterpret_cast<float*>(sout + warp * Sh::kStage) + lane;
    const float* const m_other = reinterpret_cast<const float*>(sout + other8 * Sh::kStage) + lane;
    float* const l_all = reinterpret_cast<float*>(sout + 8 * Sh::kStage) + row_t;  // [2][128]
    int ends = 0;  // parts written out
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
      float m = mine ? -INFINITY : kPast, l = 0.f;  // a row past the last never outgrows its maximum (or does so for nothing)
      float ml = m;  // what l is relative to (kPair; else m)
      for (int k = kPair ? (made ^ wg) & 1 : 0; k < n; k += kPair ? 2 : 1) {
        const int j = made + k, bi = t * Sh::kBufs + buf_of(j);
        ok = warp_wait(&s_full[bi], turn_of(j));
        if (!ok) break;
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
        const float mx = fmaxf(max3(top[0], top[1], top[2]), top[3]) * a.scale_log2;
        if (kPair && k > 0) {
          ok = warp_wait(&m_full[other8], turn_of(j - 1));
          if (!ok) break;
          m = *m_other;
        }
        float mn = m;
        if (mx - m > kLazy || m == -INFINITY) mn = fmaxf(m, mx);  // a sum m + kLazy could round to more
        if constexpr (kPair) {
          *m_own = mn;
          __syncwarp();
          if (lane == 0) mbar_arrive(&m_full[mine8]);
          if (mn != ml) l *= exp2_fast(ml - mn);
          ml = mn;
        }
        const bool grew = mn != m && m != -INFINITY;
        float mu = mn == -INFINITY ? 0.f : mn;
        const bool far = fabsf(mu) > kPast;
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
            const float alpha = grew ? exp2_fast(m - mn) : 1.f;
            if constexpr (!kPair) l *= alpha;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(to + c, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(to + c, o);
            }
          }
          // s * scale - mu in one rounding is off by what mu was rounded by, the same for all tokens of the row. Past kPast
          // it would leave the weights' range: there the scores are rounded as mu was, and then taken from it.
          if (__any_sync(0xffffffffu, far)) {
            const float back = 1.f / a.scale_log2;
#pragma unroll
            for (int c = 0; c < BN; ++c) s[c] = __fsub_rn(__fmul_rn(s[c], a.scale_log2), mu) * back;
            mu = 0.f;
          }
        }
        m = mn;
        const float from = (BF16 ? 0.f : kLift) - mu;
        const float2 sc = make_float2(a.scale_log2, a.scale_log2), off = make_float2(from, from);
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
              p[i] = pack2<BF16>(y.x, y.y);
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
        l += all.x + all.y;
      }
      if (!ok) break;
      made += n;
      if constexpr (kPair) {  // for parts without a unit too: a barrier must not run ahead of the other's wait by two phases
        if (n > 0 && ((made - 1) & 1) != wg) {
          ok = warp_wait(&m_full[other8], turn_of(made - 1));
          if (!ok) break;
          tc_fence_after();
          m = *m_other;
          if (m != ml) l *= exp2_fast(ml - m);
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
      const float inv = direct ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
      // eight rows of the warp's 32 per lane go out by this lane: row 4 i + lane / 8, 16 bytes of every 128
      int64_t to_row[8];
      uint32_t rows_out = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = (warp & 3) * 32 + i * 4 + (lane >> 3), fr = g.f0 + t * 128 + row;
        if (fr < g.rows) rows_out |= 1u << i;
        const int q = a.div_g(min(fr, g.rows - 1));
        to_row[i] = direct ? (int64_t)(g.q0 + q) * a.o_row + (int64_t)(g.h * a.G + min(fr, g.rows - 1) - q * a.G) * a.o_head
                           : (int64_t)(t * 128 + row) * D;
      }
      float* po = cut_o<T, D>(a, gridDim.x, blockIdx.x, g.slot);
      if (!direct && (!kPair || wg == 0)) cut_ml<T>(a, gridDim.x, blockIdx.x, g.slot)[t * 128 + row_t] = make_float2(m, l);
      have = take(g);
      if (!ok) break;
      if (have) load_q();
      if (!ok) break;
      if (n > 0) {
        ok = warp_wait(&o_full[t * Sh::kBufs + buf_of(made - 1)], turn_of(made - 1));
        if (!ok) break;
        tc_fence_after();
      }
      // Through shared memory, 128 bytes of each row at a time, so that a store of the warp covers four whole lines and
      // not 16 bytes of 32 of them.
      uint8_t* stage = sout + warp * Sh::kStage;
      const int step = direct ? 64 : 32;  // columns: 16-bit results, fp32 sums
#pragma unroll 1
      for (int c = kPair ? wg * (D / 2) : 0; c < (kPair ? (wg + 1) * (D / 2) : D); c += step) {
        uint4 v[8];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x == 1 && !direct) break;
          float o[32];
          __syncwarp();
          if (n > 0) {
            tmem_ld32_async(to + c + 32 * x, o);
            tmem_wait_ld();
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
            for (int i = 0; i < 8; ++i)
              v[i] = make_uint4(__float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]), __float_as_uint(o[4 * i + 2]),
                                __float_as_uint(o[4 * i + 3]));
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) = v[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = i * 4 + (lane >> 3);
          const uint4 x = *reinterpret_cast<const uint4*>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
          if (!(rows_out >> i & 1)) continue;
          if (direct) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + to_row[i] + c + (lane & 7) * 8) = x;
          else *reinterpret_cast<uint4*>(po + to_row[i] + c + (lane & 7) * 4) = x;
        }
        __syncwarp();
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
cudaError_t launch_tc_as(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, cudaStream_t s) {
  using Sh = TcShape<D>;
  static std::atomic<uint64_t> known{0};
  cudaError_t e = allow_smem(k_attn_tc<D, BF16>, Sh::kSmem, known);
  if (e == cudaSuccess)
    e = launch_pdl(k_attn_tc<D, BF16>, dim3(p.ctas), dim3(Sh::kThreads), Sh::kSmem, s, a, m.k, m.v, m.q);
  if (e != cudaSuccess) return e;
  return launch_join<D, 128 * Sh::kNT, BF16>(a, p.ctas, p.max_rows, s);
}

}  // namespace

AttnShape attn_tc_shape(int d, int sms) {
  using Wide = TcShape<256>;
  using Other = TcShape<128>;
  if (d == 256) return {128 * Wide::kNT, Wide::kBN, sms, cta_bytes(128 * Wide::kNT, d), Wide::kTileCost, Wide::kMinPart};
  return {128 * Other::kNT, Other::kBN, sms, cta_bytes(128 * Other::kNT, d), Other::kTileCost, Other::kMinPart};
}

cudaError_t launch_attn_tc(const AttnArgs& a, const AttnMaps& m, const AttnPlan& p, int d, int dtype, cudaStream_t s) {
  if (dtype == TQ_BF16)
    return d == 64    ? launch_tc_as<64, true>(a, m, p, s)
           : d == 128 ? launch_tc_as<128, true>(a, m, p, s)
                      : launch_tc_as<256, true>(a, m, p, s);
  return d == 64    ? launch_tc_as<64, false>(a, m, p, s)
         : d == 128 ? launch_tc_as<128, false>(a, m, p, s)
                    : launch_tc_as<256, false>(a, m, p, s);
}

}  // namespace tq
