// Attention of chunks of new tokens over an exact cache or an encoder's states, on the tensor cores (tcgen05).
#include <algorithm>

#include "tq_attention.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

// =============================================================================================
// k_attn_tc: one CTA takes NT tiles of 128 rows (query, head of the group) of one request and KV head, and one
// split of its tokens. The rows of a group share K and V, so a tile is full at any group size.
//   - a TMA warp keeps a ring of K and V tiles (BN tokens) in flight, in the 128-byte swizzle;
//   - an MMA warp issues S_t = Q_t K^T into TMEM, and O_t += P_t V with P_t read from TMEM and V taken as it lies
//     (tokens x channels, the MN-major operand form);
//   - a warpgroup per tile reads S_t (a thread per row, so row sums need no exchange), writes P_t = 2^(s - m) in 16
//     bits over it, and rescales O_t only where a row's maximum grew by more than 2^8: the weights stay below
//     2^8, far inside fp32 and f16, and the final division takes the factor out.
// The two tiles alternate: while one's softmax runs, the tensor pipe works for the other.
// =============================================================================================
template <int D>
struct TcShape {
  static constexpr int kNT = D == 256 ? 1 : 2;     // tiles of 128 rows: TMEM holds S and O of two up to D = 128
  static constexpr int kBN = D == 256 ? 64 : 128;  // tokens of a K or V tile
  static constexpr int kTile = kBN * D * 2;        // its bytes
  static constexpr int kStages = D == 64 ? 8 : 4;  // 128 KB of K and V in flight
  static constexpr int kThreads = kNT * 128 + 128;
  static constexpr int kQ = 128 * D * 2;           // bytes of a tile's queries
  static constexpr int kSmem = 1024 + kNT * kQ + kStages * kTile + 512;
  static constexpr uint32_t kS = 0;                // TMEM columns: S_t (P_t over it) at kS + t * 128, O_t at kO + t * D
  static constexpr uint32_t kO = 256;
};

// A warp's wait on an mbarrier: every lane waits, all go on together, and all give up if one does.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// Registers per thread from here on (executed by every warp of a warpgroup).
template <int N>
__device__ __forceinline__ void set_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// A value that all lanes of the warp hold, told to the compiler as such (the MMA operands sit in uniform registers).
template <typename T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// 32 columns of this thread's TMEM lane, without the wait.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// Shared-memory writes of this thread become visible to the async proxy (TMA, MMA operands).
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

// x * y + z and x + y on pairs of floats.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

// Rescale O when a maximum grows by more than this (in powers of two).
constexpr float kLazy = 8.0f;

template <int D, bool BF16>
__global__ void __launch_bounds__(TcShape<D>::kThreads, 1)
    k_attn_tc(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, int n_tiles) {
  using Sh = TcShape<D>;
  constexpr int NT = Sh::kNT, BN = Sh::kBN, ST = Sh::kStages;
  constexpr uint32_t kTile = Sh::kTile;
  constexpr uint32_t kType = BF16 ? 1u : 0u;
  constexpr uint32_t kIdescS = (1u << 4) | (kType << 7) | (kType << 10) | ((uint32_t)(BN >> 3) << 17) | (8u << 24);
  constexpr uint32_t kIdescO =
      (1u << 4) | (kType << 7) | (kType << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* skv = smem + NT * Sh::kQ;
  uint64_t* full = reinterpret_cast<uint64_t*>(skv + ST * kTile);
  uint64_t* empty = full + ST;
  uint64_t* s_full = empty + ST;  // per tile: scores are in TMEM
  uint64_t* p_full = s_full + NT;  // per tile and half of the unit: weights are in TMEM, O is rescaled
  uint64_t* o_full = p_full + 2 * NT;  // per tile: the product with V is done
  uint64_t* drained = o_full + NT;
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(drained + 1);
  __shared__ int gave_up;

  const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  constexpr int kMmaWarp = NT * 4, kTmaWarp = NT * 4 + 1;
  if (threadIdx.x == 0) {
    gave_up = 0;
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  pdl_wait();
  if (a.n_splits > 1) pdl_launch();  // the join may be scheduled; it waits for this kernel's end
  uint32_t err = 0;
  int x = blockIdx.x;
  const int split = x % a.n_splits;
  x /= a.n_splits;
  const int h = x % a.hkv;
  // the last tiles first: with causal masks they are the longest, and a short tail ends the launch
  const int2 where = find_tile(a, n_tiles - 1 - x / a.hkv, 128 * NT);
  const Request r = find_request(a, where.x, err);
  if (r.n_q * (int64_t)a.G > a.max_rows) err |= TQ_DEV_ERR_SPLITS;
  const int rows = err & TQ_DEV_ERR_SPLITS ? 0 : r.n_q * a.G;
  const int f0 = where.y * (128 * NT);
  const int kv = tile_kv(a, r, where.y, 128 * NT);
  const int units = (kv + BN - 1) / BN, per = units_per_split(units, a.n_splits);
  const int u0 = split * per, u1 = min(units, u0 + per);
  const bool direct = units <= per;
  if (threadIdx.x == 0 && err && a.status) atomicOr(a.status, err);
  if (where.y > (rows - 1) / (128 * NT) || f0 >= rows || (u0 >= u1 && split > 0)) return;
  // units of each tile: up to the last token that its last row sees
  int n_of[NT];
  int n_all = 0;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int kv_t = f0 + t * 128 < rows ? tile_kv(a, r, where.y * NT + t, 128) : 0;
    n_of[t] = max(0, min(u1, (kv_t + BN - 1) / BN) - u0);
    n_all = max(n_all, n_of[t]);
  }

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  // queries into shared memory, as K-major operands; rows past the last are zero
  for (int i = threadIdx.x; i < NT * 128 * (D / 8); i += Sh::kThreads) {
    const int row = i / (D / 8), c = i % (D / 8), f = f0 + row;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (f < rows) {
      const int qi = f / a.G, g = f - qi * a.G;
      v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (int64_t)(r.q0 + qi) * a.q_row +
                                          (int64_t)(h * a.G + g) * a.q_head + c * 8);
    }
    const int rr = row & 127;
    *reinterpret_cast<uint4*>(smem + (row >> 7) * Sh::kQ + (c >> 3) * 16384 + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = v;
  }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_base);
  // The softmax threads hold a row of scores: they take registers from the other warps (8 x 32 x 216 + 4 x 32 x 72 =
  // 384 x 168, what the block was launched with). One tile's warps have enough as it is.
  constexpr bool kSplitRegs = NT == 2;
  if (warp >= kMmaWarp) {
    if constexpr (kSplitRegs) set_regs_dec<72>();
    if (warp == kTmaWarp) {
      // ---- K and V tiles: ring entry 2 k holds K of unit u0 + k, entry 2 k + 1 its V ----
      int2 place = make_int2(0, 0);
      bool ok = true;
      int issued = 0;
      for (int k = 0; k < n_all && ok; ++k) {
        if ((k & 31) == 0 && k + lane < n_all) {
          const int tok = (u0 + k + lane) * BN;
          place = page_place(a, r, tok / kPage, err);
          place.y += tok % kPage;
        }
        const int w = __shfl_sync(0xffffffffu, place.x, k & 31), y = __shfl_sync(0xffffffffu, place.y, k & 31);
        if (lane == 0) {
#pragma unroll
          for (int which = 0; which < 2; ++which) {
            const int e = 2 * k + which, st = e % ST;
            if (ok && e >= ST) ok = mbar_wait(&empty[st], ((e / ST) - 1) & 1);
            if (!ok) break;
            uint8_t* dst = skv + st * kTile;
            mbar_expect_tx(&full[st], kTile);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_4d(dst + c * (BN * 128), which ? &map_v : &map_k, c * 64, y, h, w, &full[st]);
            issued = e + 1;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (lane == 0) {
        // leave only when every copy has landed (they have, unless a wait gave up)
        for (int e = max(0, issued - ST); e < issued; ++e) ok &= mbar_wait(&full[e % ST], (e / ST) & 1);
        if (!ok) {
          err |= TQ_DEV_ERR_TIMEOUT;
          atomicExch(&gave_up, 1);
        }
      }
      if (err && a.status) atomicOr(a.status, err);
    } else if (warp == kMmaWarp) {
      // ---- products: S_t(0), S_1(0), then per unit and tile O_t += P_t V and the next S_t ----
      bool ok = true;
      const bool leader = elect_one();
      n_all = uniform(n_all);
#pragma unroll
      for (int t = 0; t < NT; ++t) n_of[t] = uniform(n_of[t]);
      const uint32_t q_lo = umma_desc_sw128_lo(smem_u32(smem)), kv_lo = smem_u32(skv) >> 4;
      auto scores = [&](int t, int k) {  // S_t = Q_t K(k)^T
        if (leader) {
          const uint32_t ka = kv_lo + ((2 * k) % ST) * (kTile >> 4) + (1u << 16);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t step = (i & 3) * 2;
            umma_bf16_lo(tmem + Sh::kS + t * 128, q_lo + t * (Sh::kQ >> 4) + (i >> 2) * 1024 + step,
                         ka + (i >> 2) * (BN * 128 >> 4) + step, kIdescS, i > 0);
          }
          umma_commit(&s_full[t]);
        }
      };
      if (n_all > 0) ok = warp_wait(&full[0], 0);
      if (ok && n_all > 0) {
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < NT; ++t)
          if (n_of[t] > 0) scores(t, 0);
        if (leader) umma_commit(&empty[0]);
      }
      for (int k = 0; k < n_all && ok; ++k) {
        const int ve = 2 * k + 1, vs = ve % ST;
        ok = warp_wait(&full[vs], (ve / ST) & 1);
        if (!ok) break;
        // the unit that the sequence ends in: V rows behind it are zeroed up to the next step of 16 (0 x NaN is NaN),
        // and the steps behind them are left out
        const int valid = uniform(min(BN, kv - (u0 + k) * BN)), steps = (valid + 15) / 16;
        if (valid & 15) {
          const int n = (16 - (valid & 15)) * (D / 8);
          for (int i = lane; i < n; i += 32) {
            const int c = i % (D / 8), row = valid + i / (D / 8);
            *reinterpret_cast<uint4*>(skv + vs * kTile + (c >> 3) * (BN * 128) + row * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
          __syncwarp();
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (k < n_of[t] && ok) {
            // MN-major operand: 64-channel blocks BN x 128 bytes apart, 8-token groups 1024 bytes apart
            const uint32_t va = kv_lo + vs * (kTile >> 4) + ((uint32_t)(BN * 128 >> 4) << 16);
            const uint32_t od = tmem + Sh::kO + t * D, pa = tmem + Sh::kS + t * 128;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              ok = ok && warp_wait(&p_full[2 * t + half], k & 1);
              if (!ok) break;
              tc_fence_after();
              if (leader) {
#pragma unroll
                for (int i = half * (BN / 32); i < (half + 1) * (BN / 32); ++i)
                  if (i < steps) umma_ts_lo(od, pa + i * 8, va + i * (2048 >> 4), kIdescO, k > 0 || i > 0);
              }
            }
            if (!ok) break;
            if (leader) umma_commit(&o_full[t]);
          }
          if (t == NT - 1 && leader) umma_commit(&empty[vs]);
          if (k + 1 < n_all && ok) {
            const int ke = 2 * (k + 1), ks = ke % ST;
            if (t == 0) ok = warp_wait(&full[ks], (ke / ST) & 1);
            if (k + 1 < n_of[t] && ok) {
              ok = warp_wait(&o_full[t], k & 1);  // S_t(k + 1) goes over P_t(k)
              if (!ok) break;
              tc_fence_after();
              scores(t, k + 1);
            }
            if (t == NT - 1 && leader) umma_commit(&empty[ks]);
          }
        }
      }
      // leave only when every product is done
      if (leader) umma_commit(drained);
      const bool done = warp_wait(drained, 0);
      if ((!ok || !done) && leader) {
        atomicExch(&gave_up, 1);
        if (a.status) atomicOr(a.status, TQ_DEV_ERR_TIMEOUT);
      }
    }
  } else {
    if constexpr (kSplitRegs) set_regs_inc<216>();
    // ---- softmax of tile t: a thread per row ----
    const int t = warp >> 2;
    const int n = t == 0 ? n_of[0] : n_of[NT - 1];
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const uint32_t ts = tmem + Sh::kS + t * 128 + lanes, to = tmem + Sh::kO + t * D + lanes;
    const int f = f0 + t * 128 + (threadIdx.x & 127);
    const bool mine = f < rows;
    const int qi = mine ? f / a.G : 0;
    const int lim = mine ? seen(a, r, qi) : 0;
    // what every row of the tile sees needs no mask; rows past the last may hold anything
    const int f_first = min(f0 + t * 128, rows - 1);
    const int lim_all = seen(a, r, f_first / a.G);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int k = 0; k < n; ++k) {
      ok = warp_wait(&s_full[t], k & 1);
      if (!ok) break;
      tc_fence_after();
      float s[BN];
#pragma unroll
      for (int c = 0; c < BN; c += 32) tmem_ld32_async(ts + c, s + c);
      tmem_wait_ld();
      const int base = (u0 + k) * BN;
      if (base + BN > lim_all) {
        const int left = lim - base;
#pragma unroll
        for (int c = 0; c < BN; ++c) s[c] = c < left ? s[c] : -INFINITY;
      }
      float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < BN; c += 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], c + 4 + i < BN ? fmaxf(s[c + i], s[c + 4 + i]) : s[c + i]);
      }
      const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
      float mn = m;
      if (mx > m + kLazy || m == -INFINITY) mn = fmaxf(m, mx);
      const bool grew = mn != m && m != -INFINITY;
      if (__any_sync(0xffffffffu, grew)) {
        const float alpha = grew ? exp2_fast(m - mn) : 1.f;
        l *= alpha;
        ok = warp_wait(&o_full[t], (k - 1) & 1);  // a maximum that grew has seen a unit, so k > 0
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(to + c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(to + c, o);
        }
      }
      m = mn;
      const float mu = m == -INFINITY ? 0.f : m;
      const float2 sc = make_float2(a.scale_log2, a.scale_log2), off = make_float2(-mu, -mu);
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
          tmem_st16(ts + c / 2, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * t + half]);
      }
      const float2 both = add2(sum[0], sum[1]);
      l += both.x + both.y;
    }
    if (ok && n > 0) ok = warp_wait(&o_full[t], (n - 1) & 1);
    if (!ok) {
      if (lane == 0) {
        atomicExch(&gave_up, 1);
        if (a.status) atomicOr(a.status, TQ_DEV_ERR_TIMEOUT);
      }
    } else {
      tc_fence_after();
      const int head = h * a.G + f - qi * a.G;
      const float inv = direct ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
      const size_t slot = mine && !direct ? part_slot(a, r.q0 + qi, head, split) : 0;
      uint16_t* dst = static_cast<uint16_t*>(a.out) + (int64_t)(r.q0 + qi) * a.o_row + (int64_t)head * a.o_head;
      float* po = part_o(a) + slot * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        __syncwarp();
        if (n > 0) {
          tmem_ld32_async(to + c, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = n > 0 ? o[i] * inv : 0.f;
        if (mine && direct) {
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            *reinterpret_cast<uint4*>(dst + c + i) =
                make_uint4(pack2<BF16>(o[i], o[i + 1]), pack2<BF16>(o[i + 2], o[i + 3]),
                           pack2<BF16>(o[i + 4], o[i + 5]), pack2<BF16>(o[i + 6], o[i + 7]));
        } else if (mine) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(po + c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
      }
      if (mine && !direct) part_ml(a)[slot] = make_float2(m, l);
      tc_fence_before();
    }
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
  cudaError_t e = cudaFuncSetAttribute(k_attn_tc<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_attn_tc<D, BF16>, dim3((unsigned)p.tiles * a.hkv * a.n_splits), dim3(Sh::kThreads), Sh::kSmem, s,
                    a, m.k, m.v, (int)p.tiles);
}

}  // namespace

int attn_tc_tile_rows(int d) { return d == 256 ? TcShape<256>::kNT * 128 : TcShape<128>::kNT * 128; }
int attn_tc_unit(int d) { return d == 256 ? TcShape<256>::kBN : TcShape<128>::kBN; }

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
