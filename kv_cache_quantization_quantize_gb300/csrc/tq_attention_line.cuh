// The split of the work of one attention launch, shared by both kernels.
//
// All tiles of all requests and KV heads lie on one line, in the order (request, head, tile); each takes as much of it
// as it is estimated to cost, in 64ths of a unit (2^a.shift of them where a launch's line would pass 2^30): its tokens
// and a fixed cost for its start and end. CTA c takes
// [c Q, (c + 1) Q); a tile that is cut there has its units divided in proportion, and the parts are joined by
// k_attn_join. So CTAs get nearly the same amount of work whatever the lengths are, at most two cut tiles per CTA go
// through memory, and the host needs no lengths. Costs have closed sums, so finding a place takes one pass over the
// requests. What a cut adds, a second start and end and the join's bytes, is not in the costs, and a piece can be as short
// as one unit: in long work that is lost in the rest, short work pays for it (8 ragged prompts of 20 heads have 135 cut
// tiles in 270 pieces on 152 CTAs, 114 of the pieces of 3 units or less; 16 single tokens against 700 to 1500 states of 16 heads
// have all 256 tiles cut).
#pragma once

#include <atomic>

#include "tq_attention.cuh"

namespace tq {
namespace {

// A tile that begins in this CTA and ends in a later one.
struct CutTile {
  int32_t s, e, q;  // its place on the line, and Q
  int32_t units;    // 0: there is no such tile
  int32_t f0, rows, h, q0;
};

// What a CTA does of one tile, as its warps read it from a ring in shared memory that one warp fills. n_all < 0: no
// more.
struct Part {
  int f0, rows;                     // first row of the tile, rows of the request
  int kv;                           // tokens that any row of the tile sees
  int u0, n_all;                    // first unit, units
  int n_of[2];                      // units of each half of a tile (tq_attention_tc.cu)
  int h, q0, n_q, r_kv, row, base;  // KV head and request
  int direct, slot;                 // all of the tile: results go to out; else which part of the workspace takes them
};
constexpr int kParts = 4;

// First unit of the part of a tile [s, e) that begins at place p of the line: (p - s) units / (e - s), in fp32 steps
// that never fall with p (each rounding is monotone), so that neighbouring CTAs and the join, which compute it from the
// same numbers, cut the tile alike.
__device__ __forceinline__ int cut_at(int p, int s, int e, int units) {
  if (p <= s) return 0;
  if (p >= e) return units;
  const float x = __fmul_rn(__fmul_rn((float)(p - s), (float)units), __frcp_rn((float)(e - s)));
  return min(units, (int)x);
}

// Where a CTA starts: its part [p0, p1) of the line, and the tile that holds p0.
struct LineStart {
  int p0, p1, s, b, h, t;
  Request r;
};

// T: rows (query, head of the group) of a tile; BN: tokens of a unit; COST: fixed cost of a tile; NT: parts of a tile
// that have units of their own (n_of).
template <int T, int BN, int COST, int NT>
struct Walk {
  int p0, p1, s, e;  // this CTA's part of the line, and the tile in hand
  int fixed;         // cost of its first tile, but for the slope
  Request r;
  int b, h, t, nt, rows;

  __device__ __forceinline__ void take(const AttnArgs& a, int request, const Request& found, uint32_t& err) {
    b = request;
    r = found;
    rows = 0;
    if (r.n_q * (int64_t)a.G > a.max_rows) err |= TQ_DEV_ERR_SPLITS;
    else rows = r.n_q * a.G;
    nt = (rows + T - 1) / T;
    const int tokens = a.causal ? max(0, r.kv - r.n_q) : r.kv;
    fixed = max(1, (int)(((uint32_t)tokens / (BN / 32) * 2 + COST) >> a.shift));
  }
  __device__ __forceinline__ void load(const AttnArgs& a, int request, uint32_t& err) {
    const Request found = find_request(a, request, err);
    take(a, request, found, err);
  }
  __device__ __forceinline__ int before(const AttnArgs& a, int tile) const {
    return tile * fixed + a.slope * (int)((uint32_t)tile * (tile + 1) / 2);
  }
  // The tile in hand, or the first one of a later request.
  __device__ __forceinline__ void settle(const AttnArgs& a) {
    uint32_t err = 0;
    while (t >= nt && b < a.batch) {
      t = 0;
      if (nt > 0 && ++h < a.hkv) break;
      h = 0;
      if (b + 1 >= a.batch) {
        b = a.batch;
        break;
      }
      load(a, b + 1, err);
    }
    e = s + fixed + a.slope * (t + 1);
  }
  __device__ __forceinline__ void start(const AttnArgs& a, const LineStart& st) {
    p0 = st.p0;
    p1 = st.p1;
    b = a.batch;
    t = nt = h = 0;
    s = p1;
    // (starts that fall can give requests more rows together than there are, and sums past 32 bits: then nobody may have
    // found p0, and some outputs stay unwritten)
    if (p0 >= p1 || st.b >= a.batch) return;
    uint32_t err = 0;
    take(a, st.b, st.r, err);
    h = st.h;
    t = st.t;
    s = st.s;
  }
  // The next tile of which this CTA has a part; cut is filled for one that it begins and does not end.
  __device__ __forceinline__ bool next(const AttnArgs& a, Part& g, CutTile& cut) {
    for (;;) {
      // Behind this CTA's part there is nothing to find: 1020 requests without queries behind 4 with one each, as in a padded
      // batch, made 15 us 108.
      if (s >= p1) break;
      settle(a);  // here and not behind the last tile: a part is given out before the next request is read
      if (b >= a.batch) break;
      g.f0 = t * T;
      g.rows = rows;
      g.kv = tile_kv(a, r, t, T);
      const int units = (g.kv + BN - 1) / BN;
      g.u0 = cut_at(p0, s, e, units);
      const int u1 = cut_at(p1, s, e, units);
      g.n_all = u1 - g.u0;
      if constexpr (NT > 0) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int kv_i = g.f0 + i * (T / NT) < rows ? tile_kv(a, r, t * NT + i, T / NT) : 0;
          g.n_of[i] = max(0, min(u1, (kv_i + BN - 1) / BN) - g.u0);
        }
      }
      g.h = h;
      g.q0 = r.q0;
      g.n_q = r.n_q;
      g.r_kv = r.kv;
      g.row = r.row;
      g.base = r.base;
      g.direct = g.n_all == units;
      g.slot = s >= p0;
      if (g.slot && e > p1) {
        cut.units = units;
        cut.f0 = g.f0;
        cut.rows = rows;
        cut.h = h;
        cut.q0 = r.q0;
        cut.s = s;
        cut.e = e;
        cut.q = p1 - p0;  // a whole part: the tile goes on behind it
      }
      const bool any = g.n_all > 0 || (units == 0 && g.slot);  // a tile that sees nothing has zeros to write
      s = e;
      ++t;
      if (any) return true;
    }
    g.n_all = -1;
    return false;
  }
};

// This CTA's part of the line, into `st` in shared memory (as warp_sums, THREADS / 32 entries): prefix sums of the
// requests' costs over the block. No CTA gets less than `least`. Bad requests are reported once, by CTA 0.
template <typename W, int THREADS>
__device__ __forceinline__ void find_start(const AttnArgs& a, int least, LineStart& st, int* warp_sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  W w;
  uint32_t err = 0;
  const int per = (a.batch + THREADS - 1) / THREADS;
  const int lo = min(a.batch, (int)threadIdx.x * per), hi = min(a.batch, lo + per);
  int sum = 0;
  for (int b = lo; b < hi; ++b) {
    w.load(a, b, err);
    sum += a.hkv * w.before(a, w.nt);
  }
  if (blockIdx.x == 0 && err && a.status) atomicOr(a.status, err);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_sums[warp] = inc;
  if (threadIdx.x == 0) st.b = a.batch;
  __syncthreads();
  int start = inc - sum, total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) start += warp_sums[i];
    total += warp_sums[i];
  }
  // an equal share, a millionth up so that no rounding leaves work over
  const int q = max(max(1, least >> a.shift), (int)((float)total * __frcp_rn((float)gridDim.x) * 1.000001f) + 1);
  const int p0 = min((int64_t)total, (int64_t)q * blockIdx.x), p1 = min((int64_t)total, (int64_t)p0 + q);
  if (threadIdx.x == 0) {
    st.p0 = p0;
    st.p1 = p1;
  }
  if (p0 >= start && p0 < start + sum) {  // one thread's requests hold p0
    for (int b = lo; b < hi; ++b) {
      if (per > 1) w.load(a, b, err);
      const int one = w.before(a, w.nt);
      if (p0 >= start + a.hkv * one) {
        start += a.hkv * one;
        continue;
      }
      int head = max(0, min(a.hkv - 1, (int)((float)(p0 - start) / (float)one)));  // within a few of the quotient
      while (head > 0 && start + head * one > p0) --head;
      while (head + 1 < a.hkv && start + (head + 1) * one <= p0) ++head;
      start += head * one;
      int at = 0, n = w.nt;  // the last tile that begins at p0 or before
      while (n > 1) {
        const int half = n / 2;
        if (start + w.before(a, at + half) <= p0) {
          at += half;
          n -= half;
        } else {
          n = half;
        }
      }
      st.b = b;
      st.h = head;
      st.t = at;
      st.s = start + w.before(a, at);
      st.r = w.r;
      break;
    }
  }
  __syncthreads();
}

// Workspace: the cut tiles [CTAs], then {m, l} [CTAs][2][T] and the sums [CTAs][2][T][D] of the parts of cut tiles;
// part 0 of a CTA is of a tile that an earlier CTA began, part 1 of one that it began itself. Weights are
// exp2(score * scale_log2 - m), l their sum, the sums are of weight * value.
inline size_t cta_bytes(int T, int D) { return sizeof(CutTile) + 2 * (size_t)T * (sizeof(float2) + D * sizeof(float)); }
__device__ __forceinline__ CutTile* cut_tiles(const AttnArgs& a) { return reinterpret_cast<CutTile*>(a.part); }
template <int T>
__device__ __forceinline__ float2* cut_ml(const AttnArgs& a, int ctas, int cta, int part) {
  return reinterpret_cast<float2*>(cut_tiles(a) + ctas) + ((size_t)cta * 2 + part) * T;
}
template <int T, int D>
__device__ __forceinline__ float* cut_o(const AttnArgs& a, int ctas, int cta, int part) {
  return reinterpret_cast<float*>(reinterpret_cast<float2*>(cut_tiles(a) + ctas) + (size_t)ctas * 2 * T) +
         ((size_t)cta * 2 + part) * T * D;
}

// k_attn_join: the parts of the tile that CTA blockIdx.x began and did not end, joined with their maxima and sums:
// o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i. Latency bounds the kernel, so as many loads as possible overlap.
// Tiles of up to 32 rows can be in many parts (a long sequence over all SMs): a CTA per row, whose 8 warps share the
// parts. Larger tiles have many rows and mostly two parts: a CTA per 16 rows, four of them to a warp.
template <int T>
struct JoinShape {
  static constexpr int kGroups = T == 16 ? 8 : T == 32 ? 4 : 1;  // warps that share the parts of a row
  static constexpr int kPer = T <= 32 ? 1 : 4;                  // rows of a warp
  static constexpr int kWarps = T <= 32 ? 8 : 4;
  static constexpr int kRows = kWarps / kGroups * kPer;  // rows of a CTA
};
template <int D, int T, bool BF16>
__global__ void __launch_bounds__(JoinShape<T>::kWarps * 32) k_attn_join(const __grid_constant__ AttnArgs a, int ctas) {
  using Sh = JoinShape<T>;
  constexpr int V = D / 32, R = Sh::kPer, kStep = Sh::kWarps / Sh::kGroups;  // row j of a warp: kStep j further
  __shared__ int16_t part[kMaxAttnCtas];
  __shared__ int parts;
  __shared__ float2 s_ml[Sh::kWarps][R];
  __shared__ float s_acc[Sh::kGroups > 1 ? Sh::kWarps : 1][R][Sh::kGroups > 1 ? D : 1];
  pdl_wait();
  const CutTile c = cut_tiles(a)[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp % Sh::kGroups;
  const int row0 = blockIdx.y * Sh::kRows + warp / Sh::kGroups;
  if (!c.units || c.f0 + (int)blockIdx.y * Sh::kRows >= c.rows) return;
  const int i0 = blockIdx.x, i1 = min(ctas - 1, (c.e - 1) / c.q);
  if (warp == 0) {  // the CTAs that had units of it
    int n = 0;
    for (int base = i0; base <= i1; base += 32) {
      const int i = base + lane;
      const bool live = i <= i1 && cut_at((i + 1) * c.q, c.s, c.e, c.units) > cut_at(i * c.q, c.s, c.e, c.units);
      const uint32_t m = __ballot_sync(0xffffffffu, live);
      if (live) part[n + __popc(m & ((1u << lane) - 1))] = (int16_t)i;
      n += __popc(m);
    }
    if (lane == 0) parts = n;
  }
  __syncthreads();
  if (parts < 2) return;  // one CTA had all of it
  float top[R], sum[R], acc[R][V];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    top[j] = -INFINITY;
    sum[j] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[j][i] = 0.f;
  }
#pragma unroll 4
  for (int k = group; k < parts; k += Sh::kGroups) {
    const int i = part[k];
    const float2* pml = cut_ml<T>(a, ctas, i, i == i0) + row0;
    const float* po = cut_o<T, D>(a, ctas, i, i == i0) + (size_t)row0 * D + lane * V;
    float2 ml[R];
    float v[R][V];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (c.f0 + row0 + kStep * j >= c.rows) break;  // rows past the last are not written
      ml[j] = pml[kStep * j];
      if constexpr (V == 2) *reinterpret_cast<float2*>(v[j]) = *reinterpret_cast<const float2*>(po + kStep * j * D);
      else
#pragma unroll
        for (int q = 0; q < V; q += 4)
          *reinterpret_cast<float4*>(v[j] + q) = *reinterpret_cast<const float4*>(po + kStep * j * D + q);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (c.f0 + row0 + kStep * j >= c.rows) break;
      const float mn = fmaxf(top[j], ml[j].x), mu = mn == -INFINITY ? 0.f : mn;
      const float wa = exp2_fast(top[j] - mu), wb = exp2_fast(ml[j].x - mu);  // 0 for a part that saw no token
      top[j] = mn;
      sum[j] = sum[j] * wa + ml[j].y * wb;
#pragma unroll
      for (int x = 0; x < V; ++x) acc[j][x] = acc[j][x] * wa + v[j][x] * wb;
    }
  }
  if constexpr (Sh::kGroups > 1) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (lane == 0) s_ml[warp][j] = make_float2(top[j], sum[j]);
#pragma unroll
      for (int x = 0; x < V; ++x) s_acc[warp][j][lane * V + x] = acc[j][x];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int j = 0; j < R; ++j) {
#pragma unroll
      for (int i = 1; i < Sh::kGroups; ++i) {
        const float2 ml = s_ml[warp + i][j];
        const float mn = fmaxf(top[j], ml.x), mu = mn == -INFINITY ? 0.f : mn;
        const float wa = exp2_fast(top[j] - mu), wb = exp2_fast(ml.x - mu);
        top[j] = mn;
        sum[j] = sum[j] * wa + ml.y * wb;
#pragma unroll
        for (int x = 0; x < V; ++x) acc[j][x] = acc[j][x] * wa + s_acc[warp + i][j][lane * V + x] * wb;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int f = c.f0 + row0 + kStep * j;
    if (f >= c.rows) break;
    const float inv = sum[j] > 0.f ? 1.f / sum[j] : 0.f;
    const int qi = a.div_g(f), head = c.h * a.G + f - qi * a.G;
    uint16_t* dst = static_cast<uint16_t*>(a.out) + (int64_t)(c.q0 + qi) * a.o_row + (int64_t)head * a.o_head + lane * V;
    uint32_t out[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) out[i] = result2<BF16>(acc[j][2 * i] * inv, acc[j][2 * i + 1] * inv);
    if constexpr (V == 2) *reinterpret_cast<uint32_t*>(dst) = out[0];
    else if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// Lets a kernel use `bytes` of dynamic shared memory on the current device; asked once per device (`known`: one bit
// each).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& known) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (known.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) known.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// `rows`: the most rows that a request has (no tile has more).
template <int D, int T, bool BF16>
cudaError_t launch_join(const AttnArgs& a, int ctas, int64_t rows, cudaStream_t s) {
  using Sh = JoinShape<T>;
  const int tile = (int)(rows < T ? rows : T);
  return launch_pdl(k_attn_join<D, T, BF16>, dim3(ctas, (tile + Sh::kRows - 1) / Sh::kRows), dim3(Sh::kWarps * 32), 0, s,
                    a, ctas);
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(m) : "memory");
}
// Shared by the kernels' warps: an mbarrier wait that all lanes of a warp make together; all give up if one does.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// Rescale sums when a row's maximum grew by more than this (in powers of two): weights stay below 2^8, far inside
// fp32 and f16, and the final division takes the factor out.
constexpr float kLazy = 8.0f;
// Weights that are rounded to f16 are 2^kLift times as large, sums and statistics with them: up to 2^15 where f16 ends at 65504.
// f16 has nothing below 2^-25, so without it a weight of 2^-25 of the row's largest would be lost, which 2^15 tokens
// behind a first one that takes nearly all of the weight have; so it is 2^-32.
constexpr float kLift = 7.0f;
// Over 8 bits a row's reference is the largest of s + log2 vs, and scales can be 2^120 apart. Three things keep the statistic, which
// divides by the scale, inside fp32's range then:
//   - Where a unit's scale over the reference's, `above` in powers of two, is below kThin, its part of the statistic is not made
//     of its weights, which can be below fp32's range. The rows kernel takes exponentials of its own for it, behind its rare path. The tensor
//     cores' kernel makes the weights with a larger `above`, no larger than makes the largest of them 2^-66 (x: its score over
//     the reference's): so small they are 0 in f16 either way, and their sum is divided by what they were made with.
//   - The statistic is rescaled in two steps.
//   - A part of a tile goes to the join relative to m + mv and a power of two of its sum (below).
constexpr float kThin = -80.0f;
__device__ __forceinline__ float least_above(float above, float x) {
  return above < kThin ? fmaxf(above, fminf(0.f, -66.f - x)) : above;
}
__device__ __forceinline__ float rescaled(float l, float by) {
  const float half = exp2_fast(0.5f * by);
  return l * half * half;
}
// Of a part with the reference m + mv and the statistic l: what it is relative to in the join, in one float, and the factor of its
// sums. The rounding of that float, which far scores make large, goes into the factor.
__device__ __forceinline__ float2 part_reference(float m, float mv, float l) {
  if (m == -INFINITY) return make_float2(m, 1.f);  // it saw no token
  const int e = min(max((int)(__float_as_uint(l) >> 23) - 127, 0), 60);
  const float t = mv + (float)e, to = m + t;
  return make_float2(to, exp2_fast(((m - to) + t) - (float)e));
}

}  // namespace
}  // namespace tq
