// Rotary positions, and a step's new tokens rotated on their way into a paged cache of 16 or 8 bits: tq_rotate,
// tq_paged_extend.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "tq_device.cuh"

namespace tq {
namespace {

__device__ __forceinline__ void report(uint32_t* status, uint32_t bits) {
  if (bits && status) atomicOr(status, bits);
}

// Two floats at a time.
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float flip(float x, uint32_t sign) { return __uint_as_float(__float_as_uint(x) ^ sign); }

// ---- rotation ----

// Cosines and sines of position * turns (in 2^-64 of a whole turn) of two pairs, times factor, the sines with the sign bit
// `inverse` flipped. The product modulo 2^64 is the angle modulo a turn without error; its upper 32 bits are taken to the
// nearest quarter turn before they become a float, so that the rest x, at most a quarter of a half turn, is rounded to
// 2^-25 of itself. There sin(pi x) and cos(pi x) are their Taylor series to x^9 and x^10, whose next terms are below
// 2e-9: two pairs at a time these are half the instructions of the library's functions (65536 tokens x 8 heads into 8
// bits: 109 us with those).
__device__ __forceinline__ void turn2(int position, const uint64_t* turns, float factor, uint32_t inverse, float2& c, float2& s) {
  float x[2];
  uint32_t q[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t f = (uint32_t)(((uint64_t)(int64_t)position * turns[i]) >> 32);
    q[i] = (f + (1u << 29)) >> 30;
    x[i] = (float)(int32_t)(f - (q[i] << 30));  // in 2^-31 of a half turn
  }
  const float2 y = mul2(make_float2(x[0], x[1]), both(4.656612873077392578125e-10f)), t = mul2(y, y);
  float2 sn = fma2(t, both(0.08214588661112823f), both(-0.5992645293207921f));  // pi^9 / 9!, -pi^7 / 7!
  sn = fma2(t, sn, both(2.550164039877345f));
  sn = fma2(t, sn, both(-5.16771278004997f));
  sn = fma2(t, sn, both(3.141592653589793f));
  sn = mul2(sn, y);
  float2 cs = fma2(t, both(-0.02580689139001406f), both(0.2353306303588935f));  // -pi^10 / 10!, pi^8 / 8!
  cs = fma2(t, cs, both(-1.335262768854589f));
  cs = fma2(t, cs, both(4.058712126416768f));
  cs = fma2(t, cs, both(-4.934802200544679f));
  cs = fma2(t, cs, both(1.f));
  sn = mul2(sn, both(factor));
  cs = mul2(cs, both(factor));
  c = make_float2(flip(q[0] & 1 ? sn.x : cs.x, (q[0] + 1) << 30 & 0x80000000u), flip(q[1] & 1 ? sn.y : cs.y, (q[1] + 1) << 30 & 0x80000000u));
  s = make_float2(flip(q[0] & 1 ? cs.x : sn.x, (q[0] << 30 & 0x80000000u) ^ inverse),
                  flip(q[1] & 1 ? cs.y : sn.y, (q[1] << 30 & 0x80000000u) ^ inverse));
}

// A thread's 2 CH channels of a head: CH from lo and CH from hi on; its pairs are CH j .. CH j + CH - 1.
template <int CH>
struct Place {
  int lo, hi;
  bool turned;
  __device__ __forceinline__ Place(const Rotation& r, int j) {
    turned = j * CH < r.pairs;
    const bool apart = turned && !r.interleaved;
    lo = apart ? j * CH : 2 * CH * j;
    hi = apart ? r.pairs + j * CH : lo + CH;
  }
};

// Cosines and sines of a thread's pairs, two and two.
template <int CH>
struct Turned {
  float2 c[CH / 2], s[CH / 2];
  __device__ __forceinline__ void at(const Rotation& r, const uint64_t (&turns)[CH], int position) {
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) turn2(position, turns + 2 * i, r.factor, (uint32_t)r.inverse << 31, c[i], s[i]);
  }
  __device__ __forceinline__ void apply(const Rotation& r, float (&x)[2 * CH]) const {
    if (r.interleaved) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1], ci = i & 1 ? c[i / 2].y : c[i / 2].x, si = i & 1 ? s[i / 2].y : s[i / 2].x;
        x[2 * i] = a * ci - b * si;
        x[2 * i + 1] = b * ci + a * si;
      }
    } else {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        const float2 a = make_float2(x[2 * i], x[2 * i + 1]), b = make_float2(x[CH + 2 * i], x[CH + 2 * i + 1]);
        const float2 y = fma2(b, make_float2(-s[i].x, -s[i].y), mul2(a, c[i])), z = fma2(a, s[i], mul2(b, c[i]));
        x[2 * i] = y.x, x[2 * i + 1] = y.y, x[CH + 2 * i] = z.x, x[CH + 2 * i + 1] = z.y;
      }
    }
  }
};

template <int CH>
__device__ __forceinline__ void load_turns(const Rotation& r, int j, uint64_t (&turns)[CH]) {
#pragma unroll
  for (int i = 0; i < CH; ++i) turns[i] = r.turns[j * CH + i];
}

// ---- rows ----

// Two values of 16 bits in a word, the first in the low half.
__device__ __forceinline__ float2 unpack(uint32_t x, __nv_bfloat16) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack(uint32_t x, __half) { return __half22float2(*reinterpret_cast<__half2*>(&x)); }
__device__ __forceinline__ uint32_t pack(float lo, float hi, __nv_bfloat16) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi, __half) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// CH elements at each of two places, as words. VEC: aligned to their size, up to 16 bytes.
template <typename T, int CH, bool VEC>
struct Pieces {
  static constexpr int kWords = CH * (int)sizeof(T) / 4;
  uint32_t lo[kWords], hi[kWords];
  __device__ __forceinline__ static void load_at(const T* p, uint32_t (&w)[kWords]) {
    if constexpr (VEC && kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p + i * (4 / sizeof(T)));
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = q[2 * i] | (uint32_t)q[2 * i + 1] << 16;
    }
  }
  __device__ __forceinline__ static void store_at(T* p, const uint32_t (&w)[kWords]) {
    if constexpr (VEC && kWords == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        *reinterpret_cast<uint4*>(p + i * (4 / sizeof(T))) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
    } else {
      uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        q[2 * i] = (uint16_t)w[i];
        q[2 * i + 1] = (uint16_t)(w[i] >> 16);
      }
    }
  }
  __device__ __forceinline__ void load(const T* p, const Place<CH>& at) {
    load_at(p + at.lo, lo);
    load_at(p + at.hi, hi);
  }
  __device__ __forceinline__ void store(T* p, const Place<CH>& at) const {
    store_at(p + at.lo, lo);
    store_at(p + at.hi, hi);
  }
  __device__ __forceinline__ void floats(float (&x)[2 * CH]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(lo[i]);
        x[CH + i] = __uint_as_float(hi[i]);
      } else {
        const float2 a = unpack(lo[i], T()), b = unpack(hi[i], T());
        x[2 * i] = a.x, x[2 * i + 1] = a.y, x[CH + 2 * i] = b.x, x[CH + 2 * i + 1] = b.y;
      }
    }
  }
  __device__ __forceinline__ void round(const float (&x)[2 * CH]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) {
        lo[i] = __float_as_uint(x[i]);
        hi[i] = __float_as_uint(x[CH + i]);
      } else {
        lo[i] = pack(x[2 * i], x[2 * i + 1], T());
        hi[i] = pack(x[CH + 2 * i], x[CH + 2 * i + 1], T());
      }
    }
  }
};

// The last b in [0, n) with key(b) <= x, for keys that never fall: a warp looks at 32 places at a time.
template <typename Key>
__device__ __forceinline__ int find_last(int n, int64_t x, Key key) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    const int before = __popc(__ballot_sync(0xffffffffu, b < hi && key(b) <= x));
    lo += max(before - 1, 0) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// A request of a step: its rows, and the place of its first new token. n 0: nothing to serve.
struct StepRequest {
  int row0, n, first, table_row;
};
__device__ __forceinline__ StepRequest step_request(const StepMap& m, int b, uint32_t& err) {
  const int q0 = m.starts[b], q1 = m.starts[b + 1], total = m.totals[b], id = m.ids ? m.ids[b] : b;
  StepRequest r = {q0, 0, total - (q1 - q0), id};
  if (q0 < 0 || q1 < q0 || q1 > m.n_rows) err |= TQ_DEV_ERR_LENGTH;
  else if (q1 > q0 && total != 0) {
    if (total < q1 - q0 || (total - 1) / kPage >= m.max_pages) err |= TQ_DEV_ERR_LENGTH;
    else if (id < 0 || id >= m.max_seqs) err |= TQ_DEV_ERR_SEQ_ID;
    else r.n = q1 - q0;
  }
  return r;
}
// What is wrong with the requests is told apart from serving them: where starts fall or pass the rows, no row may lead to
// the request that does so. The n-th of `ctas` CTAs takes its part, its last warps first (the first ones look for tokens).
__device__ __forceinline__ void report_requests(const StepMap& m, uint32_t* status, int n, int ctas, int threads) {
  if (!status || (int64_t)n * threads >= m.batch) return;
  for (int64_t b = (int64_t)n * threads + threads - 1 - threadIdx.x; b < m.batch; b += (int64_t)ctas * threads) {
    uint32_t err = 0;
    step_request(m, (int)b, err);
    report(status, err);
  }
}

// =============================================================================================
// Rows of queries, keys and values, rotated or copied: a CTA takes `per` tokens with all their heads, a thread 2 CH
// channels of one token, whose cosines and sines it makes once for all heads that it meets. Everything is read and written
// once, and with many heads DRAM bounds it: 16384 rows of 32 heads of 128, a quarter of each turned, 49.8 us, 5.4 TB/s (80 % of a copy);
// 8 prompts of 1024 to 3000 tokens into a pool of 16 bits with 32 query heads 71.8 us, 5.7 TB/s. With few heads angles are made for few
// elements: the same bytes in 65536 rows of 8 heads of 128 66.9 us (59 %), 65536 rows of 2 heads of 256 43 us (46 %: issue slots 63 %
// used, the stalls are waits for loads and for results). A step of 128 tokens takes 3.6 us, a launch and four dependent
// loads (request, table, rows, results).
// =============================================================================================
struct RowsArgs {
  Rotation rot;
  StepMap map;
  const int32_t* positions;
  uint32_t* status;
  const void* x[3];  // queries, keys, values
  void* out[3];
  int64_t x_row[3], x_head[3];
  int64_t o_block[3], o_row[3], o_head[3];  // queries: block 0, their row; others: block and token of the pool
  int heads[3];
  int all;      // heads of a row that are done here: of queries, or of all three
  int d, per, n_rows, n_blocks;
  int step;     // rows go by the map (else each has its position)
  int to_bf16;  // type of the pool
};

constexpr int kRowsThreads = 256;
constexpr int kMostPer = 32;

template <typename T, int CH, bool VEC>
__device__ void rows_part(const RowsArgs& a, int cta, int ctas) {
  struct Token {
    int position, block, place;  // block: -1: no place; -2: the row is not served
  };
  __shared__ Token tokens[kMostPer];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = cta * a.per;
  for (int i = warp; i < a.per; i += kRowsThreads / 32) {
    const int row = row0 + i;
    Token t = {0, -2, 0};
    if (row < a.n_rows) {
      if (!a.step) {
        t = {a.positions[row], -1, 0};
      } else if (a.map.batch > 0) {
        const int b = find_last(a.map.batch, row, [&](int at) { return a.map.starts[at]; });
        uint32_t err = 0, bad = 0;  // of the request: report_requests
        const StepRequest r = step_request(a.map, b, bad);
        if (r.n > 0 && row >= r.row0 && row < r.row0 + r.n) {
          const int at = r.first + (row - r.row0);
          t.position = a.positions ? a.positions[row] : at;
          t.place = at % kPage;
          t.block = -1;
          if (a.all > a.heads[0]) {
            t.block = a.map.table[(int64_t)r.table_row * a.map.stride + at / kPage];
            if (t.block < 0 || t.block >= a.n_blocks) {
              err |= TQ_DEV_ERR_BLOCK;
              t.block = -1;
            }
          }
        }
        if (lane == 0) report(a.status, err);
      }
    }
    if (lane == 0) tokens[i] = t;
  }
  if (ctas > 0) report_requests(a.map, a.status, cta, ctas, kRowsThreads);
  named_barrier(1, kRowsThreads);
  const int threads = a.d / (2 * CH);  // of one head
  const int groups = kRowsThreads / threads, g = threadIdx.x / threads, j = threadIdx.x - g * threads;
  if (g >= groups - groups % a.per) return;
  const Token t = tokens[g % a.per];
  const int row = row0 + g % a.per;
  if (t.block == -2) return;
  const Place<CH> at(a.rot, j);
  Turned<CH> turned;
  if (at.turned) {
    uint64_t turns[CH];
    load_turns<CH>(a.rot, j, turns);
    turned.at(a.rot, turns, t.position);
  }
  const int step = groups / a.per;
  constexpr int kBatch = 2;  // heads whose loads are in flight together (4 leave room for two CTAs on an SM: 75.5 us, so 71.4)
  for (int h0 = g / a.per; h0 < a.all; h0 += kBatch * step) {
    Pieces<T, CH, VEC> in[kBatch];
    int which[kBatch], head[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * step;
      which[i] = h < a.heads[0] ? 0 : h < a.heads[0] + a.heads[1] ? 1 : 2;
      head[i] = h - (which[i] > 0 ? a.heads[0] : 0) - (which[i] > 1 ? a.heads[1] : 0);
      if (h >= a.all || (which[i] > 0 && t.block < 0)) which[i] = -1;
      else in[i].load(static_cast<const T*>(a.x[which[i]]) + (int64_t)row * a.x_row[which[i]] + (int64_t)head[i] * a.x_head[which[i]], at);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int w = which[i];
      if (w < 0) continue;
      float x[2 * CH];
      in[i].floats(x);
      if (at.turned && w < 2) turned.apply(a.rot, x);
      const int64_t to = w == 0 ? (int64_t)row * a.o_row[0] : (int64_t)t.block * a.o_block[w] + (int64_t)t.place * a.o_row[w];
      const int64_t off = to + (int64_t)head[i] * a.o_head[w];
      if (w == 0) {
        Pieces<T, CH, VEC> o;
        o.round(x);
        o.store(static_cast<T*>(a.out[0]) + off, at);
      } else if (a.to_bf16) {
        Pieces<__nv_bfloat16, CH, VEC> o;
        o.round(x);
        o.store(static_cast<__nv_bfloat16*>(a.out[w]) + off, at);
      } else {
        Pieces<__half, CH, VEC> o;
        o.round(x);
        o.store(static_cast<__half*>(a.out[w]) + off, at);
      }
    }
  }
}

template <typename T, int CH, bool VEC>
__global__ void __launch_bounds__(kRowsThreads, 3) k_rotate_rows(const __grid_constant__ RowsArgs a) {
  pdl_wait();
  rows_part<T, CH, VEC>(a, blockIdx.x, a.step ? gridDim.x : 0);
}

int rows_ctas(RowsArgs& a, int ch, int sms) {
  const int groups = kRowsThreads / (a.d / (2 * ch));
  // Up to 8 tokens of a CTA, where there are enough for a CTA on each SM: a thread makes its angles for more heads (2048 tokens of
  // 32 heads of 128: 15.4 us with 8 CTAs on each SM, 9.2 so). More where a token has fewer heads than threads.
  a.per = 1;
  while (a.per < kMostPer && 2 * a.per <= groups && a.n_rows / (2 * a.per) >= sms && (a.per < 8 || groups / a.per > a.all))
    a.per *= 2;
  return (a.n_rows + a.per - 1) / a.per;
}

// =============================================================================================
// Into pages of 8 bits. A CTA takes one page of one request and every Y-th of its 2 x n_kv_heads items (keys or values
// of a head). Runs of up to kShort new tokens take a warp per item, longer ones the CTA. The rows stay in registers, as they
// came, between the largest of them and their rounding, so that everything is read once; K is rotated twice for that, with
// cosines and sines that a thread makes once for all heads and keeps in shared memory of its own (4 x 8 pairs: registers
// would leave one CTA to an SM). The 14 warps that fit an SM beside that memory bound it: 65536 tokens of 8 heads of 128 in bf16
// 82 us, 4.8 TB/s (70 % of a copy) with issue slots half used; at head_dim 256, with one CTA to an SM, 66 %; at 64 58 %, with
// queries 51 %. A step of 128 tokens takes 6.4 us.
// Page j of request b has number starts[b] / 128 + 2 b + j: n new tokens touch at most n / 128 + 2 pages, so numbers
// never meet, and a CTA finds its request from starts alone.
// =============================================================================================
struct PagesArgs {
  RowsArgs rows;  // queries, and all that both need
  tq_scales scales;
  int pages, y;   // CTAs: pages * y, then those of the queries
};
constexpr int kShort = 8;
constexpr int kLeast = -60, kMost = 60;

// 16 bytes to shared memory, not waited for.
__device__ __forceinline__ void copy_async(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
// Four numbers of e4m3, to nearest even, at most 448; and two as floats.
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}\n"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_floats(uint32_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)x));
  return __half22float2(*reinterpret_cast<__half2*>(&r));
}

// The scale of values up to `top` (finite): the smallest power of two with top <= 448 = 1.75 * 2^8 scales.
__device__ __forceinline__ float scale_of(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = (int)(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return __uint_as_float((uint32_t)(min(max(e, kLeast), kMost) + 127) << 23);
}
// The smallest power of two that is at least s, a positive normal number (or 0, which stays).
__device__ __forceinline__ float power_up(float s) {
  const uint32_t u = __float_as_uint(s);
  return __uint_as_float(u & 0x7fffffu ? (u & 0x7f800000u) + 0x800000u : u);
}

template <int N>
__device__ __forceinline__ float largest(const float (&x)[N], float top) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float v = fabsf(x[i]);
    top = fmaxf(top, v < INFINITY ? v : 0.f);
  }
  return top;
}

// The largest of x and top, infinite where one is (NaN does not count).
template <int N>
__device__ __forceinline__ float largest_any(const float (&x)[N], float top) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(top), "f"(fabsf(x[i])), "f"(fabsf(x[i + 1])));
    top = r;
  }
  return top;
}

template <int CH>
__device__ __forceinline__ void store8(uint8_t* p, const Place<CH>& at, const float (&x)[2 * CH], float by) {
  uint32_t w[CH / 2];
#pragma unroll
  for (int i = 0; i < CH / 2; ++i) {
    const float2 a = mul2(make_float2(x[4 * i], x[4 * i + 1]), both(by)), b = mul2(make_float2(x[4 * i + 2], x[4 * i + 3]), both(by));
    w[i] = e4m3x4(a, b);
  }
  if constexpr (CH == 8) {
    *reinterpret_cast<uint2*>(p + at.lo) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(p + at.hi) = make_uint2(w[2], w[3]);
  } else {
    *reinterpret_cast<uint32_t*>(p + at.lo) = w[0];
    *reinterpret_cast<uint32_t*>(p + at.hi) = w[1];
  }
}

// The first `n` tokens of a page and head times `by`, by `threads` threads of which this is the id-th.
template <int D>
__device__ __forceinline__ void rescale(uint8_t* page, int64_t row, int n, float by, int id, int threads) {
  constexpr int kPer = D / 16;
  for (int i0 = id; i0 < n * kPer; i0 += 4 * threads) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * threads;
      if (i < n * kPer) v[k] = *reinterpret_cast<const uint4*>(page + (int64_t)(i / kPer) * row + (i % kPer) * 16);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * threads;
      if (i >= n * kPer) break;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v[k]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 x = e4m3x2_floats(w[q] & 0xffffu), y = e4m3x2_floats(w[q] >> 16);
        w[q] = e4m3x4(mul2(x, both(by)), mul2(y, both(by)));
      }
      *reinterpret_cast<uint4*>(page + (int64_t)(i / kPer) * row + (i % kPer) * 16) = v[k];
    }
  }
}

template <int D, int CH, int SIZE>
struct PagesShape {
  static constexpr int kThreads = D == 256 ? 512 : 256;
  static constexpr int kHead = D / (2 * CH);  // threads of a token's head
  static constexpr int kRun = kThreads / kHead;  // tokens that the CTA has in one pass
  static constexpr int kPasses = (kPage + kRun - 1) / kRun;
  // Rows of 16 bits in pieces of 16 bytes are fetched an item ahead, into shared memory that is each thread's own.
  static constexpr bool kAhead = CH == 8 && SIZE == 2;
  static constexpr int kAngles = kPasses * kThreads * CH * 8;  // bytes of cosines and sines
  static constexpr int kSmem = kAngles + (kAhead ? kPasses * kThreads * 32 : 0);
};

template <typename T, int D, int CH, bool VEC>
__device__ void pages_part(const PagesArgs& p) {
  using Sh = PagesShape<D, CH, sizeof(T)>;
  constexpr int kThreads = Sh::kThreads, kWarps = kThreads / 32, kHead = Sh::kHead, kRun = Sh::kRun, kPasses = Sh::kPasses;
  constexpr int kWarpRun = 32 / kHead, kWarpPasses = kShort / kWarpRun;
  extern __shared__ float4 angles[];  // [pass][CH / 2][thread]: cosines and sines of two pairs
  __shared__ float tops[2][kWarps];
  const RowsArgs& a = p.rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int number = blockIdx.x / p.y, y = blockIdx.x - number * p.y;
  const int b = find_last(a.map.batch, number, [&](int i) { return (int64_t)(max(a.map.starts[i], 0) / kPage) + 2 * i; });
  uint32_t bad = 0;  // report_requests
  const StepRequest r = step_request(a.map, b, bad);
  const int nth = number - (max(a.map.starts[b], 0) / kPage + 2 * b);
  if (r.n == 0 || nth < 0) return;
  const int page = r.first / kPage + nth, total = r.first + r.n;
  if (page > (total - 1) / kPage) return;
  const int lo = max(r.first, page * kPage), n = min(total, (page + 1) * kPage) - lo, at0 = lo - page * kPage;
  const int row0 = r.row0 + lo - r.first;
  const int block = a.map.table[(int64_t)r.table_row * a.map.stride + page];
  if (block < 0 || block >= a.n_blocks) {
    if (threadIdx.x == 0 && y == 0) report(a.status, TQ_DEV_ERR_BLOCK);
    return;
  }
  const int hkv = a.heads[1], items = 2 * hkv;
  auto scale_at = [&](int w, int h) {
    return (w ? p.scales.v + (int64_t)block * p.scales.v_block : p.scales.k + (int64_t)block * p.scales.k_block) + h;
  };
  const bool alone = n <= kShort;
  const int id = alone ? lane : threadIdx.x, j = id % kHead, run0 = id / kHead;
  const Place<CH> at(a.rot, j);
  uint64_t turns[CH];
  if (at.turned) load_turns<CH>(a.rot, j, turns);
  auto load = [&](int w, int h, int i, Pieces<T, CH, VEC>& in) {  // new token i of the page
    in.load(static_cast<const T*>(a.x[1 + w]) + (int64_t)(row0 + i) * a.x_row[1 + w] + (int64_t)h * a.x_head[1 + w], at);
  };
  auto turn_to = [&](int i, Turned<CH>& t) { t.at(a.rot, turns, a.positions ? a.positions[row0 + i] : lo + i); };
  if (alone) {
    for (int item = y + p.y * warp; item < items; item += p.y * kWarps) {
      const int w = item >= hkv, h = item - w * hkv;
      uint8_t* const to = static_cast<uint8_t*>(a.out[1 + w]) + (int64_t)block * a.o_block[1 + w] + (int64_t)h * a.o_head[1 + w];
      float x[kWarpPasses][2 * CH], top = 0.f;
#pragma unroll
      for (int k = 0; k < kWarpPasses; ++k) {
        const int i = k * kWarpRun + run0;
        if (i < n) {
          Pieces<T, CH, VEC> in;
          load(w, h, i, in);
          in.floats(x[k]);
          if (w == 0 && at.turned) {
            Turned<CH> t;
            turn_to(i, t);
            t.apply(a.rot, x[k]);
          }
          top = largest<2 * CH>(x[k], top);
        }
      }
      const float held = at0 ? clamp_scale(*scale_at(w, h)) : 0.f;  // a caller's need not be a power of two
      const float scale = fmaxf(power_up(held), scale_of(warp_max(top))), by = 1.f / scale;
      if (at0 && scale > held) rescale<D>(to, a.o_row[1 + w], at0, held / scale, lane, 32);
#pragma unroll
      for (int k = 0; k < kWarpPasses; ++k) {
        const int i = k * kWarpRun + run0;
        if (i < n) store8<CH>(to + (int64_t)(at0 + i) * a.o_row[1 + w], at, x[k], by);
      }
      if (lane == 0) *scale_at(w, h) = scale;
    }
    return;
  }
  float4* const mine = angles + threadIdx.x;
  uint4* const ahead = reinterpret_cast<uint4*>(angles) + Sh::kAngles / 16 + threadIdx.x;  // [pass][lo, hi][thread]
  auto fetch = [&](int item) {
    const int w = item >= hkv, h = item - w * hkv;
    const T* p = static_cast<const T*>(a.x[1 + w]) + (int64_t)(row0 + run0) * a.x_row[1 + w] + (int64_t)h * a.x_head[1 + w];
#pragma unroll
    for (int k = 0; k < kPasses; ++k, p += kRun * a.x_row[1 + w]) {
      if (k * kRun + run0 >= n) break;
      copy_async(ahead + 2 * k * kThreads, p + at.lo);
      copy_async(ahead + (2 * k + 1) * kThreads, p + at.hi);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  if (Sh::kAhead && y < items) fetch(y);
  if (at.turned && y < hkv) {
#pragma unroll 1
    for (int k = 0; k < kPasses; ++k) {
      if (k * kRun + run0 >= n) break;
      Turned<CH> t;
      turn_to(k * kRun + run0, t);
#pragma unroll
      for (int i = 0; i < CH / 2; ++i)
        mine[(k * (CH / 2) + i) * kThreads] = make_float4(t.c[i].x, t.c[i].y, t.s[i].x, t.s[i].y);
    }
  }
  int buf = 0;
  for (int item = y; item < items; item += p.y) {
    const int w = item >= hkv, h = item - w * hkv;
    uint8_t* const to = static_cast<uint8_t*>(a.out[1 + w]) + (int64_t)block * a.o_block[1 + w] + (int64_t)h * a.o_head[1 + w];
    Pieces<T, CH, VEC> in[kPasses];
    if constexpr (Sh::kAhead) asm volatile("cp.async.wait_group 0;\n" ::: "memory");
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      if (k * kRun + run0 >= n) continue;
      if constexpr (Sh::kAhead) {
        const uint4 l = ahead[2 * k * kThreads], u = ahead[(2 * k + 1) * kThreads];
        in[k].lo[0] = l.x, in[k].lo[1] = l.y, in[k].lo[2] = l.z, in[k].lo[3] = l.w;
        in[k].hi[0] = u.x, in[k].hi[1] = u.y, in[k].hi[2] = u.z, in[k].hi[3] = u.w;
      } else {
        load(w, h, k * kRun + run0, in[k]);
      }
    }
    auto values = [&](int k, float (&x)[2 * CH]) {
      in[k].floats(x);
      if (w == 0 && at.turned) {
        Turned<CH> t;
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          const float4 v = mine[(k * (CH / 2) + i) * kThreads];
          t.c[i] = make_float2(v.x, v.y);
          t.s[i] = make_float2(v.z, v.w);
        }
        t.apply(a.rot, x);
      }
    };
    auto top_of = [&](auto largest_of, bool first) {  // over the CTA
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        if (k * kRun + run0 < n) {
          float x[2 * CH];
          values(k, x);
          top = largest_of(x, top);
        }
      }
      top = warp_max(top);
      if (Sh::kAhead && first && item + p.y < items) fetch(item + p.y);  // behind the last use of what it replaces
      if (lane == 0) tops[buf][warp] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWarps; ++i) top = fmaxf(top, tops[buf][i]);
      buf ^= 1;
      return top;
    };
    const float held = at0 ? clamp_scale(*scale_at(w, h)) : 0.f;
    float top = top_of([](const float (&x)[2 * CH], float t) { return largest_any<2 * CH>(x, t); }, true);
    if (top == INFINITY) top = top_of([](const float (&x)[2 * CH], float t) { return largest<2 * CH>(x, t); }, false);
    const float scale = fmaxf(power_up(held), scale_of(top)), by = 1.f / scale;
    if (at0 && scale > held) rescale<D>(to, a.o_row[1 + w], at0, held / scale, threadIdx.x, kThreads);
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int i = k * kRun + run0;
      if (i < n) {
        float x[2 * CH];
        values(k, x);
        store8<CH>(to + (int64_t)(at0 + i) * a.o_row[1 + w], at, x, by);
      }
    }
    if (threadIdx.x == 0) *scale_at(w, h) = scale;
  }
}

template <typename T, int D, int CH, bool VEC>
__global__ void __launch_bounds__(PagesShape<D, CH, sizeof(T)>::kThreads, D == 256 ? 1 : 2) k_extend_pages(const __grid_constant__ PagesArgs p) {
  pdl_wait();
  const int queries = p.pages * p.y;
  if ((int)blockIdx.x < queries) {
    pages_part<T, D, CH, VEC>(p);
    // first by the CTAs of page number 1, which a step of single tokens leaves idle
    report_requests(p.rows.map, p.rows.status, ((int)blockIdx.x < p.y ? (int)blockIdx.x + queries : (int)blockIdx.x) - p.y, queries, blockDim.x);
  } else if (threadIdx.x < kRowsThreads) {
    rows_part<T, CH, VEC>(p.rows, blockIdx.x - queries, 0);
  }
}

template <typename T, int D, int CH, bool VEC>
cudaError_t launch_pages_as(const PagesArgs& p, unsigned grid, cudaStream_t s) {
  using Sh = PagesShape<D, CH, sizeof(T)>;
  static std::atomic<uint64_t> known{0};  // devices whose kernel may use kSmem
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (e == cudaSuccess && !(known.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k_extend_pages<T, D, CH, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e == cudaSuccess) known.fetch_or(bit, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  // without a run that the CTA takes together nothing is kept
  return launch_pdl(k_extend_pages<T, D, CH, VEC>, dim3(grid), dim3(Sh::kThreads), p.rows.n_rows > kShort ? Sh::kSmem : 0, s, p);
}

template <typename T, int CH, bool VEC>
cudaError_t launch_pages_d(PagesArgs& p, int sms, cudaStream_t s) {
  RowsArgs& a = p.rows;
  RowsArgs q = a;
  const int query_ctas = a.heads[0] ? rows_ctas(q, CH, sms) : 0;
  a.per = q.per;
  const int64_t grid = (int64_t)p.pages * p.y + query_ctas;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (a.d == 64) return launch_pages_as<T, 64, CH, VEC>(p, (unsigned)grid, s);
  if (a.d == 128) return launch_pages_as<T, 128, CH, VEC>(p, (unsigned)grid, s);
  return launch_pages_as<T, 256, CH, VEC>(p, (unsigned)grid, s);
}

template <typename T>
cudaError_t launch_pages(PagesArgs& p, bool vec, int sms, cudaStream_t s) {
  return vec ? launch_pages_d<T, 8, true>(p, sms, s) : launch_pages_d<T, 4, false>(p, sms, s);
}

// Vectors that addresses, strides and the channels' cut allow: 8 pairs of a thread in 16 bytes (2 of them in fp32), 4 pairs in
// vectors of half that, or 4 pairs one by one.
enum Width { kOneByOne, kFour, kEight };
constexpr int64_t kManyQueries = 8 << 20;  // elements

Width width_of(const Rotation& r, int d) { return r.pairs % 8 == 0 && d % 16 == 0 ? kEight : kFour; }
Width width_of(Width w, const void* p, int64_t row, int64_t head, int size) {
  while (w != kOneByOne) {
    const int bytes = w == kEight ? 16 : 4 * size;
    if ((uintptr_t)p % bytes == 0 && row * size % bytes == 0 && head * size % bytes == 0) break;
    w = (Width)(w - 1);
  }
  return w;
}

template <typename T>
cudaError_t launch_rows(RowsArgs& a, Width w, int sms, cudaStream_t s) {
  // 4 pairs also where a thread's angles serve few heads (65536 tokens of 2 heads of 256: 43 us, with 8 pairs 63; 16384 of 32
  // heads of 128 53.8 and 49.4), and in fp32, whose vectors are 16 bytes all the same (rows into bf16 50.7 and 53.3)
  if (w == kEight && (sizeof(T) == 4 || a.all <= 4)) w = kFour;
  const int ctas = rows_ctas(a, w == kEight ? 8 : 4, sms);
  if constexpr (sizeof(T) == 2) {
    if (w == kEight) return launch_pdl(k_rotate_rows<T, 8, true>, dim3(ctas), dim3(kRowsThreads), 0, s, a);
  }
  if (w == kFour) return launch_pdl(k_rotate_rows<T, 4, true>, dim3(ctas), dim3(kRowsThreads), 0, s, a);
  return launch_pdl(k_rotate_rows<T, 4, false>, dim3(ctas), dim3(kRowsThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_rotate(const Rotation& r, const void* x, void* out, int dt, const int64_t* xs, const int64_t* os,
                          const int32_t* positions, int n_tokens, int heads, int d, int sms, cudaStream_t s) {
  RowsArgs a = {};
  a.rot = r;
  a.positions = positions;
  a.x[0] = x;
  a.out[0] = out;
  a.x_row[0] = xs[0];
  a.x_head[0] = xs[1];
  a.o_row[0] = os[0];
  a.o_head[0] = os[1];
  a.heads[0] = a.all = heads;
  a.d = d;
  a.n_rows = n_tokens;
  const int size = dt == TQ_F32 ? 4 : 2;
  const Width vec = width_of(width_of(width_of(r, d), x, xs[0], xs[1], size), out, os[0], os[1], size);
  if (dt == TQ_BF16) return launch_rows<__nv_bfloat16>(a, vec, sms, s);
  if (dt == TQ_F16) return launch_rows<__half>(a, vec, sms, s);
  return launch_rows<float>(a, vec, sms, s);
}

cudaError_t launch_paged_extend(const tq_kv& pool, const tq_scales* scales, const tq_new_rows& n, const Rotation& r,
                                const StepMap& m, uint32_t* status, int sms, cudaStream_t s) {
  PagesArgs p = {};
  RowsArgs& a = p.rows;
  a.rot = r;
  a.map = m;
  a.positions = n.d_positions;
  a.status = status;
  a.step = 1;
  a.d = pool.head_dim;
  a.n_rows = n.n_rows;
  a.n_blocks = pool.outer;
  a.to_bf16 = pool.dtype == TQ_BF16;
  const int size = n.dtype == TQ_F32 ? 4 : 2;
  const void* x[3] = {n.q, n.k, n.v};
  void* out[3] = {n.q_out, pool.k, pool.v};
  const int64_t* xs[3] = {n.q_strides, n.k_strides, n.v_strides};
  const int64_t* os[3] = {n.q_out_strides, pool.k_strides, pool.v_strides};
  Width vec = width_of(r, a.d);
  for (int w = 0; w < 3; ++w) {
    a.heads[w] = w == 0 ? (n.q ? n.n_q_heads : 0) : pool.n_kv_heads;
    if (!a.heads[w]) continue;
    a.x[w] = x[w];
    a.out[w] = out[w];
    a.x_row[w] = xs[w][0];
    a.x_head[w] = xs[w][1];
    if (w > 0) a.o_block[w] = os[w][0];
    a.o_row[w] = os[w][w > 0];
    a.o_head[w] = os[w][1 + (w > 0)];
    vec = width_of(vec, x[w], a.x_row[w], a.x_head[w], size);
    // pages of 8 bits have their alignment checked
    if (w == 0 || !scales) vec = width_of(width_of(vec, out[w], a.o_row[w], a.o_head[w], w == 0 ? size : 2), nullptr, a.o_block[w], 0, 2);
  }
  a.all = a.heads[0] + (scales ? 0 : a.heads[1] + a.heads[2]);
  if (!scales) {
    if (n.dtype == TQ_BF16) return launch_rows<__nv_bfloat16>(a, vec, sms, s);
    if (n.dtype == TQ_F16) return launch_rows<__half>(a, vec, sms, s);
    return launch_rows<float>(a, vec, sms, s);
  }
  p.scales = *scales;
  // Many queries take a launch of their own, whose CTAs leave each other more room (37000 tokens of 4 heads and 16 query heads of
  // 64: 72.6 us in one launch, 65.1 in two; 8 requests of 128 tokens, 8 and 32 heads of 128, 13.1 and 16.6).
  if (a.heads[0] && (int64_t)n.n_rows * a.heads[0] * a.d >= kManyQueries) {
    RowsArgs q = a;
    const Width w = width_of(width_of(width_of(r, a.d), x[0], a.x_row[0], a.x_head[0], size), out[0], a.o_row[0], a.o_head[0], size);
    const cudaError_t e = n.dtype == TQ_BF16  ? launch_rows<__nv_bfloat16>(q, w, sms, s)
                          : n.dtype == TQ_F16 ? launch_rows<__half>(q, w, sms, s)
                                              : launch_rows<float>(q, w, sms, s);
    if (e != cudaSuccess) return e;
    a.heads[0] = a.all = 0;
  }
  p.pages = n.n_rows / kPage + 2 * m.batch;
  const int items = 2 * pool.n_kv_heads, warps = a.d == 256 ? 16 : 8;
  // Items per CTA: all warps busy in short runs; in long ones as many as leave a CTA or two to each SM, for the angles are made once
  // for all of a CTA's (37000 tokens of 4 heads of 256: 79 us with 8 CTAs to each SM, 49 with one).
  const int likely = std::max(1, n.n_rows / kPage + m.batch);
  const int most = n.n_rows / std::max(1, m.batch) > kShort ? items : (items + warps - 1) / warps;
  const int want = a.d == 256 ? sms : 2 * sms;
  p.y = std::min(most, std::max(1, (want + likely - 1) / likely));
  if (n.dtype == TQ_BF16) return launch_pages<__nv_bfloat16>(p, vec == kEight, sms, s);
  if (n.dtype == TQ_F16) return launch_pages<__half>(p, vec == kEight, sms, s);
  return launch_pages<float>(p, vec == kEight, sms, s);
}

}  // namespace tq
