// Rotary positions, and a step's new tokens rotated on their way into a paged cache of 16 or 8 bits: tq_rotate,
// tq_paged_extend.
#include <algorithm>
#include <cmath>

#include "tq_device.cuh"

namespace tq {
namespace {

__device__ __forceinline__ void report(uint32_t* status, uint32_t bits) {
  if (bits && status) atomicOr(status, bits);
}

// ---- rotation ----

// Cosine and sine of position * turns (turns in 2^-64 of a whole turn), times factor. The product modulo 2^64 is the angle
// modulo a turn without error; its upper 32 bits are taken to the nearest quarter turn before they become a float, so
// that the rest, at most an eighth of a turn, is rounded to 2^-25 of itself.
__device__ __forceinline__ void turn(int position, uint64_t turns, float factor, float& c, float& s) {
  const uint32_t f = (uint32_t)(((uint64_t)(int64_t)position * turns) >> 32);
  const uint32_t q = (f + (1u << 29)) >> 30;
  const float x = (float)(int32_t)(f - (q << 30)) * 4.656612873077392578125e-10f;  // 2^-31: in half turns
  float cx, sx;
  sincospif(x, &sx, &cx);
  cx *= factor;
  sx *= factor;
  const float a = q & 1 ? sx : cx, b = q & 1 ? cx : sx;
  c = (q + 1) & 2 ? -a : a;
  s = q & 2 ? -b : b;
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

template <int CH>
struct Turned {
  float c[CH], s[CH];
  __device__ __forceinline__ void at(const Rotation& r, const uint64_t (&turns)[CH], int position) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      turn(position, turns[i], r.factor, c[i], s[i]);
      if (r.inverse) s[i] = -s[i];
    }
  }
  __device__ __forceinline__ void apply(const Rotation& r, float (&x)[2 * CH]) const {
    if (r.interleaved) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * c[i] - b * s[i];
        x[2 * i + 1] = b * c[i] + a * s[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const float a = x[i], b = x[CH + i];
        x[i] = a * c[i] - b * s[i];
        x[CH + i] = b * c[i] + a * s[i];
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

template <typename T>
__device__ __forceinline__ float as_float(T x) {
  return static_cast<float>(x);
}

// CH elements at each of two places. VEC: 16-byte aligned.
template <typename T, int CH, bool VEC>
struct Pieces {
  alignas(16) T lo[CH], hi[CH];
  __device__ __forceinline__ void load(const T* p, const Place<CH>& at) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < (int)(CH * sizeof(T) / 16); ++i) {
        reinterpret_cast<uint4*>(lo)[i] = *(reinterpret_cast<const uint4*>(p + at.lo) + i);
        reinterpret_cast<uint4*>(hi)[i] = *(reinterpret_cast<const uint4*>(p + at.hi) + i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        lo[i] = p[at.lo + i];
        hi[i] = p[at.hi + i];
      }
    }
  }
  __device__ __forceinline__ void floats(float (&x)[2 * CH]) const {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      x[i] = as_float(lo[i]);
      x[CH + i] = as_float(hi[i]);
    }
  }
  __device__ __forceinline__ void round(const float (&x)[2 * CH]) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      lo[i] = T(x[i]);
      hi[i] = T(x[CH + i]);
    }
  }
  __device__ __forceinline__ void store(T* p, const Place<CH>& at) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < (int)(CH * sizeof(T) / 16); ++i) {
        *(reinterpret_cast<uint4*>(p + at.lo) + i) = reinterpret_cast<const uint4*>(lo)[i];
        *(reinterpret_cast<uint4*>(p + at.hi) + i) = reinterpret_cast<const uint4*>(hi)[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        p[at.lo + i] = lo[i];
        p[at.hi + i] = hi[i];
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

// =============================================================================================
// Rows of queries, keys and values, rotated or copied: a CTA takes `per` tokens with all their heads, a thread 2 CH
// channels of one token, whose cosines and sines it makes once for all heads that it meets.
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
constexpr int kMostPer = 8;

template <typename T, int CH, bool VEC>
__device__ void rows_part(const RowsArgs& a, int cta) {
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
        uint32_t err = 0;
        const StepRequest r = step_request(a.map, b, err);
        if (r.n > 0 && row >= r.row0 && row < r.row0 + r.n) {
          const int at = r.first + row - r.row0;
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
  constexpr int kBatch = sizeof(T) == 4 ? 2 : 4;  // heads whose loads are in flight together
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
__global__ void __launch_bounds__(kRowsThreads) k_rotate_rows(const __grid_constant__ RowsArgs a) {
  pdl_wait();
  rows_part<T, CH, VEC>(a, blockIdx.x);
}

int rows_ctas(RowsArgs& a, int ch, int sms) {
  const int groups = kRowsThreads / (a.d / (2 * ch));
  a.per = 1;  // up to 8 tokens of a CTA, where there are enough for 8 CTAs on each SM
  while (a.per < kMostPer && 2 * a.per <= groups && a.n_rows / (2 * a.per) >= 8 * sms) a.per *= 2;
  return (a.n_rows + a.per - 1) / a.per;
}

// =============================================================================================
// Into pages of 8 bits. A CTA takes one page of one request and every Y-th of its 2 x n_kv_heads items (keys or values
// of a head). Runs of up to kShort new tokens take a warp per item, longer ones the CTA; the rotated values stay in registers
// between the largest of them and their rounding, so that everything is read once.
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

// Two numbers of e4m3, to nearest even, at most 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
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
// The scale that a block has already; what is none counts as the least.
__device__ __forceinline__ float held_scale(float s) {
  constexpr float kLo = 8.67361737988403547205962240695953369140625e-19f;  // 2^-60
  return s >= kLo && s <= 1.f / kLo ? s : kLo;
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

template <int CH>
__device__ __forceinline__ void store8(uint8_t* p, const Place<CH>& at, const float (&x)[2 * CH], float by) {
  uint32_t w[CH / 2];
#pragma unroll
  for (int i = 0; i < CH / 2; ++i)
    w[i] = e4m3x2(x[4 * i] * by, x[4 * i + 1] * by) | e4m3x2(x[4 * i + 2] * by, x[4 * i + 3] * by) << 16;
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
        w[q] = e4m3x2(x.x * by, x.y * by) | e4m3x2(y.x * by, y.y * by) << 16;
      }
      *reinterpret_cast<uint4*>(page + (int64_t)(i / kPer) * row + (i % kPer) * 16) = v[k];
    }
  }
}

template <int D>
struct PagesShape {
  static constexpr int kThreads = D == 256 ? 512 : 256;
};

template <typename T, int D, int CH, bool VEC>
__device__ void pages_part(const PagesArgs& p) {
  constexpr int kThreads = PagesShape<D>::kThreads, kWarps = kThreads / 32;
  constexpr int kHead = D / (2 * CH);           // threads of a token's head
  constexpr int kRun = kThreads / kHead;        // tokens that the CTA has in one pass
  constexpr int kPasses = (kPage + kRun - 1) / kRun;
  constexpr int kWarpRun = 32 / kHead, kWarpPasses = kShort / kWarpRun;
  __shared__ float tops[2][kWarps];
  const RowsArgs& a = p.rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int number = blockIdx.x / p.y, y = blockIdx.x - number * p.y;
  const int b = find_last(a.map.batch, number, [&](int i) { return (int64_t)(max(a.map.starts[i], 0) / kPage) + 2 * i; });
  uint32_t err = 0;
  const StepRequest r = step_request(a.map, b, err);
  const int nth = number - (max(a.map.starts[b], 0) / kPage + 2 * b);
  const bool tells = threadIdx.x == 0 && y == 0;
  if (r.n == 0 || nth < 0) {
    if (tells && nth == 0) report(a.status, err);
    return;
  }
  const int page = r.first / kPage + nth, total = r.first + r.n;
  if (page > (total - 1) / kPage) return;
  const int lo = max(r.first, page * kPage), n = min(total, (page + 1) * kPage) - lo, at0 = lo - page * kPage;
  const int row0 = r.row0 + lo - r.first;
  const int block = a.map.table[(int64_t)r.table_row * a.map.stride + page];
  if (block < 0 || block >= a.n_blocks) {
    if (tells) report(a.status, TQ_DEV_ERR_BLOCK);
    return;
  }
  const int hkv = a.heads[1], items = 2 * hkv;
  float* const scales[2] = {p.scales.k + (int64_t)block * p.scales.k_block, p.scales.v + (int64_t)block * p.scales.v_block};
  const bool alone = n <= kShort;
  const int id = alone ? lane : threadIdx.x, j = id % kHead, run0 = id / kHead;
  const Place<CH> at(a.rot, j);
  uint64_t turns[CH];
  if (at.turned) load_turns<CH>(a.rot, j, turns);
  auto load = [&](int w, int h, int i, float (&x)[2 * CH]) {  // new token i of the page, rotated
    Pieces<T, CH, VEC> in;
    in.load(static_cast<const T*>(a.x[1 + w]) + (int64_t)(row0 + i) * a.x_row[1 + w] + (int64_t)h * a.x_head[1 + w], at);
    in.floats(x);
    if (w == 0 && at.turned) {
      Turned<CH> t;
      t.at(a.rot, turns, a.positions ? a.positions[row0 + i] : lo + i);
      t.apply(a.rot, x);
    }
  };
  if (alone) {
    for (int item = y + p.y * warp; item < items; item += p.y * kWarps) {
      const int w = item >= hkv, h = item - w * hkv;
      uint8_t* const to = static_cast<uint8_t*>(a.out[1 + w]) + (int64_t)block * a.o_block[1 + w] + (int64_t)h * a.o_head[1 + w];
      float x[kWarpPasses][2 * CH], top = 0.f;
#pragma unroll
      for (int k = 0; k < kWarpPasses; ++k) {
        const int i = k * kWarpRun + run0;
        if (i < n) {
          load(w, h, i, x[k]);
          top = largest<2 * CH>(x[k], top);
        }
      }
      const float held = at0 ? held_scale(scales[w][h]) : 0.f;
      const float scale = fmaxf(held, scale_of(warp_max(top))), by = 1.f / scale;
      if (at0 && scale > held) rescale<D>(to, a.o_row[1 + w], at0, held / scale, lane, 32);
#pragma unroll
      for (int k = 0; k < kWarpPasses; ++k) {
        const int i = k * kWarpRun + run0;
        if (i < n) store8<CH>(to + (int64_t)(at0 + i) * a.o_row[1 + w], at, x[k], by);
      }
      if (lane == 0) scales[w][h] = scale;
    }
    return;
  }
  int buf = 0;
  for (int item = y; item < items; item += p.y, buf ^= 1) {
    const int w = item >= hkv, h = item - w * hkv;
    uint8_t* const to = static_cast<uint8_t*>(a.out[1 + w]) + (int64_t)block * a.o_block[1 + w] + (int64_t)h * a.o_head[1 + w];
    float x[kPasses][2 * CH], top = 0.f;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int i = k * kRun + run0;
      if (i < n) {
        load(w, h, i, x[k]);
        top = largest<2 * CH>(x[k], top);
      }
    }
    const float held = at0 ? held_scale(scales[w][h]) : 0.f;
    top = warp_max(top);
    if (lane == 0) tops[buf][warp] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, tops[buf][i]);
    const float scale = fmaxf(held, scale_of(top)), by = 1.f / scale;
    if (at0 && scale > held) rescale<D>(to, a.o_row[1 + w], at0, held / scale, threadIdx.x, kThreads);
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int i = k * kRun + run0;
      if (i < n) store8<CH>(to + (int64_t)(at0 + i) * a.o_row[1 + w], at, x[k], by);
    }
    if (threadIdx.x == 0) scales[w][h] = scale;
  }
}

template <typename T, int D, int CH, bool VEC>
__global__ void __launch_bounds__(PagesShape<D>::kThreads) k_extend_pages(const __grid_constant__ PagesArgs p) {
  pdl_wait();
  const int queries = p.pages * p.y;
  if ((int)blockIdx.x < queries) pages_part<T, D, CH, VEC>(p);
  else if (threadIdx.x < kRowsThreads) rows_part<T, CH, VEC>(p.rows, blockIdx.x - queries);
}

template <typename T, int CH, bool VEC>
cudaError_t launch_pages_d(PagesArgs& p, int sms, cudaStream_t s) {
  RowsArgs& a = p.rows;
  RowsArgs q = a;
  const int query_ctas = a.heads[0] ? rows_ctas(q, CH, sms) : 0;
  a.per = q.per;
  const int64_t grid = (int64_t)p.pages * p.y + query_ctas;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (a.d == 64) return launch_pdl(k_extend_pages<T, 64, CH, VEC>, dim3((unsigned)grid), dim3(PagesShape<64>::kThreads), 0, s, p);
  if (a.d == 128) return launch_pdl(k_extend_pages<T, 128, CH, VEC>, dim3((unsigned)grid), dim3(PagesShape<128>::kThreads), 0, s, p);
  return launch_pdl(k_extend_pages<T, 256, CH, VEC>, dim3((unsigned)grid), dim3(PagesShape<256>::kThreads), 0, s, p);
}

template <typename T>
cudaError_t launch_pages(PagesArgs& p, bool vec, int sms, cudaStream_t s) {
  return vec ? launch_pages_d<T, 8, true>(p, sms, s) : launch_pages_d<T, 4, false>(p, sms, s);
}

template <typename T>
cudaError_t launch_rows(RowsArgs& a, bool vec, int sms, cudaStream_t s) {
  const int ctas = rows_ctas(a, vec ? 8 : 4, sms);
  return vec ? launch_pdl(k_rotate_rows<T, 8, true>, dim3(ctas), dim3(kRowsThreads), 0, s, a)
             : launch_pdl(k_rotate_rows<T, 4, false>, dim3(ctas), dim3(kRowsThreads), 0, s, a);
}

// 16-byte vectors of 8 pairs fit: addresses, strides and the channels' cut.
bool vectors(const void* p, int64_t row, int64_t head, int size) {
  return (uintptr_t)p % 16 == 0 && row * size % 16 == 0 && head * size % 16 == 0;
}
bool vectors(const Rotation& r, int d) { return r.pairs % 8 == 0 && d % 16 == 0; }

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
  const bool vec = vectors(r, d) && vectors(x, xs[0], xs[1], size) && vectors(out, os[0], os[1], size);
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
  bool vec = vectors(r, a.d);
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
    vec = vec && vectors(x[w], a.x_row[w], a.x_head[w], size);
    // pages of 8 bits have their alignment checked
    if (w == 0 || !scales) vec = vec && vectors(out[w], a.o_row[w], a.o_head[w], w == 0 ? size : 2) && a.o_block[w] % 8 == 0;
  }
  a.all = a.heads[0] + (scales ? 0 : a.heads[1] + a.heads[2]);
  if (!scales) {
    if (n.dtype == TQ_BF16) return launch_rows<__nv_bfloat16>(a, vec, sms, s);
    if (n.dtype == TQ_F16) return launch_rows<__half>(a, vec, sms, s);
    return launch_rows<float>(a, vec, sms, s);
  }
  p.scales = *scales;
  p.pages = n.n_rows / kPage + 2 * m.batch;
  const int items = 2 * pool.n_kv_heads, warps = a.d == 256 ? 16 : 8;
  // items per CTA: all warps busy in short runs, and enough CTAs for the SMs to take turns in long ones
  const int likely = std::max(1, n.n_rows / kPage + m.batch);
  const int most = n.n_rows / std::max(1, m.batch) > kShort ? items : (items + warps - 1) / warps;
  p.y = std::min(most, std::max(1, (16 * sms + likely - 1) / likely));
  if (n.dtype == TQ_BF16) return launch_pages<__nv_bfloat16>(p, vec, sms, s);
  if (n.dtype == TQ_F16) return launch_pages<__half>(p, vec, sms, s);
  return launch_pages<float>(p, vec, sms, s);
}

}  // namespace tq
