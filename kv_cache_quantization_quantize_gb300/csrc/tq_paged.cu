// Block maps and appends of the exact paged cache: tq_blocks_release, tq_blocks_map, tq_paged_append.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "tq_device.cuh"

namespace tq {
namespace {

namespace cg = cooperative_groups;

// =============================================================================================
// Block maps. One cluster of kMapCtas CTAs runs a whole call: the requests' needs are counted by one warp each
// over the cluster, exchanged through distributed shared memory, prefix-summed by every CTA alike, and the table
// entries and slots are written by all CTAs. Cluster barriers stand between the steps, so that one launch does
// what a chain of scans and scatters would, and nothing but the caller's arrays is touched in device memory.
// The work is a few KB to a few hundred KB: latency bounds it (launch, three dependent rounds of loads, three
// barriers), not bandwidth. The ids and lengths are read into shared memory in one round and never again. Measured: a
// release and a map of 256 requests 13.9 us (16.3 with each step's own loads), of 16 prompts of 4096 to 8192 tokens
// (94000 slots) 17.5 us (20.1).
// =============================================================================================
constexpr int kMaxBatch = 4096;
constexpr int kMapCtas = 8;
constexpr int kMapThreads = 512;
constexpr int kMapWarps = kMapThreads / 32;

// Slot of `id` in the table of first owners (open addressing, `mask` + 1 entries of {id, lowest request}).
__device__ __forceinline__ uint32_t hash_id(uint32_t id) { return id * 2654435761u; }

// Marks every request's id (in shared memory) with the lowest request that has it. keys start at -1, owner at INT_MAX.
__device__ void clear_owners(int32_t* keys, int32_t* owner, int mask) {
  for (int i = threadIdx.x; i <= mask; i += kMapThreads) {
    keys[i] = -1;
    owner[i] = 0x7fffffff;
  }
}
__device__ void own_ids(const int32_t* ids, int batch, int max_seqs, int32_t* keys, int32_t* owner, int mask) {
  __syncthreads();
  for (int b = threadIdx.x; b < batch; b += kMapThreads) {
    const int id = ids[b];
    if (id < 0 || id >= max_seqs) continue;
    uint32_t h = hash_id((uint32_t)id) & mask;
    for (;;) {  // ends: the table has at least twice as many entries as ids
      const int old = atomicCAS(&keys[h], -1, id);
      if (old == -1 || old == id) break;
      h = (h + 1) & mask;
    }
    atomicMin(&owner[h], b);
  }
  __syncthreads();
}

__device__ __forceinline__ bool owns_id(int b, int id, int max_seqs, const int32_t* keys, const int32_t* owner,
                                        int mask) {
  if (id < 0 || id >= max_seqs) return false;
  uint32_t h = hash_id((uint32_t)id) & mask;
  while (keys[h] != id) h = (h + 1) & mask;
  return owner[h] == b;
}

// Exclusive prefix sums, in place, of n values in shared memory by the whole CTA; returns the total. Values are
// clamped so that no sum passes `limit` (<= 2^30; the inputs are in [0, limit]).
__device__ int scan_exclusive(int32_t* x, int n, int limit, int32_t* warp_sums) {
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int per = (n + kMapThreads - 1) / kMapThreads;
  const int lo = min(n, t * per), hi = min(n, lo + per);
  int sum = 0;
  for (int i = lo; i < hi; ++i) sum = min(limit, sum + x[i]);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc = min(limit, inc + v);
  }
  __syncthreads();  // warp_sums may still be read from an earlier scan
  if (lane == 31) warp_sums[w] = inc;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kMapWarps; ++i) {
    if (i == w) before = total;
    total = min(limit, total + warp_sums[i]);
  }
  const int prev = __shfl_up_sync(0xffffffffu, inc, 1);
  int run = min(limit, before + (lane ? prev : 0));
  for (int i = lo; i < hi; ++i) {
    const int v = x[i];
    x[i] = run;
    run = min(limit, run + v);
  }
  __syncthreads();
  return total;
}

struct MapArgs {
  int32_t* table;
  int64_t stride;
  int32_t* free;
  int32_t* n_free;
  const int32_t* ids;
  const int32_t* lens;   // map: lengths; release: tokens to keep (NULL: 0)
  const int32_t* n_new;
  int32_t* starts;
  int32_t* totals;
  int32_t* slots;
  uint32_t* status;
  int max_seqs, max_pages, n_blocks, batch, max_tokens, mask;
};

__device__ __forceinline__ void report(uint32_t* status, uint32_t bits) {
  if (status && bits) atomicOr(status, bits);
}

__device__ __forceinline__ int pages_of(int tokens) { return (int)(((int64_t)tokens + kPage - 1) / kPage); }

__device__ __forceinline__ int clamped_free(const MapArgs& a, uint32_t& err) {
  const int n = *a.n_free;
  if (n < 0 || n > a.n_blocks) err |= TQ_DEV_ERR_POOL;
  return max(0, min(n, a.n_blocks));
}

__global__ void __cluster_dims__(kMapCtas, 1, 1) __launch_bounds__(kMapThreads) k_blocks_release(MapArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ int32_t warp_sums[kMapWarps];
  cg::cluster_group cl = cg::this_cluster();
  int32_t* count = sm;
  int32_t* ids = count + a.batch;   // the arrays are read once, in one round of loads
  int32_t* keeps = ids + a.batch;
  int32_t* keys = keeps + a.batch;
  int32_t* owner = keys + a.mask + 1;
  const int rank = (int)cl.block_rank(), lane = threadIdx.x & 31, gw = rank * kMapWarps + (threadIdx.x >> 5);
  uint32_t err = 0;
  cl.barrier_arrive();
  clear_owners(keys, owner, a.mask);
  pdl_wait();
  const int n_free = clamped_free(a, err);
  for (int b = threadIdx.x; b < a.batch; b += kMapThreads) {
    const int id = a.ids[b], keep = a.lens ? a.lens[b] : 0;
    ids[b] = id;
    keeps[b] = keep;
  }
  own_ids(ids, a.batch, a.max_seqs, keys, owner, a.mask);
  cl.barrier_wait();  // every CTA of the cluster has started: its shared memory can be written
  auto first_page = [&](int b, int& id) {  // the first page to give back; -1: skipped
    id = ids[b];
    const int keep = keeps[b];
    if (keep < 0) {
      err |= TQ_DEV_ERR_LENGTH;
      return -1;
    }
    if (!owns_id(b, id, a.max_seqs, keys, owner, a.mask)) {
      err |= TQ_DEV_ERR_SEQ_ID;
      return -1;
    }
    return pages_of(keep);
  };
  for (int b = gw; b < a.batch; b += kMapCtas * kMapWarps) {
    int id, n = 0;
    const int p0 = first_page(b, id);
    if (p0 >= 0) {
      const int32_t* row = a.table + (int64_t)id * a.stride;
#pragma unroll 4
      for (int p = p0 + lane; p < a.max_pages; p += 32) n += row[p] >= 0 && row[p] < a.n_blocks;
      n = __reduce_add_sync(0xffffffffu, n);
    }
    if (lane < kMapCtas) *cl.map_shared_rank(count + b, lane) = n;
  }
  cl.sync();
  const int total = scan_exclusive(count, a.batch, 1 << 30, warp_sums);
  const bool fits = total <= a.n_blocks - n_free;
  if (!fits) err |= TQ_DEV_ERR_POOL;
  if (fits) {
    for (int b = gw; b < a.batch; b += kMapCtas * kMapWarps) {
      int id, at = count[b];
      const int p0 = first_page(b, id);
      if (p0 < 0) continue;
      int32_t* row = a.table + (int64_t)id * a.stride;
      for (int base = p0; base < a.max_pages; base += 32) {
        const int p = base + lane;
        const int e = p < a.max_pages ? row[p] : -1;
        const bool mine = e >= 0 && e < a.n_blocks;
        const uint32_t m = __ballot_sync(0xffffffffu, mine);
        if (mine) a.free[n_free + total - 1 - (at + __popc(m & ((1u << lane) - 1)))] = e;
        if (e != -1) {
          row[p] = -1;
          if (!mine) err |= TQ_DEV_ERR_BLOCK;
        }
        at += __popc(m);
      }
    }
  }
  report(a.status, err);
  __threadfence();  // the table is read by kernels that start early (programmatic dependent launch)
  cl.sync();  // every CTA has read *n_free (and done with the others' shared memory)
  if (fits && rank == 0 && threadIdx.x == 0) *a.n_free = n_free + total;
}

__global__ void __cluster_dims__(kMapCtas, 1, 1) __launch_bounds__(kMapThreads) k_blocks_map(MapArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ int32_t warp_sums[kMapWarps];
  cg::cluster_group cl = cg::this_cluster();
  int32_t* need = sm;                  // blocks to take; -1: not served. Then their prefix sums
  int32_t* start = need + a.batch;     // new tokens, then their prefix sums
  int32_t* bad = start + a.batch;      // 1: not served for its arguments
  int32_t* ids = bad + a.batch;        // the arrays are read once, in one round of loads
  int32_t* lens = ids + a.batch;
  int32_t* news = lens + a.batch;
  int32_t* keys = news + a.batch;
  int32_t* owner = keys + a.mask + 1;
  const int rank = (int)cl.block_rank(), lane = threadIdx.x & 31, gw = rank * kMapWarps + (threadIdx.x >> 5);
  uint32_t err = 0;
  cl.barrier_arrive();
  clear_owners(keys, owner, a.mask);
  pdl_wait();
  const int n_free = clamped_free(a, err);
  for (int b = threadIdx.x; b < a.batch; b += kMapThreads) {
    const int id = a.ids[b], len = a.lens[b], n_new = a.n_new[b];
    ids[b] = id;
    lens[b] = len;
    news[b] = n_new;
    start[b] = max(0, min(n_new, a.max_tokens));
  }
  own_ids(ids, a.batch, a.max_seqs, keys, owner, a.mask);
  // the packed places, the same in every CTA
  const int n_tokens = scan_exclusive(start, a.batch, a.max_tokens, warp_sums);
  cl.barrier_wait();  // every CTA of the cluster has started: its shared memory can be written
  for (int b = gw; b < a.batch; b += kMapCtas * kMapWarps) {
    const int id = ids[b], len = lens[b], n_new = news[b];
    int n = 0, out = 1;
    if (!owns_id(b, id, a.max_seqs, keys, owner, a.mask)) {
      err |= TQ_DEV_ERR_SEQ_ID;
    } else if (len < 0 || n_new < 0 || (int64_t)start[b] + n_new > a.max_tokens ||
               (int64_t)len + n_new > (int64_t)a.max_pages * kPage) {
      err |= TQ_DEV_ERR_LENGTH;
    } else {
      out = 0;
      const int32_t* row = a.table + (int64_t)id * a.stride;
      const int p1 = pages_of(len + n_new);
      for (int p = pages_of(len) + lane; p < p1; p += 32) n += row[p] < 0;
      n = __reduce_add_sync(0xffffffffu, n);
    }
    if (lane < kMapCtas) {
      *cl.map_shared_rank(need + b, lane) = n;
      *cl.map_shared_rank(bad + b, lane) = out;
    }
  }
  cl.sync();
  // Served: no need, or the needs up to and with it fit. The prefix sums hold the needs of refused requests too,
  // so the first one that does not fit is followed only by requests that need nothing.
  for (int b = threadIdx.x; b < a.batch; b += kMapThreads) bad[b] |= need[b] << 1;
  __syncthreads();
  scan_exclusive(need, a.batch, 1 << 30, warp_sums);
  for (int b = threadIdx.x; b < a.batch; b += kMapThreads) {
    const int n = bad[b] >> 1;
    int out = bad[b] & 1;
    if (n > 0 && need[b] + n > n_free) {
      out = 1;
      err |= TQ_DEV_ERR_POOL;
    }
    bad[b] = out | n << 1;
    if (rank == 0) {
      a.starts[b] = start[b];
      a.totals[b] = out ? 0 : lens[b] + news[b];
    }
  }
  if (rank == 0 && threadIdx.x == 0) a.starts[a.batch] = n_tokens;
  __syncthreads();
  int taken = 0;  // blocks that leave the stack: up to the end of the last served need
  for (int b = gw; b < a.batch; b += kMapCtas * kMapWarps) {
    const int n = bad[b] >> 1;
    if ((bad[b] & 1) || n == 0) continue;
    int32_t* row = a.table + (int64_t)ids[b] * a.stride;
    const int len = lens[b], p1 = pages_of(len + news[b]);
    int at = n_free - 1 - need[b];
    for (int base = pages_of(len); base < p1; base += 32) {
      const int p = base + lane;
      const bool mine = p < p1 && row[p] < 0;
      const uint32_t m = __ballot_sync(0xffffffffu, mine);
      if (mine) row[p] = a.free[at - __popc(m & ((1u << lane) - 1))];
      at -= __popc(m);
    }
  }
  if (rank == 0)
    for (int b = threadIdx.x; b < a.batch; b += kMapThreads)
      if (!(bad[b] & 1)) taken = max(taken, (bad[b] >> 1) ? need[b] + (bad[b] >> 1) : 0);
  __shared__ int32_t most;
  if (threadIdx.x == 0) most = 0;
  __syncthreads();
  if (rank == 0 && taken > 0) atomicMax(&most, taken);
  __threadfence();  // the table is read by kernels that start early (programmatic dependent launch)
  cl.sync();  // the new table entries are seen by the whole cluster, and every CTA has read *n_free
  if (rank == 0 && threadIdx.x == 0) *a.n_free = n_free - most;
  // slots: four packed tokens per thread; the request by bisection over the starts in shared memory
  for (int i0 = (rank * kMapThreads + threadIdx.x) * 4; i0 < a.max_tokens; i0 += kMapCtas * kMapThreads * 4) {
    int32_t s[4] = {-1, -1, -1, -1};
    if (i0 < n_tokens) {
      int lo = 0, hi = a.batch - 1;  // the last request whose start is <= i0
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= i0) lo = mid; else hi = mid - 1;
      }
      int b = lo, page = -1, block = -1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j;
        if (i >= n_tokens) break;
        while (b + 1 < a.batch && start[b + 1] <= i) {
          ++b;
          page = -1;
        }
        if (bad[b] & 1) continue;
        const int pos = lens[b] + i - start[b];
        if (pos / kPage != page) {
          page = pos / kPage;
          block = a.table[(int64_t)ids[b] * a.stride + page];
          if (block < 0 || block >= a.n_blocks) {
            err |= TQ_DEV_ERR_BLOCK;
            block = -1;
          }
        }
        if (block >= 0) s[j] = block * kPage + pos % kPage;
      }
    }
    if (i0 + 4 <= a.max_tokens && (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0) {
      *reinterpret_cast<int4*>(a.slots + i0) = make_int4(s[0], s[1], s[2], s[3]);
    } else {
      for (int j = 0; j < 4 && i0 + j < a.max_tokens; ++j) a.slots[i0 + j] = s[j];
    }
  }
  report(a.status, err);
}

int owner_entries(int batch) {
  int n = 64;
  while (n < 2 * batch) n *= 2;
  return n;
}

// The most shared memory that a call can need, allowed once per device (`known`: one bit each).
template <typename K>
cudaError_t launch_map(K kernel, MapArgs& a, int arrays, std::atomic<uint64_t>& known, cudaStream_t s) {
  const int entries = owner_entries(a.batch);
  a.mask = entries - 1;
  const size_t smem = sizeof(int32_t) * ((size_t)arrays * a.batch + 2 * entries);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (e == cudaSuccess && !(known.load(std::memory_order_relaxed) & bit)) {
    const int most = (int)sizeof(int32_t) * (arrays * kMaxBatch + 2 * owner_entries(kMaxBatch));
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) known.fetch_or(bit, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(kMapCtas), dim3(kMapThreads), smem, s, a);
}

// =============================================================================================
// Append: pool[slot / 128][slot % 128][h] = round(x[t][h]) for K and V. A copy with a scatter: DRAM bounds it. Measured:
// 65536 tokens x 8 heads x 128, bf16: 80 us, 6.7 TB/s (what a plain copy reaches); 128 tokens 1.6 us.
// =============================================================================================
struct PagedAppendArgs {
  const void* x[2];
  void* pool[2];
  int64_t x_row[2], x_head[2];             // elements
  int64_t p_block[2], p_token[2], p_head[2];
  const int32_t* slots;
  uint32_t* status;
  int n_tokens, heads, d, n_slots;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return static_cast<float>(v);
}
template <typename To, typename From>
__device__ __forceinline__ To round_to(From v) {
  if constexpr (std::is_same<To, From>::value) return v;
  else return To(to_f32(v));  // the constructors from float round to nearest even
}

// Eight consecutive elements of one head per thread and tensor. VEC: every row is 16-byte aligned on both sides.
template <typename From, typename To, bool VEC>
__global__ void __launch_bounds__(256) k_paged_append(PagedAppendArgs a) {
  pdl_wait();
  const uint32_t per = (uint32_t)a.heads * (a.d / 8);  // items of one token and tensor
  const uint64_t items = (uint64_t)per * a.n_tokens;
  const uint64_t step = (uint64_t)gridDim.x * 256;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += step) {
    const uint32_t t = (uint32_t)(i / per), r = (uint32_t)(i - (uint64_t)t * per);
    const uint32_t h = r / (a.d / 8), c = (r - h * (a.d / 8)) * 8;
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) {
      if (slot != -1 && r == 0) report(a.status, TQ_DEV_ERR_BLOCK);
      continue;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const From* src = static_cast<const From*>(a.x[w]) + (int64_t)t * a.x_row[w] + (int64_t)h * a.x_head[w] + c;
      To* dst = static_cast<To*>(a.pool[w]) + (int64_t)(slot / kPage) * a.p_block[w] +
                (int64_t)(slot % kPage) * a.p_token[w] + (int64_t)h * a.p_head[w] + c;
      alignas(16) From in[8];
      alignas(16) To out[8];
      if constexpr (VEC) {
        *reinterpret_cast<uint4*>(in) = __ldg(reinterpret_cast<const uint4*>(src));
        if constexpr (sizeof(From) == 4)
          *reinterpret_cast<uint4*>(in + 4) = __ldg(reinterpret_cast<const uint4*>(src + 4));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) in[j] = src[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] = round_to<To>(in[j]);
      if constexpr (VEC) {
        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(out);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[j] = out[j];
      }
    }
  }
}

template <typename From, typename To>
cudaError_t launch_append_as(const PagedAppendArgs& a, bool vec, int sms, cudaStream_t s) {
  const uint64_t items = (uint64_t)a.heads * (a.d / 8) * a.n_tokens;
  const int grid = (int)std::min<uint64_t>((items + 255) / 256, (uint64_t)sms * 32);
  return vec ? launch_pdl(k_paged_append<From, To, true>, dim3(grid), dim3(256), 0, s, a)
             : launch_pdl(k_paged_append<From, To, false>, dim3(grid), dim3(256), 0, s, a);
}

}  // namespace

cudaError_t launch_blocks_release(const BlockMap& m, cudaStream_t s) {
  MapArgs a = {};
  a.table = m.table;
  a.stride = m.stride;
  a.free = m.free;
  a.n_free = m.n_free;
  a.ids = m.ids;
  a.lens = m.lens;
  a.status = m.status;
  a.max_seqs = m.max_seqs;
  a.max_pages = m.max_pages;
  a.n_blocks = m.n_blocks;
  a.batch = m.batch;
  static std::atomic<uint64_t> known{0};
  return launch_map(k_blocks_release, a, 3, known, s);
}

cudaError_t launch_blocks_map(const BlockMap& m, cudaStream_t s) {
  MapArgs a = {};
  a.table = m.table;
  a.stride = m.stride;
  a.free = m.free;
  a.n_free = m.n_free;
  a.ids = m.ids;
  a.lens = m.lens;
  a.n_new = m.n_new;
  a.starts = m.starts;
  a.totals = m.totals;
  a.slots = m.slots;
  a.status = m.status;
  a.max_seqs = m.max_seqs;
  a.max_pages = m.max_pages;
  a.n_blocks = m.n_blocks;
  a.batch = m.batch;
  a.max_tokens = m.max_tokens;
  static std::atomic<uint64_t> known{0};
  return launch_map(k_blocks_map, a, 6, known, s);
}

cudaError_t launch_paged_append(const tq_kv& p, const void* k, const void* v, int dt, const int64_t* ks,
                                const int64_t* vs, const int32_t* slots, int n_tokens, uint32_t* status, int sms,
                                cudaStream_t s) {
  PagedAppendArgs a;
  const void* x[2] = {k, v};
  void* pool[2] = {p.k, p.v};
  const int64_t* xs[2] = {ks, vs};
  const int64_t* ps[2] = {p.k_strides, p.v_strides};
  const int esz = dt == TQ_F32 ? 4 : 2;
  bool vec = true;
  for (int w = 0; w < 2; ++w) {
    a.x[w] = x[w];
    a.pool[w] = pool[w];
    a.x_row[w] = xs[w][0];
    a.x_head[w] = xs[w][1];
    a.p_block[w] = ps[w][0];
    a.p_token[w] = ps[w][1];
    a.p_head[w] = ps[w][2];
    vec = vec && (uintptr_t)x[w] % 16 == 0 && (uintptr_t)pool[w] % 16 == 0 && xs[w][0] * esz % 16 == 0 &&
          xs[w][1] * esz % 16 == 0 && ps[w][0] % 8 == 0 && ps[w][1] % 8 == 0 && ps[w][2] % 8 == 0;
  }
  a.slots = slots;
  a.status = status;
  a.n_tokens = n_tokens;
  a.heads = p.n_kv_heads;
  a.d = p.head_dim;
  a.n_slots = p.outer * kPage;
  if (p.dtype == TQ_BF16) {
    if (dt == TQ_BF16) return launch_append_as<__nv_bfloat16, __nv_bfloat16>(a, vec, sms, s);
    if (dt == TQ_F16) return launch_append_as<__half, __nv_bfloat16>(a, vec, sms, s);
    return launch_append_as<float, __nv_bfloat16>(a, vec, sms, s);
  }
  if (dt == TQ_BF16) return launch_append_as<__nv_bfloat16, __half>(a, vec, sms, s);
  if (dt == TQ_F16) return launch_append_as<__half, __half>(a, vec, sms, s);
  return launch_append_as<float, __half>(a, vec, sms, s);
}

}  // namespace tq
