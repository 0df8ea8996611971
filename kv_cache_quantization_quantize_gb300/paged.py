"""Exact paged cache: block maps, appends and attention of new tokens, and cross attention to an encoder's states.

Python binding of tq_blocks_map, tq_blocks_release, tq_paged_append, tq_paged_attention and tq_cross_attention
(include/tq.h has the operations). Argument checks and marshalling only: the work runs in libtq's kernels; there is
no fallback. No call reads a length, id or start on the host, so every one of them can be captured into a graph.

A page is 128 tokens, the packed cache's page: one block table serves a paged TurboQuantCache (its `block_pool`) and
the exact pools of the layers beside it.

One serving step:

    pool = BlockPool(n_blocks, max_seqs, max_ctx)            # or TurboQuantCache.block_pool
    cache = PagedCache(n_layers, pool, n_kv_heads, head_dim)
    slots, starts, totals = pool.map(seq_ids, lens, n_new, max_tokens)
    cache.append(layer, k, v, slots)                         # k, v: [tokens, n_kv_heads, head_dim]
    out = cache.attention(layer, q, seq_ids, starts, totals, max_q=..., max_kv=...)
    ...
    pool.release(seq_ids_of_finished_requests)               # keep=lengths: back to these, without packed layers
"""
import ctypes
import struct

import torch

from ._abi import (TQ_BF16, TQ_DEV_ERR_BLOCK, TQ_DEV_ERR_LENGTH, TQ_DEV_ERR_POOL, TQ_DEV_ERR_SEQ_ID,
                   TQ_DEV_ERR_SPLITS, TQ_DEV_ERR_TIMEOUT, TQ_F16, TQ_F32, check, load)

__all__ = ["PAGE", "BlockPool", "PagedCache", "map_blocks", "release_blocks", "append", "attention", "cross_attention",
           "attention_workspace_bytes", "TQ_DEV_ERR_BLOCK", "TQ_DEV_ERR_LENGTH", "TQ_DEV_ERR_POOL", "TQ_DEV_ERR_SEQ_ID",
           "TQ_DEV_ERR_SPLITS", "TQ_DEV_ERR_TIMEOUT"]

PAGE = 128
_DTYPES = {torch.bfloat16: TQ_BF16, torch.float16: TQ_F16, torch.float32: TQ_F32}
_KV = struct.Struct("@PP6q5i4x")     # tq_kv
_QUERIES = struct.Struct("@PP4qP5if")  # tq_queries
_STRIDES = struct.Struct("@2q")


_I32 = torch.int32
_HALVES = (torch.bfloat16, torch.float16)
_raw_memory = None  # see _raw_allocator


def _raw_allocator():
    """torch's stream-ordered allocation by raw address: (allocate(size, stream), free(address)). Looked up at the first call, so
    that the package can be imported with a torch that lacks the two private names; (None, None) there."""
    global _raw_memory
    if _raw_memory is None:
        names = ("_cuda_cudaCachingAllocator_raw_alloc", "_cuda_cudaCachingAllocator_raw_delete")
        _raw_memory = tuple(getattr(torch._C, n) for n in names) if all(hasattr(torch._C, n) for n in names) else (None, None)
    return _raw_memory


class _On:
    """The device and stream of a call that is not made on the current ones: outputs made inside belong to that stream, and
    the caller's tensors are recorded on it."""

    __slots__ = ("_device", "_stream")

    def __init__(self, index, stream, tensors):
        self._device = torch.cuda.device(index)
        self._stream = stream
        if stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
            self._stream = torch.cuda.stream(stream)

    def __enter__(self):
        self._device.__enter__()
        if self._stream is not None:
            self._stream.__enter__()

    def __exit__(self, *exc):
        if self._stream is not None:
            self._stream.__exit__(*exc)
        self._device.__exit__(*exc)


def _here(index, stream, tensors):
    """(raw stream, context or None) of a call on device `index`; no context where all is current."""
    current = torch._C._cuda_getDevice() == index
    raw = torch._C._cuda_getCurrentRawStream(index)
    if stream is None:
        return raw, None if current else _On(index, None, ())
    if stream.device.index != index:
        raise ValueError(f"stream of {stream.device}, tensors on cuda:{index}")
    if stream.cuda_stream == raw:
        return raw, None if current else _On(index, None, ())
    return stream.cuda_stream, _On(index, stream, tensors)


def _ints(name, t, index, n=0):
    """The address of a contiguous int32 vector on the device, with at least n entries."""
    if t.dtype is _I32 and t.get_device() == index and t.dim() == 1 and t.is_contiguous() and t.shape[0] >= n:
        return t.data_ptr()
    if t.dtype is not _I32 or t.get_device() != index or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 vector on cuda:{index}")
    raise ValueError(f"{name}: {t.shape[0]} entries, {n} are needed")


def _table(table, index):
    """(address, max_seqs, max_pages, row stride) of a block table."""
    if table.dtype is _I32 and table.dim() == 2 and table.get_device() == index >= 0:
        rows, pages = table.shape
        stride, one = table.stride()
        if rows and pages and one == 1:
            return table.data_ptr(), rows, pages, stride if rows > 1 or stride > pages else pages
    raise ValueError("table: expected int32 [max_seqs, max_pages] with contiguous rows on the others' CUDA device")


def _map_args(table, free, n_free):
    index = table.get_device()
    return index, (*_table(table, index), _ints("free", free, index, 1), free.shape[0], _ints("n_free", n_free, index, 1))


def map_blocks(table, free, n_free, seq_ids, lens, n_new, max_tokens, out=None, status=None, stream=None):
    """Blocks and slots of a step's new tokens (tq_blocks_map): (slots [max_tokens], starts [batch + 1],
    totals [batch]), int32. table, free and n_free are changed in place. out: the three tensors to write instead."""
    index, args = _map_args(table, free, n_free)
    batch = seq_ids.shape[0]
    ids = (_ints("seq_ids", seq_ids, index), _ints("lens", lens, index, batch), _ints("n_new", n_new, index, batch))
    word = None if status is None else _ints("status", status, index, 1)
    raw, on = _here(index, stream, (table, free, n_free, seq_ids, lens, n_new, status, *(out or ())))
    if on is not None:
        with on:
            return _map_blocks(args, ids, batch, max_tokens, out, word, raw, index, table.device)
    return _map_blocks(args, ids, batch, max_tokens, out, word, raw, index, table.device)


def _map_blocks(args, ids, batch, max_tokens, out, word, raw, index, device):
    if max_tokens > 1 << 30:
        raise ValueError(f"max_tokens {max_tokens}: at most 2^30")
    if out is None:  # three allocations: views of one take 5 us longer
        slots = torch.empty(max(max_tokens, 0), dtype=_I32, device=device)
        starts = torch.empty(batch + 1, dtype=_I32, device=device)
        totals = torch.empty(batch, dtype=_I32, device=device)
        out = (slots, starts, totals)
        places = (starts.data_ptr(), totals.data_ptr(), slots.data_ptr())
    else:
        slots, starts, totals = out
        places = (_ints("starts", starts, index, batch + 1), _ints("totals", totals, index, batch), _ints("slots", slots, index, max_tokens))
    check(load().tq_blocks_map(*args, *ids, batch, *places, max_tokens, word, raw))
    return out


def release_blocks(table, free, n_free, seq_ids, keep=None, status=None, stream=None):
    """Gives back the blocks behind each request's first keep[b] tokens, all of them without keep (tq_blocks_release). Only the
    table and the stack change: what else knows the requests' lengths, such as packed layers, is the caller's."""
    index, args = _map_args(table, free, n_free)
    batch = seq_ids.shape[0]
    ids = _ints("seq_ids", seq_ids, index)
    kept = None if keep is None else _ints("keep", keep, index, batch)
    word = None if status is None else _ints("status", status, index, 1)
    raw, on = _here(index, stream, (table, free, n_free, seq_ids, keep, status))
    if on is not None:
        with on:
            check(load().tq_blocks_release(*args, ids, kept, batch, word, raw))
    else:
        check(load().tq_blocks_release(*args, ids, kept, batch, word, raw))


def _kv(k, v, outer, tokens, heads, d, k_strides, v_strides):
    return _KV.pack(k.data_ptr(), v.data_ptr(), *k_strides, *v_strides, outer, tokens, heads, d, _DTYPES[k.dtype])


def _pools(k_pool, v_pool):
    """(device index, tq_kv, head_dim, heads, type) of a pool."""
    shape, dtype, index = k_pool.shape, k_pool.dtype, k_pool.get_device()
    if index < 0:
        raise ValueError("k_pool: expected a CUDA tensor")
    if (len(shape) != 4 or shape[1] != PAGE or not shape[2] or shape != v_pool.shape or dtype is not v_pool.dtype or dtype not in _HALVES
            or v_pool.get_device() != index):
        raise ValueError("k_pool, v_pool: expected two bf16 or f16 tensors [n_blocks, 128, n_kv_heads, head_dim] on one device")
    ks, vs = k_pool.stride(), v_pool.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("k_pool, v_pool: the channels of a head have to be contiguous")
    return index, _kv(k_pool, v_pool, shape[0], PAGE, shape[2], shape[3], ks[:3], vs[:3]), shape[3], shape[2], dtype


def append(k, v, k_pool, v_pool, slots, status=None, stream=None):
    """Writes k, v [tokens, n_kv_heads, head_dim] (bf16, f16 or f32, any strides with contiguous channels) into the pools
    [n_blocks, 128, n_kv_heads, head_dim] at `slots` (tq_paged_append; -1 skips a row)."""
    index, pool, d, heads, _ = _pools(k_pool, v_pool)
    shape, dtype = k.shape, k.dtype
    if (len(shape) != 3 or shape != v.shape or dtype is not v.dtype or dtype not in _DTYPES or k.get_device() != index
            or v.get_device() != index or shape[1] != heads or shape[2] != d):
        raise ValueError("k, v: expected two tensors [tokens, n_kv_heads, head_dim] of one type that fit the pools")
    ks, vs = k.stride(), v.stride()
    if ks[2] != 1 or vs[2] != 1:
        raise ValueError("k, v: the channels of a head have to be contiguous")
    n = shape[0]
    args = (pool, k.data_ptr(), v.data_ptr(), _DTYPES[dtype], _STRIDES.pack(ks[0], ks[1]), _STRIDES.pack(vs[0], vs[1]),
            _ints("slots", slots, index, n), n, None if status is None else _ints("status", status, index, 1))
    raw, on = _here(index, stream, (k, v, k_pool, v_pool, slots, status))
    if on is not None:
        with on:
            check(load().tq_paged_append(*args, raw))
    else:
        check(load().tq_paged_append(*args, raw))


def _attend(q, dtype, heads, d, index, q_starts, max_q, max_kv, softmax_scale, out, workspace, kv, stream, tensors, call):
    shape = q.shape
    if len(shape) != 3 or q.dtype is not dtype or q.get_device() != index or shape[2] != d or shape[1] % heads or not shape[1]:
        raise ValueError(f"q: expected a {dtype} tensor [rows, a multiple of {heads} heads, {d}] on cuda:{index}")
    batch = q_starts.shape[0] - 1
    if batch < 0:
        raise ValueError("q_starts: expected [batch + 1] entries")
    raw, on = _here(index, stream, (q, q_starts, out, workspace, *tensors))
    if on is not None:
        with on:
            return _attend_here(q, shape, dtype, index, batch, q_starts, max_q, max_kv, softmax_scale, out, workspace, kv, raw, call)
    return _attend_here(q, shape, dtype, index, batch, q_starts, max_q, max_kv, softmax_scale, out, workspace, kv, raw, call)


def _attend_here(q, shape, dtype, index, batch, q_starts, max_q, max_kv, softmax_scale, out, workspace, kv, raw, call):
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)  # rows behind the last request are not written
    elif out.shape != shape or out.dtype is not dtype or out.get_device() != index:
        raise ValueError("out: expected a tensor of q's shape, type and device")
    qs, os = q.stride(), out.stride()
    if qs[2] != 1 or os[2] != 1:
        raise ValueError("q, out: the channels of a head have to be contiguous")
    queries = _QUERIES.pack(q.data_ptr(), out.data_ptr(), qs[0], qs[1], os[0], os[1], _ints("q_starts", q_starts, index), shape[0], shape[1],
                            batch, max_q, max_kv, softmax_scale)
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on cuda:{index}")
        check(call(queries, kv, batch, workspace.data_ptr(), workspace.numel() * workspace.element_size(), raw))
        return out
    # Memory of the call's stream, given back to it behind the launches: what comes next on that stream may take it. Without
    # a tensor around it the call takes 11.7 us of the host instead of 17.6.
    size = load().tq_attention_workspace_bytes(queries, kv)
    alloc, free = _raw_memory or _raw_allocator()
    if alloc is None:
        ws = torch.empty(size, dtype=torch.uint8, device=q.device)  # the call's stream is current here
        check(call(queries, kv, batch, ws.data_ptr(), size, raw))
        return out
    ws = alloc(size, raw) if size else None
    try:
        check(call(queries, kv, batch, ws, size, raw))
    finally:
        if size:
            free(ws)
    return out


def attention_workspace_bytes(q, k, max_q=0, max_kv=0, batch=1):
    """Bytes of workspace that attention or cross_attention needs for q [rows, heads, d] against k (a pool, or an encoder's
    states) in `batch` requests."""
    s = k.stride()
    dims = (1, k.shape[0]) if k.dim() == 3 else tuple(k.shape[:2])
    kv = _kv(k, k, *dims, k.shape[-2], k.shape[-1], (0, 0, 0) if k.dim() == 3 else s[:3], (0, 0, 0))
    queries = _QUERIES.pack(0, 0, 0, 0, 0, 0, 0, q.shape[0], q.shape[1], batch, max_q, max_kv, 0.0)
    with torch.cuda.device(q.device):
        return load().tq_attention_workspace_bytes(queries, kv)


def attention(q, k_pool, v_pool, table, seq_ids, q_starts, kv_lens, causal=True, softmax_scale=0.0, max_q=0, max_kv=0, out=None,
              workspace=None, status=None, stream=None):
    """Attention of each request's new tokens over the paged cache that already holds them (tq_paged_attention).

    q: [rows, n_q_heads, head_dim] of the pools' type, request b's rows at [q_starts[b], q_starts[b + 1]); kv_lens[b]: its
    tokens with the new ones, in the pages of table row seq_ids[b] (None: row b). max_q: no request has more rows (0:
    unknown; few rows take a kernel of their own); max_kv: no request has more tokens (0: unknown; short calls launch fewer
    CTAs). Returns out, of q's shape; rows of no request stay as they are. What the cache holds behind a request's
    tokens does not matter; a token that any of its queries sees has to be finite."""
    index, kv, d, heads, dtype = _pools(k_pool, v_pool)
    pages = _table(table, index)
    word = None if status is None else _ints("status", status, index, 1)

    def call(queries, kv, batch, ws, size, raw):
        return load().tq_paged_attention(queries, kv, *pages, None if seq_ids is None else _ints("seq_ids", seq_ids, index, batch),
                                         _ints("kv_lens", kv_lens, index, batch), 1 if causal else 0, ws, size, word, raw)

    return _attend(q, dtype, heads, d, index, q_starts, max_q, max_kv, softmax_scale, out, workspace, kv, stream,
                   (k_pool, v_pool, table, seq_ids, kv_lens, status), call)


def cross_attention(q, k, v, q_starts, kv_lens=None, kv_starts=None, softmax_scale=0.0, max_q=0, max_kv=0, out=None, workspace=None,
                    status=None, stream=None):
    """Attention of q [rows, n_q_heads, head_dim] to an encoder's states (tq_cross_attention): packed k, v [states,
    n_kv_heads, head_dim] with kv_starts [batch + 1], or padded ones [batch, states, n_kv_heads, head_dim] with kv_lens
    [batch]. Every state of a request is visible to all its queries; a request without states gets zeros."""
    shape, dtype, index = k.shape, k.dtype, k.get_device()
    if index < 0:
        raise ValueError("k: expected a CUDA tensor")
    if shape != v.shape or dtype is not v.dtype or dtype not in _HALVES or v.get_device() != index or len(shape) not in (3, 4):
        raise ValueError("k, v: expected two bf16 or f16 tensors [states, n_kv_heads, head_dim] or [batch, states, n_kv_heads, head_dim]")
    packed = len(shape) == 3
    if packed != (kv_starts is not None) or packed == (kv_lens is not None):
        raise ValueError("packed states take kv_starts, padded ones take kv_lens")
    ks, vs = k.stride(), v.stride()
    if ks[-1] != 1 or vs[-1] != 1:
        raise ValueError("k, v: the channels of a head have to be contiguous")
    heads, d = shape[-2:]
    if not heads:
        raise ValueError("k, v: no heads")
    if packed:
        kv = _kv(k, v, 1, shape[0], heads, d, (0, ks[0], ks[1]), (0, vs[0], vs[1]))
    else:
        kv = _kv(k, v, shape[0], shape[1], heads, d, ks[:3], vs[:3])
    word = None if status is None else _ints("status", status, index, 1)

    def call(queries, kv, batch, ws, size, raw):
        return load().tq_cross_attention(queries, kv, _ints("kv_starts", kv_starts, index, batch + 1) if packed else None,
                                         None if packed else _ints("kv_lens", kv_lens, index, batch), ws, size, word, raw)

    return _attend(q, dtype, heads, d, index, q_starts, max_q, max_kv, softmax_scale, out, workspace, kv, stream,
                   (k, v, kv_lens, kv_starts, status), call)


class BlockPool:
    """The blocks of a paged cache: table [max_seqs, max_pages], the stack of free blocks, and a status word that the calls on
    it report to. `table`: another cache's block table (TurboQuantCache.block_table), whose entries are all -1 so far."""

    def __init__(self, n_blocks, max_seqs, max_ctx, device="cuda", table=None):
        if n_blocks < 1 or max_seqs < 1 or max_ctx < 1:
            raise ValueError("n_blocks, max_seqs and max_ctx have to be at least 1")
        if table is None:
            table = torch.full((max_seqs, (max_ctx + PAGE - 1) // PAGE), -1, dtype=torch.int32, device=device)
        self.table, self.device, self.n_blocks = table, table.device, n_blocks
        self.free = torch.arange(n_blocks - 1, -1, -1, dtype=torch.int32, device=self.device)  # block 0 on top
        self.n_free = torch.full((1,), n_blocks, dtype=torch.int32, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def map(self, seq_ids, lens, n_new, max_tokens, out=None, stream=None):
        """Blocks and slots of a step's new tokens: (slots, starts, totals); see map_blocks. The total of a request that is not
        served is 0."""
        return map_blocks(self.table, self.free, self.n_free, seq_ids, lens, n_new, max_tokens, out, self.status, stream)

    def release(self, seq_ids, keep=None, stream=None):
        """Ends requests, or cuts them back to their first keep[b] tokens; see release_blocks."""
        release_blocks(self.table, self.free, self.n_free, seq_ids, keep, self.status, stream)

    def check_status(self, clear=True):
        """The TQ_DEV_ERR_* bits that calls on this pool have set (waits for the current stream)."""
        word = int(self.status.item())
        if clear and word:
            self.status.zero_()
        return word


class PagedCache:
    """Exact K and V of n_layers layers in 16 bits, in the blocks of a BlockPool (which other caches may share)."""

    def __init__(self, n_layers, pool, n_kv_heads, head_dim, dtype=torch.bfloat16):
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("dtype: bf16 or f16")
        self.pool = pool
        self.kv = torch.empty((n_layers, 2, pool.n_blocks, PAGE, n_kv_heads, head_dim), dtype=dtype, device=pool.device)

    def append(self, layer, k, v, slots, stream=None):
        """Writes the step's k, v [tokens, n_kv_heads, head_dim] of one layer at the slots of pool.map."""
        append(k, v, self.kv[layer, 0], self.kv[layer, 1], slots, self.pool.status, stream)

    def attention(self, layer, q, seq_ids, q_starts, kv_lens, causal=True, softmax_scale=0.0, max_q=0, max_kv=0, out=None,
                  workspace=None, stream=None):
        """Attention of the step's q [tokens, n_q_heads, head_dim] over one layer; q_starts and kv_lens are the starts and totals
        of pool.map. See attention()."""
        return attention(q, self.kv[layer, 0], self.kv[layer, 1], self.pool.table, seq_ids, q_starts, kv_lens, causal, softmax_scale, max_q,
                         max_kv, out, workspace, self.pool.status, stream)
