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
    pool.release(seq_ids_of_finished_requests)
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


class _On:
    """The device and raw stream of a call. Outputs made inside belong to that stream; the caller's tensors are
    recorded on it where it is not the current one."""

    __slots__ = ("raw", "_device", "_stream")

    def __init__(self, device, stream, *tensors):
        index = device.index
        self._device = torch.cuda.device(index) if torch.cuda.current_device() != index else None
        self._stream = None
        if stream is None:
            self.raw = torch._C._cuda_getCurrentRawStream(index)
        else:
            if stream.device != device:
                raise ValueError(f"stream of {stream.device}, tensors on {device}")
            self.raw = stream.cuda_stream
            if self.raw != torch._C._cuda_getCurrentRawStream(index):
                self._stream = torch.cuda.stream(stream)
                for t in tensors:
                    if t is not None:
                        t.record_stream(stream)

    def __enter__(self):
        if self._device is not None:
            self._device.__enter__()
        if self._stream is not None:
            self._stream.__enter__()
        return self

    def __exit__(self, *exc):
        if self._stream is not None:
            self._stream.__exit__(*exc)
        if self._device is not None:
            self._device.__exit__(*exc)


def _ints(name, t, device, n=None):
    """The address of a contiguous int32 vector on the device, with at least n entries."""
    if t.dtype is not torch.int32 or t.device != device or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 vector on {device}")
    if n is not None and t.shape[0] < n:
        raise ValueError(f"{name}: {t.shape[0]} entries, {n} are needed")
    return t.data_ptr()


def _optional(name, t, device, n=None):
    return None if t is None else _ints(name, t, device, n)


def _cuda(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    return t.device


def _table(table, free, n_free):
    device = _cuda("table", table)
    if table.dtype is not torch.int32 or table.dim() != 2 or not table.shape[0] or not table.shape[1] or table.stride(1) != 1:
        raise ValueError("table: expected int32 [max_seqs, max_pages] with contiguous rows")
    stride = table.stride(0) if table.shape[0] > 1 else max(table.stride(0), table.shape[1])
    return device, (table.data_ptr(), table.shape[0], table.shape[1], stride, _ints("free", free, device, 1), free.shape[0],
                    _ints("n_free", n_free, device, 1))


def map_blocks(table, free, n_free, seq_ids, lens, n_new, max_tokens, out=None, status=None, stream=None):
    """Blocks and slots of a step's new tokens (tq_blocks_map): (slots [max_tokens], starts [batch + 1],
    totals [batch]), int32. table, free and n_free are changed in place. out: the three tensors to write instead."""
    device, args = _table(table, free, n_free)
    batch = seq_ids.shape[0]
    ids = (_ints("seq_ids", seq_ids, device), _ints("lens", lens, device, batch), _ints("n_new", n_new, device, batch))
    word = _optional("status", status, device, 1)
    with _On(device, stream, table, free, n_free, seq_ids, lens, n_new, status, *(out or ())) as on:
        if out is None:
            # one allocation: [slots | starts | totals], each part 16-byte aligned
            a = (max(max_tokens, 0) + 3) & ~3
            b = a + ((batch + 4) & ~3)
            buf = torch.empty(b + batch, dtype=torch.int32, device=device)
            out = (buf[:max(max_tokens, 0)], buf[a:a + batch + 1], buf[b:])
        slots, starts, totals = out
        check(load().tq_blocks_map(*args, *ids, batch, _ints("starts", starts, device, batch + 1),
                                   _ints("totals", totals, device, batch), _ints("slots", slots, device, max_tokens), max_tokens,
                                   word, on.raw))
    return slots, starts, totals


def release_blocks(table, free, n_free, seq_ids, keep=None, status=None, stream=None):
    """Gives back the blocks behind each request's first keep[b] tokens, all of them without keep (tq_blocks_release)."""
    device, args = _table(table, free, n_free)
    batch = seq_ids.shape[0]
    ids = (_ints("seq_ids", seq_ids, device), _optional("keep", keep, device, batch))
    word = _optional("status", status, device, 1)
    with _On(device, stream, table, free, n_free, seq_ids, keep, status) as on:
        check(load().tq_blocks_release(*args, *ids, batch, word, on.raw))


def _kv(k, v, outer, tokens, heads, d, k_strides, v_strides):
    return _KV.pack(k.data_ptr(), v.data_ptr(), *k_strides, *v_strides, outer, tokens, heads, d, _DTYPES[k.dtype])


def _pools(k_pool, v_pool):
    device = _cuda("k_pool", k_pool)
    if (k_pool.dim() != 4 or k_pool.shape[1] != PAGE or k_pool.shape != v_pool.shape or k_pool.dtype is not v_pool.dtype
            or k_pool.dtype not in (torch.bfloat16, torch.float16) or v_pool.device != device):
        raise ValueError("k_pool, v_pool: expected two bf16 or f16 tensors [n_blocks, 128, n_kv_heads, head_dim] on one device")
    ks, vs = k_pool.stride(), v_pool.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("k_pool, v_pool: the channels of a head have to be contiguous")
    blocks, _, heads, d = k_pool.shape
    return device, _kv(k_pool, v_pool, blocks, PAGE, heads, d, ks[:3], vs[:3])


def append(k, v, k_pool, v_pool, slots, status=None, stream=None):
    """Writes k, v [tokens, n_kv_heads, head_dim] (bf16, f16 or f32, any strides with contiguous channels) into the pools
    [n_blocks, 128, n_kv_heads, head_dim] at `slots` (tq_paged_append; -1 skips a row)."""
    device, pool = _pools(k_pool, v_pool)
    if (k.dim() != 3 or k.shape != v.shape or k.dtype is not v.dtype or k.dtype not in _DTYPES or k.device != device
            or v.device != device or k.shape[1:] != k_pool.shape[2:]):
        raise ValueError("k, v: expected two tensors [tokens, n_kv_heads, head_dim] of one type that fit the pools")
    ks, vs = k.stride(), v.stride()
    if ks[2] != 1 or vs[2] != 1:
        raise ValueError("k, v: the channels of a head have to be contiguous")
    n = k.shape[0]
    with _On(device, stream, k, v, k_pool, v_pool, slots, status) as on:
        check(load().tq_paged_append(pool, k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype], _STRIDES.pack(ks[0], ks[1]),
                                     _STRIDES.pack(vs[0], vs[1]), _ints("slots", slots, device, n), n,
                                     _optional("status", status, device, 1), on.raw))


def _attend(q, dtype, heads, d, device, q_starts, max_q, max_kv, softmax_scale, out, workspace, on, kv, call):
    if q.dim() != 3 or q.dtype is not dtype or q.device != device or q.shape[2] != d or q.shape[1] % heads or not q.shape[1]:
        raise ValueError(f"q: expected a {dtype} tensor [rows, a multiple of {heads} heads, {d}] on {device}")
    if out is None:
        # rows behind the last request are not written
        out = torch.empty(q.shape, dtype=dtype, device=device)
    elif out.shape != q.shape or out.dtype is not dtype or out.device != device:
        raise ValueError("out: expected a tensor of q's shape, type and device")
    qs, os = q.stride(), out.stride()
    if qs[2] != 1 or os[2] != 1:
        raise ValueError("q, out: the channels of a head have to be contiguous")
    batch = q_starts.shape[0] - 1
    if batch < 0:
        raise ValueError("q_starts: expected [batch + 1] entries")
    queries = _QUERIES.pack(q.data_ptr(), out.data_ptr(), qs[0], qs[1], os[0], os[1], _ints("q_starts", q_starts, device), q.shape[0],
                            q.shape[1], batch, max_q, max_kv, softmax_scale)
    if workspace is None:
        n = load().tq_attention_workspace_bytes(queries, kv)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {device}")
    ws = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    call(queries, *ws, batch, on.raw)
    return out


def attention_workspace_bytes(q, k, max_q=0, max_kv=0, batch=1):
    """Bytes of workspace that attention or cross_attention needs for q [rows, heads, d] against k (a pool, or an encoder's
    states) in `batch` requests."""
    s = k.stride()
    dims = (1, k.shape[0]) if k.dim() == 3 else tuple(k.shape[:2])
    kv = _kv(k, k, *dims, k.shape[-2], k.shape[-1], (0, 0, 0) if k.dim() == 3 else s[:3], (0, 0, 0))
    queries = _QUERIES.pack(0, 0, 0, 0, 0, 0, 0, q.shape[0], q.shape[1], batch, max_q, max_kv, 0.0)
    with _On(_cuda("q", q), None):
        return load().tq_attention_workspace_bytes(queries, kv)


def attention(q, k_pool, v_pool, table, seq_ids, q_starts, kv_lens, causal=True, softmax_scale=0.0, max_q=0, max_kv=0, out=None,
              workspace=None, status=None, stream=None):
    """Attention of each request's new tokens over the paged cache that already holds them (tq_paged_attention).

    q: [rows, n_q_heads, head_dim] of the pools' type, request b's rows at [q_starts[b], q_starts[b + 1]); kv_lens[b]: its
    tokens with the new ones, in the pages of table row seq_ids[b] (None: row b). max_q: no request has more rows (0:
    unknown; few rows take a kernel of their own); max_kv: no request has more tokens (0: unknown; short calls launch fewer
    CTAs). Returns out, of q's shape; rows behind the last request stay as they are."""
    device, kv = _pools(k_pool, v_pool)
    if table.dtype is not torch.int32 or table.dim() != 2 or table.device != device or not table.shape[0] or not table.shape[1] or table.stride(1) != 1:
        raise ValueError(f"table: expected int32 [max_seqs, max_pages] with contiguous rows on {device}")
    max_seqs, max_pages = table.shape
    stride = table.stride(0) if max_seqs > 1 else max(table.stride(0), max_pages)
    word = _optional("status", status, device, 1)

    def call(queries, ws, ws_bytes, batch, raw):
        check(load().tq_paged_attention(queries, kv, table.data_ptr(), max_seqs, max_pages, stride, _optional("seq_ids", seq_ids, device, batch),
                                        _ints("kv_lens", kv_lens, device, batch), 1 if causal else 0, ws, ws_bytes, word, raw))

    with _On(device, stream, q, k_pool, v_pool, table, seq_ids, q_starts, kv_lens, out, workspace, status) as on:
        return _attend(q, k_pool.dtype, k_pool.shape[2], k_pool.shape[3], device, q_starts, max_q, max_kv, softmax_scale, out, workspace, on, kv,
                       call)


def cross_attention(q, k, v, q_starts, kv_lens=None, kv_starts=None, softmax_scale=0.0, max_q=0, max_kv=0, out=None, workspace=None,
                    status=None, stream=None):
    """Attention of q [rows, n_q_heads, head_dim] to an encoder's states (tq_cross_attention): packed k, v [states,
    n_kv_heads, head_dim] with kv_starts [batch + 1], or padded ones [batch, states, n_kv_heads, head_dim] with kv_lens
    [batch]. Every state of a request is visible to all its queries; a request without states gets zeros."""
    device = _cuda("k", k)
    if k.shape != v.shape or k.dtype is not v.dtype or k.dtype not in (torch.bfloat16, torch.float16) or v.device != device or k.dim() not in (3, 4):
        raise ValueError("k, v: expected two bf16 or f16 tensors [states, n_kv_heads, head_dim] or [batch, states, n_kv_heads, head_dim]")
    packed = k.dim() == 3
    if packed != (kv_starts is not None) or packed == (kv_lens is not None):
        raise ValueError("packed states take kv_starts, padded ones take kv_lens")
    ks, vs = k.stride(), v.stride()
    if ks[-1] != 1 or vs[-1] != 1:
        raise ValueError("k, v: the channels of a head have to be contiguous")
    heads, d = k.shape[-2:]
    if not heads:
        raise ValueError("k, v: no heads")
    if packed:
        kv = _kv(k, v, 1, k.shape[0], heads, d, (0, ks[0], ks[1]), (0, vs[0], vs[1]))
    else:
        kv = _kv(k, v, k.shape[0], k.shape[1], heads, d, ks[:3], vs[:3])
    word = _optional("status", status, device, 1)

    def call(queries, ws, ws_bytes, batch, raw):
        check(load().tq_cross_attention(queries, kv, _optional("kv_starts", kv_starts, device, batch + 1), _optional("kv_lens", kv_lens, device, batch),
                                        ws, ws_bytes, word, raw))

    with _On(device, stream, q, k, v, q_starts, kv_lens, kv_starts, out, workspace, status) as on:
        return _attend(q, k.dtype, heads, d, device, q_starts, max_q, max_kv, softmax_scale, out, workspace, on, kv, call)


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
        """Blocks and slots of a step's new tokens: (slots, starts, totals); see map_blocks."""
        return map_blocks(self.table, self.free, self.n_free, seq_ids, lens, n_new, max_tokens, out, self.status, stream)

    def release(self, seq_ids, keep=None, stream=None):
        """Ends requests, or cuts them back to their first keep[b] tokens; see release_blocks."""
        release_blocks(self.table, self.free, self.n_free, seq_ids, keep, self.status, stream)

    def check_status(self, clear=True):
        """The TQ_DEV_ERR_* bits that calls on this pool have set (waits for the device)."""
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
