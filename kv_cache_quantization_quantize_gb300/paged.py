"""Paged caches of 16 and 8 bits: block maps, appends, rotary positions and attention of new tokens, and cross attention to an
encoder's states.

Python binding of tq_blocks_map, tq_blocks_release, tq_paged_append, tq_rotate, tq_paged_extend, tq_paged_attention,
tq_paged_attention8 and tq_cross_attention (include/tq.h has the operations). Argument checks and marshalling only: the work runs in libtq's kernels; there is
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

With rotary positions, and in a cache of 8 bits (dtype=torch.float8_e4m3fn) in any case, extend takes append's place:

    rotary = Rotary(head_dim, base=500000.0)
    q = cache.extend(layer, k, v, seq_ids, starts, totals, rotary=rotary, q=q)   # K rotated on the way, q in the same launch
"""
import ctypes
import math
import struct

import torch

from ._abi import (TQ_BF16, TQ_E4M3, TQ_DEV_ERR_BLOCK, TQ_DEV_ERR_LENGTH, TQ_DEV_ERR_POOL, TQ_DEV_ERR_SEQ_ID,
                   TQ_DEV_ERR_SPLITS, TQ_DEV_ERR_TIMEOUT, TQ_F16, TQ_F32, check, load)

__all__ = ["PAGE", "BlockPool", "PagedCache", "Rotary", "map_blocks", "release_blocks", "append", "rotate", "extend", "attention",
           "cross_attention", "attention_workspace_bytes", "TQ_DEV_ERR_BLOCK", "TQ_DEV_ERR_LENGTH", "TQ_DEV_ERR_POOL", "TQ_DEV_ERR_SEQ_ID",
           "TQ_DEV_ERR_SPLITS", "TQ_DEV_ERR_TIMEOUT"]

PAGE = 128
_DTYPES = {torch.bfloat16: TQ_BF16, torch.float16: TQ_F16, torch.float32: TQ_F32}
_KV = struct.Struct("@PP6q5i4x")     # tq_kv
_QUERIES = struct.Struct("@PP4qP5if")  # tq_queries
_STRIDES = struct.Struct("@2q")
_ROTARY = struct.Struct("@P2if4x")     # tq_rotary
_SCALES = struct.Struct("@PP2q")       # tq_scales
_NEW_ROWS = struct.Struct("@4P8qP3i4x")  # tq_new_rows


_I32 = torch.int32
_F32 = torch.float32
_HALVES = (torch.bfloat16, torch.float16)
_E4M3 = torch.float8_e4m3fn
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
    return _KV.pack(k.data_ptr(), v.data_ptr(), *k_strides, *v_strides, outer, tokens, heads, d, TQ_E4M3 if k.dtype is _E4M3 else _DTYPES[k.dtype])


def _pools(k_pool, v_pool, scaled=False):
    """(device index, tq_kv, head_dim, heads, type) of a pool, of one of e4m3 if `scaled`."""
    shape, dtype, index = k_pool.shape, k_pool.dtype, k_pool.get_device()
    if index < 0:
        raise ValueError("k_pool: expected a CUDA tensor")
    if (len(shape) != 4 or shape[1] != PAGE or not shape[2] or shape != v_pool.shape or dtype is not v_pool.dtype or v_pool.get_device() != index
            or (dtype is not _E4M3 if scaled else dtype not in _HALVES)):
        raise ValueError(f"k_pool, v_pool: expected two {'e4m3' if scaled else 'bf16 or f16'} tensors [n_blocks, 128, n_kv_heads, head_dim] on one "
                         f"device (e4m3 ones go with k_scale and v_scale)")
    ks, vs = k_pool.stride(), v_pool.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("k_pool, v_pool: the channels of a head have to be contiguous")
    return index, _kv(k_pool, v_pool, shape[0], PAGE, shape[2], shape[3], ks[:3], vs[:3]), shape[3], shape[2], dtype


def _scales(k_scale, v_scale, index, blocks, heads):
    """tq_scales, or None where both are None."""
    if k_scale is None and v_scale is None:
        return None
    if k_scale is not None and v_scale is not None and k_scale.dtype is _F32 and v_scale.dtype is _F32 and k_scale.get_device() == index:
        ks, vs = k_scale.stride(), v_scale.stride()
        if (v_scale.get_device() == index and k_scale.shape == (blocks, heads) and v_scale.shape == (blocks, heads)
                and (heads == 1 or ks[1] == 1 and vs[1] == 1) and (blocks == 1 or ks[0] >= heads and vs[0] >= heads)):
            return _SCALES.pack(k_scale.data_ptr(), v_scale.data_ptr(), max(ks[0], heads), max(vs[0], heads))
    raise ValueError(f"k_scale, v_scale: expected two float32 tensors [{blocks}, {heads}] with contiguous rows on cuda:{index}")


_TURN = 5 * 10 ** 49 * 2 ** 160 // 314159265358979323846264338327950288419716939937511  # 2^160 / (2 pi)


class Rotary:
    """Angles of rotary positions: pair i of the first rotary_dim channels of a head turns by steps[i] radians per position.

    The pairs are channels (i, i + rotary_dim / 2), or with `interleaved` (2 i, 2 i + 1). Without scaling, steps[i] =
    base^(-2 i / rotary_dim). Scalings to contexts that are `factor` times longer than the `first` tokens of training (without one
    of these, factor and first change nothing):
      "linear"  every step divided by factor (position interpolation, Chen et al. 2023)
      "base"    base * factor^(rotary_dim / (rotary_dim - 2)): the fastest pair stays, the slowest is divided by factor (NTK-aware scaling)
      "bands"   by how often a pair turns over `first` tokens: `high` times and more stays, `low` times and less is
                divided by factor, between them in proportion (model configurations publish it as rope type "llama3")
      "ramp"    in proportion over the pairs between those that turn `fast` and `slow` times over `first` tokens; cosines and sines
                are multiplied by `times`, by default 0.1 ln(factor) + 1 (YaRN, Peng et al. 2023; its ramp over whole pairs, fast 32 and slow 1)
    `times` multiplies cosines and sines with any scaling. Angles of other rules: Rotary.of(steps)."""

    def __init__(self, rotary_dim, base=10000.0, interleaved=False, scaling=None, factor=1.0, first=0, low=1.0, high=4.0, fast=32.0, slow=1.0,
                 times=None, device="cuda"):
        if rotary_dim < 8 or rotary_dim % 8:
            raise ValueError(f"rotary_dim {rotary_dim}: a multiple of 8")
        if not base > 1 or not math.isfinite(base) or not factor > 0 or not math.isfinite(factor):
            raise ValueError(f"base {base}, factor {factor}: a finite base above 1 and a finite factor above 0")
        if scaling not in (None, "linear", "base", "bands", "ramp"):
            raise ValueError(f"scaling {scaling!r}: None, 'linear', 'base', 'bands' or 'ramp'")
        if scaling in ("bands", "ramp") and not first > 0:
            raise ValueError(f"scaling {scaling!r} needs first, the tokens of the context that it starts from")
        if scaling == "bands" and not high > low or scaling == "ramp" and not fast > slow > 0:
            raise ValueError("high has to be above low, fast above slow and slow above 0")
        if scaling == "base":
            base *= factor ** (rotary_dim / (rotary_dim - 2))
        steps = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
        if scaling == "linear":
            steps = [t / factor for t in steps]
        elif scaling == "bands":
            keep = [min(1.0, max(0.0, (t * first / (2 * math.pi) - low) / (high - low))) for t in steps]
            steps = [t * x + t / factor * (1.0 - x) for t, x in zip(steps, keep)]
        elif scaling == "ramp":
            lo, hi = (rotary_dim * math.log(first / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rotary_dim - 1)
            slowed = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rotary_dim // 2)]
            steps = [t / factor * x + t * (1.0 - x) for t, x in zip(steps, slowed)]
            times = 0.1 * math.log(factor) + 1.0 if times is None else times
        self._set(steps, interleaved, 1.0 if times is None else times, device)

    @classmethod
    def of(cls, steps, interleaved=False, times=1.0, device="cuda"):
        """Angles of rotary_dim / 2 given steps, in radians per position."""
        self = cls.__new__(cls)
        self._set([float(t) for t in steps], interleaved, times, device)
        return self

    def _set(self, steps, interleaved, times, device):
        if len(steps) < 4 or len(steps) % 4 or not all(map(math.isfinite, steps)) or not math.isfinite(times):
            raise ValueError("steps: a multiple of 4 finite numbers, and a finite times")
        self.rotary_dim, self.steps, self.interleaved, self.times = 2 * len(steps), tuple(steps), bool(interleaved), float(times)
        # in 2^-64 of a whole turn, modulo 1
        ratios = [t.as_integer_ratio() for t in steps]
        turns = [((2 * n * _TURN // d >> 96) + 1 >> 1) % 2 ** 64 for n, d in ratios]  # rounded to the nearest
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)
        self._packed = None

    def _pack(self, index):
        if self._packed is None:
            self._packed = (self.turns.get_device(), _ROTARY.pack(self.turns.data_ptr(), self.rotary_dim, self.interleaved, self.times))
        if self._packed[0] != index:
            raise ValueError(f"rotary: its angles are on {self.turns.device}, the others on cuda:{index}")
        return self._packed[1]


def rotate(x, positions, rotary, out=None, inverse=False, stream=None):
    """x [tokens, heads, head_dim] (bf16, f16 or f32, any strides with contiguous channels) rotated to `positions` [tokens]
    (int32) by a Rotary (tq_rotate). inverse: the transposed rotation, which takes a gradient of the result to that of x. out: the
    tensor to write, which may be x. Returns out. Where x requires a gradient the rotation is recorded; it takes no out then."""
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out: a recorded rotation makes its result itself (torch.no_grad() records nothing)")
        return _Recorded.apply(x, positions, rotary, inverse, stream)
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    if len(shape) != 3 or dtype not in _DTYPES or index < 0:
        raise ValueError("x: expected a bf16, f16 or f32 CUDA tensor [tokens, heads, head_dim]")
    place = _ints("positions", positions, index, shape[0])
    rot = rotary._pack(index)
    raw, on = _here(index, stream, (x, positions, rotary.turns, out))
    if on is not None:
        with on:
            return _rotate(x, shape, dtype, index, place, rot, out, inverse, raw)
    return _rotate(x, shape, dtype, index, place, rot, out, inverse, raw)


class _Recorded(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, rotary, inverse, stream):
        ctx.save_for_backward(positions)
        ctx.rotary, ctx.inverse = rotary, inverse
        return rotate(x, positions, rotary, inverse=inverse, stream=stream)

    @staticmethod
    def backward(ctx, grad):
        if grad.stride(2) != 1:
            grad = grad.contiguous()
        return rotate(grad, *ctx.saved_tensors, ctx.rotary, inverse=not ctx.inverse), None, None, None, None


def _rotate(x, shape, dtype, index, place, rot, out, inverse, raw):
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
    elif out.shape != shape or out.dtype is not dtype or out.get_device() != index:
        raise ValueError("out: expected a tensor of x's shape, type and device")
    xs, os = x.stride(), out.stride()
    if xs[2] != 1 or os[2] != 1:
        raise ValueError("x, out: the channels of a head have to be contiguous")
    check(load().tq_rotate(rot, x.data_ptr(), out.data_ptr(), _DTYPES[dtype], _STRIDES.pack(xs[0], xs[1]), _STRIDES.pack(os[0], os[1]), place,
                           shape[0], shape[1], shape[2], 1 if inverse else 0, raw))
    return out


def extend(k, v, k_pool, v_pool, table, seq_ids, starts, totals, rotary=None, positions=None, q=None, q_out=None, k_scale=None, v_scale=None,
           status=None, stream=None):
    """Writes a step's new tokens into the pools, K rotated on the way (tq_paged_extend).

    k, v: [rows, n_kv_heads, head_dim] (bf16, f16 or f32, any strides with contiguous channels); request b's new rows are
    [starts[b], starts[b + 1]), the last of its totals[b] tokens in the pages of table row seq_ids[b] (None: row b), as
    map_blocks gives them. rotary: a Rotary (None: K is written as it is); positions: int32 [rows] to rotate by instead of
    the tokens' places. q: [rows, n_q_heads, head_dim] of k's type, rotated into q_out (which may be q; None: a new
    tensor, whose rows of no request are not written). k_scale, v_scale: float32 [n_blocks, n_kv_heads] of pools of
    torch.float8_e4m3fn, which are kept up with the tokens. Returns q_out. No gradient is recorded: for training, rotate()."""
    scaled = k_scale is not None or v_scale is not None
    index, pool, d, heads, _ = _pools(k_pool, v_pool, scaled)
    scales = _scales(k_scale, v_scale, index, k_pool.shape[0], heads)
    shape, dtype = k.shape, k.dtype
    if (len(shape) != 3 or shape != v.shape or dtype is not v.dtype or dtype not in _DTYPES or k.get_device() != index
            or v.get_device() != index or shape[1] != heads or shape[2] != d):
        raise ValueError("k, v: expected two tensors [rows, n_kv_heads, head_dim] of one type that fit the pools")
    ks, vs = k.stride(), v.stride()
    if ks[2] != 1 or vs[2] != 1:
        raise ValueError("k, v: the channels of a head have to be contiguous")
    n, batch = shape[0], starts.shape[0] - 1
    if batch < 0:
        raise ValueError("starts: expected [batch + 1] entries")
    args = (_table(table, index), None if seq_ids is None else _ints("seq_ids", seq_ids, index, batch), _ints("starts", starts, index),
            _ints("totals", totals, index, batch), batch, None if status is None else _ints("status", status, index, 1))
    places = 0 if positions is None else _ints("positions", positions, index, n)
    if rotary is None and (q is not None or positions is not None):
        raise ValueError("q and positions go with a rotary")
    if q is None and q_out is not None:
        raise ValueError("q_out goes with q")
    rot = None if rotary is None else rotary._pack(index)
    q_shape = None if q is None else q.shape
    if q is not None and (len(q_shape) != 3 or q_shape[0] != n or q_shape[2] != d or q.dtype is not dtype or q.get_device() != index):
        raise ValueError(f"q: expected a {dtype} tensor [{n}, n_q_heads, {d}] on cuda:{index}")
    if stream is None and torch._C._cuda_getDevice() == index:
        return _extend(k, v, ks, vs, n, dtype, pool, scales, rot, places, q, q_shape, q_out, args, torch._C._cuda_getCurrentRawStream(index))
    raw, on = _here(index, stream, (k, v, k_pool, v_pool, table, seq_ids, starts, totals, positions, q, q_out, k_scale, v_scale, status,
                                    None if rotary is None else rotary.turns))
    if on is not None:
        with on:
            return _extend(k, v, ks, vs, n, dtype, pool, scales, rot, places, q, q_shape, q_out, args, raw)
    return _extend(k, v, ks, vs, n, dtype, pool, scales, rot, places, q, q_shape, q_out, args, raw)


def _extend(k, v, ks, vs, n, dtype, pool, scales, rot, places, q, q_shape, q_out, args, raw):
    if q is None:
        queries = (0, 0, 0, 0, 0, 0, 0)
    else:
        if q_out is None:
            q_out = torch.empty(q_shape, dtype=dtype, device=q.device)
        elif q_out.shape != q_shape or q_out.dtype is not dtype or q_out.get_device() != q.get_device():
            raise ValueError("q_out: expected a tensor of q's shape, type and device")
        qs, os = q.stride(), q_out.stride()
        if qs[2] != 1 or os[2] != 1:
            raise ValueError("q, q_out: the channels of a head have to be contiguous")
        queries = (q.data_ptr(), q_out.data_ptr(), qs[0], qs[1], os[0], os[1], q_shape[1])
    rows = _NEW_ROWS.pack(k.data_ptr(), v.data_ptr(), queries[0], queries[1], ks[0], ks[1], vs[0], vs[1], *queries[2:6], places, n, queries[6],
                          _DTYPES[dtype])
    table, seq_ids, starts, totals, batch, word = args
    check(load().tq_paged_extend(pool, scales, rows, rot, *table, seq_ids, starts, totals, batch, word, raw))
    return q_out


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
              workspace=None, status=None, stream=None, k_scale=None, v_scale=None):
    """Attention of each request's new tokens over the paged cache that already holds them (tq_paged_attention; with k_scale and
    v_scale, float32 [n_blocks, n_kv_heads], over pools of torch.float8_e4m3fn: tq_paged_attention8).

    q: [rows, n_q_heads, head_dim] of the pools' type (bf16 or f16 where they are e4m3), request b's rows at [q_starts[b], q_starts[b + 1]); kv_lens[b]: its
    tokens with the new ones, in the pages of table row seq_ids[b] (None: row b). max_q: no request has more rows (0:
    unknown; few rows take a kernel of their own); max_kv: no request has more tokens (0: unknown; short calls launch fewer
    CTAs, and over e4m3 little work takes that kernel too). Returns out, of q's shape; rows of no request stay as they are. What the cache holds behind a request's
    tokens does not matter; a token that any of its queries sees has to be finite."""
    scaled = k_scale is not None or v_scale is not None
    index, kv, d, heads, dtype = _pools(k_pool, v_pool, scaled)
    pages = _table(table, index)
    word = None if status is None else _ints("status", status, index, 1)
    if scaled:
        scales = _scales(k_scale, v_scale, index, k_pool.shape[0], heads)
        dtype = q.dtype
        if dtype not in _HALVES:
            raise ValueError("q: expected a bf16 or f16 tensor")

        def call8(queries, kv, batch, ws, size, raw):
            return load().tq_paged_attention8(queries, _DTYPES[dtype], kv, scales, *pages, None if seq_ids is None else _ints("seq_ids", seq_ids, index, batch),
                                              _ints("kv_lens", kv_lens, index, batch), 1 if causal else 0, ws, size, word, raw)

        return _attend(q, dtype, heads, d, index, q_starts, max_q, max_kv, softmax_scale, out, workspace, kv, stream,
                       (k_pool, v_pool, k_scale, v_scale, table, seq_ids, kv_lens, status), call8)

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
    """K and V of n_layers layers in the blocks of a BlockPool (which other caches may share): exact in 16 bits, or in 8 bits
    (torch.float8_e4m3fn) with a scale for each block and head, `scales` [n_layers, 2, n_blocks, n_kv_heads]."""

    def __init__(self, n_layers, pool, n_kv_heads, head_dim, dtype=torch.bfloat16):
        if dtype not in (torch.bfloat16, torch.float16, _E4M3):
            raise ValueError("dtype: bf16, f16 or float8_e4m3fn")
        self.pool = pool
        if dtype is _E4M3:  # the tokens of a head together: appends and attention take them so, and a row is 64 to 256 bytes
            self.kv = torch.empty((n_layers, 2, pool.n_blocks, n_kv_heads, PAGE, head_dim), dtype=dtype, device=pool.device).transpose(3, 4)
        else:
            self.kv = torch.empty((n_layers, 2, pool.n_blocks, PAGE, n_kv_heads, head_dim), dtype=dtype, device=pool.device)
        self.scales = torch.ones((n_layers, 2, pool.n_blocks, n_kv_heads), device=pool.device) if dtype is _E4M3 else None

    def _scales(self, layer):
        return {} if self.scales is None else {"k_scale": self.scales[layer, 0], "v_scale": self.scales[layer, 1]}

    def append(self, layer, k, v, slots, stream=None):
        """Writes the step's k, v [tokens, n_kv_heads, head_dim] of one layer at the slots of pool.map (16 bits: a cache of 8 bits
        takes extend, whose scales need to know which tokens a block holds)."""
        append(k, v, self.kv[layer, 0], self.kv[layer, 1], slots, self.pool.status, stream)

    def extend(self, layer, k, v, seq_ids, starts, totals, rotary=None, positions=None, q=None, q_out=None, stream=None):
        """Writes the step's k, v [tokens, n_kv_heads, head_dim] of one layer, K rotated by a Rotary, and returns q [tokens,
        n_q_heads, head_dim] rotated; starts and totals are those of pool.map. See extend()."""
        return extend(k, v, self.kv[layer, 0], self.kv[layer, 1], self.pool.table, seq_ids, starts, totals, rotary, positions, q, q_out,
                      status=self.pool.status, stream=stream, **self._scales(layer))

    def attention(self, layer, q, seq_ids, q_starts, kv_lens, causal=True, softmax_scale=0.0, max_q=0, max_kv=0, out=None,
                  workspace=None, stream=None):
        """Attention of the step's q [tokens, n_q_heads, head_dim] over one layer; q_starts and kv_lens are the starts and totals
        of pool.map. See attention()."""
        return attention(q, self.kv[layer, 0], self.kv[layer, 1], self.pool.table, seq_ids, q_starts, kv_lens, causal, softmax_scale, max_q,
                         max_kv, out, workspace, self.pool.status, stream, **self._scales(layer))
