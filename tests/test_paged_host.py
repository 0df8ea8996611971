"""CPU tests of the exact paged cache's entry points: what the host refuses before any launch."""
import ctypes
import os
import struct
import subprocess
import sys

import pytest

from kv_cache_quantization_quantize_gb300 import _abi, paged

P = 4096  # an aligned address that no refused call reads


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_quantization_quantize_gb300 import build
    build.build()


def kv(k=P, v=P, ks=(16384, 128, 64), vs=(16384, 128, 64), outer=4, tokens=128, heads=2, d=64, dtype=0):
    return paged._KV.pack(k, v, *ks, *vs, outer, tokens, heads, d, dtype)


def queries(q=P, out=P, qs=(256, 64), os=(256, 64), starts=P, rows=3, heads=4, batch=2, max_q=0, max_kv=0, scale=0.0):
    return paged._QUERIES.pack(q, out, *qs, *os, starts, rows, heads, batch, max_q, max_kv, scale)


def test_the_packed_structs_have_the_c_layout():
    assert paged._KV.size == 88 and paged._QUERIES.size == 80
    assert struct.calcsize("@P") == 8


@pytest.mark.parametrize("over,status", [
    ({"d": 96}, _abi.TQ_ERR_UNSUPPORTED), ({"dtype": 1}, _abi.TQ_ERR_UNSUPPORTED), ({"heads": 0}, _abi.TQ_ERR_INVALID_ARG),
    ({"k": 0}, _abi.TQ_ERR_INVALID_ARG), ({"v": P + 8}, _abi.TQ_ERR_INVALID_ARG), ({"ks": (16384, 0, 64)}, _abi.TQ_ERR_INVALID_ARG),
    ({"ks": (16384, 128, 60)}, _abi.TQ_ERR_INVALID_ARG), ({"vs": (-16384, 128, 64)}, _abi.TQ_ERR_INVALID_ARG),
    ({"tokens": 64}, _abi.TQ_ERR_INVALID_ARG), ({"outer": 1 << 24}, _abi.TQ_ERR_INVALID_ARG), ({"outer": 0}, _abi.TQ_ERR_INVALID_ARG),
])
def test_attention_refuses_bad_pools(over, status):
    lib = _abi.load()
    assert lib.tq_paged_attention(queries(), kv(**over), P, 4, 4, 4, None, P, 1, None, 0, None, None) == status
    assert lib.tq_last_error()


@pytest.mark.parametrize("over,status", [
    ({"heads": 3}, _abi.TQ_ERR_INVALID_ARG), ({"heads": 0}, _abi.TQ_ERR_INVALID_ARG), ({"heads": 4096}, _abi.TQ_ERR_UNSUPPORTED),
    ({"batch": -1}, _abi.TQ_ERR_INVALID_ARG), ({"batch": 65536}, _abi.TQ_ERR_UNSUPPORTED), ({"rows": -1}, _abi.TQ_ERR_INVALID_ARG),
    ({"max_q": -1}, _abi.TQ_ERR_INVALID_ARG), ({"max_kv": -1}, _abi.TQ_ERR_INVALID_ARG), ({"q": 0}, _abi.TQ_ERR_INVALID_ARG),
    ({"out": P + 2}, _abi.TQ_ERR_INVALID_ARG), ({"starts": 0}, _abi.TQ_ERR_INVALID_ARG), ({"qs": (256, 60)}, _abi.TQ_ERR_INVALID_ARG),
    ({"os": (12, 64)}, _abi.TQ_ERR_INVALID_ARG), ({"scale": float("inf")}, _abi.TQ_ERR_INVALID_ARG),
    ({"rows": 1 << 29, "heads": 4}, _abi.TQ_ERR_UNSUPPORTED),
])
def test_attention_refuses_bad_queries(over, status):
    lib = _abi.load()
    assert lib.tq_paged_attention(queries(**over), kv(), P, 4, 4, 4, None, P, 1, None, 0, None, None) == status
    assert lib.tq_cross_attention(queries(**over), kv(), None, P, None, 0, None, None) == status


def test_attention_refuses_bad_tables_and_flags():
    lib = _abi.load()
    bad = _abi.TQ_ERR_INVALID_ARG

    def call(table=P, seqs=4, pages=4, stride=4, lens=P, causal=1):
        return lib.tq_paged_attention(queries(), kv(), table, seqs, pages, stride, None, lens, causal, None, 0, None, None)

    assert call(table=None) == bad and call(seqs=0) == bad and call(pages=0) == bad and call(stride=3) == bad
    assert call(lens=None) == bad and call(causal=2) == bad and call(seqs=1) == bad and call(pages=(1 << 20) + 1) == bad
    assert lib.tq_paged_attention(None, kv(), P, 4, 4, 4, None, P, 1, None, 0, None, None) == bad
    assert lib.tq_paged_attention(queries(), None, P, 4, 4, 4, None, P, 1, None, 0, None, None) == bad
    # an empty batch, or no rows, is done at once
    assert lib.tq_paged_attention(queries(batch=0), kv(), P, 4, 4, 4, None, P, 1, None, 0, None, None) == _abi.TQ_OK
    assert lib.tq_paged_attention(queries(rows=0), kv(), P, 4, 4, 4, None, P, 1, None, 0, None, None) == _abi.TQ_OK


def test_cross_attention_refuses_a_mixed_form():
    lib = _abi.load()
    bad = _abi.TQ_ERR_INVALID_ARG
    assert lib.tq_cross_attention(queries(), kv(), P, P, None, 0, None, None) == bad
    assert lib.tq_cross_attention(queries(), kv(), None, None, None, 0, None, None) == bad
    assert lib.tq_cross_attention(queries(), kv(outer=4), P, None, None, 0, None, None) == bad
    assert lib.tq_cross_attention(queries(), kv(outer=1), None, P, None, 0, None, None) == bad


def test_append_refuses():
    lib = _abi.load()
    st = struct.pack("@2q", 128, 64)

    def call(pool=None, k=P, v=P, dt=0, ks=st, vs=st, slots=P, n=3):
        return lib.tq_paged_append(pool or kv(), k, v, dt, ks, vs, slots, n, None, None)

    bad = _abi.TQ_ERR_INVALID_ARG
    assert call(k=None) == bad and call(v=P + 1) == bad and call(dt=3) == bad and call(dt=1, k=P + 2) == bad and call(slots=None) == bad
    assert call(ks=None) == bad and call(n=-1) == bad and call(pool=kv(tokens=64)) == bad and call(pool=kv(k=0)) == bad
    assert call(pool=kv(d=32)) == _abi.TQ_ERR_UNSUPPORTED and call(n=0) == _abi.TQ_OK


def test_block_maps_refuse():
    lib = _abi.load()
    bad = _abi.TQ_ERR_INVALID_ARG

    def release(table=P, seqs=4, pages=4, stride=4, free=P, blocks=8, n_free=P, ids=P, batch=2):
        return lib.tq_blocks_release(table, seqs, pages, stride, free, blocks, n_free, ids, None, batch, None, None)

    def mapped(table=P, seqs=4, pages=4, stride=4, free=P, blocks=8, n_free=P, ids=P, lens=P, new=P, batch=2, starts=P, totals=P, slots=P, room=3):
        return lib.tq_blocks_map(table, seqs, pages, stride, free, blocks, n_free, ids, lens, new, batch, starts, totals, slots, room, None, None)

    for f in (release, mapped):
        for over in ({"table": None}, {"seqs": 0}, {"pages": 0}, {"stride": 3}, {"free": None}, {"blocks": 0}, {"blocks": 1 << 24},
                     {"n_free": None}, {"ids": None}, {"batch": -1}):
            assert f(**over) == bad, over
        assert f(batch=4097) == _abi.TQ_ERR_UNSUPPORTED
    for over in ({"lens": None}, {"new": None}, {"starts": None}, {"totals": None}, {"slots": None}, {"room": -1}, {"room": (1 << 30) + 1}):
        assert mapped(**over) == bad, over
    assert release(batch=0) == _abi.TQ_OK


def test_the_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((3, 128, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 3), dtype=torch.int32)
    with pytest.raises(ValueError):
        paged.attention(x[0, :1].expand(1, 2, 64), x, x, i, None, i[0, :2], i[0, :1])
    with pytest.raises(ValueError):
        paged.append(x[0, :1], x[0, :1], x, x, i[0, :1])
    with pytest.raises(ValueError):
        paged.map_blocks(i, i[0], i[0], i[0], i[0], i[0], 1)
    with pytest.raises(ValueError):
        paged.cross_attention(x[0], x[0], x[0], i[0], kv_starts=i[0])
    with pytest.raises(ValueError):
        paged.BlockPool(0, 1, 1)
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_the_package_imports_without_the_raw_allocator():
    """A torch without these two private names (a CPU build) still has the host-only parts."""
    pytest.importorskip("torch")
    code = """
import torch
for name in ("_cuda_cudaCachingAllocator_raw_alloc", "_cuda_cudaCachingAllocator_raw_delete"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import kv_cache_quantization_quantize_gb300 as tqm
assert tqm.config(head_dim=64).head_dim == 64
assert tqm.paged._raw_allocator() == (None, None)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("over", [{"rows": 1, "qs": (1027, 64), "os": (3, 64)}, {"heads": 1, "batch": 1, "qs": (64, 7), "os": (64, 1)}])
def test_strides_of_a_single_row_or_head_are_not_checked(over):
    """What comes next is the device or the workspace, whichever this machine lacks."""
    lib = _abi.load()
    lib.tq_paged_attention(queries(**over), kv(heads=1), P, 4, 4, 4, None, P, 1, None, 0, None, None)
    text = lib.tq_last_error().decode()
    assert "workspace" in text or "device" in text, text
