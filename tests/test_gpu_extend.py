"""GPU tests of rotary positions, rotated appends and the paged cache of 8 bits, against plain 64-bit references."""
import math

import pytest
import torch

from kv_cache_quantization_quantize_gb300 import paged
from tests import extend_reference as ref
from tests import paged_reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn
HALVES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_quantization_quantize_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def starts_of(n):
    s = [0]
    for x in n:
        s.append(s[-1] + x)
    return s


def normal(gen, shape, dtype, layout="plain"):
    """Values at strides: rows of a wider tensor, or at an odd address."""
    x = torch.randn(shape, generator=gen, dtype=torch.float32).to(dtype)
    if layout == "fused":
        wide = torch.zeros((shape[0], shape[1] + 3, shape[2]), dtype=dtype, device=DEV)
        wide[:, 1:1 + shape[1]] = x.to(DEV)
        return wide[:, 1:1 + shape[1]]
    if layout == "odd":
        flat = torch.zeros(x.numel() + 1, dtype=dtype, device=DEV)
        flat[1:] = x.flatten().to(DEV)
        return flat[1:].view(shape)
    return x.to(DEV)


# ---- rotation ----

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,d,rd,layout", [
    (1, 1, 64, 64, "plain"), (5, 3, 128, 128, "fused"), (33, 2, 256, 64, "plain"), (7, 5, 96, 24, "plain"), (130, 4, 128, 32, "odd"), (3, 1, 8, 8, "plain"),
    (9, 7, 80, 32, "fused"), (2600, 9, 64, 64, "plain"), (20000, 1, 64, 16, "fused"), (2, 3, 1024, 1024, "plain"), (2, 1, 1000, 8, "plain"),
])
def test_rotation(dtype, interleaved, tokens, heads, d, rd, layout):
    gen = torch.Generator().manual_seed(tokens * 1000 + d)
    x = normal(gen, (tokens, heads, d), dtype, layout)
    far = torch.randint(0, 1 << 20, (tokens,), generator=gen)
    for i, p in enumerate([0, 1, 2 ** 31 - 1, -1, 131071, -2 ** 31]):
        if i < tokens:
            far[i] = p
    at = far.to(torch.int32).to(DEV)
    r = paged.Rotary(rd, base=10000.0, interleaved=interleaved, scaling="linear", factor=4.0, times=1.25)
    for inverse in (False, True):
        y = paged.rotate(x, at, r, inverse=inverse)
        want, size = ref.rotate(x, at, r.steps, r.times, interleaved, inverse)
        bound = ref.rounding(want, dtype) + ref.rotation_error(size, at, r.steps) * (1 + torch.finfo(dtype).eps)
        assert y.dtype is dtype and bool(((y.double() - want).abs() <= bound).all())
        assert torch.equal(y[..., rd:], x[..., rd:])


def test_rotation_in_place_and_into_strides():
    gen = torch.Generator().manual_seed(1)
    wide = normal(gen, (50, 12, 128), torch.bfloat16)
    at, r = torch.arange(50, dtype=torch.int32, device=DEV), paged.Rotary(64)
    q = wide[:, 2:7]
    want = paged.rotate(q.clone(), at, r)
    rest = wide.clone()
    assert paged.rotate(q, at, r, out=q) is q and torch.equal(q, want)
    rest[:, 2:7] = want
    assert torch.equal(wide, rest)
    out = torch.zeros((5, 50, 128), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    paged.rotate(wide[:, 7:], at, r, out=out)
    assert torch.equal(out, paged.rotate(wide[:, 7:].contiguous(), at, r))


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_inverse_is_the_gradient(interleaved):
    gen = torch.Generator().manual_seed(2)
    x, g = normal(gen, (6, 2, 64), torch.float32), normal(gen, (6, 2, 64), torch.float32)
    at, r = i32([0, 3, 70, 1000, 9, 131072]), paged.Rotary(32, interleaved=interleaved, scaling="ramp", factor=4.0, first=1024)
    back = paged.rotate(g, at, r, inverse=True)
    # against the formula's: autograd through the 64-bit rotation
    leaf = x.double().requires_grad_()
    rd = r.rotary_dim
    angle = at.double()[:, None, None] * torch.tensor(r.steps, dtype=torch.float64, device=DEV)
    a, b = (leaf[..., 0:rd:2], leaf[..., 1:rd:2]) if interleaved else (leaf[..., :rd // 2], leaf[..., rd // 2:rd])
    c, s = angle.cos() * r.times, angle.sin() * r.times
    y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2) if interleaved else torch.cat([a * c - b * s, b * c + a * s], -1)
    torch.cat([y, leaf[..., rd:]], -1).backward(g.double())
    _, size = ref.rotate(g, at, r.steps, r.times, interleaved, True)
    bound = ref.rounding(leaf.grad, torch.float32) + 2 * ref.rotation_error(size, at, r.steps)
    assert bool(((back.double() - leaf.grad).abs() <= bound).all())
    # against differences: the map is linear, so one step of any size gives its slope up to the rounding of both sides
    for element in [(1, 0, 0), (3, 1, 17), (5, 0, 40)]:
        moved = x.clone()
        moved[element] += 8.0
        slope = ((paged.rotate(moved, at, r).double() - paged.rotate(x, at, r).double()) * g.double()).sum() / 8.0
        assert abs(slope.item() - back[element].item()) <= 64 * 2.0 ** -22 * 12 * g.abs().max().item()


def test_rotation_of_nothing_and_refusals():
    r = paged.Rotary(64)
    x = torch.zeros(3, 2, 64, device=DEV)
    assert paged.rotate(x[:0], i32([]), r).shape == (0, 2, 64) and paged.rotate(x[:, :0], i32([1, 2, 3]), r).shape == (3, 0, 64)
    for args in [(x, i32([1, 2]), r), (x.double(), i32([1, 2, 3]), r), (x[0], i32([1, 2, 3]), r), (x.transpose(1, 2), i32([1, 2, 3]), paged.Rotary(8)),
                 (x, torch.tensor([1, 2, 3], device=DEV), r), (x, i32([1, 2, 3]), paged.Rotary(64, device="cpu"))]:
        with pytest.raises(ValueError):
            paged.rotate(*args)
    with pytest.raises(ValueError):
        paged.rotate(x, i32([1, 2, 3]), r, out=torch.zeros(3, 2, 64, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(RuntimeError):
        paged.rotate(x, i32([1, 2, 3]), paged.Rotary(128))


# ---- appends ----

def place_requests(nq, kv, seed, spare=3):
    """(table, slot, blocks): pages of requests in scrambled order, in scrambled rows."""
    pages = [-(-m // 128) for m in kv]
    blocks, g = sum(pages) + spare, torch.Generator().manual_seed(seed)
    ids, slot = torch.randperm(blocks, generator=g).tolist(), torch.randperm(len(nq) + 2, generator=g).tolist()[:len(nq)]
    table = torch.full((len(nq) + 2, max(pages, default=0) + 2), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(pages):
        table[slot[b], :p] = torch.tensor(ids[at:at + p], dtype=torch.int32)
        at += p
    return table.to(DEV), slot, blocks


def pool_of(blocks, heads, d, dtype, heads_first):
    shape = (blocks, heads, 128, d) if heads_first else (blocks, 128, heads, d)
    pool = torch.zeros(shape, dtype=torch.uint8 if dtype is E4M3 else dtype, device=DEV)
    if dtype is E4M3:  # a pattern of its own everywhere, NaN among it
        pool.copy_(torch.arange(pool.numel(), device=DEV).view(shape) % 253)
        pool = pool.view(E4M3)
    else:
        pool.fill_(-7.0)
    return pool.transpose(1, 2) if heads_first else pool


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8)) if a.dtype is E4M3 else torch.equal(a, b)


def values8(pool, scale):
    """The number that each element stands for, in 64 bits."""
    return pool.float().double() * scale.double()[:, None, :, None]


CASES = [  # (new tokens, tokens with them), hq, hkv, d, rd, layout, heads first
    (([1], [1]), 2, 1, 128, 128, "plain", False),
    (([1, 1, 0, 1], [129, 128, 0, 300]), 8, 2, 128, 128, "fused", False),
    (([8, 9, 3], [8, 200, 129]), 0, 3, 64, 32, "plain", True),
    (([128, 129, 1, 255], [128, 257, 100, 255]), 4, 4, 64, 64, "plain", False),
    (([700], [1000]), 5, 5, 128, 64, "odd", False),
    (([300, 2], [301, 130]), 6, 2, 256, 256, "plain", True),
    (([5, 130], [133, 135]), 2, 1, 256, 24, "fused", False),
    (([1] * 70, list(range(1, 71))), 4, 1, 64, 64, "plain", False),
    (([2000, 1, 700], [2000, 77, 900]), 4, 2, 128, 128, "fused", False),
]


def new_rows(case, dtype, seed, tail=2):
    (nq, kv), hq, hkv, d, rd, layout, _ = case
    gen = torch.Generator().manual_seed(seed)
    rows = sum(nq) + tail
    return [normal(gen, (rows, h, d), dtype, layout) if h else None for h in (hq, hkv, hkv)]


@pytest.mark.parametrize("src,dst", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float16), (torch.float16, torch.bfloat16)])
@pytest.mark.parametrize("interleaved,moved", [(False, False), (True, True)])
@pytest.mark.parametrize("case", CASES)
def test_extend_of_exact_pools(src, dst, interleaved, moved, case):
    (nq, kv), hq, hkv, d, rd, _, heads_first = case
    q, k, v = new_rows(case, src, 5)
    table, slot, blocks = place_requests(nq, kv, 6)
    pools = [pool_of(blocks, hkv, d, dst, heads_first) for _ in range(2)]
    r = paged.Rotary(rd, base=10000.0, interleaved=interleaved, times=1.5)
    rows, total = k.shape[0], sum(nq)
    at = torch.cat([torch.arange(m - n, m) for n, m in zip(nq, kv)]).to(torch.int32).to(DEV)
    positions = torch.randint(0, 1 << 17, (rows,), dtype=torch.int32, device=DEV) if moved else None
    q_out = None if q is None else torch.full((rows, hq, d), 3.0, dtype=src, device=DEV)
    status = i32([0])
    got = paged.extend(k, v, *pools, table, i32(slot), i32(starts_of(nq)), i32(kv), rotary=r, positions=positions, q=q, q_out=q_out, status=status)
    assert got is q_out and status.item() == 0
    turn = at if positions is None else positions[:total]
    want, size = ref.rotate(k[:total], turn, r.steps, r.times, interleaved)
    slots = torch.tensor([int(table[slot[b], p // 128]) * 128 + p % 128 for b, (n, m) in enumerate(zip(nq, kv)) for p in range(m - n, m)], device=DEV).long()
    flat = [p.transpose(1, 2).contiguous().transpose(1, 2).reshape(-1, hkv, d) if heads_first else p.view(-1, hkv, d) for p in pools]
    err = (flat[0][slots].double() - want).abs()
    assert bool((err <= ref.rounding(want, dst) + ref.rotation_error(size, turn, r.steps) * (1 + torch.finfo(dst).eps)).all())
    assert torch.equal(flat[1][slots], v[:total].to(dst))
    rest = torch.ones(flat[0].shape[0], dtype=torch.bool, device=DEV)
    rest[slots] = False
    assert bool((flat[0][rest] == -7.0).all()) and bool((flat[1][rest] == -7.0).all())
    if q is not None:
        want, size = ref.rotate(q[:total], turn, r.steps, r.times, interleaved)
        bound = ref.rounding(want, src) + ref.rotation_error(size, turn, r.steps) * (1 + torch.finfo(src).eps)
        assert bool(((q_out[:total].double() - want).abs() <= bound).all()) and bool((q_out[total:] == 3.0).all())


def check_extended(before, after, scales, new, table, slot, nq, kv, error):
    """Pages, scales and untouched places of K or V after one step. new: 64-bit rows; error: what fp32 may add to each."""
    row, touched = 0, torch.zeros(after.shape[:2], dtype=torch.bool, device=DEV)
    was, now = scales
    blocks = torch.zeros(after.shape[0], dtype=torch.bool, device=DEV)
    for b, (n, m) in enumerate(zip(nq, kv)):
        for page in range((m - n) // 128, -(-m // 128) if n else 0):
            lo, hi = max(m - n, page * 128), min(m, page * 128 + 128)
            block, at = int(table[slot[b], page]), lo - page * 128
            x, e = (t[row + lo - (m - n):row + hi - (m - n)] for t in (new, error))
            for h in range(after.shape[2]):
                finite = x[:, h].abs().nan_to_num(0.0, 0.0, 0.0)
                scale, had = float(now[block, h]), float(was[block, h]) if at else 2.0 ** ref.LEAST
                most, slack = finite.max().item(), e[:, h].nan_to_num(0.0, 0.0, 0.0).max().item()
                assert max(had, ref.scale_of(most - slack)) <= scale <= max(had, ref.scale_of(most + slack))
                got = after[block, at:at + hi - lo, h].float().double()
                y = x[:, h] / scale
                near = y.abs().nan_to_num(0.0).clamp(max=448.0) + e[:, h] / scale
                bound = ref.half_step8(near.nan_to_num(0.0).clamp(max=448.0)) + e[:, h] / scale
                assert bool(((got - y.clamp(-448.0, 448.0)).abs() <= bound)[~x[:, h].isnan()].all()) and torch.equal(got.isnan(), x[:, h].isnan())
                held = before[block, :at, h].float().double()
                if scale == had:
                    assert same(after[block, :at, h].contiguous(), before[block, :at, h].contiguous())
                else:
                    want = ref.nearest8(held * (had / scale))
                    moved = after[block, :at, h].float().double()
                    assert torch.equal(torch.where(held.isnan(), 0.0, want), torch.where(moved.isnan(), 0.0, moved)) and torch.equal(held.isnan(), moved.isnan())
            touched[block, :at + hi - lo] = True
            blocks[block] = True
        row += n
    assert same(after[~touched].contiguous(), before[~touched].contiguous()) and torch.equal(was[~blocks], now[~blocks])


def run_extend8(case, dtype, seed, interleaved=False, loud=None, change=None):
    (nq, kv), hq, hkv, d, rd, _, heads_first = case
    q, k, v = new_rows(case, dtype, seed)
    if loud is not None:  # each row and head by a loudness of its own
        gen = torch.Generator().manual_seed(seed + 1)
        for x in (k, v):
            x.copy_((x.float() * torch.exp2(torch.randint(-loud, loud + 1, x.shape[:2] + (1,), generator=gen).float()).to(DEV)).to(dtype))
    if change is not None:
        change(k, v)
    table, slot, blocks = place_requests(nq, kv, seed + 2)
    gen = torch.Generator().manual_seed(seed + 3)
    pools = [pool_of(blocks, hkv, d, E4M3, heads_first) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-12, 3, (blocks, hkv), generator=gen).float()).to(DEV) for _ in range(2)]
    before, was = [p.view(torch.uint8).clone(memory_format=torch.preserve_format).view(E4M3) for p in pools], [s.clone() for s in scales]
    r = paged.Rotary(rd, interleaved=interleaved)
    status, total = i32([0]), sum(nq)
    q_out = paged.extend(k, v, *pools, table, i32(slot), i32(starts_of(nq)), i32(kv), rotary=r, q=q, k_scale=scales[0], v_scale=scales[1], status=status)
    assert status.item() == 0
    at = torch.cat([torch.arange(m - n, m) for n, m in zip(nq, kv)]).to(torch.int32).to(DEV)
    want, size = ref.rotate(k[:total], at, r.steps, r.times, interleaved)
    host = table.cpu()
    check_extended(before[0], pools[0], (was[0], scales[0]), want, host, slot, nq, kv, ref.rotation_error(size, at, r.steps) + want.abs() * 2.0 ** -24)
    exact = v[:total].double()
    check_extended(before[1], pools[1], (was[1], scales[1]), exact, host, slot, nq, kv, torch.zeros_like(exact))
    if q is not None:
        want, size = ref.rotate(q[:total], at, r.steps, r.times, interleaved)
        bound = ref.rounding(want, dtype) + ref.rotation_error(size, at, r.steps) * (1 + torch.finfo(dtype).eps)
        assert bool(((q_out[:total].double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_extend_of_8_bits(dtype, interleaved, case):
    run_extend8(case, dtype, 11, interleaved)


@pytest.mark.parametrize("case", CASES[1:5] + CASES[6:7])
def test_extend_of_8_bits_with_loudness(case):
    run_extend8(case, torch.bfloat16, 12, loud=10)


@pytest.mark.parametrize("case", [CASES[1], CASES[3]])
def test_extend_of_8_bits_at_the_ends_of_the_scales(case):
    def ends(k, v):
        k[0] *= 2.0 ** 100  # past 448 * 2^60
        v[0] = 0.0
        if v.shape[0] > 4:
            v[1] *= 2.0 ** -100
            v[2] = torch.finfo(torch.float32).max
    run_extend8(case, torch.float32, 13, change=ends)


def test_values_that_are_no_numbers_do_not_count_for_a_scale():
    def spoil(k, v):
        v[0, 0, 3], v[1, 0, 5], v[2, 1, 0] = math.nan, math.inf, -math.inf
    run_extend8(((([3, 20], [3, 140])), 0, 2, 64, 64, "plain", False), torch.bfloat16, 14, change=spoil)


@pytest.mark.parametrize("d,heads", [(64, 3), (128, 2), (256, 1)])
def test_token_by_token_the_cache_keeps_up(d, heads):
    """Every token rounded at its block's scale of the time, and again where the scale grew: off by a step of the last at most."""
    n = 150
    gen = torch.Generator().manual_seed(d)
    k = normal(gen, (n, heads, d), torch.bfloat16)
    k *= torch.exp2(torch.linspace(-6, 6, n, device=DEV))[:, None, None].to(torch.bfloat16)
    pool = paged.BlockPool(4, 2, 256)
    cache = paged.PagedCache(1, pool, heads, d, dtype=E4M3)
    cache.kv.view(torch.uint8).fill_(0x7f)
    one = i32([1])
    for t in range(n):
        slots, starts, totals = pool.map(i32([1]), i32([t]), one, 1)
        assert cache.extend(0, k[t:t + 1], k[t:t + 1], i32([1]), starts, totals) is None
    assert pool.check_status() == 0
    ids = pool.table[1, :2].tolist()
    both = torch.cat([values8(cache.kv[0, 1], cache.scales[0, 1])[i] for i in ids])[:n]
    for page in range(2):
        x = k[page * 128:min(n, page * 128 + 128)].double()
        scale = cache.scales[0, 1][ids[page]].double()
        assert scale.tolist() == [ref.scale_of(m) for m in x.abs().amax((0, 2)).tolist()]
        y = x / scale[:, None]
        assert bool(((both[page * 128:page * 128 + len(x)] / scale[:, None] - y).abs() <= 2 * ref.half_step8(y)).all())


def test_extend_without_rotation_and_in_place():
    case = CASES[1]
    (nq, kv), hq, hkv, d, rd, _, _ = case
    q, k, v = new_rows(case, torch.bfloat16, 20)
    table, slot, blocks = place_requests(nq, kv, 21)
    args = (table, i32(slot), i32(starts_of(nq)), i32(kv))
    pools = [pool_of(blocks, hkv, d, torch.bfloat16, False) for _ in range(4)]
    slots = i32([int(table[slot[b], p // 128]) * 128 + p % 128 for b, (n, m) in enumerate(zip(nq, kv)) for p in range(m - n, m)] + [-1, -1])
    paged.extend(k, v, pools[0], pools[1], *args)
    paged.append(k, v, pools[2], pools[3], slots)
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    r = paged.Rotary(rd)
    apart = paged.extend(k, v, pools[0], pools[1], *args, rotary=r, q=q)
    padding = q[sum(nq):].clone()
    assert paged.extend(k, v, pools[2], pools[3], *args, rotary=r, q=q, q_out=q) is q
    assert torch.equal(apart[:sum(nq)], q[:sum(nq)]) and torch.equal(q[sum(nq):], padding) and torch.equal(pools[0], pools[2])
    # row b of the table without ids
    ordered = table[torch.tensor(slot, device=DEV)].contiguous()
    paged.extend(k, v, pools[2], pools[3], ordered, None, *args[2:], rotary=r)
    assert torch.equal(pools[0], pools[2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
def test_extend_reports_bad_arrays(dtype):
    hkv, d = 2, 64
    gen = torch.Generator().manual_seed(3)
    k, v, q = (normal(gen, (6, hkv, d), torch.bfloat16) for _ in range(3))
    pools = [pool_of(4, hkv, d, dtype, False) for _ in range(2)]
    scales = {"k_scale": torch.ones(4, hkv, device=DEV), "v_scale": torch.ones(4, hkv, device=DEV)} if dtype is E4M3 else {}
    table = i32([[0, 1], [2, -1], [99, 3], [-1, -1]])
    word, r = i32([0]), paged.Rotary(64)

    def run(ids, starts, totals):
        before = [p.view(torch.uint8).clone() for p in pools]
        word.zero_()
        out = torch.full_like(q, 9.0)
        paged.extend(k, v, *pools, table, i32(ids), i32(starts), i32(totals), rotary=r, q=q, q_out=out, status=word, **scales)
        changed = [(p.view(torch.uint8) != o).flatten(2).any(2) for p, o in zip(pools, before)]
        for p, o in zip(pools, before):
            p.view(torch.uint8).copy_(o)
        return word.item(), sorted({(b, t) for c in changed for b, t in c.nonzero().tolist()}), [bool((x != 9.0).any()) for x in out]

    last = [(1, t) for t in range(124, 128)]
    st, places, rows = run([0, 1], [0, 4, 6], [256, 0])  # the second request is refused by the map
    assert st == 0 and set(last) <= set(places) and all(b == 1 for b, _ in places) and rows == [True] * 4 + [False] * 2
    st, places, rows = run([7, 1], [0, 4, 6], [4, 2])
    assert st == paged.TQ_DEV_ERR_SEQ_ID and all(b == 2 for b, _ in places) and rows == [False] * 4 + [True] * 2
    st, places, rows = run([0, 1], [0, 4, 6], [3, 2])
    assert st == paged.TQ_DEV_ERR_LENGTH and all(b == 2 for b, _ in places) and rows == [False] * 4 + [True] * 2
    for starts, totals in [([0, 4, 7], [4, 3]), ([0, 4, 3], [4, 2]), ([0, 4, 6], [4, -2]), ([0, 4, 6], [4, 257]), ([0, 4, 6], [4, 2 ** 31 - 1])]:
        st, places, rows = run([0, 1], starts, totals)
        assert st == paged.TQ_DEV_ERR_LENGTH and all(b == 0 for b, _ in places) and places, (starts, totals)
    st, places, _ = run([1, 2], [0, 3, 6], [130, 3])  # two of three tokens on a page without a block, and a block outside the pool
    assert st == paged.TQ_DEV_ERR_BLOCK and all(b == 2 for b, _ in places) and (2, 127) in places
    st, places, rows = run([0, 1], [2, 2, 2], [4, 2])  # nobody has rows
    assert st == 0 and not places and not any(rows)


def test_extend_of_many_requests():
    """More requests than one look of 32 places finds, most of them with one token, some with none."""
    for batch, dtype in [(1500, E4M3), (1500, torch.float16)]:
        gen = torch.Generator().manual_seed(batch)
        nq = torch.randint(0, 3, (batch,), generator=gen).tolist()
        nq[700], kv = 300, []
        for n in nq:
            kv.append(n + int(torch.randint(0, 140, (1,), generator=gen)) if n else 0)
        table, slot, blocks = place_requests(nq, kv, 9)
        hkv, d, total = 1, 64, sum(nq)
        k, v = normal(gen, (total, hkv, d), torch.bfloat16), normal(gen, (total, hkv, d), torch.bfloat16)
        pools = [pool_of(blocks, hkv, d, dtype, False) for _ in range(2)]
        scales = {n: torch.full((blocks, hkv), 2.0 ** -6, device=DEV) for n in ("k_scale", "v_scale")} if dtype is E4M3 else {}
        paged.extend(k, v, *pools, table, i32(slot), i32(starts_of(nq)), i32(kv), **scales)
        host = table.cpu()
        slots = torch.tensor([int(host[slot[b], p // 128]) * 128 + p % 128 for b, (n, m) in enumerate(zip(nq, kv)) for p in range(m - n, m)], device=DEV).long()
        for x, p, name in ((k, pools[0], "k_scale"), (v, pools[1], "v_scale")):
            got = p.view(torch.uint8).view(p.dtype).view(-1, hkv, d)[slots] if dtype is not E4M3 else values8(p, scales[name]).view(-1, hkv, d)[slots]
            if dtype is E4M3:
                s = scales[name].double()[slots // 128][..., None]
                assert bool(((got - x.double()).abs() <= s * ref.half_step8(x.double() / s)).all())
            else:
                assert torch.equal(got, x.to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 4), (64, 20, 3), (256, 4, 2)])
def test_extend_of_long_prompts(dtype, d, hq, hkv):
    """Prompts whose queries take a launch of their own: what one call writes is what rotation, a call without queries and the
    token's round trip say."""
    nq = [(9 << 20) // (hq * d) - 200, 150, 1]
    kv = [nq[0], 400, 129]
    gen = torch.Generator().manual_seed(d)
    rows = sum(nq) + 3
    q, k, v = (normal(gen, (rows, h, d), dtype) for h in (hq, hkv, hkv))
    table, slot, blocks = place_requests(nq, kv, 1)
    args = (table, i32(slot), i32(starts_of(nq)), i32(kv))
    r, at = paged.Rotary(d, base=500000.0), torch.cat([torch.arange(m - n, m) for n, m in zip(nq, kv)]).to(torch.int32).to(DEV)
    results = []
    for queries in (q, None):
        pools = [torch.zeros(blocks, 128, hkv, d, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
        scales = [torch.ones(blocks, hkv, device=DEV) for _ in range(2)]
        out = None if queries is None else torch.full_like(q, 5.0)
        paged.extend(k, v, *pools, *args, rotary=r, q=queries, q_out=out, k_scale=scales[0], v_scale=scales[1])
        if out is not None:
            assert torch.equal(out[:sum(nq)], paged.rotate(q[:sum(nq)], at, r)) and bool((out[sum(nq):] == 5.0).all())
        results.append(pools + scales)
    assert all(same(a, b) for a, b in zip(*results))
    host = table.cpu()
    slots = torch.tensor([int(host[slot[b], p // 128]) * 128 + p % 128 for b, (n, m) in enumerate(zip(nq, kv)) for p in range(m - n, m)], device=DEV).long()
    want, size = ref.rotate(k[:sum(nq)], at, r.steps, r.times, False)
    error = ref.rotation_error(size, at, r.steps)
    for x, pool, scale, e in ((want, results[0][0], results[0][2], error), (v[:sum(nq)].double(), results[0][1], results[0][3], 0.0 * error)):
        s = scale.double()[slots // 128][..., None]
        got = values8(pool, scale).view(-1, hkv, d)[slots]
        assert bool(((got - x).abs() <= s * ref.half_step8((x.abs() + e) / s) + e).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
def test_extend_refusals(dtype):
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    pools = [pool_of(2, 2, 64, dtype, False) for _ in range(2)]
    scales = {"k_scale": torch.ones(2, 2, device=DEV), "v_scale": torch.ones(2, 2, device=DEV)} if dtype is E4M3 else {}
    good = dict(k=k, v=k, k_pool=pools[0], v_pool=pools[1], table=i32([[0, 1]]), seq_ids=i32([0]), starts=i32([0, 2]), totals=i32([2]), **scales)
    paged.extend(**good)
    r = paged.Rotary(64)
    worse = [{"k": k[:1]}, {"k": k.float()}, {"k": k[..., :32]}, {"k": k.transpose(1, 2)}, {"starts": i32([])}, {"totals": i32([])}, {"seq_ids": i32([])}, {"q": k},
             {"rotary": r, "q": k.half()}, {"rotary": r, "q": k[:1]}, {"rotary": r, "q": k, "q_out": k[:1]}, {"rotary": r, "q_out": k}, {"positions": i32([1, 2])},
             {"rotary": r, "positions": i32([1])}, {"rotary": paged.Rotary(64, device="cpu")}, {"table": i32([0, 1])}]
    worse += [{"k_scale": None}, {"v_scale": scales["v_scale"][:1]}, {"v_scale": scales["v_scale"].double()}, {"k_scale": None, "v_scale": None}] if scales else [
        {"k_scale": torch.ones(2, 2, device=DEV), "v_scale": torch.ones(2, 2, device=DEV)}]
    for over in worse:
        with pytest.raises(ValueError):
            paged.extend(**{**good, **over})
    with pytest.raises(RuntimeError):
        paged.extend(**{**good, "rotary": paged.Rotary(128)})
    if scales:
        with pytest.raises(RuntimeError):
            paged.extend(**{**good, "k_pool": torch.zeros(2, 128, 2, 72, dtype=torch.uint8, device=DEV).view(E4M3)[..., :64]})
        cache = paged.PagedCache(1, paged.BlockPool(2, 1, 256), 2, 64, dtype=E4M3)
        with pytest.raises(ValueError):
            cache.append(0, k, k, i32([0, 1]))


# ---- attention over 8 bits ----

def attend_inputs(nq, kv, hq, hkv, d, dtype, heads_first, seed, tail=0, loud=1.0):
    g = torch.Generator().manual_seed(seed)
    table, slot, blocks = place_requests(nq, kv, seed + 1)
    k, v = (torch.randn((blocks, 128, hkv, d), generator=g) for _ in range(2))
    k[..., :2] *= 3.0
    out = []
    for x in (k, v):
        x *= torch.exp2((torch.rand((blocks, 1, hkv, 1), generator=g) * 2 - 1) * loud)
        s = torch.tensor([[ref.scale_of(t) for t in row] for row in x.abs().amax((1, 3)).tolist()])
        p = (x / s[:, None, :, None]).clamp(-448.0, 448.0).to(E4M3)
        raw = p.view(torch.uint8).to(DEV)
        for b, m in enumerate(kv):  # what stands behind a sequence is not a number
            if m % 128:
                raw[table[slot[b], m // 128].item(), m % 128:] = 0x7f
        raw = raw.transpose(1, 2).contiguous().transpose(1, 2) if heads_first else raw
        out += [raw.view(E4M3), s.to(DEV)]
    q = torch.randn((sum(nq) + tail, hq, d), generator=g).to(dtype).to(DEV)
    return q, out[0], out[1], out[2], out[3], table, slot


def check_attended(out, q, k, ks, v, vs, table, slot, nq, kv, causal=True, scale=None):
    starts, host = starts_of(nq), table.cpu()
    scale = scale or q.shape[2] ** -0.5
    for b, (n, m) in enumerate(zip(nq, kv)):
        if not n:
            continue
        ids = host[slot[b], :-(-m // 128)].tolist()
        gather = lambda p: torch.cat([p.view(torch.uint8)[i] for i in ids] or [p.view(torch.uint8)[0, :0]]).view(E4M3).float().double()[:m]  # noqa: E731
        per = lambda s: torch.cat([s[i][None].expand(128, -1) for i in ids] or [s[:0]])[:m]  # noqa: E731
        rows = slice(starts[b], starts[b + 1])
        vis = [max(0, m - n + i + 1) if causal else m for i in range(n)]
        want, bound = ref.attention8(q[rows], gather(k), per(ks), gather(v), per(vs), vis, scale)
        got = out[rows].double()
        assert bool(((got - want).abs() <= bound).all()), (b, n, m, ((got - want).abs() / bound).max().item())


ATTEND = [
    ([1], [1]), ([1], [128]), ([1, 1, 1], [129, 0, 64]), ([1, 0, 1, 1], [1000, 50, 127, 65]), ([4, 1, 3], [4, 700, 130]), ([16, 2], [300, 5]),
    ([40], [40]), ([100, 1, 33], [500, 130, 33]), ([257], [900]), ([5, 200], [3, 150]),
]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [(1, 1), (8, 2), (6, 2), (5, 1)])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention_over_8_bits(dtype, d, heads, case):
    nq, kv = ATTEND[case]
    hq, hkv = heads
    q, k, ks, v, vs, table, slot = attend_inputs(nq, kv, hq, hkv, d, dtype, case % 2 == 1, case * 10 + d, tail=3)
    out, status = torch.full_like(q, 5.0), i32([0])
    hints = {"max_q": max(nq), "max_kv": max(kv)} if case % 3 else {}
    got = paged.attention(q, k, v, table, i32(slot), i32(starts_of(nq)), i32(kv), out=out, status=status, k_scale=ks, v_scale=vs, **hints)
    assert got is out and status.item() == 0 and bool((out[sum(nq):] == 5.0).all())
    check_attended(out, q, k, ks, v, vs, table, slot, nq, kv)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,nq,kv", [((8, 2), [9], [9]), ((6, 2), [11, 0, 40], [700, 0, 131]), ((5, 1), [100, 1], [257, 2000]), ((32, 1), [2, 3], [1, 3]),
                                         ((1, 1), [200, 33], [300, 33]), ((4, 4), [65], [1500]), ((8, 1), [128], [128]), ((2, 1), [17, 64], [6000, 64])])
@pytest.mark.parametrize("causal", [True, False])
def test_short_work_with_and_without_hints(dtype, d, heads, nq, kv, causal):
    """The most tokens of a request, where it is known, choose the kernel: either one has to be right, in either's workspace."""
    hq, hkv = heads
    q, k, ks, v, vs, table, slot = attend_inputs(nq, kv, hq, hkv, d, dtype, causal, d + hq + len(nq), tail=2)
    room = torch.empty(paged.attention_workspace_bytes(q, k, max_q=max(nq), batch=len(nq)), dtype=torch.uint8, device=DEV)
    least = paged.attention_workspace_bytes(q, k, max_q=max(nq), max_kv=max(kv), batch=len(nq))
    assert least <= room.numel()
    assert paged.attention_workspace_bytes(q, k, max_q=max(nq), max_kv=2 ** 31 - 1, batch=len(nq)) == room.numel()  # as if it were unknown
    for hints, ws in [({}, room), ({"max_kv": max(kv)}, room), ({"max_kv": max(kv)}, room[:least]), ({"max_kv": 1 << 20}, room)]:
        out, status = torch.full_like(q, 5.0), i32([0])
        paged.attention(q, k, v, table, i32(slot), i32(starts_of(nq)), i32(kv), causal=causal, max_q=max(nq), out=out, workspace=ws, status=status,
                        k_scale=ks, v_scale=vs, **hints)
        assert status.item() == 0 and bool((out[sum(nq):] == 5.0).all())
        check_attended(out, q, k, ks, v, vs, table, slot, nq, kv, causal)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("d,nq,kv", [(128, [1], [20000]), (64, [2], [9000]), (256, [1], [5000]), (128, [70], [6000]), (256, [130], [3000]), (64, [300], [4000])])
def test_attention_over_8_bits_of_split_sequences(dtype, d, nq, kv):
    q, k, ks, v, vs, table, slot = attend_inputs(nq, kv, 8, 2, d, dtype, False, 77)
    out = paged.attention(q, k, v, table, i32(slot), i32(starts_of(nq)), i32(kv), k_scale=ks, v_scale=vs)
    check_attended(out, q, k, ks, v, vs, table, slot, nq, kv)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("nq", [1, 3, 60])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales_far_apart(dtype, nq, d):
    """Pages whose values differ by up to 2^80: the weights' 16 bits hold what the result needs."""
    q, k, ks, v, vs, table, slot = attend_inputs([nq], [700], 4, 1, d, dtype, False, 5)
    gen = torch.Generator().manual_seed(1)
    vs = torch.exp2(torch.randint(-60 if dtype == torch.bfloat16 else -30, 20 if dtype == torch.bfloat16 else 5, vs.shape, generator=gen).float()).to(DEV)
    ks = ks * torch.exp2(torch.randint(-20, 1, ks.shape, generator=gen).float()).to(DEV)
    out = paged.attention(q, k, v, table, i32(slot), i32([0, nq]), i32([700]), k_scale=ks, v_scale=vs)
    check_attended(out, q, k, ks, v, vs, table, slot, [nq], [700])
    vs = torch.flip(vs, [0]) * 1.25  # scales of the caller's need not be powers of two
    out = paged.attention(q, k, v, table, i32(slot), i32([0, nq]), i32([700]), k_scale=ks, v_scale=vs)
    check_attended(out, q, k, ks, v, vs, table, slot, [nq], [700])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 50])
def test_queries_of_any_size(d, n):
    """bf16 rows from 2^-120 to 2^100, a row of zeros among them."""
    q, k, ks, v, vs, table, slot = attend_inputs([n], [300], 4, 2, d, torch.bfloat16, False, 6)
    gen = torch.Generator().manual_seed(2)
    q = (q.float() * torch.exp2(torch.randint(-120, 100, q.shape[:2] + (1,), generator=gen).float()).to(DEV)).to(torch.bfloat16)
    q[0, 1] = 0.0
    for scale in (2.0 ** -90, 1.0):
        out = paged.attention(q, k, v, table, i32(slot), i32([0, n]), i32([300]), softmax_scale=scale, k_scale=ks, v_scale=vs)
        assert bool(out.isfinite().all())
        mild = [i for i in range(4) if float(q[:, i].float().abs().max()) * scale < 4.0]
        for i in range(n):
            for h in range(4):
                if float(q[i, h].float().abs().max()) * scale < 4.0:
                    one = q[i:i + 1, h:h + 1].contiguous()
                    kk, vv = (x.view(torch.uint8)[:, :, h // 2:h // 2 + 1].contiguous().view(E4M3) for x in (k, v))
                    check_attended(out[i:i + 1, h:h + 1], one, kk, ks[:, h // 2:h // 2 + 1], vv, vs[:, h // 2:h // 2 + 1], table, slot, [1], [300 - n + i + 1], scale=scale)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("size,sign", [(2.0 ** 12, 1), (2.0 ** 12, -1), (2.0 ** 15, 1)])
def test_scores_far_from_zero_pick_one_token(dtype, d, n, size, sign):
    """Scores around 2^20 to 2^40, of which one is the largest by far, over pages whose values' scales are far apart: the result is that
    token's values, exact but for the result's rounding."""
    m, hkv = 700, 2
    table, slot, blocks = place_requests([n], [m], 3)
    gen = torch.Generator().manual_seed(d + n)
    k = torch.full((blocks, 128, hkv, d), 256.0)
    pick = 200
    k[int(table[slot[0], pick // 128]), pick % 128] = 256.0 + 32.0 * sign  # the neighbouring number of e4m3
    k = k.to(E4M3).to(DEV)
    v = torch.randn((blocks, 128, hkv, d), generator=gen).to(E4M3).to(DEV)
    ks = torch.full((blocks, hkv), 2.0 ** 4, device=DEV)
    most = 40 if dtype == torch.bfloat16 else 5
    vs = torch.exp2(torch.randint(-most, most, (blocks, hkv), generator=gen).float()).to(DEV)
    q = torch.full((n, 4, d), size * sign, dtype=dtype, device=DEV)
    for scale in (1.0, 2.0 ** -6):
        out = paged.attention(q, k, v, table, i32(slot), i32([0, n]), i32([m]), softmax_scale=scale, k_scale=ks, v_scale=vs)
        block = int(table[slot[0], pick // 128])
        want = (v[block, pick % 128].float().double() * vs[block].double()[:, None]).repeat_interleave(2, 0)[None].expand(n, 4, d)
        assert bool(((out.double() - want).abs() <= ref.rounding(want, dtype) + want.abs() * 2.0 ** -20).all())


def test_attention_over_8_bits_options():
    nq, kv = [3, 50], [200, 260]
    for nq in ([3, 1], [3, 50]):
        q, k, ks, v, vs, table, slot = attend_inputs(nq, kv, 6, 3, 128, torch.float16, True, 8)
        args = (i32(slot), i32(starts_of(nq)), i32(kv))
        out = paged.attention(q, k, v, table, *args, causal=False, softmax_scale=0.3, k_scale=ks, v_scale=vs)
        check_attended(out, q, k, ks, v, vs, table, slot, nq, kv, causal=False, scale=0.3)
        wide = torch.zeros(q.shape[0], 9, 128, dtype=q.dtype, device=DEV)
        ws = torch.empty(paged.attention_workspace_bytes(q, k, batch=2), dtype=torch.uint8, device=DEV)
        paged.attention(q, k, v, table, *args, out=wide[:, 2:8], workspace=ws, k_scale=ks, v_scale=vs)
        check_attended(wide[:, 2:8], q, k, ks, v, vs, table, slot, nq, kv)
        assert bool((wide[:, :2] == 0).all()) and bool((wide[:, 8:] == 0).all())
        same_place = q.clone()
        assert torch.equal(paged.attention(same_place, k, v, table, *args, out=same_place, k_scale=ks, v_scale=vs), wide[:, 2:8])


@pytest.mark.parametrize("n", [1, 40])
def test_attention_over_8_bits_reports_bad_arrays(n):
    q, k, ks, v, vs, table, slot = attend_inputs([n, n], [200, 100], 2, 1, 64, torch.bfloat16, False, 9)
    word = i32([0])

    def run(ids=slot, starts=(0, n, 2 * n), lens=(200, 100), tab=table):
        word.zero_()
        out = paged.attention(q, k, v, tab, i32(list(ids)), i32(list(starts)), i32(list(lens)), status=word, out=torch.full_like(q, 3.0), max_q=n, k_scale=ks, v_scale=vs)
        return word.item(), out

    assert run()[0] == 0
    assert run(ids=[99, slot[1]])[0] == paged.TQ_DEV_ERR_SEQ_ID and bool((run(ids=[99, slot[1]])[1][:n] == 0).all())
    assert run(lens=[10 ** 9, 100])[0] == paged.TQ_DEV_ERR_LENGTH and run(starts=(0, n, 5 * n))[0] == paged.TQ_DEV_ERR_LENGTH
    holes = table.clone()
    holes[slot[0], 1] = -1
    st, out = run(tab=holes)
    assert st == paged.TQ_DEV_ERR_BLOCK and bool(out.isfinite().all())


def test_attention_over_8_bits_refusals():
    q, k, ks, v, vs, table, slot = attend_inputs([1], [200], 2, 1, 64, torch.bfloat16, False, 9)
    args = (i32(slot), i32([0, 1]), i32([200]))
    for over in [{"k_scale": None}, {"v_scale": None}, {"k_scale": None, "v_scale": None}, {"k_scale": ks[:1]}, {"v_scale": vs.half()}, {"q": q.float()}, {"k_pool": k.view(torch.uint8)}]:
        with pytest.raises(ValueError):
            paged.attention(**{"q": q, "k_pool": k, "v_pool": v, "table": table, "seq_ids": args[0], "q_starts": args[1], "kv_lens": args[2], "k_scale": ks, "v_scale": vs, **over})


# ---- together ----

def kept_values(cache, layer, which, ids, n):
    x = cache.kv[layer, which][ids].float().double() if cache.scales is None else values8(cache.kv[layer, which], cache.scales[layer, which])[ids]
    return x.flatten(0, 1)[:n]


@pytest.mark.parametrize("dtype,qtype", [(E4M3, torch.bfloat16), (E4M3, torch.float16), (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("d", [64, 128])
def test_serving_steps(dtype, qtype, d):
    """Prompts, steps, a rejected draft and a finished request: map, extend and attention as a serving loop runs them, each
    attention against what the cache holds, the cache against the rotated rows."""
    hq, hkv, layers = 4, 2, 2
    pool = paged.BlockPool(24, 4, 1024)
    cache = paged.PagedCache(layers, pool, hkv, d, dtype=dtype)
    r = paged.Rotary(d, base=500000.0, scaling="bands", factor=8.0, first=256)
    gen = torch.Generator().manual_seed(4)
    held = {}
    for step, (ids, new) in enumerate([([0, 2], [130, 50]), ([0, 2, 3], [1, 1, 200]), ([3, 0, 2], [1, 5, 1]), ([2, 0, 3], [1, 1, 1]), ([1, 0], [300, 1])]):
        lens = [len(held.get(i, [])) for i in ids]
        rows = sum(new)
        slots, starts, totals = pool.map(i32(ids), i32(lens), i32(new), rows)
        for layer in range(layers):
            qkv = normal(gen, (rows, hq + 2 * hkv, d), qtype)
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            turned = cache.extend(layer, k, v, i32(ids), starts, totals, rotary=r, q=q)
            out = cache.attention(layer, turned, i32(ids), starts, totals, max_q=max(new))
            row = 0
            for i, n, had in zip(ids, new, lens):
                at = torch.arange(had, had + n, device=DEV)
                ks, _ = ref.rotate(k[row:row + n], at, r.steps, r.times, False)
                if layer == 0:
                    held.setdefault(i, []).extend(zip(ks, v[row:row + n].double()))
                    m = had + n
                    table = pool.table[i].tolist()
                    blocks = torch.tensor(table[:-(-m // 128)], device=DEV)
                    kk, vv = kept_values(cache, 0, 0, blocks, m), kept_values(cache, 0, 1, blocks, m)
                    for got, j in ((kk, 0), (vv, 1)):
                        want = torch.stack([t[j] for t in held[i]])
                        if dtype is E4M3:  # a step of the block's last scale for each element, at most
                            s = torch.repeat_interleave(cache.scales[0, j][blocks], 128, 0)[:m, :, None].double()
                            assert bool(((got - want).abs() <= s * 2 * ref.half_step8((want / s).clamp(-448, 448)) * (1 + 2.0 ** -10)).all())
                        else:
                            assert bool(((got - want).abs() <= want.abs() * 2.0 ** -8 + 2.0 ** -20).all())
                    vis = [had + x + 1 for x in range(n)]
                    if dtype is E4M3:
                        one = torch.ones(m, hkv, device=DEV)
                        numbers = [cache.kv[0, j].view(torch.uint8)[blocks].flatten(0, 1)[:m].view(E4M3).float() for j in (0, 1)]
                        per = [torch.repeat_interleave(cache.scales[0, j][blocks], 128, 0)[:m] for j in (0, 1)]
                        want, bound = ref.attention8(turned[row:row + n], numbers[0], per[0] * one, numbers[1], per[1] * one, vis, d ** -0.5)
                    else:
                        want, bound = paged_reference.attention(turned[row:row + n], kk, vv, vis, d ** -0.5)
                    assert bool(((out[row:row + n].double() - want).abs() <= bound).all())
                row += n
        if step == 2:  # four of request 0's five tokens were wrong guesses
            held[0] = held[0][:-4]
            pool.release(i32([0]), keep=i32([len(held[0])]))
        if step == 3:
            pool.release(i32([2, 3]))
            del held[2], held[3]
    assert pool.check_status() == 0


@pytest.mark.parametrize("dtype", [E4M3, torch.bfloat16])
def test_a_captured_step_replays(dtype):
    hq, hkv, d, batch = 8, 2, 128, 3
    pool = paged.BlockPool(40, batch, 1024)
    cache = paged.PagedCache(1, pool, hkv, d, dtype=dtype)
    cache.kv.view(torch.uint8).zero_()
    r = paged.Rotary(d)
    ids, lens, new = i32([2, 0, 1]), i32([0, 0, 0]), i32([0, 0, 0])
    qkv = torch.zeros(8, hq + 2 * hkv, d, dtype=torch.bfloat16, device=DEV)

    def step():
        _, starts, totals = pool.map(ids, lens, new, 8)
        q = cache.extend(0, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], ids, starts, totals, rotary=r, q=qkv[:, :hq])
        return q, cache.attention(0, q, ids, starts, totals, max_q=8), totals

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, out, totals = step()
    gen = torch.Generator().manual_seed(5)
    counts = [[3, 4, 1], [1, 1, 1], [0, 5, 2], [1, 1, 1]]
    eager_pool = paged.BlockPool(40, batch, 1024)
    eager = paged.PagedCache(1, eager_pool, hkv, d, dtype=dtype)
    eager.kv.view(torch.uint8).zero_()
    had = [0, 0, 0]
    for n in counts:
        qkv.copy_(torch.randn(qkv.shape, generator=gen))
        lens.copy_(i32(had))
        new.copy_(i32(n))
        graph.replay()
        _, starts, want_totals = eager_pool.map(ids, lens, new, 8)
        q2 = eager.extend(0, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], ids, starts, want_totals, rotary=r, q=qkv[:, :hq])
        out2 = eager.attention(0, q2, ids, starts, want_totals, max_q=8)
        rows = sum(n)
        assert torch.equal(totals, want_totals) and torch.equal(q[:rows], q2[:rows]) and torch.equal(out[:rows], out2[:rows])
        assert torch.equal(cache.kv.view(torch.uint8), eager.kv.view(torch.uint8))
        had = [h + x for h, x in zip(had, n)]
    assert pool.check_status() == 0


def test_calls_on_another_stream():
    q, k, ks, v, vs, table, slot = attend_inputs([2, 40], [300, 200], 4, 2, 64, torch.bfloat16, False, 10)
    args = (table, i32(slot), i32([0, 2, 42]), i32([300, 200]))
    want = paged.attention(q, k, v, *args, k_scale=ks, v_scale=vs)
    r = paged.Rotary(64)
    at = torch.arange(42, dtype=torch.int32, device=DEV)
    turned = paged.rotate(q, at, r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = paged.attention(q, k, v, *args, k_scale=ks, v_scale=vs, stream=side)
    other = paged.rotate(q, at, r, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(turned, other)
    pools = [[x.view(torch.uint8).clone().view(E4M3) for x in (k, v)] for _ in range(2)]
    scale = [[ks.clone(), vs.clone()] for _ in range(2)]
    torch.cuda.synchronize()
    new = normal(torch.Generator().manual_seed(1), (42, 2, 64), torch.bfloat16)
    torch.cuda.synchronize()
    for p, s, stream in ((pools[0], scale[0], None), (pools[1], scale[1], side)):
        paged.extend(new, new, *p, *args, rotary=r, k_scale=s[0], v_scale=s[1], stream=stream)
        torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(*pools)) and all(torch.equal(a, b) for a, b in zip(*scale))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,nq,kv", [((8, 2), [1, 1, 1], [3000, 100, 900]), ((8, 2), [33, 33, 33], [3000, 100, 900]), ((6, 2), [257], [900]),
                                         ((8, 2), [256], [1024]), ((6, 2), [100, 1, 33], [500, 130, 33])])
def test_results_repeat_bit_for_bit(d, heads, nq, kv):
    """Tiles cut between CTAs at many places, whose loads, conversions and products run ahead of one another differently each time."""
    q, k, ks, v, vs, table, slot = attend_inputs(nq, kv, *heads, d, torch.bfloat16, False, 30)
    args = (table, i32(slot), i32(starts_of(nq)), i32(kv))
    first = paged.attention(q, k, v, *args, k_scale=ks, v_scale=vs)
    check_attended(first, q, k, ks, v, vs, table, slot, nq, kv)
    differ = sum(not torch.equal(first, paged.attention(q, k, v, *args, k_scale=ks, v_scale=vs)) for _ in range(300))
    assert differ == 0


def test_offsets_past_32_bits():
    """Pools of 5.4 GB, whose blocks' places pass 32 bits: the last blocks hold the request."""
    blocks, hkv, d = 41000, 8, 128
    pools = [torch.zeros(blocks, 128, hkv, d, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
    scales = [torch.ones(blocks, hkv, device=DEV) for _ in range(2)]
    table = i32([[blocks - 1, 3, blocks - 2]])
    gen = torch.Generator().manual_seed(6)
    k, v, q = normal(gen, (300, hkv, d), torch.bfloat16), normal(gen, (300, hkv, d), torch.bfloat16), normal(gen, (300, hkv, d), torch.bfloat16)
    paged.extend(k, v, *pools, table, None, i32([0, 300]), i32([300]), k_scale=scales[0], v_scale=scales[1])
    for lo, block in ((0, blocks - 1), (128, 3), (256, blocks - 2)):
        hi = min(300, lo + 128)
        s = scales[1][block].double()[:, None]
        got = pools[1][block, :hi - lo].float().double() * s
        assert bool(((got - v[lo:hi].double()).abs() <= s * ref.half_step8(v[lo:hi].double() / s)).all())
    for n in (1, 300):
        out = paged.attention(q[:n], *pools, table, None, i32([0, n]), i32([300]), k_scale=scales[0], v_scale=scales[1])
        check_attended(out, q[:n], pools[0], scales[0], pools[1], scales[1], table, [0], [n], [300])
