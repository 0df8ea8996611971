"""GPU tests of rotary positions, rotated appends and the paged cache of 8 bits at the edges of what they take, against plain 64-bit references."""
import math

import pytest
import torch

from kv_cache_quantization_quantize_gb300 import paged
from tests import extend_reference as ref
from tests import paged_reference
from tests.test_gpu_extend import attend_inputs, check_attended, normal, place_requests, run_extend8, same, starts_of

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


def codes(x):
    return x.to(E4M3).to(DEV)


# ---- attention over 8 bits: weights far below a row's largest, scales at the ends of their range ----

def attend_shared(q, k, v, ks, vs, batch, m, scale, word=None):
    """q [n, hq, d] of each of `batch` requests, all on one sequence (so that few parts of it go to the join). Returns
    [batch, n, hq, d]."""
    n = q.shape[0]
    table = torch.arange(k.shape[0], dtype=torch.int32, device=DEV)[None]
    many = q[None].expand(batch, -1, -1, -1).reshape(batch * n, *q.shape[1:]).contiguous()
    out = paged.attention(many, k, v, table, torch.zeros(batch, dtype=torch.int32, device=DEV), torch.arange(0, (batch + 1) * n, n, dtype=torch.int32, device=DEV),
                          torch.full((batch,), m, dtype=torch.int32, device=DEV), causal=False, softmax_scale=scale, max_q=n, max_kv=m, status=word,
                          **({} if ks is None else {"k_scale": ks, "v_scale": vs}))
    return out.view(batch, *q.shape)


def sink(m, d, hkv, below):
    """Numbers of K and V of m tokens in pages: the first token's key scores `below` log2 above all others with a query of ones and the
    returned softmax scale; its value is 0, the others' are positive."""
    pages, gen = -(-m // 128), torch.Generator().manual_seed(m + d)
    k, v = torch.zeros(pages * 128, hkv, d), torch.randint(1, 9, (pages * 128, hkv, d), generator=gen) / 4
    k[0], v[0] = 1.0, 0.0
    return k.view(pages, 128, hkv, d), v.view(pages, 128, hkv, d), below * math.log(2.0) / d


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,batch", [(1, 640), (6, 640), (40, 320)])
def test_small_weights_beside_a_sink_are_kept_over_8_bits(dtype, d, n, batch):
    """A first token that takes nearly all of the weight and has no value, before 32767 others: the result is the others' alone.

    Weights are rounded to f16 as p = 2^(s - m + 7) with m at most the row's maximum: relative to 2^7 by 2^-11, or by half of f16's
    least step, 2^-25 / 2^7, below 2^-14 / 2^7. So a result is off by 2^-11 of the sum of w |v| and 2^-32 of that of |v|, over that of w,
    beside its own rounding; scores are 0 and `below` exactly, and fp32 sums of 2048 steps, of weights and of products, add 2^-13 each."""
    m, below = 32768, 25.5
    k, v, scale = sink(m, d, 1, below)
    one = torch.ones(k.shape[0], 1, device=DEV)
    out = attend_shared(torch.ones(n, 4, d, dtype=dtype, device=DEV), codes(k), codes(v), one, one, batch, m, scale)
    w, total = 2.0 ** -below, 1.0 + (m - 1) * 2.0 ** -below
    mass = v.double().sum((0, 1, 2)).to(DEV) / total  # of |v|
    want = w * mass
    bound = want * (torch.finfo(dtype).eps / 2 + 2.0 ** -11 + 2.0 ** -12) + 2.0 ** -32 * mass + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    assert bool(((out.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,batch", [(1, 640), (6, 640), (40, 320)])
def test_small_weights_beside_a_sink_are_kept_over_f16(d, n, batch):
    """The same over the exact cache in f16, whose weights are f16 too."""
    m, below = 32768, 25.5
    k, v, scale = sink(m, d, 1, below)
    out = attend_shared(torch.ones(n, 4, d, dtype=torch.float16, device=DEV), k.half().to(DEV), v.half().to(DEV), None, None, batch, m, scale)
    w, total = 2.0 ** -below, 1.0 + (m - 1) * 2.0 ** -below
    mass = v.double().sum((0, 1, 2)).to(DEV) / total
    bound = w * mass * (2.0 ** -11 + 2.0 ** -11 + 2.0 ** -12) + 2.0 ** -32 * mass + 2.0 ** -25
    assert bool(((out.double() - w * mass).abs() <= bound).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 6, 40])
@pytest.mark.parametrize("m", [70, 9000])
def test_results_past_f16_are_infinite(d, n, m):
    """All values of a request the same: the result is that, infinite where f16 has no number for it, and its largest number where
    only rounded weights carry a result past it."""
    pages, gen = -(-m // 128), torch.Generator().manual_seed(d + n)
    k, q = codes(torch.randn((pages, 128, 2, d), generator=gen)), torch.randn((n, 4, d), generator=gen).half().to(DEV)
    v, one = codes(torch.full((pages, 128, 2, d), 448.0)), torch.ones(pages, 2, device=DEV)
    v.view(torch.uint8)[..., 1::2] = 0xFE  # -448
    sign = torch.ones(d, device=DEV, dtype=torch.float64)
    sign[1::2] = -1.0
    args = (torch.arange(pages, dtype=torch.int32, device=DEV)[None], None, i32([0, n]), i32([m]))
    for scale in (2.0 ** 8, 2.0 ** 60):  # 114688 and more
        out = paged.attention(q, k, v, *args, causal=False, k_scale=one, v_scale=one * scale)
        assert torch.equal(out.double(), (sign * math.inf).expand(n, 4, d))
    out = paged.attention(q, k, v, *args, causal=False, k_scale=one, v_scale=one * (65504.0 / 448.0))
    assert bool(out.isfinite().all()) and bool(((out.double() - sign * 65504.0).abs() <= 65504.0 * 2.0 ** -10).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,batch", [(1, 640), (6, 640), (40, 320), (1, 1), (40, 1)])
def test_a_page_of_small_values_counts_beside_one_of_large_ones(d, n, batch):
    """Scales 2^60 and 2^-60, the ends of their range: the tokens of the small one have 2^-9 of the others' weight each, and
    together more than half of all."""
    m, ratio = 128 * 400, 2.0 ** -9
    k, v = torch.zeros(400, 128, 1, d), torch.full((400, 128, 1, d), 2.0)
    k[0] = 1.0
    vs = torch.full((400, 1), 2.0 ** -60, device=DEV)
    vs[0] = 2.0 ** 60
    out = attend_shared(torch.ones(n, 4, d, dtype=torch.bfloat16, device=DEV), codes(k), codes(v), torch.ones_like(vs), vs, batch, m, 9.0 * math.log(2.0) / d)
    want = 2.0 ** 61 / (1.0 + 399 * ratio)  # the small values themselves are far below half a step of that
    # the result's and a weight's rounding, fp32 sums of 3200 steps
    assert bool(((out.double() / want - 1.0).abs() <= 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -11).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,batch", [(1, 1), (6, 3), (40, 1), (1, 640), (40, 320)])
def test_a_page_of_large_values_and_no_weight(d, n, batch):
    """The first page's scale is 2^60 and all others' 2^-60, but these have 2^125 of its weight for each token: their values are the
    result, with what the first's add."""
    m, below = 128 * 200, 125.0
    k, v = torch.zeros(200, 128, 1, d), torch.full((200, 128, 1, d), 3.0)
    k[1:] = 1.0
    vs = torch.full((200, 1), 2.0 ** -60, device=DEV)
    vs[0] = 2.0 ** 60
    out = attend_shared(torch.ones(n, 4, d, dtype=torch.bfloat16, device=DEV), codes(k), codes(v), torch.ones_like(vs), vs, batch, m, below * math.log(2.0) / d)
    want = 3.0 * 2.0 ** -60 + 3.0 * 2.0 ** (60 - below) / 199
    # beside both roundings: scores up to 87 from fp32 sums of d products, off by (d + 8) 2^-24 of that, and fp32 sums of 1600 steps
    assert bool(((out.double() / want - 1.0).abs() <= 2.0 ** -8 + 2.0 ** -11 + 2 * (d + 8) * 2.0 ** -24 * 87 + 2.0 ** -12).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,m", [(1, 700), (3, 9000), (8, 700), (60, 900), (200, 5000)])
@pytest.mark.parametrize("loud", [1.0, 40.0])
def test_scales_over_their_whole_range(d, n, m, loud):
    """Each page's scale of values anywhere from 2^-60 to 2^60; with loud queries scores up to some 2^8 beside them."""
    q, k, ks, v, vs, table, slot = attend_inputs([n, n], [m, m - 129], 8, 2, d, torch.bfloat16, False, 50 + n)
    for seed in range(4):
        gen = torch.Generator().manual_seed(seed)
        vs = torch.exp2(torch.randint(-60, 61, vs.shape, generator=gen).float()).to(DEV)
        if seed == 3:  # the two ends alone
            vs = torch.where(torch.rand(vs.shape, generator=gen).to(DEV) < 0.5, 2.0 ** 60, 2.0 ** -60)
        out = paged.attention(q * loud, k, v, table, i32(slot), i32([0, n, 2 * n]), i32([m, m - 129]), max_q=n, k_scale=ks, v_scale=vs)
        check_attended(out, q * loud, k, ks, v, vs, table, slot, [n, n], [m, m - 129])


FAR = [2.0 ** 23 - 3, 2.0 ** 24 - 14, 2.0 ** 24 - 9, 2.0 ** 24 - 6, 2.0 ** 24 - 4, 2.0 ** 24 - 2, 2.0 ** 24, 2.0 ** 24 + 4]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,batch", [(1, 640), (40, 320)])
@pytest.mark.parametrize("sign", [-1, 1])
def test_weights_stay_in_f16_at_far_scores_over_8_bits(dtype, d, n, batch, sign):
    """Scores of +-2^23 to 2^24 (log2) where fp32 has steps of 1 and 2, of which later pages' are 6 to 8 above the first's, just below what moves
    the reference: weights are at their largest. Steps of 2 leave the later pages 2^4 of the first's weight at least."""
    k, v = torch.ones(6, 128, 1, d), torch.full((6, 128, 1, d), 2.0)
    v[0] = 1.0
    for far in FAR:
        for above in (6.0, 7.0, 8.0):
            ks, vs = torch.full((6, 1), 1.0 + sign * above / far, device=DEV), torch.ones(6, 1, device=DEV)
            ks[0] = 1.0
            out = attend_shared(torch.full((n, 4, d), float(sign), dtype=dtype, device=DEV), codes(k), codes(v), ks, vs, batch, 768, far * math.log(2.0) / d)
            assert bool((out >= 1.9).all()) and bool((out <= 2.0).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,batch", [(1, 640), (40, 320)])
@pytest.mark.parametrize("sign", [-1, 1])
def test_weights_stay_in_f16_at_far_scores_over_f16(d, n, batch, sign):
    """The same over the exact cache in f16."""
    v = torch.full((6, 128, 1, d), 2.0)
    v[0] = 1.0
    for far in FAR:
        for above in (6.0, 7.0, 8.0):
            k = torch.zeros(6, 128, 1, d)
            k[..., 0], k[..., 1] = sign * 4096.0, sign * (far - 4096.0 * 4096.0) / 1024.0
            k[1:, ..., 2] = above
            q = torch.zeros(n, 4, d)
            q[..., 0], q[..., 1], q[..., 2] = 4096.0, 1024.0, 1.0
            out = attend_shared(q.half().to(DEV), k.half().to(DEV), v.half().to(DEV), None, None, batch, 768, math.log(2.0))
            assert bool((out >= 1.9).all()) and bool((out <= 2.0).all())


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,batch", [(1, 640), (40, 320)])
@pytest.mark.parametrize("sign", [-1, 1])
def test_scores_a_step_of_fp32_apart(dtype, d, n, batch, sign):
    """Scores of 2^25 to 2^30 (log2) over the exact cache, later pages' one step of fp32 (2 to 64) above the first's: the values of the later
    pages, with 1/6 of the first's weight for 5 pages at most."""
    v = torch.full((6, 128, 1, d), 2.0)
    v[0] = 1.0
    for power in range(25, 31):
        step = 2.0 ** (power - 23)
        for odd in (0, 1):  # the parity of the last bit
            k, q = torch.zeros(6, 128, 1, d), torch.zeros(n, 4, d)
            k[..., 0], k[..., 1], k[1:, ..., 2] = sign * 1.25 * 2.0 ** 12, sign * odd * step, step
            q[..., 0], q[..., 1], q[..., 2] = 2.0 ** (power - 12), 1.0, 1.0
            if q.max() > 65504.0:
                k[..., 0] *= 8.0
                q[..., 0] /= 8.0
            out = attend_shared(q.to(dtype).to(DEV), k.to(dtype).to(DEV), v.to(dtype).to(DEV), None, None, batch, 768, math.log(2.0))
            assert bool((out >= 2.0 - 1.0 / 6).all()) and bool((out <= 2.0).all()), (power, odd)


# ---- rings of tiles ----

@pytest.mark.parametrize("dtype", HALVES + [E4M3])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 8])
def test_few_rows_read_their_own_tiles_every_time(dtype, d, n):
    """Steady rings on every SM, over and over: an entry that TMA fills again before its last load has returned would show as another
    result in some run."""
    gen = torch.Generator(device=DEV).manual_seed(d + n)
    batch, blocks = 96, 30
    k, v = (torch.randn((blocks, 128, 2, d), generator=gen, device=DEV).to(dtype) for _ in range(2))
    q = torch.randn((batch * n, 8, d), generator=gen, device=DEV).to(torch.bfloat16 if dtype is E4M3 else dtype)
    table = torch.stack([torch.randperm(blocks, generator=gen, device=DEV) for _ in range(batch)]).to(torch.int32)
    lens = torch.randint(2500, 128 * blocks + 1, (batch,), generator=gen, device=DEV).to(torch.int32)
    starts = torch.arange(0, (batch + 1) * n, n, dtype=torch.int32, device=DEV)
    one = {"k_scale": torch.ones(blocks, 2, device=DEV), "v_scale": torch.ones(blocks, 2, device=DEV)} if dtype is E4M3 else {}
    outs = [paged.attention(q, k, v, table, None, starts, lens, max_q=n, **one) for _ in range(200)]
    assert bool(outs[0].isfinite().all()) and sum(not torch.equal(outs[0], x) for x in outs) == 0
    for b in (0, batch - 1):  # and they are right
        m = int(lens[b])
        kk, vv = (x.view(torch.uint8)[table[b].long()].view(x.dtype).float().flatten(0, 1)[:m] for x in (k, v))
        vis = [m - n + i + 1 for i in range(n)]
        if dtype is E4M3:
            want, bound = ref.attention8(q[b * n:(b + 1) * n], kk, torch.ones(m, 2, device=DEV), vv, torch.ones(m, 2, device=DEV), vis, d ** -0.5)
        else:
            want, bound = paged_reference.attention(q[b * n:(b + 1) * n], kk, vv, vis, d ** -0.5)
        assert bool(((outs[0][b * n:(b + 1) * n].double() - want).abs() <= bound).all())


# ---- appends ----

@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("rows,starts,totals", [
    (100, [500, 600], [100]), (100, [0, 100, 700], [100, 600]), (1000, [0, 1000, 10, 20], [1000, 0, 10]), (1000, [0, 1000, 10, 20], [1000, 700, 10]),
    (300, [0, 300, 2, 300], [300, 3, 298]), (6, [0, 2, -5, 6], [2, 4, 6]), (6, [-3, 2, 6], [5, 4]), (40, [0] + [40] * 700 + [39, 40], [40] + [1] * 701),
])
def test_starts_that_fall_or_pass_the_rows_are_reported(dtype, rows, starts, totals):
    batch, d = len(totals), 64
    k = torch.randn(rows, 1, d, device=DEV).to(torch.bfloat16)
    pools = [torch.zeros(16, 128, 1, d, dtype=torch.uint8 if dtype is E4M3 else dtype, device=DEV) for _ in range(2)]
    if dtype is E4M3:
        pools = [p.view(E4M3) for p in pools]
    scales = {"k_scale": torch.ones(16, 1, device=DEV), "v_scale": torch.ones(16, 1, device=DEV)} if dtype is E4M3 else {}
    table = torch.full((batch, 8), -1, dtype=torch.int32)
    table[0], table[-1, :3] = torch.arange(8), torch.arange(8, 11)
    table[1:-1] = 15
    word = i32([0])
    paged.extend(k, k, *pools, table.to(DEV), None, i32(starts), i32(totals), status=word, **scales)
    assert word.item() == paged.TQ_DEV_ERR_LENGTH


@pytest.mark.parametrize("stored", [1.25 * 2.0 ** -3, 1.75 * 2.0 ** 9, 3.0 * 2.0 ** -61, 2.0 ** 70, math.inf, math.nan, 0.0, -1.0, 2.0 ** -70, 1.5 * 2.0 ** 60])
@pytest.mark.parametrize("had,new", [(5, 3), (100, 60)])
def test_extend_keeps_what_a_callers_scale_stands_for(stored, had, new):
    """A partly filled page with a scale that extend did not write: its numbers stand for what attention takes them for (a
    scale outside [2^-60, 2^60] counts as the nearest of the two, none as the least), also behind the step."""
    d, gen = 64, torch.Generator().manual_seed(3)
    k = torch.randn((new, 2, d), generator=gen).to(torch.bfloat16).to(DEV)
    held = torch.randn((3, 128, 2, d), generator=gen)
    pools, scales = [codes(held) for _ in range(2)], [torch.full((3, 2), stored, device=DEV) for _ in range(2)]
    before = pools[0][1, :had].float().double()
    word = i32([0])
    paged.extend(k, k, *pools, i32([[1, 2]]), None, i32([0, new]), i32([had + new]), k_scale=scales[0], v_scale=scales[1], status=word)
    was = 2.0 ** -60 if not stored > 2.0 ** -60 else min(float(torch.tensor(stored)), 2.0 ** 60)
    rounded = 2.0 ** math.ceil(math.log2(was))
    assert word.item() == 0
    for pool, scale in zip(pools, scales):
        for h in range(2):
            now = max(rounded, ref.scale_of(k[:min(new, 128 - had), h].abs().max().item()))
            assert scale[1, h].item() == now
            old = before[:, h] * (was / now)
            assert bool(((pool[1, :had, h].float().double() - old).abs() <= ref.half_step8(old) * (1 + 2.0 ** -20)).all())
            y = k[:min(new, 128 - had), h].double() / now
            assert bool(((pool[1, had:min(had + new, 128), h].float().double() - y).abs() <= ref.half_step8(y)).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rd,layout", [(24, "plain"), (8, "fused"), (64, "odd"), (24, "odd")])
@pytest.mark.parametrize("nq,kv", [([3, 1, 8], [130, 128, 300]), ([9, 40], [135, 140]), ([300], [500]), ([5, 700, 1], [5, 701, 400])])
@pytest.mark.parametrize("heads_first", [False, True])
def test_extend_of_8_bits_by_four_pairs_at_head_dim_64(dtype, rd, layout, nq, kv, heads_first):
    """Pairs or addresses that do not allow eight pairs in 16 bytes, in short and long runs across pages."""
    run_extend8(((nq, kv), 4, 3, 64, rd, layout, heads_first), dtype, 31)


@pytest.mark.parametrize("d,hq", [(64, 20), (128, 8)])
def test_queries_at_odd_addresses_beside_aligned_keys(d, hq):
    """Queries of a launch of their own take another width than keys and values: the call's results are those of rotation and of a
    call without queries."""
    nq = [(9 << 20) // (hq * d) - 200, 150]
    kv = [nq[0], 400]
    gen = torch.Generator().manual_seed(d)
    rows = sum(nq)
    q = normal(gen, (rows, hq, d), torch.bfloat16, "odd")
    k, v = (normal(gen, (rows, 2, d), torch.bfloat16) for _ in range(2))
    table, slot, blocks = place_requests(nq, kv, 1)
    args = (table, i32(slot), i32(starts_of(nq)), i32(kv))
    r, at = paged.Rotary(d), torch.cat([torch.arange(m - n, m) for n, m in zip(nq, kv)]).to(torch.int32).to(DEV)
    results = []
    for queries in (q, None):
        pools = [torch.zeros(blocks, 128, 2, d, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
        scales = [torch.ones(blocks, 2, device=DEV) for _ in range(2)]
        out = paged.extend(k, v, *pools, *args, rotary=r, q=queries, k_scale=scales[0], v_scale=scales[1])
        if queries is not None:
            assert torch.equal(out, paged.rotate(q, at, r))
        results.append(pools + scales)
    assert all(same(a, b) for a, b in zip(*results))


# ---- gradients of a rotation ----

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_rotation_records_its_gradient(dtype, interleaved):
    gen = torch.Generator().manual_seed(5)
    x, g = (torch.randn((7, 5, 64), generator=gen).to(dtype).to(DEV) for _ in range(2))
    at, r = i32([0, 5, 900, 31, 7, 131071, 2]), paged.Rotary(32, interleaved=interleaved, scaling="ramp", factor=4.0, first=1024)
    for inverse in (False, True):
        leaf = x.clone().requires_grad_()
        y = paged.rotate(leaf, at, r, inverse=inverse)
        assert torch.equal(y, paged.rotate(x, at, r, inverse=inverse)) and y.requires_grad
        y.backward(g)
        assert torch.equal(leaf.grad, paged.rotate(g, at, r, inverse=not inverse))
        # a part of a wider projection, and a gradient without strides of its own
        wide = torch.cat([x, x], 2).requires_grad_()
        paged.rotate(wide[..., 64:], at, r, inverse=inverse).sum().backward()
        assert torch.equal(wide.grad[..., 64:], paged.rotate(torch.ones_like(x), at, r, inverse=not inverse)) and not wide.grad[..., :64].any()
    leaf = x.clone().requires_grad_()
    twice = g.clone().requires_grad_()
    grad, = torch.autograd.grad(paged.rotate(leaf, at, r), leaf, twice, create_graph=True)
    grad.backward(x)
    assert torch.equal(twice.grad, paged.rotate(x, at, r))
    with torch.no_grad():
        assert not paged.rotate(leaf, at, r).requires_grad
        assert paged.rotate(leaf, at, r, out=torch.empty_like(x)).dtype is dtype
    with pytest.raises(ValueError):
        paged.rotate(leaf, at, r, out=torch.empty_like(x))


def test_a_rotations_gradient_by_differences():
    gen = torch.Generator().manual_seed(6)
    x, g = (torch.randn((3, 2, 16), generator=gen, dtype=torch.float32).to(DEV) for _ in range(2))
    at, r = i32([3, 77, 4000]), paged.Rotary(8, times=1.5)
    leaf = x.clone().requires_grad_()
    (paged.rotate(leaf, at, r) * g).sum().backward()
    for element in [(0, 0, 0), (1, 1, 5), (2, 0, 12)]:
        moved = x.clone()
        moved[element] += 8.0  # the map is linear
        slope = ((paged.rotate(moved, at, r).double() - paged.rotate(x, at, r).double()) * g.double()).sum() / 8.0
        assert abs(slope.item() - leaf.grad[element].item()) <= 16 * 2.0 ** -22 * 12 * g.abs().max().item()
