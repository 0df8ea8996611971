"""CPU tests of rotary positions, rotated appends and the paged cache of 8 bits: angles, and what the host refuses before any launch."""
import math
import struct

import pytest
import torch

from kv_cache_quantization_quantize_gb300 import _abi, paged
from tests.test_paged_host import kv, queries

P = 4096  # an aligned address that no refused call reads
BAD, NOT = _abi.TQ_ERR_INVALID_ARG, _abi.TQ_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_quantization_quantize_gb300 import build
    build.build()


def rot(turns=P, dim=64, interleaved=0, factor=1.0):
    return paged._ROTARY.pack(turns, dim, interleaved, factor)


def scales(k=P, v=P, kb=2, vb=2):
    return paged._SCALES.pack(k, v, kb, vb)


def rows(k=P, v=P, q=0, q_out=0, ks=(128, 64), vs=(128, 64), qs=(256, 64), os=(256, 64), positions=0, n=3, hq=4, dtype=0):
    return paged._NEW_ROWS.pack(k, v, q, q_out, *ks, *vs, *qs, *os, positions, n, hq, dtype)


def pool8(**over):
    return kv(**{"dtype": _abi.TQ_E4M3, **over})


def extend(pool=None, scale=None, new=None, rotary=None, table=P, seqs=4, pages=4, stride=4, ids=None, starts=P, totals=P, batch=2):
    return _abi.load().tq_paged_extend(pool or pool8(), scale, new or rows(), rotary, table, seqs, pages, stride, ids, starts, totals, batch, None, None)


def test_the_packed_structs_have_the_c_layout():
    assert paged._ROTARY.size == 24 and paged._SCALES.size == 32 and paged._NEW_ROWS.size == 120 and struct.calcsize("@P") == 8


def turns_of(rotary):
    return [(t % 2 ** 64) / 2 ** 64 for t in rotary.turns.tolist()]


@pytest.mark.parametrize("args", [{}, {"scaling": "linear", "factor": 4.0}, {"scaling": "base", "factor": 8.0}, {"scaling": "bands", "factor": 8.0, "first": 8192},
                                  {"scaling": "ramp", "factor": 16.0, "first": 4096}, {"scaling": "linear", "factor": 0.5, "times": 0.25}])
@pytest.mark.parametrize("dim,base", [(8, 100.0), (64, 10000.0), (128, 500000.0)])
def test_angles(dim, base, args):
    r = paged.Rotary(dim, base=base, device="cpu", **args)
    f, first = args.get("factor", 1.0), args.get("first", 0)
    plain = [base ** (-2 * i / dim) for i in range(dim // 2)]
    scaling = args.get("scaling")
    assert r.rotary_dim == dim and len(r.steps) == dim // 2
    if scaling == "linear":
        assert r.steps == pytest.approx([t / f for t in plain], rel=1e-14)
    elif scaling == "base":  # the fastest stays, the slowest is divided by the factor
        assert r.steps[0] == 1.0 and r.steps[-1] == pytest.approx(plain[-1] / f, rel=1e-12)
    elif scaling == "bands":
        for t, got in zip(plain, r.steps):
            n = t * first / (2 * math.pi)
            assert got == pytest.approx(t if n >= 4 else t / f if n <= 1 else t / f + (t - t / f) * (n - 1) / 3, rel=1e-12)
    elif scaling == "ramp":
        assert r.steps[0] == plain[0]
        if plain[-1] * first < math.pi:  # the slowest pair turns less than half a time
            assert r.steps[-1] == pytest.approx(plain[-1] / f, rel=1e-12)
        assert all(t / f * (1 - 1e-12) <= got <= t * (1 + 1e-12) for t, got in zip(plain, r.steps))
        ratio = [got / t for t, got in zip(plain, r.steps)]
        assert ratio == sorted(ratio, reverse=True) and r.times == pytest.approx(0.1 * math.log(f) + 1)
    else:
        assert r.steps == pytest.approx(plain, rel=1e-14)
    assert r.times == args.get("times", r.times) and (scaling == "ramp" or "times" in args or r.times == 1.0)
    for t, turn in zip(r.steps, turns_of(r)):
        assert turn == pytest.approx(t / (2 * math.pi) % 1.0, rel=1e-14)


def test_angles_of_given_steps():
    r = paged.Rotary.of([0.0, -1.0, 7.0, 2 * math.pi], interleaved=True, times=2.0, device="cpu")
    assert r.rotary_dim == 8 and r.interleaved and r.times == 2.0
    got = turns_of(r)
    assert got[0] == 0.0 and got[1] == pytest.approx(1 - 1 / (2 * math.pi)) and got[2] == pytest.approx(7 / (2 * math.pi) - 1)
    assert min(got[3], 1 - got[3]) < 1e-15


@pytest.mark.parametrize("args", [{"rotary_dim": 12}, {"rotary_dim": 0}, {"base": 1.0}, {"base": math.inf}, {"factor": 0.0}, {"factor": math.nan}, {"scaling": "other"},
                                  {"scaling": "bands", "factor": 2.0}, {"scaling": "ramp", "factor": 2.0}, {"scaling": "bands", "first": 10, "low": 4.0},
                                  {"scaling": "ramp", "first": 10, "slow": 40.0}, {"times": math.inf}])
def test_refused_angles(args):
    with pytest.raises(ValueError):
        paged.Rotary(**{"rotary_dim": 64, "device": "cpu", **args})


def test_refused_steps():
    for steps in ([], [1.0, 2.0], [1.0, 1.0, 1.0, math.nan]):
        with pytest.raises(ValueError):
            paged.Rotary.of(steps, device="cpu")


@pytest.mark.parametrize("rotary,status", [(rot(dim=4), NOT), (rot(dim=12), NOT), (rot(dim=72), NOT), (rot(interleaved=2), BAD), (rot(factor=math.inf), BAD),
                                           (rot(turns=0), BAD), (rot(turns=P + 4), BAD)])
def test_bad_rotations_are_refused(rotary, status):
    lib, st = _abi.load(), paged._STRIDES.pack(128, 64)
    assert lib.tq_rotate(rotary, P, P, 0, st, st, P, 3, 2, 64, 0, None) == status
    assert extend(scale=scales(), rotary=rotary) == status


def test_rotate_refuses():
    lib, st = _abi.load(), paged._STRIDES.pack(128, 64)
    call = lambda **o: lib.tq_rotate(*{"rot": rot(), "x": P, "out": P, "dt": 0, "xs": st, "os": st, "pos": P, "n": 3, "h": 2, "d": 64, "inv": 0, "stream": None, **o}.values())  # noqa: E731
    for over, status in [({"rot": None}, BAD), ({"d": 60}, NOT), ({"d": 1032}, NOT), ({"dt": 3}, BAD), ({"inv": 2}, BAD), ({"n": -1}, BAD), ({"h": -1}, BAD), ({"x": 0}, BAD),
                         ({"out": 0}, BAD), ({"pos": None}, BAD), ({"xs": None}, BAD), ({"x": P + 1}, BAD), ({"dt": 1, "out": P + 2}, BAD)]:
        assert call(**over) == status, over
    assert call(n=0) == call(h=0) == _abi.TQ_OK


@pytest.mark.parametrize("over,status", [
    ({"scale": None}, NOT), ({"pool": kv(), "scale": scales()}, NOT), ({"pool": pool8(ks=(16384, 120, 64))}, BAD), ({"pool": pool8(v=P + 8)}, BAD),
    ({"pool": pool8(d=96)}, NOT), ({"pool": pool8(tokens=64)}, BAD), ({"pool": pool8(outer=0)}, BAD), ({"scale": scales(k=0)}, BAD), ({"scale": scales(v=P + 2)}, BAD),
    ({"scale": scales(kb=1)}, BAD), ({"new": rows(dtype=3)}, BAD), ({"new": rows(n=-1)}, BAD), ({"new": rows(hq=-1)}, BAD), ({"new": rows(k=0)}, BAD),
    ({"new": rows(v=P + 1)}, BAD), ({"new": rows(q=P, q_out=P)}, BAD), ({"new": rows(q=P), "rotary": rot()}, BAD), ({"new": rows(q=P + 1, q_out=P), "rotary": rot()}, BAD),
    ({"batch": -1}, BAD), ({"batch": 65536}, NOT), ({"batch": 5}, BAD), ({"table": None}, BAD), ({"starts": None}, BAD), ({"totals": None}, BAD), ({"seqs": 0}, BAD),
    ({"pages": (1 << 20) + 1, "stride": 1 << 21}, BAD), ({"stride": 3}, BAD),
])
def test_extend_refuses(over, status):
    assert extend(**{"scale": scales(), **over}) == status


def test_rows_and_heads_that_32_bits_would_not_count_are_refused():
    st = paged._STRIDES.pack(0, 0)
    for n, h in [(2 ** 31 - 1, 1), (2 ** 31 - 255, 1), (1, 65536), (1, 2 ** 31 - 1)]:
        assert _abi.load().tq_rotate(rot(), P, P, 0, st, st, P, n, h, 64, 0, None) == NOT
    for n in (2 ** 31 - 1, 2 ** 31 - 255):
        assert extend(scale=scales(), new=rows(n=n)) == extend(pool=kv(), new=rows(n=n)) == NOT


def test_extend_of_nothing():
    assert extend(scale=scales(), batch=0) == extend(scale=scales(), new=rows(n=0)) == _abi.TQ_OK
    assert extend(pool=kv(), new=rows(n=0)) == _abi.TQ_OK


def test_attention_over_8_bits_refuses():
    lib = _abi.load()
    call = lambda q=queries(), dt=0, pool=pool8(), s=scales(): lib.tq_paged_attention8(q, dt, pool, s, P, 4, 4, 4, None, P, 1, None, 0, None, None)  # noqa: E731
    for over, status in [({"pool": kv()}, NOT), ({"dt": 1}, NOT), ({"dt": 3}, NOT), ({"s": None}, BAD), ({"s": scales(v=0)}, BAD), ({"pool": pool8(ks=(16384, 136, 64))}, BAD),
                         ({"q": queries(heads=3)}, BAD), ({"q": queries(out=P + 2)}, BAD)]:
        assert call(**over) == status, over
    assert lib.tq_paged_attention(queries(), pool8(), P, 4, 4, 4, None, P, 1, None, 0, None, None) == NOT
    st = paged._STRIDES.pack(128, 64)
    assert lib.tq_paged_append(pool8(), P, P, 0, st, st, P, 1, None, None) == NOT
    assert lib.tq_cross_attention(queries(), pool8(), None, P, None, 0, None, None) == NOT


def test_python_refuses_tensors_of_the_host():
    x = torch.zeros(2, 1, 64)
    r = paged.Rotary(64, device="cpu")
    with pytest.raises(ValueError):
        paged.rotate(x, torch.zeros(2, dtype=torch.int32), r)
    p = torch.zeros(2, 128, 1, 64, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        paged.extend(x, x, p, p, torch.zeros(1, 2, dtype=torch.int32), None, torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), k_scale=torch.ones(2, 1),
                     v_scale=torch.ones(2, 1))


@pytest.mark.parametrize("dim,base,args,steps", [
    # pairs that turn 32 times and once over 4096 tokens: 20.9 and 45.03, so 20 and 46; pair 32 is 0.01 (7 / 13 + 6 / 13 / 16)
    (128, 10000.0, {"scaling": "ramp", "factor": 16.0, "first": 4096},
     {0: 1.0, 19: 0.064938163157621132, 20: 0.056234132519034908, 21: 0.046940859997959401, 26: 0.018583361251098548, 32: 0.0056730769230769231,
      40: 0.00088178896293156731, 45: 0.00015177160473182493, 46: 8.3345089510207752e-5, 47: 7.2173874043091136e-5, 63: 7.2173874043091136e-6}),
    (64, 500000.0, {"scaling": "ramp", "factor": 4.0, "first": 8192},
     {0: 1.0, 8: 0.037606030930863936, 9: 0.024955408670558693, 12: 0.0054694985529128318, 15: 0.0010655597684559827, 17: 0.00031282462345246008,
      18: 0.00015569310547864899, 19: 0.00010331813749637912, 31: 7.5346453803479279e-7}),
    # base 10000 * 8^(128 / 126); pair 32 is its -1/2-th power
    (128, 10000.0, {"scaling": "base", "factor": 8.0},
     {0: 1.0, 1: 0.83784800191880243, 17: 0.049409339820143031, 32: 0.0034776640481145739, 50: 0.00014396665531557265, 63: 1.4434774808618227e-5}),
    (64, 500000.0, {"scaling": "base", "factor": 2.0},
     {0: 1.0, 1: 0.64892804304100951, 11: 0.0085933394173298561, 16: 0.00098888246841342714, 25: 2.0179646705774344e-5, 31: 1.5069290760695856e-6}),
])
def test_angles_of_middle_pairs(dim, base, args, steps):
    """Against numbers of the rules' definitions, in 60 digits."""
    r = paged.Rotary(dim, base=base, device="cpu", **args)
    assert {i: r.steps[i] for i in steps} == pytest.approx(steps, rel=1e-13)
