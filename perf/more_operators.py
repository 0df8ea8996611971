"""Cases of the rotated appends and of the 8-bit paged cache: rotary positions, a step's new tokens rotated on their way
into a paged cache of 16 or 8 bits, and attention over the cache of 8 bits.

`run` computes an operator in elementary torch operations, or (with `own`) by the framework's calls. Pages hold 128
tokens. Every length of a case follows from the case alone; the values follow from the seed.

A cache of 8 bits holds e4m3 numbers and, for each page and KV head, a scale: a power of two between 2^-60 and 2^60, the
smallest with which the largest value of the page's tokens of that head stays at most 448. A page that has tokens of
earlier steps keeps its scale unless the new ones need a larger one; then the numbers that it holds are brought to that.

One case is a dict with "op" and, by operator:
  rotate  "tokens" rows of "heads" heads of d channels, the first "rd" of them rotated; "inverse": the transposed rotation.
  extend  "batch" requests with h_lo..h_hi tokens in the cache and q_lo..q_hi new ones, the first "chunks" of them; the others
          have one new token each; "idle" requests have none. K is rotated, V is not, hq query heads are rotated beside
          them. "cache": bf16, f16 or e4m3. "tail" rows of padding stand behind the last request. "moved": the
          rotation goes by positions of the caller's instead of the tokens' places.
  attend  the same batches, whose new tokens the e4m3 cache already holds: softmax attention, causal.
"type" is the type of queries, keys and values; "fused": they are parts of one projection's rows; "heads_first": a page holds its
heads one after the other. The angles: "base", "rd", and "scaling" to longer contexts by "factor" from "first" tokens."""
import math
import random

import torch

own = False

PAGE = 128
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
LEAST, MOST = -60, 60  # exponents of a scale
MOST_FLOPS, MOST_BYTES, MOST_SCORES = 1.1e12, 4.2e8, 2 ** 31


def listed():
    r = {"rd": 128, "base": 500000.0, "interleaved": False, "scaling": "bands", "factor": 8.0, "first": 8192}
    e = {**r, "op": "extend", "type": "bf16", "fused": True, "heads_first": False, "chunks": 1 << 20, "idle": 0, "tail": 0, "moved": False}
    a = {"op": "attend", "type": "bf16", "fused": True, "heads_first": False, "chunks": 1 << 20, "idle": 0, "tail": 0}
    return [
        # the queries of one decode step, 64 requests far into their contexts
        {**r, "name": "rotate_step_64", "op": "rotate", "tokens": 64, "heads": 32, "d": 128, "type": "bf16", "fused": True, "inverse": False, "far": 131071},
        # a long prompt's queries, pairs of neighbouring channels, a quarter of the head, linearly scaled
        {**r, "name": "rotate_prompt_16384", "op": "rotate", "tokens": 16384, "heads": 32, "d": 128, "rd": 32, "base": 10000.0, "interleaved": True,
         "scaling": "linear", "factor": 4.0, "type": "f16", "fused": False, "inverse": False, "far": 16384},
        # a decode step of 128 requests into exact pools: the layer's fused projection, queries rotated in the same pass
        {**e, "name": "extend_step_128", "batch": 128, "h_lo": 100, "h_hi": 8191, "q_lo": 1, "q_hi": 1, "hq": 32, "hkv": 8, "d": 128, "cache": "bf16", "idle": 2, "tail": 3,
         "lens": 1},
        # eight prompts into exact pools, with their queries
        {**e, "name": "extend_prompts_8", "batch": 8, "h_lo": 0, "h_hi": 0, "q_lo": 1024, "q_hi": 3000, "hq": 32, "hkv": 8, "d": 128, "cache": "bf16", "lens": 2},
        # the same decode step into a cache of 8 bits
        {**e, "name": "extend8_step_128", "batch": 128, "h_lo": 100, "h_hi": 8191, "q_lo": 1, "q_hi": 1, "hq": 32, "hkv": 8, "d": 128, "cache": "e4m3", "idle": 2, "tail": 3,
         "lens": 3},
        # drafted tokens of a small model's 64 requests: heads of 64 channels, pairs of neighbours, half of the head
        {**e, "name": "extend8_draft_64", "batch": 64, "h_lo": 1, "h_hi": 16384, "q_lo": 2, "q_hi": 8, "hq": 16, "hkv": 4, "d": 64, "rd": 32, "interleaved": True,
         "base": 10000.0, "scaling": "none", "type": "f16", "cache": "e4m3", "moved": True, "lens": 4},
        # a bulk prefill of up to 65536 tokens x 8 KV heads, scores' queries elsewhere
        {**e, "name": "extend8_prompts_16", "batch": 16, "h_lo": 0, "h_hi": 300, "q_lo": 3500, "q_hi": 4500, "hq": 0, "hkv": 8, "d": 128, "cache": "e4m3", "fused": False,
         "lens": 5},
        # one user's decode step after 32K tokens
        {**a, "name": "attend8_step_32k", "batch": 1, "h_lo": 32767, "h_hi": 32767, "q_lo": 1, "q_hi": 1, "hq": 32, "hkv": 8, "d": 128, "lens": 6},
        # a decode step of 32 requests of ragged lengths, with one idle slot and a captured batch's padding rows
        {**a, "name": "attend8_step_32", "batch": 32, "h_lo": 4096, "h_hi": 8192, "q_lo": 1, "q_hi": 1, "hq": 32, "hkv": 8, "d": 128, "type": "f16", "idle": 1, "tail": 2,
         "heads_first": True, "lens": 7},
        # drafted tokens of a small model's 8 requests, scored in one pass
        {**a, "name": "attend8_draft_8", "batch": 8, "h_lo": 100, "h_hi": 16384, "q_lo": 2, "q_hi": 8, "hq": 16, "hkv": 4, "d": 64, "lens": 8},
        # a long prompt's last chunk: 2048 new tokens after 30720
        {**a, "name": "attend8_chunk_2048", "batch": 1, "h_lo": 30720, "h_hi": 30720, "q_lo": 2048, "q_hi": 2048, "hq": 32, "hkv": 8, "d": 128, "lens": 9},
        # continuous batching at head_dim 256: one chunk of a prompt beside seven decoding requests
        {**a, "name": "attend8_mixed_8", "batch": 8, "h_lo": 500, "h_hi": 8192, "q_lo": 500, "q_hi": 512, "hq": 16, "hkv": 4, "d": 256, "fused": False, "chunks": 1, "lens": 10},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def _draw_angles(rng, d):
    return {"rd": rng.choice([16, d // 4, d // 2, d, d, d]), "base": rng.choice([10000.0, 500000.0]), "interleaved": rng.random() < 0.4,
            "scaling": rng.choice(["none", "linear", "base", "bands", "ramp"]), "factor": rng.choice([2.0, 4.0, 8.0, 16.0]), "first": rng.choice([2048, 4096, 8192])}


def _draw_batch(rng):
    kind = rng.choice(["step", "draft", "chunk", "mixed"])
    batch = _spread(rng, 1, 256 if kind == "step" else 64 if kind == "draft" else 16)
    q = {"step": 1, "draft": rng.randint(2, 16), "chunk": _spread(rng, 17, 8192), "mixed": _spread(rng, 17, 2048)}[kind]
    hist = _spread(rng, 1, 65536)
    return {"batch": batch, "h_lo": rng.choice([0, hist // 2, hist]), "h_hi": hist, "q_lo": rng.choice([1, q]), "q_hi": q, "type": rng.choice(["bf16", "f16"]),
            "fused": rng.random() < 0.5, "heads_first": rng.random() < 0.5, "chunks": 1 + batch // 4 if kind == "mixed" else 1 << 20,
            "idle": rng.choice([0, 0, 1]) if batch > 1 else 0, "tail": rng.choice([0, 0, 5]), "lens": rng.randrange(1 << 30)}


def _draw_once(rng):
    op = rng.choice(["rotate", "extend", "extend", "extend", "attend", "attend", "attend"])
    if op == "rotate":
        d = rng.choice([64, 96, 128, 256])
        return {"op": op, "tokens": _spread(rng, 1, 65536), "heads": rng.choice([1, 2, 3, 5, 8, 16, 32]), "d": d, **_draw_angles(rng, d), "type": rng.choice(["bf16", "f16", "f32"]),
                "fused": rng.random() < 0.5, "inverse": rng.random() < 0.3, "far": _spread(rng, 1, 1 << 20)}
    d, hkv, g = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([1, 1, 2, 3, 4, 4, 6, 8, 16])
    heads = {"hq": hkv * g, "hkv": hkv, "d": d}
    if op == "attend":
        return {"op": op, **_draw_batch(rng), **heads}
    kind = rng.choice(["bf16", "f16", "f32"])
    return {"op": op, **_draw_batch(rng), **heads, **_draw_angles(rng, d), "type": kind, "hq": rng.choice([0, hkv * g]), "moved": rng.random() < 0.3,
            "cache": rng.choice(["bf16", "f16", "e4m3", "e4m3", "e4m3"])}


def draw(rng):
    while True:
        case = _draw_once(rng)
        w = work(case)
        if w["bytes"] > MOST_BYTES or w["flops"] > MOST_FLOPS:
            continue
        if case["op"] != "rotate":
            nq, kv = _lengths(case)
            if not sum(nq) or case["batch"] * max(kv) * case["hkv"] * case["d"] > 2 ** 29 and case["op"] == "attend":
                continue
            if case["op"] == "attend" and case["batch"] * case["hq"] * max(nq) * max(kv) > MOST_SCORES:
                continue
        return case


def _lengths(case):
    """(new tokens, tokens in the cache with them) of every request."""
    r = random.Random(case["lens"])
    nq, kv = [], []
    for b in range(case["batch"]):
        n = r.randint(case["q_lo"], case["q_hi"]) if b < case["chunks"] else 1
        h = r.randint(case["h_lo"], case["h_hi"])
        if b >= case["batch"] - case["idle"]:
            n = h = 0
        nq.append(n)
        kv.append(h + n)
    return nq, kv


def work(case):
    size = TYPES[case["type"]].itemsize
    if case["op"] == "rotate":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2.0 * n * case["d"] * size + 4.0 * case["tokens"], "flops": 3.0 * n * case["rd"]}
    nq, kv = _lengths(case)
    rows, read = sum(nq), sum(k for n, k in zip(nq, kv) if n)
    if case["op"] == "extend":
        store = TYPES[case["cache"]].itemsize
        pages = sum((k + PAGE - 1) // PAGE - (k - n) // PAGE for n, k in zip(nq, kv) if n)
        scales = 2.0 * pages * case["hkv"] * 8 if store == 1 else 0.0
        return {"bytes": 2.0 * rows * case["hkv"] * case["d"] * (size + store) + 2.0 * rows * case["hq"] * case["d"] * size + scales + 8.0 * len(nq),
                "flops": 3.0 * rows * (case["hq"] + case["hkv"]) * case["rd"]}
    pairs = sum(n * k - n * (n - 1) // 2 for n, k in zip(nq, kv))
    return {"bytes": 2.0 * read * case["hkv"] * (case["d"] + 4.0 / PAGE) + 2.0 * size * rows * case["hq"] * case["d"], "flops": 4.0 * pairs * case["hq"] * case["d"]}


# ---- the angles' steps ----

def _steps(case):
    """(angle of each pair for one position, in radians and 64 bits; what cosines and sines are multiplied with)."""
    rd, base, factor, first = case["rd"], case["base"], case["factor"], case["first"]
    kind = case["scaling"]
    if kind == "base":  # a larger base, so that the slowest pair is slowed by the factor and the fastest stays
        base *= factor ** (rd / (rd - 2))
    steps = [base ** (-2.0 * i / rd) for i in range(rd // 2)]
    times = 1.0
    if kind == "linear":
        steps = [t / factor for t in steps]
    elif kind == "bands":  # by how often a pair turns over the first context: 4 times and more stays, once and less is slowed
        turns = [t * first / (2.0 * math.pi) for t in steps]
        keep = [min(1.0, max(0.0, (n - 1.0) / 3.0)) for n in turns]
        steps = [t * k + t / factor * (1.0 - k) for t, k in zip(steps, keep)]
    elif kind == "ramp":  # over the pairs between those that turn 32 times and once
        def pair(turns):
            return rd * math.log(first / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rd - 1)
        slow = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rd // 2)]
        steps = [t / factor * s + t * (1.0 - s) for t, s in zip(steps, slow)]
        times = 0.1 * math.log(factor) + 1.0
    return steps, times


# ---- inputs ----

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"rotate": _prepare_rotate, "extend": _prepare_extend, "attend": _prepare_attend}[case["op"]](case, gen)
    s["op"] = case["op"]
    if case["op"] != "attend":
        steps, times = _steps(case)
        s.update(steps=torch.tensor(steps, dtype=torch.float64, device="cuda"), times=times, interleaved=case["interleaved"])
        if own:  # a program makes it once
            from kv_cache_quantization_quantize_gb300 import paged
            s["rotary"] = paged.Rotary(case["rd"], base=case["base"], interleaved=case["interleaved"],
                                       scaling=None if case["scaling"] == "none" else case["scaling"], factor=case["factor"], first=case["first"])
    return s


def _prepare_rotate(case, gen):
    t, h, d = case["tokens"], case["heads"], case["d"]
    x = _normal(gen, (t, h + 2, d), TYPES[case["type"]])[:, :h] if case["fused"] else _normal(gen, (t, h, d), TYPES[case["type"]])
    at = torch.randint(0, case["far"] + 1, (t,), generator=gen, device="cuda")
    return {"x": x, "at": at.to(torch.int32), "out": torch.empty((t, h, d), dtype=x.dtype, device="cuda"), "inverse": case["inverse"]}


def _batch(case, nq, kv):
    """Ids, starts and totals of a step, and where its rows are in the requests: what a batch's builder knows."""
    starts = [0]
    for n in nq:
        starts.append(starts[-1] + n)
    counts = torch.tensor(nq, device="cuda")
    row_b = torch.repeat_interleave(torch.arange(len(nq), device="cuda"), counts, output_size=sum(nq))
    row_i = torch.arange(sum(nq), device="cuda") - torch.tensor(starts[:-1], device="cuda")[row_b]
    return {"starts": _i32(starts), "kv": _i32(kv), "row_b": row_b, "row_i": row_i, "max_q": max(nq), "max_kv": max(kv), "total": sum(nq)}


def _e4m3_pages(gen, blocks, heads, d, strong, loud):
    """Pages [blocks, 128, heads, d] of an e4m3 cache and their scales: normal values, each page by a loudness of its own."""
    x = torch.randn((blocks, PAGE, heads, d), generator=gen, device="cuda", dtype=torch.float32)
    x *= torch.exp2(torch.rand((blocks, 1, heads, 1), generator=gen, device="cuda") * 2 * loud - loud)
    if strong:
        x[..., torch.randperm(d, generator=gen, device="cuda")[:4]] *= 3.0
    scale = _scale_of(x.abs().amax((1, 3)))
    return (x / scale[:, None, :, None]).to(torch.float8_e4m3fn), scale


def _heads_first(pool):
    """The same pages with each page's heads one after the other."""
    return pool.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool.transpose(1, 2).contiguous().transpose(1, 2)


def _prepare_extend(case, gen):
    nq, kv = _lengths(case)
    batch, h, d = case["batch"], case["hkv"], case["d"]
    first = [(k - n) // PAGE for n, k in zip(nq, kv)]  # pages before it are full and elsewhere
    pages = [-(-k // PAGE) - f if n else 0 for n, k, f in zip(nq, kv, first)]
    blocks, width = sum(pages) + 3, max(-(-k // PAGE) for k in kv) + 1
    ids = torch.randperm(blocks, generator=gen, device="cuda").cpu()
    table = torch.full((batch + 2, width), -1, dtype=torch.int32)
    slot = torch.randperm(batch + 2, generator=gen, device="cuda").cpu()[:batch]
    at = 0
    for b in range(batch):
        table[slot[b], :first[b]] = ids[blocks - 1].int()
        table[slot[b], first[b]:first[b] + pages[b]] = ids[at:at + pages[b]].int()
        at += pages[b]
    rows = sum(nq) + case["tail"]
    t = TYPES[case["type"]]
    if case["fused"]:  # one projection for queries, keys and values
        every = _normal(gen, (rows, case["hq"] + 2 * h, d), t)
        q, k, v = every[:, :case["hq"]], every[:, case["hq"]:case["hq"] + h], every[:, case["hq"] + h:]
    else:
        q, k, v = (_normal(gen, (rows, x, d), t) for x in (case["hq"], h, h))
    s = {"k": k, "v": v, "table": table.cuda(), "slot": slot.to(torch.int32).cuda(), **_batch(case, nq, kv)}
    if case["hq"]:
        s.update(q=q, q_out=torch.full((rows, case["hq"], d), 1 / 64, dtype=t, device="cuda"))
    if case["moved"]:
        s["at"] = torch.randint(0, 1 << 17, (rows,), generator=gen, device="cuda").to(torch.int32)
    for name in ("k", "v"):
        if case["cache"] == "e4m3":
            pool, s[name + "_scale"] = _e4m3_pages(gen, blocks, h, d, False, 3.0)
        else:
            pool = torch.zeros((blocks, PAGE, h, d), dtype=TYPES[case["cache"]], device="cuda")
        s[name + "_pool"] = _heads_first(pool) if case["heads_first"] else pool
    return s


def _prepare_attend(case, gen):
    nq, kv = _lengths(case)
    batch, h, d, t = case["batch"], case["hkv"], case["d"], TYPES[case["type"]]
    pages = [-(-k // PAGE) for k in kv]
    width, blocks = max(pages) + 1, sum(pages) + 2
    s = _batch(case, nq, kv)
    for name in ("k", "v"):
        s[name + "_pool"], s[name + "_scale"] = _e4m3_pages(gen, blocks, h, d, name == "k", 1.0)
    ids = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.full((batch + 1, width), -1, dtype=torch.int32)
    slot = torch.randperm(batch + 1, generator=gen, device="cuda").cpu()[:batch]
    at, last, cut = 0, [], []
    for b in range(batch):
        table[slot[b], :pages[b]] = ids[at:at + pages[b]]
        at += pages[b]
        if kv[b] % PAGE:
            last.append(int(ids[at - 1]))
            cut.append(kv[b] % PAGE)
    for name in ("k_pool", "v_pool"):
        if last:  # what nobody has written yet is whatever the memory held: not a number
            stale = torch.arange(PAGE, device="cuda")[None] >= torch.tensor(cut, device="cuda")[:, None]
            raw, where = s[name].view(torch.uint8), torch.tensor(last, device="cuda")
            raw[where] = raw[where].masked_fill(stale[:, :, None, None], 0x7f)
        if case["heads_first"]:
            s[name] = _heads_first(s[name])
    rows = sum(nq) + case["tail"]
    q = _normal(gen, (rows, case["hq"] + 2 * h, d), t)[:, :case["hq"]] if case["fused"] else _normal(gen, (rows, case["hq"], d), t)
    s.update(q=q, out=torch.full((rows, case["hq"], d), 1 / 64, dtype=t, device="cuda"), table=table.cuda(), slot=slot.to(torch.int32).cuda())
    return s


# ---- one pass ----

def run(state):
    return {"rotate": _run_rotate, "extend": _run_extend, "attend": _run_attend}[state["op"]](state)


def _rotated(s, x, at, inverse=False):
    """x [tokens, heads, d] in 32 bits with its first 2 * pairs channels rotated by at * steps."""
    pairs = s["steps"].shape[0]
    angle = at.double()[:, None] * s["steps"]
    c, n = (angle.cos() * s["times"]).float()[:, None], (angle.sin() * s["times"]).float()[:, None]
    if inverse:
        n = -n
    x = x.float()
    turned, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
    if s["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        return torch.cat([torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2), rest], -1)
    a, b = turned[..., :pairs], turned[..., pairs:]
    return torch.cat([a * c - b * n, b * c + a * n, rest], -1)


def _run_rotate(s):
    if own:
        from kv_cache_quantization_quantize_gb300 import paged
        return paged.rotate(s["x"], s["at"], s["rotary"], out=s["out"], inverse=s["inverse"])
    s["out"].copy_(_rotated(s, s["x"], s["at"], s["inverse"]))
    return s["out"]


def _scale_of(top):
    """The smallest power of two between 2^LEAST and 2^MOST with which values up to `top` stay at most 448 = 0.875 * 2^9."""
    part, power = torch.frexp(top)
    power = torch.where(top > 0, power - 9 + (part > 0.875), LEAST).clamp(LEAST, MOST)
    return torch.ldexp(torch.ones_like(top), power)


def _store8(x, pool, scale, block, place):
    """Rows x [rows, heads, d] in 32 bits into pages of an e4m3 cache, whose numbers follow where a scale grows."""
    blocks, heads = scale.shape
    raw = pool.view(torch.uint8)
    top = scale.new_zeros(blocks, heads).scatter_reduce(0, block[:, None].expand(-1, heads), x.abs().amax(-1), "amax")
    since = place.new_full((blocks,), PAGE).scatter_reduce(0, block, place, "amin")  # the first new place of each page
    had = torch.where((since == 0)[:, None], 2.0 ** LEAST, scale)
    now = torch.where((since < PAGE)[:, None], torch.maximum(had, _scale_of(top)), scale)
    held = (torch.arange(PAGE, device=x.device) < since[:, None]) & (since < PAGE)[:, None]
    moved = (pool.float() * (had / now)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    raw.copy_(torch.where(held[:, :, None, None], moved, raw))
    raw[block, place] = (x / now[block][..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(now)


def _run_extend(s):
    names = [n for n in ("k_pool", "v_pool", "k_scale", "v_scale", "q_out") if n in s]
    if own:
        from kv_cache_quantization_quantize_gb300 import paged
        paged.extend(s["k"], s["v"], s["k_pool"], s["v_pool"], s["table"], s["slot"], s["starts"], s["kv"], rotary=s["rotary"], positions=s.get("at"), q=s.get("q"),
                     q_out=s.get("q_out"), k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
        return {n: s[n] for n in names}
    n, b = s["total"], s["row_b"]
    lens, counts = s["kv"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    at = (lens - counts)[b] + s["row_i"]
    block, place = s["table"][s["slot"].long()[b], at // PAGE].long(), at % PAGE
    turn = s["at"][:n] if "at" in s else at
    k, v = _rotated(s, s["k"][:n], turn), s["v"][:n]
    if "k_scale" in s:
        _store8(k, s["k_pool"], s["k_scale"], block, place)
        _store8(v.float(), s["v_pool"], s["v_scale"], block, place)
    else:
        s["k_pool"][block, place] = k.to(s["k_pool"].dtype)
        s["v_pool"][block, place] = v.to(s["v_pool"].dtype)
    if "q" in s:
        s["q_out"][:n] = _rotated(s, s["q"][:n], turn).to(s["q"].dtype)
    return {n: s[n] for n in names}


def _run_attend(s):
    if own:
        from kv_cache_quantization_quantize_gb300 import paged
        return paged.attention(s["q"], s["k_pool"], s["v_pool"], s["table"], s["slot"], s["starts"], s["kv"], max_q=s["max_q"], max_kv=s["max_kv"], out=s["out"],
                               k_scale=s["k_scale"], v_scale=s["v_scale"])
    pages, most = -(-s["max_kv"] // PAGE), s["max_kv"]
    blocks = s["table"][s["slot"].long(), :pages].long().clamp_(min=0)
    batch, (_, _, h, d) = blocks.shape[0], s["k_pool"].shape
    k, v = (s[n + "_pool"].view(torch.uint8)[blocks].view(torch.float8_e4m3fn).float().mul_(s[n + "_scale"][blocks][:, :, None, :, None])
            .reshape(batch, pages * PAGE, h, d)[:, :most] for n in ("k", "v"))
    g, lens, counts = s["q"].shape[1] // h, s["kv"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    at = (s["starts"][:-1].long()[:, None] + torch.arange(s["max_q"], device=k.device)).clamp_(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(batch, s["max_q"], h, g, d).permute(0, 2, 3, 1, 4).reshape(batch, h, g * s["max_q"], d)
    col = torch.arange(most, device=k.device)
    seen = col <= ((lens - counts)[:, None] + torch.arange(s["max_q"], device=k.device))[:, :, None]
    seen &= (col < lens[:, None])[:, None]
    x = (q @ k.permute(0, 2, 3, 1)).view(batch, h, g, s["max_q"], most)
    x.mul_(1.0 / math.sqrt(d)).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    v = torch.where((col < lens[:, None])[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)
    o = (x.view(batch, h, g * s["max_q"], most) @ v).view(batch, h, g, s["max_q"], d) / torch.where(total == 0, 1.0, total)
    s["out"][:s["total"]] = o.permute(0, 3, 1, 2, 4)[s["row_b"], s["row_i"]].reshape(s["total"], h * g, d).to(s["q"].dtype)
    return s["out"]


# ---- 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "extend": _exact_extend, "attend": _exact_attend}[case["op"]](case, s)


def _turned(case, x, at, inverse=False):
    """The rotation as a product of complex numbers."""
    steps, times = _steps(case)
    rd = case["rd"]
    angle = at.double()[:, None, None] * torch.tensor(steps, dtype=torch.float64, device=x.device)
    by = torch.polar(torch.full_like(angle, times), -angle if inverse else angle)
    x = x.double()
    pairs = x[..., :rd].unflatten(-1, (rd // 2, 2)) if case["interleaved"] else x[..., :rd].unflatten(-1, (2, rd // 2)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
    y = y.flatten(-2) if case["interleaved"] else y.transpose(-1, -2).flatten(-2)
    return torch.cat([y, x[..., rd:]], -1)


def _exact_rotate(case, s):
    return _turned(case, s["x"], s["at"], case["inverse"])


def _nearest8(x):
    """x in 64 bits to the nearest e4m3 number, ties to even: steps of 2^-9 below 2^-6, three bits behind the first above."""
    power = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(power - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_extend(case, s):
    nq, kv = _lengths(case)
    places = s["table"].tolist()
    slot = s["slot"].tolist()
    res = {n: s[n].double() for n in ("k_pool", "v_pool", "k_scale", "v_scale", "q_out") if n in s}
    row = 0
    for b, (n, m) in enumerate(zip(nq, kv)):
        mine = slice(row, row + n)
        row += n
        if not n:
            continue
        turn = s["at"][mine] if case["moved"] else torch.arange(m - n, m, device="cuda")
        new = {"k": _turned(case, s["k"][mine], turn), "v": s["v"][mine].double()}
        if case["hq"]:
            res["q_out"][mine] = _turned(case, s["q"][mine], turn)
        for page in range((m - n) // PAGE, (m - 1) // PAGE + 1):
            lo, hi = max(m - n, page * PAGE), min(m, (page + 1) * PAGE)
            block, at = places[slot[b]][page], lo - page * PAGE
            for name, x in new.items():
                x, pool = x[lo - (m - n):hi - (m - n)], res[name + "_pool"]
                if case["cache"] != "e4m3":
                    pool[block, at:at + hi - lo] = x
                    continue
                most = x.abs().amax((0, 2)).clamp(min=1e-300)
                scale = torch.exp2(torch.ceil(torch.log2(most / 448.0)).clamp(LEAST, MOST))
                if at:
                    was = res[name + "_scale"][block].clone()
                    scale = torch.maximum(scale, was)
                    pool[block, :at] = _nearest8(pool[block, :at] * (was / scale)[:, None])
                pool[block, at:at + hi - lo] = _nearest8(x / scale[:, None])
                res[name + "_scale"][block] = scale
    return res


def _exact_attend(case, s):
    nq, kv = _lengths(case)
    d, g = case["d"], case["hq"] // case["hkv"]
    out, row = s["out"].double(), 0
    for b, (n, m) in enumerate(zip(nq, kv)):
        ids = s["table"][int(s["slot"][b]), :-(-m // PAGE)].long()
        for h in range(case["hkv"] if n else 0):
            k, v = ((s[x + "_pool"].view(torch.uint8)[:, :, h][ids].view(torch.float8_e4m3fn).double() * s[x + "_scale"].double()[ids, h][:, None, None]).reshape(-1, d)[:m]
                    for x in ("k", "v"))
            hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu_(m - n + 1)
            for i in range(h * g, (h + 1) * g):
                x = (s["q"][row:row + n, i].double() @ k.T) / math.sqrt(d)
                out[row:row + n, i] = torch.softmax(x.masked_fill_(hidden, -math.inf), dim=-1) @ v
        row += n
    return out
