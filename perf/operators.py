"""Cases of the paged serving operators: block maps, paged appends, attention of new tokens over a paged cache,
and cross attention to an encoder's states.

`run` computes an operator in elementary torch operations, or (with `own`) by the framework's calls. Pages hold 128
tokens. Every length of a case follows from the case alone; the values follow from the seed.

One case is a dict with "op" and, by operator:
  map     "batch" requests whose tables are cut back to "hist" tokens (between h_lo and h_hi) and then extended by
          q_lo..q_hi new ones; "spare" is the share of blocks that the pool has beyond (below 0: short of) the need.
  append  "tokens" new rows of K and V, some of them padding without a slot, written from type "from" into pools of
          type "type"; "fused": K and V are parts of one projection's rows.
  paged   "batch" requests with hist tokens in the cache and q_lo..q_hi new ones (already appended), the first
          "chunks" of them; the others have one new token each; "idle" requests have none and no history. "tail" rows of
          q and out behind the last request are padding that stays as it is. "heads_first": a page holds its heads
          one after the other.
  cross   q_lo..q_hi decoder tokens against h_lo..h_hi encoder states each, in packed rows or ("padded") in rows of
          equal length."""
import math
import random

import numpy as np
import torch

own = False

PAGE = 128
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MOST_FLOPS, MOST_BYTES, MOST_SCORES = 1.0e12, 5.0e8, 2 ** 31


def listed():
    a = {"type": "bf16", "fused": True, "heads_first": False, "chunks": 1 << 20, "idle": 0, "tail": 0}
    return [
        # a speculative decoder's step: 256 requests drop their rejected draft tokens and map 1 to 5 new ones
        {"name": "map_step_256", "op": "map", "batch": 256, "h_lo": 1, "h_hi": 8191, "q_lo": 1, "q_hi": 5, "spare": 0.3, "lens": 1},
        # a prefill step: 16 new prompts of 4096 to 8192 tokens
        {"name": "map_prompts_16", "op": "map", "batch": 16, "h_lo": 0, "h_hi": 0, "q_lo": 4096, "q_hi": 8192, "spare": 0.3, "lens": 2},
        # the tokens of one decode step, straight from the layer's fused projection
        {"name": "append_step_128", "op": "append", "tokens": 128, "hkv": 8, "d": 128, "from": "bf16", "type": "bf16", "fused": True, "pad": 3, "lens": 3},
        # a bulk prefill of 65536 tokens x 8 KV heads
        {"name": "append_prompt_65536", "op": "append", "tokens": 65536, "hkv": 8, "d": 128, "from": "bf16", "type": "bf16", "fused": False, "pad": 0, "lens": 4},
        # one user's decode step after 32K tokens
        {**a, "name": "paged_step_32k", "op": "paged", "batch": 1, "h_lo": 32767, "h_hi": 32767, "q_lo": 1, "q_hi": 1, "hq": 32, "hkv": 8, "d": 128, "lens": 5},
        # a decode step of 16 requests of ragged lengths, with one idle slot and a captured batch's padding rows
        {**a, "name": "paged_step_16", "op": "paged", "batch": 16, "h_lo": 4096, "h_hi": 8192, "q_lo": 1, "q_hi": 1, "hq": 32, "hkv": 8, "d": 128, "lens": 6,
         "type": "f16", "idle": 1, "tail": 2},
        # drafted tokens of a small model's 8 requests, scored by the target in one pass
        {**a, "name": "paged_draft_8", "op": "paged", "batch": 8, "h_lo": 100, "h_hi": 16384, "q_lo": 2, "q_hi": 8, "hq": 16, "hkv": 4, "d": 64, "lens": 7},
        # a long prompt's last chunk: 2048 new tokens after 30720
        {**a, "name": "paged_chunk_2048", "op": "paged", "batch": 1, "h_lo": 30720, "h_hi": 30720, "q_lo": 2048, "q_hi": 2048, "hq": 32, "hkv": 8, "d": 128, "lens": 8},
        # continuous batching at head_dim 256: one chunk of a prompt beside seven decoding requests
        {**a, "name": "paged_mixed_8", "op": "paged", "batch": 8, "h_lo": 500, "h_hi": 8192, "q_lo": 500, "q_hi": 512, "hq": 16, "hkv": 4, "d": 256, "lens": 9,
         "fused": False, "heads_first": True, "chunks": 1},
        # an encoder-decoder's step: one token each against up to 1500 states
        {"name": "cross_step_16", "op": "cross", "batch": 16, "q_lo": 1, "q_hi": 1, "h_lo": 700, "h_hi": 1500, "hq": 16, "hkv": 16, "d": 64, "type": "f16",
         "padded": True, "fused": False, "lens": 10},
        # the decoder's prompts against packed encoder states
        {"name": "cross_prompts_8", "op": "cross", "batch": 8, "q_lo": 1, "q_hi": 448, "h_lo": 100, "h_hi": 1500, "hq": 20, "hkv": 20, "d": 64, "type": "bf16",
         "padded": False, "fused": True, "lens": 11},
        # long documents: up to 2048 decoder tokens against up to 4096 states, grouped heads
        {"name": "cross_long_4", "op": "cross", "batch": 4, "q_lo": 1024, "q_hi": 2048, "h_lo": 2048, "h_hi": 4096, "hq": 32, "hkv": 8, "d": 128, "type": "bf16",
         "padded": False, "fused": True, "lens": 12},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def _draw_heads(rng):
    hkv, g = rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([1, 1, 2, 3, 4, 4, 6, 8, 16])
    return {"hq": hkv * g, "hkv": hkv, "d": rng.choice([64, 128, 128, 256]), "type": rng.choice(["bf16", "f16"])}


def _draw_once(rng):
    op = rng.choice(["map", "append", "paged", "paged", "paged", "cross", "cross"])
    lens = rng.randrange(1 << 30)
    if op == "map":
        q = _spread(rng, 1, 8192)
        return {"op": op, "batch": _spread(rng, 1, 1024), "h_lo": 0, "h_hi": _spread(rng, 1, 32768), "q_lo": rng.choice([0, 1, q]), "q_hi": q,
                "spare": rng.choice([0.0, 0.5, -0.3]), "lens": lens}
    if op == "append":
        return {"op": op, "tokens": _spread(rng, 1, 65536), "hkv": rng.randint(1, 16), "d": rng.choice([64, 128, 256]), "from": rng.choice(["bf16", "f16", "f32"]),
                "type": rng.choice(["bf16", "f16"]), "fused": rng.random() < 0.5, "pad": rng.choice([0, 0, 1, 9]), "lens": lens}
    if op == "paged":
        kind = rng.choice(["step", "draft", "chunk", "mixed"])
        batch = _spread(rng, 1, 64 if kind in ("step", "draft") else 8)
        q = {"step": 1, "draft": rng.randint(2, 16), "chunk": _spread(rng, 17, 4096), "mixed": _spread(rng, 17, 1024)}[kind]
        hist = _spread(rng, 1, 65536)
        return {"op": op, "batch": batch, "h_lo": rng.choice([0, hist // 2, hist]), "h_hi": hist, "q_lo": rng.choice([1, q]), "q_hi": q, **_draw_heads(rng),
                "fused": rng.random() < 0.5, "heads_first": rng.random() < 0.5, "chunks": 1 + batch // 4 if kind == "mixed" else 1 << 20,
                "idle": rng.choice([0, 0, 1]) if batch > 1 else 0, "tail": rng.choice([0, 0, 5]), "lens": lens}
    q, states = rng.choice([1, _spread(rng, 1, 2048)]), _spread(rng, 1, 8192)
    return {"op": op, "batch": _spread(rng, 1, 32), "q_lo": rng.choice([0, 1, q]), "q_hi": q, "h_lo": rng.choice([0, states // 2, states]), "h_hi": states,
            **_draw_heads(rng), "padded": rng.random() < 0.5, "fused": rng.random() < 0.5, "lens": lens}


def draw(rng):
    while True:
        case = _draw_once(rng)
        if case["op"] == "map" and case["batch"] * case["q_hi"] > 1 << 18:
            continue
        w = work(case)
        if w["bytes"] > MOST_BYTES or w["flops"] > MOST_FLOPS:
            continue
        if case["op"] in ("paged", "cross"):
            nq, kv = _lengths(case)
            if not sum(n * k for n, k in zip(nq, kv)) or case["batch"] * case["hq"] * max(nq) * max(kv) > MOST_SCORES or case["batch"] * max(kv) * case["hkv"] * case["d"] > 2 ** 29:
                continue
        if case["op"] == "map" and not sum(_lengths(case)[0]):
            continue
        return case


def _lengths(case):
    """(new or decoder tokens, tokens to attend to) of every request."""
    r = random.Random(case["lens"])
    nq, kv = [], []
    for b in range(case["batch"]):
        n = r.randint(case["q_lo"], case["q_hi"]) if b < case.get("chunks", 1 << 20) else 1
        h = r.randint(case["h_lo"], case["h_hi"])
        if b >= case["batch"] - case.get("idle", 0):
            n = h = 0
        nq.append(n)
        kv.append(h if case["op"] in ("cross", "map") else h + n)
    return nq, kv


def _starts(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return s


def work(case):
    if case["op"] == "map":
        nq, hist = _lengths(case)
        pages = sum(-(-(h + n) // PAGE) - -(-h // PAGE) for n, h in zip(nq, hist))
        # lengths, ids and counts in; starts, totals, slots and new table entries out (and the same entries freed)
        return {"bytes": 4.0 * (5 * len(nq) + sum(nq) + 6 * pages), "flops": 0.0}
    if case["op"] == "append":
        size = TYPES[case["from"]].itemsize + TYPES[case["type"]].itemsize
        return {"bytes": 2.0 * (case["tokens"] - case["pad"]) * case["hkv"] * case["d"] * size + 4.0 * case["tokens"], "flops": 0.0}
    nq, kv = _lengths(case)
    pairs = sum(n * k - (n * (n - 1) // 2 if case["op"] == "paged" else 0) for n, k in zip(nq, kv))
    read = sum(k for n, k in zip(nq, kv) if n)
    return {"bytes": 4.0 * read * case["hkv"] * case["d"] + 4.0 * sum(nq) * case["hq"] * case["d"], "flops": 4.0 * pairs * case["hq"] * case["d"]}


# ---- inputs ----

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _keys(gen, shape, dtype):
    """Keys with a few strong channels, as the layers of such models have them."""
    k = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    strong = torch.randperm(shape[-1], generator=gen, device="cuda")[:4]
    k[..., strong] *= 3.0
    return k.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"map": _prepare_map, "append": _prepare_append, "paged": _prepare_paged, "cross": _prepare_cross}[case["op"]](case, seed, gen)


def _prepare_map(case, seed, gen):
    nq, hist = _lengths(case)
    batch = len(nq)
    r = np.random.RandomState(seed % (1 << 31))
    now = [-(-h // PAGE) for h in hist]
    need = [-(-(h + n) // PAGE) - p for n, h, p in zip(nq, hist, now)]
    left = np.zeros(batch, np.int64)  # pages that the last step's rejected tokens left behind
    left[r.permutation(batch)[:batch // 2]] = 1
    width = max(n + max(e, 1) for n, e in zip(now, need)) + 2
    n_blocks = sum(now) + batch // 2 + max(int(sum(need) * (1 + case["spare"])) - batch // 2, 1)
    ids = r.permutation(n_blocks).astype(np.int32)
    table = np.full((batch + 3, width), -1, np.int32)
    rows = r.permutation(batch + 3)[:batch]
    at = 0
    for b in range(batch):
        k = now[b] + int(left[b])
        table[rows[b], :k] = ids[at:at + k]
        at += k
    free = np.full(n_blocks, -1, np.int32)
    free[:n_blocks - at] = ids[at:]
    return {"op": "map", "table": torch.from_numpy(table).cuda(), "free": torch.from_numpy(free).cuda(), "n_free": _i32([n_blocks - at]),
            "rows": _i32(rows.tolist()), "lens": _i32(hist), "n_new": _i32(nq), "tokens": sum(nq)}


def _prepare_append(case, seed, gen):
    t, h, d = case["tokens"], case["hkv"], case["d"]
    if case["fused"]:  # the K and V parts of rows that also hold 4 query heads for each KV head
        both = _normal(gen, (t, 6 * h, d), TYPES[case["from"]])
        k, v = both[:, 4 * h:5 * h], both[:, 5 * h:]
    else:
        k, v = _normal(gen, (t, h, d), TYPES[case["from"]]), _normal(gen, (t, h, d), TYPES[case["from"]])
    blocks = -(-t // PAGE) + 4
    pool = torch.zeros((2, blocks, PAGE, h, d), dtype=TYPES[case["type"]], device="cuda")
    # runs of tokens in scrambled blocks, the first run from the middle of a block on
    order = torch.randperm(blocks, generator=gen, device="cuda")
    at = torch.arange(t, device="cuda") + 77
    slots = (order[at // PAGE] * PAGE + at % PAGE).to(torch.int32)
    slots[t - min(case["pad"], t - 1):] = -1
    return {"op": "append", "k": k, "v": v, "k_pool": pool[0], "v_pool": pool[1], "slots": slots}


def _plan(nq, rows):
    """Where the flat rows are in the requests: what a batch's builder knows."""
    row_b = np.repeat(np.arange(len(nq)), nq)
    row_i = np.arange(sum(nq)) - np.repeat(np.array(_starts(nq)[:-1], dtype=np.int64), nq)
    return {"starts": _i32(_starts(nq)), "row_b": torch.from_numpy(row_b).cuda(), "row_i": torch.from_numpy(row_i).cuda(), "max_q": max(nq), "total": sum(nq), "rows": rows}


def _queries(case, gen, rows):
    if case["fused"]:  # the query part of a fused projection's rows
        return _normal(gen, (rows, case["hq"] + 2 * case["hkv"], case["d"]), TYPES[case["type"]])[:, :case["hq"]]
    return _normal(gen, (rows, case["hq"], case["d"]), TYPES[case["type"]])


def _prepare_paged(case, seed, gen):
    nq, kv = _lengths(case)
    batch, h, d, t = case["batch"], case["hkv"], case["d"], TYPES[case["type"]]
    pages = [-(-k // PAGE) for k in kv]
    width, blocks = max(pages) + 1, sum(pages) + 2
    shape = (blocks, h, PAGE, d) if case["heads_first"] else (blocks, PAGE, h, d)
    pools = [_keys(gen, shape, t), _normal(gen, shape, t)]
    if case["heads_first"]:
        pools = [p.transpose(1, 2) for p in pools]
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
    if last:  # what nobody has written yet is whatever the memory held
        stale = torch.arange(PAGE, device="cuda")[None] >= torch.tensor(cut, device="cuda")[:, None]
        for p in pools:
            rows = p[torch.tensor(last, device="cuda")]
            rows.masked_fill_(stale[:, :, None, None], float("nan"))
            p[torch.tensor(last, device="cuda")] = rows
    rows = sum(nq) + case["tail"]
    return {"op": "paged", "q": _queries(case, gen, rows), "k": pools[0], "v": pools[1], "table": table.cuda(), "slot": slot.to(torch.int32).cuda(), "kv": _i32(kv),
            "max_kv": max(kv), "out": torch.full((rows, case["hq"], d), 1 / 64, dtype=t, device="cuda"), **_plan(nq, rows)}


def _prepare_cross(case, seed, gen):
    nq, kv = _lengths(case)
    batch, h, d, t = case["batch"], case["hkv"], case["d"], TYPES[case["type"]]
    state = {"op": "cross", "q": _queries(case, gen, sum(nq)), "kv": _i32(kv), "kv_starts": _i32(_starts(kv)), "max_kv": max(kv), "padded": case["padded"], **_plan(nq, sum(nq))}
    rows = (batch, max(kv, default=0)) if case["padded"] else (sum(kv),)
    if case["fused"]:  # one projection for both
        both = _normal(gen, rows + (2 * h, d), t)
        state["k"], state["v"] = both[..., :h, :], both[..., h:, :]
    else:
        state["k"], state["v"] = _keys(gen, rows + (h, d), t), _normal(gen, rows + (h, d), t)
    if case["padded"]:  # padding states are whatever the encoder left there
        stale = torch.arange(rows[1], device="cuda")[None] >= state["kv"][:, None]
        for x in (state["k"], state["v"]):
            x.masked_fill_(stale[:, :, None, None], float("nan"))
    return state


# ---- one pass ----

def run(state):
    return {"map": _run_map, "append": _run_append, "paged": _run_paged, "cross": _run_cross}[state["op"]](state)


def _run_map(s):
    if own:
        from kv_cache_quantization_quantize_gb300 import paged
        paged.release_blocks(s["table"], s["free"], s["n_free"], s["rows"], keep=s["lens"])
        slots, starts, totals = paged.map_blocks(s["table"], s["free"], s["n_free"], s["rows"], s["lens"], s["n_new"], s["tokens"])
        return {"slots": slots, "starts": starts, "totals": totals, "table": s["table"], "free": s["free"], "n_free": s["n_free"]}
    table, free, n_blocks = s["table"], s["free"], s["free"].shape[0]
    rows, lens, n_new = s["rows"].long(), s["lens"].long(), s["n_new"].long()
    page = torch.arange(table.shape[1], device=table.device)[None]
    held = (lens + PAGE - 1) // PAGE
    # release: the pages past the kept tokens go back, the first one on top
    mine = table[rows].long()
    gone = (page >= held[:, None]) & (mine >= 0)
    nth = gone.flatten().cumsum(0).view_as(gone)
    n_gone = nth[-1, -1]
    stack = torch.cat([free, free.new_zeros(1)])  # one more entry takes what is not meant
    to = torch.where(gone, s["n_free"].long() + n_gone - nth, n_blocks)
    stack[to.flatten()] = mine.to(torch.int32).flatten()
    n_free = s["n_free"].long() + n_gone
    mine = torch.where(gone, -1, mine)
    # map: a block for every new page that has none, from the top of the stack, in the order of requests and pages
    total = lens + n_new
    new = (page >= held[:, None]) & (page < ((total + PAGE - 1) // PAGE)[:, None]) & (mine < 0)
    need = new.sum(1)
    served = (need == 0) | (need.cumsum(0) <= n_free)
    new &= served[:, None]
    nth = new.flatten().cumsum(0).view_as(new)
    mine = torch.where(new, stack[torch.where(new, n_free - nth, n_blocks)].long(), mine)
    table[rows] = mine.to(torch.int32)
    free.copy_(stack[:n_blocks])
    s["n_free"].copy_(n_free - nth[-1, -1])
    starts = torch.cat([n_new.new_zeros(1), n_new.cumsum(0)])
    i = torch.arange(s["tokens"], device=table.device)
    b = torch.searchsorted(starts[1:], i, right=True)
    pos = lens[b] + i - starts[b]
    block = mine[b, pos // PAGE]
    slots = torch.where(served[b] & (block >= 0), block * PAGE + pos % PAGE, -1)
    return {"slots": slots.to(torch.int32), "starts": starts.to(torch.int32), "totals": torch.where(served, total, 0).to(torch.int32),
            "table": table, "free": free, "n_free": s["n_free"]}


def _run_append(s):
    if own:
        from kv_cache_quantization_quantize_gb300 import paged
        paged.append(s["k"], s["v"], s["k_pool"], s["v_pool"], s["slots"])
        return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    slots = s["slots"].long()
    there = (slots >= 0)[:, None, None]
    # a row without a slot writes what the row with the highest slot writes, to the same place
    at, top = torch.where(slots >= 0, slots, slots.max()), slots.argmax()
    for x, pool in ((s["k"], s["k_pool"]), (s["v"], s["v_pool"])):
        pool.view(-1, *pool.shape[2:])[at] = torch.where(there, x, x[top][None]).to(pool.dtype)
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain(s, k, v, causal):
    """Softmax attention of padded requests in 32 bits: k, v [batch, states, kv heads, d]."""
    batch, span, h, d = k.shape
    g = s["q"].shape[1] // h
    kv, n = s["kv"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    at = (s["starts"][:-1].long()[:, None] + torch.arange(s["max_q"], device=k.device)).clamp_(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(batch, s["max_q"], h, g, d).permute(0, 2, 3, 1, 4).reshape(batch, h, g * s["max_q"], d)
    col = torch.arange(span, device=k.device)
    there = col[None] < kv[:, None]
    seen = there[:, None, :].expand(batch, s["max_q"], span)
    if causal:
        pos = (kv - n)[:, None] + torch.arange(s["max_q"], device=k.device)
        seen = seen & (col <= pos[:, :, None])
    x = (q @ k.float().permute(0, 2, 3, 1)).view(batch, h, g, s["max_q"], span)
    x.mul_(1.0 / math.sqrt(d)).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    v = torch.where(there[:, :, None, None], v, 0).float().permute(0, 2, 1, 3)
    o = (x.view(batch, h, g * s["max_q"], span) @ v).view(batch, h, g, s["max_q"], d)
    o = o / torch.where(total == 0, 1.0, total)
    return o.permute(0, 3, 1, 2, 4)[s["row_b"], s["row_i"]].reshape(s["total"], h * g, d).to(s["q"].dtype)


def _run_paged(s):
    if own:
        from kv_cache_quantization_quantize_gb300 import paged
        return paged.attention(s["q"], s["k"], s["v"], s["table"], s["slot"], s["starts"], s["kv"], max_q=s["max_q"], max_kv=s["max_kv"], out=s["out"])
    pages = -(-s["max_kv"] // PAGE)
    blocks = s["table"][s["slot"].long(), :pages].long().clamp_(min=0)
    batch = blocks.shape[0]
    k, v = (p[blocks].reshape(batch, pages * PAGE, p.shape[2], p.shape[3])[:, :s["max_kv"]] for p in (s["k"], s["v"]))
    s["out"][:s["total"]] = _plain(s, k, v, True)
    return s["out"]


def _run_cross(s):
    if own:
        from kv_cache_quantization_quantize_gb300 import paged
        if s["padded"]:
            return paged.cross_attention(s["q"], s["k"], s["v"], s["starts"], kv_lens=s["kv"], max_q=s["max_q"])
        return paged.cross_attention(s["q"], s["k"], s["v"], s["starts"], kv_starts=s["kv_starts"], max_q=s["max_q"], max_kv=s["max_kv"])
    k, v = s["k"], s["v"]
    if not s["padded"] and k.shape[0]:
        at = (s["kv_starts"][:-1].long()[:, None] + torch.arange(s["max_kv"], device=k.device)).clamp_(max=k.shape[0] - 1)
        k, v = k[at], v[at]
    elif not s["padded"]:
        k, v = (x.new_zeros((s["kv"].shape[0], 1) + x.shape[1:]) for x in (k, v))
    elif not k.shape[1]:
        k, v = (x.new_zeros((x.shape[0], 1) + x.shape[2:]) for x in (k, v))
    return _plain(s, k, v, False)


# ---- 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "map":
        return _exact_map(s)
    if case["op"] == "append":
        k, v, slots = s["k"].double(), s["v"].double(), s["slots"]
        keep = slots >= 0
        res = {}
        for name, x in (("k_pool", k), ("v_pool", v)):
            pool = s[name].double()
            blocks, page = torch.div(slots[keep], PAGE, rounding_mode="floor").long(), (slots[keep] % PAGE).long()
            pool[blocks, page] = x[keep]
            res[name] = pool
        return res
    nq, kv = _lengths(case)
    d, g = case["d"], case["hq"] // case["hkv"]
    out = s["out"].double() if case["op"] == "paged" else torch.zeros((sum(nq), case["hq"], d), dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for b, (n, m) in enumerate(zip(nq, kv)):
        if case["op"] == "paged":
            ids = s["table"][int(s["slot"][b]), :-(-m // PAGE)].tolist()
            ks, vs = ([p[i] for i in ids] for p in (s["k"], s["v"]))
            ks, vs = (torch.cat(x)[:m].double() if m else None for x in (ks, vs))
        elif case["padded"]:
            ks, vs = s["k"][b, :m].double(), s["v"][b, :m].double()
        else:
            ks, vs = s["k"][k0:k0 + m].double(), s["v"][k0:k0 + m].double()
        for h in range(case["hq"] if n else 0):
            if not m:
                out[q0:q0 + n, h] = 0.0
                continue
            x = (s["q"][q0:q0 + n, h].double() @ ks[:, h // g].T) / math.sqrt(d)
            if case["op"] == "paged":
                hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu_(m - n + 1)
                x[hidden] = -math.inf
            out[q0:q0 + n, h] = torch.softmax(x, dim=-1) @ vs[:, h // g]
        q0, k0 = q0 + n, k0 + m
    return out


def _exact_map(s):
    table, free, n = s["table"].tolist(), s["free"].tolist(), s["n_free"].tolist()[0]
    rows, lens, n_new = s["rows"].tolist(), s["lens"].tolist(), s["n_new"].tolist()
    back = []
    for row, length in zip(rows, lens):
        for p in range(-(-length // PAGE), len(table[row])):
            if table[row][p] >= 0:
                back.append(table[row][p])
                table[row][p] = -1
    for block in reversed(back):
        free[n] = block
        n += 1
    slots, starts, totals, wanted, had = [], [0], [], 0, n
    for row, length, new in zip(rows, lens, n_new):
        pages = [p for p in range(-(-length // PAGE), -(-(length + new) // PAGE)) if table[row][p] < 0]
        wanted += len(pages)
        fits = not pages or wanted <= had
        if fits:
            for p in pages:
                n -= 1
                table[row][p] = free[n]
        totals.append(length + new if fits else 0)
        starts.append(starts[-1] + new)
        slots += [table[row][t // PAGE] * PAGE + t % PAGE if fits else -1 for t in range(length, length + new)]
    as_i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"slots": as_i32(slots), "starts": as_i32(starts), "totals": as_i32(totals), "table": as_i32(table), "free": as_i32(free), "n_free": as_i32([n])}
