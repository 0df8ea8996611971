"""Plain 64-bit references of the paged operators, and error bounds that follow from the operands (test infrastructure)."""
import math

import torch

PAGE = 128


def pages(n):
    return -(-n // PAGE)


def release(table, free, n_free, ids, keep):
    """Lists in, changed in place; returns the new n_free (the plain, serial form of tq_blocks_release)."""
    back, seen = [], set()
    cleared = []
    for b, i in enumerate(ids):
        k = keep[b] if keep is not None else 0
        if not 0 <= i < len(table) or i in seen or k < 0:
            seen.add(i)
            continue
        seen.add(i)
        for p in range(pages(k), len(table[i])):
            if 0 <= table[i][p] < len(free):
                back.append(table[i][p])
            if table[i][p] != -1:
                cleared.append((i, p))
    if n_free + len(back) > len(free):
        return n_free
    for i, p in cleared:
        table[i][p] = -1
    for block in reversed(back):
        free[n_free] = block
        n_free += 1
    return n_free


def map_(table, free, n_free, ids, lens, n_new, max_tokens):
    """(slots, starts, totals, n_free): the plain, serial form of tq_blocks_map; table is changed in place."""
    starts, totals, slots, seen = [0], [], [-1] * max_tokens, set()
    wanted, had = 0, n_free
    for i, n, new in zip(ids, lens, n_new):
        start = starts[-1]
        starts.append(min(max_tokens, start + max(new, 0)))
        served = 0 <= i < len(table) and i not in seen and n >= 0 and new >= 0 and start + new <= max_tokens
        seen.add(i)
        served = served and pages(n + new) <= len(table[i])
        if served:
            need = [p for p in range(pages(n), pages(n + new)) if table[i][p] < 0]
            wanted += len(need)
            served = not need or wanted <= had
            if served:
                for p in need:
                    n_free -= 1
                    table[i][p] = free[n_free]
        totals.append(n + new if served else 0)
        if served:
            for t in range(n, n + new):
                block = table[i][t // PAGE]
                if 0 <= block < len(free):
                    slots[start + t - n] = block * PAGE + t % PAGE
    return slots, starts, totals, n_free


def attention(q, k, v, visible, scale):
    """q [n, Hq, d], k, v [m, Hkv, d] of one request in 64 bits; query i sees the first visible[i] tokens. Returns (out, bound):
    bound is the error a kernel with fp32 scores and sums and 16-bit weights and results may have, per element:
      u |o|                   the result's rounding, u = eps / 2 of the type,
      u A                     each weight's rounding, A = sum w |v| (w the normalised weights),
      2 E A                   the scores: fp32 sums of d products, scaled, and 2^x: E = (d + 8) 2^-24 max|q||k| scale + 2^-20,
      f16: 2^-25 sum |v| / l  weights below f16's normal range, relative to the largest weight (l = sum exp(s - max) >= 1)."""
    dt = q.dtype
    u = torch.finfo(dt).eps / 2
    n, hq, d = q.shape
    m, hkv = k.shape[0], k.shape[1]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    if not n or not m:
        return out, bound
    col = torch.arange(m, device=q.device)
    vis = torch.as_tensor(visible, device=q.device)
    for h in range(hq):
        qh, kh, vh = q[:, h].double(), k[:, h * hkv // hq].double(), v[:, h * hkv // hq].double()
        seen = col[None] < vis[:, None]
        kh, vh = (torch.where((col < vis.max())[:, None], x, 0.0) for x in (kh, vh))
        s = (qh @ kh.T * scale).masked_fill(~seen, -math.inf)
        top = s.amax(1, keepdim=True)
        w = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
        l = w.sum(1, keepdim=True)
        safe = torch.where(l == 0, 1.0, l)
        out[:, h] = w @ vh / safe
        a = w @ vh.abs() / safe
        e = (d + 8) * 2.0 ** -24 * ((qh.abs() @ kh.abs().T) * scale).masked_fill(~seen, 0).amax(1, keepdim=True) + 2.0 ** -20
        bound[:, h] = u * (out[:, h].abs() + a) + 2 * e * a
        if dt == torch.float16:
            bound[:, h] += 2.0 ** -25 * (seen.double() @ vh.abs()) / safe + 2.0 ** -25
    return out, bound
