"""Plain 64-bit references of rotary positions, rotated appends and the paged cache of 8 bits, with error bounds that follow from
the operands (test infrastructure)."""
import math

import torch

PAGE = 128
LEAST, MOST = -60, 60


def rotate(x, positions, steps, times, interleaved, inverse=False):
    """(y, size): x [tokens, heads, d] rotated in 64 bits, and times (|a| + |b|) of each element's pair (0 behind the pairs)."""
    rd = 2 * len(steps)
    angle = positions.double()[:, None, None] * torch.tensor(steps, dtype=torch.float64, device=x.device)
    c, s = angle.cos() * times, angle.sin() * times * (-1 if inverse else 1)
    x = x.double()
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if interleaved else (x[..., :rd // 2], x[..., rd // 2:rd])
    y, size = x.clone(), torch.zeros_like(x)
    pair = (slice(0, rd, 2), slice(1, rd, 2)) if interleaved else (slice(0, rd // 2), slice(rd // 2, rd))
    y[..., pair[0]], y[..., pair[1]] = a * c - b * s, b * c + a * s
    size[..., pair[0]] = size[..., pair[1]] = abs(times) * (a.abs() + b.abs())
    return y, size


def rotation_error(size, positions, steps):
    """What fp32 arithmetic may add: cosines and sines to 2^-22.7 (their argument is rounded to 2^-25 of up to pi / 4, the functions
    to 2 units of 2^-24, the factor once), two products and a sum to 2^-24 each: below 2^-22 + 2^-23 of the pair's size. The
    reference's own angle is rounded to 2^-52 of itself."""
    far = positions.double().abs()[:, None, None] * max(abs(t) for t in steps)
    return size * (2.0 ** -22 + 2.0 ** -23 + far * 2.0 ** -52)


def rounding(y, dtype):
    """Half a step of dtype at y, its subnormal steps among them."""
    least = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}[dtype]
    return y.abs() * (torch.finfo(dtype).eps / 2) + least


def nearest8(x):
    """64-bit x to the nearest e4m3 number, ties to even, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def half_step8(x):
    """Half the distance of neighbouring e4m3 numbers at |x| <= 448."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 4)


def scale_of(top):
    """The smallest power of two in [2^-60, 2^60] with top <= 448 scales."""
    if not top > 0:
        return 2.0 ** LEAST
    part, power = math.frexp(top)
    return 2.0 ** min(max(power - 9 + (part > 0.875), LEAST), MOST)


def attention8(q, k, ks, v, vs, visible, scale):
    """q [n, hq, d] over numbers k, v [m, hkv, d] with scales ks, vs [m, hkv] in 64 bits. Returns (out, bound): as
    paged_reference.attention, with weights of f16 (u_w = 2^-11) whose steps below f16's normal range, 2^-25, are relative to the largest
    weight times scale: sum of 2^-25 |v| / sum(p / vs) for p = exp(s) vs / max(exp(s) vs)."""
    n, hq, d = q.shape
    m, hkv = k.shape[:2]
    u = torch.finfo(q.dtype).eps / 2
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    if not n or not m:
        return out, bound
    col, vis = torch.arange(m, device=q.device), torch.as_tensor(visible, device=q.device)
    seen = col[None] < vis[:, None]
    for h in range(hq):
        g = h * hkv // hq
        qh, kn, vn = q[:, h].double(), k[:, g].double(), v[:, g].double()
        kn, vn = (torch.where((col < vis.max())[:, None], x, 0.0) for x in (kn, vn))
        kh, vh = kn * ks[:, g, None].double(), vn * vs[:, g, None].double()
        s = (qh @ kh.T * scale).masked_fill(~seen, -math.inf)
        top = s.amax(1, keepdim=True)
        w = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
        total = w.sum(1, keepdim=True)
        safe = torch.where(total == 0, 1.0, total)
        out[:, h] = w @ vh / safe
        a = w @ vh.abs() / safe
        e = (d + 8) * 2.0 ** -24 * ((qh.abs() @ kh.abs().T) * scale).masked_fill(~seen, 0).amax(1, keepdim=True) + 2.0 ** -20
        most = (w * vs[:, g].double()).amax(1, keepdim=True)
        bound[:, h] = u * out[:, h].abs() + 2.0 ** -11 * a + 2 * e * a + 2.0 ** -25 * most * (seen.double() @ vn.abs()) / safe
        if q.dtype == torch.float16:
            bound[:, h] += 2.0 ** -25
    return out, bound
