"""Plain 64-bit forms of the paged-cache operators, on the CPU, for the tests.

Errors that the tests allow follow from the kernels' arithmetic: a value
rounded to fp16 is off by at most 2^-11 of itself (2^-25 where fp16 is
subnormal), an fp32 operation by 2^-24 of its result."""

import math

import torch

HALF = 2.0 ** -11      # half a step of fp16, relative
TINY = 2.0 ** -25      # half of fp16's smallest step


def frequencies(rot, theta=10000.0, scaling=None, factor=1.0, original_max=4096, fast=None, slow=1.0):
    """(angle per position of each pair, multiplier)."""
    fast = fast or (4.0 if scaling == "bands" else 32.0)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = theta ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            lo, hi = (rot * math.log(original_max / (n * 2 * math.pi)) / (2 * math.log(theta)) for n in (fast, slow))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0), 1)
            f = f * (1 - r) + f / factor * r
        if scaling == "bands":
            s = min(max((original_max * f / (2 * math.pi) - slow) / (fast - slow), 0), 1)
            f = f * s + f / factor * (1 - s)
        out.append(f)
    return torch.tensor(out, dtype=torch.float64), (0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)


def turn(x, pos, rot, interleaved=False, **kw):
    """x [T, H, d] float64 turned at pos [T]; (y, |x_a| + |x_b| of each value's pair)."""
    f, m = frequencies(rot, **kw)
    ang = pos.double()[:, None] * f
    c, s = (m * ang.cos())[:, None], (m * ang.sin())[:, None]
    y, size = x.clone(), x.abs()
    if interleaved:
        ia, ib = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    else:
        ia, ib = torch.arange(rot // 2), torch.arange(rot // 2, rot)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = m * (a.abs() + b.abs())
    return y, size


def norm(x, w, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def turn_error(y, size):
    """Angle (2^-25 half turns of argument, sine and cosine to 2^-23), two products, a sum, a norm's 20 operations:
    below 32 fp32 roundings of the pair's size; then one rounding to fp16."""
    return y.abs() * HALF + size * 2.0 ** -19 + TINY


def quantise(x):
    """Codes and fp16 scales of rows of float64 values."""
    scale = (x.abs().amax(-1) / 127).half()
    s = scale.double()[..., None]
    return torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0).round().clamp(-127, 127).to(torch.int8), scale


def pool_values(x, scales=None):
    """Pages as float64 values."""
    x = x.cpu().double()
    return x if scales is None else x * scales.cpu().double()[..., None]


def rows_of(pool, pages, n):
    """First n positions of a list of pages."""
    page = pool.shape[1]
    idx = [int(p) for p in pages[:-(-n // page)]] if n else []
    return pool[idx].flatten(0, 1)[:n] if idx else pool[:0].flatten(0, 1)


def attention(q, pools, table, kv_lens, new, prefix_pages=(), prefix_len=0, causal=True):
    """(out, error allowed) [T, Hq, d], 64 bits.  pools: float64 K and V pages.

    Error: a score sums d products (2^-24 of their absolute sum each) and is
    scaled; a weight is its exponential (to 2^-18), rounded to fp16 (2^-11, or 2^-31 of the
    largest below fp16's normal range); the sums run in fp32 in any order; the
    result is rounded once."""
    kp, vp = pools
    T, hq, d = q.shape
    hkv = kp.shape[2]
    g = hq // hkv
    out, tol = torch.zeros(T, hq, d, dtype=torch.float64), torch.full((T, hq, d), TINY, dtype=torch.float64)
    t0 = 0
    for b, n in enumerate(new):
        lk = int(kv_lens[b])
        k = torch.cat((rows_of(kp, prefix_pages, prefix_len), rows_of(kp, table[b], lk)))
        v = torch.cat((rows_of(vp, prefix_pages, prefix_len), rows_of(vp, table[b], lk)))
        j = torch.arange(prefix_len + lk)
        for h in range(hq):
            qh = q[t0:t0 + n, h].cpu().double()
            kh, vh = k[:, h // g], v[:, h // g]
            s = qh @ kh.T / math.sqrt(d)
            seen = torch.ones(n, prefix_len + lk, dtype=torch.bool)
            if causal:
                seen = j[None] < prefix_len + (torch.arange(n) + lk - n + 1)[:, None].clamp(min=0)
            s = s.masked_fill(~seen, -math.inf)
            if not s.shape[1]:
                continue
            w = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300))
            w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
            out[t0:t0 + n, h] = w @ vh
            total = w @ vh.abs()
            ds = (qh.abs() @ kh.abs().T / math.sqrt(d)).masked_fill(~seen, 0).amax(-1, keepdim=True)
            ds = ds * (d + 8) * 2.0 ** -24 + 2.0 ** -21
            steps = len(j) * 2.0 ** -24 + 2.0 ** -17      # the exponential counts in the weight and in their sum
            tol[t0:t0 + n, h] += (total * (HALF + steps) + (total + out[t0:t0 + n, h].abs()) * 2 * ds
                                  + out[t0:t0 + n, h].abs() * HALF + len(j) * 2.0 ** -31 * vh.abs().amax(0))
        t0 += n
    return out, tol
