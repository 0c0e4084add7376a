"""Plain forms of the 4-bit cache operators for the tests: host tensors, 64
bits, one formula after the other. The order of bytes in a page is not known
here; tests compare what the cache holds through what it gives back."""
import torch


def f64(t):
    return t.detach().cpu().double()


def rotate(x, cos_sin, positions, interleaved):
    """x (T, H, D) -> its rotation in 64 bits."""
    x, r = f64(x).clone(), cos_sin.shape[1]
    cs = f64(cos_sin)[positions.cpu().long()]
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    if interleaved:
        a, b = x[..., 0:r:2].clone(), x[..., 1:r:2].clone()
        x[..., 0:r:2], x[..., 1:r:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :r // 2].clone(), x[..., r // 2:r].clone()
        x[..., :r // 2], x[..., r // 2:r] = a * c - b * s, b * c + a * s
    return x


def quantize(x, group):
    """x bf16 (T, H, D) -> (codes, scales, minima) in 64 bits, scales and minima spread over the dimensions. Every step
    is one operation in fp32, as the operator defines it."""
    y = x.detach().cpu().float().reshape(*x.shape[:2], x.shape[2] // group, group)
    m = y.amin(-1, keepdim=True).half().float()
    s = ((y.amax(-1, keepdim=True) - m) / 15).half().float()
    n = torch.where(s == 0, torch.zeros_like(y), ((y - m) / s).round().clamp(0, 15)).nan_to_num(0.0)
    sh = x.shape
    return n.double().reshape(sh), s.double().expand_as(y).reshape(sh), m.double().expand_as(y).reshape(sh)


def attention(q, kv, ctx, starts, scale, window=0):
    """q (T, Hq, D); kv: per request (k, v parts) with k (ctx, Hkv, D) in 64 bits and v = (n, s, m) of the same shape.
    Returns (out, lse, mass): mass is sum_t p_t (|s (n - 8)| + |m + 8 s|), what the rounding of a weight can move."""
    q = f64(q)
    T, Hq, D = q.shape
    out, mass = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -float("inf"), dtype=torch.float64)
    for b, (k, (n, s, m)) in enumerate(kv):
        v, a = n * s + m, (s * (n - 8)).abs() + (m + 8 * s).abs()
        nq = starts[b + 1] - starts[b]
        for i in range(nq):
            pos = ctx[b] - nq + i
            lo = max(0, pos - window + 1) if window else 0
            if pos < lo:
                continue
            t = starts[b] + i
            g = Hq // k.shape[1]
            for h in range(Hq):
                x = (k[lo:pos + 1, h // g] @ q[t, h]) * scale
                lse[t, h] = torch.logsumexp(x, 0)
                p = torch.softmax(x, 0)
                out[t, h] = p @ v[lo:pos + 1, h // g]
                mass[t, h] = p @ a[lo:pos + 1, h // g]
    return out, lse, mass
