"""Plain 64-bit forms of the 8-bit cache's operators, and seeded inputs."""
import math

import numpy as np
import torch

BLOCK = 64


def parents(kind, t, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "chain":
        return [i - 1 for i in range(t)]
    if kind == "bfs":
        return [-1] + [(i - 1) // 3 for i in range(1, t)]
    if kind == "star":
        return [-1] + [0] * (t - 1)
    return [-1] + [int(rng.integers(0, i)) for i in range(1, t)]


def depths(parent):
    d = [0] * len(parent)
    for i in range(1, len(parent)):
        d[i] = d[parent[i]] + 1
    return d


def sees(parent):
    """[T, T] truth values: node i's root path, itself included."""
    t = len(parent)
    m = torch.zeros(t, t, dtype=torch.bool)
    for i in range(t):
        a = i
        while a >= 0:
            m[i, a] = True
            a = parent[a]
    return m


def e4m3(x):
    """x (float64) to the nearest e4m3 value, ties to even; |x| <= 448."""
    size = torch.frexp(x.abs().clamp_min(2.0 ** -6))[1] - 1
    step = torch.ldexp(torch.ones_like(x), size - 3)
    return torch.round(x / step) * step


def quantize(x):
    """(code values float64, scale bytes) of bf16 rows [H, 64 m, D] on the CPU."""
    h, n, d = x.shape
    b = x.double().reshape(h, n // BLOCK, BLOCK * d)
    codes = torch.zeros_like(b)
    byte = torch.zeros(b.shape[:2], dtype=torch.uint8)
    for i in range(h):
        for j in range(n // BLOCK):
            row = b[i, j]
            if not torch.isfinite(row).all():
                byte[i, j] = 255
                continue
            top, e = float(row.abs().max()), -100
            while top > 448 * 2.0 ** e:
                e += 1
            codes[i, j] = e4m3(row / 2.0 ** e)
            byte[i, j] = e + 127
    return codes.reshape(h, n, d), byte


def factors(byte):
    f = torch.ldexp(torch.ones(byte.shape, dtype=torch.float64), byte.cpu().to(torch.int64) - 127)
    return torch.where(byte.cpu() == 255, torch.full_like(f, math.nan), f)


def rows(codes, byte):
    """8-bit rows as float64 on the CPU; codes e4m3 [H, n, D]."""
    return codes.float().cpu().double() * factors(byte).repeat_interleave(BLOCK, 1)[:, :codes.shape[1], None]


def attention(q, k, v, n_ctx, parent, scale):
    """(out, bound, root, root bound), float64 on the CPU.  q: bf16 [T, Hq, D]; k, v:
    float64 [Hkv, n_ctx + T, D].

    bound: how far a kernel's bf16 output may be.  Its weights carry one
    rounding to bf16, its result another (2^-8 of each).  With the weights' sum
    taken before their rounding, w_j (1 + e_j) in place of w_j moves the result
    by sum w_j e_j v_j, at most 2^-8 sum w_j |v_j|; with the rounded weights'
    own sum by sum w_j e_j (v_j - out) / (1 + sum w_j e_j), at most
    2^-8 sum w_j |v_j - out| (1 + 2^-7).  Sums are taken in 32 bits.  A score sums D products in 32 bits, where each addition (the
    tensor core may cut instead of round) loses at most 2^-23 of the sum of
    magnitudes, and 2^-20 of it for the query's split into 8-bit parts; a
    score's error e changes a weight by the factor exp(e), and the weights'
    sum as well.  Exponentials and the remaining sums: 2^-18 in all.
    """
    t, hq, d = q.shape
    hkv = k.shape[0]
    g = hq // hkv
    qd = q.cpu().double()
    out = torch.empty(t, hq, d, dtype=torch.float64)
    bound = torch.empty_like(out)
    root = torch.empty(hq, n_ctx, dtype=torch.float64)
    root_bound = torch.empty_like(root)
    vis = sees(parent)
    for h in range(hq):
        kh, vh = k[h // g], v[h // g]
        x = qd[:, h] @ kh.T * scale                                  # [T, n + T]
        mag = qd[:, h].abs() @ kh.abs().T * abs(scale)
        per = (d + 8) * 2.0 ** -23 + 2.0 ** -20
        root[h] = x[0, :n_ctx] / math.log(2)
        root_bound[h] = mag[0, :n_ctx] / math.log(2) * per + 1e-30
        for i in range(t):
            at = torch.cat([torch.arange(n_ctx), n_ctx + vis[i].nonzero()[:, 0]])
            w = torch.softmax(x[i, at], 0)
            o, a = w @ vh[at], w @ vh[at].abs()
            move = torch.maximum(a, w @ (vh[at] - o).abs())
            out[i, h] = o
            eta = 2 * float(mag[i, at].max()) * per + 2.0 ** -18
            bound[i, h] = 2.0 ** -8 * (move + o.abs()) * (1 + 2.0 ** -7) + a * eta + 1e-30
    return out, bound, root, root_bound


def rotate(x, pos, freq, interleaved, mscale):
    """Float64 [n, H, D] on the CPU."""
    y = x.cpu().double().clone()
    r = 2 * len(freq)
    if not r:
        return y
    a = torch.as_tensor(pos, dtype=torch.float64)[:, None, None] * freq.cpu().double()
    c, s = torch.cos(a) * mscale, torch.sin(a) * mscale
    if interleaved:
        u, w = y[..., 0:r:2].clone(), y[..., 1:r:2].clone()
        y[..., 0:r:2], y[..., 1:r:2] = u * c - w * s, w * c + u * s
    else:
        u, w = y[..., :r // 2].clone(), y[..., r // 2:r].clone()
        y[..., :r // 2], y[..., r // 2:r] = u * c - w * s, w * c + u * s
    return y


def rotate_bound(x, freq, interleaved, mscale):
    """One rounding to bf16 of a value of at most m (|u| + |w|) after 32-bit
    products, and an angle off by 2^-21: [n, H, D] added to 2^-8 |y|."""
    y = x.cpu().double().abs()
    r = 2 * len(freq)
    b = torch.zeros_like(y)
    if r:
        if interleaved:
            s = y[..., 0:r:2] + y[..., 1:r:2]
            b[..., 0:r:2] = b[..., 1:r:2] = s
        else:
            s = y[..., :r // 2] + y[..., r // 2:r]
            b[..., :r // 2] = b[..., r // 2:r] = s
    return b * abs(mscale) * 2.0 ** -20


def bf16(rng, *shape, spread=0.5):
    """bf16 rows [H, n, D] whose size differs by block and by channel."""
    x = rng.standard_normal(shape).astype(np.float32)
    if len(shape) == 3:
        h, n, d = shape
        b = np.exp(spread * rng.standard_normal((h, n // BLOCK + 1, 1))).repeat(BLOCK, 1)[:, :n]
        x = x * b * np.exp(spread * rng.standard_normal((1, 1, d)))
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def cache_inputs(seed, hkv, d, n_q8, n_tail, t, cap=None, tail_cap=None, tail_row0=0, poison=True):
    """Tensors of an 8-bit cache on the CPU.  What no call may read (8-bit rows
    past n_q8, tail rows outside the used ones) is NaN."""
    rng = np.random.default_rng(seed)
    cap = n_q8 if cap is None else cap
    used = n_tail + t
    tail_cap = tail_row0 + used if tail_cap is None else tail_cap
    out = {}
    for name in ("k", "v"):
        codes, byte = quantize(bf16(rng, hkv, n_q8, d)) if n_q8 else (
            torch.zeros(hkv, 0, d, dtype=torch.float64), torch.zeros(hkv, 0, dtype=torch.uint8))
        full = torch.full((hkv, cap, d), 0x7F if poison else 0, dtype=torch.uint8)
        full[:, :n_q8] = codes.float().to(torch.float8_e4m3fn).view(torch.uint8)
        sc = torch.full((hkv, cap // BLOCK), 255 if poison else 0, dtype=torch.uint8)
        sc[:, :n_q8 // BLOCK] = byte
        tail = torch.full((hkv, tail_cap, d), math.nan if poison else 0.0).to(torch.bfloat16)
        tail[:, tail_row0:tail_row0 + used] = bf16(rng, hkv, used, d)
        out[name + "8"], out[name + "_scale"] = full.view(torch.float8_e4m3fn), sc
        out[name + "_tail"] = tail
    return out


def cache_rows(c, name, n_q8, tail_row0, used):
    """Context and tree rows as float64 [Hkv, n_q8 + used, D]."""
    return torch.cat([rows(c[name + "8"][:, :n_q8], c[name + "_scale"][:, :n_q8 // BLOCK]),
                      c[name + "_tail"][:, tail_row0:tail_row0 + used].double()], 1)
