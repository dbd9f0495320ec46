"""Plain 64-bit forms of the operators around the FP8 linear layer (the norm,
the paged cache, attention), for the tests; nothing of the library is used."""
import numpy as np
import torch

E4M3, E5M2 = 0, 1
FMT_MAX = {E4M3: 448.0, E5M2: 57344.0}
EMAX = {E4M3: 8, E5M2: 15}
MBITS = {E4M3: 3, E5M2: 2}
EMIN = {E4M3: -6, E5M2: -14}


def code_values(fmt):
    """float64[256]: the value of every code."""
    c = np.arange(256)
    m, off = MBITS[fmt], 1 - EMIN[fmt]
    e, f = (c & 0x7F) >> m, c & ((1 << m) - 1)
    v = np.where(e == 0, f * 2.0 ** (EMIN[fmt] - m), (1 + f / 2.0 ** m) * 2.0 ** (e.astype(float) - off))
    if fmt == E4M3:
        v[(c & 0x7F) == 0x7F] = np.nan
    else:
        v[(e == 31) & (f == 0)] = np.inf
        v[(e == 31) & (f != 0)] = np.nan
    return np.where(c & 0x80, -v, v)


def round_fp8(x, fmt):
    """x (float64) rounded to the format: nearest, ties to even, saturating;
    NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        a = np.minimum(np.abs(x), FMT_MAX[fmt] * 2)
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), EMIN[fmt])
        e = np.where(2.0 ** (e + 1) <= a, e + 1, np.where(2.0 ** e > a, np.maximum(e - 1, EMIN[fmt]), e))
        q = 2.0 ** (e - MBITS[fmt])
        r = np.minimum(np.rint(a / q) * q, FMT_MAX[fmt])
    return np.where(np.isnan(x), np.nan, np.copysign(r, x))


def encode_fp8(x, fmt):
    """uint8 codes of round_fp8(x)."""
    v = round_fp8(x, fmt)
    m = MBITS[fmt]
    a = np.abs(np.where(np.isnan(v), 0.0, v))
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), EMIN[fmt])
    sub = a < 2.0 ** EMIN[fmt]
    code = np.where(sub, a / 2.0 ** (EMIN[fmt] - m),
                    (e - EMIN[fmt] + 1) * 2 ** m + (a / 2.0 ** e - 1) * 2 ** m).astype(np.int64)
    code = np.where(np.isnan(v), 0x7F, code)
    return (code | np.where(np.signbit(np.asarray(x, dtype=np.float64)), 0x80, 0)).astype(np.uint8)


def bias_of(amax, fmt):
    """Largest b with amax * 2^b <= the format's maximum (amax > 0, finite)."""
    b = int(np.floor(np.log2(FMT_MAX[fmt] / amax)))
    while amax * 2.0 ** b > FMT_MAX[fmt]:
        b -= 1
    while amax * 2.0 ** (b + 1) <= FMT_MAX[fmt]:
        b += 1
    return b


# ------------------------------------------------------------------ norm
def norm_h(x, r):
    """round(x + r) to r's type, float64; x, r CPU tensors."""
    if r is None:
        return x.double().numpy()
    return (x.double() + r.double()).float().to(r.dtype).double().numpy()


def norm_y(h, w, eps):
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def norm_grads(dy, h, w, rstd, dh):
    xh = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdims=True))
    return dx + (0 if dh is None else dh), (dy * xh).sum(0)


# ------------------------------------------------------------------ cache
def rotate(x, pos, cos, sin, pairs):
    """fp32 rotation of x [T, H, D], each product and sum rounded."""
    x = x.astype(np.float32)
    D = x.shape[-1]
    c, s = cos[pos][:, None], sin[pos][:, None]
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :D // 2], x[..., D // 2:])
    lo, hi = a * c - b * s, b * c + a * s
    if pairs:
        return np.stack((lo, hi), -1).reshape(x.shape)
    return np.concatenate((lo, hi), -1)


def append(codes, bias, x, seqs, table, block_size, fmt, values):
    """New tokens x [T, H, D] (float32) into codes / bias (numpy, in place).
    seqs: (first row, new, length) of each sequence."""
    vals = code_values(fmt)
    for i, (first, n, length) in enumerate(seqs):
        start = length - n
        for at in range(start // block_size, -(-length // block_size) if n else 0):
            p0, p1 = max(start, at * block_size), min(length, (at + 1) * block_size)
            blk = table[i][at] if at < len(table[i]) else -1
            if p0 >= p1 or not 0 <= blk < bias.shape[0]:
                continue
            s0, s1 = p0 - at * block_size, p1 - at * block_size
            for h in range(bias.shape[1]):
                t = x[first + p0 - start:first + p1 - start, h].astype(np.float64)
                fin = np.abs(t[np.isfinite(t)])
                amax = fin.max() if fin.size else 0.0
                b = 126 if amax == 0 else min(126, bias_of(amax, fmt))
                if s0 > 0:
                    old = int(bias[blk, h])
                    if b < old:
                        view = codes[blk, h][:, :s0] if values else codes[blk, h][:s0]
                        fin = np.isfinite(vals[view])   # codes of NaN and infinity stay
                        view[...] = np.where(fin, encode_fp8(np.where(fin, vals[view], 0) * 2.0 ** (b - old), fmt), view)
                    b = min(b, old)
                bias[blk, h] = b
                c = encode_fp8(t * 2.0 ** b, fmt)
                if values:
                    codes[blk, h][:, s0:s1] = c.T
                else:
                    codes[blk, h][s0:s1] = c


def gather(codes, bias, table, length, block_size, fmt, values):
    """[length, H, D] float64 of one sequence."""
    vals = code_values(fmt)
    H = codes.shape[1]
    D = codes.shape[2] if values else codes.shape[3]
    out = np.zeros((length, H, D))
    for p in range(length):
        blk = table[p // block_size]
        c = codes[blk][:, :, p % block_size] if values else codes[blk][:, p % block_size]
        out[p] = vals[c] * 2.0 ** (-bias[blk].astype(np.float64))[:, None]
    return out


def attend(q, k, v, pos, scale, causal, window):
    """q [n, Hq, D] at positions pos over k, v [L, H, D] (float64): (out, lse,
    sum_j p_j |v_j|, largest scale * sum_d |q_d k_jd|).  Invisible keys and
    values have no influence whatever they hold."""
    n, Hq, D = q.shape
    L, H, _ = k.shape
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    mag, big = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for t in range(n):
        j = np.arange(L)
        see = np.ones(L, bool)
        if causal:
            see &= j <= pos[t]
        if window:
            see &= j > pos[t] - window
        idx = j[see]
        if not idx.size:
            continue
        for a in range(Hq):
            kk, vv = k[idx, a * H // Hq], v[idx, a * H // Hq]
            s = scale * (kk @ q[t, a])
            big[t, a] = scale * np.max(np.abs(kk) @ np.abs(q[t, a]))
            m = s.max()
            p = np.exp(s - m)
            lse[t, a] = m + np.log(p.sum())
            p /= p.sum()
            out[t, a] = p @ vv
            mag[t, a] = p @ np.abs(vv)
    return out, lse, mag, big


def bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)
