"""Plain 64-bit references of the norm + rotary pass and of the 4-bit store (numpy), written
from the formulas; no library code."""
import math

import numpy as np

D = 128


def frequencies(theta, rotary_dim, scaling="none", factor=1.0, low=1.0, high=32.0,
                original_len=32768.0):
    out = []
    for i in range(rotary_dim // 2):
        f = theta ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "by_parts":
            turns = original_len * f / (2 * math.pi)
            g = 0.0 if turns <= low else 1.0 if turns >= high else (turns - low) / (high - low)
            f = g * f + (1 - g) * f / factor
        elif scaling == "yarn":
            def index(turns):
                return rotary_dim * math.log(original_len / (2 * math.pi * turns)) \
                    / (2 * math.log(theta))
            a = max(0, math.floor(index(high)))
            b = min(rotary_dim - 1, math.ceil(index(low)))
            b = b if b > a else a + 0.001
            g = 1.0 if i <= a else 0.0 if i >= b else 1 - (i - a) / (b - a)
            f = g * f + (1 - g) * f / factor
        out.append(f)
    return np.array(out)


def pair_index(layout, rotary_dim):
    i = np.arange(rotary_dim // 2)
    return (i, i + rotary_dim // 2) if layout == "half" else (2 * i, 2 * i + 1)


def rotate(x, pos, freq, layout, attn=1.0, back=False):
    """x [N, H, D] float64 turned at pos [N]."""
    a, b = pair_index(layout, 2 * len(freq))
    ang = pos.astype(np.float64)[:, None, None] * freq
    c, s = np.cos(ang) * attn, np.sin(ang) * attn * (-1 if back else 1)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, w, eps, pos, freq, layout, attn=1.0):
    if w is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w
    return rotate(x, pos, freq, layout, attn)


def norm_rope_bwd(x, w, eps, pos, freq, layout, dy, attn=1.0):
    g = rotate(dy, pos, freq, layout, attn, back=True)
    if w is None:
        return g, None
    r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    n = x * r
    return r * (w * g - n * (w * g * n).mean(-1, keepdims=True)), (g * n).sum((0, 1))


def bf16(x):
    """Round to bf16 (nearest even) and back, float64."""
    u = np.asarray(x, np.float32).view(np.uint32)
    u = (u + 0x7fff + ((u >> 16) & 1)) & np.uint32(0xffff0000)
    return u.view(np.float32).astype(np.float64)


def quantise(x):
    """x [..., 128] on the bf16 grid -> codes [..., 2, 64], s, m [..., 2, 1]."""
    x = np.asarray(x, np.float64).reshape(*x.shape[:-1], 2, 64)
    m = x.min(-1, keepdims=True)
    s = bf16((x.max(-1, keepdims=True) - m).astype(np.float32) / np.float32(15))
    u = np.where(s > 0, np.clip(np.rint((x - m) / np.where(s > 0, s, 1)), 0, 15), 0)
    return u, s, m


def values(u, s, m):
    return (m + s * u).reshape(*u.shape[:-2], 128)


def unpack(payload):
    """uint8 [..., 64] -> codes [..., 2, 64], by the documented bit of every dim."""
    words = np.ascontiguousarray(payload).view(np.uint32)  # little endian
    u = np.empty(payload.shape[:-1] + (2, 64), np.float64)
    for g in range(2):
        for b in range(8):
            for e in range(8):
                u[..., g, 8 * b + e] = (words[..., 2 * b + g] >> (4 * (e >> 1) + 16 * (e & 1))) & 15
    return u


def pack(u):
    words = np.zeros(u.shape[:-2] + (16,), np.uint32)
    for g in range(2):
        for b in range(8):
            for e in range(8):
                words[..., 2 * b + g] |= u[..., g, 8 * b + e].astype(np.uint32) << np.uint32(
                    4 * (e >> 1) + 16 * (e & 1))
    return words.view(np.uint8)


def attend(q, k, v, scale):
    """q [hq, D], k/v [n, hkv, D] -> out [hq, D], lse [hq]."""
    hq, hkv = q.shape[0], k.shape[1]
    out, lse = np.zeros((hq, D)), np.full(hq, -np.inf)
    for h in range(hq):
        s = k[:, h // (hq // hkv)] @ q[h] * scale
        m = s.max()
        p = np.exp(s - m)
        out[h] = p @ v[:, h // (hq // hkv)] / p.sum()
        lse[h] = m + math.log(p.sum())
    return out, lse
