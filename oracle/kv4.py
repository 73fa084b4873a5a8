"""Plain fp64 definitions of the operations on rotary positions and the paged 4-bit KV cache."""

from __future__ import annotations

import numpy as np


def rope_frequencies(rotary_dim, theta=10000.0, scaling="none", factor=1.0, original_ctx=4096, beta_fast=32.0,
                     beta_slow=1.0):
    """Radians per position of each pair, and the magnitude."""
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    if scaling == "ntk":
        theta = theta * factor ** (rotary_dim / (rotary_dim - 2))
    f = theta ** (-2 * i / rotary_dim)
    if scaling == "linear":
        f = f / factor
    if scaling != "yarn":
        return f, 1.0
    # the pair index at which a pair turns `beta` times over the original context
    index = [rotary_dim * np.log(original_ctx / (b * 2 * np.pi)) / (2 * np.log(theta)) for b in (beta_fast, beta_slow)]
    low, high = max(np.floor(index[0]), 0), min(np.ceil(index[1]), rotary_dim - 1)
    ramp = np.clip((i - low) / max(high - low, 0.001), 0, 1)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * np.log(factor) + 1


def rotate(x, pos, rotary_dim, layout="half", transposed=False, **scaling):
    """x [T][H][d], pos [T]."""
    f, m = rope_frequencies(rotary_dim, **scaling)
    a = np.asarray(pos, np.float64)[:, None] * f
    c, s = m * np.cos(a)[:, None, :], m * np.sin(a)[:, None, :] * (-1 if transposed else 1)
    y = np.array(x, np.float64)
    i = np.arange(rotary_dim // 2)
    p, q = (i, i + rotary_dim // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y[..., p], y[..., q] = x[..., p] * c - x[..., q] * s, x[..., q] * c + x[..., p] * s
    return y


MAX_SCALE_BYTE = 0xD2


def scale_values():
    """What each scale byte stands for: fp16 with the byte as its upper bits, no sign."""
    return (np.arange(256, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)


def quantise(x):
    """x [..][d] -> codes [..][d] (1 .. 15), scale bytes [..][d / 16]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    top = np.nanmax(np.concatenate([np.abs(g), np.zeros_like(g[..., :1])], -1), -1)
    byte = np.searchsorted(7 * scale_values()[:MAX_SCALE_BYTE + 1], top).clip(max=MAX_SCALE_BYTE)
    s = scale_values()[byte][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where((s > 0) & ~np.isnan(g), np.rint(g / s), 0).clip(-7, 7)
    return (q + 8).astype(np.uint8).reshape(x.shape), byte.astype(np.uint8)


def pack(codes):
    """codes [..][d] -> bytes [..][d / 2]: of dims 8 w .. 8 w + 7, dim 8 w + 2 j is nibble j of a little-endian
    32-bit word and dim 8 w + 2 j + 1 nibble j + 4."""
    u = codes.reshape(*codes.shape[:-1], codes.shape[-1] // 8, 4, 2).astype(np.uint32)
    shift = 4 * np.arange(4, dtype=np.uint32)
    word = (u[..., 0] << shift).sum(-1) | (u[..., 1] << (shift + 16)).sum(-1)
    return word.astype("<u4").view(np.uint8).reshape(*codes.shape[:-1], codes.shape[-1] // 2)


def unpack(code_bytes, scale_bytes):
    """Bytes -> values [..][d]."""
    word = np.ascontiguousarray(code_bytes).view("<u4")
    shift = 4 * np.arange(4, dtype=np.uint32)
    low, high = (word[..., None] >> shift) & 15, (word[..., None] >> (shift + 16)) & 15
    q = np.stack([low, high], -1).reshape(*code_bytes.shape[:-1], 2 * code_bytes.shape[-1]).astype(np.float64) - 8
    return q * np.repeat(scale_values()[scale_bytes], 16, -1)


def attend(q, k, v, scale, limits):
    """q [n][H][d], k and v [keys][Hkv][d]; query i sees keys below limits[i]. Returns out, lse, and what
    bounds of the error need: sum of weight * |v|, and the largest sum over dims of |q k| * scale."""
    n, H, d = q.shape
    group = H // k.shape[1]
    out, mass = np.zeros((n, H, d)), np.zeros((n, H, d))
    lse, size = np.full((n, H), -np.inf), np.zeros((n, H))
    for i in range(n):
        m = max(0, min(int(limits[i]), len(k)))
        if m == 0:
            continue
        for h in range(H):
            kk, vv = k[:m, h // group], v[:m, h // group]
            s = kk @ q[i, h] * scale
            top = s.max()
            w = np.exp(s - top)
            lse[i, h] = top + np.log(w.sum())
            w /= w.sum()
            out[i, h], mass[i, h] = w @ vv, w @ np.abs(vv)
            size[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return out, lse, mass, size
