"""Plain reference of the 4-bit cache (numpy): where each channel's code stands, the writer's
rounding in fp32 step by step, the values that rows stand for, and the bifocal decode in 64 bits."""
import numpy as np
import torch


def key_place(d, c):
    """(byte, shift) of key channel c."""
    pair, high = c % (d // 2), c // (d // 2)
    w, r = divmod(pair, d // 8)
    t, e = divmod(r, d // 32)
    return (16 * t + 4 * w + e if d == 128 else 8 * t + 4 * (w // 2) + 2 * e + w % 2), 4 * high


def value_place(d, c):
    return (d // 16) * (c % 8) + c // 16, 4 * (c % 16 // 8)


def key_group(d, c):
    return c % (d // 2) // (d // 8)


def value_group(d, c):
    return c // (d // 4)


def codes(packed, d, place):
    """uint8 [.., d/2] -> codes [.., d]."""
    at = [place(d, c) for c in range(d)]
    byte, shift = np.array([a for a, _ in at]), np.array([s for _, s in at])
    return (packed[..., byte] >> shift) & 15


def f32(t):
    return t.detach().float().cpu().numpy()


def values(k_codes, v_codes, scales):
    """The keys and values (float64) that cache rows stand for."""
    d = 2 * k_codes.shape[-1]
    kc, vc, s = k_codes.cpu().numpy(), v_codes.cpu().numpy(), f32(scales).astype(np.float64)
    gk, gv = np.array([key_group(d, c) for c in range(d)]), np.array([4 + value_group(d, c) for c in range(d)])
    return (codes(kc, d, key_place).astype(np.float64) - 8) * s[..., gk], \
        (codes(vc, d, value_place).astype(np.float64) - 8) * s[..., gv]


def tables(n, d, base):
    ang = np.arange(n)[:, None] * base ** (-2.0 * np.arange(d // 2) / d)
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def rotate_f32(x, cos, sin):
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return np.concatenate([a * cos - b * sin, b * cos + a * sin], -1)


def quantise(x, group):
    """(codes, scales as float32) of float32 rows x [.., d]; group(d, c) numbers the scale of a channel."""
    d = x.shape[-1]
    g = np.array([group(d, c) for c in range(d)])
    with np.errstate(all="ignore"):
        top = np.stack([np.abs(x[..., g == w]).max(-1) for w in range(4)], -1)
        scale = torch.from_numpy(top * np.float32(1 / 7)).to(torch.bfloat16).float().numpy()
        scale = np.where(scale < np.float32(2.0**-100), np.float32(0), scale)
        scale = np.where(np.isfinite(top), scale, np.float32("nan"))
        wide = scale[..., g]
        code = np.where(wide > 0, np.clip(np.rint(x / wide), -7, 7) + 8, 8)
    return code.astype(np.uint8), scale


def rope64(x, pos, base):
    """R(pos) x in 64 bits (x [.., d], pos broadcast against x's leading dimensions)."""
    d = x.shape[-1]
    ang = np.asarray(pos, dtype=np.float64)[..., None] * base ** (-2.0 * np.arange(d // 2) / d)
    z = (x[..., : d // 2] + 1j * x[..., d // 2:]) * np.exp(1j * ang)
    return np.concatenate([z.real, z.imag], -1)


def decode(q, k, v, w0, w_pre, base, scale=None):
    """One entry: q [Hq][d] (rotated), k, v [L][Hkv][d], all float64 -> out [Hq][d], lse [Hq]."""
    L, hkv, d = k.shape
    hq = q.shape[0]
    if L == 0:
        return np.zeros((hq, d)), np.full(hq, -np.inf)
    grow, i = max(1, -(-L // w_pre)), L - 1
    j = np.arange(L)
    remote = (i - j >= w0) & (grow > 1)
    k = np.where(remote[:, None, None], rope64(k, (j // grow - j)[:, None], base), k)
    far = rope64(q, i // grow - i, base)
    kv = np.arange(hq) // (hq // hkv)
    s = np.where(remote[None], np.einsum("hd,jhd->hj", far, k[:, kv]), np.einsum("hd,jhd->hj", q, k[:, kv]))
    s *= (1 / np.sqrt(d)) if scale is None else scale
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    return np.einsum("hj,jhd->hd", p, v[:, kv]) / p.sum(-1)[:, None], (m + np.log(p.sum(-1, keepdims=True)))[:, 0]
