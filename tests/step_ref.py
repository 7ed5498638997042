"""Plain references of positions, of a cache in 4 bits and of the sampling policy, in float64 and
whole numbers (NumPy only; nothing of the library is used)."""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------------ positions

def turn(x, pos, inv_freq, interleaved, factor):
    """x [..., H, D] turned by positions pos [...], and how much of each element an error of one
    unit in a cosine or sine is worth."""
    R = 2 * len(inv_freq)
    t = (np.asarray(pos, np.float64)[..., None] * inv_freq.astype(np.float64))[..., None, :]
    c, s = factor * np.cos(t), factor * np.sin(t)
    y, size = x.astype(np.float64).copy(), np.zeros(x.shape)
    first, second = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a, b = x[..., first].astype(np.float64), x[..., second].astype(np.float64)
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = abs(factor) * (np.abs(a) + np.abs(b))
    return y, size


# ------------------------------------------------------------------ 4 bits

def encode(x):
    """Codes [..., D] and scale bytes [..., D / 32] of float32 values."""
    x = np.asarray(x, np.float32).astype(np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    odd = ~np.isfinite(b).all(-1)
    b = np.where(odd[..., None], 0.0, b)
    m, e = np.frexp(np.abs(b).max(-1))
    e = np.where(m == 0, -120, np.clip(np.where(m <= 0.75, e - 3, e - 2), -120, 125))
    r = np.ldexp(np.abs(b), -e[..., None])
    code = np.zeros(b.shape, np.int64)
    for lo, strict in ((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)):
        code += (r > lo) if strict else (r >= lo)  # a tie goes to the even code
    code += 8 * np.signbit(b)
    code = np.where(odd[..., None], 0, code)
    return code.reshape(x.shape), np.where(odd, 255, e + 127)


def decode(code, byte):
    """The float64 values that they stand for."""
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    f = np.where(byte == 255, np.nan, np.ldexp(1.0, np.where(byte == 255, 0, byte) - 127))
    return v * np.repeat(f, 32, -1)


class Pool4:
    """One layer's keys or values in 4 bits: code [P, H, page, D] and byte [P, H, page, D / 32]."""

    def __init__(self, rng, P, H, page, D):
        self.code = rng.integers(0, 16, (P, H, page, D))
        self.byte = rng.integers(100, 150, (P, H, page, D // 32))

    def arrays(self, values: bool):
        """Codes and scales in the library's layout."""
        P, H, page, D = self.code.shape
        b = (self.code[..., 0::2] | (self.code[..., 1::2] << 4)).astype(np.uint8)  # [P, H, page, D / 2]
        if values:
            S = 512 // D
            b = b.reshape(P, H, page // S, S, 16, D // 32).transpose(0, 1, 2, 4, 3, 5)
        else:
            b = b.reshape(P, H, page, D // 32, 16).transpose(0, 1, 3, 2, 4)
        return np.ascontiguousarray(b), np.ascontiguousarray(self.byte.astype(np.uint8).transpose(0, 1, 3, 2))

    def put(self, x, t, ids):
        """x [H, D] (float32 values) into slot t of a sequence with these pages."""
        p, at = ids[t // self.code.shape[2]], t % self.code.shape[2]
        self.code[p, :, at], self.byte[p, :, at] = encode(x)

    def get(self, t, ids):
        p, at = ids[t // self.code.shape[2]], t % self.code.shape[2]
        return self.code[p, :, at].copy(), self.byte[p, :, at].copy()

    def set(self, entry, t, ids):
        p, at = ids[t // self.code.shape[2]], t % self.code.shape[2]
        self.code[p, :, at], self.byte[p, :, at] = entry

    def value(self, t, ids):
        return decode(*self.get(t, ids))


# ------------------------------------------------------------------ the policy

def kept(z, T, k=0, p=1.0, m=0.0):
    """The smallest logit that the policy keeps of the row z (float64), from groups of equal logits,
    and how near a cut was to falling elsewhere (relative to the total weight)."""
    T, p, m = (float(np.float32(x)) for x in (T, p, m))
    z = z[z > -np.inf]
    value, count = np.unique(z, return_counts=True)
    value, count = value[::-1], count[::-1].astype(np.float64)
    e = np.exp((value - value[0]) / T)
    keep, near = e >= m, 1.0
    if m > 0:
        near = min(near, np.abs(e[1:] / m - 1).min(initial=1.0))
    if 0 < k < len(z):
        keep &= np.cumsum(count) - count < k
    if p < 1:
        w = np.where(keep, count * e, 0.0)
        before = np.cumsum(w) - w
        near = min(near, np.abs(before / w.sum() - p).min())
        keep &= before < p * w.sum()
    return value[keep].min(), near


def draw(z, u, T, k=0, p=1.0, m=0.0):
    """The token, and how near (relative to the total) a boundary was."""
    z = z.astype(np.float64)
    if T == 0:
        return int(np.argmax(z)), 1.0
    low, near = kept(z, T, k, p, m)
    w = np.where(z >= low, np.exp((z - z.max()) / float(np.float32(T))), 0.0)
    cdf = np.cumsum(w)
    x = float(np.float32(u)) * cdf[-1]
    # a boundary in front of every kept token is at 0 exactly, on both sides
    return int(np.searchsorted(cdf, x, side="right")), min(near, np.abs(cdf[w > 0] / cdf[-1] - x / cdf[-1]).min())
