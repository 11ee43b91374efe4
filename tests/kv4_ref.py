"""The 4-bit paged cache and the norm with rotation restated in numpy (float64, or the one
fp32 rounding per operation that the contract names), from include/pnmix.h alone."""
from __future__ import annotations

import math

import numpy as np

LIMIT = 61440.0


def bf16(x: np.ndarray) -> np.ndarray:
    """Round to nearest even to bf16, as float32 (from float64 without a stop at fp32)."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        m, e = np.frexp(x)
        q = np.ldexp(np.rint(np.ldexp(m, 8)), np.maximum(e, -125) - 8)
        small = np.rint(np.ldexp(x, 133)) * 2.0 ** -133
    return np.where(np.isfinite(x), np.where(e < -125, small, q), x).astype(np.float32)


def bf16_from_f32(x: np.ndarray) -> np.ndarray:
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    return np.where(np.isnan(x), np.float32(np.nan), u.view(np.float32))


def norm_rope(x, weight, positions, inv_freq, axis, rot, interleaved, eps):
    """float64 [n][heads][D], before the rounding to bf16; and a bound on what fp32 loses."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y = x.copy()
    mag = np.abs(x)
    half = rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = np.asarray(positions[axis[i]], np.float64) * float(np.float32(inv_freq[i]))
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, mag


def quantise(x):
    """(codes [..., D], scale, zero fp16 [..., D/32]) of rows x, fp32 op order of the contract."""
    x = np.asarray(x, dtype=np.float32)
    x = np.where(np.isnan(x), np.float32(0), np.clip(x, -LIMIT, LIMIT).astype(np.float32))
    g = x.reshape(*x.shape[:-1], -1, 32)
    mn, mx = g.min(-1), g.max(-1)
    s16 = ((mx - mn).astype(np.float32) / np.float32(15)).astype(np.float16)
    z16 = mn.astype(np.float16)
    s, z = s16.astype(np.float32)[..., None], z16.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.clip(np.rint((g - z).astype(np.float32) / s), 0, 15)
    c = np.where(s > 0, c, 0).astype(np.uint8)
    return c.reshape(x.shape), s16, z16


def stand_for(c, s16, z16):
    """float32 code * s + z, one rounding."""
    g = c.reshape(*c.shape[:-1], -1, 32).astype(np.float64)
    v = g * s16.astype(np.float64)[..., None] + z16.astype(np.float64)[..., None]
    return v.astype(np.float32).reshape(c.shape)


class Pages:
    """The pages of a cache as bytes: [n_pages][Hkv][blocks][20 D]."""

    def __init__(self, n_pages, Hkv, D, page, raw=None):
        self.D, self.page, self.H = D, page, Hkv
        self.raw = np.zeros((n_pages, Hkv, page // 16, 20 * D), np.uint8) if raw is None else raw.copy()

    def _code(self, side, t, ch):
        """(byte, shift) of the code of channel ch of block token t."""
        D, n = self.D, self.D // 32
        g, e = divmod(ch, 32)
        if side == 0:
            w, i = divmod(e, 8)
            bit = 32 * g + 4 * i
            at = t * (D // 2) + w * 4 * n
        else:
            w, i = divmod(e, 4)
            bit = 16 * g + 4 * i
            place = w ^ (4 * ((t // 2) % 2)) if D == 128 else w
            at = 10 * D + t * (D // 2) + place * 2 * n
        return at + bit // 8, bit % 8

    def put(self, page, t, side, c, s16, z16):
        """One token's side: codes [H][D], scales [H][D/32]."""
        blk, r = divmod(t, 16)
        for ch in range(self.D):
            at, sh = self._code(side, r, ch)
            b = self.raw[page, :, blk, at]
            self.raw[page, :, blk, at] = (b & ~np.uint8(15 << sh)) | (c[:, ch] << sh)
        sz = np.stack([s16, z16], -1).reshape(self.H, -1).view(np.uint8)
        o = side * 10 * self.D + 8 * self.D + r * (self.D // 8)
        self.raw[page, :, blk, o:o + self.D // 8] = sz

    def get(self, page, t, side):
        """float32 [H][D] of one token's side."""
        blk, r = divmod(t, 16)
        c = np.empty((self.H, self.D), np.uint8)
        for ch in range(self.D):
            at, sh = self._code(side, r, ch)
            c[:, ch] = (self.raw[page, :, blk, at] >> sh) & 15
        o = side * 10 * self.D + 8 * self.D + r * (self.D // 8)
        sz = np.ascontiguousarray(self.raw[page, :, blk, o:o + self.D // 8]).view(np.float16).reshape(self.H, -1, 2)
        return stand_for(c, sz[..., 0], sz[..., 1])


def dequant_all(raw, D):
    """(k, v, v - z) float64 [pages][H][tokens][D] of page bytes, vectorised."""
    P, H, nb, _ = raw.shape
    ref = Pages(1, 1, D, 16)
    out = []
    for side in (0, 1):
        codes = np.empty((P, H, nb, 16, D), np.float64)
        for r in range(16):
            for ch in range(D):
                at, sh = ref._code(side, r, ch)
                codes[:, :, :, r, ch] = (raw[..., at] >> sh) & 15
        o = side * 10 * D + 8 * D
        sz = np.ascontiguousarray(raw[..., o:o + 2 * D]).view(np.float16).reshape(P, H, nb, 16, D // 32, 2)
        s = np.repeat(sz[..., 0].astype(np.float64), 32, -1)
        z = np.repeat(sz[..., 1].astype(np.float64), 32, -1)
        out.append((codes * s + z).reshape(P, H, nb * 16, D))
        if side:
            out.append((codes * s).reshape(P, H, nb * 16, D))
    return out


def attention(raw, table, kv_len, q_start, q, scale, page, D):
    """(out float64 [n][Hq][D], tolerance of the same shape).

    The tolerance is what the contract's roundings can do: half a bf16 step of the result;
    the fp16 operands of the tensor cores, 2^-11 of every key (the logit then moves by at most
    2^-11 sum |q k| scale) and on the value side either 2^-11 of a weight and 2^-11 of a value
    (2^-10 p |v|), or 2^-11 of the product weight * scale, which multiplies the code: the error
    is then 2^-11 p |code * s| whatever the zero point leaves of it in v = code * s + z (a token
    with v = 0.03 out of code * s = 2.6 moves by 2.6 * 2^-11 = 1.3e-3); fp32 sums, 2^-20 of the sum of magnitudes of a logit, and 2^-18 of the values' weighted
    magnitude for exp2 and the sums over up to some thousand tokens."""
    k_all, v_all, cs_all = dequant_all(raw, D)
    n, Hq = q.shape[0], q.shape[1]
    G = Hq // raw.shape[1]
    out, tol = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    for b in range(len(kv_len)):
        r0, r1 = int(q_start[b]), int(q_start[b + 1])
        L, T = int(kv_len[b]), r1 - r0
        if not T or not L:
            continue
        ids = table[b, : -(-L // page)]
        k = k_all[ids].transpose(1, 0, 2, 3).reshape(raw.shape[1], -1, D)[:, :L]
        v = v_all[ids].transpose(1, 0, 2, 3).reshape(raw.shape[1], -1, D)[:, :L]
        cs = cs_all[ids].transpose(1, 0, 2, 3).reshape(raw.shape[1], -1, D)[:, :L]
        for j in range(T):
            seen = L - T + j + 1
            if seen <= 0:
                continue
            for h in range(Hq):
                qq = q[r0 + j, h].astype(np.float64)
                kk, vv = k[h // G, :seen], v[h // G, :seen]
                x = kk @ qq * scale
                p = np.exp(x - x.max())
                p /= p.sum()
                o = p @ vv
                out[r0 + j, h] = o
                dx = (2.0 ** -11 + 2.0 ** -20) * (np.abs(kk) @ np.abs(qq)) * scale
                spread = (p * np.minimum(np.expm1(2 * dx), 2.0)) @ np.abs(vv - o)
                mag = p @ np.abs(vv)
                span = 2 * mag + p @ cs[h // G, :seen]
                tol[r0 + j, h] = np.abs(o) * 2.0 ** -8 + spread + 2.0 ** -11 * span + 2.0 ** -18 * mag + 2.0 ** -24
    return out, tol


def default_scale(D):
    return 1.0 / math.sqrt(D)
