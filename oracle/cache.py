"""fp64 oracle of the target pass's cache: block tables as lists, the norm and
rotation, the 4-bit format from its bits, and attention one request at a time.

Plain and slow (numpy, one thread); shares no code with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------ block tables
class Tables:
    """The page pool and block tables of a batch."""

    def __init__(self, B, max_pages, free):
        self.width = max_pages
        self.rows = [[] for _ in range(B)]
        self.free = list(free)

    def plan(self, ctx, ell, G, P):
        """(q_start, kv_len, slot, pos, full)"""
        start, kv, slot, pos, full, dry = [0], [], [], [], False, False
        for b, (c, e) in enumerate(zip(ctx, ell)):
            row = self.rows[b]
            if c < 0:
                start.append(start[-1])
                kv.append(0)
                continue
            e = min(max(e, 0), G)
            n = min(e + 1, self.width * P - c)
            full |= n < e + 1
            need = max(0, -(-(c + n) // P) - len(row))
            dry |= need > len(self.free)
            if need and dry:
                full = True
                n = max(0, min(n, len(row) * P - c))
                need = 0
            for _ in range(need):
                row.append(self.free.pop())
            for t in range(c, c + n):
                pos.append(t)
                slot.append(row[t // P] * P + t % P)
            start.append(start[-1] + n)
            kv.append(c + n)
        pad = [-1] * (len(ctx) * (G + 1) - len(slot))
        return start, kv, slot + pad, pos + pad, full

    def commit(self, ctx, start, nout, done, P):
        out, back = [], []
        for b, c in enumerate(ctx):
            n = start[b + 1] - start[b]
            o = -1 if c < 0 or (done is not None and done[b]) else c + min(max(nout[b], 0), n)
            keep = -(-max(o, 0) // P)
            back += self.rows[b][keep:]
            self.rows[b] = self.rows[b][:keep]
            out.append(o)
        self.free += back[::-1]
        return out

    def table(self):
        t = np.full((len(self.rows), self.width), -1, np.int32)
        for b, r in enumerate(self.rows):
            t[b, : len(r)] = r
        return t


# ------------------------------------------------------- norm and rotation
def norm_rope(x, w, eps, pos, inv_freq, interleaved):
    """x [T, H, D], w [D] or None, pos [T], inv_freq [rot/2] -> fp64 [T, H, D]"""
    x = np.asarray(x, np.float64)
    y = x.copy() if w is None else x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    h = len(inv_freq)
    if h == 0:
        return y
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    ia = np.arange(0, 2 * h, 2) if interleaved else np.arange(h)
    ib = ia + 1 if interleaved else ia + h
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


# ------------------------------------------------------------ 4-bit format
def _e4m3_values():
    v = np.empty(128)
    for i in range(128):
        e, m = i >> 3, i & 7
        v[i] = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
    return v


E4M3 = _e4m3_values()          # magnitudes by code; code 127 (NaN) is never produced


def _nearest(x, grid):
    """Index of the nearest grid value, ties to the even index."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantise(x, g=1.0):
    """[..., D] -> (codes uint8 [..., D], scale codes uint8 [..., D/16])"""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), 0.0, x)
    y = x.reshape(*x.shape[:-1], -1, 16)
    with np.errstate(invalid="ignore", over="ignore"):
        sc = _nearest(np.minimum(np.abs(y).max(-1) / (6 * g), 448.0), E4M3[:127]).astype(np.uint8)
        s = (E4M3[sc] * g)[..., None]
        a = np.where(s > 0, np.minimum(np.abs(y) / np.where(s > 0, s, 1.0), 6.0), 0.0)
    code = _nearest(a, GRID).astype(np.uint8) | np.where((y < 0) & (s > 0), 8, 0).astype(np.uint8)
    return code.reshape(x.shape), sc


def dequantise(code, sc, g=1.0):
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    y = v.reshape(*v.shape[:-1], -1, 16) * (E4M3[sc & 127] * g)[..., None]
    return y.reshape(v.shape)


def write(cache, slot, k, v, P, kg=1.0, vg=1.0):
    """Store rows k, v [T, Hkv, D] at their slots of cache [pages, Hkv, R] (uint8, in place)."""
    D = k.shape[-1]
    half = P * D // 16 * 9
    for part, (x, g) in enumerate(((k, kg), (v, vg))):
        code, sc = quantise(x, g)
        byte = code[..., 0::2] | (code[..., 1::2] << 4)
        for t, s in enumerate(slot):
            if s < 0:
                continue
            pg, off = s // P, s % P
            for c in range(D // 32):
                at = part * half + c * P * 16 + off * 16
                cache[pg, :, at:at + 16] = byte[t, :, 16 * c:16 * c + 16]
            at = part * half + P * D // 2 + off * (D // 16)
            cache[pg, :, at:at + D // 16] = sc[t]


def read(cache, slot, P, D, kg=1.0, vg=1.0):
    """fp64 (k, v) [T, Hkv, D] of the slots."""
    half = P * D // 16 * 9
    slot = np.asarray(slot)
    pg, off = slot // P, slot % P
    out = []
    for part, g in ((0, kg), (1, vg)):
        rec = cache[pg][:, :, part * half:(part + 1) * half]
        t = np.arange(len(slot))
        codes = rec[:, :, :P * D // 2].reshape(len(slot), -1, D // 32, P, 16)[t, :, :, off]
        codes = codes.reshape(len(slot), -1, D // 2)
        nib = np.stack((codes & 15, codes >> 4), -1).reshape(len(slot), -1, D)
        sc = rec[:, :, P * D // 2:].reshape(len(slot), -1, P, D // 16)[t, :, off]
        out.append(dequantise(nib, sc, g))
    return out


# --------------------------------------------------------------- attention
def attention(q, cache, table, q_start, kv_len, P, scale, window=0, kg=1.0, vg=1.0):
    """q [T, Hq, D] -> (out, bound), both fp64 [rows, Hq, D] of the q_start[B] packed rows.

    bound: what a computation that rounds each probability to f16 and works in
    fp32 may be off by, before the output's own rounding."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    Hkv = cache.shape[1]
    grp = Hq // Hkv
    out = np.zeros((q_start[-1], Hq, D))
    bound = np.zeros_like(out)
    for b in range(len(kv_len)):
        n, L = int(q_start[b + 1]) - int(q_start[b]), int(kv_len[b])
        if n == 0 or L == 0:
            continue
        t = np.arange(L)
        k, v = read(cache, table[b][t // P].astype(np.int64) * P + t % P, P, D, kg, vg)
        for j in range(n):
            p_ = L - n + j
            lo = max(0, p_ - window + 1) if window > 0 else 0
            if p_ < lo:
                continue
            for h in range(Hq):
                kk, vv = k[lo:p_ + 1, h // grp], v[lo:p_ + 1, h // grp]
                qq = q[q_start[b] + j, h]
                x = kk @ qq * scale
                p = np.exp(x - x.max())
                p /= p.sum()
                out[q_start[b] + j, h] = p @ vv
                # scores: D products summed in fp32 (2^-23 a term, for sums that truncate)
                dx = D * 2.0 ** -23 * (np.abs(kk) @ np.abs(qq)).max() * abs(scale) + 2.0 ** -21 + \
                    2.0 ** -22 * np.abs(x - x.max()).max()
                # probabilities: half an f16 step each in the numerator and the sum, the score error twice, the
                # fp32 sums, and half of f16's smallest step, 2^-32 of the largest (lifted by 2^7), where p is subnormal
                rel = 2 * (2.0 ** -11 + dx) + len(p) * 2.0 ** -23
                bound[q_start[b] + j, h] = rel * (p @ np.abs(vv)) + 2 * len(p) * 2.0 ** -32 * p.max() * np.abs(vv).max()
    return out, bound
