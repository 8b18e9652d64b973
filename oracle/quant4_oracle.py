"""fp64 oracle of rotary positions and of the 4-bit block cache (numpy; test infrastructure only).

Written from the definitions in ``include/nosa.h``: the rotation, the unit's layout, the
quantisation rule and masked attention.
"""
from __future__ import annotations

import numpy as np

B = 64
f32, f16 = np.float32, np.float16


def unit_bytes(d: int) -> int:
    raw = 71 * d + 4 * B + 8
    return raw + (-raw) % 32


# ---- rotation ----
def rotate(x, table, positions, axes, interleaved, round_to, backward=False):
    """Rows x [batch][n][heads][d] by positions [axes][batch][n]; every product and sum is rounded to
    fp32 and the result by `round_to` (None: nothing is rounded)."""
    F = np.float64 if round_to is None else f32
    y = np.array(x, dtype=F)
    pairs = table.shape[1]
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        p = np.clip(positions[axes[i] if axes is not None else 0], 0, len(table) - 1)
        c, s = (table[p, i, k].astype(F)[:, :, None] for k in (0, 1))
        if backward:
            s = -s
        u, v = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y if round_to is None else np.asarray(round_to(y))


# ---- layout ----
def code_places(d: int):
    """Byte offsets [64][d] and bit shifts [64][d] of the key codes, and of the value codes."""
    t, x = np.arange(B)[:, None], np.arange(d)[None]
    tt = t % 16
    word = lambda m, lane, w: 512 * m + 16 * lane + 4 * w  # noqa: E731
    kw = word(x // 16, 4 * (2 * (tt // 4) + tt % 2) + x % 16 // 4, t // 16)
    kn = tt % 4 // 2 + 2 * (x % 4 // 2) + 4 * (x % 2)
    vw = 32 * d + word(x // 16, 4 * (x % 8) + tt // 4, t // 16)
    vn = x % 16 // 8 + 2 * (t % 4 // 2) + 4 * (t % 2)
    return (kw + kn // 2, 4 * (kn % 2)), (vw + vn // 2, 4 * (vn % 2))


def order(n: int):
    """Place of each of n steps (or zeros)."""
    x = np.arange(n)
    return 4 * (x % 16 // 4 * (n // 16) + x // 16) + x % 4


def places(d: int):
    """Byte offsets: key steps [d], key zeros [d], value steps [64][d / 64], value zeros."""
    o, run = order(d), 64 * np.arange(d // 64)[None] + order(64)[:, None]
    return 64 * d + o, 65 * d + 2 * o, 67 * d + 2 * run, 69 * d + 2 * run


def _f16(units, at):
    return (units[:, at].astype(np.uint16) | units[:, at + 1].astype(np.uint16) << 8).view(f16).astype(np.float64)


def parts(units, d: int):
    """Codes, steps, zeros of keys ([n][64][d], [n][1][d] twice) and of values ([n][64][d] three times),
    scales [n][2], logits [n][64] of unit images [n][bytes]."""
    (kb, ks), (vb, vs) = code_places(d)
    p = places(d)
    kstep = (units[:, p[0]].astype(np.uint16) << 8).view(f16).astype(np.float64)[:, None]
    vals = [np.repeat(_f16(units, q), 64, axis=2) for q in p[2:]]
    at = 71 * d
    e = np.ascontiguousarray(units[:, at:at + 4 * B]).view(f32).astype(np.float64)
    scales = np.ascontiguousarray(units[:, at + 4 * B:at + 4 * B + 8]).view(f32).astype(np.float64)
    return ((units[:, kb] >> ks & 15).astype(np.float64), kstep, _f16(units, p[1])[:, None]), \
        ((units[:, vb] >> vs & 15).astype(np.float64), *vals), scales, e


def decode(units, d: int):
    """keys, values [n][64][d], logits [n][64], and what bounds an error: step * n + |zero| of both."""
    k, v, s, e = parts(units, d)
    with np.errstate(invalid="ignore"):
        out = [(c * st + z) * s[:, i, None, None] for i, (c, st, z) in enumerate((k, v))]
        size = [(c * st + np.abs(z)) * s[:, i, None, None] for i, (c, st, z) in enumerate((k, v))]
    return out[0], out[1], e, size[0], size[1]


# ---- quantisation ----
def down16(x):
    h = x.astype(f16)
    return np.where(h.astype(np.float64) > x, np.nextafter(h, f16(-np.inf)), h)


def up16(x, drop=0):
    h = x.astype(f16)
    h = np.where(h.astype(np.float64) < x, np.nextafter(h, f16(np.inf)), h)
    bits = h.view(np.uint16).astype(np.uint32)
    low = (1 << drop) - 1
    return ((bits + low) & ~np.uint32(low)).astype(np.uint16).view(f16)


def _group(y, drop):
    """Codes, step, zero of groups y [g][m] (masked elements NaN)."""
    some = ~np.isnan(y).all(1)
    yy = np.where(some[:, None], y, 0.0)
    zero = down16(np.fmin.reduce(yy, 1) + 0.0)
    room = (np.fmax.reduce(yy, 1) - zero.astype(np.float64)).astype(f32) * (f32(1) / f32(15))
    step = up16(room.astype(np.float64), drop)
    inv = np.divide(f32(1), step.astype(f32), out=np.zeros(len(y), f32), where=step > 0)
    n = np.rint((yy - zero.astype(np.float64)[:, None]).astype(f32).astype(np.float64) * inv.astype(np.float64)[:, None])
    return np.nan_to_num(n).astype(np.uint8), step, zero


def encode(k, v, e):
    """Unit images of blocks k, v [n][64][d], e [n][64]."""
    n, _, d = k.shape
    out = np.zeros((n, unit_bytes(d)), np.uint8)
    (kb, ks), (vb, vs) = code_places(d)
    p = places(d)

    def put(at, h):
        bits = np.ascontiguousarray(h).view(np.uint16)
        out[:, at], out[:, at + 1] = bits & 255, bits >> 8

    def codes(at, shift, c):  # two codes of a byte
        for half in (0, 4):
            own = shift == half
            out[:, at[own]] |= c[:, own] << np.uint8(half)

    live = ~np.isneginf(e)
    scales = np.zeros((n, 2), f32)
    for i, x in enumerate((k, v)):
        with np.errstate(invalid="ignore"):
            top = np.where(live[..., None], np.abs(x), 0.0).max((1, 2))
            ok = np.isfinite(top) & (top >= 2.0 ** -100)
            power = 2.0 ** (np.frexp(np.where(ok, top, 1.0))[1] - 3)
            scales[:, i] = np.where(ok, power, np.where(np.isfinite(top), 0.0, np.nan))
            y = np.where(live[..., None] & ok[:, None, None], x / power[:, None, None], np.nan)
        if i == 0:
            c, st, z = _group(y.transpose(0, 2, 1).reshape(-1, B), 8)
            codes(kb, ks, c.reshape(n, d, B).transpose(0, 2, 1))
            out[:, p[0]] = st.reshape(n, d).view(np.uint16) >> 8
            put(p[1], z.reshape(n, d))
        else:
            c, st, z = _group(y.reshape(-1, 64), 0)
            codes(vb, vs, c.reshape(n, B, d))
            put(p[2], st.reshape(n, B, d // 64))
            put(p[3], z.reshape(n, B, d // 64))
    at = 71 * d
    out[:, at:at + 4 * B] = np.ascontiguousarray(e.astype(f32)).view(np.uint8)
    out[:, at + 4 * B:at + 4 * B + 8] = scales.view(np.uint8)
    return out


def attend(q, K, V, e, sees, Ks, Vs):
    """Rows q [R][d] over tokens K, V [n][d], e [n]; row r sees the first sees[r] tokens.
    Returns out [R][d], lse [R], weights [R][n], and for error bounds the weighted mean of Vs [R][d]
    and the largest sum |q_x| Ks_x / sqrt(d) over the visible tokens [R]."""
    R, d = q.shape
    n = K.shape[0]
    out, mean = np.zeros((R, d)), np.zeros((R, d))
    lse, w, size = np.full(R, -np.inf), np.zeros((R, n)), np.zeros(R)
    for r in range(R):
        ids = np.flatnonzero(~np.isneginf(e) & (np.arange(n) < sees[r]))
        if not ids.size:
            continue
        with np.errstate(invalid="ignore"):
            l = K[ids] @ q[r] / np.sqrt(d) + e[ids]
            size[r] = (Ks[ids] @ np.abs(q[r])).max() / np.sqrt(d)
            m = l.max()
            p = np.exp(l - m)
            lse[r] = m + np.log(p.sum())
            p /= p.sum()
        w[r, ids] = p
        out[r] = p @ V[ids]
        mean[r] = p @ Vs[ids]
    return out, lse, w, mean, size
