"""fp64 oracle of the 8-bit block cache (numpy; test infrastructure only).

Written from the definitions in ``include/nosa.h``: the unit's layout, the e4m3
numbers, the quantisation rule, masked attention and the eviction rule.
"""
from __future__ import annotations

import numpy as np

B = 64


def unit_bytes(d: int) -> int:
    raw = 2 * B * d + 4 * B + 8
    return raw + (-raw) % 32


def code_offsets(d: int):
    """Byte offsets [64][d] of the key codes and of the value codes."""
    t, x = np.arange(B)[:, None], np.arange(d)[None]
    tt = t % 16
    key = 16 * (32 * (x // 32) + 4 * (2 * (tt // 4) + tt % 2) + x % 16 // 4) + 4 * (2 * (x % 32 // 16) + tt % 4 // 2) + x % 4
    val = 16 * d + 16 * (32 * (x // 32) + 4 * (x % 8) + tt // 4) + 4 * (x % 32 // 8) + tt % 4
    base = 32 * d * (t // 16)
    return base + key, base + val


def e4m3_values() -> np.ndarray:
    """The number that each of the 256 codes stands for (1-4-3 bits, bias 7, no infinities)."""
    c = np.arange(256)
    exp, man = (c >> 3) & 15, c & 7
    v = np.where(exp == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * 2.0 ** (exp - 7.0))
    v = np.where((exp == 15) & (man == 7), np.nan, v)
    return np.where(c & 128, -v, v)


E4M3 = e4m3_values()
_POS = E4M3[:127]  # ascending: 0 .. 448


def nearest_distance(y: np.ndarray) -> np.ndarray:
    """Distance of each y to the nearest e4m3 number."""
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    return np.minimum(np.abs(_POS[hi] - a), np.abs(a - _POS[lo])) + (np.abs(y) - a)


def decode(units: np.ndarray, d: int):
    """(key numbers, value numbers [n][64][d], logits [n][64], scales [n][2]) of unit images [n][bytes]."""
    ko, vo = code_offsets(d)
    e = np.ascontiguousarray(units[:, 2 * B * d:2 * B * d + 4 * B]).view(np.float32).astype(np.float64)
    s = np.ascontiguousarray(units[:, 2 * B * d + 4 * B:2 * B * d + 4 * B + 8]).view(np.float32).astype(np.float64)
    return E4M3[units[:, ko]], E4M3[units[:, vo]], e, s


def encode(k, v, e) -> np.ndarray:
    """Unit images of blocks k, v [n][64][d], e [n][64] (finite values; ties to even)."""
    n, _, d = k.shape
    out = np.zeros((n, unit_bytes(d)), np.uint8)
    ko, vo = code_offsets(d)
    live = ~np.isneginf(e)[..., None]
    scales = np.zeros((n, 2), np.float32)
    for i, (x, at) in enumerate(((k, ko), (v, vo))):
        x = np.where(live, x, 0.0)
        scales[:, i] = np.abs(x).max((1, 2)) / 448
        s = scales[:, i].astype(np.float64)[:, None, None]
        y = np.divide(x, s, out=np.zeros_like(x), where=s > 0)
        a = np.minimum(np.abs(y), 448.0)
        hi = np.clip(np.searchsorted(_POS, a), 1, 126)
        dl, dh = a - _POS[hi - 1], _POS[hi] - a
        up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
        code = np.where(up, hi, hi - 1) | np.where(y < 0, 128, 0)
        for b in range(n):
            out[b, at] = code[b]
    out[:, 2 * B * d:2 * B * d + 4 * B] = np.ascontiguousarray(e.astype(np.float32)).view(np.uint8)
    out[:, 2 * B * d + 4 * B:2 * B * d + 4 * B + 8] = scales.view(np.uint8)
    return out


def attend(q, K, V, e, sees):
    """Rows q [R][d] over tokens K, V [n][d], e [n]; row r sees the first sees[r] tokens.
    Returns out [R][d], lse [R], weights [R][n], and for error bounds the weighted mean
    of |v| [R][d] and the largest sum |q_x k_x| / sqrt(d) over the visible tokens [R]."""
    R, d = q.shape
    n = K.shape[0]
    out, mean_abs = np.zeros((R, d)), np.zeros((R, d))
    lse, w, size = np.full(R, -np.inf), np.zeros((R, n)), np.zeros(R)
    for r in range(R):
        ids = np.flatnonzero(~np.isneginf(e) & (np.arange(n) < sees[r]))
        if not ids.size:
            continue
        with np.errstate(invalid="ignore"):
            l = K[ids] @ q[r] / np.sqrt(d) + e[ids]
            size[r] = (np.abs(K[ids]) @ np.abs(q[r])).max() / np.sqrt(d)
            m = l.max()
            p = np.exp(l - m)
            lse[r] = m + np.log(p.sum())
            p /= p.sum()
        w[r, ids] = p
        out[r] = p @ V[ids]
        mean_abs[r] = p @ np.abs(V[ids])
    return out, lse, w, mean_abs, size


def evict(tab, mass, n, budget, recent):
    """One unit: (table row, mass row, length, order) after eviction."""
    cap = len(tab)
    full = n // B
    over = max(0, full - budget)
    rank = lambda i: (np.isnan(mass[i]), 0.0 if np.isnan(mass[i]) else float(mass[i]), -i)  # noqa: E731
    gone = set(sorted(range(full - recent), key=rank)[:over]) if over else set()
    order = [i for i in range(full) if i not in gone] + sorted(gone) + list(range(full, cap))
    new = np.array(mass, dtype=np.float32)
    if over:
        new[:full - over] = [mass[i] for i in order[:full - over]]
        tail = mass[full] if full < cap else 0.0
        new[full - over:min(full + 1, cap)] = 0.0
        new[full - over] = tail
    return np.array([tab[i] for i in order], dtype=np.int32), new, n - B * over, np.array(order, np.int32)
