"""Float64 references of prompt attention and the 4-bit cache (test infrastructure only).

Plain NumPy from the formulas: causal grouped-query attention with its log-sum-exp, the weight
that prompt tokens collect, the 4-bit group quantiser with its page format, decode attention over
quantised entries, and the order of eviction.
"""
from __future__ import annotations

import numpy as np


def prompt_attend(q, k, v):
    """One sequence: q [n][Hq][D], k, v [n][Hkv][D] -> out [n][Hq][D], lse [n][Hq], and for error
    bounds sum_j p |v| [n][Hq][D] and max_j sum_d |q k| / sqrt(D) [n][Hq]."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, aout = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, sabs = np.zeros((n, Hq)), np.zeros((n, Hq))
    see = np.tril(np.ones((n, n), bool))
    for h in range(Hq):
        kh, vh, qh = (x.astype(np.float64) for x in (k[:, h // G], v[:, h // G], q[:, h]))
        s = np.where(see, qh @ kh.T / np.sqrt(D), -np.inf)
        sabs[:, h] = np.where(see, np.abs(qh) @ np.abs(kh).T / np.sqrt(D), 0).max(1)
        m = s.max(1, keepdims=True)
        e = np.exp(s - m)
        l = e.sum(1, keepdims=True)
        lse[:, h] = (m + np.log(l))[:, 0]
        out[:, h], aout[:, h] = (e / l) @ vh, (e / l) @ np.abs(vh)
    return out, lse, aout, sabs


def prompt_mass(q, k, lse):
    """One sequence: mass [n][Hkv] from q [n][Hq][D], k [n][Hkv][D], lse [n][Hq]."""
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    mass = np.zeros((n, Hkv))
    see = np.tril(np.ones((n, n), bool))
    for h in range(Hq):
        s = q[:, h].astype(np.float64) @ k[:, h // (Hq // Hkv)].astype(np.float64).T / np.sqrt(D)
        mass[:, h // (Hq // Hkv)] += np.exp(np.where(see, s - lse[:, h:h + 1], -np.inf)).sum(0)
    return mass


def int4_quantize(x):
    """x [..., D] -> codes [..., D] uint8, scales, zeros [..., D / 32] float16. The steps are those of
    the definition, each rounded to float32 (a 64-bit step rounded once more to 32 is the 32-bit one)."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    f32 = lambda y: np.asarray(y, np.float32).astype(np.float64)
    s = f32(f32(g.max(-1) - g.min(-1)) / 15.0).astype(np.float32).astype(np.float16)
    z = g.min(-1).astype(np.float32).astype(np.float16)
    sf, zf = s.astype(np.float64)[..., None], z.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(sf > 0, np.clip(np.rint(f32(f32(g - zf) / sf)), 0, 15), 0)
    return c.reshape(x.shape).astype(np.uint8), s, z


def int4_values(codes, s, z):
    """Float64 values of codes [..., D] with scales and zeros [..., D / 32]."""
    c = codes.astype(np.float64).reshape(*codes.shape[:-1], codes.shape[-1] // 32, 32)
    return (c * s.astype(np.float64)[..., None] + z.astype(np.float64)[..., None]).reshape(codes.shape)


def int4_page(k, v):
    """The 20 D bytes of a page of 16 entries k, v [16][D], byte for byte."""
    D = k.shape[1]
    NG = D // 32
    page = np.zeros(20 * D, np.uint8)
    (kc, ks, kz), (vc, vs, vz) = int4_quantize(k), int4_quantize(v)
    halves = page[16 * D:].view(np.float16)
    for i in range(16):
        for g in range(NG):
            for t in range(4):
                for j in range(8):
                    page[i * D // 2 + (t * NG + g) * 4 + j // 2] |= kc[i, 32 * g + 8 * t + j] << (4 * (j % 2))
            for r in range(8):
                for j in range(4):
                    page[8 * D + i * D // 2 + (r * NG + g) * 2 + j // 2] |= vc[i, 32 * g + 4 * r + j] << (4 * (j % 2))
            hi, t, e = i // 8, (i % 8) // 2, i % 2
            halves[i * NG + g], halves[D // 2 + i * NG + g] = ks[i, g], kz[i, g]
            at = ((t * NG + g) * 2 + hi) * 2 + e
            halves[D + at], halves[3 * D // 2 + at] = vs[i, g], vz[i, g]
    return page


def int4_attend(q, k, v):
    """One unit: q [G][D], the entries' values k, v [L][D] -> out [G][D], weights p [L][G]."""
    G, D = q.shape
    if len(k) == 0:
        return np.zeros((G, D)), np.zeros((0, G))
    s = np.asarray(k, np.float64) @ np.asarray(q, np.float64).T / np.sqrt(D)
    e = np.exp(s - s.max(0))
    p = e / e.sum(0)
    return p.T @ np.asarray(v, np.float64), p


def int4_evict(mass, pos, seen, budget, recent):
    """One unit: the kept entries' indices, in order."""
    mass, pos = np.asarray(mass, np.float64), np.asarray(pos, np.int64)
    newest = pos >= int(seen) - recent

    def rank(i):
        if newest[i]:
            return (0, 0.0, i)
        return (2, 0.0, i) if np.isnan(mass[i]) else (1, -mass[i], i)
    return np.array(sorted(sorted(range(len(mass)), key=rank)[:budget]), np.int64)
