"""fp64 CPU oracle of the 4-bit key/value cache and of attention over it.

Plain numpy, no code shared with the library.  The storing rule's roundings
(the scale to bf16, the reciprocal and the quotient to fp32) are emulated
exactly; everything else is fp64.
"""

from __future__ import annotations

import numpy as np

from .qlora_oracle import fp4_levels_f32, nf4_levels_f32, uniform4_levels_f32

BLOCK = 64
BF16_MAX_BITS = np.uint16(0x7F7F)


def levels_f32(table: int) -> np.ndarray:
    return np.asarray((nf4_levels_f32, uniform4_levels_f32, fp4_levels_f32)[table](), dtype=np.float32)


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """fp32 -> bf16 bits, round to nearest even (finite input)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bits_f64(b: np.ndarray) -> np.ndarray:
    return (np.asarray(b, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def store(x: np.ndarray, table: int):
    """x fp32 [..., D] -> (codes uint8 [..., D/2], scale bits uint16 [..., D/64])."""
    x = np.asarray(x, dtype=np.float32)
    runs = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = np.max(np.abs(runs), axis=-1)                      # NaN stays NaN
    ok = np.isfinite(top)
    sb = np.minimum(bf16_bits(np.where(ok, top, 0)), BF16_MAX_BITS)
    sb = np.where(ok & (top < np.float32(2.0 ** -126)), np.uint16(0), sb)
    s = bits_f64(sb)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        r = np.where(s > 0, 1.0 / np.where(s > 0, s, 1.0), 0.0).astype(np.float32).astype(np.float64)
        q = (runs.astype(np.float64) * r[..., None]).astype(np.float32).astype(np.float64)
    lv = levels_f32(table).astype(np.float64)
    code = np.sum(q[..., None] > (lv[1:] + lv[:-1]) / 2, axis=-1).astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(ok, sb, np.uint16(0x7FC0))


def values(codes: np.ndarray, scale_bits: np.ndarray, table: int) -> np.ndarray:
    """fp64 values of packed codes; level * scale is exact in fp64."""
    code = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = levels_f32(table).astype(np.float64)[code]
    return (v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK) * bits_f64(scale_bits)[..., None]).reshape(v.shape)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, causal: bool, window: int, absent=None):
    """One sequence: q [n, Hq, D], k, v [len, Hkv, D] fp64, absent [len] (positions nobody sees).

    Returns out [n, Hq, D], lse [n, Hq], spread [n, Hq, D] = sum_j p_j |v_j| and
    size [n, Hq] = max_j sum_d |scale q_d k_jd| over the seen positions.
    """
    n, hq, d = q.shape
    length, hkv, _ = k.shape
    out = np.zeros((n, hq, d))
    spread = np.zeros((n, hq, d))
    lse = np.full((n, hq), -np.inf)
    size = np.zeros((n, hq))
    j, p = np.arange(length), length - n + np.arange(n)[:, None]
    seen = np.ones((n, length), bool) if absent is None else np.repeat(~absent[None], n, 0)
    if causal:
        seen &= j <= p
    if window > 0:
        seen &= j > p - window
    # queries that see a position which is not finite: by themselves, over what they see alone
    odd = ~(np.isfinite(k).all((1, 2)) & np.isfinite(v).all((1, 2)))
    alone = seen[:, odd].any(1)
    kf, vf = np.where(odd[:, None, None], 0.0, k), np.where(odd[:, None, None], 0.0, v)
    for h in range(hq):
        for rows, keys in [(np.flatnonzero(seen.any(1) & ~alone), slice(None))] + \
                [(np.array([i]), seen[i]) for i in np.flatnonzero(alone)]:
            if not len(rows):
                continue
            ks, vs = ((x if alone[rows[0]] else y)[keys, h // (hq // hkv)] for x, y in ((k, kf), (v, vf)))
            there = seen[rows][:, keys]
            s = np.where(there, q[rows, h] @ ks.T * scale, -np.inf)
            m = s.max(1, keepdims=True)
            w = np.exp(s - m)
            t = w.sum(1, keepdims=True)
            out[rows, h] = w @ vs / t
            spread[rows, h] = w @ np.abs(vs) / t
            lse[rows, h] = (m + np.log(t))[:, 0]
            size[rows, h] = np.where(there, np.abs(q[rows, h]) @ np.abs(ks).T * abs(scale), 0.0).max(1)
    return out, lse, spread, size
