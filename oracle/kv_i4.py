"""The 4-bit KV cache and its decode attention, in float64 from their definition.

A row of D values is held as codes c and a pair (s, m) and stands for
c s + m: m = min x, s = bf16((max x - m) / 15), c = clamp(rne((x - m) / s), 0,
15), with the difference, the quotient by 15 and the quotient by s each
rounded to float32 as the definition says (a float64 quotient of two float32
values, rounded to float32, is the float32 quotient: 53 >= 2 * 24 + 2 bits).
Test infrastructure: it shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def bf16_to_f64(h) -> np.ndarray:
    return (np.asarray(h, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f32_to_bf16(x) -> np.ndarray:
    """BF16 bit patterns of float32 values, ties to even (finite values, infinities)."""
    u = np.asarray(x, np.float32).view(np.uint32)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(np.asarray(x, np.float32)), np.uint16(0x7FC0), r)


def quant_rows(x_bf16):
    """codes [..., D / 2] uint8 and meta [..., 2] (BF16 bits of s, m) of rows [..., D]."""
    with np.errstate(all="ignore"):
        x = bf16_to_f64(x_bf16)
        lo = x.min(-1, keepdims=True)
        rng = (x.max(-1, keepdims=True) - lo).astype(np.float32)
        s16 = f32_to_bf16((rng.astype(np.float64) / 15.0).astype(np.float32))
        s = bf16_to_f64(s16)
        d = (x - lo).astype(np.float32).astype(np.float64)
        q = np.where(s > 0, (d / np.where(s > 0, s, 1.0)).astype(np.float32), 0.0)
        c = np.clip(np.rint(q.astype(np.float64)), 0, 15)
    bad = ~np.isfinite(rng)
    c = np.where(bad, 0, c).astype(np.uint8)
    lo16 = (lo.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)   # exact: a BF16 value
    nan = np.uint16(0x7FC0)
    meta = np.concatenate((np.where(bad, nan, s16), np.where(bad, nan, lo16)), axis=-1)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8), meta.astype(np.uint16)


def unpack(codes) -> np.ndarray:
    codes = np.asarray(codes, np.uint8)
    return np.stack((codes & 15, codes >> 4), axis=-1).reshape(*codes.shape[:-1], -1)


def dequant_rows(codes, meta) -> np.ndarray:
    """The float64 values c s + m (exact: 4 + 8 bits, then a sum of two such values)."""
    m = bf16_to_f64(meta)
    return unpack(codes) * m[..., :1] + m[..., 1:]


def kv_write(k, v, slots, k_codes, v_codes, k_meta, v_meta) -> int:
    """Rows k, v [T, Hkv, D] into the caches at slots [T]; the number of slots out of range."""
    bad = 0
    for t, slot in enumerate(np.asarray(slots)):
        if slot < 0:
            continue
        if slot >= k_codes.shape[0]:
            bad += 1
            continue
        k_codes[slot], k_meta[slot] = quant_rows(k[t])
        v_codes[slot], v_meta[slot] = quant_rows(v[t])
    return bad


def attention(q, k_codes, v_codes, k_meta, v_meta, block_table, ctx_lens, page, scale=None):
    """Decode attention [B, Hq, D] in float64, and an elementwise bound on how far a float32
    evaluation that takes the weights p s to FP16 may be from it:

      scores: at most (D + 16) roundings of 2^-24 of sum |q| |c s| + |m| sum |q| (the codes' and
        the minimum's part apart, as they are added), and 2^-34 of max |q| where q's smallest
        parts leave FP16's range; d(exp) = exp d(score), and 2^-21 for the exponential itself;
      weights: 2^-11 relative to p s, times the code; 2^-34 of the largest p s per token (below
        FP16's range);
      sums: 2^-20 of their absolute terms;
      a bad block id counts as rows of zeros."""
    q = bf16_to_f64(q)
    B, Hq, D = q.shape
    Hkv = k_codes.shape[1]
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    blocks = k_codes.shape[0] // page
    out, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b in range(B):
        n = int(ctx_lens[b])
        if n <= 0 or n > block_table.shape[1] * page:
            continue
        t = np.arange(n)
        blk = block_table[b][t // page]
        ok = (blk >= 0) & (blk < blocks)
        slot = np.where(ok, blk, 0) * page + t % page
        for h in range(Hkv):
            km, vm = bf16_to_f64(k_meta[slot, h]), bf16_to_f64(v_meta[slot, h])
            km, vm = np.where(ok[:, None], km, 0.0), np.where(ok[:, None], vm, 0.0)
            kc, vc = unpack(k_codes[slot, h]) * 1.0, unpack(v_codes[slot, h]) * 1.0
            K, V = kc * km[:, :1] + km[:, 1:], vc * vm[:, :1] + vm[:, 1:]
            for g in range(G):
                x = q[b, h * G + g]
                with np.errstate(invalid="ignore"):
                    s = scale * (K @ x)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    o = p @ V
                    a = np.abs(x)
                    mag = (kc @ a) * np.abs(km[:, 0]) + np.abs(km[:, 1]) * a.sum()
                    ds = abs(scale) * ((D + 16) * 2.0 ** -24 * mag
                                       + 2.0 ** -34 * a.max() * kc.sum(1) * np.abs(km[:, 0]))
                    dp = p * (np.expm1(np.minimum(ds, 50.0)) + 2.0 ** -21)
                    w = p * np.abs(vm[:, 0])
                    bound[b, h * G + g] = (dp @ np.abs(V) + dp.sum() * np.abs(o)
                                           + 2.0 ** -11 * (w @ vc) + 2.0 ** -34 * w.max() * vc.sum(0)
                                           + 2.0 ** -20 * (p @ (np.abs(vm[:, :1]) * vc
                                                                + np.abs(vm[:, 1:]))))
                out[b, h * G + g] = o
    return out, bound
