"""A chunk of new tokens past a paged cache, in float64: the QKV rows' norm, rotation and
placing (append), and the attention of the chunk's rows, with an elementwise bound on how far a
float32 evaluation with rounded weights may be from it. Written from the definitions; shares no
code with the kernels."""
import numpy as np

from . import bf16_from_f64, bf16_to_f64


def rotated_heads(x, w, eps, pos, theta):
    """Heads x [H, D] (BF16 bits) of one token: normed (where w is given) and rotated, BF16 bits."""
    x = bf16_to_f64(x)
    D = x.shape[-1]
    if w is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + float(np.float32(eps))) * bf16_to_f64(w)
        x = bf16_to_f64(bf16_from_f64(x))
    a = pos * theta ** (-2.0 * np.arange(D // 2) / D)
    c, s = np.cos(a), np.sin(a)
    lo, hi = x[:, :D // 2], x[:, D // 2:]
    return bf16_from_f64(np.concatenate((lo * c - hi * s, hi * c + lo * s), axis=-1))


def append(qkv, Hq, Hkv, D, positions, max_pos, theta, q_norm_w=None, k_norm_w=None, eps=1e-6):
    """q_rot [T, Hq, D], k and v [T, Hkv, D] (BF16 bits) and which tokens have a place."""
    T = qkv.shape[0]
    x = np.ascontiguousarray(qkv[:, :(Hq + 2 * Hkv) * D]).reshape(T, Hq + 2 * Hkv, D)
    q = np.zeros((T, Hq, D), np.uint16)
    k = np.zeros((T, Hkv, D), np.uint16)
    live = (positions >= 0) & (positions < max_pos)
    for t in np.flatnonzero(live):
        q[t] = rotated_heads(x[t, :Hq], q_norm_w, eps, int(positions[t]), theta)
        k[t] = rotated_heads(x[t, Hq:Hq + Hkv], k_norm_w, eps, int(positions[t]), theta)
    return q, k, x[:, Hq + Hkv:], live


def attention(q, K, V, block_table, ctx_lens, q_starts, page, scale=None, kind="bf16"):
    """Chunk attention of q [T, Hq, D] (BF16 bits) over cache rows K, V [slots, Hkv, D] (float64):
    out [T, Hq, D] (NaN rows marked by NaN; rows of no request 0), the bound on the distance of a
    kernel's result before its last rounding, and which rows belong to a request.

    The bound, u = 2^-24:
      scores: D + 16 roundings of sum |q k|; with FP16 operands (INT8, 4-bit) K's value and an INT8
        scale's rounding, 2^-11 each of |q k|, and 2^-25 of the block's largest |K| times |q| and
        the row's largest |q| times |K| for what FP16 cannot hold; d(exp) = exp d(score), and 2^-21
        for the exponential;
      weights: 2^-8 (BF16) or 2^-11 (FP16) of themselves, and for FP16 2^-24 of the largest;
      values: as K's, the largest so far in their place;
      sums: 2^-20 of their absolute terms."""
    q = bf16_to_f64(q)
    T, Hq, D = q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    blocks = K.shape[0] // page
    out, bound = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    owned = np.zeros(T, bool)
    f16 = kind != "bf16"
    for b in range(len(ctx_lens)):
        r0 = min(max(int(q_starts[b]), 0), T)
        n = max(min(int(q_starts[b + 1]), T) - r0, 0)
        ctx = int(ctx_lens[b])
        if ctx < 0 or ctx > block_table.shape[1] * page:
            ctx = 0
        owned[r0:r0 + n] = True
        if n == 0 or ctx == 0:
            continue
        t = np.arange(ctx)
        blk = block_table[b][t // page]
        ok = (blk >= 0) & (blk < blocks)
        slot = np.where(ok, blk, 0) * page + t % page
        seen = t[None] <= (ctx - n + np.arange(n))[:, None]                 # [n, ctx]
        some = seen.any(1)
        for h in range(Hkv):
            k, v = (np.where(ok[:, None], x[slot, h], 0.0) for x in (K, V))
            for g in range(h * G, (h + 1) * G):
                x = q[r0:r0 + n, g]
                with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
                    s = np.where(seen, scale * (x @ k.T), -np.inf)
                    p = np.exp(s - s.max(1, keepdims=True, initial=-1e308))
                    p = np.where(seen, p, 0.0)
                    w = p / p.sum(1, keepdims=True)
                    # (a value no row's weight reaches counts for nothing)
                    o = np.stack([np.where(seen[i, :, None], w[i, :, None] * v, 0.0).sum(0)
                                  for i in range(n)]) if not np.isfinite(v).all() else w @ v
                    vf = np.where(np.isfinite(v), v, 0.0)
                    kf = np.where(np.isfinite(k), k, 0.0)
                    a = np.abs(x)
                    mag = a @ np.abs(kf).T
                    ds = abs(scale) * (D + 16) * 2.0 ** -24 * mag
                    dv = 0.0
                    if f16:
                        kmax = np.abs(kf).max()
                        ds += abs(scale) * (2.0 ** -10 * mag + 2.0 ** -25 * kmax * a.sum(1, keepdims=True)
                                            + 2.0 ** -25 * a.max(1, keepdims=True) * np.abs(kf).sum(1)[None])
                        dv = 2.0 ** -10 * (w @ np.abs(vf)) + 2.0 ** -25 * np.abs(vf).max()
                    dw = w * (np.expm1(np.minimum(ds, 50.0)) + 2.0 ** -21)
                    rw = w * (2.0 ** -11 if f16 else 2.0 ** -8)
                    if f16:
                        rw = rw + np.where(seen, 2.0 ** -24 * w.max(1, keepdims=True), 0.0)
                    e = (dw + rw) @ np.abs(vf) + dw.sum(1, keepdims=True) * np.abs(o) \
                        + 2.0 ** -20 * (w @ np.abs(vf)) + dv
                out[r0:r0 + n, g] = np.where(some[:, None], o, 0.0)
                bound[r0:r0 + n, g] = np.where(some[:, None], e, 0.0)
    return out, bound, owned
