"""fp64 numpy definitions of the operators between two LUT linears (residual
norm, low-rank adapters, rotary positions) and the error bounds their kernels
are held to."""
import numpy as np

U24 = 2.0 ** -24     # half a step of fp32, relative


def f64(t):
    return t.detach().cpu().numpy().astype(np.float64)


# ---------------------------------------------------------------- residual norm


def norm(v, kind, w, b, eps):
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    v = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    if w is not None:
        v = v * w
    return v if b is None else v + b


def residual_norm(resid, y, kind, eps, pre, post, gate, rs, bs):
    """resid numpy fp16 / fp32, the rest fp64 arrays; pre / post: (w, b) or None.
    Returns (r', x) in the stored types."""
    r = resid
    if y is not None:
        v = y if post is None else norm(y, kind, post[0], post[1], eps)
        if gate is not None:
            v = v * gate
        r = (rs * resid.astype(np.float64) + bs * v).astype(resid.dtype)
    x = norm(r.astype(np.float64), kind, pre[0], pre[1], eps)
    return r, x.astype(np.float16)


# ---------------------------------------------------------------- low-rank adapters


def lora_add(x, ids, a, b, scale, ranks, y):
    """All fp64 (ids, ranks int).  Returns (out, bound).

    The bound adds up, with u = 2^-24 and 2u for an addition inside the tensor
    core (it may truncate):
      t_j = sum_k x a: products exact; a chain of at most K/16 + 64 additions
        (K/16 steps of one warp, then warps and CTAs) -> 2u (K/16 + 64) sum|x a|
      t carried with 20 bits of its row's largest entry -> 2^-20 max|t|
      sum over r <= 128 entries: at most r + 8 additions and the two products
        by scale -> 2u (r + 12) |scale| sum|b t|
      the addition to y -> u |out|, and u |y| for a product rounded before it."""
    M, K = x.shape
    out, tol = y.copy(), np.zeros_like(y)
    for m in range(M):
        i = ids[m]
        if i < 0 or i >= a.shape[0]:
            continue
        k = int(np.clip(ranks[i], 0, a.shape[1]))
        A, B = a[i, :k], b[i, :, :k]
        t = A @ x[m]
        out[m] += scale[i] * (B @ t)
        if k:
            dt = 2 * U24 * (K / 16 + 64) * (np.abs(A) @ np.abs(x[m])) + 2.0 ** -20 * np.abs(t).max()
            tol[m] = abs(scale[i]) * (np.abs(B) @ dt + 2 * U24 * (k + 12) * (np.abs(B) @ np.abs(t)))
        tol[m] += U24 * (np.abs(out[m]) + np.abs(y[m]))
    return out, tol


# ---------------------------------------------------------------- rotary positions


def rope_qkv(qkv, positions, inv_freq, nq, nkv, D, interleaved, attn_scale, qw, kw, eps):
    """All fp64.  Returns ((q, k, v), (bounds)).

    Before its rounding a value is off by at most 1.6e-6 attn_scale (|a| + |b|)
    of its pair: the reduced angle rounded to fp32 (at most half a turn:
    pi 2^-24 = 1.9e-7 rad), sincospi (2 ulp: 2.4e-7), the two products, the sum
    and attn_scale (4 * 2^-24 = 2.4e-7), and the norm (a sum of at most 256
    squares in a tree of 8 + 5 additions, halved by the root, a division, a root
    and two products: (13 / 2 + 4) * 2^-24 = 6.3e-7, rounded up).  The rounding
    to fp16 adds 2^-11 of the value, or half the smallest step 2^-25."""
    M = qkv.shape[0]
    z = qkv.reshape(M, nq + 2 * nkv, D).copy()
    for lo, hi, w in ((0, nq, qw), (nq, nq + nkv, kw)):
        if w is not None:
            t = z[:, lo:hi]
            z[:, lo:hi] = t / np.sqrt((t * t).mean(-1, keepdims=True) + eps) * w
    size = np.abs(z)
    if inv_freq is not None:
        half = len(inv_freq)
        i = np.arange(half)
        p, s = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = positions[:, None, None] * inv_freq
        c, sn = np.cos(ang) * attn_scale, np.sin(ang) * attn_scale
        t = z[:, : nq + nkv]
        a, b = t[..., p].copy(), t[..., s].copy()
        t[..., p], t[..., s] = a * c - b * sn, a * sn + b * c
        both = attn_scale * (np.abs(a) + np.abs(b))
        size[:, : nq + nkv][..., p] = both
        size[:, : nq + nkv][..., s] = both
    tol = 1.6e-6 * size + 2.0 ** -11 * np.abs(z) * (1 + 1e-6) + 2.0 ** -25
    cut = (slice(0, nq), slice(nq, nq + nkv), slice(nq + nkv, None))
    return tuple(z[:, c] for c in cut), tuple(tol[:, c] for c in cut)
