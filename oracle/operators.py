"""Float64 oracle of the operators around the expert FFN: products of NVFP4 weights with
unquantized activations, the router's balance loss, and the norms around a block.

Each is written from its definition.  Where a test needs an error bound, the functions also give
the sum of magnitudes that a rounding in the sum is relative to.
"""

import numpy as np


def linear(x, w):
    """x (M, K) times w (N, K) transposed: (result, sum of |x||w|)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def moe_ffn(x, ids, weights, w1, w2):
    """The expert FFN on (T, H) activations with (T, k) routing (ids outside [0, E) dropped); w1
    (E, 2I, H) gate rows then up rows, w2 (E, H, I).

    Returns (out, bound): bound is how far float32 sums (relative error cs each, on sums of
    magnitudes), a few float32 operations, and one rounding of h to 11 bits can move out, before
    its own rounding."""
    cs = 2.0 ** -16
    x = np.asarray(x, np.float64)
    T, k = ids.shape
    E, two_i, _ = w1.shape
    n = two_i // 2
    out, bound = np.zeros_like(x), np.zeros_like(x)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0 or e >= E:
                continue
            a = w1[e] @ x[t]
            s = np.abs(w1[e]) @ np.abs(x[t])
            g, u = a[:n], a[n:]
            sg, su = s[:n], s[n:]
            silu = g / (1.0 + np.exp(-g))
            h = silu * u
            # |silu'| <= 1.1
            dh = 1.1 * cs * sg * np.abs(u) + np.abs(silu) * cs * su + (2.0 ** -11 + 2.0 ** -19) * np.abs(h)
            dh += 2.0 ** -38 * np.abs(h).max()
            w = float(weights[t, j])
            out[t] += w * (w2[e] @ h)
            bound[t] += abs(w) * (np.abs(w2[e]) @ (dh * (1 + cs) + cs * np.abs(h)))
    return out, bound


def balance(logits, ids, alpha, offs=None, mask=None, dloss=1.0):
    """Loss, counts (S, E), tokens (S,) and the logits' gradient."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    k = ids.shape[1]
    offs = [0, T] if offs is None else [int(v) for v in offs]
    keep = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    S = len(offs) - 1
    counts, tokens = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    p = np.zeros((T, E))
    for t in range(T):
        m = z[t].max()
        if m > -np.inf:
            ex = np.exp(z[t] - m)
            p[t] = ex / ex.sum()
    rows = []
    for s in range(S):
        r = [t for t in range(offs[s], offs[s + 1]) if keep[t]]
        rows.append(r)
        tokens[s] = len(r)
        for t in r:
            for e in ids[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
    busy = int((tokens > 0).sum())
    loss, grad = 0.0, np.zeros((T, E))
    for s in range(S):
        if tokens[s] == 0:
            continue
        f = E * counts[s] / (k * tokens[s])
        loss += alpha / busy * float((f * p[rows[s]].mean(0)).sum())
        for t in rows[s]:
            grad[t] = dloss * alpha / (busy * tokens[s]) * p[t] * (f - float(f @ p[t]))
    return loss, counts, tokens, grad


def _rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def residual_norm(r, y, post_gamma=None, gate=1.0, scale=1.0, pre_gamma=None, eps=1e-6):
    """(r', n, rstd(y), rstd(r'), what is added to r); gate broadcasts against (T, H)."""
    r = np.asarray(r, np.float64)
    add, rs_y = np.zeros_like(r), None
    if y is not None:
        z = np.asarray(y, np.float64)
        if post_gamma is not None:
            rs_y = _rstd(z, eps)
            z = z * rs_y * post_gamma
        add = scale * gate * z
    rn = r + add
    rs_r = n = None
    if pre_gamma is not None:
        rs_r = _rstd(rn, eps)
        n = rn * rs_r * pre_gamma
    return rn, n, rs_y, rs_r, add


def residual_norm_grad(dr_new, dn, r, y, post_gamma=None, gate=1.0, scale=1.0, pre_gamma=None,
                       eps=1e-6):
    """Gradients as a dict of (value, sum of the magnitudes it is made of): dr, dy, dpost_gamma,
    dpre_gamma, dgate (elementwise (T, H), for the caller to sum over what was broadcast)."""
    rn, _, rs_y, rs_r, add = residual_norm(r, y, post_gamma, gate, scale, pre_gamma, eps)
    H = rn.shape[1]
    a = np.zeros_like(rn) if dr_new is None else np.asarray(dr_new, np.float64).copy()
    mag_a = np.abs(a)
    out = {}
    if dn is not None:
        u, hat = dn * pre_gamma, rn * rs_r
        # r' is a sum itself: a rounding in it is relative to |r| + |what is added|
        mag_hat = (np.abs(np.asarray(r, np.float64)) + np.abs(add)) * rs_r
        mean, mag = (u * hat).mean(1, keepdims=True), (np.abs(u) * mag_hat).mean(1, keepdims=True)
        a = a + rs_r * (u - hat * mean)
        mag_a = mag_a + rs_r * (np.abs(u) + mag_hat * mag)
        out["dpre_gamma"] = ((dn * hat).sum(0), (np.abs(dn) * mag_hat).sum(0))
    out["dr"] = (a, mag_a)
    if y is None:
        return out
    y = np.asarray(y, np.float64)
    post = 1.0 if post_gamma is None else post_gamma
    rs = 1.0 if post_gamma is None else rs_y
    yhat = y * rs
    dz, mag_z = scale * gate * a, np.abs(scale * gate) * mag_a
    d, mag_d = dz * post, mag_z * np.abs(post)
    if post_gamma is None:
        out["dy"] = (d, mag_d)
    else:
        mean = (d * yhat).sum(1, keepdims=True) / H
        mag = (mag_d * np.abs(yhat)).sum(1, keepdims=True) / H
        out["dy"] = (rs * (d - yhat * mean), rs * (mag_d + np.abs(yhat) * mag))
        out["dpost_gamma"] = ((dz * yhat).sum(0), (mag_z * np.abs(yhat)).sum(0))
    out["dgate"] = (scale * a * yhat * post, abs(scale) * mag_a * np.abs(yhat * post))
    return out
