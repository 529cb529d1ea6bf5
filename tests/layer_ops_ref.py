"""Plain 64-bit references of the operators in front of, between and beside the experts'
products (numpy), and the bounds that their GPU results are held to.

Bounds count roundings of fp32 (U32 = 2^-24, relative, of one operation). What enters
several bounds:
  a row's sum of H products: a thread adds at most 65 of them, its wave 7 times and its
  block at most 16 times, so a product passes through fewer than 90 roundings;
  exp: 2 U32; its argument x - top, rounded once: |x - top| U32 more, relative;
  1 / sqrt(mean + eps): half of the sum's, and 5 of its own: 50 U32."""
import numpy as np

from tests.expert_ops_ref import U32, f64, quantize  # noqa: F401

DEPTH = 90


def f32(a):
    return np.asarray(a, np.float32).astype(np.float64)


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
def scores(x, score):
    """Scores in 64 bits; 0 for a -inf logit."""
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
        top = x.max(axis=1, keepdims=True)
        d = np.where(x == top, 0.0, x - top)
        e = np.where(x == -np.inf, 0.0, np.exp(d))
        return e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)


def route(x, K, score, bias, groups, top_groups, group_top, renormalize, scale):
    """(ids, weights) of finite or -inf logits, one token at a time."""
    T, E = x.shape
    s = scores(x, score)
    b = np.zeros(E) if bias is None else bias
    ids, w = np.full((T, K), -1), np.zeros((T, K))
    S = E // groups
    for t in range(T):
        if bias is None and (groups == 1 or group_top == 1):
            key = x[t].copy()  # both scores rise with the logit
        else:
            key = s[t] + b
        key = np.where((x[t] == -np.inf) | (b == -np.inf), -np.inf, key)
        if groups > 1:
            best = np.sort(key.reshape(groups, S), axis=1)[:, ::-1][:, :group_top]
            total = np.where(best[:, 0] == -np.inf, -np.inf, np.where(best == -np.inf, 0.0, best).sum(axis=1))
            keep = np.argsort(-total, kind="stable")[:top_groups]
            mask = np.ones(groups, bool)
            mask[keep] = False
            key = np.where(np.repeat(mask, S), -np.inf, key)
        order = np.argsort(-key, kind="stable")[:K]
        order = order[key[order] > -np.inf]
        n = len(order)
        ids[t, :n] = order
        if n and renormalize:
            l = x[t, order] if score == "softmax" else np.minimum(x[t, order], 0.0)
            top = l.max()
            v = np.exp(np.where(l == top, 0.0, l - top))
            v = v if score == "softmax" else v / (1 + np.exp(-np.abs(x[t, order])))
            w[t, :n] = scale * v / v.sum()
        elif n:
            w[t, :n] = scale * s[t, order]
    return ids, w


def route_slack(x, score, K, renormalize):
    """Relative bound of a weight: the exponents' roundings of the largest distance that
    enters, the sum, and a dozen operations."""
    E = x.shape[1]
    fin = np.where(np.isfinite(x), x, 0.0)
    reach = fin.max(axis=1) - fin.min(axis=1) + np.abs(fin).max(axis=1)
    return ((reach + (K if renormalize else E) + 12) * U32)[:, None]


def route_grad(dw, x, ids, score, renormalize, scale):
    """(dx, what its terms add up to in magnitude)."""
    T, E = x.shape
    dx, mag = np.zeros((T, E)), np.zeros((T, E))
    s = scores(x, score)
    for t in range(T):
        at = [(int(i), float(q) * scale) for i, q in zip(ids[t], dw[t]) if 0 <= i < E and x[t, i] > -np.inf]
        if not at:
            continue
        i = np.array([a for a, _ in at])
        q = np.array([b for _, b in at])
        if renormalize:
            l = x[t, i] if score == "softmax" else np.minimum(x[t, i], 0.0)
            v = np.exp(l - l.max())
            v = v if score == "softmax" else v / (1 + np.exp(-np.abs(x[t, i])))
            p = v / v.sum()
            rest = 1.0 if score == "softmax" else scores(-x[t:t + 1, i], "sigmoid")[0]
            np.add.at(dx[t], i, p * rest * (q - (p * q).sum()))
            np.add.at(mag[t], i, p * rest * (np.abs(q) + (p * np.abs(q)).sum()))
        elif score == "sigmoid":
            d = q * s[t, i] * scores(-x[t:t + 1, i], "sigmoid")[0]
            np.add.at(dx[t], i, d)
            np.add.at(mag[t], i, np.abs(d))
        else:
            g, m = np.zeros(E), np.zeros(E)
            np.add.at(g, i, q)
            np.add.at(m, i, np.abs(q))
            dx[t] = s[t] * (g - (s[t] * g).sum())
            mag[t] = s[t] * (m + (s[t] * m).sum())
    return dx, mag


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def inverse_rms(h, eps):
    with np.errstate(all="ignore"):
        size = np.abs(h).max(axis=1, keepdims=True)
        size = np.where(size > 0, size, 1.0)  # squares of 1e200 and more stay in range
        return 1.0 / (size * np.sqrt(((h / size) ** 2).mean(axis=1, keepdims=True) + eps / size / size))


def norm_grad(dy, h, w, eps, dtotal):
    """(dx, bound before rounding to the type, dweight, its bound): r is off by 50 U32, a sum
    of g h by DEPTH + 2 of its terms' magnitudes, and so on: below 300 in all."""
    r = inverse_rms(h, eps)
    n, g = h * r, dy * w
    dx = r * (g - n * (g * n).mean(axis=1, keepdims=True))
    bound = 300 * U32 * r * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True))
    if dtotal is not None:
        dx = dx + dtotal
        bound = bound + 2 * U32 * np.abs(dtotal)
    return dx, bound, (dy * n).sum(axis=0), (len(dy) + 60) * U32 * np.abs(dy * n).sum(axis=0)


# ---------------------------------------------------------------------------
# activation
# ---------------------------------------------------------------------------
def activation(h, act):
    if act == "relu2":
        return np.maximum(h, 0.0) ** 2
    I = h.shape[1] // 2
    return h[:, :I] * scores(h[:, :I], "sigmoid") * h[:, I:]


def activation_grad(da, h, act, w):
    """(dh, bound before rounding); sig and 1 - sig are off by 5 U32 each."""
    d = da * w[:, None]
    if act == "relu2":
        dh = 2 * d * np.maximum(h, 0.0)
        return dh, 4 * U32 * np.abs(dh)
    I = h.shape[1] // 2
    g, u = h[:, :I], h[:, I:]
    sig, rest = scores(g, "sigmoid"), scores(-g, "sigmoid")
    dh = np.concatenate([d * u * sig * (1 + g * rest), d * g * sig], axis=1)
    return dh, np.concatenate([16 * U32 * np.abs(d * u) * sig * (1 + np.abs(g) * rest), 10 * U32 * np.abs(d * g * sig)], axis=1)


# ---------------------------------------------------------------------------
# adapters
# ---------------------------------------------------------------------------
def adapt(base, x, ids, a, b, scales, part):
    """(out, bound before rounding). part: what the two parts of v leave out, relative."""
    out, bound = base.copy(), np.zeros_like(base)
    H, r = x.shape[1], a.shape[1]
    for t, e in enumerate(ids):
        if not 0 <= e < len(a):
            continue
        v = a[e] @ x[t]
        off = H * U32 * (np.abs(a[e]) @ np.abs(x[t])) + part * np.abs(v) + 2.0 ** -24 * np.abs(v).max()
        d = b[e] @ v
        s = abs(scales[e])
        out[t] += scales[e] * d
        bound[t] = s * (np.abs(b[e]) @ off + (2 * r + 4) * U32 * (np.abs(b[e]) @ np.abs(v))) + 2 * U32 * np.abs(out[t])
    return out, bound
