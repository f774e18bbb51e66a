"""The operators of a training step around the blocks in 64 bits (numpy), test
infrastructure: each from its definition, pinned in test_training_cpu.py."""
import numpy as np


def layernorm_stats(x, eps):
    mean = x.mean(1)
    return mean, 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)


def layernorm(x, gain, bias, eps):
    mean, rstd = layernorm_stats(x, eps)
    return (x - mean[:, None]) * rstd[:, None] * gain + bias


def layernorm_backward(x, gain, eps, dy, dres=0.0, stats=None):
    """dx, dgain, dbias, and for the tolerances: the size of dx's terms, sum |dy xh|, sum |dy|."""
    mean, rstd = layernorm_stats(x, eps) if stats is None else stats
    r = rstd[:, None]
    xh = (x - mean[:, None]) * r
    g = dy * gain
    gx = (g * xh).mean(1, keepdims=True)
    dx = dres + r * (g - g.mean(1, keepdims=True) - xh * gx)
    terms = np.abs(dres) + r * (np.abs(g) + np.abs(g).mean(1, keepdims=True) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0), terms, np.abs(dy * xh).sum(0), np.abs(dy).sum(0)


def embedding(ids, E, scale):
    out = np.zeros((len(ids), E.shape[1]))
    ok = (ids >= 0) & (ids < len(E))
    out[ok] = scale * E[ids[ok]]
    return out


def embedding_backward(ids, v, dOut, scale):
    """dE, and for the tolerances scale * sum |dOut| and the number of tokens of each word."""
    dE, size = np.zeros((v, dOut.shape[1])), np.zeros((v, dOut.shape[1]))
    count = np.zeros(v)
    for m, r in enumerate(ids):
        if 0 <= r < v:
            dE[r] += scale * dOut[m]
            size[r] += abs(scale) * np.abs(dOut[m])
            count[r] += 1
    return dE, size, count


def loss(z, labels, dloss):
    """Loss and the gradient of the logits; the probabilities with the label's negated complement for the tolerances."""
    n, v = z.shape
    out, grad = np.zeros(n), np.zeros((n, v))
    with np.errstate(all="ignore"):
        for m, y in enumerate(labels):
            if y == -100:
                continue
            if not 0 <= y < v or not (z[m] < np.inf).all() or (z[m] == -np.inf).all():
                out[m], grad[m] = np.nan, np.nan
                continue
            most = z[m].max()
            e = np.exp(z[m] - most)
            others = e.sum() - e[y] if e[y] < 0.5 * e.sum() else np.delete(e, y).sum()
            out[m] = np.log1p(others / e[y]) if e[y] > 0 else np.inf
            if e[y] > 0 and others / e[y] == np.inf:
                out[m] = most - z[m, y] + np.log(others)
            grad[m] = dloss[m] * e / (others + e[y])
            grad[m, y] = -dloss[m] * others / (others + e[y])
    return out, grad


def clip(grads, max_norm):
    norm = np.sqrt(sum((g ** 2).sum() for g in grads))
    by = 1.0 if not norm > max_norm or not np.isfinite(norm) else max_norm / norm
    return norm, [g * by for g in grads]
