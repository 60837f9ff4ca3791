"""The language-model operators' definitions in 64 bits (numpy), and the error
bounds that binary32 sums and one final rounding allow them.

U is binary32's unit roundoff, UNIT[t] that of an element type, TINY[t] half
its smallest subnormal.  chain(n) bounds the additions that any one term of a
sum of n terms passes through: the kernels give each of at least 256 lanes
every 256th term (rows too narrow for that: a warp's 32 lanes, at most 64 terms
each) and add the lanes in a tree of at most 16 levels, 16 more for good measure.
"""
import numpy as np

U = 2.0 ** -24
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def chain(n):
    return min(n, n / 256 + 96)


def rounding(t, value):
    """Allowance for storing a result of about `value` in type t."""
    return UNIT[t] * np.abs(value) * 1.0001 + TINY[t]


def embedding_grad(ids, dout, dtable, scale, beta, t):
    """(dtable, bound): every sum of n terms in any order is off by at most n U
    of the sum of magnitudes; scaling and adding beta * dtable add three roundings."""
    vocab = dtable.shape[0]
    valid = (ids >= 0) & (ids < vocab)
    total = np.zeros(dtable.shape)
    size = np.zeros(dtable.shape)
    np.add.at(total, ids[valid], dout[valid])
    np.add.at(size, ids[valid], np.abs(dout[valid]))
    n = np.bincount(ids[valid], minlength=vocab)[:, None]
    old = np.zeros(dtable.shape) if beta == 0 else beta * dtable
    ref = old + scale * total
    bound = U * ((n + 3) * abs(scale) * size + 3 * np.abs(old)) + rounding(t, ref) * (1 + 1e-3)
    return ref, bound


def layer_norm(x, w, b, eps, t):
    """((y, bound), (mean, bound), (rstd, bound))."""
    dim = x.shape[1]
    mean = x.mean(1, keepdims=True)
    dev = x - mean
    var = (dev * dev).mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    xhat = dev * rstd
    y = xhat * w + b
    d_mean = U * (chain(dim) + 2) * np.abs(x).mean(1, keepdims=True)
    # each deviation is off by d_mean and one rounding; their squares' mean moves by
    # d_mean^2 (the deviations sum to zero) and the sum's own error
    d_var = d_mean ** 2 + 2 * U * (chain(dim) + 4) * var + 2 * d_mean * U * np.abs(dev).mean(
        1, keepdims=True)
    d_rstd = rstd * (0.5 * d_var / (var + eps) + 6 * U)
    d_xhat = (d_mean + 2 * U * np.abs(dev)) * (rstd + d_rstd) + np.abs(dev) * d_rstd
    d_y = np.abs(w) * d_xhat + 3 * U * (np.abs(w * xhat) + np.abs(b))
    return ((y, d_y + rounding(t, y)), (mean[:, 0], d_mean[:, 0] + U * np.abs(mean[:, 0])),
            (rstd[:, 0], d_rstd[:, 0]))


def layer_norm_grad(dy, x, mean, rstd, w, t, pt):
    """((dx, bound), (dweight, bound), (dbias, bound)); mean and rstd are inputs."""
    rows, dim = x.shape
    r = rstd[:, None]
    xhat = (x - mean[:, None]) * r
    g = dy * w
    a = g.mean(1, keepdims=True)
    b = (g * xhat).mean(1, keepdims=True)
    dx = r * (g - a - xhat * b)
    d_a = U * (chain(dim) + 4) * np.abs(g).mean(1, keepdims=True)
    d_b = U * (chain(dim) + 6) * np.abs(g * xhat).mean(1, keepdims=True)
    d_dx = np.abs(r) * (d_a + np.abs(xhat) * d_b
                        + 6 * U * (np.abs(g) + np.abs(a) + np.abs(xhat * b)))
    # rows are dealt to blocks, then joined: no term passes more than this many additions
    n = min(rows, rows / 8 + 96)
    dw, db = (dy * xhat).sum(0), dy.sum(0)
    d_dw = U * (n + 4) * np.abs(dy * xhat).sum(0)
    d_db = U * (n + 1) * np.abs(dy).sum(0)
    return ((dx, d_dx + rounding(t, dx)), (dw, d_dw + rounding(pt, dw)),
            (db, d_db + rounding(pt, db)))


def token_logprob(x, targets, alpha):
    """lse, logprob, entropy of each row and their bounds.  x may hold -inf and NaN."""
    rows, vocab = x.shape
    out = {k: np.zeros(rows) for k in ("lse", "logprob", "entropy")}
    tol = {k: np.zeros(rows) for k in out}
    for r in range(rows):
        z = alpha * x[r]
        t = -1 if targets is None else int(targets[r])
        has = 0 <= t < vocab
        if np.isnan(z).any() or np.isposinf(z).any():
            for k in out:
                out[k][r] = np.nan if k != "logprob" or has else 0.0
            continue
        live = z[z > -np.inf]
        if live.size == 0:
            out["lse"][r] = -np.inf
            out["logprob"][r] = -np.inf if has else 0.0
            continue
        m = live.max()
        e = np.exp(live - m)
        s = e.sum()
        p = e / s
        lse = m + np.log(s)
        far = float((p * np.abs(live - m)).sum())      # how far from the maximum, on average
        # a term's exponent is off by 4 U of its distance, the exponential by 4 U; the sum by
        # its chain; the base (alpha m) and the result by their own roundings
        d_lse = U * (chain(vocab) + 8 + 4 * far + 4 * abs(m) + 2 * abs(lse))
        second = float((p * (live - m) ** 2).sum())
        out["lse"][r], tol["lse"][r] = lse, d_lse
        out["entropy"][r] = np.log(s) - (p * (live - m)).sum()
        tol["entropy"][r] = U * ((chain(vocab) + 12) * (1 + 2 * far) + 8 * second
                                 + 4 * abs(np.log(s)))
        if has:
            out["logprob"][r] = z[t] - lse
            if z[t] > -np.inf:
                tol["logprob"][r] = d_lse + U * (2 * abs(z[t]) + abs(z[t] - lse))
    return out, tol


def top(x, k):
    """Indices of the k largest logits (lowest index first among equals), -1 where none."""
    rows, vocab = x.shape
    out = np.full((rows, k), -1, np.int32)
    for r in range(rows):
        live = np.flatnonzero(x[r] > -np.inf)
        order = live[np.lexsort((live, -x[r][live]))][:k]
        out[r, :order.size] = order
    return out


def token_logprob_grad(x, targets, lse, entropy, up, de, alpha, t):
    """(dlogits, bound); lse and entropy are inputs."""
    rows, vocab = x.shape
    z = alpha * x
    with np.errstate(invalid="ignore", over="ignore"):
        q = z - lse[:, None]
        p = np.where((z > -np.inf) & (lse[:, None] > -np.inf), np.exp(q), 0.0)
    q = np.where(p > 0, q, 0.0)
    d = np.zeros((rows, vocab))
    bound = np.zeros((rows, vocab))
    # the exponent is off by 2 U of its terms, the exponential by 4 U
    eps = U * (3 * np.abs(np.where(p > 0, z, 0.0)) + 3 * np.abs(
        np.where(lse > -np.inf, lse, 0.0))[:, None] + 8)
    if up is not None:
        has = (targets >= 0) & (targets < vocab)
        u = np.where(has, up, 0.0)[:, None]
        d -= u * p
        bound += np.abs(u) * p * (eps + 2 * U)
        at = np.flatnonzero(has & (lse > -np.inf))
        d[at, targets[at]] += up[at]
        bound[at, targets[at]] += 3 * U * np.abs(up[at])
    if de is not None:
        ent = entropy[:, None]
        d -= de[:, None] * p * (q + ent)
        bound += np.abs(de)[:, None] * p * ((eps + 4 * U) * np.abs(q + ent)
                                            + 3 * U * (np.abs(np.where(p > 0, z, 0.0))
                                                       + np.abs(q) + np.abs(ent)))
        bound += 2 * U * np.abs(d)
    d *= alpha
    return d, alpha * bound + 2 * U * np.abs(d) + rounding(t, d)
