"""Plain 64-bit restatements (numpy) of the operators of a prompt of text and images over existing
states, for the tests.  They share no code with the library."""
import numpy as np


def axis_of_pair(sections, order):
    """Pair by pair: each axis's pairs together, or in rounds that take one of every axis not used up."""
    left = list(sections)
    if order == "blocks":
        return np.repeat(np.arange(len(left)), left)
    out = []
    while sum(left):
        for x in range(len(left)):
            if left[x]:
                out.append(x)
                left[x] -= 1
    return np.array(out)


def rotate(x, positions, axis, freqs, layout, mscale=1.0):
    """x [N, ..., d] float64, pair j turned by positions[n, axis[j]] * freqs[j] -> the values, and
    |a| + |b| of each value's pair (for error bounds)."""
    d = x.shape[-1]
    th = positions.astype(np.float64)[:, axis] * freqs
    z = (mscale * np.exp(1j * th)).reshape((x.shape[0],) + (1,) * (x.ndim - 2) + (d // 2,))
    ia = np.arange(0, d, 2) if layout == "interleaved" else np.arange(d // 2)
    ib = ia + 1 if layout == "interleaved" else ia + d // 2
    w = (x[..., ia] + 1j * x[..., ib]) * z
    y, pair = np.empty_like(x), np.empty_like(x)
    y[..., ia], y[..., ib] = w.real, w.imag
    pair[..., ia] = pair[..., ib] = np.abs(x[..., ia]) + np.abs(x[..., ib])
    return y, pair


def logprobs(x, tokens, scale, top):
    """x [N, V] float64 (-inf: masked) -> logprob, entropy, rank, ids, alternatives, and what error
    bounds need: the mean distance below the maximum under p, and ln of the sum (both in nats)."""
    N, V = x.shape
    y = x * scale
    m = y.max(1, keepdims=True)
    none = m[:, 0] == -np.inf
    d = y - np.where(m == -np.inf, 0.0, m)
    e = np.exp(d)
    total = e.sum(1)
    with np.errstate(divide="ignore", invalid="ignore"):
        logs = np.where(none, 0.0, np.log(total))
        p = d - logs[:, None]
        below = np.where(none, 0.0, -(e * np.where(e > 0, d, 0.0)).sum(1) / total)
    entropy = np.where(none, 0.0, logs + below)
    order = np.argsort(-x, axis=1, kind="stable")
    rank, logprob = np.full(N, -1), np.zeros(N)
    for n in range(N):
        t = int(tokens[n])
        if t >= V:
            logprob[n] = np.nan
        elif t >= 0:
            rank[n] = int(np.nonzero(order[n] == t)[0][0])
            logprob[n] = -np.inf if none[n] else p[n, t]
    ids, alt = np.full((N, top), -1), np.full((N, top), -np.inf)
    k = min(top, V)
    ids[:, :k] = order[:, :k]
    alt[:, :k] = np.take_along_axis(p, order[:, :k], 1)
    alt[none] = -np.inf
    ids[:, :k][np.take_along_axis(x, order[:, :k], 1) == -np.inf] = -1
    return logprob, entropy, rank, ids, alt, below, logs


def cross(q, k, v, cu_q, cu_k, scale, causal, before=None):
    """q [Nq, H, d], k [H, Nk, d], v [H, Nk, 128] float64 -> out [Nq, H, 128], lse [Nq, H], the mean of
    |v| under the weights [Nq, H, 128], and the largest sum_d |q_d k_d| of a row's keys [Nq, H]
    (NaN in rows outside every run)."""
    Nq, H = q.shape[:2]
    out, lse = np.full((Nq, H, 128), np.nan), np.full((Nq, H), np.nan)
    mean, dot = out.copy(), lse.copy()
    for b in range(len(cu_q) - 1):
        i0, i1, j0, j1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        n, m = i1 - i0, j1 - j0
        for h in range(H):
            qs, ks, vs = q[i0:i1, h], k[h, j0:j1], v[h, j0:j1]
            s = scale * qs @ ks.T
            if causal:
                s = np.where(np.arange(m)[None, :] <= np.arange(n)[:, None] + m - n, s, -np.inf)
            top = s.max(1, initial=-np.inf, keepdims=True)
            e = np.exp(s - np.where(top == -np.inf, 0.0, top))
            total = e.sum(1, keepdims=True)
            some = total > 0
            w = np.where(some, e / np.where(some, total, 1.0), 0.0)
            with np.errstate(divide="ignore"):
                lse[i0:i1, h] = (np.log(total) + top)[:, 0]
            out[i0:i1, h], mean[i0:i1, h] = w @ vs, w @ np.abs(vs)
            seen = np.isfinite(s)
            dot[i0:i1, h] = np.where(seen, np.abs(qs) @ np.abs(ks).T, 0.0).max(1, initial=0.0)
    if before is not None:
        o1, l1 = before
        for b in range(len(cu_q) - 1):
            r = slice(cu_q[b], cu_q[b + 1])
            with np.errstate(invalid="ignore"):
                both = np.logaddexp(l1[r], lse[r])
                a1 = np.where(l1[r] == -np.inf, 0.0, np.exp(l1[r] - both))[..., None]
                a2 = np.where(lse[r] == -np.inf, 0.0, np.exp(lse[r] - both))[..., None]
            first = np.where(a1 > 0, o1[r], 0.0)
            out[r], mean[r], lse[r] = a1 * first + a2 * out[r], a1 * np.abs(first) + a2 * mean[r], both
    return out, lse, mean, dot
