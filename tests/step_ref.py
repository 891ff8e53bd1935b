"""Plain 64-bit restatements (numpy) of the operators of a speculative decoding step, for the
tests.  They share no code with the library."""
import numpy as np


def bf16(x):
    """float64 -> nearest bf16 value (ties to even), as float64 (finite, normal range)."""
    b = np.asarray(x, dtype=np.float32).view(np.uint32)
    r = (b + 0x7FFF + ((b >> 16) & 1)) & np.uint32(0xFFFF0000)
    return r.view(np.float32).astype(np.float64)


def rotate(x, positions, freqs, layout, mscale):
    """x [N, ..., d] float64 turned by positions[n] * freqs[j] in pair j."""
    d = x.shape[-1]
    th = positions.astype(np.float64).reshape((-1,) + (1,) * (x.ndim - 1)) * freqs
    c, s = mscale * np.cos(th), mscale * np.sin(th)
    y = np.empty_like(x)
    ia = np.arange(0, d, 2) if layout == "interleaved" else np.arange(d // 2)
    ib = ia + 1 if layout == "interleaved" else ia + d // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    pair = np.empty_like(x)
    pair[..., ia] = pair[..., ib] = np.abs(a) + np.abs(b)
    return y, pair  # the values, and |a| + |b| of each value's pair (for error bounds)


def verify(target, draft, tokens, uniforms, parents=None, lens=None):
    """One request at a time, as the header defines it; float64."""
    B, T = tokens.shape
    V = target.shape[2]
    num, depths, nxt = np.zeros(B, int), np.full((B, T), -1), np.zeros(B, int)
    clean = lambda r: np.clip(np.nan_to_num(r.astype(np.float64), nan=0.0), 0.0, 1.0)
    for b in range(B):
        at, depth, left, mass = -1, 0, clean(target[b, 0]), 1.0
        n = T if lens is None else int(np.clip(lens[b], 0, T))
        for i in range(n):
            par = i - 1 if parents is None else int(parents[b, i])
            x = int(tokens[b, i])
            if par != at or not 0 <= x < V:
                continue
            q = clean(draft[b, i]) if draft is not None else (np.arange(V) == x).astype(np.float64)
            if float(uniforms[b, i]) * q[x] * mass < left[x]:
                depths[b, i], depth, at = depth, depth + 1, i
                left, mass = clean(target[b, i + 1]), 1.0
            else:
                left = np.maximum(left - mass * q, 0.0)
                mass = left.sum()
        num[b] = depth
        if left.sum() == 0:
            left = clean(target[b, at + 1])
        upto = np.cumsum(left)
        nxt[b] = -1 if upto[-1] == 0 else int(np.searchsorted(upto, float(uniforms[b, T]) * upto[-1], side="right"))
    return num, depths, nxt
