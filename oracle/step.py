"""Plain numpy oracles of the feed-forward half of a decode step and of the
model's answer, in 64 bits: the residual's addition and norm, the gated
projections, log probabilities.  They share no code with the HIP path.  Test
infrastructure only."""
import numpy as np

F32 = np.float32


def norm_sum(x, residual, to_residual):
    """h: one fp32 addition, rounded to the residual's type by `to_residual`
    (float32 -> float32 values of that type); x itself without a residual."""
    x = np.asarray(x, F32)
    if residual is None:
        return x
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(to_residual(x + np.asarray(residual, F32)), F32)


def rms_norm(h, w, eps):
    """The norm of rows h in 64 bits."""
    h = np.asarray(h, np.float64)
    y = h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + float(F32(eps)))
    return y if w is None else y * np.asarray(w, np.float64)


def rms_norm_steps(h, w, eps):
    """The norm of rows h (float32) in the definition's fp32 steps, their root from 64 bits."""
    h = np.asarray(h, F32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        h64 = h.astype(np.float64)
        r = (1 / np.sqrt(np.sum(h64 * h64, axis=-1, keepdims=True) / h.shape[-1] + float(F32(eps)))).astype(F32)
        y = h * r
        return y if w is None else y * np.asarray(w, F32)


def codes8(y, s=None):
    """(codes, scales [T]) of rows y (float32): with the scale s, or a row's own."""
    y = np.asarray(y, F32)
    if s is None:
        s = (np.max(np.abs(y), axis=-1) / F32(127)).astype(F32)
    else:
        s = np.full(y.shape[0], F32(s))
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint(y / s[:, None])
    return np.where(s[:, None] == 0, 0, np.clip(c, -128, 127)).astype(np.int8), s


def dense(codes, scales):
    """[N][K] of packed weights (uint8 [N][K/4], float16 [N][K/256]) in 64 bits."""
    codes = np.asarray(codes)
    q = np.stack([(codes >> (2 * j)) & 3 for j in range(4)], -1).reshape(codes.shape[0], -1)
    return (q.astype(np.float64) - 1) * np.repeat(np.asarray(scales).astype(np.float64), 256, axis=1)


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1 + np.exp(-v))


def gated(wg, wu, x):
    """(h, g, u, and the sums of |w x| of both) for x [M][K] in 64 bits."""
    x = np.asarray(x, np.float64)
    g, u = x @ wg.T, x @ wu.T
    return silu(g) * u, g, u, np.abs(x) @ np.abs(wg).T, np.abs(x) @ np.abs(wu).T


def logprobs(logits, scale=1.0):
    """(log probabilities [T][V], entropy [T]) in 64 bits, by the definition's cases."""
    x = np.asarray(logits, np.float64) * float(F32(scale))
    lp, H = np.empty_like(x), np.empty(len(x))
    for t, row in enumerate(x):
        if np.isnan(row).any() or np.isposinf(row).any():
            lp[t], H[t] = np.nan, np.nan
        elif np.isneginf(row).all():
            lp[t], H[t] = -np.inf, 0
        else:
            d = row - row.max()
            lp[t] = d - np.log(np.sum(np.exp(d)))
            some = np.isfinite(lp[t])
            H[t] = -np.sum(np.exp(lp[t][some]) * lp[t][some])
    return lp, H


def top_tokens(logits, top):
    """The places of the largest values of each row, of equal ones the first; -1 in rows without a distribution."""
    x = np.asarray(logits, np.float64)
    out = np.argsort(-x, axis=-1, kind="stable")[:, :top].astype(np.int64)
    out[np.isnan(x).any(-1) | np.isposinf(x).any(-1)] = -1
    return out
