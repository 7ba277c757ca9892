"""Float64 reference of the 4-bit floating-point operators and of the token
statistics.  Written from the definitions: codes are decided by distance to
the eight magnitudes, values read bit by bit, sums in one expression.

Parity unpinned (conventions of the library, no source gives values): the
power of a block, the order of equal logits.
"""

import numpy as np

__all__ = ["mx_quantize", "mx_values", "mx_gate", "mx_gate_slope", "mx_gated_backward",
           "token_stats", "token_grad"]

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_quantize(x):
    """(codes [n, 16 nb], scale bytes [n, nb], values [n, d]) of x [n, d]."""
    x = np.asarray(x, np.float64)
    n, d = x.shape
    nb = -(-d // 32)
    v = np.zeros((n, nb * 32))
    v[:, :d] = x
    v = v.reshape(n, nb, 32)
    bad = ~np.isfinite(v).all(2)
    top = np.where(bad, 1.0, np.abs(np.where(np.isfinite(v), v, 0.0)).max(2))
    _, e = np.frexp(top)                       # top = f 2^e, f in [1/2, 1)
    power = np.where(top > 0, np.maximum(e - 3, -127), -127)
    a = np.abs(np.where(np.isfinite(v), v, 0.0)) / np.ldexp(1.0, power)[:, :, None]
    # nearest magnitude; between two equally near the one with an even code
    off = np.abs(a[..., None] - LEVELS)
    off[..., 1::2] = np.nextafter(off[..., 1::2], np.inf)
    code = off.argmin(-1)
    code[a >= 6.0] = 7
    code = code | np.where(np.signbit(v), 8, 0)
    code[bad] = 0
    scales = np.where(bad, 255, power + 127).astype(np.uint8)
    code = code.reshape(n, nb * 32).astype(np.uint8)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    return codes, scales, mx_values(codes, scales, d)


def mx_values(codes, scales, d):
    """The values [rows, d] that codes and scale bytes stand for."""
    col = np.arange(d)
    code = (codes[:, col // 2].astype(int) >> (4 * (col % 2))) & 15
    ex, man = (code >> 1) & 3, code & 1
    v = np.where(ex > 0, np.ldexp(1.0 + 0.5 * man, ex - 1), 0.5 * man)
    s = scales[:, col // 32].astype(int)
    with np.errstate(invalid="ignore"):
        return np.where(code & 8, -v, v) * np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))


def mx_gate(g, act):
    if act == "silu":
        return g / (1.0 + np.exp(-g))
    return np.where(g > 0, g, 0.0) if act == "relu" else g


def mx_gate_slope(g, act):
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return s + g * s * (1.0 - s)
    return (g > 0).astype(np.float64) if act == "relu" else np.ones_like(g)


def mx_gated_backward(dY, G, U, Wg, Wu, act):
    """(dX, dG, dU) of Y = act(G) U, G = X Wg^T, U = X Wu^T."""
    dU, dG = dY * mx_gate(G, act), dY * U * mx_gate_slope(G, act)
    return dG @ Wg + dU @ Wu, dG, dU


def token_stats(z, tokens, k, T):
    """(logp, entropy, lse, top logits, top ids) of rows of logits z [n, vocab]."""
    z = np.asarray(z, np.float64)
    n = len(z)
    top = np.full((n, k), -np.inf)
    idx = np.full((n, k), -1, np.int64)
    logp, entropy, lse = np.zeros(n), np.full(n, np.nan), np.full(n, np.nan)
    for r in range(n):
        number = np.flatnonzero(~np.isnan(z[r]))
        best = number[np.argsort(-z[r][number], kind="stable")[:k]]
        top[r, :len(best)], idx[r, :len(best)] = z[r][best], best
        m = z[r].max()
        if m == -np.inf:
            lse[r] = -np.inf
        elif np.isfinite(m):
            with np.errstate(over="ignore"):
                d = (z[r] - m) / T
            lse[r] = m / T + np.log(np.exp(d).sum())
            q = np.exp(d) / np.exp(d).sum()
            entropy[r] = -(q[q > 0] * np.log(q[q > 0])).sum()
        t = int(tokens[r])
        if 0 <= t < z.shape[1]:
            logp[r] = d[t] - np.log(np.exp(d).sum()) if np.isfinite(m) else np.nan
    return logp, entropy, lse, top, idx


def token_grad(z, tokens, g, h, T):
    """Gradient of sum(g logp + h entropy) with respect to z."""
    z = np.asarray(z, np.float64)
    out = np.zeros_like(z)
    for r in range(len(z)):
        t = int(tokens[r])
        up = g[r] if 0 <= t < z.shape[1] else 0.0
        if up == 0 and h[r] == 0:
            continue
        m = z[r].max()
        e = np.exp((z[r] - m) / T)
        q = e / e.sum()
        with np.errstate(divide="ignore"):
            lq = np.log(q)
        ent = -(q[q > 0] * lq[q > 0]).sum()
        out[r] = -up * q - h[r] * np.where(q > 0, q * (np.where(q > 0, lq, 0.0) + ent), 0.0)
        if up:
            out[r, t] += up
    return out / T
