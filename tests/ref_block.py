"""64-bit references of the norms, the 8-bit rows, the causal convolution and the selective scan, written from their
formulas, with bounds on what binary32 arithmetic in any order may differ by.  E is half a last place of binary32."""
import numpy as np

E = 2.0 ** -24
SMALLEST = np.float32(127.0 * 2.0 ** -126)


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def norm(x, weight, residual=None, gate=None, groups=1, eps=1e-5):
    """(n, v, bound of n)."""
    v, extra = x, np.ones_like(x)                      # roundings of v
    if residual is not None:
        v = x + residual
    if gate is not None:                               # exp within |z| + 3, 1 + e, the reciprocal within 2, two products
        v, extra = x * silu(gate), 8.0 + np.abs(gate)
    parts = v.reshape(v.shape[0], groups, -1)
    n = parts / np.sqrt((parts ** 2).mean(-1, keepdims=True) + eps)
    n = n.reshape(v.shape) * weight
    # The sum of squares: up to 64 of them one after another in a lane, then 10 levels of halves and 16 waves; a squared
    # v carries its roundings twice, and the root halves all of it.  Then mean, root and quotient, and two products.
    return n, v, np.abs(n) * E * (extra + (64 + 10 + 16 + 2 * extra.max()) / 2 + 3 + 2)


def row_scale(most):
    """The scale of rows with these largest magnitudes, in binary32."""
    most = most.astype(np.float32)
    scale = most * np.float32(1.0 / 127.0)
    scale = np.where(most < SMALLEST, np.float32(0), scale)
    return np.where(np.isfinite(most), scale, np.float32(np.nan))


def rows(x):
    """Codes and scales of rows of binary32 numbers, exactly: the quotient of two numbers of 24 bits is nearer to a
    tie than a double can tell only where it is one."""
    scale = row_scale(np.abs(x).max(-1) if np.isfinite(x).all() else np.where(np.isfinite(x).all(-1), np.abs(x).max(-1), np.inf))
    safe = np.where(scale > 0, scale, 1).astype(np.float64)[:, None]
    with np.errstate(invalid="ignore"):
        codes = np.rint(np.where(scale[:, None] > 0, x.astype(np.float64) / safe, 0.0))
    return codes.astype(np.int8), scale


def spans(sequences, tokens, offsets):
    if offsets is None:
        length = tokens // sequences
        return [(s * length, (s + 1) * length) for s in range(sequences)]
    return [(int(lo), int(hi)) for lo, hi in zip(offsets, offsets[1:])]


def conv(x, weight, bias, state, sequences, offsets, activate=True):
    """(out, the last inputs, bound of out) over (tokens, channels)."""
    tokens, channels = x.shape
    width = weight.shape[1]
    out, bound, kept = np.zeros_like(x), np.zeros_like(x), np.zeros((sequences, width - 1, channels))
    for s, (lo, hi) in enumerate(spans(sequences, tokens, offsets)):
        past = state[s] if state is not None else np.zeros((width - 1, channels))
        wide = np.concatenate([past, x[lo:hi]])
        kept[s] = wide[len(wide) - (width - 1):]
        a = np.zeros((hi - lo, channels)) + (0.0 if bias is None else bias)
        size = np.abs(a)
        for k in range(width):
            a = a + wide[k:k + hi - lo] * weight[:, k]
            size = size + np.abs(wide[k:k + hi - lo] * weight[:, k])
        wrong = (width + 1) * E * size
        if activate:                                   # |SiLU'| < 1.1; exp within |a| + 3, 1 + e, reciprocal, product
            out[lo:hi] = silu(a)
            wrong = 1.1 * wrong + np.abs(out[lo:hi]) * (np.abs(a) + 8) * E
        else:
            out[lo:hi] = a
        bound[lo:hi] = wrong
    return out, kept, bound


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def scan(u, delta, A, B, C, D, z, delta_bias, h0, sequences, offsets, positive=True):
    """(y, h_final, bound of y, bound of h_final) over (tokens, channels)."""
    tokens, channels = u.shape
    n = A.shape[1]
    y, wrong_y = np.zeros_like(u), np.zeros_like(u)
    final = np.zeros((sequences, channels, n)) if h0 is None else h0.astype(np.float64).copy()
    wrong_final = np.zeros_like(final)
    raw = delta + (0.0 if delta_bias is None else delta_bias)
    d = softplus(raw) if positive else raw
    # d: the sum with the bias rounded once, moved on by a slope of at most 1 (but relatively never more than |raw| times);
    # then exp(-|raw|), which may be off by |raw| + 3, and log(1 + that), of at most its size, within 5 more
    wrong_d = E * (2 * np.abs(raw) * np.minimum(1.0, np.abs(d) if positive else 1.0) + 8 * np.abs(d))
    for s, (lo, hi) in enumerate(spans(sequences, tokens, offsets)):
        h, size, wrong = final[s].copy(), np.abs(final[s]), np.zeros((channels, n))
        for t in range(lo, hi):
            x = d[t][:, None] * A
            a = np.exp(x)
            b = (d[t] * u[t])[:, None] * B[t]
            # a: the product and the factor log2(e) each rounded, d's error, the exponential within 3
            wrong = a * wrong + np.abs(a * h) * (E * (3 * np.abs(x) + 3) + np.abs(A) * wrong_d[t][:, None])
            wrong = wrong + np.abs(b) * 3 * E + np.abs(u[t][:, None] * B[t]) * wrong_d[t][:, None]
            h = a * h + b
            size = a * size + np.abs(b)
            wrong = wrong + E * size
            # Work split along the sequence carries a state over up to 256 tokens at once, by exp(A sum d): the sum's
            # roundings, 256 of them, count |A sum d| exp(-|A sum d|) <= 0.37 times; per state, over all such parts,
            # its decay keeps the total below twice that of the last one or two
            split = 2 * 0.37 * 256 * E * size
            read = (C[t] * h).sum(-1)
            wrong_read = (np.abs(C[t]) * (wrong + split)).sum(-1) + (n + 2) * E * (np.abs(C[t]) * size).sum(-1)
            if D is not None:
                read = read + D * u[t]
                wrong_read = wrong_read + 2 * E * np.abs(D * u[t])
            if z is not None:
                g = silu(z[t])
                y[t] = read * g
                wrong_y[t] = wrong_read * np.abs(g) + np.abs(y[t]) * (np.abs(z[t]) + 10) * E   # exp within |z| + 3
            else:
                y[t], wrong_y[t] = read, wrong_read
        final[s] = h
        wrong_final[s] = wrong + (2 * 0.37 * 256 * E * size if hi > lo else 0.0)
    return y, final, wrong_y, wrong_final
