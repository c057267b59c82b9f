"""The gated linear recurrence, its gradient and the 8-bit checkpoint in numpy, token by token in 64 bits,
with bounds on the error that binary32 evaluation in any association of the scan can have.

Error model (e = 2^-24).  A result is a sum over earlier tokens s of (product of a over s+1..t) times
an input.  Each factor a carries at most 6 e (exp within 3 e; for a logit gate the sum 1 + exp, a
reciprocal and a product), each product and each sum that joins it to the rest 1 e more: 8 e per token
of distance.  A scan by tiles joins partial results in at most 24 further products or sums (5 levels
in a wave, 3 waves, up to 15 tiles and a state).  With N the recurrence over magnitudes, N_t = a_t
N_{t-1} + |b_t|, and S_t = a_t S_{t-1} + N_t (which counts every term once per token of distance),

    |computed h_t - h_t| <= e (8 S_t + 24 N_t),

before the one rounding to the output's type (half a step, eps / 2 relative).  (For 16-bit tensors exp is within
(|x| + 2) e instead: a term that passed gates of logarithms x carries y e more, y the sum of their |x|, which
the 8 per token and the 24 cover up to y = 24 + 3 per token; beyond that the term has decayed below exp(-24).)  The same holds for
the gradient's recurrence k from behind; a product formed from it adds at most 8 e of its magnitude."""
from __future__ import annotations

import numpy as np

E = 2.0 ** -24
BLOCK = 64


def gate_terms(gate, kind):
    gate = np.asarray(gate, dtype=np.float64)
    with np.errstate(over="ignore"):
        if kind == "log":
            return np.exp(gate), np.ones_like(gate)
        return 1.0 / (1.0 + np.exp(-gate)), 1.0 / (1.0 + np.exp(gate))


def spans(tokens, sequences, offsets):
    if offsets is None:
        n = tokens // sequences
        return [(s * n, (s + 1) * n) for s in range(sequences)]
    return [(int(offsets[s]), int(offsets[s + 1])) for s in range(sequences)]


def forward(gate, u, h0, kind, sequences, offsets=None):
    """gate, u (tokens, C), h0 (sequences, C) or None -> h, h_final and the error bounds of both."""
    a, c = gate_terms(gate, kind)
    b = c * np.asarray(u, dtype=np.float64)
    T, C = a.shape
    h, bound = np.zeros((T, C)), np.zeros((T, C))
    final, final_bound = np.zeros((sequences, C)), np.zeros((sequences, C))
    for s, (lo, hi) in enumerate(spans(T, sequences, offsets)):
        now = np.zeros(C) if h0 is None else np.asarray(h0[s], dtype=np.float64)
        N, S = np.abs(now), np.zeros(C)
        for t in range(lo, hi):
            now = a[t] * now + b[t]
            N = a[t] * N + np.abs(b[t])
            S = a[t] * S + N
            h[t], bound[t] = now, E * (8 * S + 24 * N)
        final[s] = now
        final_bound[s] = E * (8 * S + 24 * N) if hi > lo else 0.0
    return h, final, bound, final_bound


def backward(gate, u, saved, h0, dh, dh_final, kind, sequences, offsets=None):
    """saved: the states h as the gradient sees them (tokens, C).  Returns dgate, du, dh0 and their bounds."""
    a, c = gate_terms(gate, kind)
    T, C = a.shape
    u = np.zeros((T, C)) if u is None else np.asarray(u, dtype=np.float64)
    dh = np.asarray(dh, dtype=np.float64)
    out = [np.zeros((T, C)) for _ in range(4)]
    dgate, du, bgate, bu = out
    dh0, b0 = np.zeros((sequences, C)), np.zeros((sequences, C))
    for s, (lo, hi) in enumerate(spans(T, sequences, offsets)):
        k = np.zeros(C) if dh_final is None else np.asarray(dh_final[s], dtype=np.float64)
        N, S, err = np.abs(k), np.zeros(C), np.zeros(C)
        for t in range(hi - 1, lo - 1, -1):
            before = saved[t - 1] if t > lo else (np.zeros(C) if h0 is None else h0[s])
            before = np.asarray(before, dtype=np.float64)
            d, Nd, errd = dh[t] + k, np.abs(dh[t]) + N, err
            k, N = a[t] * d, a[t] * Nd
            S = a[t] * S + N
            err = E * (8 * S + 24 * N)
            du[t] = c[t] * d
            bu[t] = c[t] * (errd + 8 * E * Nd)
            if kind == "log":
                dgate[t] = k * before
                bgate[t] = (err + 8 * E * N) * np.abs(before)
            else:
                dgate[t] = k * c[t] * (before - u[t])
                bgate[t] = c[t] * (err + 8 * E * N) * (np.abs(before) + np.abs(u[t]))
        dh0[s], b0[s] = k, err
    return dgate, du, dh0, bgate, bu, b0


def checkpoint(x):
    """Codes and scales of float32 rows (rows, C), exactly: the quotient of two binary32 numbers in binary64
    is on the right side of every tie (distinct from a half-integer by more than 2^-26 of itself, or equal)."""
    x = np.asarray(x, dtype=np.float32)
    rows, C = x.shape
    nb = -(-C // BLOCK)
    codes, scale = np.zeros((rows, C), np.int8), np.zeros((rows, nb), np.float32)
    for k in range(nb):
        blk = x[:, k * BLOCK:(k + 1) * BLOCK]
        m = np.abs(blk).max(axis=1)                        # NaN where one is
        with np.errstate(all="ignore"):
            sc = (m * (np.float32(1) / np.float32(127))).astype(np.float32)
            sc = np.where(m < np.float32(127 * 2.0 ** -126), np.float32(0), sc)
            sc = np.where(np.isfinite(m), sc, np.float32(np.nan))
            q = np.rint(blk.astype(np.float64) / sc[:, None].astype(np.float64))
        codes[:, k * BLOCK:(k + 1) * BLOCK] = np.where((sc > 0)[:, None], q, 0).astype(np.int8)
        scale[:, k] = sc
    return codes, scale


def values(codes, scale):
    """What a checkpoint stands for, in 64 bits."""
    wide = np.repeat(np.asarray(scale, dtype=np.float64), BLOCK, axis=-1)[..., :codes.shape[-1]]
    return codes.astype(np.float64) * wide
