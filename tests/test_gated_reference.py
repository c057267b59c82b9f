"""Pins of the gated recurrence's 64-bit reference that need no GPU: closed forms, gradients against
central differences, packed against dense, and the 8-bit checkpoint against exact rationals."""
from fractions import Fraction

import numpy as np
import pytest

import ref_gated as ref


def draw(seed, tokens, channels, sequences, kind):
    rng = np.random.default_rng(seed)
    gate = -np.abs(rng.normal(0.4, 0.3, (tokens, channels))) if kind == "log" else rng.normal(1, 1, (tokens, channels))
    return (gate, rng.normal(size=(tokens, channels)), rng.normal(size=(sequences, channels)),
            rng.normal(size=(tokens, channels)), rng.normal(size=(sequences, channels)))


def test_closed_forms():
    u = np.arange(1.0, 7.0).reshape(6, 1)
    h, final, _, _ = ref.forward(np.zeros((6, 1)), u, None, "log", 1)           # a = 1: prefix sums
    assert np.array_equal(h[:, 0], np.cumsum(u[:, 0])) and final[0, 0] == 21.0
    h, _, _, _ = ref.forward(np.full((6, 1), -np.inf), u, [[5.0]], "log", 1)    # a = 0: the input itself
    assert np.array_equal(h, u)
    h, _, _, _ = ref.forward(np.zeros((6, 1)), u, [[4.0]], "logit", 1)          # a = b = 1/2, by hand
    assert h[0, 0] == 2.5 and h[1, 0] == 2.25


@pytest.mark.parametrize("kind", ["log", "logit"])
@pytest.mark.parametrize("offsets", [None, (0, 3, 3, 4, 9)])
def test_gradients_against_differences(kind, offsets):
    tokens, channels = (8, 3) if offsets is None else (9, 3)
    sequences = 2 if offsets is None else 4
    gate, u, h0, dh, dfin = draw(3, tokens, channels, sequences, kind)

    def loss(g, v, s):
        h, final, _, _ = ref.forward(g, v, s, kind, sequences, offsets)
        return float((h * dh).sum() + (final * dfin).sum())

    h, _, _, _ = ref.forward(gate, u, h0, kind, sequences, offsets)
    got = ref.backward(gate, u, h, h0, dh, dfin, kind, sequences, offsets)[:3]
    step = 1e-5
    for which, grad in enumerate(got):
        args = [gate, u, h0]
        for i in np.ndindex(grad.shape):
            ends = []
            for sign in (1, -1):
                moved = [a.copy() for a in args]
                moved[which][i] += sign * step
                ends.append(loss(*moved))
            # a central difference is off by step^2 / 6 of the third derivative, and by rounding / step
            assert abs((ends[0] - ends[1]) / (2 * step) - grad[i]) < 1e-7


@pytest.mark.parametrize("kind", ["log", "logit"])
def test_packed_equals_each_sequence_alone(kind):
    offsets = (0, 4, 4, 5, 11)
    gate, u, h0, dh, dfin = draw(5, 11, 2, 4, kind)
    h, final, _, _ = ref.forward(gate, u, h0, kind, 4, offsets)
    grads = ref.backward(gate, u, h, h0, dh, dfin, kind, 4, offsets)
    for s, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        one, fin, _, _ = ref.forward(gate[lo:hi], u[lo:hi], h0[s:s + 1], kind, 1)
        assert np.array_equal(one, h[lo:hi]) and np.array_equal(fin[0], final[s])
        g = ref.backward(gate[lo:hi], u[lo:hi], one, h0[s:s + 1], dh[lo:hi], dfin[s:s + 1], kind, 1)
        assert np.array_equal(g[0], grads[0][lo:hi]) and np.array_equal(g[1], grads[1][lo:hi])
        assert np.array_equal(g[2][0], grads[2][s])


def test_checkpoint_against_rationals():
    rng = np.random.default_rng(7)
    x = (rng.normal(size=(6, 100)) * np.exp(rng.normal(size=(6, 1)) * 3)).astype(np.float32)
    x[0, 64:] = 0                                       # a block of zeros
    x[1, :3] = (254.0, 1.0, 3.0)                        # scale 2: 1 / 2 and 3 / 2 are ties
    x[1, 3:64] = -5.0                                   # -5 / 2 is a tie as well
    x[2, :64] = np.float32(1e-37)                       # below the smallest scale
    codes, scale = ref.checkpoint(x)
    for r in range(6):
        for i in range(100):
            m = max(abs(Fraction(float(v))) for v in x[r, i // 64 * 64:i // 64 * 64 + 64])
            s = Fraction(float(scale[r, i // 64]))
            if s == 0:
                assert m < 127 * Fraction(2) ** -126 and codes[r, i] == 0
                continue
            assert abs(s - m / 127) <= m / 127 * Fraction(1, 1 << 23)   # the constant and the product, rounded each
            assert int(codes[r, i]) == round(Fraction(float(x[r, i])) / s)   # round() of a Fraction: ties to even
    assert list(codes[1, :4]) == [127, 0, 2, -2]
