"""Calls of the block's operators that are large enough to take other ways: stores past the caches above 256 MiB, four
sequences a lane, offsets past 32 bits."""
import numpy as np
import pytest
import torch

import ref_block as ref
import test_gpu_rows
import test_gpu_selective
from test_gpu_selective import DEV, TYPES, Scan, close, cuts, lib

CACHE = 256 << 20     # bytes touched, above which stores pass the caches by
STEPS = [(67, 4096, 16), (130, 2050, 13), (66, 1025, 64), (1030, 257, 3), (259, 1000, 8), (129, 1031, 33)]


@pytest.mark.parametrize("batch,channels,n", STEPS)
def test_steps_of_four_sequences_a_lane(batch, channels, n):
    assert lib().selective_step_plan(batch, channels, n) == 4 and batch % 4


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,channels,n", STEPS)
def test_step(dtype, batch, channels, n):
    """Two tokens of every sequence; the last sequence, beside a call with it alone: its state moves once a call."""
    s = lib()
    assert s.selective_step_plan(batch, channels, n) == 4 and s.selective_step_plan(1, channels, n) == 1
    d = Scan(n, dtype, batch, batch * 2, channels, n)
    state, last = d.h0.clone(), d.h0[-1:].clone()
    want, want_final, wrong, wrong_final = d.reference()
    for t in range(2):
        at = lambda x: x[:, t].clone()
        end = lambda x: x[-1:, t].clone()
        y = s.selective_step(state, at(d.u), at(d.delta), d.A, at(d.B), at(d.C), d.D, at(d.z), d.bias)
        alone = s.selective_step(last, end(d.u), end(d.delta), d.A, end(d.B), end(d.C), d.D, end(d.z), d.bias)
        assert torch.equal(y[-1:], alone) and torch.equal(state[-1:], last)
        w = lambda x: x.reshape(batch, 2, channels)[:, t]
        close(y, w(want), w(wrong), d.dtype, f"token {t}")
    close(state, want_final, wrong_final, torch.float32, "state")


def device(seed, shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(seed))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("source", ["plain", "same", "f32", "gate"])
@pytest.mark.parametrize("channels,groups", [(4099, 1), (1000, 1), (200, 1), (8192, 8)])
def test_norms_of_more_than_the_caches_hold(dtype, source, channels, groups):
    s, t = lib(), TYPES[dtype]
    if source != "gate":
        groups = 1
    rows = CACHE // (channels * (t.itemsize + 1)) + 1001     # norms to codes, the fewest bytes, are above it too
    x, w = device(1, (rows, channels), t), device(2, (channels,), torch.float32)
    other = device(3, (rows, channels), torch.float32 if source == "f32" else t) if source != "plain" else None
    some = torch.from_numpy(np.unique(np.concatenate([[0, 1, rows - 2, rows - 1], np.random.default_rng(1).integers(0, rows, 200)]))).to(DEV)
    of = lambda v: None if v is None else v[some].double().cpu().numpy()
    kw = {"gate": of(other), "groups": groups} if source == "gate" else {"residual": of(other)}
    n, v, bound = ref.norm(of(x), w.double().cpu().numpy(), **kw)
    static = torch.tensor([0.02], device=DEV)
    if source == "gate":
        out, moved = s.gated_rms_norm(x, other, w, groups=groups), None
        codes, scale = s.gated_rms_norm_i8(x, other, w, groups=groups)
        fixed, _ = s.gated_rms_norm_i8(x, other, w, groups=groups, scale=static)
    else:
        out, moved = s.rms_norm(x, w, other)
        codes, scale, moved8 = s.rms_norm_i8(x, w, other)
        fixed, _, _ = s.rms_norm_i8(x, w, other, scale=static)
        assert (moved is None) == (moved8 is None) and (moved is None or torch.equal(moved, moved8))
    close(out[some], n, bound, t, "norm")
    test_gpu_rows.check_codes(codes[some], scale[some], n, bound)
    quotient = n / static.double().item()
    off = np.abs(fixed[some].cpu().numpy() - np.clip(quotient, -127, 127))
    assert np.all(off <= 0.5 + np.minimum(np.abs(quotient), 128) * (np.max(bound / np.maximum(np.abs(n), 1e-300)) + 2 * ref.E))
    if moved is not None:
        close(moved[some], v, np.abs(v) * ref.E, moved.dtype, "residual")
    # every row, against the same rows in calls that stay within the caches
    edges = np.linspace(0, rows, 8).astype(int).tolist()
    for part in map(slice, edges, edges[1:]):
        if source == "gate":
            assert torch.equal(out[part], s.gated_rms_norm(x[part].clone(), other[part].clone(), w, groups=groups))
            got = s.gated_rms_norm_i8(x[part].clone(), other[part].clone(), w, groups=groups)
        else:
            more = None if other is None else other[part].clone()
            assert torch.equal(out[part], s.rms_norm(x[part].clone(), w, more)[0])
            got = s.rms_norm_i8(x[part].clone(), w, more)
        assert torch.equal(codes[part], got[0]) and torch.equal(scale[part], got[1])


class Convolution:
    """A convolution made on the device, with the reference over some of the channels."""

    def __init__(self, dtype, sequences, tokens, channels, width, offsets):
        t = TYPES[dtype]
        self.type, self.sequences, self.at, self.channels = t, sequences, offsets, channels
        lead = (tokens,) if offsets is not None else (sequences, tokens // sequences)
        self.offsets = None if offsets is None else torch.from_numpy(offsets).to(DEV)
        self.x, self.state = device(1, (*lead, channels), t), device(4, (sequences, width - 1, channels), t)
        self.weight, self.bias = device(2, (channels, width), torch.float32), device(3, (channels,), torch.float32)

    def run(self, **more):
        return lib().causal_conv(self.x, self.weight, self.bias, self.state, offsets=self.offsets, **more)

    def check(self, selected, rows, out, kept):
        """Rows `rows` (a slice that begins with a sequence's first) of the selected channels."""
        pick, host = torch.from_numpy(selected).to(DEV), lambda v: v.double().cpu().numpy()
        flat = lambda v: host(v.view(-1, self.channels)[rows].index_select(1, pick))
        tokens = self.x.numel() // self.channels
        cuts_ = ref.spans(self.sequences, tokens, self.at)
        which = [s for s, (lo, hi) in enumerate(cuts_) if rows.start <= lo and hi <= rows.stop]
        at = np.array([cuts_[s][0] for s in which] + [cuts_[which[-1]][1]]) - rows.start
        want, want_kept, bound = ref.conv(flat(self.x), host(self.weight[pick]), host(self.bias[pick]),
                                          host(self.state[which].index_select(2, pick)), len(which), at)
        inside = slice(at[0], at[-1])
        close(torch.from_numpy(flat(out)[inside]), want[inside], bound[inside], self.type, "conv")
        assert np.array_equal(host(kept[which].index_select(2, pick)), want_kept)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("channels,sequences,packed", [(4099, 3, False), (2050, 300, True), (3, 2, True)])
def test_convolutions_of_more_than_the_caches_hold(dtype, width, channels, sequences, packed):
    """(with 3 channels a lane has fewer than four)"""
    tokens = CACHE // (2 * channels * TYPES[dtype].itemsize) + 999
    tokens -= 0 if packed else tokens % sequences
    at = cuts(5, sequences, tokens, 3, 9) if packed else None
    d = Convolution(dtype, sequences, tokens, channels, width, at)
    out, kept = d.run(out=torch.full_like(d.x, 9.0))
    selected = np.unique(np.concatenate([[0, channels - 1], np.random.default_rng(2).integers(0, channels, 30)]))
    spans = ref.spans(sequences, tokens, at)
    if channels > 3:
        d.check(selected, slice(0, tokens), out, kept)
    if packed:
        assert bool((out[:3] == 9.0).all()) and bool((out[-9:] == 9.0).all())
    # all channels and rows, against the same sequences in calls that stay within the caches
    flat, flat_out = d.x.view(-1, channels), out.view(-1, channels)
    for s in range(0, sequences, 1 if sequences < 9 else 37):
        lo, hi = spans[s]
        state, length = d.state[s:s + 1].clone(), 4 * (CACHE // 16 // channels // 4)
        for first in range(lo, hi, length):
            last = min(first + length, hi)
            got, state = lib().causal_conv(flat[first:last].clone().view(1, -1, channels), d.weight, d.bias, state)
            assert torch.equal(got[0], flat_out[first:last])
        assert torch.equal(state, kept[s:s + 1])


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_a_convolution_past_32_bit_offsets(packed):
    tokens, channels = 70000, 32768                          # 2.3e9 elements
    at = np.array([0, 10, 65000, 65530, 65530, 65600, 69990], np.int32) if packed else None
    d = Convolution("bf16", len(at) - 1 if packed else 70, tokens, channels, 4, at)
    out, kept = d.run()
    selected = np.array([0, 1, 255, 256, 16385, channels - 2, channels - 1])
    for rows in (slice(0, 1000),) * (not packed) + (slice(65000, 66000), slice(65600 if packed else 69000, 70000)):
        d.check(selected, rows, out, kept)
