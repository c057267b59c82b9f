"""The selective scan in chunks of several tiles of 16 rows, against the 64-bit reference.

A chunk has as many rows as fill the waves of the device a whole number of times, so long chunks take many channels; the
reference follows some of them, since channels do not meet.  Every size's plan is asserted, on the CPU too."""
import numpy as np
import pytest
import torch

import ref_block as ref
from test_gpu_selective import DEV, TYPES, close, lib, put

TILE = 16

# (sequences, tokens, channels, states, rows of a chunk): up to 8, 16, 32 and 64 states; chunks that end in tiles of 4, 8 and
# 12 rows and, of 256 rows, the longest
DENSE = [(1, 2001, 4096, 8, 44), (1, 2001, 4096, 5, 44), (2, 2002, 4096, 16, 44), (1, 1301, 2500, 13, 20),
         (1, 2001, 4096, 24, 84), (1, 2001, 4090, 32, 84), (1, 2001, 4096, 64, 168), (2, 4002, 2000, 41, 168)]
PACKED = [(2001, 4096, 8, 44), (2001, 4096, 16, 44), (3003, 4000, 13, 64), (2001, 4096, 24, 84), (2001, 4090, 64, 168),
          (1000, 3000, 1, 16)]
LONGEST = [(512, 196608, 8, 256), (512, 196608, 16, 256), (512, 98304, 30, 256), (512, 49152, 64, 256)]


@pytest.mark.parametrize("sequences,tokens,channels,n,chunk", DENSE)
def test_dense_sizes_have_these_chunks(sequences, tokens, channels, n, chunk):
    assert lib().selective_scan_plan(sequences, tokens, channels, n) == chunk


@pytest.mark.parametrize("tokens,channels,n,chunk", PACKED + LONGEST)
def test_packed_sizes_have_these_chunks(tokens, channels, n, chunk):
    assert lib().selective_scan_plan(9, tokens, channels, n, True) == chunk


def some_channels(seed, channels, count=150):
    edges = [0, 1, 63, 64, 65, 127, 128, 255, 256, channels // 2, channels - 65, channels - 2, channels - 1]
    more = np.random.default_rng(seed).integers(0, channels, count - len(edges))
    return np.unique(np.concatenate([edges, more]) % channels)


def cuts_of(chunk, tokens, before, behind):
    """Sequences that begin and end at chunk edges, in first and later tiles, beside tiles' edges and inside of groups of 4
    rows; some of one token, some empty, one over several chunks."""
    at = [before, chunk, chunk, chunk + 1, chunk + TILE - 1, chunk + TILE, chunk + TILE + 5, 2 * chunk - 1, 2 * chunk,
          2 * chunk + min(2 * TILE + 3, chunk - 2), 3 * chunk - 3, 3 * chunk - 2, 3 * chunk, 4 * chunk - 1, 4 * chunk + 2]
    at = [t for t in at if before <= t <= tokens - behind]
    return np.array(sorted(at) + [tokens - behind] * 2, np.int32)


class Wide:
    """Inputs made on the device, and the reference over some of the channels."""

    def __init__(self, seed, dtype, sequences, tokens, channels, n, offsets=None):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=gen, device=DEV)
        t = TYPES[dtype]
        self.type, self.sequences, self.tokens, self.at = t, sequences, tokens, offsets
        self.offsets = None if offsets is None else torch.from_numpy(offsets).to(DEV)
        lead = (tokens,) if offsets is not None else (sequences, tokens // sequences)
        self.u, self.z = normal(*lead, channels).to(t), (normal(*lead, channels) * 2).to(t)
        # steps of 0.001 to 1: states that live for some tokens and ones that live for many chunks
        self.delta = (normal(*lead, channels) * 0.5).to(t)
        self.bias = -torch.rand(channels, generator=gen, device=DEV) * 7
        self.A = -torch.exp(torch.log(torch.arange(1, n + 1, device=DEV)) + 0.1 * normal(channels, n))
        self.B, self.C, self.D = normal(*lead, n).to(t), normal(*lead, n).to(t), normal(channels)
        self.h0 = normal(sequences, channels, n)

    def run(self, **more):
        return lib().selective_scan(self.u, self.delta, self.A, self.B, self.C, self.D, self.z, self.bias, self.h0,
                                    offsets=self.offsets, **more)

    def check(self, selected, **more):
        y, final = self.run(**more)
        pick = torch.from_numpy(selected).to(DEV)
        host = lambda x: x.double().cpu().numpy()
        flat = lambda x: x.reshape(-1, x.shape[-1])
        of = lambda x: host(flat(x).index_select(1, pick))
        want, want_final, wrong, wrong_final = ref.scan(
            of(self.u), of(self.delta), host(self.A[pick]), host(flat(self.B)), host(flat(self.C)), host(self.D[pick]),
            of(self.z), host(self.bias[pick]), host(self.h0.index_select(1, pick)), self.sequences, self.at)
        inside = np.zeros(self.tokens, bool)
        for lo, hi in ref.spans(self.sequences, self.tokens, self.at):
            inside[lo:hi] = True
        got = flat(y).index_select(1, pick)[torch.from_numpy(inside).to(DEV)]
        close(got, want[inside], wrong[inside], self.type, "y")
        close(final.index_select(1, pick), want_final, wrong_final, torch.float32, "h_final")
        return y, final, torch.from_numpy(~inside).to(DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sequences,tokens,channels,n,chunk", DENSE)
def test_dense(dtype, sequences, tokens, channels, n, chunk):
    assert lib().selective_scan_plan(sequences, tokens, channels, n) == chunk > TILE
    Wide(tokens + n, dtype, sequences, tokens, channels, n).check(some_channels(n, channels))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("before,behind", [(0, 0), (7, 29)])
@pytest.mark.parametrize("tokens,channels,n,chunk", PACKED)
def test_packed(dtype, before, behind, tokens, channels, n, chunk):
    at = cuts_of(chunk, tokens, before, behind)
    assert lib().selective_scan_plan(len(at) - 1, tokens, channels, n, True) == chunk
    d = Wide(tokens + n, dtype, len(at) - 1, tokens, channels, n, at)
    y, _, outside = d.check(some_channels(n, channels), y=torch.full_like(d.u, 9.0))
    assert bool((y[outside] == 9.0).all())                                   # rows of no sequence stay


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,channels,n,chunk", LONGEST)
def test_longest_chunks(tokens, channels, n, chunk):
    at = np.array([0, 100, 300, 512], np.int32)                              # one carried over the edge at 256
    assert lib().selective_scan_plan(3, tokens, channels, n, True) == chunk
    Wide(n, "bf16", 3, tokens, channels, n, at).check(some_channels(n, channels))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [8, 16, 24, 64])
def test_same_bits_in_any_workspace_and_what_is_not_finite_stays(n):
    sequences, tokens, channels = 9, 2001, 4096
    at = np.array([0, 30, 30, 31, 500, 700, 1001, 1500, 1999, 2001], np.int32)
    assert lib().selective_scan_plan(sequences, tokens, channels, n, True) > 2 * TILE
    d = Wide(n, "f32", sequences, tokens, channels, n, at)
    need = lib().selective_scan_workspace_size(sequences, tokens, channels, n, True)
    y, final = d.run(workspace=torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV))
    again, final2 = d.run(workspace=torch.zeros(need, dtype=torch.uint8, device=DEV))
    assert torch.equal(y, again) and torch.equal(final, final2)
    d.u[550, 70], d.delta[900, 4000], d.z[1200, 5], d.h0[7, 9, 0] = (float("nan"),) * 4
    d.B[1450, n - 1] = float("nan")
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[550:700, 70] = bad[900:1001, 4000] = bad[1200, 5] = bad[1500:1999, 9] = bad[1450:1500] = True
    got, got_final = d.run()
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], y[~bad])
    same = torch.ones(sequences, channels, dtype=torch.bool, device=DEV)
    same[4, 70] = same[5, 4000] = same[7, 9] = False
    same[6] = False
    assert torch.equal(got_final[same], final[same])
    assert torch.isnan(got_final[4, 70]).all() and torch.isnan(got_final[5, 4000]).all() and torch.isnan(got_final[7, 9, 0])
    assert torch.isnan(got_final[6, :, n - 1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_rows_past_32_bit_offsets(packed):
    """2.3e9 elements: the last rows, against the reference and beside a call that has them alone."""
    length, sequences, channels, n = 1000, 70, 32768, 16
    tokens = length * sequences
    plan = lib().selective_scan_plan(sequences, tokens, channels, n, packed)
    assert plan == 0 if not packed else plan > TILE
    gen = torch.Generator(device=DEV).manual_seed(1)
    wide = lambda: torch.empty(tokens, channels, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    u, delta, z = wide(), wide(), wide()
    B, C = (torch.empty(tokens, n, dtype=torch.bfloat16, device=DEV).normal_(generator=gen) for _ in "BC")
    A = -torch.rand(channels, n, generator=gen, device=DEV) * 4
    h0 = torch.randn(sequences, channels, n, generator=gen, device=DEV)
    lead = (tokens,) if packed else (sequences, length)
    at = (torch.arange(sequences + 1, device=DEV) * length).int() if packed else None
    y, final = lib().selective_scan(u.view(*lead, channels), delta.view(*lead, channels), A, B.view(*lead, n), C.view(*lead, n),
                                    z=z.view(*lead, channels), h0=h0, offsets=at)
    y, pick, host = y.view(tokens, channels), torch.from_numpy(some_channels(2, channels, 40)).to(DEV), lambda x: x.double().cpu().numpy()
    for s in (0, 65, sequences - 1):                         # (the one that 2^31 elements end in, too)
        rows = slice(s * length, (s + 1) * length)
        of = lambda x: host(x[rows].index_select(1, pick))
        want, want_final, wrong, wrong_final = ref.scan(of(u), of(delta), host(A[pick]), host(B[rows]), host(C[rows]), None, of(z),
                                                        None, host(h0[s:s + 1].index_select(1, pick)), 1, None)
        close(y[rows].index_select(1, pick), want, wrong, torch.bfloat16, f"y {s}")
        close(final[s:s + 1].index_select(1, pick), want_final, wrong_final, torch.float32, f"h_final {s}")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 5, 13, 20, 41])
def test_an_infinity_stays_in_its_channel_with_any_number_of_states(n):
    """Whole and in chunks; numbers of states that the kernels fill up."""
    for sequences, tokens, channels in ((2, 2002, 2200), (60, 600, 1100)):
        d = Wide(n, "f32", sequences, tokens, channels, n)
        y, final = d.run()
        half = tokens // sequences // 2
        d.u[1, half, 3] = float("inf")
        got, got_final = d.run()
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[1, half:, 3] = True
        assert not torch.isfinite(got[bad]).any() and torch.equal(got[~bad], y[~bad])
        assert not torch.isfinite(got_final[1, 3]).any()
        got_final[1, 3] = final[1, 3]
        assert torch.equal(got_final, final)
