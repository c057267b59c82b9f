"""Packed calls with very many sequences without tokens: a run of them is left by a search, not walked one by one."""
import numpy as np
import pytest
import torch

import ref_block as ref
from test_gpu_selective import DEV, close, lib

pytestmark = pytest.mark.gpu
EMPTY = 1 << 18


def case(tokens, channels, n, seed=1):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=gen, device=DEV)
    # real sequences between runs of empty ones: at the front, inside a chunk, at a chunk's edge, behind
    real = [5, 20, 64, 101, tokens - 7]
    at = np.concatenate([np.full(EMPTY, real[0]), [real[1]], np.full(EMPTY, real[1]), [real[2]], np.full(EMPTY, real[2]), [real[3]],
                         np.full(EMPTY, real[3]), np.full(EMPTY, real[4])]).astype(np.int32)
    which = [EMPTY - 1, 2 * EMPTY, 3 * EMPTY + 1, 4 * EMPTY + 2]
    for s, lo, hi in zip(which, real, real[1:]):
        assert at[s] == lo and at[s + 1] == hi
    return at, np.array(real), torch.tensor(which, device=DEV), normal


def timed(run):
    run()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    result = run()
    end.record()
    torch.cuda.synchronize()
    print(f"  {start.elapsed_time(end):.2f} ms", flush=True)
    return result, start.elapsed_time(end)


@pytest.mark.parametrize("n", [2, 16, 20, 50])
def test_scan(n):
    tokens, channels = 150, 5
    at, real, which, normal = case(tokens, channels, n)
    sequences = len(at) - 1
    assert lib().selective_scan_plan(sequences, tokens, channels, n, True) == 16
    u, delta, z, B, C = normal(tokens, channels), normal(tokens, channels), normal(tokens, channels), normal(tokens, n), normal(tokens, n)
    A, h0 = -normal(channels, n).abs(), normal(sequences, channels, n)
    y, offsets = torch.full_like(u, 9.0), torch.from_numpy(at).to(DEV)
    (_, final), ms = timed(lambda: lib().selective_scan(u, delta, A, B, C, z=z, h0=h0, y=y, offsets=offsets))
    host = lambda t: t.double().cpu().numpy()
    want, want_final, wrong, wrong_final = ref.scan(host(u), host(delta), host(A), host(B), host(C), None, host(z), None,
                                                    host(h0[which]), 4, real)
    rows = slice(real[0], real[-1])
    close(y[rows], want[rows], wrong[rows], torch.float32, "y")
    close(final[which], want_final, wrong_final, torch.float32, "h_final")
    assert bool((y[:real[0]] == 9).all()) and bool((y[real[-1]:] == 9).all())
    rest = torch.ones(sequences, dtype=torch.bool, device=DEV)
    rest[which] = False
    assert torch.equal(final[rest], h0[rest])
    assert ms < 20                                           # (one by one 58 to 81, the convolution 37)


def test_convolution():
    tokens, channels = 150, 5
    at, real, which, normal = case(tokens, channels, 1)
    sequences = len(at) - 1
    x, weight, state = normal(tokens, channels), normal(channels, 4), normal(sequences, 3, channels)
    out, offsets = torch.full_like(x, 9.0), torch.from_numpy(at).to(DEV)
    (_, kept), ms = timed(lambda: lib().causal_conv(x, weight, None, state, offsets=offsets, out=out))
    host = lambda t: t.double().cpu().numpy()
    want, want_kept, bound = ref.conv(host(x), host(weight), None, host(state[which]), 4, real)
    rows = slice(real[0], real[-1])
    close(out[rows], want[rows], bound[rows], torch.float32, "conv")
    assert np.array_equal(host(kept[which]), want_kept)
    assert bool((out[:real[0]] == 9).all()) and bool((out[real[-1]:] == 9).all())
    rest = torch.ones(sequences, dtype=torch.bool, device=DEV)
    rest[which] = False
    assert torch.equal(kept[rest], state[rest])
    assert ms < 20
