"""8-bit activation checkpoints on the GPU: codes and scales equal to the exact ones, and their values."""
import numpy as np
import pytest
import torch

import ref_gated as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda:0"


def lib():
    import quantized_selective_state_amd as ssdq
    return ssdq


def check(x):
    ssdq = lib()
    codes, scale = ssdq.checkpoint_save(x)
    want_codes, want_scale = ref.checkpoint(x.float().cpu().numpy().reshape(-1, x.shape[-1]))
    torch.cuda.synchronize()
    got = scale.cpu().numpy().reshape(want_scale.shape)
    assert np.array_equal(got, want_scale, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy().reshape(want_codes.shape), want_codes)
    # values: one product in binary32, one rounding
    wide = torch.from_numpy(np.repeat(want_scale, 64, axis=1)[:, :x.shape[-1]])
    values = torch.from_numpy(want_codes).float() * wide
    for t in TYPES.values():
        back = ssdq.checkpoint_load(codes, scale, t)
        assert back.dtype == t and torch.equal(torch.nan_to_num(back.cpu().view(values.shape), nan=1e4),
                                               torch.nan_to_num(values.to(t), nan=1e4))
    return codes, scale


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 1), (1, 64), (3, 65), (5, 7), (77, 1000), (64, 4096), (2, 3, 130), (1000, 8),
                                   (33, 200), (4097, 64)], ids=str)
def test_against_the_exact_codes(shape, dtype):
    g = torch.Generator(device=DEV).manual_seed(sum(shape))
    x = torch.randn(shape, generator=g, device=DEV) * torch.randn(shape[-1], generator=g, device=DEV).exp()
    check(x.to(TYPES[dtype]))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_ties_zeros_and_extremes(dtype):
    t = TYPES[dtype]
    x = torch.zeros(12, 128, device=DEV)
    x[0, :64] = torch.arange(-32, 32, device=DEV) * 0.5 + 0.5            # with 127 below: scale 1, every half a tie
    x[0, 5] = 127.0
    x[1, :64] = torch.arange(64, device=DEV).float()                     # with 254: scale 2, every odd number a tie
    x[1, 7] = -254.0
    x[2, 3] = torch.finfo(t).max
    x[3, 64:] = torch.finfo(t).tiny
    x[4, 9] = float("nan")
    x[5, 100] = float("inf")
    x[6, 1] = -float("inf")
    x[7, :64] = -1.0                                                     # every element the largest
    x[8, 2] = 127 * 2.0 ** -14                                           # scale 2^-14
    x[9, 4] = torch.finfo(t).tiny * 0.5                                  # a subnormal of fp16
    x[10, 6] = 1e-37 if t != torch.float16 else 0.0                      # below the smallest scale
    check(x.to(t))


def test_reads_any_code():
    codes = torch.arange(-128, 128, device=DEV).to(torch.int8).view(2, 128)
    scale = torch.tensor([[0.1, 3.0], [1e-30, 0.0]], device=DEV)
    got = lib().checkpoint_load(codes, scale, torch.float32)
    want = codes.cpu().float() * scale.cpu().repeat_interleave(64, 1)
    assert torch.equal(got.cpu(), want)


def test_empty_and_given_buffers():
    ssdq = lib()
    codes, scale = ssdq.checkpoint_save(torch.empty(0, 70, device=DEV))
    assert codes.shape == (0, 70) and scale.shape == (0, 2) and ssdq.checkpoint_load(codes, scale, torch.half).numel() == 0
    x = torch.randn(5, 70, device=DEV)
    out = ssdq.checkpoint_empty(x)
    again = ssdq.checkpoint_save(x, out=out)
    assert again[0] is out[0] and again[1] is out[1]
    back = torch.empty_like(x)
    assert ssdq.checkpoint_load(*out, x.dtype, out=back) is back
    # a code is off by at most half a scale, plus the rounding of the scale and of the product
    wide = out[1].repeat_interleave(64, 1)[:, :70]
    assert bool(((back - x).abs() <= wide * (0.5 + 127 * 2.0 ** -23)).all())


def test_refusals():
    ssdq = lib()
    x = torch.randn(4, 128, device=DEV)
    codes, scale = ssdq.checkpoint_save(x)
    for call in (lambda: ssdq.checkpoint_save(x.double()), lambda: ssdq.checkpoint_save(x.t()),
                 lambda: ssdq.checkpoint_save(x, out=(codes, scale[:2])), lambda: ssdq.checkpoint_save(x, out=(codes.float(), scale)),
                 lambda: ssdq.checkpoint_load(codes, scale[:, :1].contiguous(), torch.half),
                 lambda: ssdq.checkpoint_load(codes, scale, torch.float64),
                 lambda: ssdq.checkpoint_load(codes, scale, torch.half, out=x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ssdq.SSDQError):
        ssdq.checkpoint_load(torch.zeros(129, dtype=torch.int8, device=DEV)[1:].view(1, 128), scale[:1], torch.half)


def test_more_blocks_than_a_launch_holds():
    """A grid holds fewer than 2^32 threads and a row of one channel takes 16: 2^28 rows are several launches."""
    ssdq, rows = lib(), 2 ** 28 + 5
    x = torch.randn(rows, 1, device=DEV, dtype=torch.bfloat16)
    x[::1000] = 0
    codes, scale = ssdq.checkpoint_save(x)
    assert torch.equal(codes, (127 * x.sign()).to(torch.int8))               # a block of one channel: code 127
    assert torch.equal(scale, x.float().abs() * torch.tensor(1 / 127, device=DEV))
    back = ssdq.checkpoint_load(codes, scale, torch.bfloat16)
    assert torch.equal(back, (codes.float() * scale).to(torch.bfloat16))


@pytest.mark.parametrize("channels", [2 ** 31 - 1, 2 ** 31 - 8], ids=["one-lane-each", "vectors"])
def test_the_longest_rows(channels):
    """Rows of nearly 2^31 channels: 2^25 blocks, whose last one equals the same channels as a row alone."""
    ssdq = lib()
    x = torch.full((1, channels), 0.5, device=DEV, dtype=torch.bfloat16)
    lo = channels // 64 * 64 - 6400                                           # the last blocks, a partial one among them
    x[0, lo:] = torch.randn(channels - lo, device=DEV)
    codes, scale = ssdq.checkpoint_save(x)
    assert scale.shape == (1, 2 ** 25)
    want_codes, want_scale = ssdq.checkpoint_save(x[:, lo:].clone())
    assert torch.equal(codes[:, lo:], want_codes) and torch.equal(scale[:, lo // 64:], want_scale)
    assert bool((codes[:, :lo] == 127).all())
    assert bool((scale[:, :lo // 64] == torch.tensor(0.5, device=DEV) * torch.tensor(1 / 127, device=DEV)).all())
    back = ssdq.checkpoint_load(codes, scale, torch.bfloat16)
    assert torch.equal(back[:, lo:], ssdq.checkpoint_load(want_codes, want_scale, torch.bfloat16))
    assert bool((back[:, :lo] == 0.5).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(8192, 1531), (2048, 4095)], ids=str)
def test_large_activations_in_widths_that_no_vector_divides(shape, dtype):
    g = torch.Generator(device=DEV).manual_seed(shape[1])
    check(torch.randn(shape, generator=g, device=DEV).to(TYPES[dtype]))


@pytest.mark.parametrize("channels", [1, 63, 65, 1531])
def test_ragged_rows_leave_their_neighbours(channels):
    """Codes, scales and values written inside larger buffers: nothing before or behind them changes."""
    ssdq, rows = lib(), 77
    blocks = -(-channels // 64)
    for t in TYPES.values():
        x = torch.randn(rows, channels, device=DEV).to(t)
        edge = 1024
        rooms = [torch.full((rows * w + 2 * edge,), 77, dtype=kind, device=DEV)
                 for w, kind in ((channels, torch.int8), (blocks, torch.float32), (channels, t))]
        codes, scale, back = (r[edge:-edge].view(rows, -1) for r in rooms)
        ssdq.checkpoint_save(x, out=(codes, scale))
        ssdq.checkpoint_load(codes, scale, t, out=back)
        want = ssdq.checkpoint_save(x)
        assert torch.equal(codes, want[0]) and torch.equal(scale, want[1])
        assert torch.equal(back, ssdq.checkpoint_load(*want, t))
        assert all(bool((r[:edge] == 77).all()) and bool((r[-edge:] == 77).all()) for r in rooms)
