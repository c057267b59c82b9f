"""Norms of rows whose squares are beyond binary32's small end, with an eps of 0 or too small to stand in for them."""
import numpy as np
import pytest
import torch

import ref_block as ref
from test_gpu_rows import DEV, TYPES, check_codes, close, draw, host, lib

pytestmark = pytest.mark.gpu
# largest magnitudes of the rows: ordinary, squares that lose digits, squares of 0, subnormal numbers
SIZES = [1.0, 300.0, 1e-3, 1e-17, 1e-19, 1e-21, 1e-23, 1e-30, 1e-36, 3e-39, 1e-42, 1e15]


def rows_of(seed, channels, dtype, tiny=0.0):
    """One row of every size (below `tiny` none); what the type rounds to zero throughout becomes ones."""
    x = draw(seed, (len(SIZES), channels), torch.float32)
    x = x / x.abs().amax(-1, keepdim=True)
    size = torch.tensor([max(s, tiny) for s in SIZES], dtype=torch.float64, device=DEV)
    x = (x.double() * size[:, None]).to(dtype)
    x[x.abs().amax(-1) == 0] = 1
    x[torch.isinf(x).any(-1)] = 1
    return x


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 1e-30, 1e-20])
@pytest.mark.parametrize("channels", [1, 7, 64, 1531, 4096, 16391, 32768])
def test_norm(dtype, eps, channels):
    s, t = lib(), TYPES[dtype]
    x, w = rows_of(channels, channels, t), draw(7, (channels,), torch.float32)
    for res in (None, rows_of(3, channels, t), rows_of(4, channels, torch.float32)):
        with np.errstate(invalid="ignore"):
            n, v, bound = ref.norm(host(x), host(w), None if res is None else host(res), eps=float(np.float32(eps)))
        out, moved = s.rms_norm(x, w, res, eps=eps)
        codes, scale, _ = s.rms_norm_i8(x, w, res, eps=eps)
        at = lambda rows: torch.from_numpy(rows).to(DEV)
        some = v.any(-1) | (float(np.float32(eps)) > 0)                      # (one channel may cancel: 0 / 0)
        assert torch.isnan(out[at(~some)]).all() and torch.isnan(scale[at(~some)]).all() and not codes[at(~some)].any()
        # (outputs that are subnormal are rounded to multiples of 2^-149, twice)
        close(out[at(some)], n[some], bound[some] + 2.0 ** -148, t, f"norm {eps}")
        if res is not None:
            close(moved, v, np.abs(v) * ref.E, res.dtype, "residual")
        big = some & (np.abs(np.where(some[:, None], n, 0)).max(-1) > 1e-30)   # (below, codes may be zero)
        check_codes(codes[at(big)], scale[at(big)], n[big], bound[big])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("channels,groups", [(64, 4), (1000, 5), (4096, 16), (8192, 8), (16384, 2), (16384, 256), (77, 7)])
def test_groups_of_different_sizes(dtype, channels, groups):
    """A group of ordinary numbers beside one whose squares underflow, and rows of any size."""
    s, t = lib(), TYPES[dtype]
    x, z, w = rows_of(1, channels, t, 1e-30), draw(2, (len(SIZES), channels), t), draw(3, (channels,), torch.float32)
    x[2, :channels // groups] = x[7, :channels // groups]
    n, _, bound = ref.norm(host(x), host(w), gate=host(z), groups=groups, eps=0.0)
    close(s.gated_rms_norm(x, z, w, groups=groups, eps=0.0), n, bound, t, "gated")
    check_codes(*s.gated_rms_norm_i8(x, z, w, groups=groups, eps=0.0), n, bound)
    static = torch.tensor([0.02], device=DEV)
    codes, _ = s.gated_rms_norm_i8(x, z, w, groups=groups, eps=0.0, scale=static)
    quotient = n / host(static)
    off = np.abs(codes.cpu().numpy() - np.clip(quotient, -127, 127))
    assert np.all(off <= 0.5 + np.minimum(np.abs(quotient), 128) * (np.max(bound / np.maximum(np.abs(n), 1e-300)) + 2 * ref.E))


@pytest.mark.parametrize("channels", [40, 5000])
def test_zeros_and_what_is_not_finite_with_eps_0(channels):
    s = lib()
    x, w = rows_of(1, channels, torch.float32), torch.ones(channels, device=DEV)
    clean, _ = s.rms_norm(x, w, eps=0.0)
    x[1], x[3, 5], x[5, 0], x[7] = 0, float("nan"), float("inf"), 3e38       # the last one's squares overflow
    out, _ = s.rms_norm(x, w, eps=0.0)
    codes, scale, _ = s.rms_norm_i8(x, w, eps=0.0)
    for row in range(len(SIZES)):
        if row in (1, 3, 5, 7):
            assert torch.isnan(out[row]).all() and torch.isnan(scale[row]) and not codes[row].any()
        else:
            assert torch.equal(out[row], clean[row]) and torch.isfinite(scale[row])
    x[1] = 0
    assert not s.rms_norm(x, w, eps=1e-40)[0][1].any()


def test_ordinary_rows_have_the_same_bits_with_any_small_eps():
    """An eps that vanishes beside mean(v^2) changes no bit, whichever way the sum is formed."""
    s = lib()
    for channels in (100, 3000, 20000):
        x, w = draw(1, (50, channels), torch.float32), draw(2, (channels,), torch.float32)
        want, _ = s.rms_norm(x, w, eps=1e-15)
        for eps in (0.0, 1e-40, 1e-25):
            assert torch.equal(s.rms_norm(x, w, eps=eps)[0], want)


def test_many_rows_past_the_caches():
    s = lib()
    x, w = draw(1, (40000, 1700), torch.float32), draw(2, (1700,), torch.float32)
    x[5::7] *= 1e-25
    out, _ = s.rms_norm(x, w, eps=0.0)
    some = torch.arange(0, 40000, 611, device=DEV)
    n, _, bound = ref.norm(host(x[some]), host(w), eps=0.0)
    close(out[some], n, bound, torch.float32, "norm")


@pytest.mark.parametrize("power", [-126, -100, 0, 100, 114])
def test_static_scales_of_every_size(power):
    """From the smallest scale that is allowed to the largest."""
    s = lib()
    x, w = draw(1, (40, 1000), torch.float32), draw(2, (1000,), torch.float32)
    w = (w.double() * 2.0 ** (power + 5)).float()                            # quotients around 32, some beyond 127
    scale = torch.tensor([1.1 * 2.0 ** power], dtype=torch.float64).float().to(DEV)
    n, _, bound = ref.norm(host(x), host(w))
    codes, _, _ = s.rms_norm_i8(x, w, scale=scale)
    quotient = n / host(scale)
    # (at the lower end products and n are subnormal: off by 2^-149 each, 2^-23 of the scale)
    off = np.abs(codes.cpu().numpy() - np.clip(quotient, -127, 127))
    assert np.all(off <= 0.5 + 2.0 ** -20 + np.minimum(np.abs(quotient), 128) * (np.max(bound / np.abs(n)) + 2 * ref.E))
    assert np.abs(codes.cpu().numpy()).max() == 127 and (np.abs(quotient) < 60).any()
