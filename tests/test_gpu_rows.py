"""Row norms, rows of codes and their values on the GPU against the 64-bit references."""
import numpy as np
import pytest
import torch

import ref_block as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda:0"


def lib():
    import quantized_selective_state_amd as ssdq
    return ssdq


def half_step(dtype, values):
    info = torch.finfo(dtype)
    return np.abs(values) * info.eps / 2 + info.tiny * info.eps / 2


def draw(seed, shape, dtype, spread=1.0):
    rng = np.random.default_rng(seed)
    a = rng.normal(size=shape) * np.exp(rng.uniform(-spread, spread, shape[-1]))
    return torch.from_numpy(a.astype(np.float32)).to(dtype).to(DEV)


def host(t):
    return t.double().cpu().numpy()


def close(got, want, bound, dtype, what):
    allowed = bound + half_step(dtype, np.abs(want) + bound)
    off = np.abs(host(got).reshape(want.shape) - want)
    print(f"  {what}: {np.max(off / allowed) if want.size else 0.0:.3f} of the bound", flush=True)
    assert np.all(off <= allowed), what


# widths with whole and partial packs of 8, rows of one lane to 1024, and the widest
WIDTHS = [1, 7, 8, 63, 64, 65, 250, 511, 512, 1000, 1531, 2048, 2050, 4096, 5120, 8192, 16384, 16391, 32768]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("channels", WIDTHS)
def test_norm_with_residual(dtype, channels):
    s = lib()
    t = TYPES[dtype]
    for rows, kind in ((1, "f32"), (37, dtype), (300, None)):
        x, w = draw(channels + rows, (rows, channels), t), draw(7, (channels,), torch.float32)
        res = None if kind is None else draw(rows, (rows, channels), TYPES[kind], 0.5)
        n, v, bound = ref.norm(host(x), host(w), None if res is None else host(res))
        out, res_out = s.rms_norm(x, w, res)
        close(out, n, bound, t, f"norm {rows} {kind}")
        assert (res_out is None) == (res is None)
        codes, scale, res_out8 = s.rms_norm_i8(x, w, res)
        check_codes(codes, scale, n, bound)
        if res is not None:
            close(res_out, v, np.abs(v) * ref.E, res.dtype, "residual")
            assert torch.equal(res_out, res_out8)


def check_codes(codes, scale, n, bound):
    most = np.abs(n).max(-1)
    want = ref.row_scale(most).astype(np.float64)
    worst = np.max(bound / np.maximum(np.abs(n), 1e-300)) + 2 * ref.E       # relative, of n and of the largest |n|
    got = host(scale)
    assert np.all(np.abs(got - want) <= want * worst)
    q = codes.cpu().numpy().astype(np.float64)
    quotient = n / np.where(want > 0, want, 1.0)[:, None]
    assert np.all(np.abs(q - quotient) <= 0.5 + 127 * 2 * worst)
    assert np.all(np.abs(q) <= 127) and np.all(np.abs(q).max(-1) == np.where(want > 0, 127, 0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("channels,groups", [(8, 8), (64, 4), (96, 3), (1000, 5), (1536, 8), (4096, 2), (4096, 16), (8192, 8),
                                             (5120, 1), (16384, 256), (16384, 1), (16380, 4), (300, 100), (7 * 11, 7)])
def test_gated_norm_in_groups(dtype, channels, groups):
    s = lib()
    t = TYPES[dtype]
    for rows in (1, 29, 1025):
        if rows * channels > 1 << 23:
            continue
        x, z, w = draw(channels, (rows, channels), t), draw(groups, (rows, channels), t), draw(5, (channels,), torch.float32)
        n, _, bound = ref.norm(host(x), host(w), gate=host(z), groups=groups)
        close(s.gated_rms_norm(x, z, w, groups=groups), n, bound, t, f"gated {rows}")
        check_codes(*s.gated_rms_norm_i8(x, z, w, groups=groups), n, bound)


@pytest.mark.parametrize("dtype", TYPES)
def test_static_scale(dtype):
    s = lib()
    t = TYPES[dtype]
    x, w, res = draw(1, (53, 777), t), draw(2, (777,), torch.float32), draw(3, (53, 777), torch.float32)
    scale = torch.tensor([0.013], device=DEV)                                # many codes saturate
    n, _, bound = ref.norm(host(x), host(w), host(res))
    codes, got, _ = s.rms_norm_i8(x, w, res, scale=scale)
    assert got is scale
    q, quotient = codes.cpu().numpy().astype(np.float64), n / host(scale)
    assert np.all(np.abs(q - np.clip(quotient, -127, 127)) <= 0.5 + np.minimum(np.abs(quotient), 128) * (np.max(bound / np.abs(n)) + 2 * ref.E))
    assert (np.abs(q) == 127).any() and np.abs(q).max() == 127
    x[3, 5] = float("nan")
    x[4, 6] = float("inf")
    codes, _, _ = s.rms_norm_i8(x, w, res, scale=scale)
    assert not codes[3].any() and not codes[4].any()
    keep = [r for r in range(53) if r not in (3, 4)]
    assert np.array_equal(codes.cpu().numpy()[keep], q[keep])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("channels", [1, 8, 13, 64, 777, 2560, 4096, 32768])
def test_rows_are_exact(dtype, channels):
    s = lib()
    x = draw(channels, (65, channels), TYPES[dtype])
    x[3] = 0
    x[4, channels // 2] = float("nan")
    x[5, 0] = float("-inf")
    if dtype == "f32":
        x[6] = 1e-37                                                         # its scale would be subnormal
        x[7] *= 1e30
    codes, scale = s.quantize_rows(x)
    want_codes, want_scale = ref.rows(x.float().cpu().numpy())
    assert np.array_equal(scale.cpu().numpy(), want_scale, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    for t in TYPES.values():
        values = s.dequantize_rows(codes, scale, t)
        want = torch.from_numpy(want_codes.astype(np.float32) * want_scale[:, None]).to(t)
        assert torch.equal(values.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


def test_ties_to_even():
    s = lib()
    x = torch.zeros(2, 256, device=DEV)
    x[0] = torch.arange(256, device=DEV) * 0.5 - 63.5
    x[:, 0] = 127.0                                                          # scale: 127 * (1/127 in binary32)
    codes, scale = s.quantize_rows(x)
    want_codes, want_scale = ref.rows(x.cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), want_codes) and np.array_equal(scale.cpu().numpy(), want_scale)


@pytest.mark.parametrize("channels,groups", [(40, 1), (3000, 1), (3000, 3)])
def test_rows_that_are_not_finite(channels, groups):
    s = lib()
    x, z, w = (draw(k, (9, channels), torch.bfloat16) for k in (1, 2, 3))
    w = w[0].float()
    clean = s.gated_rms_norm(x, z, w, groups=groups)
    codes0, scale0 = s.gated_rms_norm_i8(x, z, w, groups=groups)
    x[2, channels - 1] = float("nan")
    x[4, 0] = float("inf")
    x[6] = 3e38                                                              # finite, but its square is not
    out = s.gated_rms_norm(x, z, w, groups=groups)
    codes, scale = s.gated_rms_norm_i8(x, z, w, groups=groups)
    size = channels // groups
    for row in range(9):
        if row in (2, 4, 6):
            assert torch.isnan(scale[row]) and not codes[row].any()
            bad = slice(channels - size, channels) if row == 2 else slice(0, size) if row == 4 else slice(0, channels)
            assert torch.isnan(out[row, bad]).all()
            if row != 6 and groups > 1:
                good = slice(0, channels - size) if row == 2 else slice(size, channels)
                assert torch.equal(out[row, good], clean[row, good])
        else:
            assert torch.equal(out[row], clean[row]) and torch.equal(codes[row], codes0[row]) and scale[row] == scale0[row]


def test_zero_rows_and_no_rows():
    s = lib()
    w = torch.ones(96, device=DEV)
    x = torch.zeros(3, 96, device=DEV, dtype=torch.float16)
    out, _ = s.rms_norm(x, w)
    codes, scale, _ = s.rms_norm_i8(x, w)
    assert not out.any() and not codes.any() and not scale.any()
    out, _ = s.rms_norm(x[:0], w)
    assert out.shape == (0, 96)
    assert s.quantize_rows(x[:0])[1].shape == (0,)
    assert s.dequantize_rows(codes[:0], scale[:0], torch.float32).shape == (0, 96)


def test_residual_in_place_and_given_buffers():
    s = lib()
    x, w, res = draw(1, (77, 1000), torch.float16), draw(2, (1000,), torch.float32), draw(3, (77, 1000), torch.float32)
    want, v = s.rms_norm(x, w, res)
    out = torch.empty_like(x)
    got, same = s.rms_norm(x, w, res, out=out, residual_out=res)
    assert got is out and same is res and torch.equal(out, want) and torch.equal(res, v)


def test_more_rows_than_the_grid_and_other_shapes():
    s = lib()
    x, w = draw(4, (5, 8000, 72), torch.bfloat16), draw(5, (72,), torch.float32)
    n, _, bound = ref.norm(host(x).reshape(-1, 72), host(w))
    out, _ = s.rms_norm(x, w)
    close(out, n, bound, torch.bfloat16, "three axes")
    codes, scale, _ = s.rms_norm_i8(x, w)
    assert codes.shape == x.shape and scale.shape == (5, 8000)
    check_codes(codes.view(-1, 72), scale.view(-1), n, bound)


def test_rows_past_32_bit_offsets():
    s = lib()
    rows, channels = 140000, 16384                                           # 2.3e9 elements
    x = torch.zeros(rows, channels, device=DEV, dtype=torch.float16)
    tail = draw(9, (40, channels), torch.float16)
    x[-40:] = tail
    codes, scale = s.quantize_rows(x)
    small = s.quantize_rows(tail)
    assert torch.equal(codes[-40:], small[0]) and torch.equal(scale[-40:], small[1])
    assert not codes[:1000].any() and not scale[:-40].any()
    s.dequantize_rows(codes, scale, torch.float16, out=x)
    assert torch.equal(x[-40:], s.dequantize_rows(*small, torch.float16))
