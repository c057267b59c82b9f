"""The 8-bit matrix product on the GPU: sums against exact integers, outputs within the roundings of the epilogue."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda:0"
E = 2.0 ** -24


def lib():
    import quantized_selective_state_amd as ssdq
    return ssdq


def codes(seed, *shape):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=gen, device=DEV, dtype=torch.int32).to(torch.int8)


def scales(seed, n):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.exp(torch.randn(n, generator=gen, device=DEV)) * 1e-3


def check(a, sa, b, sb, bias, dtype):
    """Outputs within: the sum's conversion, two products and the sum with the bias rounded to binary32, then to dtype.  The
    integers are exact in doubles."""
    got = lib().matmul_i8(a, sa, b, sb, bias=bias, dtype=dtype)
    assert got.dtype == dtype and got.shape == (a.shape[0], b.shape[0])
    product = a.double() @ b.double().T * sa.double().view(-1, 1) * sb.double()
    want = product if bias is None else product + bias.double()
    bound = 3 * E * product.abs() + E * want.abs()
    info = torch.finfo(dtype)
    allowed = bound + (want.abs() + bound) * info.eps / 2 + info.tiny * info.eps / 2
    off = (got.double() - want).abs()
    over = (want.abs() > info.max)                                           # beyond a type's range: infinite
    assert bool(((off <= allowed) | over).all()), float((off / allowed).max())


# each kind of tile and its remainders: single tokens, a few, many; inner sizes with and without whole 16-byte pieces
SIZES = [(1, 1, 1), (1, 16, 16), (1, 4096, 512), (1, 1531, 1000), (2, 64, 130), (3, 100, 77), (5, 2560, 4096), (8, 4097, 333),
         (15, 64, 64), (16, 128, 256), (17, 192, 250), (31, 320, 1000), (32, 8192, 96), (33, 4096, 2048), (48, 65, 129),
         (64, 1024, 1024), (65, 1008, 1030), (100, 2048, 8512), (127, 127, 127), (128, 4096, 512), (129, 129, 129),
         (200, 8192, 520), (256, 256, 256), (257, 2048, 4096), (300, 1531, 999), (512, 640, 2000), (777, 1531, 1000),
         (1000, 4096, 1000), (1024, 4096, 4096), (2048, 64, 2560), (2500, 2560, 2570), (4096, 192, 4100),
         (16, 5003, 700), (700, 8192, 130), (3000, 333, 2800), (8200, 1040, 4200), (20, 131071, 40), (6, 131056, 300)]


@pytest.mark.parametrize("m,k,n", SIZES)
def test_sizes(m, k, n):
    a, b = codes(m + k, m, k), codes(n + k, n, k)
    sa, sb = scales(m, m), scales(n, n)
    for i, dtype in enumerate(TYPES.values()):
        check(a, sa, b, sb, None if i == 1 else scales(3, n) * 100, dtype)
    check(a, sa[:1], b, sb, None, torch.float32)


@pytest.mark.parametrize("m", [1, 20, 300, 1024])
def test_largest_sums(m):
    """-128 times -128 all along the longest inner axis: 131071 * 16384 is 2^31 - 16384."""
    k, n = 131071, 256
    a, b = torch.full((m, k), -128, dtype=torch.int8, device=DEV), torch.full((n, k), -128, dtype=torch.int8, device=DEV)
    b[1] = 127
    one = torch.ones(1, device=DEV)
    got = lib().matmul_i8(a, one, b, torch.ones(n, device=DEV), dtype=torch.float32)
    assert bool((got[:, 0] == float(np.float32(131071 * 16384))).all())
    assert bool((got[:, 1] == float(np.float32(-131071 * 128 * 127))).all())


def test_every_position_counts():
    """One code of a and one of b not zero: the output is where they say, for positions all over the tiles."""
    m, k, n = 300, 1000, 700
    rng = np.random.default_rng(5)
    one = torch.ones(1, device=DEV)
    for _ in range(20):
        i, j, p = rng.integers(m), rng.integers(n), rng.integers(k)
        a, b = torch.zeros(m, k, dtype=torch.int8, device=DEV), torch.zeros(n, k, dtype=torch.int8, device=DEV)
        a[i, p], b[j, p] = 3, -5
        got = lib().matmul_i8(a, one, b, torch.ones(n, device=DEV), dtype=torch.float32)
        want = torch.zeros_like(got)
        want[i, j] = -15
        assert torch.equal(got, want), (i, j, p)


@pytest.mark.parametrize("m", [2, 40, 600, 2048])
def test_what_is_not_finite_stays_in_its_row_and_column(m):
    k, n = 512, 2048 if m == 2048 else 300
    a, b, sa, sb, bias = codes(1, m, k), codes(2, n, k), scales(3, m), scales(4, n), scales(5, n)
    clean = lib().matmul_i8(a, sa, b, sb, bias=bias, dtype=torch.float32)
    sa2, sb2, bias2 = sa.clone(), sb.clone(), bias.clone()
    sa2[1], sb2[7], bias2[9] = float("nan"), float("inf"), float("nan")
    got = lib().matmul_i8(a, sa2, b, sb2, bias=bias2, dtype=torch.float32)
    assert torch.isnan(got[1]).all() and torch.isnan(got[:, 9]).all() and not torch.isfinite(got[:, 7]).any()
    rows, cols = [r for r in range(m) if r != 1], [c for c in range(n) if c not in (7, 9)]
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])


def test_no_tokens_given_output_and_more_axes():
    s = lib()
    b, sb = codes(1, 96, 64), scales(2, 96)
    assert s.matmul_i8(codes(3, 0, 64), scales(4, 0), b, sb).shape == (0, 96)
    a, sa = codes(5, 2, 3, 64), scales(6, 6).view(2, 3)
    out = torch.empty(2, 3, 96, device=DEV, dtype=torch.bfloat16)
    assert s.matmul_i8(a, sa, b, sb, dtype=torch.bfloat16, out=out) is out
    assert torch.equal(out.view(6, 96), s.matmul_i8(a.view(6, 64), sa.view(6), b, sb, dtype=torch.bfloat16))


@pytest.mark.parametrize("m,k,n", [(1, 4096, 4096), (130, 1531, 700), (2048, 2048, 2048)])
def test_nothing_is_written_outside(m, k, n):
    """Output, operands and scales inside larger buffers: what lies around the output stays as it was."""
    a, b, sa, sb = codes(1, m, k), codes(2, n, k), scales(3, m), scales(4, n)
    want = lib().matmul_i8(a, sa, b, sb, dtype=torch.float16)
    pad = 4096
    room = torch.full((m * n + 2 * pad,), 7.0, device=DEV, dtype=torch.float16)
    out = room[pad:pad + m * n].view(m, n)
    lib().matmul_i8(a, sa, b, sb, dtype=torch.float16, out=out)
    assert torch.equal(out, want) and bool((room[:pad] == 7).all()) and bool((room[-pad:] == 7).all())


def test_outputs_past_32_bit_offsets():
    m, k, n = 70000, 64, 32768                                               # 2.3e9 outputs
    a, b, sa, sb = codes(1, m, k), codes(2, n, k), scales(3, m), scales(4, n)
    got = lib().matmul_i8(a, sa, b, sb, dtype=torch.bfloat16)
    for rows in (slice(0, 64), slice(65500, 65600), slice(m - 100, m)):
        assert torch.equal(got[rows], lib().matmul_i8(a[rows].contiguous(), sa[rows].contiguous(), b, sb, dtype=torch.bfloat16))
