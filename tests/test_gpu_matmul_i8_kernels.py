"""Every kernel of the 8-bit product at sizes that reach it, against exact integers: several slabs of the inner axis, more
tiles than a device holds, remainders along every axis, the largest sums, and outputs beyond their type's range."""
import numpy as np
import pytest
import torch

from test_gpu_matmul_i8 import DEV, E, TYPES, codes, lib, scales

# each kernel: a slab of the inner axis is 128 codes; blocks on the device at once 256 (256x256), 512 (the other tiles), 768
# (odd 64x64), 512 (odd 128x128); halves have one tile each
SIZES = [
    ("stream 16", 13, 1040, 2050), ("stream 16", 8, 2064, 18565), ("stream 32", 29, 1040, 2050),
    ("tiles 256x256", 5000, 1040, 6000),        # 480 tiles, 9 slabs
    ("tiles 256x256", 8200, 272, 8200),         # 1089 tiles, 3 slabs
    ("tiles 256x256", 4081, 64, 4095),          # one tile a block, half a slab
    ("tiles 128x128", 1100, 1040, 3900), ("tiles 128x128", 8200, 656, 4201),
    ("tiles 128x64", 1500, 2064, 1500), ("tiles 128x64", 76700, 400, 63), ("tiles 128x64", 900, 656, 3901),
    ("tiles 64x64", 257, 2064, 4100), ("tiles 64x64", 61, 1040, 38401), ("tiles 64x64", 63, 144, 70401),
    ("tiles 64x64 halves", 250, 2064, 1001), ("tiles 64x64 halves", 65, 16, 130), ("tiles 64x64 halves", 257, 1168, 999),
    ("odd stream 16", 16, 2051, 3001), ("odd 128x128", 2100, 1531, 2200), ("odd 128x128", 3000, 333, 2900),
    ("odd 64x64", 1100, 333, 1100), ("odd 64x64", 1300, 1531, 1101), ("odd 64x64", 1900, 261, 1899), ("odd 64x64", 1100, 127, 1100),
    ("odd 64x64 halves", 900, 1291, 1000), ("odd 64x64 halves", 40, 33, 50)]


@pytest.mark.parametrize("plan,m,k,n", SIZES)
def test_sizes_reach_these_kernels(plan, m, k, n):
    assert lib().matmul_i8_plan(m, k, n) == plan


def test_every_kernel_has_sizes():
    assert {plan for plan, *_ in SIZES} == set(lib().MATMUL_I8_PLANS)


def agree(a, sa, b, sb, bias, dtype):
    """Within the roundings of the epilogue (the conversion, two products and the sum with the bias, then the type's own);
    beyond the type's range by more than half a step the infinity of the right sign, and nothing else."""
    got = lib().matmul_i8(a, sa, b, sb, bias=bias, dtype=dtype).double()
    product = a.double() @ b.double().T * sa.double().view(-1, 1) * sb.double()
    want = product if bias is None else product + bias.double()
    bound = 3 * E * product.abs() + E * want.abs()
    del product
    info = torch.finfo(dtype)
    allowed = bound + (want.abs() + bound) * info.eps / 2 + info.tiny * info.eps / 2
    # Rounds to infinity from half a step past the largest number on: max is (2 - eps) 2^e, half a step there eps / 2 2^e
    limit = info.max * (1 + info.eps / 2 / (2 - info.eps))
    infinite = torch.copysign(torch.full_like(want, float("inf")), want)
    good = ((got - want).abs() <= allowed) & (want.abs() - bound <= limit)
    good |= (got == infinite) & (want.abs() + bound >= limit)
    assert bool(good.all()), (int((~good).sum()), (~good).nonzero()[:4].tolist(), got[~good][:4].tolist(), want[~good][:4].tolist())
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("plan,m,k,n", SIZES)
def test_sums(plan, m, k, n):
    assert lib().matmul_i8_plan(m, k, n) == plan
    a, b = codes(m + k, m, k), codes(n + k, n, k)
    sa, sb = scales(m, m), scales(n, n)
    for i, dtype in enumerate(TYPES.values()):
        print(f"  {dtype}", flush=True)
        agree(a, sa, b, sb, None if i == 1 else scales(3, n) * 100, dtype)
    agree(a, sa[:1], b, sb, None, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("plan,m,k,n", SIZES[::2])
def test_beyond_the_types_range(plan, m, k, n):
    a, b = codes(m, m, k), codes(n, n, k)
    sa, sb = scales(m, m), scales(n, n).clamp(max=2e-2)
    spread = float(k) ** 0.5 * 128 * 128 / 3                 # of the sums
    for dtype in TYPES.values():                             # (sum * a_scale stays far inside binary32)
        got = agree(a, sa, b, (sb.double() * (1e6 * torch.finfo(dtype).max / spread)).float(), None, dtype)
        infinite = torch.isinf(got).sum().item()
        assert 0 < infinite < got.numel() and bool((got == float("inf")).any()) and bool((got == -float("inf")).any())


LARGEST = [("stream 16", 9, 131056, 200), ("stream 32", 20, 131056, 200), ("tiles 256x256", 4096, 131056, 4096),
           ("tiles 128x128", 2048, 131056, 2560), ("tiles 128x64", 1024, 131056, 4096), ("tiles 64x64", 257, 131056, 4096),
           ("tiles 64x64 halves", 70, 131056, 300), ("odd stream 16", 9, 131071, 200), ("odd 128x128", 2100, 131071, 2100),
           ("odd 64x64", 1100, 131071, 1100), ("odd 64x64 halves", 70, 131071, 300)]


@pytest.mark.gpu
@pytest.mark.parametrize("plan,m,k,n", LARGEST)
def test_largest_sums(plan, m, k, n):
    """-128 times -128, and times 127, all along the longest inner axes: the sums fill int32."""
    assert lib().matmul_i8_plan(m, k, n) == plan
    a, b = torch.full((m, k), -128, dtype=torch.int8, device=DEV), torch.full((n, k), -128, dtype=torch.int8, device=DEV)
    b[1::2] = 127
    got = lib().matmul_i8(a, torch.ones(1, device=DEV), b, torch.ones(n, device=DEV), dtype=torch.float32)
    assert bool((got[:, ::2] == float(np.float32(k * 16384))).all())
    assert bool((got[:, 1::2] == float(np.float32(-k * 128 * 127))).all())


@pytest.mark.gpu
@pytest.mark.parametrize("plan,m,k,n", SIZES)
def test_every_position_counts(plan, m, k, n):
    """One code of a and one of b not zero: the output is where they say, at first, last and other positions."""
    rng = np.random.default_rng(5)
    one, ones = torch.ones(1, device=DEV), torch.ones(n, device=DEV)
    a, b = torch.zeros(m, k, dtype=torch.int8, device=DEV), torch.zeros(n, k, dtype=torch.int8, device=DEV)
    for p in [0, k - 1, *rng.integers(0, k, 4).tolist()]:
        i, j = (m - 1, 0) if p == 0 else (0, n - 1) if p == k - 1 else (rng.integers(m), rng.integers(n))
        a[i, p], b[j, p] = 3, -5
        got = lib().matmul_i8(a, one, b, ones, dtype=torch.float32)
        assert got[i, j] == -15 and int(got.count_nonzero()) == 1, (i, j, p)
        a[i, p], b[j, p] = 0, 0
