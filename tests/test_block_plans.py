"""Which kernel a size takes: the queries of the 8-bit product, the selective scan and its single-token form.  Without a GPU
the library plans for 256 compute units, as an MI355X has them."""
import pytest

ssdq = pytest.importorskip("quantized_selective_state_amd")


@pytest.mark.parametrize("m,k,n", [(0, 64, 64), (-1, 64, 64), (4, 0, 64), (4, 64, 0), (4, 131072, 64), (2 ** 31, 64, 64),
                                   (2 ** 20, 64, 2 ** 20), (2 ** 63, 64, 64), (4, 2 ** 31, 64), (4, 64, 2 ** 31)])
def test_no_plan_of_a_product(m, k, n):
    assert ssdq.matmul_i8_plan(m, k, n) is None


def test_no_plan_of_a_scan():
    plan = ssdq.selective_scan_plan
    assert plan(3, 8, 64, 16) == -1 and plan(0, 8, 64, 16) == -1 and plan(1, 8, 0, 16) == -1 and plan(1, 8, 64, 65) == -1
    assert plan(1, 2 ** 31, 64, 16) == -1 and plan(-1, 8, 64, 16) == -1 and plan(2 ** 23, 2 ** 23, 64, 16) == -1
    step = ssdq.selective_step_plan
    assert step(0, 64, 16) == -1 and step(1, 0, 16) == -1 and step(1, 64, 65) == -1 and step(2 ** 24, 1, 16) == -1
    assert step(2 ** 31, 64, 16) == -1


def test_every_kernel_of_the_product_has_its_sizes():
    """Few tokens, tiles by their number, two halves where there are no more tiles than compute units; the same for odd
    inner sizes."""
    seen = {}
    for m in (1, 8, 9, 16, 17, 32, 33, 256, 1024, 1100, 2048, 8192):
        for k in (1040, 333):
            for n in (256, 1100, 4096, 8192, 18560):
                seen.setdefault(ssdq.matmul_i8_plan(m, k, n), []).append((m, k, n))
    assert set(seen) == set(ssdq.MATMUL_I8_PLANS)
    assert (1, 1040, 18560) in seen["stream 16"] and (32, 1040, 8192) in seen["stream 32"]
    assert (8192, 1040, 8192) in seen["tiles 256x256"] and (256, 1040, 4096) in seen["tiles 64x64 halves"]


def test_a_scan_goes_whole_or_in_chunks():
    plan = ssdq.selective_scan_plan
    assert plan(16, 16 * 2048, 8192, 16) == 0                    # sequences and channels give waves enough
    assert plan(1, 16384, 5120, 16) == 216                       # a long one does not
    assert plan(37, 9001, 1531, 13, True) == 72                  # the host does not know packed lengths
    for sequences, tokens, channels, n, packed in ((1, 5000, 4096, 8, False), (3, 2001, 100, 33, True), (1, 1, 1, 1, True)):
        chunk = plan(sequences, tokens, channels, n, packed)
        assert 16 <= chunk <= 256 and chunk % 4 == 0
        number = -(-tokens // chunk)
        bytes_of = lambda k: -(-k // 256) * 256
        carried = number if number > 1 else 0                    # a chunk's states, sums and whether it ends a sequence
        need = bytes_of(carried * n * channels * 4) + bytes_of(carried * channels * 4) + bytes_of(carried * 4)
        assert ssdq.selective_scan_workspace_size(sequences, tokens, channels, n, packed) == max(256, need)


def test_a_step_takes_four_sequences_once_there_are_many():
    step = ssdq.selective_step_plan
    assert step(64, 4096, 16) == 4 and step(1, 4096, 16) == 1 and step(3, 2 ** 18, 64) == 1 and step(70, 129, 16) == 1
