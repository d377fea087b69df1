"""The serving calls at long inner dimensions, up to ffn 14336: rings that turn many times, an odd
number of 128s, several tiles per pair of SMs; the second 4-bit product streams its rows there
(past ffn 1024) instead of keeping them."""
import pytest

import test_few_gpu as few
import test_mx4_gpu as mx4

pytestmark = pytest.mark.gpu

name = lambda s: "-".join(map(str, s))


@pytest.mark.parametrize("shape", [
    (200, 256, 4224, 4, 2, 0),     # 33 tiles of K, one tile per pair of SMs
    (3000, 1024, 4224, 8, 2, 0),   # ... several, in rounds and shares
    (1500, 384, 4096, 5, 3, 0x1),  # K even, three column tiles
    (257, 512, 14336, 3, 1, 0),
    (300, 4224, 256, 4, 2, 0),     # a long first product
], ids=name)
def test_mx4_forward_long(shape):
    mx4.test_mx4_forward_parity(shape)


def test_mx4_forward_long_rows_do_not_depend_on_the_batch():
    mx4.test_mx4_forward_rows_do_not_depend_on_the_batch((2000, 768, 2176, 12, 3, 0))


@pytest.mark.parametrize("four_bits", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("shape", [(1, 512, 14336, 8, 2), (5, 4224, 128, 4, 2), (40, 256, 14208, 6, 2),
                                   (128, 384, 4224, 4, 2)], ids=name)
def test_few_long(shape, four_bits):
    few.test_few_parity(shape, four_bits)
