"""Sizes and addresses at the edge of what the operators' kernels can index are
refused at the C entry points (no GPU needed: nothing is launched)."""
import pytest

from weight_only_quantized_qmoe_gb300 import binding as b

P = 4096   # an aligned address that no call here gets to use


@pytest.fixture(scope="module", autouse=True)
def lib():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    return b.load()


def refused(status, word):
    assert status == b.QMOE_ERR_INVALID_ARG, (status, b.qmoe_op_last_error())
    assert word in b.qmoe_op_last_error()


# A tile of the product reaches up to 191 rows past the last one of either
# operand, in 31-bit coordinates.
@pytest.mark.parametrize("rows,experts,n", [(2 ** 31 - 2, 1, 64), (2 ** 31 - 256, 1, 64), (64, 2, 2 ** 30 - 1), (64, 2, 2 ** 30 - 128)])
def test_product_tiles_stay_within_31_bits(rows, experts, n):
    refused(b.qmoe_mx4_matmul(P, P, rows, P, P, P, experts, n, 32, b.QMOE_BF16, P, n, None), "31 bits")
