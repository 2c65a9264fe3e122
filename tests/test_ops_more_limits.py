"""Row counts at the edge of what the 8-bit product and the weight gradient can
index are refused at their C entry points (no GPU needed: nothing is launched).

A split weight gradient hands each of 8 ranks ceil(steps / 8) stages of 64 rows, so
that the last one's end lies up to 511 rows past the last row; with the rows below
2^31 - 512 it stays within 31 bits."""
import pytest

from test_ops_abi import P
from test_ops_limits import lib, refused  # noqa: F401
from weight_only_quantized_qmoe_gb300 import binding as b


@pytest.mark.parametrize("rows", [2 ** 31 - 512, 2 ** 31 - 300, 2 ** 31 - 258, 2 ** 31 - 257])
def test_rows(rows):
    refused(b.qmoe_weight_grad(P, 16, P, 16, None, rows, 1, 16, 16, b.QMOE_BF16, b.QMOE_F32, P, None, 0, None), "31 bits")
    refused(b.qmoe_fp8_matmul(P, P, rows, P, P, None, 1, 64, 64, 0, b.QMOE_BF16, P, 64, None), "31 bits")


@pytest.mark.parametrize("experts,n", [(1, 2 ** 31 - 512), (2, 2 ** 30 - 256), (1024, 2 ** 21)])
def test_weight_rows(experts, n):
    refused(b.qmoe_weight_grad(P, n, P, 16, P, 8, experts, n, 16, b.QMOE_BF16, b.QMOE_F32, P, P, 1 << 30, None), "31 bits")
    refused(b.qmoe_fp8_matmul(P, P, 8, P, P, P, experts, n, 64, 0, b.QMOE_BF16, P, n, None), "31 bits")
