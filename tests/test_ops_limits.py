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


# --- addresses ---------------------------------------------------------------------
# (function, its arguments with every address aligned, {position of an address:
# bytes it has to be a multiple of}); f32 needs 4, 16-bit types 2, int32 and
# fp32 vectors 4
F32, BF16 = b.QMOE_F32, b.QMOE_BF16
WORK = 1 << 20
ADDRESSES = [
    ("qmoe_expert_sort", [P, 4, 2, 8, 2, 4, P, P, P, None], {0: 4, 6: 4, 7: 4, 8: 4}),
    ("qmoe_expert_sort", [P, 8, 2, 8, 2, 4, P, P, P, None], {0: 8, 6: 4, 7: 4, 8: 4}),
    ("qmoe_dispatch", [P, 16, P, P, 8, 2, 4, 16, F32, P, None], {0: 4, 2: 4, 3: 4, 9: 4}),
    ("qmoe_dispatch", [P, 16, P, P, 8, 2, 4, 16, BF16, P, None], {0: 2, 2: 4, 3: 4, 9: 2}),
    ("qmoe_dispatch_grad", [P, 16, P, 8, 2, 16, F32, P, None], {0: 4, 2: 4, 7: 4}),
    ("qmoe_combine", [P, 16, P, P, 8, 2, 16, BF16, P, None], {0: 2, 2: 4, 3: 4, 8: 2}),
    ("qmoe_combine_grad", [P, 16, P, 16, P, P, P, 8, 2, 4, 16, BF16, P, P, None],
     {0: 2, 2: 2, 4: 4, 5: 4, 6: 4, 12: 2, 13: 4}),
    ("qmoe_mx4_quantize", [P, 64, 8, 64, F32, b.QMOE_ACT_NONE, P, P, 2, 4, 16, P, P, None], {0: 4, 6: 4, 7: 4, 11: 16, 12: 4}),
    ("qmoe_mx4_quantize", [P, 64, 8, 64, BF16, b.QMOE_ACT_NONE, 0, 0, 1, 1, 8, P, P, None], {0: 2, 11: 16, 12: 4}),
    ("qmoe_mx4_dequantize", [P, P, 8, 64, 8, F32, P, 64, None], {0: 4, 6: 4}),
    ("qmoe_mx4_dequantize", [P, P, 8, 64, 8, BF16, P, 64, None], {0: 4, 6: 2}),
    ("qmoe_mx4_matmul", [P, P, 8, P, P, P, 2, 16, 64, F32, P, 16, None], {0: 16, 1: 4, 3: 16, 4: 4, 5: 4, 10: 4}),
    ("qmoe_mx4_matmul", [P, P, 8, P, P, P, 2, 16, 64, BF16, P, 16, None], {0: 16, 1: 4, 3: 16, 4: 4, 5: 4, 10: 2}),
    ("qmoe_block_norm", [P, 16, P, 16, P, b.QMOE_GATE_CHANNEL, 0, P, P, 1.0, 1e-6, 8, 16, F32, P, P, P, P, None],
     {0: 4, 2: 4, 4: 4, 7: 4, 8: 4, 14: 4, 15: 4, 16: 4, 17: 4}),
    ("qmoe_block_norm", [P, 16, P, 16, P, b.QMOE_GATE_FULL, 16, P, P, 1.0, 1e-6, 8, 16, BF16, P, P, P, P, None],
     {0: 2, 2: 2, 4: 2, 7: 2, 8: 2, 14: 2, 15: 2, 16: 4, 17: 4}),
    ("qmoe_block_norm_grad", [P, 16, P, 16, P, 16, P, 16, P, b.QMOE_GATE_TOKEN, 0, P, P, P, P, 1.0, 8, 16, F32, P, P, P, P, P,
                              P, WORK, None],
     {0: 4, 2: 4, 4: 4, 6: 4, 8: 4, 11: 4, 12: 4, 13: 4, 14: 4, 19: 4, 20: 4, 21: 4, 22: 4, 23: 4, 24: 4}),
    ("qmoe_block_norm_grad", [P, 16, P, 16, P, 16, P, 16, P, b.QMOE_GATE_TOKEN, 0, P, P, P, P, 1.0, 8, 16, BF16, P, P, P, P, P,
                              P, WORK, None],
     {0: 2, 2: 2, 4: 2, 6: 2, 8: 2, 11: 2, 12: 2, 13: 4, 14: 4, 19: 2, 20: 2, 21: 2, 22: 2, 23: 2, 24: 4}),
]
MISPLACED = [(i, at) for i, (_, _, places) in enumerate(ADDRESSES) for at in places]


@pytest.mark.parametrize("i,at", MISPLACED)
def test_an_address_off_its_elements_is_refused(i, at):
    # a GPU cannot read an element that does not start on a multiple of its size
    name, args, places = ADDRESSES[i]
    args = list(args)
    for off in {1, places[at] // 2}:
        args[at] = P + off
        refused(getattr(b, name)(*args), "aligned")
