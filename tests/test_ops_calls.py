"""Calls of the operators that lie beside their ordinary arguments: padding that
is not used, empty and unusually shaped arguments, forward-mode derivatives."""
import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


# --- microscaled rows ----------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("K", [1, 32, 65, 160, 257, 288, 1111, 2880])
@pytest.mark.parametrize("R,N", [(3, 40), (300, 400)])
def test_padding_scales_are_not_used(ops, R, N, K):
    # what follows the last block's scale in its word of four: 255 (NaN) must
    # not meet the padding codes
    g = torch.Generator().manual_seed(R + K)
    a, w = (ops.mx4_quantize(torch.randn((n, K), generator=g).cuda()) for n in (R, N))
    nb = -(-K // 32)

    def poisoned(q):
        s = q.scales.clone()
        if nb % 4:
            s[-1, :, nb % 4:] = 255
        return ops.MX4Tensor(q.codes, s, K)

    want = ops.mx4_matmul(a, w, out_dtype=torch.float32)
    assert torch.isfinite(want).all()
    assert torch.equal(ops.mx4_matmul(poisoned(a), poisoned(w), out_dtype=torch.float32), want)
    assert torch.equal(ops.mx4_dequantize(poisoned(a)), ops.mx4_dequantize(a))
