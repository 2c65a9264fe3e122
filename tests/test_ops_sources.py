"""What holds for the operators' sources as text (no GPU needed)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "weight_only_quantized_qmoe_gb300", "csrc")
OPERATORS = ["qmoe_ops.cuh", "qmoe_sort.cu", "qmoe_mx4.cu", "qmoe_mx4_gemm.cu", "qmoe_norm.cuh", "qmoe_norm.cu",
             "qmoe_norm_grad.cu"]


def code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", OPERATORS)
def test_tensors_are_read_by_coherent_loads(name):
    # an operator's kernel starts while the one before it may still write the
    # tensors it reads; non-coherent loads need memory nobody writes meanwhile
    # and may be moved ahead of the wait
    found = re.findall(r"__ldg\w*|ld\.global\.nc|ld\.global[\w.:]*\.nc|ld_nc_\w+|ldu\.|__restrict__", code(name))
    assert not found, found


@pytest.mark.parametrize("name", [n for n in OPERATORS if n.endswith(".cu")])
def test_every_kernel_waits_for_the_one_before(name):
    text = code(name)
    kernels = re.findall(r"__global__\s+void[\s\S]*?\n}\n", text)
    assert kernels
    for k in kernels:
        assert k.count("op_begin();") == 1, k.split("(", 1)[0]
