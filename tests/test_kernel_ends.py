"""How the tensor-core kernels end, as their sources say it (no GPU needed: what goes
wrong without it is a race, which nothing shows on purpose)."""
import re

import pytest

from test_ops_sources import code


def kernels(name):
    """{kernel: its text}."""
    found = re.findall(r"__global__\s+void[\s\S]*?\n}\n", code(name))
    return {re.search(r"(\w+_kernel)\(", k).group(1): k for k in found}


@pytest.mark.parametrize("name,kernel", [("qmoe_fp8_gemm.cu", "fp8_matmul_pair_kernel"), ("qmoe_wgrad.cu", "weight_grad_pair_kernel")])
def test_every_commit_to_both_ctas_is_waited_for(name, kernel):
    # a commit's arrival comes on its own: none may come to a CTA that has left, in
    # the first CTA of the pair or the second
    text = kernels(name)[kernel]
    barriers = set(re.findall(r"(?:tc_commit_pair_elect\(|&)(\w*empty|acc_full|drain_bar)\b", text)) - {"acc_empty"}
    assert barriers >= {"empty", "acc_full", "drain_bar"}
    for bar in barriers:
        if bar == "drain_bar":       # the issuer, and the other CTA
            assert "mbar_wait_bounded(drain_bar, 0" in text and "pair_end(drain_bar, rank" in text
        elif bar == "acc_full":      # the epilogue of either CTA
            assert re.search(r"warp >= \d\) \{[\s\S]*wait_or_abort\(&acc_full\[ab\]", text)
        else:                        # by a role that both CTAs have, whatever its waits gave
            wait = re.search(r"\n *if \(warp == \d\) drain_ring<\w>\(%s, " % bar, text)
            assert wait, bar
            role = re.findall(r"\n  (?:} else )?if \((warp[^\n]*)\) {", text[:wait.start()])[-1]
            assert "rank" not in role, (bar, role)


WITH_TMEM = ["qmoe_prefill.cu", "qmoe_mx4_gemm.cu", "qmoe_fp8_gemm.cu", "qmoe_wgrad.cu"]


@pytest.mark.parametrize("name", WITH_TMEM)
def test_a_whole_warp_releases_tensor_memory(name):
    # the lanes of the issuing warp leave its last wait one by one, and a barrier of
    # the CTA does not bring them together again for an instruction of a whole warp
    releases = re.findall(r"([^\n]*)\n[ \t]*if \(warp == 1\) tmem_dealloc\w*\(", re.sub(r"[ \t]+\n", "\n", code(name)))
    assert releases and all(line.strip() == "__syncwarp();" for line in releases), releases


def test_no_other_kernel_has_tensor_memory():
    import os

    from test_ops_sources import CSRC
    users = [n for n in sorted(os.listdir(CSRC)) if n.endswith((".cu", ".cuh")) and re.search(r"\btmem_dealloc\w*\(tmem", code(n))]
    assert users == sorted(WITH_TMEM)


@pytest.mark.parametrize("name,kernel", [("qmoe_prefill.cu", "gemm_kernel"), ("qmoe_mx4_gemm.cu", "mx4_matmul_kernel"),
                                         ("qmoe_fp8_gemm.cu", "fp8_matmul_kernel"), ("qmoe_wgrad.cu", "weight_grad_kernel")])
def test_a_cta_waits_for_its_own_commits(name, kernel):
    # the producer for the stages', the epilogue for the accumulators', the issuer for
    # its last one
    text = kernels(name)[kernel]
    assert set(re.findall(r"tc_commit_elect\(&?(\w+)", text)) <= {"empty", "acc_full", "drain_bar"}
    producer = text[text.index("if (warp == 0) {"):text.index("else if (warp == ")]
    assert re.search(r"\n    drain_ring<\w+>\(empty, ", producer)
    assert "wait_or_abort(&acc_full[ab]" in text and "mbar_wait_bounded(drain_bar, 0" in text
