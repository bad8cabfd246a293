"""Instruction selection in the 8-bit cache's kernels (CPU only; our own gfx950 code): products of attention are matrix
instructions, of 32 rows in the kernel of many rows, and numbers become codes, and codes numbers, by conversions."""
import os
import re

import pytest

pytest.importorskip("torch")

from tests.test_tkv_isa import LLVM, kernels, objects  # noqa: E402,F401

pytestmark = pytest.mark.skipif(not os.path.exists(f"{LLVM}/llvm-objdump"), reason="llvm-objdump not available")

FAMILIES = {  # of a kernel's name: what it has to have
    "rows8_kernel": ["v_mfma_f32_32x32x16_f16", "v_cvt_scalef32_pk_f16_fp8"],
    "append8_kernel": ["v_cvt_pk_fp8_f32"],
    "append8_few_kernel": ["v_cvt_pk_fp8_f32"],
    "read8_kernel": ["v_cvt_pk_f32_fp8"],
}


def test_conversions_and_products(kernels):  # noqa: F811
    count = dict.fromkeys(FAMILIES, 0)
    for name, body in kernels.items():
        found = re.search(r"(rows8|append8|append8_few|read8)_kernel", name)
        if found:
            count[found.group(0)] += 1
            words = {word for word, _ in body}
            for need in FAMILIES[found.group(0)]:
                assert any(w.startswith(need) for w in words), (name, need)
    # four head sizes; of rows8 for both types, of append with a rotation and without
    assert count == {"rows8_kernel": 8, "append8_kernel": 8, "append8_few_kernel": 8, "read8_kernel": 4}


def test_attention_in_8_bits_converts_by_the_instruction(kernels):  # noqa: F811
    """attend_kernel of a cache without groups: D, then 0"""
    seen = 0
    for name, body in kernels.items():
        if re.search(r"attend_kernelILi\d+ELi0E", name):
            seen += 1
            assert any(word.startswith("v_cvt_scalef32_pk_f16_fp8") for word, _ in body), name
    assert seen >= 16
