"""Instruction selection in libtkv.so (CPU only; our own gfx950 code), kernel by kernel:
  - every store and every atomic is a vector, LDS or scratch one, and nothing but an invalidation is done to a cache
    from a scalar unit;
  - no packed fp32 arithmetic;
  - pool, tokens and tables are reached as global memory: no access has to find out what it is an access to;
  - the products of attention are matrix instructions, and its loops over few rows load straight into LDS;
  - what does not fit the registers is a few numbers.
"""
import os
import re
import shutil
import subprocess

import pytest

pytest.importorskip("torch")

from tiled_tensor_bulk_amd import tkv as T  # noqa: E402

LLVM = "/opt/rocm/llvm/bin"
pytestmark = pytest.mark.skipif(not os.path.exists(f"{LLVM}/llvm-objdump"), reason="llvm-objdump not available")


def tool(name, *args, cwd):
    return subprocess.run([f"{LLVM}/{name}", *args], cwd=cwd, check=True, capture_output=True, text=True).stdout


@pytest.fixture(scope="module")
def objects(tmp_path_factory):
    d = tmp_path_factory.mktemp("isa")
    shutil.copy(T.LIB_PATH, d / "lib.so")
    tool("llvm-objdump", "--offloading", "lib.so", cwd=d)
    names = sorted(p for p in os.listdir(d) if p.endswith("gfx950"))
    assert names, "no gfx950 code object in the library"
    return d, names


@pytest.fixture(scope="module")
def kernels(objects):
    """{name: [(mnemonic, line)]}"""
    d, names = objects
    out = {}
    for o in names:
        for line in tool("llvm-objdump", "-d", "--mcpu=gfx950", o, cwd=d).splitlines():
            m = re.match(r"^[0-9a-f]+ <(.+)>:", line)
            if m:
                body = out.setdefault(m.group(1), [])
            elif out and (word := re.match(r"^\s+([a-z]\w+)", line)):
                body.append((word.group(1), line))
    assert len(out) >= 100
    return out


def test_stores_and_atomics_are_vector_ones(kernels):
    for name, body in kernels.items():
        for word, line in body:
            if "store" in word or "atomic" in word:
                assert word.startswith(("global_", "buffer_", "ds_", "scratch_")), (name, line)
            if word.startswith("s_") and "cache" in word:
                assert word.endswith("_inv"), (name, line)


def test_no_packed_fp32_and_no_flat_access(kernels):
    for name, body in kernels.items():
        for word, line in body:
            assert not re.fullmatch(r"v_pk_\w+_f32\w*", word), (name, line)
            assert not word.startswith("flat_"), (name, line)


def test_attention_multiplies_in_the_matrix_unit(kernels):
    seen = set()
    for name, body in kernels.items():
        family = re.search(r"(attend|rows|scores)_kernel", name)
        if family:
            seen.add(family.group(1))
            assert any(w.startswith("v_mfma_f32_16x16x32_f16") for w, _ in body), name
            straight = any(w.startswith("buffer_load_dwordx4") and re.search(r"\blds\b", line) for w, line in body)
            assert straight == (family.group(1) != "rows"), name
    assert seen == {"attend", "rows", "scores"}


def test_few_numbers_are_spilled(objects):
    d, names = objects
    seen = 0
    for o in names:
        notes = tool("llvm-readobj", "--notes", o, cwd=d)
        for size, name in zip(re.findall(r"\.private_segment_fixed_size:\s*(\d+)", notes), re.findall(r"\.symbol:\s*(\S+)", notes)):
            seen += 1
            assert int(size) <= 24, name
    assert seen >= 100
