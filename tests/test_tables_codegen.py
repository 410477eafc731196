"""gfx950 code generation of the weight-table kernels, from the assembly hipcc
writes for this repository's sources (CPU only).

- No kernel selects or branches on the scalar condition code where the compare
  before it set a vector one: hipcc (clang 22) has compiled  a < b ? a : b  of
  uniform 64-bit values so, which then always took the same side.
- No atomics in the products, lookups and gradients: sums do not depend on the
  order in which workgroups run."""
import os
import re
import subprocess

import pytest

from spmv_storage_formats_amd import _build

SOURCES = ["quant.hip", "quant_run_fp32.hip", "quant_run_fp16.hip", "quant_run_bf16.hip",
           "lookup.hip"]
SCC_COMPARES = ("s_cmp", "s_bitcmp", "s_and", "s_or", "s_xor", "s_andn", "s_nor", "s_not")
SCC_WRITERS = re.compile(r"s_(add|addc|sub|subb|cmp\w*|bitcmp\w*|and|or|xor|not|nand|nor|xnor|"
                         r"andn\w*|orn\w*|lshl|lshr|ashr|bfe|abs|min|max|bcnt\w*|absdiff|addk|"
                         r"cmpk\w*|lshl\d_add)_")


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    if not os.path.exists(_build.HIPCC):
        pytest.skip("hipcc not installed")
    d = tmp_path_factory.mktemp("asm")
    out = {}
    for name in SOURCES:
        s = d / (name + ".s")
        r = subprocess.run([_build.HIPCC, *_build.CFLAGS, "--cuda-device-only", "-S",
                            os.path.join(_build.CSRC, name), "-o", str(s)],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        out[name] = s.read_text()
    return out


def misread_conditions(text):
    found, last, vector = [], None, False
    for line in text.splitlines():
        if re.match(r"(\.LBB|_Z)\S*:", line):
            last, vector = None, False
        op = line.strip().split(" ")[0].split("\t")[0]
        if op.startswith("v_cmp"):
            vector = True
        if op.startswith(("s_cselect", "s_cbranch_scc", "s_cmov")):
            if vector and last and not last.startswith(SCC_COMPARES):
                found.append(line.strip())
        if SCC_WRITERS.match(op):
            last, vector = op, False
    return found


def test_scan_finds_the_pattern():
    bad = ("\ts_addc_u32 s1, s41, s39\n\tv_cmp_lt_i64_e32 vcc, s[0:1], v[10:11]\n"
           "\ts_cselect_b32 s1, s1, s11\n")
    good = ("\ts_addc_u32 s1, s41, s39\n\tv_cmp_lt_i64_e32 vcc, s[0:1], v[10:11]\n"
            "\ts_cmp_lg_u64 vcc, 0\n\ts_cselect_b32 s1, s1, s11\n")
    assert len(misread_conditions(bad)) == 1
    assert misread_conditions(good) == []


@pytest.mark.parametrize("name", SOURCES)
def test_conditions_are_read_where_they_were_set(listings, name):
    assert misread_conditions(listings[name]) == []


@pytest.mark.parametrize("name", SOURCES[1:])
def test_no_global_atomics(listings, name):
    assert not re.search(r"\b(global|flat|buffer)_atomic_", listings[name])


@pytest.mark.parametrize("name", SOURCES[1:4])
def test_narrow_products_have_a_grid_of_tiles_alone(listings, name):
    """One pass covers the vectors of every product that k_quant_mfma serves, so its code
    reads no second index of a workgroup; k_quant_wide's reads all three."""
    found = re.findall(r"\.amdhsa_kernel (\S+)(.*?)\.end_amdhsa_kernel", listings[name], re.S)
    ids = {"k_quant_mfma": "100", "k_quant_wide": "111"}
    for kernel, want in ids.items():
        bodies = [b for k, b in found if kernel in k]
        assert bodies
        for b in bodies:
            got = [re.search(rf"workgroup_id_{d} (\d)", b).group(1) for d in "xyz"]
            assert "".join(got) == want
