"""Register budget of the kernels of the operators on the whole distribution,
checked at build time on the CPU (as test_build_resources.py does for the
kernels of linear_logp).

The tile kernels run eight waves per workgroup, two to a SIMD: a wave has half
of a SIMD lane's 512 registers.  The few-row kernels that keep a ring of
stages in LDS take one workgroup per compute unit and may use more.
"""
import os
import re
import subprocess

import pytest

from selected_token_lm_amd import build as B

TILES = {"logit_tiles": 2, "soft_dz_tiles": 2, "part_grad_tiles": 4}  # kernels and their instances
FEW = {"few_tiles": 12, "few_grad_h": 8, "few_grad_w": 4, "few_rows_grad": 2}
ROWS = {"gather_rows_fill": 1, "gather_rows_grad": 2, "distill_rows": 1, "bucket_entries": 2, "top_merge": 1,
        "distill_merge": 1, "distill_scatter": 1, "grad_h_sum": 1, "zero_bytes": 1}


@pytest.fixture(scope="module")
def resources():
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not available")
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    out = subprocess.run([B.HIPCC, *flags, "-DRLK_WAVES=4", "--cuda-device-only", "-c", "-o", os.devnull,
                          "-Rpass-analysis=kernel-resource-usage", "-I", os.path.join(B.ROOT, "include"),
                          os.path.join(B.CSRC, "rlk_vocab.hip")], capture_output=True, text=True, check=True).stderr
    res, at = {}, None
    for line in out.splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        if m:
            at = res.setdefault(m.group(1), {})
            continue
        m = re.search(r"(VGPRs|AGPRs|ScratchSize \[bytes/lane\]|Occupancy \[waves/SIMD\]|LDS Size \[bytes/block\]): (\d+)", line)
        if m and at is not None:
            at[m.group(1).split()[0]] = int(m.group(2))
    return res


def short(mangled):
    """Kernel name without namespace rlk::vocab:: and signature."""
    m = re.match(r"_ZN3rlk5vocab(\d+)", mangled)
    return mangled[m.end():m.end() + int(m.group(1))]


def test_every_kernel_is_reported(resources):
    count = {}
    for k in resources:
        count[short(k)] = count.get(short(k), 0) + 1
    assert count == {**TILES, **FEW, **ROWS}


def test_no_scratch(resources):
    assert not {k: v for k, v in resources.items() if v["ScratchSize"]}


def test_tile_kernels_fit_two_waves_to_a_simd(resources):
    for k, v in resources.items():
        if short(k) in TILES:
            assert v["AGPRs"] + v["VGPRs"] <= 256 and v["Occupancy"] >= 2, (k, v)
        assert v["LDS"] <= 160 << 10, (k, v)
