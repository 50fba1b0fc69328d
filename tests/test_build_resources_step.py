"""Register and scratch budget of the kernels before and behind the LM head,
checked at build time on the CPU (as test_build_resources.py does for the
kernels of linear_logp)."""
import os
import re
import subprocess

import pytest

from selected_token_lm_amd import build as B

# kernels and their instances: types of input and output (4), with and
# without a mean (2), sums or not (2), widths
KERNELS = {"norm_fwd": 8 * 8, "norm_fwd_wide": 8, "norm_bwd": 16 * 7, "norm_bwd_wide": 8, "norm_sums_wide": 8,
           "norm_grad_sum": 1, "embed_rows": 4 * 2, "embed_rank": 2, "radix_count": 1, "radix_scan": 1,
           "radix_scatter": 1, "embed_grad": 4, "embed_grad_join": 2, "grads_square": 1, "grads_norm": 1,
           "grads_scale": 1}


@pytest.fixture(scope="module")
def resources():
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not available")
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    out = subprocess.run([B.HIPCC, *flags, "-DRLK_WAVES=4", "--cuda-device-only", "-c", "-o", os.devnull,
                          "-Rpass-analysis=kernel-resource-usage", "-I", os.path.join(B.ROOT, "include"),
                          os.path.join(B.CSRC, "rlk_step.hip")], capture_output=True, text=True, check=True).stderr
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
    """Kernel name without namespace rlk::step:: and signature."""
    m = re.match(r"_ZN3rlk4step(\d+)", mangled)
    return mangled[m.end():m.end() + int(m.group(1))]


def test_every_kernel_is_reported(resources):
    count = {}
    for k in resources:
        count[short(k)] = count.get(short(k), 0) + 1
    assert count == KERNELS


def test_no_scratch(resources):
    assert not {k: v for k, v in resources.items() if v["ScratchSize"]}


def test_waves_that_hide_the_memory(resources):
    """Two waves to a SIMD at the least; LDS that lets two blocks share a unit."""
    for k, v in resources.items():
        assert v["Occupancy"] >= 2 and v["LDS"] <= 80 << 10, (k, v)
