"""Global loads of the kernels, in the sources.  Every launch is programmatic:
a kernel begins while the one before it may still write what it reads.  So no
kernel reads through the non-coherent path (__ldg, ld.global.nc, a const
__restrict__ pointer), nor by a load intrinsic with a cache hint, which the
compiler may move over the wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lora_linear_layer_b200", "csrc")
FILES = sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh")))


def code(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        text = re.sub(r"/\*.*?\*/", " ", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", FILES)
def test_no_load_that_may_pass_the_wait(name):
    found = re.findall(r"__ldg\b|__ldc[agsv]\b|__ldlu\b|ld\.global\.nc|__restrict__", code(name))
    assert not found, (name, found)


@pytest.mark.parametrize("name,kernel", [("adapter_pass.cuh", "adapter_pass_kernel"), ("token.cuh", "token_prep_kernel")])
def test_kernels_in_front_of_an_early_reader_wait_before_they_let_it_go(name, kernel):
    """token_stream_kernel and dX's lowrank_gemm_kernel read before their own
    wait what was written before the kernel in front of them: that kernel
    calls griddep_wait directly before every griddep_launch_dependents."""
    body = code(name).split(kernel + "(", 1)[1].split("__global__", 1)[0]
    calls = re.findall(r"griddep_\w+\(\);", body)
    assert calls and calls == ["griddep_wait();", "griddep_launch_dependents();"] * (len(calls) // 2)
    assert len(re.findall(r"griddep_wait\(\);\s*griddep_launch_dependents\(\);", body)) == len(calls) // 2
