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
