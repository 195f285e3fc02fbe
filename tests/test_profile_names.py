"""The per-kernel timing has a place for every kernel of the library (CPU: the
names are counted in the sources). Without one, a program that runs many forms
under the timing would miss kernels without a word."""

import glob
import os
import re

from kernelized_linear_attention_kata_b200 import build as kbuild


def names():
    """String literals with which a ProfileScope is made, there or through `name`."""
    found = set()
    for path in glob.glob(os.path.join(kbuild.CSRC, "*.cu*")):
        text = open(path).read()
        for scope in re.findall(r"ProfileScope \w+\(([^;]*)\);", text):
            found |= set(re.findall(r'"(\w+)"', scope))
        if re.search(r"ProfileScope \w+\(name,", text):
            found |= set(re.findall(r'\("(\w+)", a,', text))
    return found


def test_every_kernel_has_a_place():
    places = int(re.search(r"kMaxKernels = (\d+)", open(os.path.join(kbuild.CSRC, "profile.cu")).read())[1])
    assert {"gd_tc_forward", "gd_tc_save", "gd_step", "tc_segment_pass", "simt_delta"} <= names()
    assert len(names()) <= places
