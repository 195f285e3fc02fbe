"""The hand-overs of the gated delta rule's chain kernels, walked through every
order of events on the host: the kernels' rules (csrc/gated_delta_sync.h) in a
model of their roles and barriers, compiled here."""

import os
import shutil
import subprocess

import pytest

from kernelized_linear_attention_kata_b200 import build as kbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    program = str(tmp_path_factory.mktemp("model") / "model")
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-O1", "-Wall", f"-I{kbuild.CSRC}",
                    os.path.join(HERE, "gated_delta_sync_model.cpp"), "-o", program], check=True)

    def run(*args):
        return subprocess.run([program, *map(str, args)], check=True, capture_output=True, text=True,
                              timeout=120).stdout.strip()
    return run


@pytest.mark.parametrize("stages", [2, 3, 4])
def test_no_ready_dv_is_missed(model, stages):
    """Reverse chain: however late the storing warp looks, it sees every round of
    dV (2 to 4 stages of loads, as the head sizes leave room for)."""
    assert model("dv", stages, 3 * stages + 1, "kernel") == "ok"


@pytest.mark.parametrize("stages", [2, 3, 4])
def test_one_barrier_for_all_rounds_is_caught(model, stages):
    """With a single barrier the storing warp can miss two rounds at once and wait
    for good: the model finds it."""
    assert model("dv", stages, 3 * stages + 1, "one") != "ok"
