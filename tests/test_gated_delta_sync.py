"""The hand-overs of the gated delta rule's chain kernels. On the host, the
kernels' rules (csrc/gated_delta_sync.h) in a model of their roles and
barriers, walked through every order of events; on the GPU, the helpers
themselves in a kernel of the same roles whose loads stop for good."""

import os
import shutil
import subprocess

import pytest

from kernelized_linear_attention_kata_b200 import build as kbuild

HERE = os.path.dirname(os.path.abspath(__file__))
CHAINS = ("forward", "forward_apart", "save", "effect", "reverse")
STATUS_DEVICE_TIMEOUT = 2


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


@pytest.mark.parametrize("chain", CHAINS)
@pytest.mark.parametrize("warps, chunks", [(1, 6), (2, 4), (3, 2)])
def test_a_wait_that_gives_up_leaves_no_role_behind(model, chain, warps, chunks):
    """Whichever waits of the state warps give up, and whenever: all roles come to
    their ends, and no wait of a warp that has not given up ends early."""
    assert model(chain, warps, chunks, "kernel") == "ok"


@pytest.mark.parametrize("chain", CHAINS)
def test_passing_after_giving_up_is_caught(model, chain):
    """State warps that go on passing the hand-overs can come twice for one round;
    an issuer then waits for good."""
    assert model(chain, 2, 3, "pass") == "stuck"


def test_one_place_for_the_outputs_is_caught(model):
    assert model("forward_apart", 2, 3, "place") == "stuck"


@pytest.mark.parametrize("loads, stages, rounds", [("loads", 2, 6), ("loads", 3, 8), ("loads", 4, 9),
                                                   ("own_loads", 2, 6)])
def test_loads_start_and_end_in_order(model, loads, stages, rounds):
    """No load starts on a barrier whose last one has not landed, and none is in flight
    when the block ends, whichever waits give up."""
    assert model(loads, stages, rounds, "kernel") == "ok"


@pytest.mark.parametrize("loads", ["loads", "own_loads"])
def test_loads_after_giving_up_are_caught(model, loads):
    assert model(loads, 2, 6, "waited") == "a load started over another"
    assert model(loads, 2, 6, "leave") == "a load in flight at the end"


@pytest.fixture(scope="module")
def handover(tmp_path_factory):
    program = str(tmp_path_factory.mktemp("handover") / "handover")
    subprocess.run([kbuild.nvcc_path(), *kbuild.ARCH_FLAGS, "-std=c++17", "-O2", "--expt-relaxed-constexpr",
                    "-I", kbuild.CSRC, os.path.join(HERE, "gated_delta_handover.cu"), "-o", program], check=True)
    return program


def test_handover_program_builds(handover):
    assert os.path.exists(handover)


@pytest.mark.gpu
def test_blocks_whose_loads_stop_end_and_report_it(handover):
    done = subprocess.run([handover], check=True, capture_output=True, text=True, timeout=60).stdout.split("\n")
    blocks, ms = [[int(x) for x in line.split()] for line in done if " " in line], float(done[-2])
    assert len(blocks) == 56
    for stop, chunks, status, issued, outputs, walked in blocks:
        assert issued == outputs == walked == chunks
        assert (status & STATUS_DEVICE_TIMEOUT != 0) == (stop < chunks)
    assert 1900 <= ms <= 10000                              # one limit, then straight to the end
