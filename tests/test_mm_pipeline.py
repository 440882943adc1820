"""The order of csa_fp8_matmul's pipeline (copies, two MMA issuers, epilogue) on the host: the kernel's own
issuer walk and shapes (csrc/mm_pipeline.h), compiled by the host compiler into a model with mbarriers that tell a
phase by its parity alone, run under random orders in which every warp, copy and MMA may be late."""
import os
import shutil
import subprocess

import pytest

from compressed_sparse_attention_indexer_gb300 import build as csa_build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path_factory.mktemp("mm") / "order")
    subprocess.run([cc, "-std=c++17", "-O2", "-I", csa_build.CSRC, os.path.join(HERE, "mm_pipeline_order.cpp"), "-o", exe],
                   check=True)
    return lambda *args: subprocess.run([exe, *args], capture_output=True, text=True)


def test_every_order_gives_each_block_its_own_codes(model):
    r = model("800")
    assert r.returncode == 0 and r.stdout.count(": ok") == 5, r.stdout


def test_a_stage_waited_for_before_the_buffer_is_found(model):
    # with an odd number of stages and two issuers a stage's phase before is the other issuer's: the model sees
    # MMAs on a stage whose codes have not landed
    r = model("800", "stage-first")
    assert r.returncode > 0 and "MMAs on a stage that does not hold their block" in r.stdout, r.stdout


def test_a_ring_of_scales_that_comes_round_too_soon_is_found(model):
    # the epilogue gives a buffer back before it reads the last of the block's scales
    r = model("800", "one-slot-less")
    assert r.returncode > 0 and "scales read that are another block's" in r.stdout, r.stdout
