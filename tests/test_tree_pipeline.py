"""The order of csa_tree_attn's tcgen05 kernel on the host: the kernel's own ring (csrc/tree_pipeline.h), compiled by the
host compiler into a model with mbarriers that tell a phase by its parity alone, run under random orders in which
every warp, copy and product may be late, and waits may give up: every one reads the chunk it means, every order ends, and
nothing lands behind its block's end."""
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
    exe = str(tmp_path_factory.mktemp("tree") / "order")
    subprocess.run([cc, "-std=c++20", "-O2", "-I", csa_build.CSRC, os.path.join(HERE, "tree_pipeline_order.cpp"), "-o", exe],
                   check=True)
    return lambda *args: subprocess.run([exe, *args], capture_output=True, text=True, timeout=600)


def test_every_order_gives_each_product_its_own_chunk_and_ends(model):
    r = model("4000")
    assert r.returncode == 0 and r.stdout.count(": ok") == 3, r.stdout


@pytest.mark.parametrize("mistake,found", [
    ("unseen", "a product with a V that is not its tile's"),          # a slot that gives back a phase it has not seen
    ("one-slot", "warps that wait for one another"),                  # two phases where one is meant: the same parity
    ("no-drain", "a copy or a product behind its block's end"),       # a loader that leaves before its copies have landed
    ("unlooked", "a V's rows apart that are another chunk's"),
    ("few-scales", "scales that are another tile's"),
])
def test_a_planted_mistake_is_found(model, mistake, found):
    r = model("400", mistake)
    assert r.returncode > 0 and found in r.stdout, r.stdout
