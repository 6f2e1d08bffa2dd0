"""The plan of the head's loss (csrc/head_plan.h, compiled for the host): the sizes of
tests/head_loss_paths.py take the paths they stand for, and every plan fits the workspace."""
import json
import os
import random
import subprocess

import pytest

from mixture_experts_transformer_moe_amd import binding as M
from mixture_experts_transformer_moe_amd.build import CSRC
from tests.head_loss_paths import PATHS


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = tmp_path_factory.mktemp("plan") / "head_plan"
    src = os.path.join(os.path.dirname(__file__), "head_plan.cpp")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, src, "-o", str(exe)], check=True)

    def run(sizes):
        text = "\n".join("%d %d %d" % s for s in sizes)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [json.loads(line) for line in out.splitlines()]
    return run


def path_of(p):
    first, last = p["pieces"][0], p["pieces"][-1]
    ends = lambda k: (first[k], last[k])  # noqa: E731
    return p["forward"], ends("probs"), ends("dw"), p["dx"], len(p["pieces"]), ends("parts")


@pytest.mark.parametrize("name", PATHS)
def test_sizes_take_their_paths(plans, name):
    size, forward, probs, dw, dx, pieces, parts = PATHS[name]
    both = lambda t: t if isinstance(t, tuple) else (t, t)  # noqa: E731
    assert path_of(plans([size])[0]) == (forward, both(probs), both(dw), dx, pieces, parts)


def test_every_path_has_a_size(plans):
    """whatever kernels and forms random sizes reach, the tests' sizes reach"""
    rng = random.Random(5)
    sizes = []
    while len(sizes) < 20000:
        s = int(2 ** rng.uniform(0, 18)), 8 * int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 23))
        if s[0] * s[2] < 2 ** 38 and s[1] <= 65536:
            sizes.append(s)
    def reached(ps):
        out = set()
        for p in ps:
            out.add(("forward", p["forward"]))
            # dx: its tile, through sums or not, in parts or not, over pieces or not
            out.add(("dx", p["dx"], p["sums"], p["parts"] > 1, len(p["pieces"]) > 1))
            for q in p["pieces"]:
                out |= {("probs", q["probs"]), ("dw", q["dw"])}
        return out
    mine = reached(plans([p[0] for p in PATHS.values()]))
    # (small batches and single parts of every tile are in the other tests of the loss)
    more = reached(plans([(1, 8, 1), (33, 128, 300), (300, 520, 777), (65, 256, 513), (129, 192, 4099), (32, 64, 4096)]))
    assert reached(plans(sizes)) <= mine | more


def test_plans_fit_their_workspace(plans):
    rng = random.Random(6)
    sizes = []
    while len(sizes) < 20000:
        s = int(2 ** rng.uniform(0, 22)), 8 * int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 23))
        if s[0] * s[2] < 2 ** 38 and s[1] <= 65536:
            sizes.append(s)
    for s, p in zip(sizes, plans(sizes)):
        assert p["bytes"] <= p["bound"] == M.moe_head_loss_workspace_bytes(*s), s
        # forward: 8 bytes a row and column tile, 4 a row
        tile = 128 if p["forward"] == "mid" else 256
        assert s[0] * (8 * -(-s[2] // tile) + 4) <= p["bound"], s
