"""The barrier protocol of the few-token kernels as random interleavings on the
CPU (few_model.py), with the pipeline constants of each kernel as compiled."""
import os
import random
import subprocess

import pytest

import few_model

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ["gate_up_16", "gate_up_64", "down_16", "down_64", "linear_16_bf16", "linear_16", "linear_64"]
# two MMA warps, eight promotion warps in two groups, rows of codes by TMA
WIDE = dict(stages=5, slots=16, buffers=2, epi_warps=8, groups=2, token_warps=4, mma_warps=2, red_tokens=4, max_s=4, copies=1,
            ring=0)


@pytest.fixture(scope="module")
def configs(tmp_path_factory):
    exe = tmp_path_factory.mktemp("few") / "few_config"
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O0", "-std=c++17",
                    "-I", os.path.join(ROOT, "fine_grained_fp8_token_b200", "csrc"),
                    "-o", str(exe), os.path.join(ROOT, "tests", "host", "few_config.cu")], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    lines = [line.split() for line in out.splitlines()]
    return {name: {k: int(v) for k, v in (f.split("=") for f in rest)} for name, *rest in lines}


def segments(rng, n):
    return [rng.choice([1, 1, 2, 3, 4, 7]) for _ in range(n)]


@pytest.mark.parametrize("name", NAMES)
def test_one_rank(configs, name):
    """Segments of any length, one after the other."""
    for seed in range(250):
        rng = random.Random(seed)
        assert few_model.run(configs[name], [segments(rng, 16)], seed=seed) == 0


@pytest.mark.parametrize("name", NAMES)
def test_ranks_meet(configs, name):
    """Clusters whose ranks have different work and meet at its end, ranks
    without any work among them."""
    for seed in range(60):
        rng = random.Random(seed)
        S = rng.choice([2, 4, configs[name]["max_s"]])
        work = [segments(rng, rng.choice([0, 1, 3])) for _ in range(S)]
        assert few_model.run(configs[name], work, S=S, meetings=rng.choice([1, 2, 5]), seed=seed) == 0


@pytest.mark.parametrize("name", NAMES)
def test_a_withheld_tile_unwinds(configs, name):
    """One weight tile never comes: every role of every rank ends."""
    for seed in range(80):
        rng = random.Random(seed)
        S = rng.choice([1, 2, 4])
        work = [segments(rng, 6) for _ in range(S)]
        at = rng.randrange(sum(work[0]))
        assert few_model.run(configs[name], work, S=S, meetings=2, withhold=at, seed=seed, patience=400) > 0


def caught(c, runs, **kw):
    n = 0
    for seed in range(runs):
        rng = random.Random(seed)
        work = [segments(rng, 6) for _ in range(kw.get("S", 1))]
        try:
            few_model.run(c, work, seed=seed, **kw)
        except AssertionError:
            n += 1
    return n


def test_the_model_sees_a_second_wait_for_the_cluster(configs):
    """A meeting that is counted only when it succeeds: after the first one
    expires the role waits again for a phase it has waited for."""
    kw = dict(S=2, meetings=1, withhold=1, patience=400)
    for name in ("gate_up_16", "linear_16", "down_16"):
        assert caught(configs[name], 20, count_first=False, **kw) == 20
        assert caught(configs[name], 20, **kw) == 0


def test_the_model_sees_broken_pipelines():
    """Forms whose parity waits are not sound: two MMA warps over three stages,
    a ring of scales that is too short."""
    assert caught(dict(WIDE, stages=3), 40) > 0
    assert caught(dict(WIDE, mma_warps=1, stages=8, slots=9), 40) > 0
    assert caught(WIDE, 200) == 0


def test_the_model_sees_copies_that_nobody_waited_for():
    """Two MMA warps: behind a withheld tile the other warp's blocks go on, and
    with them the token rows' copies, past the last tile that the TMA warp
    waits for.  The token warps wait for their own."""
    for c in (WIDE, dict(WIDE, stages=8)):
        assert caught(c, 40, withhold=4, patience=400, wait_copies=False) > 0
        assert caught(c, 40, withhold=4, patience=400) == 0
