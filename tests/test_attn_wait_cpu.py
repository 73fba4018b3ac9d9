"""The limit of the attention's device waits grows with the work that a wait may span (CPU)."""
import os
import random
import subprocess

import pytest

from test_attn_plan_cpu import HERE, ROOT, cut, one


@pytest.fixture(scope="module")
def limits(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("wait") / "attn_wait_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "audio_dit_gb300", "csrc"),
                    "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include",
                    os.path.join(HERE, "attn_wait_check.cpp"), "-o", exe], check=True)

    def run(limit, problems):
        text = "\n".join(" ".join(str(x) for x in (limit, M, T, C, Hq, Hkv, D, len(q) - 1, *q, *k))
                         for M, T, C, Hq, Hkv, D, q, k in problems)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        return [tuple(int(x) for x in line.split()) for line in out]
    return run


STEP_NS = 2300  # a step of two query tiles and, with a mask, its part of the scan


def test_longest_units(limits):
    """Whole units of 1.7 million tiles: 2.7 s of work, more than the default of 2 s."""
    keys = 213_000_000
    (limit, tiles), = limits(2_000_000_000, [one(152 * 256, keys, 0, 1, 1, 8)])
    assert tiles == 4 * ((keys + 127) // 128) and limit >= 2_000_000_000 + tiles * STEP_NS


def test_limits_of_random_problems(limits):
    rng = random.Random(3)
    problems = []
    for _ in range(300):
        n = rng.choice([1, 2, 7, 100])
        M, T, C = int(2 ** rng.uniform(0, 16)), int(2 ** rng.uniform(0, 20)), rng.choice([0, int(2 ** rng.uniform(0, 18))])
        Hkv = rng.choice([1, 3, 24])
        problems.append((M, T, C, Hkv * rng.choice([1, 4]), Hkv, rng.choice([64, 128]), cut(rng, M, n), cut(rng, T, n)))
    for given in (1, 2_000_000, 2_000_000_000):
        got = limits(given, problems)
        assert len(got) == len(problems) and all(limit >= given + tiles * STEP_NS for limit, tiles in got)


def test_largest_limit_stays(limits):
    most = (1 << 64) - 1
    assert limits(most, [one(1, 1 << 20, 0, 1, 1)])[0][0] == most


def test_small_calls_keep_a_short_limit(limits):
    """The time-out self-test's one tile."""
    assert limits(2_000_000, [one(1, 1, 0, 1, 1, 64)])[0][0] == 2_020_000
