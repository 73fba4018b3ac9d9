"""How attention work is cut into pieces: every key tile of every unit is walked once and partial sums stay in their
slots (attn_plan.h, walked on the host as the kernels walk it)."""
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "attn_plan_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "audio_dit_gb300", "csrc"),
                    "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include",
                    os.path.join(HERE, "attn_plan_check.cpp"), "-o", exe], check=True)

    def run(problems):
        text = "\n".join(" ".join(str(x) for x in (M, T, C, Hq, Hkv, D, len(q) - 1, *q, *k))
                         for M, T, C, Hq, Hkv, D, q, k in problems)
        return subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    return run


def cut(rng, total, n):
    return [0] + sorted(rng.randint(0, total) for _ in range(n - 1)) + [total]


def one(M, T, C, Hq, Hkv, D=128):
    return (M, T, C, Hq, Hkv, D, [0, M], [0, T])


def test_named_sizes(check):
    got = check([one(30720, 512, 0, 24, 24), one(1024, 30720, 0, 24, 24), one(1, 32768, 0, 32, 8), one(1, 1, 0, 1, 1),
                 (16384, 16384, 1024, 24, 24, 128, [0, 8192, 16384], [0, 8192, 16384]),
                 one(500, 70000, 0, 24, 24), one(130, 70000, 0, 24, 8),
                 (48, 9000, 16384, 32, 8, 128, list(range(49)), [i * 9000 // 48 for i in range(49)])])
    assert [g.split()[:4] for g in got] == [
        ["ok", "0", "0", "0"], ["ok", "0", "0", "1"], ["ok", "1", "0", "1"], ["ok", "1", "0", "0"],
        ["ok", "0", "0", "1"], ["ok", "0", "0", "1"], ["ok", "0", "0", "1"], ["ok", "1", "1", "1"]], got
    # side by side where the keys of a head's units would be read once for each


def test_lanes(check):
    lanes = [int(g.split()[5]) for g in check([one(1024, 30720, 0, 24, 24), one(500, 70000, 0, 24, 24),
                                               one(1024, 1024, 0, 24, 24), one(1, 32768, 0, 32, 8)])]
    assert lanes[0] == 4 and lanes[1] == 2 and lanes[2:] == [1, 1], lanes


def test_random_problems(check):
    rng = random.Random(1)
    problems = []
    for _ in range(1500):
        n = rng.choice([1, 1, 2, 3, 7, 40, 256])
        M = int(2 ** rng.uniform(0, 15))
        T = int(2 ** rng.uniform(0, 16)) - 1
        C = rng.choice([0, 0, 1, 128, int(2 ** rng.uniform(0, 15))])
        Hkv = rng.choice([1, 2, 3, 8, 24])
        Hq = Hkv * rng.choice([1, 1, 2, 3, 5, 7, 8, 24, 130])
        problems.append((M, T, C, Hq, Hkv, rng.choice([64, 128]), cut(rng, M, n), cut(rng, T, n)))
    got = check(problems)
    assert len(got) == len(problems)
    bad = [(g, p[:6], len(p[6]) - 1) for g, p in zip(got, problems) if not g.startswith("ok")]
    assert not bad, bad[:5]
    kinds = {tuple(g.split()[1:4]) for g in got}
    # pair and solo units, with and without cuts, the separate plan
    assert {("0", "0", "0"), ("0", "0", "1"), ("1", "0", "0"), ("1", "0", "1"), ("1", "1", "1")} <= kinds, kinds


def test_more_steps_than_32_bits_are_refused(check):
    big = (1 << 31) - 256
    assert check([one(big // 24, big, 0, 24, 24)]) == ["refused"]
