"""Pieces without the tiles behind the last keys that masks keep: every kept tile is walked once (attn_plan.h, walked on the
host as the kernel's describing warp walks it)."""
import os
import random
import subprocess

import pytest

from test_attn_plan_cpu import HERE, ROOT, cut


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("trim") / "attn_trim_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "audio_dit_gb300", "csrc"),
                    "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include",
                    os.path.join(HERE, "attn_trim_check.cpp"), "-o", exe], check=True)

    def run(problems):
        text = "\n".join(" ".join(str(x) for x in (M, T, C, Hq, Hkv, D, len(q) - 1, *q, *k, ctx, *own))
                         for M, T, C, Hq, Hkv, D, q, k, ctx, own in problems)
        return subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    return run


def tiles(n):
    return (n + 127) // 128


def keep(rng, n):
    return rng.choice([0, tiles(n), rng.randint(0, tiles(n)), min(1, tiles(n))])


def test_one_segment_kept_at_every_length(check):
    for M, T, C, Hkv in ((3, 9000, 0, 2), (700, 2500, 1000, 4), (5000, 700, 300, 8)):
        problems = [(M, T, C, 8, Hkv, 128, [0, M], [0, T], c, [o])
                    for c in range(tiles(C) + 1) for o in range(0, tiles(T) + 1, 1 if C else 5)]
        got = check(problems)
        assert len(got) == len(problems) and set(got) == {"ok"}, got


def test_random_problems(check):
    rng = random.Random(11)
    problems = []
    for _ in range(1500):
        n = rng.choice([1, 1, 2, 5, 40, 256])
        M, T = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 15)) - 1
        C = rng.choice([0, 1, 128, int(2 ** rng.uniform(0, 15))])
        Hkv = rng.choice([1, 2, 8, 24])
        k = cut(rng, T, n)
        problems.append((M, T, C, Hkv * rng.choice([1, 3, 4]), Hkv, rng.choice([64, 128]), cut(rng, M, n), k,
                         keep(rng, C), [keep(rng, b - a) for a, b in zip(k, k[1:])]))
    got = check(problems)
    bad = [(g, p[:6]) for g, p in zip(got, problems) if g != "ok"]
    assert len(got) == len(problems) and not bad, bad[:5]
