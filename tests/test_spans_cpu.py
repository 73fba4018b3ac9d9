"""Which views share memory (spans.h, compiled by itself) against sets of their bytes, and what the entry points refuse for it
(no GPU: only calls that are refused are made)."""
import ctypes as C
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("spans") / "spans_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "audio_dit_gb300", "csrc"), os.path.join(HERE, "spans_check.cpp"), "-o", exe], check=True)

    def run(pairs):
        text = "\n".join(" ".join(str(x) for x in (*a, *b)) for a, b in pairs)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [o == "1" for o in out]
    return run


def places(s):
    p, rows, row, heads, head, width = s
    return {p + r * row + h * head + i for r in range(rows) for h in range(heads) for i in range(width)}


def test_against_sets_of_bytes(check):
    rng = random.Random(1)
    pairs = []
    for _ in range(6000):
        same = rng.random() < 0.6
        s = []
        for i in range(2):
            width = rng.choice([1, 2, 3, 8])
            strides = s[0][2::2][:2] if same and i else (rng.randint(1, 60), rng.randint(1, 60))
            s.append((rng.randint(1, 120), rng.randint(1, 6), strides[0], rng.randint(1, 6), strides[1], width))
        pairs.append(tuple(s))
    want = [bool(places(a) & places(b)) for a, b in pairs]
    assert 1500 < sum(want) < 4500
    assert check(pairs) == want


def test_long_views(check):
    P, M, H, D = 1 << 40, 1 << 24, 8, 256                             # a packed projection: rows of Q, K and V heads
    row = 3 * H * D
    q, k, v = ((P + i * H * D, M, row, H, D, D) for i in range(3))
    late = (P + M * row - 16, 1, 0, 1, 0, 64)                         # a run over the end of the last V
    far = (P, (1 << 31) - 256, 1 << 39, 4096, 1 << 39, 512)           # no memory holds it
    assert check([(q, k), (k, v), (v, q), (q, q), (q, (P + D - 2, *q[1:])), (k, (k[0] + row * 5, *k[1:])),
                  ((v[0] + 2, *v[1:]), q), (v, late), (q, late), (far, far)]) == [False] * 3 + [True] * 5 + [False] * 2
    ends = (P + M * row, 1, 0, 1, 0, 64)
    assert check([(v, ends), (ends, v), ((P, 1, 7, H, D, D), (P + H * D, 1, 9, H, D, D))]) == [False] * 3


@pytest.fixture(scope="module")
def lib():
    from audio_dit_gb300 import build
    build.build()
    import audio_dit_gb300 as A
    return A.load_library()


INVALID, MB = 1, 1 << 20


def view(ptr, row=256, head=64):
    from audio_dit_gb300 import _Heads
    return C.byref(_Heads(ptr, row, head))


def cache(pool=MB, table=2 * MB, length=3 * MB, row_off=4 * MB, kg=17 * MB, vg=18 * MB):
    # 10 pages of 64 tokens and 2 heads of 64 (92160 bytes), 3 sequences of up to 4 pages
    return C.byref((C.c_int64 * 12)(pool, 10, 64, 2, 64, table, 4, length, row_off, 3, kg, vg))


@pytest.mark.parametrize("what,at", [("pool", MB), ("pool", MB + 92160 - 16), ("table", 2 * MB + 32), ("length", 3 * MB),
                                     ("row_off", 4 * MB), ("k_gscale", 17 * MB), ("v_gscale", 18 * MB)])
def test_cache_calls_refuse_outputs_over_the_cache(lib, what, at):
    ok = view(5 * MB)
    assert lib.h3fp4_cache_read(view(at), ok, 3, cache(), None) == INVALID
    assert lib.h3fp4_cache_read(ok, view(at), 3, cache(), None) == INVALID
    if what == "pool":
        assert lib.h3fp4_cache_append(view(at), ok, 3, cache(), None) == INVALID
        assert lib.h3fp4_cache_append(ok, view(at), 3, cache(), None) == INVALID

    def attend(out=view(6 * MB), lse=7 * MB, ws=8 * MB):
        return lib.h3fp4_cache_attn(ok, 3, 4, cache(), 0.1, out, lse, 4096, ws, 1 << 40, None)
    assert attend(out=view(at)) == INVALID and attend(lse=at) == INVALID
    assert attend(ws=at) == INVALID


def test_cache_calls_refuse_outputs_over_their_rows(lib):
    # rows of 2 heads of 64: 256 elements apart; the other view between them, and one element into them
    for at in (5 * MB, 5 * MB + 16, 5 * MB + 128 + 16, 5 * MB + 512 - 16, 5 * MB + 2 * 512 + 128):
        assert lib.h3fp4_cache_read(view(5 * MB), view(at), 3, cache(), None) == INVALID, at - 5 * MB

    def attend(q=view(5 * MB), out=view(6 * MB), lse=7 * MB, ws=8 * MB):
        return lib.h3fp4_cache_attn(q, 3, 4, cache(), 0.1, out, lse, 4096, ws, 1 << 40, None)
    for kw in (dict(out=view(5 * MB + 16)), dict(out=view(5 * MB + 3 * 512 - 16)), dict(out=view(5 * MB + 16, 512)),
               dict(lse=5 * MB + 128), dict(lse=6 * MB + 3 * 512 - 4), dict(ws=7 * MB + 32), dict(ws=6 * MB + 1024),
               dict(q=view(9 * MB)), dict(out=view(9 * MB)), dict(lse=9 * MB)):
        assert attend(**kw) == INVALID, kw
