"""A CTA's part of a tile (csrc/cache_share.h), compiled for the host: shares that begin more
than 2^31 units behind a tile, as in a causal prompt of a million tokens with 96 heads."""
import ctypes
import os
import random
import subprocess

import pytest

from ragged_gqa_attention_varlen_gb300 import _build


@pytest.fixture(scope="module")
def steps(tmp_path_factory):
    d = tmp_path_factory.mktemp("share")
    src, lib = d / "share.cpp", d / "share.so"
    src.write_text('#include "cache_share.h"\n'
                   'extern "C" void steps(int64_t b, int64_t e, int64_t at, int n, int* out) {\n'
                   '  const attn::kv::Steps s = attn::kv::share_steps(b, e, at, n);\n'
                   '  out[0] = s.from, out[1] = s.to;\n}\n')
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC", "-I", _build.CSRC, str(src),
                    "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).steps
    f.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.POINTER(ctypes.c_int)]

    def call(b, e, at, n):
        out = (ctypes.c_int * 2)()
        f(b, e, at, n, out)
        return range(out[0], out[1])

    return call


def test_tiles_far_before_a_share_have_no_step_in_it(steps):
    # 750000 row tiles of 1 to 7813 steps, the tile cost of 2: a head of 2.9e9 units
    begin, n = 2_900_000_000, 7813
    for at in (2, 10, 700_000_000, begin - 2 ** 31, begin - 2 ** 31 - 1, begin - n):
        assert len(steps(begin, begin + 20_000_000, at, n)) == 0
    assert steps(begin, begin + 100, begin - n + 5, n) == range(n - 5, n)


def test_every_step_belongs_to_one_share(steps):
    r = random.Random(1)
    for _ in range(300):
        big = r.choice([0, 2 ** 31 - 50, 2 ** 31 + 7, 2 ** 33 + 1])
        per, n, at = r.randint(1, 60), r.randint(0, 100), big + r.randint(0, 400)
        got = []
        for c in range(12):
            got += steps(big + c * per, big + (c + 1) * per, at, n)
        want = [s for s in range(n) if big <= at + s < big + 12 * per]
        assert got == want
        assert len(steps(0, 10, at, n)) == sum(at + s < 10 for s in range(n))
