"""Which row tiles a call with shared prefixes is planned with, and that each of its launches
has a kernel of that tile: the rules' header, compiled alone (no GPU needed)."""
import ctypes
import itertools
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lossless_bit_weight_encode_gb300",
                    "csrc")
SOURCE = """
#include "kv_tiles.hpp"
using namespace w12::launch;
// rows of the prefixes' and the own tokens' tiles, launches, and rows of the kernels launched
extern "C" void tiles(int tokens, int max_new, int requests, int groups, int max_requests, int group, int kv_heads,
                      int q8, int sms, int *out) {
    const SharedTiles t = shared_tiles(tokens, max_new, requests, groups, max_requests, group, kv_heads, q8, sms);
    out[0] = t.prefix, out[1] = t.own, out[2] = t.lines();
    out[3] = shared_kernel_rows(t.kind(0), q8, t.prefix);
    out[4] = t.lines() == 1 ? out[3] : shared_kernel_rows(t.kind(1), q8, t.own);
}
extern "C" int rows(int kind, int q8, int rows) {
    return shared_kernel_rows(static_cast<w12::dev::KvSpans>(kind), q8, rows);
}
"""
SMS = 152


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    at = tmp_path_factory.mktemp("tiles")
    (at / "tiles.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-I", CSRC, str(at / "tiles.cpp"), "-o",
                    str(at / "tiles.so")], check=True)
    return ctypes.CDLL(str(at / "tiles.so"))


def tiles(rules, *args):
    out = (ctypes.c_int * 5)()
    rules.tiles(*args, out)
    return list(out)


def test_every_launch_has_a_kernel_of_its_tile(rules):
    """Requests per group understated, few tokens for many requests, all cache types."""
    seen = set()
    for group, kv_heads, requests, new, q8 in itertools.product(
            (1, 2, 3, 4, 6, 8, 9, 12, 16, 17, 40), (1, 2, 4, 8, 40), (1, 9, 18, 19, 23, 24, 64, 114, 120, 300, 1000, 5000),
            (0, 1, 2, 3, 17, 300), (0, 1)):
        for groups, most, tokens in itertools.product({1, 2, min(requests, 20), requests}, {0, 1, 2, 8, requests},
                                                      {1, requests, requests * max(new, 1)}):
            a, b, lines, launched, own = tiles(rules, tokens, new, requests, groups, most, group, kv_heads, q8, SMS)
            what = (group, kv_heads, requests, new, q8, groups, most, tokens)
            assert (launched, own) == (a, b), what
            assert a >= b and lines == (1 if a == b else 2), what
            seen.add((q8, a, b))
    # all plans that there are
    assert seen == {(0, 8, 8), (0, 16, 16), (0, 128, 128), (0, 16, 8), (0, 128, 8),
                    (1, 8, 8), (1, 16, 16), (1, 128, 128), (1, 16, 8), (1, 128, 8), (1, 128, 16)}


def test_few_requests_per_group_said(rules):
    # one prompt, 128 requests of two new tokens, 48 heads over 8: one launch of the tcgen05 kernel
    assert tiles(rules, 256, 2, 128, 1, 1, 6, 8, 0, SMS) == [128, 128, 1, 128, 128]
    # one of 128 requests has a new token, 12 heads per key head
    assert tiles(rules, 1, 1, 128, 1, 128, 12, 8, 0, SMS) == [128, 128, 1, 128, 128]
    # six rows a request: two launches
    assert tiles(rules, 128, 1, 128, 1, 128, 6, 8, 0, SMS) == [128, 8, 2, 128, 8]


def test_no_kernel(rules):
    assert [rules.rows(0, q, r) for q in (0, 1) for r in (8, 16, 128, 32, 0)] == [8, 16, 128, 0, 0] * 2
    assert [rules.rows(1, q, r) for q in (0, 1) for r in (8, 16, 128)] == [0, 16, 128] * 2
    assert [rules.rows(2, q, r) for q in (0, 1) for r in (8, 16, 128)] == [8, 0, 0, 8, 16, 0]
