"""The cache kernels' range rules (csrc/kvslot.h), compiled for the host and run
over small cases: whatever the offsets, lengths, table and pages hold, what the
rules let through lies inside the arrays, and what they refuse does not."""
import ctypes
import itertools
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_quantized_rtn_b200", "csrc")
SRC = """
#include "kvslot.h"
extern "C" int seq(long long r0, long long r1, long long kv, long long mq, long long t) { return wlq::kv_sequence(r0, r1, kv, mq, t); }
extern "C" int entry(long long pos, long long w, int sh, long long* e, int* p) {
    int64_t x; int r = wlq::kv_entry(pos, w, sh, &x, p); *e = x; return r; }
extern "C" int covered(long long kv, long long w, int sh) { return wlq::kv_covered(kv, w, sh); }
extern "C" int page_ok(long long p, long long n) { return wlq::kv_page_ok(p, n); }
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("kvslot")
    (d / "r.cpp").write_text(SRC)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "r.so"), str(d / "r.cpp")])
    L = ctypes.CDLL(str(d / "r.so"))
    i64 = ctypes.c_longlong
    L.seq.argtypes = [i64] * 5
    L.entry.argtypes = [i64, i64, ctypes.c_int, ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_int)]
    L.page_ok.argtypes = [i64, i64]
    L.covered.argtypes = [i64, i64, ctypes.c_int]
    return L


def test_sequences(rules):
    vals = (-(1 << 31), -1, 0, 1, 2, 3, 5, (1 << 31) - 1)
    for r0, r1, kv in itertools.product(vals, vals, vals):
        for mq, t in ((0, 0), (2, 3), (5, 5), ((1 << 31) - 1, (1 << 31) - 1)):
            r = rules.seq(r0, r1, kv, mq, t)
            good = 0 <= r0 <= r1 <= t and r1 - r0 <= mq and kv >= r1 - r0
            assert r == (2 if not good else (0 if r1 > r0 else 1)), (r0, r1, kv, mq, t)


def test_entries(rules):
    e, p = ctypes.c_longlong(), ctypes.c_int()
    for shift in (4, 5, 8):
        size = 1 << shift
        for pos in (-(1 << 31), -size, -1, 0, 1, size - 1, size, 3 * size - 1, 3 * size, (1 << 31) - 1):
            for width in (0, 1, 3):
                r = rules.entry(pos, width, shift, ctypes.byref(e), ctypes.byref(p))
                assert (r == 0) == (0 <= pos < width * size)
                if r == 0:
                    assert e.value * size + p.value == pos and 0 <= p.value < size and 0 <= e.value < width


def test_pages(rules):
    for page in (-(1 << 31), -1, 0, 1, 4, 5, (1 << 31) - 1):
        for n in (0, 1, 5):
            assert bool(rules.page_ok(page, n)) == (0 <= page < n)


def test_covered_tokens(rules):
    for kv in (-1, 0, 1, 16, 47, 48, 49, (1 << 31) - 1):
        for width in (0, 1, 3, 1 << 24, 1 << 40):
            for shift in (4, 8):
                want = max(0, min(kv, width << shift))
                assert rules.covered(kv, width, shift) == want
