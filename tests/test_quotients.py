"""The quotients that decide 8-bit and 4-bit codes: the kernels form x / s as q + (x - q s) y from one rounded reciprocal
y = 1 / s (Markstein's correction), whose theorem excepts divisors with a significand of ones alone.  Compared on the CPU with the
machine's own division, for dividends at and up to four fp32 steps from every border between two codes.  Only significands matter
(the kernels divide otherwise where a step could leave the normal range): a divisor in [1, 2), and borders as odd multiples of 1/16 or
1/8 up to 2, which stand for those of E4M3 and E2M1 in every octave."""
import ctypes
import os
import subprocess

import pytest

SOURCE = r"""
#include <math.h>
#include <stdint.h>
#include <string.h>
static float of_bits(uint32_t b) { float f; memcpy(&f, &b, 4); return f; }
static uint32_t bits_of(float f) { uint32_t b; memcpy(&b, &f, 4); return b; }
/* divisors 1 + d 2^-23 for d = from, from + step, ... below 2^23; returns the quotients that differ */
long wrong(long from, long step, const double* borders, int n, long* seen) {
  long bad = 0;
  for (long d = from; d < 1l << 23; d += step) {
    const float s = of_bits(0x3F800000u + (uint32_t)d), y = 1.0f / s;
    for (int i = 0; i < n; ++i) {
      const uint32_t at = bits_of((float)(borders[i] * (double)s));
      for (int k = -4; k <= 4; ++k) {
        const float x = of_bits(at + (uint32_t)k), q = x * y, r = fmaf(-q, s, x);
        bad += fmaf(r, y, q) != x / s;
        ++*seen;
      }
    }
  }
  return bad;
}
"""
BORDERS = sorted({(8 + m + 0.5) / 8 for m in range(8)} | {(4 + m + 0.5) / 4 for m in range(4)} | {1.0, 1.25, 1.5, 1.75})


@pytest.fixture(scope="module")
def wrong(tmp_path_factory):
    folder = tmp_path_factory.mktemp("quotients")
    src, lib = os.path.join(folder, "quotients.c"), os.path.join(folder, "quotients.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.check_call(["gcc", "-O2", "-fPIC", "-shared", "-ffp-contract=off", src, "-o", lib, "-lm"])
    fn = ctypes.CDLL(lib).wrong
    fn.restype = ctypes.c_long
    borders = (ctypes.c_double * len(BORDERS))(*BORDERS)

    def call(first, step):
        seen = ctypes.c_long(0)
        bad = fn(ctypes.c_long(first), ctypes.c_long(step), borders, len(BORDERS), ctypes.byref(seen))
        return bad, seen.value

    return call


def test_borders_of_the_codes_are_covered():
    def significand(v):
        while v >= 2:
            v /= 2
        while v < 1:
            v *= 2
        return v

    e4m3 = [(8 + c % 8) * 2.0 ** (c // 8) if c >= 8 else 2.0 * c for c in range(127)]
    e2m1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for table in (e4m3, e2m1):
        for a, b in zip(table, table[1:]):
            assert significand((a + b) / 2) in BORDERS


def test_divisors_of_ones_alone_and_their_neighbours(wrong):
    bad, seen = wrong((1 << 23) - 1000, 1)
    assert bad == 0 and seen == 1000 * len(BORDERS) * 9


def test_every_ninth_divisor(wrong):
    """(All 2^23 take nine times as long, and agree as well.)"""
    bad, seen = wrong(0, 9)
    assert bad == 0 and seen > (1 << 23) // 9 * len(BORDERS) * 9
