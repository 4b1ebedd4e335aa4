"""The quotients of the cache write (one correctly rounded reciprocal, two fused
products) against IEEE division, on the host: fp32 rows come from the rotation, so that
dividend and divisor can have any 24-bit mantissa."""

import shutil
import subprocess

import pytest

SOURCE = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
static float of(uint32_t b) { float f; memcpy(&f, &b, 4); return f; }
static uint32_t bits(float f) { uint32_t b; memcpy(&b, &f, 4); return b; }
static int wrong(float v, float s, float y) {
  float q = v * y;
  return fmaf(-fmaf(s, q, -v), y, q) != v / s;
}
int main(void) {
  unsigned long bad = 0, tried = 0;
  uint32_t x = 1;
  for (uint32_t m = 0; m < (1u << 23); m += 61) {
    float s = of(0x3f800000u | m), y = 1.0f / s;
    /* quotients at and next to every tie between two e4m3 codes: t / 16 times a
       power of two (odd t between normal codes, the others between small ones) */
    for (int t = 16; t < 32; ++t)
      for (int d = -4; d <= 4; ++d, ++tried)
        bad += wrong(of(bits((float)(t / 16.0 * s)) + d), s, y);
    for (int i = 0; i < 20; ++i, ++tried) {   /* and anywhere */
      x = x * 1664525u + 1013904223u;
      bad += wrong(of(0x3f800000u | x >> 9), s, y);
    }
  }
  printf("%lu %lu\n", bad, tried);
  return 0;
}
"""


def test_quotients_round_like_division(tmp_path):
    compiler = shutil.which("gcc")
    if compiler is None:
        pytest.skip("needs a C compiler")
    source, program = tmp_path / "quotient.c", tmp_path / "quotient"
    source.write_text(SOURCE)
    subprocess.run([compiler, "-O2", "-ffp-contract=off", "-o", program, source, "-lm"],
                   check=True)
    bad, tried = map(int, subprocess.run([program], check=True, capture_output=True,
                                         text=True).stdout.split())
    assert bad == 0 and tried > 20_000_000
