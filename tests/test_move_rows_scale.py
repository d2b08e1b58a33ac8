"""The scale that the moved rows' encodings make without a division (scale_of in
csrc/move_rows.cu, built for the CPU) against the division, for every mantissa of
a row's largest value and every exponent."""
import os
import re
import shutil
import subprocess

import pytest

import skvtest as T

MAIN = r"""
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#define __device__
#define __forceinline__ inline
using __half = _Float16;
static float last;  // what was rounded to fp16
static __half __float2half_rn(float x) { last = x; return static_cast<__half>(x); }
// SCALE_OF

static float of(uint32_t u) { float f; std::memcpy(&f, &u, 4); return f; }
static uint16_t bits(__half h) { uint16_t u; std::memcpy(&u, &h, 2); return u; }

template <int TOP>
static int check() {
  for (uint32_t m = 0; m < 1u << 23; m++) {  // one binade: the fp32 quotient itself
    const float x = of(127u << 23 | m);
    scale_of<TOP>(x);
    if (last != x / TOP) return std::printf("%d: %a gives %a, not %a\n", TOP, x, last, x / TOP);
  }
  for (uint32_t e = 0; e < 255; e++)  // from zero and the smallest numbers on: its fp16 rounding
    for (uint32_t m = 0; m < 1u << 23; m += e > 90 && e < 160 ? 257 : 4099) {
      const float x = of(e << 23 | m);
      if (bits(scale_of<TOP>(x)) != bits(static_cast<__half>(x / TOP))) return std::printf("%d: fp16 of %a\n", TOP, x);
    }
  for (float x : {of(0x7f7fffffu), of(0x7f800000u), of(1u), of(0x007fffffu)})
    if (bits(scale_of<TOP>(x)) != bits(static_cast<__half>(x / TOP))) return std::printf("%d: fp16 of %a\n", TOP, x);
  return 0;
}

int main() { return check<127>() || check<7>(); }
"""


def test_scales_without_a_division_are_the_divisions(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("needs a C++ compiler")
    src = open(os.path.join(T.ROOT, "sparse_kv_long_gb300", "csrc", "move_rows.cu")).read()
    fn = re.search(r"template <int TOP>\n__device__ __forceinline__ __half scale_of\(.*?\n}\n", src, re.S)
    assert fn
    (tmp_path / "main.cpp").write_text(MAIN.replace("// SCALE_OF", fn.group(0)))
    cmd = [cxx, "-std=c++17", "-O2", "-ffp-contract=off", str(tmp_path / "main.cpp"), "-o", str(tmp_path / "check")]
    subprocess.run(cmd, check=True, capture_output=True)
    r = subprocess.run([str(tmp_path / "check")], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
