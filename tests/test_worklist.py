"""The entries of the paged attention's work list, from offsets that may be
anything: csrc/worklist.cuh built for the CPU, with every array checked for
reads outside it."""
import os
import shutil
import subprocess

import pytest

import skvtest as T

CSRC = os.path.join(str(T.ROOT), "sparse_kv_long_gb300", "csrc")

# What the header takes from the CUDA headers and from common.cuh.
STAND_IN = r"""
#pragma once
#include <algorithm>
#include <climits>
#include <cstdint>
#define __device__
#define __forceinline__ inline
#define __noinline__
#define SKV_DEV_RANGE 2
struct __half;
struct int4;
struct float2;
using std::max;
using std::min;
inline void set_status(int32_t* st, unsigned bits) { *st |= static_cast<int32_t>(bits); }
"""

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include <memory>
#include <vector>
#include "worklist.cuh"
using namespace skv;

static std::unique_ptr<int32_t[]> exact(const std::vector<int32_t>& x) {  // no byte more than the call names
  std::unique_ptr<int32_t[]> p(new int32_t[x.size()]);
  std::copy(x.begin(), x.end(), p.get());
  return p;
}

static bool ascending(const std::vector<int32_t>& x, int most) {
  for (size_t i = 0; i < x.size(); i++)
    if (x[i] < 0 || x[i] > most || (i && x[i] < x[i - 1])) return false;
  return true;
}

// Every entry as the kernel asks for it: once, and where something was out of order again.
template <bool PRE>
static void go(const std::vector<int32_t>& groups, const std::vector<int32_t>& starts, int B, int n_tok, int tpt,
               const std::vector<int32_t>& prefix, const std::vector<int32_t>& lens) {
  auto g = exact(groups), q = exact(starts), p = exact(prefix), l = exact(lens);
  PagedArgs a{};
  int32_t status = 0;
  a.B = B, a.n_tok = n_tok, a.Hkv = 2, a.G = 4, a.tpc = tpt, a.tpt = tpt, a.page = 16, a.n_pages = 100;
  a.q_start = starts.empty() ? nullptr : q.get();
  a.lengths = l.get(), a.status = &status;
  if (PRE) {
    a.n_groups = static_cast<int>(prefix.size()), a.group_start = g.get(), a.prefix_lengths = p.get();
    a.n_prefix_pages = 300;
  }
  int disorder = 0;
  const int n = B + a.n_groups;
  for (int i = 0; i < n + 3; i++) request_of<64, PRE>(a, i, true, &disorder, false);
  const bool good = (!PRE || prefix.empty() || ascending(groups, B)) && (starts.empty() || ascending(starts, n_tok));
  if ((disorder == 0) != good || ((status & SKV_DEV_RANGE) == 0 && !good)) {
    std::printf("disorder %d, status %d, good %d\n", disorder, status, good);
    std::exit(1);
  }
  int64_t tokens = 0;
  for (int i = 0; i < n + 3; i++) {
    const auto r = request_of<64, PRE>(a, i, false, &disorder, true);
    if (r.nq < 0 || (r.nq > 0 && (r.start < 0 || r.start + r.nq > n_tok))) std::exit(2);
    if (i >= a.n_groups) tokens += r.nq;
  }
  if (PRE && !good && tokens != 0) std::exit(3);  // nothing is written
  if (tokens > n_tok) std::exit(4);               // requests are disjoint
}

int main() {
  const int lo = -(1 << 30), hi = 1 << 30;
  const std::vector<std::vector<int32_t>> groups = {
      {0, 1, 3}, {0, 0, 3}, {1, 1, 2}, {0, -1, 3}, {-1, 1, 3}, {lo, 1, 3}, {0, lo, 3}, {INT_MIN, INT_MIN, 3}, {-1, 3, 3},
      {-2, -1, 3}, {0, 1, 4}, {0, 1, hi}, {0, hi, 3}, {hi, 1, 3}, {3, 2, 0}, {2, 1, 3}, {0, 3, 2}, {INT_MAX, INT_MIN, INT_MAX}};
  const std::vector<std::vector<int32_t>> starts = {{},           {0, 40, 80, 120}, {5, 5, 6, 100}, {0, 80, 40, 120}, {-1, 40, 80, 120},
                                                    {0, 40, 80, hi}, {lo, 40, 80, 120}, {0, -9, 80, 120}, {0, 40, 40, lo}};
  for (auto& g : groups)
    for (auto& s : starts)
      for (int tpt : {1, 32, 64}) {
        const int n_tok = s.empty() ? 3 : 120;
        go<true>(g, s, 3, n_tok, tpt, {100, 700}, {64, 700, 64});
        go<false>(g, s, 3, n_tok, tpt, {}, {64, 700, 64});
      }
  std::srand(1);
  for (int i = 0; i < 20000; i++) {  // mostly ascending, now and then a wild one
    const int B = 1 + std::rand() % 40, m = std::rand() % 6, n_tok = B + std::rand() % 200;
    auto offsets = [&](int n, int most) {
      std::vector<int32_t> x(n + 1);
      for (auto& y : x) y = std::rand() % (most + 1);
      std::sort(x.begin(), x.end());
      if (std::rand() % 2) x[std::rand() % (n + 1)] = (std::rand() % 3 ? 1 : 1 << 20) * (std::rand() % 400 - 200);
      return x;
    };
    auto lengths = [&](int n) {
      std::vector<int32_t> x(n);
      for (auto& y : x) y = std::rand() % 10 ? std::rand() % 3000 : std::rand() - RAND_MAX / 2;
      return x;
    };
    go<true>(offsets(m, B), offsets(B, n_tok), B, n_tok, 1 + std::rand() % 64, lengths(m), lengths(B));
    go<false>({}, offsets(B, n_tok), B, n_tok, 1 + std::rand() % 64, {}, lengths(B));
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    """The program, built with the header beside a stand-in for what it includes."""
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("needs a C++ compiler")
    at = tmp_path_factory.mktemp("worklist")
    shutil.copy(os.path.join(CSRC, "worklist.cuh"), at)
    (at / "common.cuh").write_text(STAND_IN)
    (at / "main.cpp").write_text(MAIN)
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-w", "-fsanitize=address", str(at / "main.cpp"), "-o", str(at / "check")]
    subprocess.run(cmd, check=True, capture_output=True)
    return str(at / "check")


def test_offsets_of_any_value_are_read_within_their_arrays(check):
    env = {**os.environ, "ASAN_OPTIONS": "detect_leaks=0"}  # looking for leaks takes rights that a container may not have
    r = subprocess.run([check], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[:3000]
