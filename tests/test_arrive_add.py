"""The arrival by atomic add (csrc/pa_arrive.h, arrive_add) driven on the CPU: the header is
compiled as plain C++ with counters in host memory.  A pair of n pieces must see counts 1..n
in whatever order its arrivals' loads, swaps and adds interleave; stale tags count as zero; the
counter ends at zero, so a replay with the same tag counts from zero again; a counter that
another call keeps changing ends in -1, not in a loop."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_cache_149_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <functional>
#include "pa_arrive.h"

typedef unsigned long long u64;
struct Cas {
  u64 operator()(u64* a, u64 e, u64 d) const {
    const u64 old = *a;
    if (old == e) *a = d;
    return old;
  }
};
struct Load { u64 operator()(u64* a) const { return *a; } };
struct Add { u64 operator()(u64* a) const { return (*a)++; } };
struct Store { void operator()(u64* a, u64 v) const { *a = v; } };
// another arrival of the same pair runs whole between this one's load and its swap
struct Between {
  std::function<void()>* f;
  u64 operator()(u64* a, u64 e, u64 d) const {
    if (*f) { auto g = *f; *f = nullptr; g(); }
    return Cas()(a, e, d);
  }
};
struct Never { u64 operator()(u64* a, u64, u64) const { return *a += 1ull << 24; } };

int one(u64* c, u64 tag, int n) { return pa::arrive_add(c, tag, n, Cas(), Load(), Add(), Store()); }

int main() {
  const u64 tag = 0x123456789aull, other = 0x0fedcba987ull;
  u64 ctr = 0xdeadbeefcafef00dull;  // never written
  for (int i = 0; i < 4; ++i) printf("a %d\n", one(&ctr, tag, 4));
  printf("after %llx\n", ctr);
  for (int i = 0; i < 4; ++i) printf("r %d\n", one(&ctr, tag, 4));
  ctr = (other << 24) | 3;
  for (int i = 0; i < 2; ++i) printf("s %d\n", one(&ctr, tag, 2));
  printf("after2 %llx\n", ctr);
  ctr = (other << 24) | 1;
  printf("n %d\n", one(&ctr, tag, 1));
  printf("after3 %llx\n", ctr);
  // k arrivals come between the load of a stale tag and the swap, of n = k + 1 and k + 2
  for (int k = 1; k <= 3; ++k)
    for (int more = 1; more <= 2; ++more) {
      ctr = other << 24;
      std::function<void()> f = [&]() { for (int i = 0; i < k; ++i) printf("b%d%d %d\n", k, more, one(&ctr, tag, k + more)); };
      printf("b%d%d %d\n", k, more, pa::arrive_add(&ctr, tag, k + more, Between{&f}, Load(), Add(), Store()));
      if (more == 2) printf("b%d%d %d\n", k, more, one(&ctr, tag, k + more));
      printf("end %llx\n", ctr);
    }
  ctr = other << 24;
  printf("g %d\n", pa::arrive_add(&ctr, tag, 2, Never(), Load(), Add(), Store()));
  return 0;
}
"""


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("arrive_add")
    src, exe = d / "arrive.cpp", d / "arrive"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    return [line.split() for line in out.strip().splitlines()]


def values(lines, key):
    return [v for k, v in lines if k == key]


TAG = 0x123456789A << 24


def test_counts_run_one_to_n_and_the_last_resets(lines):
    assert values(lines, "a") == ["1", "2", "3", "4"]
    assert int(values(lines, "after")[0], 16) == TAG
    assert values(lines, "r") == ["1", "2", "3", "4"]     # a replay with the same tag


def test_another_tag_is_stale(lines):
    assert values(lines, "s") == ["1", "2"]
    assert int(values(lines, "after2")[0], 16) == TAG
    assert values(lines, "n") == ["1"]                     # a pair of one piece
    assert int(values(lines, "after3")[0], 16) == TAG


@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("more", [1, 2])
def test_arrivals_between_a_load_and_its_swap(lines, k, more):
    assert values(lines, "b%d%d" % (k, more)) == [str(i + 1) for i in range(k + more)]
    assert all(int(v, 16) == TAG for v in values(lines, "end"))


def test_gives_up_when_the_counter_keeps_changing(lines):
    assert values(lines, "g") == ["-1"]
