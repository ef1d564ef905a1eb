"""What the library remembers about a device it remembers for that device only
(csrc/per_device.h), checked by a small program of its own on the CPU."""

import glob
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_layer_ep_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
enum Error { kFine = 0, kBroken = 7 };
int main() {
  moe::PerDevice numbers;
  int made = 0, v = -1;
  auto of = [&](int n, Error e = kFine) { return [&made, n, e](int* out) { ++made; *out = n; return e; }; };
  // each device's own number, made once
  for (int turn = 0; turn < 3; ++turn)
    for (int device = 0; device < 4; ++device) {
      CHECK(numbers.get(device, &v, of(100 + device)) == kFine);
      CHECK(v == 100 + device);
    }
  CHECK(made == 4);
  // 0 is a number like others
  made = 0;
  CHECK(numbers.get(9, &v, of(0)) == kFine && v == 0);
  CHECK(numbers.get(9, &v, of(5)) == kFine && v == 0 && made == 1);
  // what failed is tried again
  made = 0;
  CHECK(numbers.get(10, &v, of(3, kBroken)) == kBroken);
  CHECK(numbers.get(10, &v, of(4)) == kFine && v == 4 && made == 2);
  // devices beyond the table are asked every time
  made = 0;
  for (int device : {-1, moe::PerDevice::kMaxDevices, moe::PerDevice::kMaxDevices})
    CHECK(numbers.get(device, &v, of(6)) == kFine && v == 6);
  CHECK(made == 3);
  // threads that ask at once see the number, and what was set up before it
  moe::PerDevice shared;
  static int setup[8];
  std::vector<std::thread> threads;
  std::vector<int> good(16, 0);
  for (int t = 0; t < 16; ++t)
    threads.emplace_back([&, t] {
      int ok = 1;
      for (int i = 0; i < 1000; ++i) {
        const int device = (t + i) % 8;
        int x = -1;
        shared.get(device, &x, [&](int* out) {
          __atomic_store_n(&setup[device], 1, __ATOMIC_RELAXED);
          *out = device * 3;
          return kFine;
        });
        ok &= x == device * 3 && __atomic_load_n(&setup[device], __ATOMIC_RELAXED) == 1;
      }
      good[t] = ok;
    });
  for (auto& t : threads) t.join();
  for (int g : good) CHECK(g == 1);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_numbers_belong_to_a_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_no_function_remembers_the_first_device():
    """A kernel's attributes and occupancy are not kept in a plain variable of a function."""
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        text = open(path).read()
        assert not re.search(r"^\s+static (bool|int|int32_t)\s+\w+\s*=", text, flags=re.M), path
