"""Host state that belongs to a device: kernel attributes and SM counts (CPU; per_device.h has no CUDA in it)."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "eagle_speculative_decoding_round_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>

#include <initializer_list>

#include "per_device.h"

#define WANT(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  static e3::OncePerDevice<int> once;
  int ran = 0;
  auto ok = [&] { ++ran; return 0; };
  auto fails = [&] { ++ran; return 7; };
  WANT(once.run(0, fails) == 7 && ran == 1);
  WANT(once.run(0, ok) == 0 && ran == 2);     // a failure is tried again
  WANT(once.run(0, fails) == 0 && ran == 2);  // a success is not
  WANT(once.run(1, ok) == 0 && ran == 3);     // another device has its own
  WANT(once.run(63, ok) == 0 && ran == 4);
  for (int i = 0; i < 2; ++i) WANT(once.run(64, ok) == 0 && once.run(-1, ok) == 0);
  WANT(ran == 8);                             // beyond the table: every time
  for (int d : {0, 1, 63}) WANT(once.run(d, fails) == 0 && ran == 8);
  static e3::NumberPerDevice number;
  int asked = 0, answer = 0;
  auto ask = [&] { ++asked; return answer; };
  WANT(number.get(0, ask) == 0 && asked == 1);
  answer = 152;
  WANT(number.get(0, ask) == 152 && asked == 2);
  answer = 148;
  WANT(number.get(0, ask) == 152 && asked == 2);
  WANT(number.get(5, ask) == 148 && asked == 3);
  WANT(number.get(99, ask) == 148 && number.get(99, ask) == 148 && asked == 5);
  return 0;
}
"""


def test_once_and_numbers_are_kept_per_device(tmp_path):
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_every_kernel_attribute_is_set_per_device():
    """Each cudaFuncSetAttribute stands in a once_per_device call, behind a check of the device, or runs on every call."""
    for f in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, f)).read()
        for m in re.finditer(r"cudaFuncSetAttribute\(", text):
            before = text[:m.start()]
            since = before[max(before.rfind("\n}\n"), 0):]  # the function so far
            every_call = f == "k_tree.cu"
            assert "once_per_device(" in since or "cached_dev != dev" in since or every_call, (f, before.count("\n") + 1)
