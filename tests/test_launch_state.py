"""State that launches share (no GPU): calls of two threads must not race on it, since the bindings release the interpreter."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_precision_05_b200", "csrc")


def test_no_launcher_keeps_plain_statics():
    """Function-local statics that change after their initialisation are atomic or behind a mutex of their own."""
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh", ".h", ".cpp")):
            continue
        body = open(os.path.join(CSRC, name)).read()
        for m in re.finditer(r"^[ \t]+static (?!constexpr\b|const\b|__device__\b|_assert\b)([^;({\[]*)", body, re.M):
            seen += 1
            kind = m.group(1)
            guarded = "static std::mutex" in body[m.start():m.start() + 200]
            assert kind.startswith(("PerDevice", "std::mutex", "EncodeTiledFn fn =")) or guarded, f"{name}: static {kind}"
    assert seen >= 5


PROGRAM = r"""
#include <thread>
#include <vector>
#include "per_device.h"
static int lookup(int device) {
  static bsp::PerDevice known;
  int v = known.get(device);
  if (v == 0) known.set(device, v = 7 + device);
  return v;
}
int main() {
  std::vector<std::thread> t;
  int bad[8] = {};
  for (int i = 0; i < 8; ++i) t.emplace_back([&bad, i] { for (int k = 0; k < 20000; ++k) bad[i] += lookup(k % 64) != 7 + k % 64; });
  for (auto& x : t) x.join();
  int sum = 0;
  for (int b : bad) sum += b;
  return sum != 0;
}
"""


def test_per_device_values_from_many_threads(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    base = [gxx, "-O1", "-std=c++17", "-pthread", "-I", CSRC, str(src), "-o", str(exe)]
    r = subprocess.run([*base, "-fsanitize=thread"], capture_output=True, text=True)
    if r.returncode != 0 and "tsan" in r.stderr:  # a compiler without the sanitizer's library
        r = subprocess.run(base, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and "data race" not in r.stderr, r.stderr[:2000]
