"""What the library asks each GPU once (csrc/per_device.h), with devices that are only numbers: the
choice of a product's form on one GPU must not come from another one's counts."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <cstdio>
#include <thread>
#include <vector>

#include "per_device.h"

int main() {
  gb300::PerDevice<int> known;
  int asked = 0, v = -1;
  const auto device = [&](int n, bool works) {
    return [&asked, n, works](int* out) { ++asked; *out = 10 * n + 7; return works; };
  };
  const auto get = [&](int n, int answer_of, bool works) {
    const int ok = known.get(n, &v, device(answer_of, works));
    std::printf("%d %d ", ok, v);
  };
  get(0, 0, false);   // could not: nothing is kept
  get(0, 0, true);
  get(5, 5, true);
  get(63, 63, true);
  get(0, 1, true);    // known: not asked again
  std::printf("asked %d ", asked);
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([&] { int w = 0; known.get(9, &w, device(9, true)); });
  for (std::thread& t : threads) t.join();
  std::printf("asked %d\n", asked);
}
"""


def test_each_device_is_asked_until_it_answers(tmp_path):
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(SOURCE)
    csrc = os.path.join(ROOT, "multistage_smem_pipeline_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I" + csrc, str(src), "-o", str(exe)], check=True)
    said = subprocess.run([str(exe)], check=True, text=True, capture_output=True).stdout
    assert said == "0 -1 1 7 1 57 1 637 1 7 asked 4 asked 5\n"
