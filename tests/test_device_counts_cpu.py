"""The launchers' table of what they have asked of each device (host code, no GPU)."""

import subprocess
from pathlib import Path

HEADER = Path(__file__).resolve().parents[1] / "kimi_delta_attention_04_gb300" / "csrc" / "kda_device_counts.h"

MAIN = r'''
#include "%s"
#include <cstdio>
int main() {
  kda::DeviceCounts<9> counts;
  int asked = 0;
  auto on = [&](int device, int size) {  // device d holds 100 / size - 10 d clusters, none below that
    int n = -1;
    const int e = counts.get(device, size, &n, [&](int* c) {
      ++asked;
      *c = device < 10 ? 100 / size - 10 * device : 0;
      if (*c < 0) *c = 0;
      return 0;
    });
    return e == 0 ? n : -1;
  };
  auto print = [&](int device, int size) { std::printf("%%d ", on(device, size)); };
  // each device by itself, whichever asked first, and once only
  for (int again = 0; again < 2; ++again) print(0, 2), print(1, 2), print(0, 8), print(2, 8);
  std::printf("%%d\n", asked);
  // ordinals outside the table are asked each time
  asked = 0;
  print(64, 2), print(64, 2), print(-1, 2);
  std::printf("%%d\n", asked);
  // an error is passed on and asked again
  int n = -1;
  std::printf("%%d ", counts.get(3, 2, &n, [](int*) { return 7; }));
  std::printf("%%d\n", on(3, 2));
}
'''


def test_counts_by_device(tmp_path):
    src, exe = tmp_path / "counts.cpp", tmp_path / "counts"
    src.write_text(MAIN % HEADER)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    assert lines == ["50 40 12 0 50 40 12 0 4", "0 0 60 3", "7 20"]
