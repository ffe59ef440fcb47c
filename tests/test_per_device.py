"""What the library asks the runtime once a device (csrc/per_device.h), with a stand-in for
the runtime: a failed answer is not kept, a good one is, device by device, and threads
that ask at once share one question.  Plain C++ on the CPU."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "constant_state_recurrence_gb300", "csrc")
CODE = r"""
#include "per_device.h"
#include <cstdio>
#include <thread>
#include <vector>
#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
int main() {
  enum Error { kOk = 0, kBroken = 7 };
  sanatan::PerDevice<int, 4> known;
  int asked = 0, out = -1;
  auto fails = [&](int* v) { ++asked; *v = 5; return kBroken; };
  auto works = [&](int* v) { ++asked; *v = 40 + asked; return kOk; };
  CHECK(known.get(1, &out, fails) == kBroken && asked == 1);
  CHECK(known.get(1, &out, fails) == kBroken && asked == 2);   // asked again
  CHECK(known.get(1, &out, works) == kOk && out == 43);        // and taken
  CHECK(known.get(1, &out, fails) == kOk && out == 43 && asked == 3);   // kept
  CHECK(known.get(0, &out, works) == kOk && out == 44);        // a device's own
  CHECK(known.get(9, &out, works) == kOk && known.get(9, &out, works) == kOk && asked == 6);
  sanatan::PerDevice<int, 4> shared;
  std::atomic<int> count{0}, bad{0};
  std::vector<std::thread> all;
  for (int i = 0; i < 16; ++i)
    all.emplace_back([&] {
      int v = 0;
      auto ask = [&](int* p) { *p = 3; return ++count > 2 ? kOk : kBroken; };
      while (shared.get(2, &v, ask) != kOk) {}
      if (v != 3) ++bad;
    });
  for (auto& t : all) t.join();
  CHECK(bad == 0 && count == 3);
  return 0;
}
"""


def test_failures_are_not_kept(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    (tmp_path / "t.cc").write_text(CODE)
    exe = str(tmp_path / "t")
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(tmp_path / "t.cc"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
