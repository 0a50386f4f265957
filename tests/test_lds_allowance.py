"""csrc/lds_allowance.h compiled and run on the host: when a launch has to be allowed its LDS."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_quantized_int8_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


def run_cpp(tmp_path, body):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text('#include "lds_allowance.h"\n' + body)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout


def test_static_arrays_count(tmp_path):
    out = run_cpp(tmp_path, """
#include <stdio.h>
int main() {
  const unsigned sizes[][2] = {{0, 0}, {65536, 0}, {65472, 64}, {65473, 64}, {65536, 64}, {65537, 0}, {0xFFFFFFFFu, 64}};
  for (auto &s : sizes) printf("%d", int8w::needs_lds_allowance(s[0], s[1]));
}
""")
    assert out == "0001111"


def test_asked_once_on_each_device(tmp_path):
    out = run_cpp(tmp_path, """
#include <stdio.h>
int main() {
  static int8w::LdsAllowance a;
  int asked = 0;
  auto launch = [&](int device, int answer) { return a.once(device, 0, [&] { ++asked; return answer; }); };
  printf("%d ", launch(0, 0) || launch(0, 7));  // the second does not ask
  printf("%d ", asked);
  printf("%d ", launch(1, 5));                  // another device: its own request, which fails
  printf("%d ", launch(1, 0) || launch(1, 7));  // and is made again
  printf("%d ", asked);
  printf("%d ", launch(63, 0) || launch(63, 7) || launch(0, 7));
  printf("%d ", asked);
  launch(64, 0), launch(64, 0), launch(-1, 0);  // not kept
  printf("%d", asked);
}
""")
    assert out == "0 1 5 0 3 0 4 7"


def test_threads_that_launch_at_the_same_time(tmp_path):
    # none may go on before a request for its device has succeeded
    out = run_cpp(tmp_path, """
#include <stdio.h>
#include <thread>
#include <vector>
int main() {
  int early = 0, most = 0;
  for (int round = 0; round < 200; ++round) {
    int8w::LdsAllowance a;
    std::atomic<int> granted[2] = {{0}, {0}}, asked{0}, bad{0};
    std::vector<std::thread> t;
    for (int i = 0; i < 8; ++i)
      t.emplace_back([&, i] {
        a.once(i % 2, 0, [&] { ++asked; granted[i % 2] = 1; return 0; });
        if (!granted[i % 2]) ++bad;
      });
    for (auto &x : t) x.join();
    int again = 0;
    a.once(0, 0, [&] { ++again; return 0; });
    a.once(1, 0, [&] { ++again; return 0; });
    early += bad + again;
    if (asked > most) most = asked;
  }
  printf("%d %d", early, most >= 2 && most <= 8);
}
""")
    assert out == "0 1"


def test_every_kernel_asks_through_it():
    # hipFuncSetAttribute is called in one place
    hits = [f for f in sorted(os.listdir(CSRC)) if "hipFuncSetAttribute" in open(os.path.join(CSRC, f)).read()]
    assert hits == ["launch.h"]
