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
