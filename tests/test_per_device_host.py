"""What the launchers keep of a kernel (its shared-memory limit, its resident CTAs) is kept per
device: PerDevice of common.cuh, compiled for the host with a stand-in for cudaGetDevice."""
import os
import re
import subprocess

import pytest

from int2_rotated_kv_rotate_gb300 import build

PROGRAM = """
#include <atomic>
#include <cstdio>
#include <initializer_list>
typedef int cudaError_t;
const int cudaSuccess = 0;
static int device = 0, error = 0, made[70];
static int cudaGetDevice(int* d) { *d = device; return error; }
%s
int main() {
  static PerDevice p;
  auto call = [] { ++made[device]; return device == 2 ? -9 : 10 + device; };
  for (int round = 0; round < 3; ++round)
    for (int d : {0, 1, 2, 63, 64}) { device = d; std::printf("%%d ", p.get(call)); }
  error = 3;
  std::printf("%%d : %%d %%d %%d %%d %%d", p.get(call), made[0], made[1], made[2], made[63], made[64]);
}
"""


def test_values_belong_to_their_device(tmp_path):
    text = open(os.path.join(build.CSRC, "common.cuh")).read()
    source = tmp_path / "per_device.cpp"
    source.write_text(PROGRAM % re.search(r"^struct PerDevice \{.*?^\};$", text, re.M | re.S).group(0))
    subprocess.run(["g++", "-std=c++17", "-o", str(tmp_path / "per_device"), str(source)], check=True)
    out = subprocess.run([str(tmp_path / "per_device")], check=True, capture_output=True, text=True).stdout
    # an error is not kept, nor is what lies beyond the table
    assert out == "10 11 -9 73 74 " * 3 + "-3 : 1 1 3 1 3"


@pytest.mark.parametrize("name", ["append.cu", "bf16.cu", "decode.cu", "evict.cu", "shared.cu"])
def test_launchers_keep_nothing_per_process(name):
    text = open(os.path.join(build.CSRC, name)).read()
    assert not re.search(r"static (bool|int) \w+ = ", text)
