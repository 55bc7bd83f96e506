"""The widest cluster that a kernel is launched with: 16 CTAs where the runtime says they fit, else the portable 8.
Host code of csrc/host.cuh, compiled into a program of its own with a runtime that answers as the test says."""

import os
import subprocess

from speculative_decode_draft_b200 import build

PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "host.cuh"
using namespace wmtp;
int main(int argc, char** argv) {
  static WidestOnce once;
  for (int i = 1; i < argc; ++i) {  // DEVICE:CLUSTERS THAT FIT
    int asked = 0, fit = 0, dev = 0;
    std::sscanf(argv[i], "%d:%d", &dev, &fit);
    const int most = widest_cluster(once, dev, 16, [&] { ++asked; return fit; });
    std::printf("%d%s ", most, asked ? "?" : "");
  }
}
"""


def test_clusters_of_16_only_where_they_fit(tmp_path):
    src, exe = tmp_path / "choice.cu", tmp_path / "choice"
    src.write_text(PROGRAM)
    csrc = os.path.join(build.HERE, "csrc")
    subprocess.run([build.nvcc(), "-std=c++17", "-I" + csrc, "-I" + os.path.join(build.ROOT, "include"), "-o", str(exe),
                    str(src)], check=True, capture_output=True)

    def run(*answers):
        return subprocess.run([str(exe), *answers], check=True, capture_output=True, text=True).stdout.split()
    assert run("0:37", "0:0") == ["16?", "16"]  # asked once
    assert run("0:0", "0:37") == ["8?", "8"]
    assert run("0:-1", "0:-1", "0:5", "0:0") == ["8?", "8?", "16?", "16"]  # a failure is not remembered
    assert run("0:1", "1:0", "0:0", "1:9") == ["16?", "8?", "16", "8"]  # each device for itself
