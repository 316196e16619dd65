"""Stage tracing from several host threads at once (calls may come from any),
built with the compiler's thread sanitizer: no GPU is needed, since no event can
be made without one and the stages are counted all the same."""

import os
import shutil
import subprocess

import pytest

from rnn_joint_network_02_b200 import build as B

PROGRAM = """
#include <thread>
#include <vector>
#include "frnnt_internal.h"
int main() {
  std::vector<std::thread> all;
  for (int i = 0; i < 4; ++i)
    all.emplace_back([i] {
      for (int k = 0; k < 200; ++k) {
        frnnt::StageScope scope(i & 1 ? "one" : "two", nullptr);
        frnnt::note_launch();
        if (i == 0) frnnt_profile(k & 1);
        if (i == 3 && k % 50 == 0) frnnt_profile_read(nullptr, 0, nullptr);
      }
    });
  for (std::thread& t : all) t.join();
  return 0;
}
"""


def test_switching_and_reading_while_others_call(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(B._nvcc()):
        pytest.skip("needs nvcc and g++")
    main, exe = tmp_path / "main.cu", tmp_path / "main"
    main.write_text(PROGRAM)
    flags = [*B.ARCH, "-O1", "-g", "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, "--expt-relaxed-constexpr",
             "-Xcompiler", "-fsanitize=thread"]
    made = subprocess.run([B._nvcc(), *flags, str(main), os.path.join(B.CSRC, "frnnt_profile.cu"), "-o", str(exe)],
                          capture_output=True, text=True)
    if made.returncode and "tsan" in made.stderr:
        pytest.skip("no thread sanitizer here")
    assert made.returncode == 0, made.stderr
    ran = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120,
                         env=dict(os.environ, TSAN_OPTIONS="exitcode=66", CUDA_VISIBLE_DEVICES=""))
    assert ran.returncode == 0, ran.stderr[-3000:]
