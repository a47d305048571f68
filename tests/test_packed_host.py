"""Host test of where a wave is in a packed batch.

Compiles ``tests/packed_host_check.cpp`` against the library's
``gdn2_packed.h`` with g++ and runs it: sequence starts, ends and indices of
every 8 tokens, as the recurrence's and the convolution's kernels look them
up, against a plain list of boundaries, with more sequences than the 64 that a
wave holds at once, empty ones among them; and each lane's channels at every
width (no GPU).
"""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_slices_see_every_boundary(tmp_path):
    exe = tmp_path / "packed_host_check"
    src = os.path.join(ROOT, "tests", "packed_host_check.cpp")
    inc = os.path.join(ROOT, "linear_attention_rnn_gdn2_amd", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wno-unknown-pragmas", "-I", inc, src, "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "ok"
