"""A call of two launches whose second fails: the workspace's counters, which the second
kernel would have reset, are cleared, so that the next call finds them as it needs them.
The failure is made on the host: a child process runs the library with its launch, its
facts of the device and its memset replaced by a fake (no GPU, nothing runs)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_decode_attention_v2_gb300", "csrc")

FAKE = r"""
#include <stdio.h>
#include "pa_host.h"
namespace pa {
pa_status_t host_sm_count(int *sms) { *sms = 152; return PA_OK; }
pa_status_t host_ensure_smem(const void *, size_t) { return PA_OK; }
pa_status_t host_cache_map(CUtensorMap *, const void *, int, int, long long, int) { return PA_OK; }
pa_status_t host_rows_map(CUtensorMap *, const void *, int, int, long long, int) { return PA_OK; }
void host_clear(void *at, size_t bytes, void *stream) {
  printf("clear %zu %zu %zu\n", (size_t)at, bytes, (size_t)stream);
}
pa_status_t host_launch(const void *, unsigned, unsigned, int, size_t, void *, void **, const char *what) {
  static int n = 0;
  printf("launch %d\n", ++n);
  return n == FAILS ? PA_ERR_CUDA : PA_OK;
}
}
"""

CHILD = r"""
import ctypes, sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import paged_decode_attention_v2_gb300 as pa
import test_latent, test_q4
lib = pa.load_library()
if sys.argv[2] == "q4":
    print("status", lib.pa_q4_forward(*dict(test_q4.FORWARD, stream=77).values()), flush=True)
else:
    print("status", lib.pa_latent_forward(*dict(test_latent.FORWARD, stream=77).values()), flush=True)
"""


@pytest.mark.parametrize("which", ["q4", "latent"])
@pytest.mark.parametrize("fails", [1, 2, 3])
def test_counters_after_a_failed_launch(tmp_path, which, fails):
    import __graft_entry__
    import paged_decode_attention_v2_gb300 as pa
    from test_q4 import FAKE as WORKSPACE
    __graft_entry__.build()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc")))
    src, so = tmp_path / "fake.cpp", tmp_path / "fake.so"
    src.write_text(FAKE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", f"-DFAILS={fails}", "-I", CSRC, "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(cuda, "include"), str(src), "-o", str(so)], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, which], env=dict(os.environ, LD_PRELOAD=str(so), CUDA_VISIBLE_DEVICES=""),
                       capture_output=True, text=True, timeout=600)
    said = r.stdout.split("\n")
    assert r.returncode == 0, r.stderr
    assert f"status {pa.PA_OK if fails > 2 else pa.PA_ERR_CUDA}" in said
    assert f"launch {min(fails, 2)}" in said and "launch 3" not in said
    # the four counters behind the sixteenth word of the status block, on the call's stream
    cleared = [line for line in said if line.startswith("clear")]
    assert cleared == ([f"clear {WORKSPACE + 64} 16 77"] if fails == 2 else [])
