"""AddressSanitizer + UBSan build of the host code of the attention block's operators (layouts,
workspace sizes, argument checks), driven by tests/host_sanitize_attention_main.cpp.

The host units are rebuilt with g++ and the sanitizers and linked with the
device objects of the normal build; nothing is launched.  Leak detection is on.
"""
import glob
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "equivariant_gnn_tensor_receiver_amd", "csrc")
BUILD = os.path.join(ROOT, "_build")
HOST_UNITS = ("api", "plan", "timing", "stream_dispatch", "layers", "attention")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_attention_host_code_under_asan_and_ubsan(tmp_path):
    objs = [o for o in sorted(glob.glob(os.path.join(BUILD, "*.o")))
            if os.path.basename(o)[:-2] not in HOST_UNITS]
    if not any(o.endswith("attention_join.o") for o in objs) or not os.path.exists(os.path.join(BUILD, "gen", "cg_tables.inc")):
        pytest.skip("library objects not built")
    inc = ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(BUILD, "gen")]
    host = []
    for src in [os.path.join(CSRC, u + ".cpp") for u in HOST_UNITS] + [
            os.path.join(ROOT, "tests", "host_sanitize_attention_main.cpp")]:
        host.append(str(tmp_path / (os.path.basename(src) + ".o")))
        subprocess.run(["g++", "-O1", "-g", "-std=c++17"] + SAN + inc + ["-c", src, "-o", host[-1]], check=True)
    exe = str(tmp_path / "host_sanitize_attention")
    subprocess.run(["g++"] + SAN + ["-o", exe] + host + objs +
                   ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "host sanitizer checks passed" in r.stdout
