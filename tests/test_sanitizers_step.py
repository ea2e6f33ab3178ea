"""AddressSanitizer + UndefinedBehaviorSanitizer over the host validation of the calls between the projections:
osc_api.hip rebuilt with the sanitizers on its host pass, linked with all of the library's other objects,
and tests/test_abi_step.py run against it in a child process."""
import glob
import os
import subprocess

import pytest


def test_step_validation_under_sanitizers(tmp_path):
    san = pytest.importorskip("test_sanitizers", reason="a checkout without it")
    objs = [o for o in sorted(glob.glob(os.path.join(san.PKG_BUILD, "*.o"))) if os.path.basename(o) != "osc_api.o"]
    if not os.path.exists(san.HIPCC) or len(objs) < 7:
        pytest.skip("needs hipcc and the library's objects (python w4a4_outlier_split_amd/build.py)")
    rt = glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so")
    if not rt:
        pytest.skip("no clang ASan runtime")
    host_san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    api, lib = str(tmp_path / "osc_api_san.o"), str(tmp_path / "libosc_san.so")
    subprocess.run([san.HIPCC, "-std=c++17", "-O1", "-g", "-fPIC", "--offload-arch=gfx950",
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *host_san,
                    "-I", os.path.join(san.ROOT, "include"), "-I", san.CSRC, "-c", os.path.join(san.CSRC, "osc_api.hip"),
                    "-o", api], check=True, capture_output=True)
    subprocess.run([san.HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", api, *objs, "-o", lib], check=True,
                   capture_output=True)
    san.run_child(["tests/test_abi_step.py"], rt[0], {"OSC_LIBRARY": lib}, tmp_path)
