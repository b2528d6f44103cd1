"""The residual-block operators' host-side argument handling (block_abi.cpp) under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: rebuilt with the sanitizers, linked with the kernels' objects as
built, and taken through tests/test_block_host.py in a child process, as test_sanitizers.py does for
delta_abi.cpp."""
import glob
import os
import subprocess

import pytest

base = pytest.importorskip("test_sanitizers")

RUN = base.ABI_RUN.replace("tests/test_abi_host.py", "tests/test_block_host.py")


def test_block_abi_host_checks_under_asan_ubsan(tmp_path):
    clang = os.path.join(base.ROCM, "lib", "llvm", "bin", "clang++")
    rt = sorted(glob.glob(os.path.join(base.ROCM, "lib", "llvm", "lib", "clang", "*", "lib", "linux",
                                       "libclang_rt.asan-x86_64.so")))
    pkg = os.path.join(base.ROOT, "chunkwise_delta_rule_chunked_amd")
    objs = [o for o in sorted(glob.glob(os.path.join(pkg, "_build", "*.o"))) if os.path.basename(o) != "block_abi.o"]
    if not os.path.exists(clang) or not rt or len(objs) < 5:
        pytest.skip("needs ROCm's clang, its sanitizer runtime and the library's built objects")
    abi, lib = str(tmp_path / "block_abi_san.o"), str(tmp_path / "libdelta_san.so")
    subprocess.run([clang, "-x", "c++", "-std=c++17", "-O1", "-g", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                    "-I" + os.path.join(base.ROCM, "include")] + base.SAN +
                   ["-c", os.path.join(pkg, "csrc", "block_abi.cpp"), "-o", abi], check=True)
    subprocess.run([os.path.join(base.ROCM, "bin", "hipcc"), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", lib, abi] + objs,
                   check=True, capture_output=True)
    undef = subprocess.run(["nm", "-D", "--undefined-only", lib], capture_output=True, text=True).stdout
    assert "__asan_" in undef and "__ubsan_" in undef
    out = base._child(RUN % lib, rt[-1])
    assert " passed" in out and " failed" not in out
