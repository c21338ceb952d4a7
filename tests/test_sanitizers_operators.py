"""The delta rule's and the page operators' host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only).

Their argument checks and workspace layouts are built with both sanitizers on the host side only and driven by
tests/sanitize/operators_driver.c with values at the edges of every type and limit; no call there reaches a launch."""
import os
import shutil
import subprocess

import pytest

SAN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "sanitize")
HIPCC = os.environ.get("HIPCC") or "/opt/rocm/bin/hipcc"


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
    return r


def test_operators_host_code_under_asan_and_ubsan(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.exists(HIPCC):
        pytest.skip("gcc or hipcc not found")
    from device_wide_prefix_amd import build as hip_build
    host_sources = ("dws_delta_abi.cpp", "dws_pages_abi.cpp")
    others = [os.path.join(hip_build.BUILD_DIR, os.path.splitext(s)[0] + ".o")
              for s in hip_build.SOURCES if s not in host_sources]
    if not all(os.path.exists(o) for o in others):
        hip_build.build(verbose=False)
    flags = [f"--offload-arch={hip_build.ARCH}", "-O1", "-g", "-std=c++17", "-fPIC", "-fno-omit-frame-pointer",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             f"-I{hip_build.INCLUDE}", f"-I{hip_build.CSRC}",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all"]
    objs = []
    for src in host_sources:
        obj = str(tmp_path / (os.path.splitext(src)[0] + ".o"))
        _run([HIPCC, *flags, "-x", "hip", "-c", os.path.join(hip_build.CSRC, src), "-o", obj])
        objs.append(obj)
    drv = str(tmp_path / "operators_driver.o")
    _run([gcc, "-std=c11", "-O1", "-g", "-fno-omit-frame-pointer", "-Wall", "-Wextra", "-Werror",
          f"-I{hip_build.INCLUDE}", "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__",
          "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-c", os.path.join(SAN, "operators_driver.c"),
          "-o", drv])
    exe = str(tmp_path / "operators_driver")
    _run([HIPCC, f"--offload-arch={hip_build.ARCH}", "-fno-gpu-sanitize", "-fsanitize=address,undefined",
          drv, *objs, *others, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = _run([exe], env=env, timeout=120)
    assert "operators driver: ok" in r.stdout
