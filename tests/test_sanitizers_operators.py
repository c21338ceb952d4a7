"""The delta rule's and the page operators' host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only).

Their argument checks and workspace layouts are built with both sanitizers on the host side only and driven by
tests/sanitize/operators_driver.c with values at the edges of every type and limit; no call there reaches a launch."""
import os

import pytest

from test_sanitizers import ENV_UBSAN, HIPCC, ROOT, SAN, _gcc, _run


def test_operators_host_code_under_asan_and_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not found")
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
    _run([_gcc(), "-std=c11", "-O1", "-g", "-fno-omit-frame-pointer", "-Wall", "-Wextra", "-Werror",
          f"-I{hip_build.INCLUDE}", "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__",
          "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-c", os.path.join(SAN, "operators_driver.c"),
          "-o", drv])
    exe = str(tmp_path / "operators_driver")
    _run([HIPCC, f"--offload-arch={hip_build.ARCH}", "-fno-gpu-sanitize", "-fsanitize=address,undefined",
          drv, *objs, *others, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS=ENV_UBSAN)
    r = _run([exe], env=env, timeout=120)
    assert "operators driver: ok" in r.stdout
