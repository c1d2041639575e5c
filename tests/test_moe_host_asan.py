"""The mixture-of-experts calls' host code under AddressSanitizer (CPU only, where no GPU is visible)."""

import os
import shutil
import subprocess

import pytest

from tests.test_host_asan import ROOT, _hipcc


@pytest.mark.skipif(_hipcc() is None or shutil.which("g++") is None, reason="hipcc and g++ are needed")
@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="runs only where no GPU is visible")
def test_moe_host_code_under_asan(tmp_path):
    from sparse_matmul_ffns_amd import build
    build.build()
    objs = [os.path.join(build.BUILD, os.path.splitext(s)[0] + ".o") for s in build.SOURCES if s != "api.cpp"]
    api_o, main_o, exe = tmp_path / "api_asan.o", tmp_path / "main.o", tmp_path / "moe_asan"
    flags = [f for f in build.FLAGS if not f.startswith("-O")]
    steps = [
        [_hipcc(), "-x", "hip", *flags, "-O1", "-g", "-Xarch_host", "-fsanitize=address", "-c",
         os.path.join(ROOT, "sparse_matmul_ffns_amd", "csrc", "api.cpp"), "-o", str(api_o)],
        ["g++", "-std=c++17", "-g", "-fsanitize=address", f"-I{os.path.join(ROOT, 'include')}", "-c",
         os.path.join(ROOT, "tests", "asan_moe_main.cpp"), "-o", str(main_o)],
        [_hipcc(), f"--offload-arch={build.ARCH}", "-Xarch_host", "-fsanitize=address", str(main_o), str(api_o), *objs,
         "-o", str(exe)],
    ]
    for cmd in steps:
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:exitcode=23")
    res = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert res.returncode == 0 and "asan moe ok" in res.stdout, (res.returncode, res.stdout[-2000:], res.stderr[-4000:])
