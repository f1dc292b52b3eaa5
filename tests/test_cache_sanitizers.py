"""Sanitizer tier of the serving calls (CPU only): their C ABI's host code under AddressSanitizer and
UndefinedBehaviorSanitizer, driven by calls that validation refuses, linked with the regular build's kernels."""
import os
import shutil
from pathlib import Path

import pytest

from test_sanitizers import BUILD, HOST_SAN, KERNEL_OBJS, ROOT, SAN, _run

OBJS = KERNEL_OBJS + ["kda_api.o", "kda_heads.o", "kda_pages.o", "kda_tree.o"]


def test_serving_calls_under_asan_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    objs = [BUILD / o for o in OBJS]
    if not all(o.exists() for o in objs):
        pytest.skip("kernel objects not built (python -m gated_delta_rule_07_amd.build)")
    csrc = Path(ROOT) / "gated_delta_rule_07_amd" / "csrc"
    common = ["-x", "hip", "--offload-host-only", "-O1", "-g", "-std=c++17", f"-I{ROOT / 'include'}", f"-I{csrc}", *HOST_SAN]
    api_o, main_o, exe = tmp_path / "api.o", tmp_path / "main.o", tmp_path / "cache_san"
    _run([hipcc, *common, "-c", str(csrc / "kda_cache_api.cpp"), "-o", str(api_o)])
    _run([hipcc, *common, "-c", str(SAN / "cache_main.cpp"), "-o", str(main_o)])
    _run([hipcc, *HOST_SAN, "--offload-arch=gfx950", str(main_o), str(api_o), *map(str, objs), "-o", str(exe)])
    # the HIP runtime's own allocations at load are not ours to judge: leaks off
    r = _run([str(exe)], env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert "clean" in r.stdout and "runtime error" not in r.stderr
