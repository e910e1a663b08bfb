"""The decoder operators' host layer under AddressSanitizer and UndefinedBehaviorSanitizer (no GPU):
tests/host/decoder_host_test.cpp links capi.cpp, capi_decoder.cpp and both plans as shipped against
stand-in launchers that perform the kernels' workspace writes on exact-size buffers."""
import os
import subprocess

import pytest

from test_host_sanitized import CSRC, HIP_INC, ROOT

import shutil


def _run(tmp_path, plan):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(HIP_INC, "hip", "hip_runtime.h")):
        pytest.skip("g++ or the HIP headers are missing")
    exe = str(tmp_path / "decoder_host_test")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-Wno-unused-function", f"-I{HIP_INC}",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", *(os.path.join(CSRC, f) for f in
                                                               ("capi.cpp", "capi_decoder.cpp", "plan.cpp")), plan,
           os.path.join(ROOT, "tests", "host", "decoder_host_test.cpp"), "-o", exe]
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert p.returncode == 0, p.stdout
    return subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600,
                          env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))


def test_decoder_host_layer_sanitized(tmp_path):
    p = _run(tmp_path, os.path.join(CSRC, "decoder_plan.cpp"))
    assert p.returncode == 0, p.stdout[-4000:]
    assert " 0 failures" in p.stdout


def test_the_harness_catches_an_undersized_workspace(tmp_path):
    """A planted mistake in a copy of the plan (the decode parts without their maxima) must fail."""
    src = open(os.path.join(CSRC, "decoder_plan.cpp")).read()
    good = "p.units * p.splits * decode_part_floats(head_dim)"
    assert good in src
    bad = tmp_path / "plan_undersized.cpp"
    bad.write_text(src.replace(good, "p.units * p.splits * (size_t)kDecHeads * head_dim").replace(
        '#include "decoder_plan.h"', f'#include "{os.path.join(CSRC, "decoder_plan.h")}"'))
    p = _run(tmp_path, str(bad))
    assert p.returncode != 0
    assert "heap-buffer-overflow" in p.stdout or "FAIL" in p.stdout
