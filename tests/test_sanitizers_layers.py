"""Host code of the convolution, the selective scan and the verification under
AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: argument checks
and workspace sizes, driven by tests/sanitize/layers_harness.cpp (device code
is compiled but never launched).  A sanitizer report fails the test."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN_ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")


def test_argument_checks_under_sanitizers(tmp_path):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "layers_harness")
    csrc = os.path.join(ROOT, "linear_attention_rnn_gdn_amd", "csrc")
    # host-side sanitizers only (each -fsanitize after -Xarch_host)
    cmd = [hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "gdn_conv.hip"),
           os.path.join(csrc, "gdn_ssm.hip"), os.path.join(csrc, "gdn_verify.hip"), os.path.join(ROOT, "tests", "sanitize", "layers_harness.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, env=SAN_ENV, timeout=300)
    assert r.returncode == 0 and "all checks passed" in r.stdout, (r.stdout[-2000:], r.stderr[-2000:])
