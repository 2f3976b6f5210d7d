"""A check of the kernels' listings that needs no GPU: where paths join, nothing
is done to vector registers before the lanes that took the other path are
switched on again.  This compiler once put copies of live addresses (to
accumulation registers, in a kernel that needed more than 256) there, and with
the lanes off they were lost: the kernel read wild addresses."""
import os
import re
import shutil
import subprocess

import pytest

from linear_attention_rnn_gdn_amd import build as hip_build

VECTOR = ("v_", "global_", "ds_", "buffer_", "flat_", "scratch_")
LANES = ("v_readlane", "v_writelane", "v_readfirstlane")   # (do not depend on which lanes are on)


def early(text):
    """(kernel, first such instruction) of every join with vector work before its lanes are restored."""
    lines = [line.strip() for line in text.split("\n")]
    targets = set(re.findall(r"s_cbranch_execz (\.LBB\d+_\d+)", text))
    found, kernel = [], None
    for i, line in enumerate(lines):
        if re.match(r"^_Z\w+:", line):
            kernel = line.split(":")[0]
        m = re.match(r"^(\.LBB\d+_\d+):", line)
        if not m or m.group(1) not in targets:
            continue
        first = None
        for t in lines[i + 1:]:
            if re.match(r"s_or_b64 exec, exec", t):
                if first:
                    found.append((kernel, first))
                break
            if re.match(r"(\.LBB\d+_\d+|\.Lfunc_end\d+):", t) or (t.startswith("s_") and ("branch" in t or "exec" in t or "endpgm" in t)):
                break
            if t.startswith(VECTOR) and not t.startswith(LANES):
                first = first or t
    return found


def test_the_check_finds_an_early_copy():
    text = """_Zk:
  s_and_saveexec_b64 s[0:1], vcc
  s_cbranch_execz .LBB0_2
  v_mov_b32 v0, 1
.LBB0_2:
  s_mov_b32 s4, 1
  {}
  s_or_b64 exec, exec, s[0:1]
  v_mov_b32 v1, v0
  s_endpgm
"""
    assert early(text.format("v_accvgpr_write_b32 a2, v112")) == [("_Zk", "v_accvgpr_write_b32 a2, v112")]
    assert early(text.format("v_readlane_b32 s3, v255, 1")) == []


@pytest.mark.parametrize("name", ["gdn_conv", "gdn_ssm", "gdn_verify"])
def test_joins_restore_their_lanes_first(name, tmp_path):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not os.path.exists(hipcc) and not shutil.which(hipcc):
        pytest.skip("hipcc not available")
    flags = [f for f in hip_build.HIPCC_FLAGS if f != "-shared"]
    out = str(tmp_path / "x.s")
    r = subprocess.run([hipcc] + flags + ["-S", "--offload-device-only", os.path.join(hip_build.CSRC, name + ".hip"), "-o", out],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    assert "s_endpgm" in text and early(text) == []
    # and none of these kernels needs accumulation registers as room for others
    assert "v_accvgpr" not in text
