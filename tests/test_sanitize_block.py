"""Sanitizer build of the block map's lookup (CPU only, no GPU): a launch covers
moe_max_blocks entries, and those behind the map are not read
(tests/sanitize/block_main.hip, as tests/test_sanitize_host.py builds its drivers)."""

from __future__ import annotations

import os
import subprocess

import pytest

from test_sanitize_host import ENV, HIPCC, OUT, ROOT, SAN, _run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_block_map_under_asan():
    os.makedirs(OUT, exist_ok=True)
    exe = os.path.join(OUT, "block_san")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
           "-Xarch_host", "-fsanitize=address",
           "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "w4_dequant_expert_amd", "csrc"),
           os.path.join(SAN, "block_main.hip"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "block map sanitizer driver ok" in _run(exe, ENV)
