"""The segments the E4M3 decode's merge reads (csrc/segment_range.h): within the workspace whatever the split
left there, a rule checked on the host."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "exact_tiled_attention_36_b200", "csrc")


def test_segments_stay_in_the_workspace(tmp_path):
    exe = tmp_path / "segment_range_check"
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "segment_range_check.cpp"),
                           "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.strip() == "ok"


def test_the_merge_takes_the_rule_from_the_header():
    src = open(os.path.join(CSRC, "fa_decode_fp8.cuh")).read()
    assert '#include "segment_range.h"' in src
    merge = src[src.index("fa_decode8_combine"):]
    assert merge.count("segment_range(") == 1 and merge.count("a.meta[item]") == 1
