"""The notices of looked-through value tiles in the decode over an 8-bit cache (csrc/notice_ring.h):
every order of the warps' steps is walked through on the host, so it runs without a GPU."""
import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "exact_tiled_attention_36_b200", "csrc")


def test_every_order_of_steps_ends(tmp_path):
    exe = tmp_path / "notice_ring_check"
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-I", CSRC, os.path.join(HERE, "notice_ring_check.cpp"),
                           "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.strip() == "ok"


def test_both_kernels_take_the_barriers_from_the_header():
    for name in ("fa_decode_fp8.cuh", "fa_decode_fp8_rows.cuh"):
        src = open(os.path.join(CSRC, name)).read()
        assert "kNotices >= ring_values(kUnits)" in src, name
        assert len(re.findall(r"v_seen\[notice_bar\(\w+\)\]", src)) == 2, name  # the notice, the wait
        assert len(re.findall(r"v_due\[notice_bar\(\w+\)\]", src)) == 2, name
        assert len(re.findall(r"notice_parity\(\w+\)", src)) == 2, name
        assert not re.search(r"mbar_(arrive|wait)\(v_(seen|due)\b(?!\[)", src), name
