"""How decode_int4 joins segments cut between CTAs, on the CPU: tests/c/join_int4.cpp takes the CTAs of many splits
through the rounds of csrc/join_int4.h in random orders.  Every cut segment gets each of its shares exactly once, in the
order of the line, and all counters end at zero; a mistake planted in the model is found."""

from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_int4_join_gives_every_share_once_in_any_order(tmp_path):
    exe = tmp_path / "join_int4"
    build = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                            os.path.join(ROOT, "paged_kv_cache_330_b200", "csrc"),
                            os.path.join(ROOT, "tests", "c", "join_int4.cpp"), "-o", str(exe)],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "0 wrong", run.stdout + run.stderr
    # the state of a CTA's second segment overwritten by the first one's second round
    run = subprocess.run([str(exe), "planted"], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and int(run.stdout.split()[0]) > 100, run.stdout + run.stderr
