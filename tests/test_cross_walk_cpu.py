"""How the cross attention kernel cuts its work into runs, compiled for the host (tests/cross_walk_host.cpp)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("walk") / "cross_walk_host")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-I" + os.path.join(ROOT, "qwen3_vl_text_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "cross_walk_host.cpp"), "-o", out], check=True, timeout=300)
    return out


def _run(program, *args):
    r = subprocess.run([program, *args], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.startswith("ok "), (r.returncode, r.stdout[-500:])


def test_runs_of_segments_in_order(program):
    """Every step once, cut or whole, over 1500 calls; memory that a walk does not set is filled with another pattern."""
    _run(program)
