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


def test_runs_of_any_offsets(program):
    """Offsets that run back or lie outside: the weights stay within the bound that the call is accepted by (so 32 bits hold
    them), and every item within its tensors.  1024 offsets that go between 0 and 16,384 queries, and 0 and 200,000 keys,
    in turns would come to 6.6e9 (64 heads over 8) where the bound is 3.8e7."""
    _run(program, "any")
