"""Host-side records that calls from several threads share, in C++ programs of
their own against a model of the CUDA runtime (no GPU)."""
import os
import subprocess

import pytest

from structured_state_space_dplr_b200 import build as s4build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "structured_state_space_dplr_b200", "csrc")
HOST = os.path.join(ROOT, "tests", "host")


def run(tmp_path, source, *flags):
    exe = str(tmp_path / "program")
    cuda = os.path.join(os.path.dirname(os.path.dirname(s4build._nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", *flags, "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    "-isystem", cuda, os.path.join(HOST, source), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("flags", [(), ("-fsanitize=thread",)])
def test_shared_memory_limit_from_two_threads(tmp_path, flags):
    run(tmp_path, "smem_limit.cpp", *flags)


def test_resident_blocks_from_four_threads(tmp_path):
    run(tmp_path, "resident.cpp", "-fsanitize=thread")


def test_the_last_copy_of_every_stage_is_waited_for(tmp_path):
    exe = str(tmp_path / "program")
    subprocess.run([s4build._nvcc(), *s4build.NVCC_FLAGS, os.path.join(HOST, "last_parity.cu"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
