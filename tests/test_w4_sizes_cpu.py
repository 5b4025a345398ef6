"""What the 4-bit products' kernels rely on, checked by host programs that include their headers (CPU only)."""
import os
import subprocess

from tests.helpers import ROOT


def run_host_program(name, tmp_path):
    exe = str(tmp_path / name)
    src = os.path.join(ROOT, "tests", "c", name + ".cpp")
    inc = os.path.join(ROOT, "moe_expert_offload_router_gb300", "csrc")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-Wall", "-Werror", "-I", inc, src, "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_a_tile_s_block_has_its_sm_to_itself(tmp_path):
    """The kernel takes all of an SM's tensor memory, for a pair of blocks at once: two blocks on an SM would wait for one
    another's."""
    run_host_program("w4_tile_alone", tmp_path)


def test_scales_and_zero_points_are_read_inside_their_arrays(tmp_path):
    run_host_program("four_of_row", tmp_path)
