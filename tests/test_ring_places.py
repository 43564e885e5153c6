"""The weight rings of the few-row kernels on the host (csrc/ring_places.cuh), with waits that give up:
no load may be in flight when a CTA ends, since its shared memory is another's then."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "combine_ep_layout_03_gb300", "csrc")


def test_no_load_outlives_its_ring(tmp_path):
    exe = str(tmp_path / "ring_places_model")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-x", "c++", "-I", CSRC, "-o", exe,
                    os.path.join(HERE, "ring_places", "ring_places_model.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
