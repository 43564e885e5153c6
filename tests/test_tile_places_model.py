"""The arithmetic by which the tensor-core kernels find a tile, their ring positions and the rule on the FP8 product's stages
(csrc/tile_places.cuh), compiled for the host; and copies of it with a mistake, each of which is found."""
import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "combine_ep_layout_03_gb300", "csrc")


def configurations():
    with open(os.path.join(CSRC, "matmul_fp8.cu")) as f:
        text = f.read()
    assert "static_assert(no_warp_laps(STAGES, ACCS)" in text
    found = re.findall(r"using \w+ = Config<\d+, \d+, \d+, (\d+), (\d+), \d+>", text)
    assert len(found) == 4
    return "".join(f" X({stages}, {accs})" for stages, accs in found)


def run(tmp_path, include):
    exe = str(tmp_path / "tile_places_model")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-x", "c++", "-I", include, f"-DCONFIGS={configurations()}", "-o", exe,
                    os.path.join(HERE, "tile_places", "tile_places_model.cpp")], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=120)


def test_tiles_and_rings(tmp_path):
    r = run(tmp_path, CSRC)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("was,wrong", [
    ("return q + (n - q * d.of >= d.of);", "return q;"),
    ("if (rest < 0) q -= 1, rest += d;\n    else if", "if"),
    ("else if (rest >= (int32_t)d) q += 1, rest -= d;", ""),
    ("divide(local - before * ctiles, kGroup < left ? kGroup : left)", "divide(local - before * ctiles, kGroup)"),
    ("(int)(before + q.rest)", "(int)q.rest"),
    ("32 * (j * each + (j < more ? j : more))", "32 * j * each"),
    ("most < rows - first ? most : rows - first", "most"),
    ("stages >= accs + 2", "stages >= accs + 1"),
    ("{ stage = 0; parity ^= 1; }", "{ stage = 0; }"),
])
def test_mistakes_are_found(was, wrong, tmp_path):
    with open(os.path.join(CSRC, "tile_places.cuh")) as f:
        text = f.read()
    assert text.count(was) == 1
    (tmp_path / "tile_places.cuh").write_text(text.replace(was, wrong))
    assert run(tmp_path, str(tmp_path)).returncode != 0
