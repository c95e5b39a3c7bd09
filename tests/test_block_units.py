"""Which unit of attention over blocks a block of the launch has: every one is covered once, those of the last turn in
halves where that fits."""
import os
import subprocess

from nvfp4_activation_quantize_gb300 import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))


def test_blocks_cover_all_units(tmp_path):
    exe = str(tmp_path / "block_units")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", libbuild.CSRC, os.path.join(HERE, "host", "block_units.cpp"), "-o", exe],
                   check=True)
    cases = [(u, s) for s in (0, 1, 2, 3, 8, 152) for u in (*range(0, 20), 76, 77, 151, 152, 153, 228, 229, 640, 7168)]
    out = subprocess.run([exe], input="\n".join(f"{u} {s}" for u, s in cases), text=True, check=True,
                         capture_output=True).stdout.split()
    assert out == ["ok"] * len(cases), [c for c, o in zip(cases, out) if o != "ok"]
