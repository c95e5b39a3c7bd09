"""Every unit of the prompt kernel is taken, in whatever order its blocks start and are taken over (compiled
for the host)."""
import os
import re
import subprocess

from nvfp4_activation_quantize_gb300 import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_unit_is_taken_once(tmp_path):
    exe = str(tmp_path / "units_taken")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    os.path.join(HERE, "host", "units_taken.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert int(out.stdout) > 10000


def test_the_kernel_goes_by_it():
    text = re.sub(r"//.*", "", open(os.path.join(libbuild.CSRC, "attention.cu")).read())
    assert len(re.findall(r"\bblock = ", text)) == 2 and "block = next_block(" in text   # (the first: its own)
