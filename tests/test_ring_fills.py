"""What a CTA that gives up waits for: the fills of a ring that may still be under way (compiled for the host)."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_no_fill_is_under_way_after_the_waits(tmp_path):
    exe = str(tmp_path / "ring_fills")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    os.path.join(HERE, "host", "ring_fills.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert int(out.stdout) == 15000
