"""Tests that need no GPU reach none: a session of such tests hides the devices, and one that also has gpu
tests leaves out those whose accepted calls name addresses of no memory."""
import os
import subprocess
import sys
from pathlib import Path

import conftest

HERE = os.path.dirname(os.path.abspath(__file__))


class Item:
    def __init__(self, file, gpu):
        self.path, self.gpu = Path("/somewhere/tests") / file, gpu

    def get_closest_marker(self, name):
        return self.gpu if name == "gpu" else None


def test_a_session_of_both_kinds():
    items = [Item("test_gpu_quantize.py", True), Item("test_abi.py", False), Item("test_attention_abi.py", False),
             Item("test_oracle_quantize.py", False)]
    before = os.environ.get("CUDA_VISIBLE_DEVICES")
    assert conftest.reaches_no_gpu(items, lambda: True) == [items[0], items[3]]
    assert conftest.reaches_no_gpu(items, lambda: False) == items
    assert os.environ.get("CUDA_VISIBLE_DEVICES") == before


def _session(tmp_path, *args):
    (tmp_path / "test_one.py").write_text(
        "import os\nimport pytest\n"
        "def test_host():\n    assert os.environ['CUDA_VISIBLE_DEVICES'] == ''\n"
        "@pytest.mark.gpu\ndef test_device():\n    assert os.environ['CUDA_VISIBLE_DEVICES'] == '0'\n")
    env = {**os.environ, "PYTHONPATH": HERE, "CUDA_VISIBLE_DEVICES": "0"}
    return subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "conftest", "-p", "no:cacheprovider", *args,
                           str(tmp_path / "test_one.py")], env=env, cwd=tmp_path, capture_output=True, text=True)


def test_a_session_without_gpu_tests_sees_no_device(tmp_path):
    for args in (("-m", "not gpu"), ("-k", "host")):
        run = _session(tmp_path, *args)
        assert run.returncode == 0, run.stdout + run.stderr


def test_a_session_of_gpu_tests_keeps_its_device(tmp_path):
    run = _session(tmp_path, "-m", "gpu")
    assert run.returncode == 0, run.stdout + run.stderr


def test_the_files_exist():
    assert all(os.path.exists(os.path.join(HERE, name)) for name in conftest.NO_MEMORY)
