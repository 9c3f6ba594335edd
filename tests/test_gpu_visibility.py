"""A run that holds a test without the gpu mark never reaches a GPU.

Tests of argument checks call the library with made-up device addresses and valid arguments; what ends these calls
before a launch is that there is no device. So conftest.py hides the GPUs of a machine that has some from every run but
those of gpu tests alone. The runs below are child processes with a copy of that conftest; none of them uses CUDA."""

import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
MODULE = """
import os
import pytest

seen = os.environ.get("CUDA_VISIBLE_DEVICES")  # while the module is imported

def record(name):
    with open(os.environ["RECORD"], "a") as f:
        f.write(f"{name} {seen!r} {os.environ.get('CUDA_VISIBLE_DEVICES')!r}\\n")

@pytest.mark.gpu
def test_marked():
    record("marked")

def test_unmarked():
    record("unmarked")
"""


@pytest.mark.parametrize("visible", ["0", None])
@pytest.mark.parametrize("args,ran", [
    ((), ["unmarked '' ''"]),                       # the gpu test is skipped
    (("-m", "not gpu"), ["unmarked '' ''"]),
    (("-m", "gpu"), ["marked '' {}"]),
    (("-k", "test_marked"), ["marked '' {}"]),
])
def test_gpus_are_hidden_from_tests_without_the_mark(tmp_path, args, ran, visible):
    shutil.copy(os.path.join(HERE, "conftest.py"), tmp_path / "conftest.py")
    (tmp_path / "test_it.py").write_text(MODULE)
    record = tmp_path / "record"
    env = {k: v for k, v in os.environ.items() if "VISIBLE_DEVICES" not in k and not k.startswith("PYTEST")}
    env["RECORD"] = str(record)
    if visible is not None:
        env["CUDA_VISIBLE_DEVICES"] = visible
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "--rootdir", str(tmp_path), *args,
                        str(tmp_path)], env=env, cwd=tmp_path, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert record.read_text().splitlines() == [x.format(repr(visible)) for x in ran]


def test_this_run():
    assert os.environ.get("CUDA_VISIBLE_DEVICES") == ""
