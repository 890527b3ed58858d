"""The library's build runs no more compilers at a time than the machine has cores and memory for, and
waits for all of them before it complains about one."""
import os
import subprocess
import threading
import time

import pytest

from ternary_weight_bit_absmean_b200 import build_lib

pytestmark = pytest.mark.cpu


class Compilers:
    """subprocess.run that writes the output file and counts how many run at once."""

    def __init__(self, fails=()):
        self.lock, self.now, self.most, self.ended, self.fails = threading.Lock(), 0, 0, 0, fails

    def __call__(self, cmd, check=False, **kw):
        with self.lock:
            self.now += 1
            self.most = max(self.most, self.now)
        time.sleep(0.02)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("object")
        with self.lock:
            self.now -= 1
            self.ended += 1
        return subprocess.CompletedProcess(cmd, int(any(name in " ".join(cmd) for name in self.fails)))


@pytest.fixture
def build(monkeypatch, tmp_path):
    monkeypatch.setattr(build_lib, "PKG", str(tmp_path))
    monkeypatch.setattr(build_lib, "LIB", str(tmp_path / "lib.so"))

    def run(compilers, cores=64, memory=64 << 30, limit=None):
        monkeypatch.setattr(build_lib.subprocess, "run", compilers)
        monkeypatch.setattr(build_lib.subprocess, "Popen", None)
        monkeypatch.setattr(build_lib.os, "sched_getaffinity", lambda pid: set(range(cores)))
        monkeypatch.setattr(build_lib, "free_memory", lambda: memory)
        if limit is None:
            monkeypatch.delenv("BL_BUILD_JOBS", raising=False)
        else:
            monkeypatch.setenv("BL_BUILD_JOBS", str(limit))
        return build_lib.build(force=True)
    return run


@pytest.mark.parametrize("cores,memory,limit,most", [
    (64, 64 << 30, None, len(build_lib.SOURCES)), (3, 64 << 30, None, 3), (64, (4 << 30) + 5, None, 4), (1, 0, None, 1),
    (64, 64 << 30, 2, 2), (2, 64 << 30, 8, 2)])
def test_no_more_compilers_than_cores_and_memory(build, cores, memory, limit, most):
    compilers = Compilers()
    lib = build(compilers, cores, memory, limit)
    assert os.path.exists(lib)
    assert compilers.most <= most and compilers.ended == len(build_lib.SOURCES) + 1  # and the linker
    assert build_lib.jobs() == most


def test_all_have_ended_before_one_is_complained_about(build):
    compilers = Compilers(fails=("k_tl5.cu",))
    with pytest.raises(subprocess.CalledProcessError):
        build(compilers, cores=4)
    assert compilers.ended == len(build_lib.SOURCES) and compilers.now == 0
    assert not os.path.exists(build_lib.LIB)


def test_free_memory_is_known_here():
    assert build_lib.free_memory() > 1 << 20
