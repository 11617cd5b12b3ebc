"""The layer calls' host code over a CUDA runtime that only keeps books
(tests/cpu_layers_launch.cpp), for what no GPU test can bring about at will: a
launch that falls between another thread's limit and launch, or fails."""
import importlib.util
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "sign_muon_optimizer_b200")


def _build_module():
    spec = importlib.util.spec_from_file_location("signmuon_build", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    build = _build_module()
    if shutil.which(build._nvcc()) is None or shutil.which("g++") is None:
        pytest.skip("no nvcc or no g++")
    build.build()                         # (objects that are up to date stay)
    exe = str(tmp_path_factory.mktemp("launch") / "cpu_layers_launch")
    cuda = os.path.join(os.path.dirname(os.path.dirname(build._nvcc())), "include")
    cmd = ["g++", "-std=c++17", "-O1", "-I", cuda, os.path.join(ROOT, "tests", "cpu_layers_launch.cpp")]
    cmd += [os.path.join(build.BUILD, s + ".o") for s in build.SOURCES] + ["-o", exe, "-ldl", "-lpthread"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    return exe


def _run(program, what):
    res = subprocess.run([program, what], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and "layer launches ok" in res.stdout, res.stdout + res.stderr


def test_a_kernels_shared_memory_limit_is_never_lowered(program):
    """The limit belongs to the kernel, for all handles and host threads: another
    thread's launch, made ready before it was lowered, would be refused."""
    _run(program, "limits")


def test_a_distillation_that_fails_between_its_launches_clears_its_counters(program):
    _run(program, "counters")
