"""A process with two GPUs, on CPU: the library's own objects linked with a stand-in for the CUDA runtime
(tests/fake_cudart.cpp).  What a call launches on one device does not depend on what ran on the other before, and a
kernel that needs more than 48 KB of shared memory gets it on both."""
import json
import os
import subprocess
import sys

import pytest

from fp4_compressed_sparse_02_gb300 import build

TESTS = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    objects = [os.path.join(build.BUILD, u.replace(".cu", ".o")) for u in build.UNITS]
    lib = build.build()
    if not all(os.path.exists(o) and os.path.getmtime(o) <= os.path.getmtime(lib) for o in objects):
        build.build(force=True)
    out = str(tmp_path_factory.mktemp("fake") / "libcsa2_fake.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", cuda, "-o", out,
                        os.path.join(TESTS, "fake_cudart.cpp"), *objects, "-lpthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


def run(library, order):
    r = subprocess.run([sys.executable, os.path.join(TESTS, "two_devices.py"), library, order], capture_output=True, text=True,
                       cwd=build.ROOT, env={**os.environ, "PYTHONPATH": build.ROOT}, timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout)


@pytest.fixture(scope="module")
def alone(library):
    out = run(library, "1")
    assert all(status == 0 and launches for _, status, _, launches in out), [o[:3] for o in out if o[1] or not o[3]]
    return out


def test_a_second_device_launches_what_it_would_alone(library, alone):
    both = run(library, "01")
    bad = [(i, b[:3], a[3], b[3]) for i, (a, b) in enumerate(zip(alone, both)) if a != b]
    assert not bad, bad


def test_first_calls_from_several_threads(library, alone):
    threads = run(library, "threads")
    bad = [(i, b[:3]) for i, (a, b) in enumerate(zip(alone, threads)) if b[1] != 0 or b[3] != sorted(4 * a[3])]
    assert not bad, bad
