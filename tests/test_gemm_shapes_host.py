"""The choice of a product's kernel, tile and split of K (csrc/gemm_shape.h), compiled
with g++: each size of tests/gemm_sizes.py runs the kernel it stands for, and no drawn
size runs one that the list lacks, so a change of the choice cannot leave a kernel
without its GPU tests.  No GPU is used."""

import os
import shutil
import subprocess

import pytest

from gemm_sizes import INSTANCES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("g++ missing")
    out = tmp_path_factory.mktemp("shapes") / "shapes"
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                        "-I", os.path.join(ROOT, "mxfp8_weight_repack_amd", "csrc"),
                        os.path.join(ROOT, "tests", "host_gemm_shapes.cpp"), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return str(out)


def test_every_size_runs_the_kernel_it_stands_for(exe):
    rows = [(name, size) for name, sizes in INSTANCES.items() for size in sizes if size]
    text = "".join(f"{int(' nn' in name)} {m} {n} {k} {int('bf16' in name)}\n" for name, (m, n, k) in rows)
    r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.splitlines() == [name for name, _ in rows]


def test_no_size_runs_a_kernel_without_a_test(exe):
    r = subprocess.run([exe, "2000000"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0
    assert {line.split(",")[0] for line in r.stdout.splitlines()} == set(INSTANCES)
