"""Which kernels the sizes of the fused operators' GPU tests reach, on the host: every tile of
the dense products and of the gradients, whole and in parts, with whole words of scales and
without, so that a change of a constant that makes the tests miss one fails here; and that no
kernel is compiled that none of them reaches."""
import itertools
import os
import random
import re
import shutil

import pytest

import dequant_gemv_nf4_amd as nf4
import test_gpu_fused as fused
import test_gpu_fused_edges as edges
from test_sanitizers import CSRC, HERE, _run

# of nf4::mx::dense_tile(): rows, columns, K-groups, in order
DENSE = [(128, 256, 1), (128, 192, 1), (128, 128, 1), (96, 128, 1), (64, 128, 1), (32, 128, 1),
         (32, 64, 1), (32, 64, 2), (16, 64, 1), (16, 64, 2), (16, 32, 4)]
# of nf4::mx::plan_dense(): row fragments, waves, K-groups
GRAD = [(1, 2, 2), (2, 2, 2), (4, 4, 1), (4, 4, 2)]


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("plans")
    exe = str(d / "plans")
    rc, out = _run([cxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-Wall", "-Werror", "-I", CSRC, os.path.join(HERE, "plans_driver.cpp"), "-o", exe])
    assert rc == 0, out

    def ask(kind, sizes):
        rc, out = _run([exe], input="".join(f"{kind} {m} {n} {k}\n" for m, n, k in sizes))
        assert rc == 0, out
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


def cases_of(test):
    """The sizes that a test is parametrised with."""
    return [mark.args[1] for mark in test.pytestmark if mark.name == "parametrize" and mark.args[0] == "m,n,k"][0]


def test_dense_tiles_are_all_tested(plans):
    sizes = fused.TILES + edges.MORE_TILES
    got = {(DENSE[i], k % 128 == 0) for (i,), (_, _, k) in zip(plans("t", sizes), sizes)}
    assert got == set(itertools.product(DENSE, (True, False)))


def test_gradient_tiles_are_all_tested(plans):
    sizes = cases_of(fused.test_grad_shapes) + edges.MORE_GRADIENTS
    got = {((mf, wv, kg), splits > 1, k % 128 == 0)
           for (mf, wv, kg, splits), (_, _, k) in zip(plans("g", sizes), sizes)}
    assert got == set(itertools.product(GRAD, (True, False), (True, False)))


def test_plans_hold_over_the_whole_range(plans):
    """Plans of any size: a tile that there is, parts within their limit and of four stages."""
    rng = random.Random(1)
    sizes = [(1, 8, 32), (1 << 21, 1 << 23, 32), (1 << 21, 65528, 32768), (1, 1 << 23, 256)]
    for _ in range(4000):
        k = 32 * int(2 ** rng.uniform(0, 10))
        n = 8 * int(2 ** rng.uniform(0, 20))
        if n * k // 2 < 1 << 31:
            sizes.append((int(2 ** rng.uniform(0, 21)), n, k))
    tiles, grads = plans("t", sizes), plans("g", sizes)
    assert len(tiles) == len(grads) == len(sizes)
    for (m, n, k), (tile,), (mf, wv, kg, splits) in zip(sizes, tiles, grads):
        assert 0 <= tile < len(DENSE) and (mf, wv, kg) in GRAD and splits >= 1
        if splits > 1:
            assert splits * m * k * 4 <= 1 << 28 and (n + 63) // 64 >= 4 * kg * splits


def kernels(name):
    """The template arguments of every kernel `name` of the library."""
    nm = shutil.which("nm")
    if nm is None or not os.path.exists(nf4.lib_path()):
        pytest.skip("no nm, or no library")
    rc, out = _run([nm, "-C", nf4.lib_path()])
    assert rc == 0, out
    return [tuple(a.strip() for a in m.split(",")) for m in re.findall(rf"__device_stub__{name}<([^>]*)>", out)]


def test_no_gradient_kernel_is_out_of_reach():
    """Sums in parts are compiled for the tiles of plan_dense() and no others."""
    found = {(tuple(map(int, k[:3])), k[3]) for k in kernels("mx_grad_kernel") if k[5] == "true"}
    assert found == set(itertools.product(GRAD, ("true", "false")))
    assert sorted(kernels("mx_act_grad_kernel")) == [("false",), ("true",)]
