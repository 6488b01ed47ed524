"""Which kernels the products' cost model picks, asked of the library on the host
(CPU), and that the shapes of test_gpu_product_plans.py run all of them."""
import math
import random
import subprocess

import pytest

from product_shapes import SHAPES
from test_abi_block_edges import host_program


def plans(exe, calls):
    """The kernels of each (call, dtype, rows, K, N), without how the rows are split."""
    text = "".join("%s %s %d %d %d\n" % c for c in calls)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120, check=True).stdout
    return [{k.replace(",split", "") for k in b.split("\n") if k} for b in out.split("\n\n")[:len(calls)]], out


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return host_program("plans", tmp_path_factory.mktemp("plans"))


def steps_inside(call, dtype, rows, K, N, kernel):
    """The kernel's contractions take more than two steps and end inside one."""
    part = kernel.split()[2]
    step = 64 if dtype == "f16" else 32
    along = {"y": [K], "gx": [N], "gw": [rows], "pair": [N, rows]}[part]
    return all(c > 2 * step and c % step for c in along)


def test_every_kernel_that_is_picked_has_a_shape(program):
    ours = [(*k, *s) for k, shapes in SHAPES.items() for s in shapes]
    run = set()
    kernels, text = plans(program, ours)
    for c, ks in zip(ours, kernels):
        run |= {k for k in ks if steps_inside(*c, k)}
    assert ",split" in text
    r = random.Random(7)
    size = lambda a, b: round(math.exp(r.uniform(math.log(a), math.log(b))))
    calls = []
    for call, dtype in SHAPES:
        for _ in range(20000):
            c = (call, dtype, size(1, 30000), size(1, 512) * 8, size(1, 512) * 8)
            if c[2] * c[3] * c[4] <= 8e10:
                calls.append(c)
    kernels, _ = plans(program, calls)
    missing = {}
    for c, ks in zip(calls, kernels):
        for k in ks - run:
            if steps_inside(*c, k):
                missing.setdefault(k, c)
    assert not missing, f"add to product_shapes.py: {missing}"


def test_the_kernels_are_those_that_there_are(program):
    """All tiles of either type in every place that they are compiled for."""
    ours = [(*k, *s) for k, shapes in SHAPES.items() for s in shapes]
    run = set().union(*plans(program, ours)[0])
    small = ["128x128by1", "128x128by2", "64x64by1", "64x64by2", "64x64by4", "32x32by4", "32x32by8"]
    wide = ["320x256by1", "256x256by1", "192x256by1", "128x256by1"]
    for dtype in ("f16", "f32"):
        for call in ("linear", "gated"):
            for tile in small + ["few"] + (wide if dtype == "f16" else []):
                assert f"{call} {dtype} y {tile}" in run
            for tile in small:
                assert f"{call}_bwd {dtype} pair {tile}" in run and f"{call}_bwd {dtype} gx {tile}" in run
            for tile in wide if dtype == "f16" else []:
                assert f"{call}_bwd {dtype} gx {tile}" in run
