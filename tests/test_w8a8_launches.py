"""The host side of the 8-bit calls without a device: libgptq's objects linked
to a runtime that writes launches down (fake_runtime.cpp), so that what each
call would launch, and what two threads do to each other, can be looked at."""
import ctypes
import glob
import os
import re
import shutil
import subprocess
import threading

import pytest

from post_weight_quantization_accumulate_b200 import binding as B
from post_weight_quantization_accumulate_b200 import build as build_mod

HERE = os.path.dirname(os.path.abspath(__file__))
P = ctypes.c_void_p
FAKE = P(1 << 20)      # never dereferenced


def _objects():
    build_mod.build()
    objs = [os.path.join(build_mod.BUILD, os.path.basename(s) + ".o") for s in glob.glob(os.path.join(build_mod.CSRC, "*.cu"))]
    if not all(os.path.exists(o) for o in objs):
        build_mod.build(force=True)
    return objs


@pytest.fixture(scope="module")
def linked(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    cuda = os.path.dirname(os.path.dirname(build_mod.nvcc()))
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I",
                    os.path.join(cuda, "include"), os.path.join(HERE, "fake_runtime.cpp"), *_objects(), "-o", path, "-lpthread"],
                   check=True)
    return path


@pytest.fixture
def lib(linked, tmp_path):
    """A library of its own for each test: what calls remember starts anew."""
    handle = ctypes.CDLL(shutil.copy(linked, tmp_path / "own.so"))
    for name, res, args in B.SIGNATURES:
        fn = getattr(handle, name)
        fn.restype, fn.argtypes = res, args
    return handle


def gemm(lib, M, N, K, ty=0, zeros=True):
    ld = (K + 15) // 16 * 16
    return lib.gptq_w8a8_gemm(FAKE, N, ty, FAKE, ld, FAKE, FAKE, FAKE, ld, FAKE, FAKE if zeros else None, None, M, N, K, None)


def launches(lib):
    """(kernel, its template's arguments, what it was launched with) of each launch so far, which are forgotten."""
    out = []
    name, v = ctypes.create_string_buffer(4096), (ctypes.c_longlong * 7)()
    for i in range(lib.fake_launches()):
        lib.fake_launch(i, name, len(name), v)
        m = re.search(r"(\w+)_kernel<(.*?)>\(", name.value.decode())
        out.append((m[1], m[2], dict(zip(("x", "y", "z", "threads", "smem", "cluster", "early"), v))))
    lib.fake_forget()
    return out


def test_two_threads_that_first_use_a_kernel_at_once(lib):
    """Two products whose launches ask for different shared memory, at once and
    as the first of their kernel: neither takes the other's limit away."""
    big, small = (24, 4096, 4096), (24, 11008, 4096)
    lib.fake_hold(400)
    status = {}
    threads = [threading.Thread(target=lambda s=s: status.__setitem__(s, gemm(lib, *s))) for s in (big, small)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    lib.fake_hold(0)
    assert status == {big: 0, small: 0}
    assert gemm(lib, *big) == 0 and gemm(lib, *small) == 0
    found = launches(lib)
    assert len(found) == 4 and {n for n, _, _ in found} == {"w8a8_split"}
    assert len({a for _, a, _ in found}) == 1 and len({v["smem"] for _, _, v in found}) == 2     # one kernel, two sizes
    assert lib.fake_most_limits() == 1


def test_launches_stay_within_their_limits(lib):
    """Every launch asks for no more shared memory than its kernel's limit, which is
    set to one value, whatever order the sizes come in."""
    sizes = [(M, N, K) for K in (100, 700, 1100, 4096, 11008, 65536) for N in (64, 1000, 4096, 11008) for M in (1, 17, 40, 100, 200, 600, 5000)]
    for M, N, K in sizes + sizes[::-1]:
        for ty in (0, 2):
            assert gemm(lib, M, N, K, ty) == 0, (M, N, K)
    assert lib.fake_launches() == 4 * len(sizes)
    assert lib.fake_most_limits() == 1


# Products (M, N, K) for every kernel: with rings of stages that go round within a
# tile, and pairs of CTAs that take three tiles and more.
PRODUCTS = [(8, 1000, 4096), (5, 7200, 2100), (13, 3000, 5000), (27, 1100, 3500),                      # few tokens
            (24, 11008, 4096), (24, 20000, 2000), (40, 300, 3000), (24, 4096, 4096),                   # 32 a tile; clusters of 3, 1, 8, 4
            (100, 4096, 4096), (60, 4096, 4093), (256, 4096, 4096), (130, 3000, 5000),                 # 64 and 128 a tile
            (200, 4096, 2000), (37, 39990, 1300), (300, 5000, 2000), (150, 20000, 1300),               # pairs, 64 and 128
            (600, 8200, 1100), (1100, 11000, 1000), (2048, 4096, 4096)]                                # and 256


def test_the_listed_products_reach_every_kernel(lib):
    name, compiled, i = ctypes.create_string_buffer(4096), set(), 0
    while lib.fake_kernel(i, name, len(name)):
        m = re.search(r"(w8a8_(?:few|split|pair))_kernel<(.*), float>\(", name.value.decode())
        compiled |= {m.groups()} if m else set()
        i += 1
    reached, laps, turns = set(), set(), set()
    for M, N, K in PRODUCTS:
        assert gemm(lib, M, N, K, 2) == 0
        (kernel, arguments, v), = launches(lib)
        which = (kernel, arguments.rsplit(", ", 1)[0])
        reached.add(which)
        if kernel == "w8a8_few":
            continue
        tokens, blocks = int(which[1]), -(-K // 128)
        if kernel == "w8a8_split":
            stages, blocks = (v["smem"] - 1024) // (128 * (128 + tokens)), blocks // v["cluster"]
        else:
            stages = 192 * 1024 // (128 * (128 + tokens // 2))
            if -(-N // 256) * -(-M // tokens) > 2 * (v["x"] // 2):
                turns.add(which)
        if blocks > stages:
            laps.add(which)
    assert len(compiled) == 10 and reached == compiled
    tiled = {k for k in compiled if k[0] != "w8a8_few"}
    assert laps == tiled and turns == {k for k in compiled if k[0] == "w8a8_pair"}
