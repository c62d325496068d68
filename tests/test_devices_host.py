"""Every call on the second device of one process, without a GPU.

What a kernel is allowed (dynamic shared memory past 48 KB, clusters past eight
CTAs) belongs to a device, so each device has to be given it. The library's host
code runs here on a runtime that keeps that rule for two devices and checks
launches instead of running them (fake_cudart.c); its kernels are compiled to an
intermediate form only, which nothing loads.
"""
import ctypes
import glob
import os
import shutil
import subprocess

import pytest

from conftest import ROOT
from fp8_block_scaled_group_b200 import _lib, build

BUF = ctypes.create_string_buffer(4096)
BASE = (ctypes.addressof(BUF) + 255) // 256 * 256  # aligned; never read: nothing runs
BIG = 1 << 40


def declare(lib):
    for name, (restype, argtypes) in _lib.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = restype, argtypes
    return lib


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    out = tmp_path_factory.mktemp("devices")
    so = str(out / "libfp8q_checked.so")
    cuda = os.path.dirname(os.path.dirname(build.nvcc()))
    subprocess.check_call(["gcc", "-c", "-fPIC", "-O1", "-Wall", "-I", os.path.join(cuda, "include"),
                           os.path.join(ROOT, "tests", "fake_cudart.c"), "-o", str(out / "fake.o")])
    subprocess.check_call([build.nvcc(), "-t", "0", "-gencode", "arch=compute_100a,code=compute_100a", "-std=c++17", "-cudart", "none",
                           "-shared", "-Xcompiler", "-fPIC,-O1", "-Xlinker", "-Bsymbolic", "-I", build.INCLUDE, "-I", build.CSRC, *build.sources(),
                           str(out / "fake.o"), "-o", so])
    return so


@pytest.fixture(scope="module")
def lib(library):
    return declare(ctypes.CDLL(library))


N, K, E = 384, 1152, 8
CALLS = {
    "route of few slots": ("fp8q_moe_route", [BASE] * 4 + [25, 8, E]),
    "route of many slots": ("fp8q_moe_route", [BASE] * 4 + [1000, 8, E]),
    "route of the most slots": ("fp8q_moe_route", [BASE] * 4 + [16384, 8, E]),
    **{f"linear, {m} rows": ("fp8q_linear_ex", [BASE, BASE, BASE, 0, BASE, BASE, BIG, m, N, K]) for m in (1, 32, 33, 64, 65, 1168)},
    **{f"NVFP4 linear, {m} rows": ("fp8q_nvfp4_linear", [BASE, 1.0, BASE, BASE, 1.0, BASE, BASE, BIG, m, N, 1024]) for m in (17, 100, 1168)},
    "fused decode": ("fp8q_linear_decode_fused", [BASE, BASE, BASE, 0, BASE, BASE, BIG, 17, N, K]),
    **{f"grouped, {rows} rows an expert": ("fp8q_grouped_linear", [BASE] * 5 + [0, BASE, BASE, BIG, rows * E, rows * E, E, N, K])
       for rows in (1, 56, 57, 152, 153)},
    **{f"FFN, {t} tokens": ("fp8q_moe_ffn", [BASE] * 7 + [0, BASE, BASE, BIG, t, 2, E, N, 256]) for t in (1, 300, 2000)},
    **{f"adapters of rank {r}, {m} rows": ("fp8q_lora_linear", [BASE, BASE, BASE, 0] + [BASE] * 6 + [BIG, m, N, K, 5, r])
       for m in (1, 32, 33, 64, 65, 256, 257) for r in (8, 256)},
    "adapters, long K": ("fp8q_lora_linear", [BASE, BASE, BASE, 0] + [BASE] * 6 + [BIG, 3, 128, 1563 * 128, 5, 256]),
}


@pytest.mark.parametrize("what", CALLS)
def test_each_device_is_prepared(lib, what):
    name, args = CALLS[what]
    for device in (0, 1):
        lib.fake_set_device(device)
        before, refused = lib.fake_launches(device), lib.fake_refused()
        assert getattr(lib, name)(*args, None) == 0, f"{what} on device {device}"
        assert lib.fake_launches(device) > before and lib.fake_refused() == refused


def test_two_copies_of_the_library_in_one_process(lib, library, tmp_path):
    """A copy that another package brings along has kernels of its own, which it has to prepare itself whatever the first
    one has done: no state of one is the other's."""
    for name, args in CALLS.values():
        assert getattr(lib, name)(*args, None) == 0
    second = str(tmp_path / "libfp8q_second.so")
    shutil.copy(library, second)
    other = declare(ctypes.CDLL(second))
    for what, (name, args) in CALLS.items():
        assert getattr(other, name)(*args, None) == 0, what
    assert other.fake_refused() == 0
