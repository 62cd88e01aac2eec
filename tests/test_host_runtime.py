"""The library's host code against a CUDA runtime without a device (fake_cudart.cpp):
what it waits for, what it refuses and which pointers it hands to which kernel."""

from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from lora_adapter_execution_b200 import build as cuda_build

vp = ctypes.c_void_p
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def linked(tmp_path_factory):
    """The library's objects linked with the fake runtime."""
    objs = [os.path.join(cuda_build.BUILD_DIR, os.path.basename(s) + ".o") for s in cuda_build.SOURCES]
    if not all(os.path.exists(o) for o in objs):
        cuda_build.build(force=True)
    out = str(tmp_path_factory.mktemp("fake") / "liblora_fake.so")
    inc = os.path.join(os.path.dirname(os.path.dirname(cuda_build.NVCC)), "include")
    # -Bsymbolic: the fake's own symbols, whatever runtime this process has loaded
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I", inc, "-o", out,
                           os.path.join(HERE, "fake_cudart.cpp"), *objs])
    return out


@pytest.fixture
def lib(linked, tmp_path):
    """A fresh copy of it: nothing is initialised yet."""
    path = str(tmp_path / "lib.so")
    shutil.copy(linked, path)
    L = ctypes.CDLL(path)
    L.fake_launch_name.restype = ctypes.c_char_p
    L.fake_launch_arg.restype = ctypes.c_uint64
    return L


def test_muon_create_waits_for_its_tables(lib):
    """lora_muon_create returns once its tables are on the device: the first call may be
    on a stream that does not wait for the default one."""
    ranks = np.array([4, 70, 16], np.int32)
    mu = vp()
    assert lib.lora_muon_create(ranks.ctypes.data_as(vp), 3, ctypes.c_int64(512), ctypes.byref(mu)) == 0
    assert lib.fake_pending() == 0
    lib.lora_muon_destroy(mu)
