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


def built_plan(lib, T=64, d_in=256, d_out=128, ranks=(4, 8)):
    """A plan whose tokens are scattered over its adapters (so rows are gathered)."""
    ids, ranks = np.arange(T, dtype=np.int32) % len(ranks), np.array(ranks, np.int32)
    plan = vp()
    assert lib.lora_plan_build(ids.ctypes.data_as(vp), ctypes.c_int64(T), ranks.ctypes.data_as(vp), len(ranks),
                               ctypes.c_int64(d_in), ctypes.c_int64(d_out), None, ctypes.byref(plan)) == 0
    lib.fake_clear()
    return plan


def launches(lib):
    return [(lib.fake_launch_name(i).decode(), [lib.fake_launch_arg(i, k) for k in range(lib.fake_launch_args(i))])
            for i in range(lib.fake_launches())]


P = vp(0x10000)  # stands for an aligned device array: nothing reads it
BIG = ctypes.c_size_t(1 << 30)


def backward(lib, plan, eight_bit, keep_bits):
    zero = ctypes.c_uint64(5)
    base = (P, P) if eight_bit else (P,)
    fn = lib.lora_linear_bwd_multi_fp8 if eight_bit else lib.lora_linear_bwd_multi
    return fn(plan, P, *base, P, P, P, ctypes.c_double(0.1), zero, P, P, P, P, P, P, BIG, keep_bits, None)


@pytest.mark.parametrize("eight_bit", [False, True])
def test_keep_bits_of_four_byte_alignment(lib, eight_bit):
    """Keep bits need 4-byte alignment only: the kernels that gather rows in pieces of 16
    bytes get no other address."""
    plan = built_plan(lib)
    for bits in (0x20000, 0x20004, 0x20008):
        lib.fake_clear()
        assert backward(lib, plan, eight_bit, vp(bits)) == 0
        gathers = [a for n, a in launches(lib) if "lora_gather_" in n and a]
        assert gathers
        sources = [a[5] if len(a) == 6 else a[0] for a in gathers]
        assert all(s % 16 == 0 for s in sources), (hex(bits), sources)
        assert (bits in sources) == (bits % 16 == 0)
    lib.lora_plan_destroy(plan)


def test_a_short_register_count_refuses_the_8_bit_product_alone(lib):
    """A build whose 8-bit product got too few registers for its split (it would wait for
    them for ever) refuses the calls that launch that product, before any launch, and
    no other."""
    lib.fake_set_regs(160)
    n = ctypes.c_int64
    assert lib.lora_base_gemm(P, P, P, n(64), n(256), n(128), None) == 0
    assert lib.lora_fp8_quantize_rows(P, n(64), n(256), P, P, None) == 0
    assert lib.lora_fp8_quantize_weight(P, n(256), n(128), P, P, None) == 0
    ranks = np.array([4, 70, 16], np.int32)
    mu = vp()
    assert lib.lora_muon_create(ranks.ctypes.data_as(vp), 3, n(512), ctypes.byref(mu)) == 0
    assert lib.lora_muon_orthogonalize(mu, P, vp(0x1000000), None, None) == 0
    lib.lora_muon_destroy(mu)
    plan = built_plan(lib)
    assert backward(lib, plan, False, None) == 0
    lib.fake_clear()
    CUDA = -4
    assert lib.lora_base_gemm_fp8(P, P, P, P, P, n(64), n(256), n(128), 0, None) == CUDA
    assert lib.lora_linear_fwd_fp8(plan, P, P, P, P, P, P, ctypes.c_double(0.0), ctypes.c_uint64(0), P, P, P, BIG, None,
                                   None) == CUDA
    assert backward(lib, plan, True, None) == CUDA
    assert launches(lib) == []
    lib.lora_plan_destroy(plan)


def test_enough_registers_launch_the_8_bit_product(lib):
    n = ctypes.c_int64
    assert lib.lora_base_gemm_fp8(P, P, P, P, P, n(64), n(256), n(128), 0, None) == 0
    assert [name for name, _ in launches(lib) if "lora_fp8_gemm_kernel" in name]
