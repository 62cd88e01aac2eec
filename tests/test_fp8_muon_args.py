"""What the 8-bit base's and the Muon step's entry points refuse, without a GPU: every
check runs on the host before any CUDA call (the pointers are never read)."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import lora_adapter_execution_b200 as lora
from lora_adapter_execution_b200 import abi

vp = ctypes.c_void_p
P, ODD = vp(0x1000), vp(0x1004)  # 16-byte aligned; not
ARG, RANK, WORKSPACE = -1, -3, -8


def host_plan(ids, ranks, d_in, d_out):
    L = abi.load_library()
    ids, ranks = np.ascontiguousarray(ids, np.int32), np.ascontiguousarray(ranks, np.int32)
    h = vp()
    assert L.lora_plan_build_host(ids.ctypes.data_as(vp), len(ids), ranks.ctypes.data_as(vp), len(ranks), d_in, d_out,
                                  ctypes.byref(h)) == 0
    return h


@pytest.mark.parametrize("args", [
    (None, 4, 64, P, P), (P, 4, 64, None, P), (P, 4, 64, P, None),   # null
    (P, 0, 64, P, P), (P, -1, 64, P, P), (P, 1 << 31, 64, P, P),     # rows
    (P, 4, 8, P, P), (P, 4, 72, P, P), (P, 4, 0, P, P), (P, 4, -16, P, P),  # width: a multiple of 16
    (ODD, 4, 64, P, P), (P, 4, 64, ODD, P), (P, 4, 64, P, vp(0x1002))])
def test_quantize_refuses(args):
    L = abi.load_library()
    assert L.lora_fp8_quantize_rows(*args, None) == ARG
    X, T, d, Q, S = args
    if T in (4, 0, -1):  # the weight's first extent has the width's rules
        assert L.lora_fp8_quantize_weight(X, d if T == 4 else T, 64, Q, S, None) == ARG


@pytest.mark.parametrize("change", [
    dict(Xq=None), dict(Sx=None), dict(Wq=None), dict(Sw=None), dict(Y=None), dict(Xq=ODD), dict(Wq=ODD), dict(Y=ODD),
    dict(Sx=vp(0x1001)), dict(Sw=vp(0x1002)), dict(T=0), dict(T=-5), dict(d_in=24), dict(d_out=40), dict(d_in=0),
    dict(transpose=2), dict(transpose=-1)])
def test_product_refuses(change):
    a = dict(Xq=P, Sx=P, Wq=P, Sw=P, Y=P, T=4, d_in=64, d_out=64, transpose=0, stream=None)
    a.update(change)
    assert abi.load_library().lora_base_gemm_fp8(*a.values()) == ARG


def test_layer_refuses():
    L = abi.load_library()
    h = host_plan([0, 1, 0], [4, 8], 64, 48)
    fwd = [h, P, P, P, P, P, P, 0.0, 0, P, None, P, 1 << 30, None, None]
    assert L.lora_linear_fwd_fp8(*fwd) == ARG  # a host-only plan
    assert L.lora_linear_fwd_fp8(None, *fwd[1:]) == ARG
    assert L.lora_linear_fwd_fp8_workspace_size(None) == 0
    need = L.lora_linear_fwd_fp8_workspace_size(h)
    assert need >= 3 * 64 + 4 * 3
    assert L.lora_linear_bwd_multi_fp8_workspace_size(h) > L.lora_linear_bwd_multi_workspace_size(h) > 0
    bwd = [h, P, P, P, P, P, P, 0.0, 0, P, P, P, P, P, P, 1 << 30, None, None]
    assert L.lora_linear_bwd_multi_fp8(*bwd) == ARG
    assert L.lora_linear_bwd_multi_fp8(None, *bwd[1:]) == ARG
    L.lora_plan_destroy(h)
    # widths that the bf16 layer takes and the 8-bit one does not
    h = host_plan([0], [4], 72, 48)
    assert L.lora_linear_fwd_fp8_workspace_size(h) == 0 and L.lora_linear_bwd_multi_fp8_workspace_size(h) == 0
    assert L.lora_linear_fwd_fp8(h, *fwd[1:]) == ARG and L.lora_linear_bwd_multi_fp8(h, *bwd[1:]) == ARG
    L.lora_plan_destroy(h)


def test_muon_create_refuses():
    L = abi.load_library()
    out = vp()

    def create(ranks, d):
        r = np.ascontiguousarray(ranks, np.int32)
        return L.lora_muon_create(r.ctypes.data_as(vp), len(r), d, ctypes.byref(out))

    assert create([], 64) == ARG
    for d in (0, 4, 12, -8):
        assert create([4], d) == ARG
    for r in ([0], [257], [4, -1]):
        assert create(r, 64) == RANK
    assert L.lora_muon_create(None, 1, 64, ctypes.byref(out)) == ARG
    r = np.array([4], np.int32)
    assert L.lora_muon_create(r.ctypes.data_as(vp), 1, 64, None) == ARG
    L.lora_muon_destroy(None)  # ignored


def test_muon_calls_refuse_a_null_context():
    L = abi.load_library()
    assert L.lora_muon_orthogonalize(None, P, P, None, None) == ARG
    assert L.lora_muon_step(None, P, P, P, P, P, P, 0.1, 0.9, 1, 0.0, 0.2, None, None) == ARG


def test_binding_names_what_is_wrong():
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    X, Q, S = torch.zeros(4, 256, dtype=bf), torch.zeros(4, 256).to(f8), torch.zeros(2, 4)

    def says(text, fn, *a, **k):
        with pytest.raises(lora.LoraError, match=text) as e:
            fn(*a, **k)
        assert e.value.code == ARG

    says("S has shape", lora.quantize_rows, X, Q, torch.zeros(4, 2))
    says("Q has dtype", lora.quantize_rows, X, Q.float(), S)
    says("X is not contiguous", lora.quantize_rows, torch.zeros(256, 4, dtype=bf).t(), Q, S)
    says("X must be a 2-D tensor", lora.quantize_rows, X[0], Q, S)
    says("X is not a CUDA tensor", lora.quantize_rows, X, Q, S)
    says("S has shape", lora.quantize_weight, X, Q, S)
    W, Sw, Y = torch.zeros(256, 128).to(f8), torch.zeros(2, 1), torch.zeros(4, 128, dtype=bf)
    says("Xq is not a CUDA tensor", lora.base_gemm_fp8, Q, S, W, Sw, Y)
    says("Xq has shape", lora.base_gemm_fp8, Q, S, W, Sw, Y, transpose=True)
    says("Y has shape", lora.base_gemm_fp8, Q, S, W, Sw, Y.t().contiguous())
    says("Sw has shape", lora.base_gemm_fp8, Q, S, W, Sw.t().contiguous(), Y)
    plan = lora.Plan(np.zeros(4, np.int32), np.array([8], np.int32), 256, 128, host_only=True)
    A, B, sc = torch.zeros(8, 256, dtype=bf), torch.zeros(8, 128, dtype=bf), torch.ones(1)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    says("Wq has dtype", lora.linear_fwd_fp8, plan, X, W.float(), Sw, A, B, sc, Y, ws)
    says("A_pool has shape", lora.linear_fwd_fp8, plan, X, W, Sw, A[:4], B, sc, Y, ws)
    says("U_save is required", lora.linear_bwd_multi_fp8, plan, X, W, Sw, A, B, sc, None, Y, X, A.float(), B.float(), ws)
    says("dB_pool has dtype", lora.linear_bwd_multi_fp8, plan, X, W, Sw, A, B, sc, torch.zeros(4, 8), Y, X, A.float(), B,
         ws)
    plan.destroy()
