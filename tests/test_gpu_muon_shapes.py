"""The Muon step on the GPU at shapes and on streams of its own: first calls on
non-blocking streams, odd padded ranks over several CTAs, the largest slices. Bounds as
derived in test_gpu_muon.

The factor 485 of its bound on a step is the largest slope of the whole composition of
five quintics on [0, 1]: p'(0)^5 = 3.4445^5, reached at 0. (A single quintic is steeper
elsewhere, 3.96 at 1.20, the largest value an iterate takes, but only behind quintics
that are flat there.)
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import lora_adapter_execution_b200 as lora
from test_gpu_muon import bound, f64, newton_schulz, pools, segments

pytestmark = pytest.mark.gpu


def test_first_call_on_a_non_blocking_stream():
    """A fresh context's first call, on a stream that does not wait for the default one:
    its tables (some megabytes) are on the device when lora_muon_create returns."""
    d, n = 64, 40000
    ranks = [(3, 8, 17, 70)[i % 4] for i in range(n)]
    U = pools(ranks[:8], d, seed=1)(1.0)
    U = U.repeat(n // 8, 1)
    few, O = torch.empty_like(U[:196]), torch.empty_like(U)
    assert U[:196].shape[0] == sum(ranks[:8])
    lora.Muon(ranks[:8], d).orthogonalize(U[:196].clone(), few)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        mu = lora.Muon(ranks, d)
        mu.orthogonalize(U, O, stream=stream)
        torch.cuda.synchronize()
        assert lora.device_status() == 0
        assert torch.equal(O.view(n // 8, -1, d), few.expand(n // 8, -1, -1))
        O.zero_()
        torch.cuda.synchronize()
        mu.destroy()
