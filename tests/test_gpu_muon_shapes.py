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
import test_gpu_muon as base
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


# the one-launch kernel's builds and cluster sizes that other tests leave out: padded rank
# 56; odd numbers of rank blocks (40, 56) whose iteration several CTAs share; rank 64 with
# the most shared memory; ranks of 9 to 48 on eight CTAs
SHAPES = [([49, 53, 56], 4096), ([56], 392), ([33, 40], 2056), ([57, 64], 4096), ([41, 48, 37], 4096), ([9, 24, 31], 4096),
          ([1, 8], 16384)]


@pytest.mark.parametrize("ranks,d", SHAPES)
def test_orthogonalize(ranks, d):
    base.test_orthogonalize(ranks, d)


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("ranks,d", SHAPES)
def test_step(ranks, d, nesterov):
    base.test_step(ranks, d, nesterov)


@pytest.mark.parametrize("ranks,d", SHAPES + [([70, 200], 1032)])
def test_after_a_call_of_nans(ranks, d):
    """What a call of NaNs leaves in shared memory and scratch does not reach the next one."""
    U = pools(ranks, d, seed=2)(1.0)
    mu = lora.Muon(ranks, d)
    O, clean = torch.empty_like(U), torch.empty_like(U)
    mu.orthogonalize(U, clean)
    for _ in range(3):
        mu.orthogonalize(torch.full_like(U, float("nan")), O)
        assert torch.isnan(O).all()
        mu.orthogonalize(U, O)
        assert torch.equal(O, clean)
    u = f64(U)
    for _, s in segments(ranks):
        assert (np.abs(f64(clean)[s] - newton_schulz(u[s])) <= bound(u[s])).all()


def test_two_contexts_on_two_streams_and_one_in_a_graph():
    """Steps of two contexts queued alternately on two streams, and a third context's
    replayed graph beside them: the serial calls' bits."""
    ranks, d = [24, 7, 64, 130, 53], 2048
    make = pools(ranks, d, seed=3)
    ins = [(make(1e-2), make(1e-3), make(1.0)) for _ in range(3)]
    mus = [lora.Muon(ranks, d) for _ in ins]
    outs = lambda: [[torch.zeros_like(i[0]), torch.zeros_like(i[0])] for i in ins]
    want, got = outs(), outs()
    for mu, i, o in zip(mus, ins, want):
        mu.step(*i, *o, lr=0.1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mus[2].step(*ins[2], *got[2], lr=0.1)
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    for _ in range(8):
        for k in range(2):
            mus[k].step(*ins[k], *got[k], lr=0.1, stream=streams[k])
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    assert lora.device_status() == 0
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])
