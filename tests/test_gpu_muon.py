"""The Muon step and its orthogonalisation on the GPU against numpy in 64 bits.

Tolerances. O = P·X0 with P exact to 64 bits and rounded once to fp32; a row of O
is a sum over the rank of products P[i, k]·X0[k, :] in fp32, so an element is off
by at most (r + 3) · 2^-24 · sum_k |P[i, k]|·|X0[k, :]| (one rounding of P, of X0's
scale and of u's two terms, one addition per rank), which is what the tests allow,
plus 2^-24 of the result for its own rounding. The update adds 2^-24 of each of its
two terms (three roundings: allowed 2^-22), bf16 copies half a step, 2^-8.
"""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import lora_adapter_execution_b200 as lora

pytestmark = pytest.mark.gpu
A_, B_, C_ = 3.4445, -4.7750, 2.0315
EPS32 = 2.0**-24


def newton_schulz(U):
    X = U / (np.linalg.norm(U) + 1e-7)
    for _ in range(5):
        G = X @ X.T
        X = A_ * X + (B_ * G + C_ * G @ G) @ X
    return X


def polynomial(U):
    """P with O = P·X0."""
    X = U / (np.linalg.norm(U) + 1e-7)
    G, P = X @ X.T, np.eye(len(U))
    for _ in range(5):
        Q = A_ * np.eye(len(U)) + B_ * G + C_ * G @ G
        P, G = P @ Q, Q @ G @ Q
    return P


def bound(U):
    """The allowed error of O, element by element."""
    X = np.abs(U) / (np.linalg.norm(U) + 1e-7)
    return (len(U) + 3) * EPS32 * (np.abs(polynomial(U)) @ X) + EPS32 * np.abs(newton_schulz(U)) + 1e-30


def pools(ranks, d, seed, fall=1.0):
    rng = np.random.default_rng(seed)
    rows = np.concatenate([np.arange(1, r + 1.0) ** -fall for r in ranks])
    make = lambda std: torch.from_numpy((rng.standard_normal((len(rows), d)) * rows[:, None] * std).astype(np.float32)).cuda()
    return make


def f64(t):
    return t.double().cpu().numpy()


def segments(ranks):
    at = 0
    for a, r in enumerate(ranks):
        yield a, slice(at, at + r)
        at += r


CASES = [([1], 8), ([1, 2, 3], 16), ([4, 8, 8, 16], 256), ([17, 33, 5], 200), ([64], 1000), ([32, 64, 48], 4104),
         ([65, 1, 128], 520), ([256], 64), ([200, 7, 256], 1032), (list(range(1, 22)) * 3, 264), ([16], 20000)]


@pytest.mark.parametrize("ranks,d", CASES)
def test_orthogonalize(ranks, d):
    U = pools(ranks, d, seed=len(ranks) * 1000 + d)(1e-3)
    O = torch.full((U.shape[0] + 1, d), 3.0, device="cuda")
    mu = lora.Muon(ranks, d)
    mu.orthogonalize(U, O[:-1])
    assert lora.device_status() == 0
    assert (O[-1] == 3.0).all()
    got, u = f64(O[:-1]), f64(U)
    for _, s in segments(ranks):
        ref = newton_schulz(u[s])
        assert (np.abs(got[s] - ref) <= bound(u[s])).all(), (ranks, d, np.abs(got[s] - ref).max())
    mu.destroy()


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("ranks,d", CASES)
def test_step(ranks, d, nesterov):
    make = pools(ranks, d, seed=d + len(ranks))
    g, m, w = make(1e-2), make(3e-3), make(0.5)
    mo, wo = torch.empty_like(m), torch.empty_like(w)
    pool = torch.empty(w.shape, dtype=torch.bfloat16, device="cuda")
    lr, beta, wd, rms = 0.02, 0.9, 0.1, 0.2
    mu = lora.Muon(ranks, d)
    mu.step(g, m, w, mo, wo, pool, lr=lr, beta=beta, nesterov=nesterov, weight_decay=wd, rms=rms)
    assert lora.device_status() == 0
    G, M, W = f64(g), f64(m), f64(w)
    m2 = beta * M + (1 - beta) * G
    assert (np.abs(f64(mo) - m2) <= 3 * EPS32 * (np.abs(M) + np.abs(G))).all()
    u = (1 - beta) * G + beta * m2 if nesterov else m2
    for _, s in segments(ranks):
        gain = rms * math.sqrt(max(s.stop - s.start, d))
        O = newton_schulz(u[s])
        ref = (1 - lr * wd) * W[s] - lr * gain * O
        tol = lr * gain * update_bound(u[s], [(1 - beta) * G[s], M[s]]) + 2.0**-22 * np.linalg.norm(
            np.abs(W[s]) + lr * gain * np.abs(O))
        assert np.linalg.norm(f64(wo)[s] - ref) <= tol
    assert torch.equal(pool, wo.to(torch.bfloat16))
    # in place, without a bf16 copy
    mu.step(g, m, w, lr=lr, beta=beta, nesterov=nesterov, weight_decay=wd, rms=rms)
    assert torch.equal(m, mo) and torch.equal(w, wo)
    mu.destroy()


def update_bound(u, terms):
    """How far O may be off, in the Frobenius norm, when u = sum of `terms` is itself
    rounded: u is off by at most 3 · 2^-24 of its terms' magnitudes, X0 by twice
    that over |u| (its norm moves too), and five quintic steps, each of slope at
    most 3.4445 on [0, 1.3], stretch a difference by at most 3.4445^5 = 485."""
    return np.linalg.norm(bound(u)) + 485 * 6 * EPS32 * np.linalg.norm(sum(np.abs(t) for t in terms)) / np.linalg.norm(u)


def test_rms_zero_and_lr_zero():
    ranks, d = [3, 8], 64
    make = pools(ranks, d, seed=1)
    g, m, w = make(1e-2), make(1e-3), make(1.0)
    mo, wo, wo0 = torch.empty_like(m), torch.empty_like(w), torch.empty_like(w)
    mu = lora.Muon(ranks, d)
    mu.step(g, m, w, mo, wo, lr=0.5, rms=0.0, beta=0.0)
    for _, s in segments(ranks):
        u = f64(g)[s]
        # beta 0: u = g exactly, so the bounds of O hold element by element
        tol = 0.5 * bound(u) + 2.0**-22 * (np.abs(f64(w)[s]) + np.abs(newton_schulz(u)))
        assert (np.abs(f64(wo)[s] - (f64(w)[s] - 0.5 * newton_schulz(u))) <= tol).all()
    mu.step(g, m, w, mo, wo0, lr=0.0)
    assert torch.equal(wo0, w)


def test_singular_values_come_together():
    """What the iteration is for: every singular value above 1/100 of the norm ends in (0.6, 1.3)."""
    U = pools([24], 512, seed=2, fall=0.8)(1.0)
    O = torch.empty_like(U)
    lora.Muon([24], 512).orthogonalize(U, O)
    s = np.linalg.svd(f64(O), compute_uv=False)
    assert s.min() > 0.6 and s.max() < 1.3


@pytest.mark.parametrize("r", [8, 40, 100])
def test_zero_rank_deficient_and_non_finite(r):
    """Zeros stay zeros; equal rows (rank one) are no trouble; a NaN keeps to its adapter."""
    d, ranks = 136, [r] * 5
    U = pools(ranks, d, seed=3)(1.0)
    U[:r] = 0.0
    U[r:2 * r] = U[r:r + 1]
    U[2 * r + r // 2, d // 2] = float("nan")
    U[3 * r, 1] = float("inf")
    O = torch.empty_like(U)
    lora.Muon(ranks, d).orthogonalize(U, O)
    assert (O[:r] == 0).all()
    u = f64(U)[r:2 * r]
    assert (np.abs(f64(O)[r:2 * r] - newton_schulz(u)) <= bound(u)).all()
    assert torch.isnan(O[2 * r:3 * r]).all()
    assert not torch.isfinite(O[3 * r:4 * r]).any()
    u = f64(U)[4 * r:]
    assert (np.abs(f64(O)[4 * r:] - newton_schulz(u)) <= bound(u)).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e6, 1e18])
def test_scales_of_the_update(scale):
    """Far below the norm's floor of 1e-7 and far above one (squares beyond fp32's range)."""
    ranks, d = [5, 20], 96
    U = pools(ranks, d, seed=4)(scale)
    O = torch.empty_like(U)
    lora.Muon(ranks, d).orthogonalize(U, O)
    for _, s in segments(ranks):
        u = f64(U)[s]
        assert (np.abs(f64(O)[s] - newton_schulz(u)) <= bound(u)).all()


def test_adapters_do_not_depend_on_their_neighbours():
    """The same rows give the same bits alone, among others, and with others left out."""
    d = 264
    ranks = [7, 64, 21, 130, 3]
    U = pools(ranks, d, seed=5)(1.0)
    O = torch.empty_like(U)
    lora.Muon(ranks, d).orthogonalize(U, O)
    for a, s in segments(ranks):
        alone = torch.empty_like(U[s])
        lora.Muon([ranks[a]], d).orthogonalize(U[s].clone(), alone)
        assert torch.equal(alone, O[s]), a
    active = torch.tensor([1, 0, 1, 0, 1], dtype=torch.int32, device="cuda")
    some = torch.full_like(U, 9.0)
    lora.Muon(ranks, d).orthogonalize(U, some, active=active)
    for a, s in segments(ranks):
        assert torch.equal(some[s], O[s]) if active[a] else (some[s] == 9.0).all()
    w = torch.ones_like(U)
    m = torch.full_like(U, 0.5)
    pool = torch.full(U.shape, 2.0, dtype=torch.bfloat16, device="cuda")
    lora.Muon(ranks, d).step(U, m, w, pool=pool, lr=0.1, active=active)
    for a, s in segments(ranks):
        same = (m[s] == 0.5).all() and (w[s] == 1.0).all() and (pool[s] == 2.0).all()
        assert bool(same) == (not bool(active[a]))


def test_graph_replays_equal_the_eager_call():
    ranks, d = [16, 5, 70], 512
    U = pools(ranks, d, seed=6)(1.0)
    mu = lora.Muon(ranks, d)
    O, Z = torch.empty_like(U), torch.empty_like(U)
    mu.orthogonalize(U, O)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        mu.orthogonalize(U, Z)
    for _ in range(3):
        Z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, Z)


def test_refuses_overlap():
    ranks, d = [4], 64
    mu = lora.Muon(ranks, d)
    t = [torch.zeros(4, d, device="cuda") for _ in range(5)]
    with pytest.raises(lora.LoraError):
        mu.orthogonalize(t[0], t[0])
    for kw in (dict(momentum_out=t[0]), dict(momentum_out=t[2]), dict(master_out=t[1]), dict(master_out=t[0]),
               dict(momentum_out=t[3], master_out=t[3])):
        with pytest.raises(lora.LoraError):
            mu.step(t[0], t[1], t[2], lr=0.1, **kw)


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: its last adapters equal the same rows alone."""
    d, n = 8192, 16500
    ranks = [16] * n + [70]
    U = torch.zeros(sum(ranks), d, device="cuda")
    assert U.numel() > 2**31
    tail = pools([16, 16, 70], d, seed=9)(1.0)
    U[-102:] = tail
    O = torch.empty_like(U)
    lora.Muon(ranks, d).orthogonalize(U, O)
    assert lora.device_status() == 0
    alone = torch.empty_like(tail)
    lora.Muon([16, 16, 70], d).orthogonalize(tail, alone)
    assert torch.equal(O[-102:], alone)
    assert (O[:1000] == 0).all()


def test_two_contexts_on_two_streams():
    ranks, d = [24, 7, 64, 130], 1024
    Us = [pools(ranks, d, seed=20 + i)(1.0) for i in range(2)]
    mus = [lora.Muon(ranks, d) for _ in Us]
    alone = [torch.empty_like(u) for u in Us]
    for m, u, o in zip(mus, Us, alone):
        m.orthogonalize(u, o)
    torch.cuda.synchronize()
    both = [torch.empty_like(u) for u in Us]
    streams = [torch.cuda.Stream() for _ in Us]
    for _ in range(3):
        for st, m, u, o in zip(streams, mus, Us, both):
            m.orthogonalize(u, o, stream=st)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert torch.equal(a, b)
