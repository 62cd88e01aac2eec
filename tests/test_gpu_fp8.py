"""The 8-bit frozen base on the GPU: the quantiser bit for bit, the block-scaled
product and the layer's forward and backward over it, against 64-bit values.

Tolerances. An output is rounded once to bf16: half a step is 2^-8 of its value
(torch.finfo(bfloat16).eps / 2). Before that, a block's product is summed by the
tensor cores in fp32 (taken as 2^-21 of the sum of its terms' magnitudes: 128
terms in four instructions, each addition good to at least 2^-23) and the KB
blocks are added in fp32 (KB roundings of 2^-24 of the running sum, which the
sum of the magnitudes bounds).
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import lora_adapter_execution_b200 as lora
import oracle
from helpers import check_close, dev_bf16, host_f64
from lora_adapter_execution_b200 import workloads as wl

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


def blocks(d):
    return -(-d // 128)


def ref_scale(amax):
    """The definition, in 64 bits: the smallest power of two s with 448·s >= amax."""
    amax = np.asarray(amax, dtype=np.float64)
    out = np.ones_like(amax)
    for i, a in np.ndenumerate(amax):
        if not np.isfinite(a):
            out[i] = np.nan
        elif a > 0:
            e = -126
            while 448.0 * 2.0**e < a:
                e += 1
            out[i] = 2.0**e
    return out


def ref_e4m3(v):
    """Nearest e4m3 value, ties to even, |v| <= 448."""
    with np.errstate(invalid="ignore", divide="ignore"):
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0**-6))) - 3)
        return np.rint(v / step) * step


def ref_rows(x):
    T, d = x.shape
    q, s = np.empty_like(x), np.empty((blocks(d), T))
    for b in range(blocks(d)):
        c = slice(128 * b, min(128 * b + 128, d))
        s[b] = ref_scale(np.abs(x[:, c]).max(1))
        q[:, c] = ref_e4m3(x[:, c] / s[b][:, None])
    return q, s


def ref_weight(w):
    q, s = np.empty_like(w), np.empty((blocks(w.shape[0]), blocks(w.shape[1])))
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            c = np.s_[128 * i:min(128 * i + 128, w.shape[0]), 128 * j:min(128 * j + 128, w.shape[1])]
            s[i, j] = ref_scale(np.abs(w[c]).max())
            q[c] = ref_e4m3(w[c] / s[i, j])
    return q, s


def rows_value(q, s):
    out = q.copy()
    for b in range(s.shape[0]):
        out[:, 128 * b:128 * b + 128] *= s[b][:, None]
    return out


def weight_value(q, s):
    return q * np.repeat(np.repeat(s, 128, 0)[:q.shape[0]], 128, 1)[:, :q.shape[1]]


def f64(t):
    return t.to(torch.float32).double().cpu().numpy()


def quantize_rows(X):
    T, d = X.shape
    # a guard row behind the values and a guard element behind the scales
    Q = torch.full((T + 1, d), 1.5, device="cuda").to(FP8)
    S = torch.full((blocks(d) * T + 1,), 7.0, device="cuda")
    lora.quantize_rows(X, Q[:T], S[:-1].view(blocks(d), T))
    assert (f64(Q[T:]) == 1.5).all() and float(S[-1]) == 7.0
    return Q[:T], S[:-1].view(blocks(d), T)


@pytest.mark.parametrize("T,d", [(1, 16), (1, 4096), (3, 128), (5, 144), (37, 400), (130, 1008), (257, 4112)])
def test_quantize_rows_bit_for_bit(T, d):
    rng = np.random.default_rng(T * 1000 + d)
    x = rng.standard_normal((T, d)) * np.exp2(rng.integers(-60, 60, size=(T, 1)).astype(np.float64))
    X = torch.from_numpy(x).to(torch.bfloat16).cuda()
    X[T // 2, : min(d, 128)] = 0.0  # a block of zeros
    Q, S = quantize_rows(X)
    q, s = ref_rows(f64(X))
    assert np.array_equal(f64(S), s)
    assert np.array_equal(f64(Q), q)
    assert lora.device_status() == 0


def test_quantize_values_at_the_borders():
    """Ties, the largest value on and just over 448·2^k, subnormal scales' floor, -0, inf and NaN."""
    d = 128
    x = np.zeros((9, d))
    x[0, :8] = [448, 17, 19, 21, -17, 2.0**-10, 3 * 2.0**-10, 2.0**-9]  # ties between e4m3 values
    x[1, :3] = [450, 1, -1]          # bf16 450 > 448: the next power of two
    x[2, :2] = [2.0**-130, 2.0**-133]  # amax below 448·2^-126: the scale's floor
    x[3, :2] = [3.0e38, 1.0]
    x[4, :2] = [-448.0 * 2**10, 448.0]
    x[5, :2] = [-0.0, 0.0]
    x[6, 5] = np.inf
    x[7, 127] = np.nan
    x[8, :2] = [2.0**-126 * 448, 2.0**-126]
    X = torch.from_numpy(x).to(torch.bfloat16).cuda()
    Q, S = quantize_rows(X)
    q, s = ref_rows(f64(X))
    ok = np.r_[0:6, 8]
    assert np.array_equal(f64(S)[:, ok], s[:, ok]) and np.array_equal(f64(Q)[ok], q[ok])
    assert np.isnan(f64(S)[0, 6:8]).all() and np.isnan(f64(Q)[6:8]).all()


@pytest.mark.parametrize("di,do", [(16, 16), (128, 128), (144, 400), (272, 1008), (400, 16)])
def test_quantize_weight_bit_for_bit(di, do):
    rng = np.random.default_rng(di + do)
    w = rng.standard_normal((di, do)) * np.exp2(rng.integers(-3, 3, size=(di, do)).astype(np.float64))
    W = torch.from_numpy(w).to(torch.bfloat16).cuda()
    Q, S = torch.empty(di, do, device="cuda").to(FP8), torch.empty(blocks(di), blocks(do), device="cuda")
    lora.quantize_weight(W, Q, S)
    q, s = ref_weight(f64(W))
    assert np.array_equal(f64(S), s) and np.array_equal(f64(Q), q)


# sizes that take each tile width, the K split (1 to 8 CTAs), ragged tiles and short blocks
SIZES = [(1, 16, 16), (1, 4096, 128), (2, 144, 272), (7, 1040, 400), (64, 256, 256), (129, 272, 1008), (200, 2064, 528),
         (300, 128, 4096), (1000, 400, 4112), (5000, 144, 1040), (2100, 1168, 2576)]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("T,di,do", SIZES)
def test_product_integers_exact(T, di, do, transpose):
    """Small integers on scales of one: every sum is an exact fp32 integer, so the
    result is the one bf16 rounding of the exact product, bit for bit."""
    k, n = (do, di) if transpose else (di, do)
    g = torch.Generator(device="cuda").manual_seed(T + di + do)
    X = torch.randint(-3, 4, (T, k), generator=g, device="cuda").float()
    W = torch.randint(-3, 4, (di, do), generator=g, device="cuda").float()
    Y = torch.full((T + 1, n), 5.0, dtype=torch.bfloat16, device="cuda")
    lora.base_gemm_fp8(X.to(FP8), torch.ones(blocks(k), T, device="cuda"), W.to(FP8),
                       torch.ones(blocks(di), blocks(do), device="cuda"), Y[:T], transpose=transpose)
    assert lora.device_status() == 0
    ref = (X.double() @ (W.T if transpose else W).double()).to(torch.bfloat16)
    assert torch.equal(Y[:T], ref)
    assert (Y[T] == 5.0).all()


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("T,di,do", SIZES)
def test_product_any_scales(T, di, do, transpose):
    k, n = (do, di) if transpose else (di, do)
    g = torch.Generator(device="cuda").manual_seed(T * 7 + di + do)
    Xq = torch.randn(T, k, generator=g, device="cuda").mul(20).clamp(-448, 448).to(FP8)
    Wq = torch.randn(di, do, generator=g, device="cuda").mul(20).clamp(-448, 448).to(FP8)
    Sx = torch.rand(blocks(k), T, generator=g, device="cuda") + 0.01
    Sw = torch.rand(blocks(di), blocks(do), generator=g, device="cuda") - 0.3
    Y = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
    lora.base_gemm_fp8(Xq, Sx, Wq, Sw, Y, transpose=transpose)
    assert lora.device_status() == 0
    X = rows_value(f64(Xq), f64(Sx))
    W = weight_value(f64(Wq), f64(Sw))
    W = W.T if transpose else W
    ref, mag = X @ W, np.abs(X) @ np.abs(W)
    tol = 2.0**-8 * np.abs(ref) + (2.0**-21 + (blocks(k) + 3) * 2.0**-24) * mag
    assert (np.abs(f64(Y) - ref) <= tol).all()


def test_product_runs_the_same_twice_and_in_a_graph():
    T, di, do = 33, 2048, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    Xq = torch.randn(T, di, generator=g, device="cuda").to(FP8)
    Wq = torch.randn(di, do, generator=g, device="cuda").to(FP8)
    Sx, Sw = torch.rand(blocks(di), T, generator=g, device="cuda"), torch.rand(blocks(di), blocks(do), device="cuda")
    Y, Z = (torch.empty(T, do, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lora.base_gemm_fp8(Xq, Sx, Wq, Sw, Y)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        lora.base_gemm_fp8(Xq, Sx, Wq, Sw, Z)
    for _ in range(3):
        Z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, Z)


def test_nan_and_inf_stay_in_their_rows_and_blocks():
    """A NaN in a row of X makes that row NaN; one in W makes its block's columns NaN."""
    T, d = 40, 512
    g = torch.Generator(device="cuda").manual_seed(2)
    X = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn(d, d, generator=g, device="cuda").to(torch.bfloat16)
    X[3, 200] = float("inf")
    W[100, 300] = float("nan")
    Xq, Sx = quantize_rows(X)
    Wq, Sw = torch.empty(d, d, device="cuda").to(FP8), torch.empty(4, 4, device="cuda")
    lora.quantize_weight(W, Wq, Sw)
    Y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    lora.base_gemm_fp8(Xq, Sx, Wq, Sw, Y)
    bad = torch.isnan(Y).cpu().numpy()
    want = np.zeros((T, d), bool)
    want[3] = True
    want[:, 256:384] = True
    assert np.array_equal(bad, want)


# ------------------------------------------------------------------ the layer
def layer(T, di, do, ranks, ids, p, seed=0, with_dy=True):
    n = len(ranks)
    spec = wl.Spec("case", T, di, do, n, ("list", tuple(ranks)), ("uniform",), 2.0, p_drop=p, with_dy=with_dy, seed=seed)
    inp = wl.make_inputs(spec)
    inp.ids[:] = ids
    return inp


def run_layer(inp, use_bits=True, backward=True):
    dev = "cuda"
    plan = lora.Plan(inp.ids, inp.ranks, inp.d_in, inp.d_out)
    X, A, B = dev_bf16(inp.X), dev_bf16(inp.A_pool), dev_bf16(inp.B_pool)
    W = dev_bf16(inp.W)
    Wq, Sw = torch.empty(W.shape, device=dev).to(FP8), torch.empty(blocks(inp.d_in), blocks(inp.d_out), device=dev)
    lora.quantize_weight(W, Wq, Sw)
    scale = torch.from_numpy(inp.scale).to(dev)
    bits = None
    if inp.p_drop > 0 and use_bits:
        bits = torch.empty(inp.T, -(-inp.d_in // 32), dtype=torch.int32, device=dev)
        lora.dropout_keep_bits(inp.mask_seed, inp.p_drop, bits, inp.d_in)
    Y = torch.empty(inp.T, inp.d_out, dtype=torch.bfloat16, device=dev)
    U = torch.empty(inp.T, plan.r_max, device=dev)
    kw = dict(p_drop=inp.p_drop, seed=inp.mask_seed, keep_bits=bits)
    ws = torch.empty(lora.fwd_fp8_workspace_size(plan), dtype=torch.uint8, device=dev)
    lora.linear_fwd_fp8(plan, X, Wq, Sw, A, B, scale, Y, ws, U_save=U, **kw)
    assert lora.device_status() == 0
    out = [Y, U]
    if backward:
        dY = dev_bf16(inp.dY)
        dX = torch.empty(inp.T, inp.d_in, dtype=torch.bfloat16, device=dev)
        dA, dB = torch.zeros(A.shape, device=dev), torch.zeros(B.shape, device=dev)
        ws = torch.empty(lora.bwd_multi_fp8_workspace_size(plan), dtype=torch.uint8, device=dev)
        lora.linear_bwd_multi_fp8(plan, X, Wq, Sw, A, B, scale, U, dY, dX, dA, dB, ws, **kw)
        assert lora.device_status() == 0
        out += [dX, dA, dB]
    plan.destroy()
    return out


def ref_layer(inp):
    b = wl.bf16_bits_to_f32
    X, W, A, B, dY = (b(v).astype(np.float64) for v in (inp.X, inp.W, inp.A_pool, inp.B_pool, inp.dY))
    W = weight_value(*ref_weight(W))
    keep = 1.0
    if inp.p_drop > 0:
        keep = (1 - oracle.mask(inp.mask_seed, inp.p_drop, inp.T, inp.d_in)) / (1 - inp.p_drop)
    Y = rows_value(*ref_rows(X)) @ W
    dX = rows_value(*ref_rows(dY)) @ W.T
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    Xd = X * keep
    for a in range(inp.n_adapters):
        t = np.flatnonzero(inp.ids == a)
        r = slice(int(inp.offsets[a]), int(inp.offsets[a + 1]))
        s = float(inp.scale[a])
        U = Xd[t] @ A[r].T
        Y[t] += s * U @ B[r]
        dU = s * dY[t] @ B[r].T
        low = dU @ A[r]
        dX[t] += low * (keep[t] if inp.p_drop > 0 else 1.0)
        dA[r], dB[r] = dU.T @ Xd[t], s * U.T @ dY[t]
    return Y, dX, dA, dB


LAYERS = [
    # T, d_in, d_out, ranks, ids, p: one token; a single adapter; ranks off 16; many small runs; wide tiles
    (1, 256, 272, [5], lambda T: 0, 0.0),
    (40, 144, 400, [16], lambda T: 0, 0.1),
    (64, 256, 256, [4, 8, 8, 16], lambda T: np.arange(T) % 4, 0.1),
    (200, 400, 272, [1, 21, 64, 33], lambda T: (np.arange(T) // 50) % 4, 0.0),
    (300, 1040, 656, list(range(1, 22)), lambda T: (np.arange(T) * 7) % 21, 0.1),
    (130, 256, 512, [256, 3], lambda T: (np.arange(T) > 100).astype(np.int32), 0.1),
    (2600, 656, 2064, [8, 16, 32], lambda T: (np.arange(T) // 512) % 3, 0.0),
    (2600, 2064, 656, [8, 13, 32], lambda T: (np.arange(T) * 5) % 3, 0.1),
]


@pytest.mark.parametrize("case", range(len(LAYERS)))
def test_layer_forward_and_backward(case):
    T, di, do, ranks, ids, p = LAYERS[case]
    inp = layer(T, di, do, ranks, ids(T), p, seed=case)
    Y, U, dX, dA, dB = run_layer(inp)
    rY, rdX, rdA, rdB = ref_layer(inp)
    check_close(host_f64(Y), rY, "Y")
    check_close(host_f64(dX), rdX, "dX")
    check_close(host_f64(dA), rdA, "dA")
    check_close(host_f64(dB), rdB, "dB")


def test_layer_mask_from_the_generator_equals_the_bits():
    inp = layer(200, 400, 272, [5, 16], np.arange(200) % 2, 0.3, seed=4)
    for a, b in zip(run_layer(inp, True), run_layer(inp, False)):
        assert torch.equal(a, b)


def test_U_to_fp32():
    """U = X·A: products of bf16 are exact in fp32; each MMA's 16 are summed to 2^-21 of
    their magnitudes, and the d_in / 16 partial sums are added in fp32 (2^-24 each)."""
    T, di = 70, 1040
    inp = layer(T, di, 128, [16, 40, 5], np.arange(T) % 3, 0.0, seed=5)
    U = f64(run_layer(inp, backward=False)[1])
    X, A = (wl.bf16_bits_to_f32(v).astype(np.float64) for v in (inp.X, inp.A_pool))
    for a in range(3):
        t = np.flatnonzero(inp.ids == a)
        r = slice(int(inp.offsets[a]), int(inp.offsets[a + 1]))
        ref, mag = X[t] @ A[r].T, np.abs(X[t]) @ np.abs(A[r]).T
        assert (np.abs(U[t][:, :inp.ranks[a]] - ref) <= (2.0**-21 + (di / 16 + 4) * 2.0**-24) * mag).all()
        assert (U[t][:, inp.ranks[a]:] == 0).all()


def test_dB_to_fp32():
    """dB = s·U^T·dY from the saved U: U enters as three bf16 parts (24 bits, 2^-24 left
    over), each 16-token step's products are summed in fp32 by one to three MMAs (taken
    as 2^-21 of their magnitudes), the T/16 steps and the segment's pieces are added
    in fp32 (2^-24 of the running sum each) and scaled (one more rounding)."""
    T = 3000
    inp = layer(T, 128, 256, [16, 5], (np.arange(T) % 7 == 0).astype(np.int32), 0.0, seed=6)
    _, U, _, _, dB = run_layer(inp)
    U, dY = f64(U), wl.bf16_bits_to_f32(inp.dY).astype(np.float64)
    for a in range(2):
        t = np.flatnonzero(inp.ids == a)
        r = slice(int(inp.offsets[a]), int(inp.offsets[a + 1]))
        u, s = U[t][:, :inp.ranks[a]], float(inp.scale[a])
        ref, mag = s * u.T @ dY[t], s * np.abs(u).T @ np.abs(dY[t])
        steps = len(t) / 16 + len(t) / 1024 + 4
        assert (np.abs(f64(dB)[r] - ref) <= (2.0**-21 + steps * 2.0**-24) * mag).all()


def test_gradient_of_the_input_against_differences():
    """dX against central differences of L = sum(Y·G) along random directions, on
    an input and gradient that e4m3 holds exactly: the layer is then linear in X
    between the two points, which e4m3 holds too, and only roundings remain. Y is
    rounded to bf16 (2^-8 of each element), so L is off by at most
    2^-8 · sum |Y||G| at each point, and the difference by twice that over 2h = 2."""
    T, di, do, r = 24, 256, 128, 8
    rng = np.random.default_rng(6)
    dev = "cuda"
    ints = lambda *s, lo=-4, hi=5: torch.from_numpy(rng.integers(lo, hi, size=s).astype(np.float32)).to(dev)
    X, D, G = ints(T, di), ints(T, di, lo=-1, hi=2), ints(T, do)
    X[:, ::128] = 8.0  # every block of every point has the largest value 8 or 9: one scale throughout
    D[:, ::128] = 0.0
    W, A, B = ints(di, do), ints(r, di, lo=-1, hi=2), ints(r, do, lo=-1, hi=2)
    plan = lora.Plan(np.zeros(T, np.int32), np.array([r], np.int32), di, do)
    bf = torch.bfloat16
    Wq, Sw = W.to(FP8), torch.ones(blocks(di), blocks(do), device=dev)
    scale = torch.ones(1, device=dev)
    ws = torch.empty(max(lora.fwd_fp8_workspace_size(plan), lora.bwd_multi_fp8_workspace_size(plan)), dtype=torch.uint8,
                     device=dev)

    def loss(x):
        Y = torch.empty(T, do, dtype=bf, device=dev)
        U = torch.empty(T, r, device=dev)
        lora.linear_fwd_fp8(plan, x.to(bf), Wq, Sw, A.to(bf), B.to(bf), scale, Y, ws, U_save=U)
        return (Y.double() * G.double()).sum().item(), (Y.double() * G.double()).abs().sum().item(), U

    lp, mp, _ = loss(X + D)
    lm, mm, _ = loss(X - D)
    _, _, U = loss(X)
    dX = torch.empty(T, di, dtype=bf, device=dev)
    dA, dB = torch.empty(r, di, device=dev), torch.empty(r, do, device=dev)
    lora.linear_bwd_multi_fp8(plan, X.to(bf), Wq, Sw, A.to(bf), B.to(bf), scale, U, G.to(bf), dX, dA, dB, ws)
    want = (lp - lm) / 2
    got = (dX.double() * D.double()).sum().item()
    tol = 2.0**-8 * ((mp + mm) / 2 + (dX.double() * D.double()).abs().sum().item())
    assert abs(got - want) <= tol
    plan.destroy()


def test_layer_two_streams_two_plans():
    """Two calls at once, each with its own plan and workspace, equal the calls one after the other."""
    inps = [layer(150 + 50 * i, 512, 384, [8, 16], np.arange(150 + 50 * i) % 2, 0.0, seed=7 + i) for i in range(2)]
    alone = [run_layer(i, backward=False) for i in inps]
    streams = [torch.cuda.Stream() for _ in inps]
    got = []
    for s, i in zip(streams, inps):
        with torch.cuda.stream(s):
            got.append(run_layer(i, backward=False))
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_workspace_too_small_and_out_of_place_arguments():
    inp = layer(20, 64, 48, [4], np.zeros(20, np.int32), 0.0)
    plan = lora.Plan(inp.ids, inp.ranks, 64, 48)
    X, A, B = dev_bf16(inp.X), dev_bf16(inp.A_pool), dev_bf16(inp.B_pool)
    Wq, Sw = torch.zeros(64, 48, device="cuda").to(FP8), torch.ones(1, 1, device="cuda")
    Y, sc = torch.empty(20, 48, dtype=torch.bfloat16, device="cuda"), torch.ones(1, device="cuda")
    need = lora.fwd_fp8_workspace_size(plan)
    big = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    for ws in (big[:need - 1], big[16:16 + need]):  # one byte short; not 256-byte aligned
        with pytest.raises(lora.LoraError) as e:
            lora.linear_fwd_fp8(plan, X, Wq, Sw, A, B, sc, Y, ws)
        assert e.value.code == -8
    with pytest.raises(lora.LoraError) as e:
        lora.linear_fwd_fp8(plan, X, Wq, Sw, A, B, sc, Y, big, p_drop=1.0)
    assert e.value.code == -1
    lora.linear_fwd_fp8(plan, X, Wq, Sw, A, B, sc, Y, big[:need])
    assert lora.device_status() == 0
    plan.destroy()


def test_offsets_past_32_bits():
    """Rows whose bytes lie past 2^31 and elements past 2^31: the last rows equal the same rows alone."""
    T, d = 270000, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    tail = torch.randn(300, d, generator=g, device="cuda").to(torch.bfloat16)
    X = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    X[-300:] = tail
    Q, S = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(blocks(d), T, device="cuda")
    lora.quantize_rows(X, Q, S)
    Qt, St = quantize_rows(tail)
    assert torch.equal(Q[-300:], Qt.view(torch.uint8)) and torch.equal(S[:, -300:], St)
    assert (Q[:100] == 0).all() and (S[:, :100] == 1).all()
    del X
    Wq = torch.randn(d, 16, generator=g, device="cuda").to(FP8)
    Sw = torch.ones(blocks(d), 1, device="cuda")
    Y = torch.empty(T, 16, dtype=torch.bfloat16, device="cuda")
    lora.base_gemm_fp8(Q, S, Wq, Sw, Y)
    assert lora.device_status() == 0
    W, Xv = f64(Wq), rows_value(f64(Qt), f64(St))
    ref, mag = Xv @ W, np.abs(Xv) @ np.abs(W)
    assert (np.abs(f64(Y[-300:]) - ref) <= 2.0**-8 * np.abs(ref) + (2.0**-21 + (blocks(d) + 3) * 2.0**-24) * mag).all()
    assert (Y[:100] == 0).all()


def test_fine_tuning_steps_over_an_8_bit_base():
    """The pieces as they are used: quantise the base once; per step the forward, a
    gradient of the output, the backward, a Muon step of both pools in place, the next
    step reading the bf16 pools. The first step's gradients and updates equal the
    formulas' in 64 bits, adapters without tokens stay as they were, and further steps run."""
    T, di, do, ranks = 200, 256, 384, [8, 3, 16, 21]
    rng = np.random.default_rng(8)
    ids = rng.integers(0, 3, size=T).astype(np.int32)  # adapter 3 has no token
    inp = layer(T, di, do, ranks, ids, 0.0, seed=9)
    dev, bf = "cuda", torch.bfloat16
    plan = lora.Plan(ids, ranks, di, do)
    X, W = dev_bf16(inp.X), dev_bf16(inp.W)
    Wq, Sw = torch.empty(di, do, dtype=FP8, device=dev), torch.empty(blocks(di), blocks(do), device=dev)
    lora.quantize_weight(W, Wq, Sw)
    scale = torch.from_numpy(inp.scale).to(dev)
    pools = [dev_bf16(inp.A_pool), dev_bf16(inp.B_pool)]
    masters = [p.float() for p in pools]
    moms = [torch.zeros_like(m) for m in masters]
    muons = [lora.Muon(ranks, di), lora.Muon(ranks, do)]
    active = torch.tensor([1, 1, 1, 0], dtype=torch.int32, device=dev)
    Y, U = torch.empty(T, do, dtype=bf, device=dev), torch.empty(T, plan.r_max, device=dev)
    dX, grads = torch.empty(T, di, dtype=bf, device=dev), [torch.full_like(m, float("nan")) for m in masters]
    ws = torch.empty(max(lora.fwd_fp8_workspace_size(plan), lora.bwd_multi_fp8_workspace_size(plan)), dtype=torch.uint8,
                     device=dev)
    dY = dev_bf16(inp.dY)
    before = [m.clone() for m in masters]
    lr, rms = 0.05, 0.2
    for step in range(3):
        lora.linear_fwd_fp8(plan, X, Wq, Sw, *pools, scale, Y, ws, U_save=U)
        lora.linear_bwd_multi_fp8(plan, X, Wq, Sw, *pools, scale, U, dY, dX, *grads, ws)
        for mu, g, m, w, p in zip(muons, grads, moms, masters, pools):
            mu.step(g, m, w, pool=p, lr=lr, beta=0.0, rms=rms, active=active)
        assert lora.device_status() == 0
        if step == 0:
            rY, rdX, rdA, rdB = ref_layer(inp)
            check_close(host_f64(Y), rY, "Y")
            check_close(host_f64(dX), rdX, "dX")
            for w, b, rg in zip(masters, before, (rdA, rdB)):
                for a in range(3):
                    r = slice(int(inp.offsets[a]), int(inp.offsets[a + 1]))
                    x = rg[r] / np.linalg.norm(rg[r])
                    for _ in range(5):
                        G = x @ x.T
                        x = 3.4445 * x + (-4.7750 * G + 2.0315 * G @ G) @ x
                    want = f64(b)[r] - lr * rms * np.sqrt(max(ranks[a], w.shape[1])) * x
                    check_close(f64(w)[r], want, f"adapter {a}")
    last = slice(int(inp.offsets[3]), int(inp.offsets[4]))
    for w, b, p, m in zip(masters, before, pools, moms):
        assert torch.equal(w[last], b[last]) and torch.equal(p[last], b[last].to(bf)) and (m[last] == 0).all()
        assert torch.isfinite(w).all() and torch.equal(p, w.to(bf)) and not torch.equal(w, b)
    plan.destroy()


@pytest.mark.parametrize("runs", [False, True])  # tokens of an adapter together, or scattered
def test_a_captured_step_replays_as_the_eager_one(runs):
    """Forward, backward and the Muon step of one pool in one graph, replayed over new
    inputs in the same buffers: bit for bit the eager calls' results."""
    T, di, do, ranks = 300, 384, 272, [8, 33, 16, 70]
    rng = np.random.default_rng(12)
    ids = rng.integers(0, 4, size=T).astype(np.int32)
    ids = np.sort(ids) if runs else ids
    inp = layer(T, di, do, ranks, ids, 0.1, seed=13)
    bf, dev = torch.bfloat16, "cuda"
    plan = lora.Plan(ids, ranks, di, do)
    X, A, B, dY = dev_bf16(inp.X), dev_bf16(inp.A_pool), dev_bf16(inp.B_pool), dev_bf16(inp.dY)
    Wq, Sw = torch.empty(di, do, dtype=FP8, device=dev), torch.empty(blocks(di), blocks(do), device=dev)
    lora.quantize_weight(dev_bf16(inp.W), Wq, Sw)
    scale = torch.from_numpy(inp.scale).to(dev)
    mu = lora.Muon(ranks, di)
    mom, master = torch.randn(A.shape, device=dev), A.float()
    ws = torch.empty(max(lora.fwd_fp8_workspace_size(plan), lora.bwd_multi_fp8_workspace_size(plan)), dtype=torch.uint8,
                     device=dev)

    def buffers():
        return [torch.zeros(T, do, dtype=bf, device=dev), torch.zeros(T, plan.r_max, device=dev),
                torch.zeros(T, di, dtype=bf, device=dev), torch.zeros(A.shape, device=dev),
                torch.zeros(B.shape, device=dev), torch.zeros_like(mom), torch.zeros_like(master), torch.zeros_like(A)]

    def step(o):
        Y, U, dX, dA, dB, m2, w2, pool = o
        lora.linear_fwd_fp8(plan, X, Wq, Sw, A, B, scale, Y, ws, U_save=U, p_drop=0.1, seed=5)
        lora.linear_bwd_multi_fp8(plan, X, Wq, Sw, A, B, scale, U, dY, dX, dA, dB, ws, p_drop=0.1, seed=5)
        mu.step(dA, mom, master, m2, w2, pool, lr=0.02)

    eager, captured = buffers(), buffers()
    step(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for k in range(3):
        if k:
            X.mul_(-2)
            dY.mul_(0.5)
            step(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert lora.device_status() == 0
        for e, c in zip(eager, captured):
            assert torch.equal(e, c)
    plan.destroy()


@pytest.mark.parametrize("runs", [False, True])  # tokens of an adapter together, or scattered
def test_keep_bits_of_four_byte_alignment(runs):
    """Keep bits may start at any 4-byte boundary: forward and backward over both bases give
    what they give with the same bits on a 16-byte one."""
    T, di, do, ranks, p, seed = 200, 256, 272, [8, 21], 0.3, 11
    ids = np.arange(T, dtype=np.int32) % 2
    ids = np.sort(ids) if runs else ids
    inp = layer(T, di, do, ranks, ids, p, seed=21)
    dev, bf = "cuda", torch.bfloat16
    plan = lora.Plan(ids, ranks, di, do)
    X, W, A, B, dY = (dev_bf16(v) for v in (inp.X, inp.W, inp.A_pool, inp.B_pool, inp.dY))
    Wq, Sw = torch.empty(di, do, dtype=FP8, device=dev), torch.empty(blocks(di), blocks(do), device=dev)
    lora.quantize_weight(W, Wq, Sw)
    scale = torch.from_numpy(inp.scale).to(dev)
    ws = torch.empty(max(lora.fwd_fp8_workspace_size(plan), lora.bwd_multi_fp8_workspace_size(plan)), dtype=torch.uint8,
                     device=dev)
    room = torch.empty(T * (di // 32) + 4, dtype=torch.int32, device=dev)

    def results(shift):
        bits = room[shift:shift + T * (di // 32)].view(T, di // 32)
        assert bits.data_ptr() % 16 == 4 * shift
        lora.dropout_keep_bits(seed, p, bits, di)
        kw = dict(p_drop=p, seed=seed, keep_bits=bits)
        out = []
        for fwd, bwd, base in ((lora.linear_fwd_fp8, lora.linear_bwd_multi_fp8, (Wq, Sw)),
                               (lora.linear_fwd, lora.linear_bwd_multi, (W,))):
            Y, U = torch.empty(T, do, dtype=bf, device=dev), torch.empty(T, plan.r_max, device=dev)
            dX = torch.empty(T, di, dtype=bf, device=dev)
            dA, dB = torch.zeros(A.shape, device=dev), torch.zeros(B.shape, device=dev)
            fwd(plan, X, *base, A, B, scale, Y, *([ws] if len(base) == 2 else []), U_save=U, **kw)
            bwd(plan, X, *base, A, B, scale, U, dY, dX, dA, dB, ws, **kw)
            assert lora.device_status() == 0
            out += [Y, U, dX, dA, dB]
        return out

    want = results(0)
    for shift in (1, 2, 3):
        for a, b in zip(want, results(shift)):
            assert torch.equal(a, b)
    plan.destroy()


@pytest.mark.parametrize("ex,ew", [(-60, -60), (100, 5), (-126, 100), (120, -140), (-145, 120)])
@pytest.mark.parametrize("T,di,do", [(8, 512, 256), (300, 512, 8192)])  # split K; wide tiles
def test_product_scales_at_the_ends_of_fp32(T, di, do, ex, ew):
    """Scales at either end of fp32's range, subnormal ones among them, whose products are
    normal numbers: as exact as others. A scale's own bits below fp32's are taken from
    the tensor, so subnormal scales are what they are."""
    g = torch.Generator(device="cuda").manual_seed(T + ex)
    Xq = torch.randn(T, di, generator=g, device="cuda").mul(100).clamp(-448, 448).to(FP8)
    Wq = torch.randn(di, do, generator=g, device="cuda").mul(100).clamp(-448, 448).to(FP8)
    wide = lambda *s, e: ((torch.rand(*s, generator=g, device="cuda", dtype=torch.float64) + 1) * 2.0**e).float()
    Sx, Sw = wide(blocks(di), T, e=ex), wide(blocks(di), blocks(do), e=ew)
    Y = torch.empty(T, do, dtype=torch.bfloat16, device="cuda")
    lora.base_gemm_fp8(Xq, Sx, Wq, Sw, Y)
    assert lora.device_status() == 0
    X, W = rows_value(f64(Xq), f64(Sx)), weight_value(f64(Wq), f64(Sw))
    ref, mag = X @ W, np.abs(X) @ np.abs(W)
    tol = 2.0**-8 * np.abs(ref) + (2.0**-21 + (blocks(di) + 3) * 2.0**-24) * mag
    assert (np.abs(f64(Y) - ref) <= tol).all()


class Prepared:
    """A layer's plan, inputs, outputs and workspace, made beforehand, so that run() only queues."""

    def __init__(self, inp):
        dev, bf = "cuda", torch.bfloat16
        self.plan = lora.Plan(inp.ids, inp.ranks, inp.d_in, inp.d_out)
        self.X, W, self.A, self.B, self.dY = (dev_bf16(v) for v in (inp.X, inp.W, inp.A_pool, inp.B_pool, inp.dY))
        self.Wq = torch.empty(W.shape, dtype=FP8, device=dev)
        self.Sw = torch.empty(blocks(inp.d_in), blocks(inp.d_out), device=dev)
        lora.quantize_weight(W, self.Wq, self.Sw)
        self.scale = torch.from_numpy(inp.scale).to(dev)
        self.ws = torch.empty(max(lora.fwd_fp8_workspace_size(self.plan), lora.bwd_multi_fp8_workspace_size(self.plan)),
                              dtype=torch.uint8, device=dev)
        self.kw = dict(p_drop=inp.p_drop, seed=inp.mask_seed)
        self.new_outputs = lambda: [torch.zeros(inp.T, inp.d_out, dtype=bf, device=dev),
                                    torch.zeros(inp.T, self.plan.r_max, device=dev),
                                    torch.zeros(inp.T, inp.d_in, dtype=bf, device=dev),
                                    torch.zeros(self.A.shape, device=dev), torch.zeros(self.B.shape, device=dev)]

    def run(self, out):
        Y, U, dX, dA, dB = out
        base = (self.Wq, self.Sw, self.A, self.B, self.scale)
        lora.linear_fwd_fp8(self.plan, self.X, *base, Y, self.ws, U_save=U, **self.kw)
        lora.linear_bwd_multi_fp8(self.plan, self.X, *base, U, self.dY, dX, dA, dB, self.ws, **self.kw)


def test_layers_overlap_on_two_streams_and_in_a_graph():
    """Forwards and backwards of two layers queued alternately on two streams, and a third
    layer's replayed graph beside them, nothing waited for in between: the serial bits."""
    shapes = [(900, 1024, 768, [8, 16, 70]), (700, 768, 1040, [21, 5]), (64, 2048, 512, [16, 4, 33])]
    layers = [Prepared(layer(T, di, do, r, np.arange(T) % len(r), 0.1, seed=30 + i))
              for i, (T, di, do, r) in enumerate(shapes)]
    want, got = ([l.new_outputs() for l in layers] for _ in range(2))
    for l, o in zip(layers, want):
        l.run(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers[2].run(got[2])
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(10):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                layers[k].run(got[k])
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    assert lora.device_status() == 0
    for w, g in zip(want, got):
        for a, b in zip(w, g):
            assert torch.equal(a, b)
    for l in layers:
        l.plan.destroy()


@pytest.mark.parametrize("case", range(len(LAYERS)))
def test_layer_outputs_to_their_rounding(case):
    """Y and dX element by element. Each is rounded once to bf16 (2^-8). The base term is the
    product's (see above). The adapter term is s·U (or s·dU) times the pool's rows: U is
    summed to (2^-21 + (d/16 + 4)·2^-24) of its terms' magnitudes (see test_U_to_fp32),
    s·U is held as two bf16 parts, each rounded to half a step (2^-8 · 2^-8 = 2^-16 left
    over), and its products are summed by MMAs in fp32, 16 ranks an MMA (2^-21 of the
    magnitudes each time, ranks to 256 in two parts: 32 of them at most, 2^-16)."""
    T, di, do, ranks, ids, p = LAYERS[case]
    inp = layer(T, di, do, ranks, ids(T), p, seed=case)
    Y, _, dX, _, _ = run_layer(inp)
    b = wl.bf16_bits_to_f32
    X, W, A, B, dY = (b(v).astype(np.float64) for v in (inp.X, inp.W, inp.A_pool, inp.B_pool, inp.dY))
    W = weight_value(*ref_weight(W))
    keep = np.ones((T, di))
    if p > 0:
        keep = (1 - oracle.mask(inp.mask_seed, p, T, di)) / (1 - p)
    for got, rows, w, first, second, masked_in in ((Y, X, W, A, B, True), (dX, dY, W.T, B, A, False)):
        k = rows.shape[1]
        xq = rows_value(*ref_rows(rows))
        ref, tol = xq @ w, (2.0**-21 + (blocks(k) + 3) * 2.0**-24) * (np.abs(xq) @ np.abs(w))
        for a in range(inp.n_adapters):
            t = np.flatnonzero(inp.ids == a)
            r, sc = slice(int(inp.offsets[a]), int(inp.offsets[a + 1])), float(inp.scale[a])
            x = rows[t] * keep[t] if masked_in else rows[t]
            m = 1.0 if masked_in else keep[t]
            u, mag = sc * x @ first[r].T, sc * np.abs(x) @ np.abs(first[r]).T
            ref[t] += m * (u @ second[r])
            tol[t] += m * ((2.0**-16 + 2.0**-16) * np.abs(u) @ np.abs(second[r])
                           + (2.0**-21 + (k / 16 + 4) * 2.0**-24) * mag @ np.abs(second[r]))
        tol += 2.0**-8 * (np.abs(ref) + tol)
        assert (np.abs(f64(got) - ref) <= tol).all(), (np.abs(f64(got) - ref) / tol).max()
