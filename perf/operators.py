"""Measured cases of the layer over an 8-bit frozen base and of the adapters' Muon step.

Six operators, each through the package's public entry points (``own`` true) or
in elementary torch operations in 32 bits (``own`` false):

  quantize       blocks of 128 held in e4m3 with a power-of-two scale: a row's
                 1 x 128 (activations) or a weight's 128 x 128
  product        Y = Xq·Wq with a scale for each block of 128, and the same
                 weight read the other way (dX = dYq·Wq^T)
  forward        Y[t] = X[t]·W + s_a·((D ⊙ X)[t]·A_a)·B_a over an 8-bit W
  backward       dX, dA, dB of a mixed batch over an 8-bit W
  step           one Muon step of a pool of adapter factors
  orthogonalize  the Newton-Schulz products alone

Layouts: W [d_in, d_out] with scales [ceil(d_in/128), ceil(d_out/128)];
activations [T, d] with scales [ceil(d/128), T]; adapter a owns rows off_a ..
off_a + r_a - 1 of the pools [R, d_in] and [R, d_out].
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128
NS = (3.4445, -4.7750, 2.0315)  # the quintic's coefficients; five products of it
EPS = 1e-7
DEV = "cuda"
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # activations of a prefill batch on the way into the down projection's gradient
        dict(name="quantize rows", op="quantize", what="rows", T=8192, d=11008),
        # an up projection's weight, quantised once when the base is loaded
        dict(name="quantize weight", op="quantize", what="weight", T=4096, d=11008),
        # one token through one projection while serving: latency and the weight's bytes
        dict(name="product 1 token", op="product", T=1, d_in=4096, d_out=4096, transpose=False),
        # the input gradient of a ragged fine-tuning batch
        dict(name="product dX ragged", op="product", T=5003, d_in=4096, d_out=11008, transpose=True),
        # a decode batch: every token its own adapter
        dict(name="forward decode", op="forward", T=256, d_in=4096, d_out=4096, adapters=64, ranks="16-16",
             ids="uniform", p=0.0),
        # prefill requests of 512 tokens, mixed ranks, the up projection
        dict(name="forward prefill", op="forward", T=8192, d_in=4096, d_out=11008, adapters=200, ranks="8,16,32,64",
             ids="request", p=0.0),
        # the smallest training batch: four adapters on a small layer
        dict(name="backward tiny", op="backward", T=64, d_in=256, d_out=256, adapters=4, ranks="4,8,8,16",
             ids="uniform", p=0.1),
        # a fleet's fine-tuning step: a thousand adapters of ranks 1 to 21, dropout
        dict(name="backward fleet", op="backward", T=4096, d_in=4096, d_out=4096, adapters=1000, ranks="1-21",
             ids="zipf", p=0.1),
        # the optimiser's smallest call: the four adapters of the small layer
        dict(name="step tiny", op="step", d=256, adapters=4, ranks="4,8,8,16"),
        # every adapter of the fleet stepped at once
        dict(name="step fleet", op="step", d=4096, adapters=1000, ranks="1-21"),
        # common ranks of trained adapters
        dict(name="orthogonalize mixed", op="orthogonalize", d=4096, adapters=50, ranks="8,16,32,64"),
        # the largest rank an adapter may have
        dict(name="orthogonalize rank 256", op="orthogonalize", d=4096, adapters=6, ranks="256-256"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "forward", "backward", "step", "orthogonalize"))
    if op == "quantize":
        what = rng.choice(("rows", "weight"))
        c = dict(op=op, what=what, T=_log(rng, 1, 16384, 16 if what == "weight" else 1), d=_log(rng, 64, 12288, 16))
        c["T"] = max(16, c["T"]) if what == "weight" else c["T"]
        return c
    ranks = rng.choice(("16-16", "8,16,32,64", "1-21", "3-40"))
    if op in ("step", "orthogonalize"):
        ranks = rng.choice((ranks, "1-64", "100-256")) if op == "orthogonalize" else ranks
        n = _log(rng, 1, 12) if ranks == "100-256" else _log(rng, 1, 150)
        return dict(op=op, d=_log(rng, 64, 8192, 8), adapters=n, ranks=ranks)
    # tokens mostly below a thousand (serving), up to a long training batch
    c = dict(op=op, T=_log(rng, 1, 8192), d_in=_log(rng, 128, 4864, 16), d_out=_log(rng, 128, 11008, 16))
    if op == "product":
        return dict(c, transpose=rng.random() < 0.4)
    c.update(adapters=_log(rng, 1, 300), ranks=ranks, ids=rng.choice(("uniform", "zipf", "request")),
             p=rng.choice((0.0, 0.1)))
    return c


def _ranks_ids(case, seed):
    """The adapters' ranks, the same for every seed, and, where the case has tokens, each token's adapter."""
    r = np.random.default_rng(case["adapters"])
    n, text = case["adapters"], case["ranks"]
    if "-" in text:
        lo, hi = (int(v) for v in text.split("-"))
        ranks = r.integers(lo, hi + 1, size=n)
    else:
        choice = np.array([int(v) for v in text.split(",")])
        ranks = np.resize(choice, n) if n == len(choice) else r.choice(choice, size=n)
    ids = None
    if "T" in case:
        r = np.random.default_rng(seed)
        T, kind = case["T"], case["ids"]
        p = np.arange(1, n + 1) ** (-1.2 if kind == "zipf" else -1.0)
        p /= p.sum()
        if kind == "uniform":
            ids = r.integers(0, n, size=T)
        elif kind == "zipf":
            ids = r.choice(n, size=T, p=p)
        else:
            ids = np.repeat(r.choice(n, size=-(-T // 512), p=p), 512)[:T]
        ids = ids.astype(np.int32)
        ids[0] = np.argmax(ranks)  # every batch has the largest rank
    return ranks.astype(np.int32), ids


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * std


def _keep_bits(seed, p, T, d):
    """Dropout keep bits [T, ceil(d/32)] of the layer's generator: SplitMix64
    output t·d + i of `seed` is below p·2^64 where element (t, i) is dropped."""
    def shr(z, k):
        return (z >> k) & ((1 << (64 - k)) - 1)

    def i64(v):
        return v - (1 << 64) if v >= 1 << 63 else v

    z = torch.arange(1, T * d + 1, device=DEV) * i64(0x9E3779B97F4A7C15) + seed
    z = (z ^ shr(z, 30)) * i64(0xBF58476D1CE4E5B9)
    z = (z ^ shr(z, 27)) * i64(0x94D049BB133111EB)
    z = z ^ shr(z, 31)
    top = -(1 << 63)  # unsigned order as signed: flip the top bit
    keep = ((z ^ top) >= (int(p * 2.0**64) + top)).view(T, d)
    keep = torch.nn.functional.pad(keep, (0, -d % 32)).view(T, -1, 32).to(torch.int64)
    words = (keep << torch.arange(32, device=DEV)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _weight_fp8(W):
    """A checkpoint's 8-bit weight: the block's largest value on 448, any fp32 scale."""
    s = _block_amax(W) / 448.0
    return (W / _over_blocks(s, *W.shape)).clamp(-448.0, 448.0).to(FP8), s


def prepare(case, seed):
    """Inputs from the seed; where the package runs, its plan, context, outputs and workspace too."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, bf = case["op"], torch.bfloat16
    s = dict(case=case, op=op)
    if op == "quantize":
        T, d = case["T"], case["d"]
        x = _normal(g, T, d, std=d**-0.5 if case["what"] == "weight" else 1.0)
        if case["what"] == "rows":  # a few channels much larger than the rest, as activations have
            x = x * torch.where(torch.rand(d, generator=g, device=DEV) < 0.003, 30.0, 1.0)
        s["X"] = x.to(bf)
        nb = -(-d // BLOCK)
        s["S"] = torch.empty((nb, T) if case["what"] == "rows" else (-(-T // BLOCK), nb), device=DEV)
        s["Q"] = torch.empty(T, d, dtype=FP8, device=DEV)
        return s
    if op in ("step", "orthogonalize"):
        ranks, _ = _ranks_ids(case, seed)
        d, R = case["d"], int(ranks.sum())
        # a factor's gradient falls off over its rows, as a trained update's spectrum does
        fall = torch.tensor(np.concatenate([1.0 / np.arange(1, r + 1) for r in ranks]), dtype=torch.float32, device=DEV)
        s["G"] = _normal(g, R, d, std=1e-3) * fall[:, None]
        s["ranks"] = torch.from_numpy(ranks).to(DEV)
        if op == "step":
            s["m"] = _normal(g, R, d, std=5e-4) * fall[:, None]
            s["w"] = _normal(g, R, d, std=d**-0.5)
            s["hyper"] = dict(lr=2e-3, beta=0.95, weight_decay=0.1, rms=0.2)
            s["m_out"], s["w_out"] = torch.empty_like(s["m"]), torch.empty_like(s["w"])
            s["pool"] = torch.empty(R, d, dtype=bf, device=DEV)
        else:
            s["O"] = torch.empty_like(s["G"])
        if own:
            import lora_adapter_execution_b200 as lora
            s["muon"] = lora.Muon(ranks, d)
        return s
    T, di, do = case["T"], case["d_in"], case["d_out"]
    s["Wq"], s["Sw"] = _weight_fp8(_normal(g, di, do, std=di**-0.5))
    if op == "product":
        k, n = (do, di) if case["transpose"] else (di, do)
        s["Xq"], s["Sx"] = _rows_fp8(_normal(g, T, k).to(bf))
        s["Y"] = torch.empty(T, n, dtype=bf, device=DEV)
        return s
    ranks, ids = _ranks_ids(case, seed)
    R, n = int(ranks.sum()), len(ranks)
    s["ranks"], s["ids"] = torch.from_numpy(ranks).to(DEV), torch.from_numpy(ids).to(DEV)
    s["X"] = _normal(g, T, di).to(bf)
    s["A"] = _normal(g, R, di, std=di**-0.5).to(bf)
    per_row = torch.repeat_interleave(s["ranks"].float(), s["ranks"].long()).rsqrt()
    s["B"] = (_normal(g, R, do) * per_row[:, None]).to(bf)
    s["scale"] = 16.0 / s["ranks"].float()
    s["p"], s["seed"] = case["p"], seed
    s["keep"] = _keep_bits(seed, case["p"], T, di) if case["p"] > 0 else None
    r_max = int(ranks[np.unique(ids)].max())
    if op == "forward":
        s["Y"] = torch.empty(T, do, dtype=bf, device=DEV)
        s["U"] = torch.empty(T, r_max, device=DEV)
    else:
        own_rows, rows = _own_rows(s["ranks"], s["ids"], r_max)
        s["U"] = torch.where(own_rows, (_dropped(s) @ s["A"].float().T).gather(1, rows), 0.0)
        s["dY"] = _normal(g, T, do).to(bf)
        s["dX"] = torch.empty(T, di, dtype=bf, device=DEV)
        s["dA"], s["dB"] = torch.zeros(R, di, device=DEV), torch.zeros(R, do, device=DEV)
    if own:
        import lora_adapter_execution_b200 as lora
        s["plan"] = lora.Plan(ids, ranks, di, do)
        need = (lora.fwd_fp8_workspace_size if op == "forward" else lora.bwd_multi_fp8_workspace_size)(s["plan"])
        s["work"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------- plain forms
def _blocks(x, rows):
    """x padded with zeros to whole blocks, as [.., 128] along d (rows) or [.., 128, .., 128]."""
    T, d = x.shape
    x = torch.nn.functional.pad(x, (0, -d % BLOCK, 0, 0 if rows else -T % BLOCK))
    return x.view(T, -1, BLOCK) if rows else x.view(x.shape[0] // BLOCK, BLOCK, -1, BLOCK)


def _block_amax(W):
    return _blocks(W.float().abs(), False).amax((1, 3))


def _over_blocks(s, rows, cols):
    return s.repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def _scale_of(amax):
    """The smallest power of two >= amax / 448 (448 = 0.875 · 2^9), >= 2^-126; 1 for zeros."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875)).clamp(min=-126))
    return torch.where(amax > 0, s, 1.0)


def _rows_fp8(X):
    x = X.float()
    s = _scale_of(_blocks(x.abs(), True).amax(2))  # [T, blocks]
    q = x / s.repeat_interleave(BLOCK, 1)[:, : x.shape[1]]
    return q.to(FP8), s.T.contiguous()


def _weight_q(W):
    w = W.float()
    s = _scale_of(_block_amax(w))
    return (w / _over_blocks(s, *w.shape)).to(FP8), s


def _rows_value(Q, S):
    return Q.float() * S.T.repeat_interleave(BLOCK, 1)[:, : Q.shape[1]]


def _weight_value(Q, S):
    return Q.float() * _over_blocks(S, *Q.shape)


def _own_rows(ranks, ids, r_max):
    """Which of the columns 0 .. r_max-1 are ranks of the token's adapter, and their pool rows."""
    off = ranks.cumsum(0) - ranks
    k = torch.arange(r_max, device=ids.device)
    mine = k < ranks[ids.long()][:, None]
    return mine, torch.where(mine, off[ids.long()][:, None] + k, 0)


def _row_adapter(ranks):
    return torch.repeat_interleave(torch.arange(len(ranks), device=ranks.device), ranks.long())


def _keep(s):
    """The kept elements' factor, 0 or 1/(1-p), [T, d_in]."""
    T, d = s["X"].shape
    bits = (s["keep"].long()[:, :, None] >> torch.arange(32, device=DEV)) & 1
    return bits.view(T, -1)[:, :d].float() / (1.0 - s["p"])


def _dropped(s):
    return s["X"].float() * _keep(s) if s["keep"] is not None else s["X"].float()


def _plain_forward(s):
    Xd, B = _dropped(s), s["B"].float()
    mine = s["ids"].long()[:, None] == _row_adapter(s["ranks"])  # [T, R]: the token's own factor rows
    U = (Xd @ s["A"].float().T) * mine
    Y = _rows_value(*_rows_fp8(s["X"])) @ _weight_value(s["Wq"], s["Sw"])
    Y = Y + (U * s["scale"][s["ids"].long()][:, None]) @ B
    own_rows, rows = _own_rows(s["ranks"], s["ids"], s["U"].shape[1])
    return Y.to(torch.bfloat16), torch.where(own_rows, U.gather(1, rows), 0.0)


def _plain_backward(s):
    dY, sc = s["dY"].float(), s["scale"][s["ids"].long()][:, None]
    mine = s["ids"].long()[:, None] == _row_adapter(s["ranks"])
    dU = (dY @ s["B"].float().T) * mine * sc
    low = dU @ s["A"].float()
    dX = _rows_value(*_rows_fp8(s["dY"])) @ _weight_value(s["Wq"], s["Sw"]).T
    dX = dX + (low * _keep(s) if s["keep"] is not None else low)
    own_rows, rows = _own_rows(s["ranks"], s["ids"], s["U"].shape[1])
    U = torch.zeros_like(dU).scatter_add(1, rows, torch.where(own_rows, s["U"], 0.0))
    return dX.to(torch.bfloat16), dU.T @ _dropped(s), (U * sc).T @ dY


def _quintic(X):
    A = X @ X.transpose(1, 2)
    return NS[0] * X + (NS[1] * A + NS[2] * (A @ A)) @ X


def _plain_orthogonalize(U, ranks):
    """The pool's adapters as one stack padded with rows of zeros, which stay zeros."""
    r_max, R = int(ranks.max()), U.shape[0]
    off = ranks.cumsum(0) - ranks
    k = torch.arange(r_max, device=U.device)
    rows = torch.where(k < ranks[:, None], off[:, None] + k, R)
    X = torch.cat([U, torch.zeros_like(U[:1])])[rows]
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    X = _quintic(_quintic(_quintic(_quintic(_quintic(X)))))
    return X[k < ranks[:, None]]


def _plain_step(s):
    h, ranks, d = s["hyper"], s["ranks"], s["G"].shape[1]
    m = h["beta"] * s["m"] + (1 - h["beta"]) * s["G"]
    O = _plain_orthogonalize((1 - h["beta"]) * s["G"] + h["beta"] * m, ranks)
    gain = h["rms"] * ranks.clamp(min=d).float().sqrt()
    w = (1 - h["lr"] * h["weight_decay"]) * s["w"] - h["lr"] * gain[_row_adapter(ranks)][:, None] * O
    return m, w, w.to(torch.bfloat16)


def run(s):
    """One pass through the case's operator, and its outputs."""
    op = s["op"]
    if own:
        import lora_adapter_execution_b200 as lora
        if op == "quantize":
            (lora.quantize_rows if s["case"]["what"] == "rows" else lora.quantize_weight)(s["X"], s["Q"], s["S"])
            return s["Q"], s["S"]
        if op == "product":
            lora.base_gemm_fp8(s["Xq"], s["Sx"], s["Wq"], s["Sw"], s["Y"], transpose=s["case"]["transpose"])
            return s["Y"]
        if op == "forward":
            lora.linear_fwd_fp8(s["plan"], s["X"], s["Wq"], s["Sw"], s["A"], s["B"], s["scale"], s["Y"], s["work"],
                                p_drop=s["p"], seed=s["seed"], U_save=s["U"], keep_bits=s["keep"])
            return s["Y"], s["U"]
        if op == "backward":
            lora.linear_bwd_multi_fp8(s["plan"], s["X"], s["Wq"], s["Sw"], s["A"], s["B"], s["scale"], s["U"], s["dY"],
                                      s["dX"], s["dA"], s["dB"], s["work"], p_drop=s["p"], seed=s["seed"],
                                      keep_bits=s["keep"])
            return s["dX"], s["dA"], s["dB"]
        if op == "step":
            s["muon"].step(s["G"], s["m"], s["w"], s["m_out"], s["w_out"], s["pool"], nesterov=True, **s["hyper"])
            return s["m_out"], s["w_out"], s["pool"]
        s["muon"].orthogonalize(s["G"], s["O"])
        return s["O"]
    if op == "quantize":
        return (_rows_fp8 if s["case"]["what"] == "rows" else _weight_q)(s["X"])
    if op == "product":
        W = _weight_value(s["Wq"], s["Sw"])
        return (_rows_value(s["Xq"], s["Sx"]) @ (W.T if s["case"]["transpose"] else W)).to(torch.bfloat16)
    if op == "forward":
        return _plain_forward(s)
    if op == "backward":
        return _plain_backward(s)
    if op == "step":
        return _plain_step(s)
    return _plain_orthogonalize(s["G"], s["ranks"])


# ---------------------------------------------------------------------------- work and 64-bit values
def work(case):
    op = case["op"]
    if op == "quantize":
        T, d = case["T"], case["d"]
        blocks = (T if case["what"] == "rows" else -(-T // BLOCK)) * -(-d // BLOCK)
        return {"bytes": 3 * T * d + 4 * blocks, "flops": 2 * T * d}
    if op in ("step", "orthogonalize"):
        ranks, _ = _ranks_ids(case, 0)
        r, d = ranks.astype(np.float64), case["d"]
        # the Gram matrix (one half of it), the r x r products and the polynomial's application
        flops = (r * (r + 1) * d + 17 * 2 * r**3 + 2 * r * r * d).sum()
        return {"bytes": float(r.sum() * d * (22 if op == "step" else 8)), "flops": float(flops)}
    T, di, do = case["T"], case["d_in"], case["d_out"]
    if op == "product":
        k, n = (do, di) if case["transpose"] else (di, do)
        kb = -(-k // BLOCK)
        return {"bytes": T * k + di * do + 2 * T * n + 4 * kb * (T + -(-n // BLOCK)), "flops": 2 * T * di * do}
    ranks, ids = _ranks_ids(case, 0)
    used, per_token = float(ranks[np.unique(ids)].sum()), float(ranks[ids].sum())
    u_save, keep = 4 * T * int(ranks[np.unique(ids)].max()), (T * di // 8 if case["p"] > 0 else 0)
    pools = 2 * used * (di + do)
    if op == "forward":
        return {"bytes": 2 * T * di + di * do + pools + 2 * T * do + u_save + keep,
                "flops": 2.0 * T * di * do + 2 * per_token * (di + do)}
    return {"bytes": 2 * T * (2 * di + do) + di * do + pools + 2 * pools + u_save + keep,
            "flops": 2.0 * T * di * do + 4 * per_token * (di + do)}


def _e4m3_64(v):
    """The e4m3 value nearest to v (ties to the even one): steps of 2^(e-3), no finer than 2^-9."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0**-6))) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _pow2_scale_64(amax):
    e = torch.ceil(torch.log2(amax.clamp(min=2.0**-140) / 448.0))
    e = torch.where(torch.exp2(e - 1) * 448.0 >= amax, e - 1, e)  # log2 rounded up over a whole number
    e = torch.where(torch.exp2(e) * 448.0 < amax, e + 1, e)
    return torch.where(amax > 0, torch.exp2(e.clamp(min=-126.0)), torch.ones_like(amax))


def _quant_64(x, br):
    """(values on the scale, scales) of blocks of br x 128, column block by column block."""
    T, d = x.shape
    q, cols = torch.empty_like(x), []
    for c in range(0, d, BLOCK):
        a = x[:, c:c + BLOCK].abs().amax(1)
        a = torch.stack([t.amax() for t in a.split(br)]) if br > 1 else a
        s = _pow2_scale_64(a)
        q[:, c:c + BLOCK] = _e4m3_64(x[:, c:c + BLOCK] / s.repeat_interleave(br)[:T, None])
        cols.append(s)
    return q, torch.stack(cols)  # scales [column blocks, row blocks]


def _times_scale_64(q, s, br):
    out = q.double()
    for i in range(s.shape[0]):
        out[:, i * BLOCK:(i + 1) * BLOCK] *= s[i].double().repeat_interleave(br)[: q.shape[0], None]
    return out


def _kept_64(s):
    T, d = s["X"].shape
    x, f = torch.empty(T, d, dtype=torch.float64, device=DEV), 1.0 / (1.0 - s["p"])
    for j in range(d):
        x[:, j] = ((s["keep"][:, j // 32] >> (j % 32)) & 1).double() * f
    return x


def exact(case, seed):
    """run()'s outputs in 64 bits: adapter by adapter, block by block."""
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantize":
        q, sc = _quant_64(s["X"].double(), 1 if case["what"] == "rows" else BLOCK)
        return q, sc if case["what"] == "rows" else sc.T
    if op in ("step", "orthogonalize"):
        G, ranks = s["G"].double(), s["ranks"].tolist()
        out, h = torch.empty_like(G), s.get("hyper")
        b = h["beta"] if h else 0.0
        m = b * s["m"].double() + (1 - b) * G if h else None
        U = (1 - b) * G + b * m if h else G
        at = 0
        for r in ranks:
            X = U[at:at + r]
            X = X / (torch.linalg.norm(X) + EPS)
            for _ in range(5):
                A = X @ X.T
                X = NS[0] * X + (NS[1] * A + NS[2] * A @ A) @ X
            if h:
                gain = h["rms"] * math.sqrt(max(r, case["d"]))
                X = (1 - h["lr"] * h["weight_decay"]) * s["w"][at:at + r].double() - h["lr"] * gain * X
            out[at:at + r] = X
            at += r
        return (m, out, out) if h else out
    W = _times_scale_64(s["Wq"], s["Sw"].T, BLOCK)
    if op == "product":
        X = _times_scale_64(s["Xq"], s["Sx"], 1)
        return X @ (W.T if case["transpose"] else W)
    ranks, ids = s["ranks"].tolist(), s["ids"]
    keep = _kept_64(s) if s["keep"] is not None else None
    X = s["X"].double()
    Xd = X * keep if keep is not None else X
    if op == "forward":
        Y = _times_scale_64(*_quant_64(X, 1), 1) @ W
        U = torch.zeros(s["U"].shape, dtype=torch.float64, device=DEV)
    else:
        dY = s["dY"].double()
        dX = _times_scale_64(*_quant_64(dY, 1), 1) @ W.T
        dA, dB = torch.zeros_like(s["dA"], dtype=torch.float64), torch.zeros_like(s["dB"], dtype=torch.float64)
    at = 0
    for a, r in enumerate(ranks):
        t = (ids == a).nonzero().flatten()
        if len(t):
            A, B, sc = s["A"][at:at + r].double(), s["B"][at:at + r].double(), s["scale"][a].double()
            if op == "forward":
                U[t, :r] = Xd[t] @ A.T
                Y[t] += sc * U[t, :r] @ B
            else:
                dU = sc * dY[t] @ B.T
                low = dU @ A
                dX[t] += low * keep[t] if keep is not None else low
                dA[at:at + r] = dU.T @ Xd[t]
                dB[at:at + r] = sc * s["U"][t, :r].double().T @ dY[t]
        at += r
    return (Y, U) if op == "forward" else (dX, dA, dB)
