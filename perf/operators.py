"""Cases that time the training-step operators: the loss head (softmax cross
entropy over the vocabulary with its gradient) and the 8-bit activation
checkpoints with the backward pass that reads them.

``run`` computes them in their plain form (elementary torch operations in
fp32), or, with ``own`` set, through the package's entry points.
"""

import math
from statistics import NormalDist

import torch

own = False

BLOCK = 64          # elements per NF4 block constant and per activation exponent
IGNORE = -100       # label of a token that does not count

# ------------------------------------------------------------------ cases


def listed():
    return [
        # 8-bit checkpoints: the input of a 512-wide linear at 64 tokens (latency),
        # and the input of a layer's down projection at a full training batch
        {"name": "act8 quantize 64x512", "op": "quantize", "M": 64, "K": 512},
        {"name": "act8 quantize 16384x11008", "op": "quantize", "M": 16384, "K": 11008},
        # the same read back: an odd token count, and a hidden state of the wide model
        {"name": "act8 dequantize 1001x4096", "op": "dequantize", "M": 1001, "K": 4096},
        {"name": "act8 dequantize 16384x8192", "op": "dequantize", "M": 16384, "K": 8192},
        # backward through one projection at 4x1024 tokens, from the 8-bit input;
        # and through a gate/up group at a ragged token count
        {"name": "bwd act8 4096x4096 m4096", "op": "bwd", "M": 4096, "N": 4096, "K": 4096, "r": 64, "G": 1},
        {"name": "bwd act8 2x11008x4096 m6001", "op": "bwd", "M": 6001, "N": 22016, "K": 4096, "r": 16, "G": 2},
        # log-probability of a single token, and a validation batch
        {"name": "loss fwd t1 v32000", "op": "fwd", "T": 1, "V": 32000, "D": 4096, "nf4": False},
        {"name": "loss fwd t8192 v32000", "op": "fwd", "T": 8192, "V": 32000, "D": 4096, "nf4": False},
        # gradient of per-token losses (preference losses): an odd vocabulary on a
        # narrow model, and an NF4 head
        {"name": "loss bwd t1000 v50257", "op": "bwd_loss", "T": 1000, "V": 50257, "D": 1024, "nf4": False},
        {"name": "loss bwd t4096 v32000 nf4", "op": "bwd_loss", "T": 4096, "V": 32000, "D": 4096, "nf4": True},
        # loss and gradient in one call: one short sequence, and a full batch over a
        # large vocabulary
        {"name": "loss step t200 v32001 nf4", "op": "step", "T": 200, "V": 32001, "D": 2048, "nf4": True},
        {"name": "loss step t8192 v128000", "op": "step", "T": 8192, "V": 128000, "D": 4096, "nf4": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _multiple(rng, lo, hi, of):
    return max(lo, _log_int(rng, lo, hi) // of * of)


def draw(rng):
    op = rng.choice(["quantize", "dequantize", "bwd", "fwd", "bwd_loss", "step"])
    if op in ("quantize", "dequantize"):
        return {"op": op, "M": _log_int(rng, 1, 16384), "K": _multiple(rng, 64, 11008, 64)}
    if op == "bwd":
        G = rng.choice([1, 1, 2, 3])
        r = rng.choice([16, 32, 48, 64] if G > 1 else [16, 32, 64, 80, 128])
        N = G * _multiple(rng, 128, 8192, 128)
        return {"op": op, "M": _log_int(rng, 1, 8192), "N": N, "K": _multiple(rng, 128, 8192, 64), "r": r, "G": G}
    V, D, nf4 = _log_int(rng, 1000, 128000), _multiple(rng, 256, 8192, 64), rng.random() < 0.4
    while V * D > 128000 * 4096:
        V = V * 3 // 4
    return {"op": op, "T": _log_int(rng, 1, 8192), "V": V, "D": D, "nf4": nf4}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _nf4_random(g, rows, cols):
    """NF4 storage of a [rows, cols] weight of about N(0, 0.02): codes are close
    to uniform by the type's construction, the block constants close to 2.5 sigma."""
    numel = rows * cols
    nb = numel // BLOCK
    codes = torch.randint(0, 256, (numel // 2,), generator=g, device="cuda", dtype=torch.uint8)
    c8 = torch.randint(0x70, 0x7F, (nb,), generator=g, device="cuda", dtype=torch.uint8)
    s2 = torch.rand((nb + 255) // 256, generator=g, device="cuda") * 5e-5 + 1.5e-4
    return {"codes": codes, "c8": c8, "s2": s2, "n": rows, "k": cols}


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("quantize", "dequantize"):
        # activations: unit scale, a few channels an order of magnitude larger
        M, K = case["M"], case["K"]
        chan = 1.0 + 20.0 * (torch.rand(K, generator=g, device="cuda") < 0.01)
        X = (torch.randn(M, K, generator=g, device="cuda") * chan).to(torch.bfloat16)
        if op == "quantize":
            return {"case": case, "X": X}
        codes, exps = _plain_quantize(X)
        return {"case": case, "codes": codes.view(torch.uint8), "exps": exps}
    if op == "bwd":
        M, N, K, r, G = (case[k] for k in ("M", "N", "K", "r", "G"))
        X = _randn(g, M, K)
        A = _randn(g, G * r, K, std=K ** -0.5)
        codes, exps = _plain_quantize(X)
        return {"case": case, "W": _nf4_random(g, N, K), "A": A, "B": _randn(g, N, r, std=0.01),
                "dY": _randn(g, M, N), "U": X.float() @ A.float().t(), "s": 16.0 / r,
                "codes": codes.view(torch.uint8), "exps": exps}
    T, V, D = case["T"], case["V"], case["D"]
    if case["nf4"]:
        head = _nf4_random(g, V, D)
        rows = torch.randint(0, V, (T,), generator=g, device="cuda")
        lean = None
    else:
        head = _randn(g, V, D, std=0.02)
        rows = torch.randint(0, V, (T,), generator=g, device="cuda")
        lean = head[rows].float()
    H = torch.randn(T, D, generator=g, device="cuda")
    if lean is not None:
        # hidden states that lean towards their label: probabilities from 1/V to near 1
        H = H + lean * (15.0 * torch.rand(T, 1, generator=g, device="cuda") / (4e-4 * D))
    H = H.to(torch.bfloat16)
    # a quarter of the tokens (a prompt) does not count
    out = torch.rand(T, generator=g, device="cuda") < 0.25
    out[-1] = False
    labels = torch.where(out, torch.full_like(rows, IGNORE), rows)
    state = {"case": case, "H": H, "head": head, "labels": labels}
    if op == "bwd_loss":
        state["dloss"] = torch.randn(T, generator=g, device="cuda") / T
        state["lse"] = _plain_lse(_plain_logits(state))
    return state


# ------------------------------------------------------------------ plain forms


def _levels(dtype):
    """The 16 NF4 levels: standard-normal quantiles, 8 positive, 7 negative, 0."""
    delta, q = 0.5 * ((1 - 1 / 30) + (1 - 1 / 32)), NormalDist().inv_cdf
    lv = [q(delta + i * (0.5 - delta) / 8) for i in range(8)]
    lv += [-q(delta + i * (0.5 - delta) / 7) for i in range(7)] + [0.0]
    top = max(abs(v) for v in lv)
    return torch.tensor(sorted(v / top for v in lv), dtype=torch.float32, device="cuda").to(dtype)


def _plain_weight(w):
    """The bf16 weight an NF4 storage stands for, as fp32; a bf16 weight as it is."""
    if isinstance(w, torch.Tensor):
        return w.float()
    n = w["n"] * w["k"]
    code = torch.stack((w["codes"] & 15, w["codes"] >> 4), -1).reshape(-1, BLOCK)
    c = w["c8"].view(torch.float8_e4m3fn).float() * w["s2"].repeat_interleave(256)[:n // BLOCK]
    v = _levels(torch.float32)[code.int()] * c[:, None]
    return v.to(torch.bfloat16).float().reshape(w["n"], w["k"])


def _plain_quantize(X):
    """E4M3 codes and one exponent byte per 64: the smallest e with max|x| <= 448 2^e."""
    b = X.float().reshape(X.shape[0], -1, BLOCK)
    top = b.abs().amax(-1)
    mant, ex = torch.frexp(top)          # top = mant 2^ex, mant in [1/2, 1)
    e = torch.where(top > 0, ex - 9 + (mant > 0.875).to(ex.dtype), torch.full_like(ex, -118)).clamp(-118, 120)
    codes = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn)
    return codes.reshape(X.shape), (e + 127).to(torch.uint8)


def _plain_dequantize(codes, exps):
    v = codes.view(torch.float8_e4m3fn).float().reshape(codes.shape[0], -1, BLOCK)
    return torch.ldexp(v, exps.int()[..., None] - 127).reshape(codes.shape)


def _plain_bwd(s):
    c = s["case"]
    G, r, n = c["G"], c["r"], c["N"] // c["G"]
    dY, A, B, U = s["dY"].float(), s["A"].float(), s["B"].float(), s["U"]
    X = _plain_dequantize(s["codes"], s["exps"])
    parts = torch.arange(c["N"], device=dY.device) // n                 # member of an output
    cols = torch.arange(G * r, device=dY.device) // r                   # member of a rank column
    same = (parts[:, None] == cols[None, :]).float()
    Bd = B.repeat(1, G) * same                                          # block diagonal [N, G r]
    dU = s["s"] * (dY @ Bd)
    dX = dY @ _plain_weight(s["W"]) + dU @ A
    full = (s["s"] * (dY.t() @ U)).reshape(c["N"], G, r)
    dB = full.gather(1, parts[:, None, None].expand(-1, 1, r))[:, 0]
    return dX.to(torch.bfloat16), dU.t() @ X, dB.contiguous()


def _plain_logits(s):
    return s["H"].float() @ _plain_weight(s["head"]).t()


def _plain_lse(logits):
    top = logits.amax(-1, keepdim=True)
    return (torch.log(torch.exp(logits - top).sum(-1, dtype=torch.float64)) + top[:, 0].double()).float()


def _plain_loss(s, logits):
    lse = _plain_lse(logits)
    counted = s["labels"] != IGNORE
    at = s["labels"].clamp(min=0)
    loss = torch.where(counted, lse - logits.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    count = counted.sum()
    mean = loss.double().sum() / count.clamp(min=1)
    return loss, lse, torch.stack((mean, count.double())).float()


def _plain_grad(s, logits, lse, g):
    p = torch.exp(logits - lse[:, None])
    at = s["labels"].clamp(min=0)
    p = p.scatter_add(1, at[:, None], torch.full_like(p[:, :1], -1.0))
    g = torch.where(s["labels"] != IGNORE, g, torch.zeros_like(g))
    return ((p @ _plain_weight(s["head"])) * g[:, None]).to(torch.bfloat16)


def _plain(s):
    op = s["case"]["op"]
    if op == "quantize":
        return _plain_quantize(s["X"])
    if op == "dequantize":
        return _plain_dequantize(s["codes"], s["exps"]).to(torch.bfloat16)
    if op == "bwd":
        return _plain_bwd(s)
    logits = _plain_logits(s)
    if op == "fwd":
        return _plain_loss(s, logits)
    if op == "bwd_loss":
        return _plain_grad(s, logits, s["lse"], s["dloss"])
    loss, lse, stats = _plain_loss(s, logits)
    g = (1.0 / stats[1].clamp(min=1)).expand_as(lse)
    return loss, lse, stats, _plain_grad(s, logits, lse, g)


# ------------------------------------------------------------------ the package's calls


def _own_weight(lib, w):
    return w if isinstance(w, torch.Tensor) else lib.NF4Weight(w["codes"], w["c8"], w["s2"], w["n"], w["k"])


def _own(s):
    import bit_nf4_quantized_26_b200 as lib
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        x8 = lib.act8_quantize(s["X"])
        return x8.codes.view(torch.float8_e4m3fn), x8.exps
    if op == "dequantize":
        return lib.act8_dequantize(lib.Act8(s["codes"], s["exps"]))
    if op == "bwd":
        x8, W = lib.Act8(s["codes"], s["exps"]), _own_weight(lib, s["W"])
        if c["G"] == 1:
            return lib.qlora_linear_bwd_act8(s["dY"], x8, s["U"], W, s["A"], s["B"], s["s"])
        return lib.qlora_group_bwd_act8(s["dY"], x8, s["U"], W, [c["N"] // c["G"]] * c["G"], s["A"], s["B"], s["s"])
    head = _own_weight(lib, s["head"])
    if op == "fwd":
        return lib.qlora_head_loss_fwd(s["H"], head, s["labels"])
    if op == "bwd_loss":
        return lib.qlora_head_loss_bwd(s["H"], head, s["labels"], s["lse"], s["dloss"])
    return lib.qlora_head_loss_step(s["H"], head, s["labels"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ floors


def work(case):
    """Each input read once, each output written once; the products the operator
    cannot do without (the gradient of the loss needs the logits and one more
    product of the same size)."""
    op = case["op"]
    if op in ("quantize", "dequantize"):
        n = case["M"] * case["K"]
        return {"bytes": n * (3 + 1 / BLOCK), "flops": 0}
    if op == "bwd":
        M, N, K, r, G = (case[k] for k in ("M", "N", "K", "r", "G"))
        nf4 = N * K * (0.5 + 1 / 64 + 4 / 16384)
        return {"bytes": nf4 + M * N * 2 + M * K * (1 + 1 / BLOCK) + M * K * 2 + G * r * K * (2 + 4) + N * r * (2 + 4)
                + M * G * r * 4,
                "flops": 2 * M * N * K + 4 * M * N * r + 4 * M * G * r * K}
    T, V, D = case["T"], case["V"], case["D"]
    head = V * D * (0.5 + 1 / 64 + 4 / 16384 if case["nf4"] else 2)
    if op == "fwd":
        return {"bytes": head + T * D * 2 + T * 16, "flops": 2 * T * V * D}
    return {"bytes": head + T * D * 4 + T * 16, "flops": 4 * T * V * D}


# ------------------------------------------------------------------ 64 bits


def _exact_weight(w):
    if isinstance(w, torch.Tensor):
        return w.double()
    byte = w["codes"].long()
    code = torch.empty(2 * byte.numel(), dtype=torch.long, device=byte.device)
    code[0::2], code[1::2] = byte % 16, byte // 16
    c8 = w["c8"].long()
    ex, m = c8 // 8, (c8 % 8).double()
    const = torch.where(ex == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(ex.double() - 7))
    block = torch.arange(const.numel(), device=const.device)
    # the storage's own roundings: the constant and the weight once each to fp32, then bf16
    const = (const * w["s2"].double()[block // 256]).float()
    v = (_levels(torch.float64)[code].reshape(-1, BLOCK) * const.double()[:, None]).float()
    return v.to(torch.bfloat16).double().reshape(w["n"], w["k"])


def _exact_values(codes, exps):
    c = codes.long()
    mag, sign = c % 128, 1.0 - 2.0 * (c // 128).double()
    ex, m = mag // 8, (mag % 8).double()
    v = sign * torch.where(ex == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(ex.double() - 7))
    return v * torch.exp2(exps.double() - 127).repeat_interleave(BLOCK, 1)


def _exact_quantize(X):
    x = X.double().reshape(X.shape[0], -1, BLOCK)
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -200)))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e))
    e = e.clamp(-118, 120)
    v = x * torch.exp2(-e)[..., None]
    # E4M3: three mantissa bits, subnormal step 2^-9; ties to even
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).reshape(X.shape), (e + 127).to(torch.uint8)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(s["X"])
    if op == "dequantize":
        return _exact_values(s["codes"], s["exps"])
    if op == "bwd":
        G, r, n = case["G"], case["r"], case["N"] // case["G"]
        dX, dA, dB = 0.0, [], []
        W, X = _exact_weight(s["W"]), _exact_values(s["codes"], s["exps"])
        for k in range(G):
            dY = s["dY"][:, k * n:(k + 1) * n].double()
            A, B = s["A"][k * r:(k + 1) * r].double(), s["B"][k * n:(k + 1) * n].double()
            dU = (dY @ B) * s["s"]
            dX = dX + dY @ W[k * n:(k + 1) * n] + dU @ A
            dA.append(dU.t() @ X)
            dB.append((dY.t() @ s["U"][:, k * r:(k + 1) * r].double()) * s["s"])
        return dX, torch.cat(dA), torch.cat(dB)
    H, W, labels = s["H"].double(), _exact_weight(s["head"]), s["labels"]
    T, counted = case["T"], labels != IGNORE
    count = int(counted.sum())
    lse = torch.empty(T, dtype=torch.float64, device="cuda")
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    dH = torch.zeros_like(H)
    for t in range(0, T, 1024):
        z = H[t:t + 1024] @ W.t()
        c, y = counted[t:t + 1024], labels[t:t + 1024]
        lse[t:t + 1024] = torch.logsumexp(z, 1)
        i = torch.nonzero(c)[:, 0]
        loss[t + i] = lse[t + i] - z[i, y[i]]
        if op == "fwd":
            continue
        z = torch.softmax(z, 1)
        if op == "bwd_loss":  # the definition's lse is the call's input
            z = z * torch.exp(lse[t:t + 1024] - s["lse"][t:t + 1024].double())[:, None]
        z[i, y[i]] -= 1.0
        g = s["dloss"][t:t + 1024].double() if op == "bwd_loss" else torch.full_like(lse[t:t + 1024], 1.0 / max(count, 1))
        dH[t + i] = (z[i] @ W) * g[i, None]
    stats = torch.stack((loss.sum() / max(count, 1), torch.tensor(float(count), dtype=torch.float64, device="cuda")))
    if op == "fwd":
        return loss, lse, stats
    return dH if op == "bwd_loss" else (loss, lse, stats, dH)
