"""GPU parity of the 8-bit activation checkpoints: codes and exponents bit for
bit, decoded values exactly, and the backward passes that read them, against
the fp64 oracle on the decoded input.

dX keeps the linears' 2e-3.  dA and dB are held to 4e-6 (relative Frobenius
error): sums of exact products join every 32 accumulator steps, each step at
most 2^-24 of the sum off towards zero, 32 2^-24 = 1.9e-6 at most; dU and s U
enter as three bf16 parts, exact but for 2^-26; dA has the drift of dU as well:
2 * 1.9e-6 and the fp32 joins' 2^-24 each, randomly."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_26_b200 as q
import synth
from oracle import act8
from tests._util import bits

pytestmark = pytest.mark.gpu


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def _x(M, K, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(4 * torch.randn(M, 1, generator=g))
    x[:, K // 3] *= 300.0
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("M,K", [(1, 64), (3, 128), (64, 512), (1001, 4096), (7, 11008), (4097, 192)])
def test_quantize_and_dequantize_match_oracle(M, K):
    x = _x(M, K)
    x8 = q.act8_quantize(x.cuda())
    codes, exps = act8.quantize(bits(x))
    assert np.array_equal(x8.codes.cpu().numpy(), codes) and np.array_equal(x8.exps.cpu().numpy(), exps)
    out = q.act8_dequantize(x8)
    assert np.array_equal(out.double().cpu().numpy(), act8.dequantize(codes, exps))


def test_every_finite_bf16_value():
    b = np.arange(1 << 16, dtype=np.uint16)
    b = b[(b & 0x7F80) != 0x7F80]
    rng = np.random.default_rng(0)
    b = np.concatenate([b, rng.permutation(b), np.zeros(-2 * b.size % 128, dtype=np.uint16)]).reshape(-1, 128)
    x = torch.from_numpy(b.view(np.int16)).view(torch.bfloat16)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    x8 = q.act8_quantize(x.cuda(), status=status)
    codes, exps = act8.quantize(b)
    assert np.array_equal(x8.codes.cpu().numpy(), codes) and np.array_equal(x8.exps.cpu().numpy(), exps)
    v = act8.dequantize(codes, exps)
    v = np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)
    assert np.array_equal(q.act8_dequantize(x8).double().cpu().numpy(), v)
    assert int(status[0]) == 0


@pytest.mark.parametrize("ld,o", [(320, 64), (320, 8), (328, 64), (200, 8)])
def test_strided_rows_and_the_gap_between_them(ld, o):
    """Rows aligned to 32 bytes, and to the 16 that are asked for."""
    M, K = 37, 192
    buf = torch.full((M, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    x = _x(M, K, 3)
    buf[:, o:o + K] = x.cuda()
    x8 = q.act8_quantize(buf[:, o:o + K])
    codes, exps = act8.quantize(bits(x))
    assert np.array_equal(x8.codes.cpu().numpy(), codes) and np.array_equal(x8.exps.cpu().numpy(), exps)
    out = torch.full((M, ld), 9.0, dtype=torch.bfloat16, device="cuda")
    q.act8_dequantize(x8, out=out[:, o:o + K])
    assert np.array_equal(out[:, o:o + K].double().cpu().numpy(), act8.dequantize(codes, exps))
    assert bool((out[:, :o] == 9).all()) and bool((out[:, o + K:] == 9).all())


def test_non_finite_values_keep_their_place():
    x = torch.ones(4, 128, dtype=torch.bfloat16)
    x[1, 5], x[2, 70], x[3, 0] = float("nan"), float("inf"), -float("inf")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = q.act8_dequantize(q.act8_quantize(x.cuda(), status=status)).float().cpu()
    assert int(status[0]) == q.DEV_NONFINITE
    assert torch.isnan(out[1, 5]) and out[2, 70] == float("inf") and out[3, 0] == -float("inf")
    assert int(torch.isnan(out).sum()) == 1 and int(torch.isinf(out).sum()) == 2
    assert bool((out[0] == 1).all()) and bool((out[1, 64:] == 1).all())


def test_no_rows():
    x8 = q.act8_quantize(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"))
    assert x8.codes.shape == (0, 128) and q.act8_dequantize(x8).shape == (0, 128)


# tokens, outputs, inputs, rank: every GEMM path, ragged stages and tiles, rank chunks
SHAPES = [(1, 64, 64, 16), (64, 512, 512, 16), (65, 192, 320, 48), (200, 512, 640, 32), (600, 512, 768, 64),
          (1000, 384, 448, 64), (150, 384, 448, 144), (700, 512, 768, 256), (4096, 4096, 4096, 64),
          (577, 256, 256, 64), (16384, 128, 4096, 16), (1153, 8192, 128, 64)]


@pytest.mark.parametrize("M,N,K,r", SHAPES)
@pytest.mark.parametrize("dt", [q.DTYPE_BF16, q.DTYPE_F32])
def test_linear_bwd_act8(M, N, K, r, dt):
    d = synth.linear_inputs(synth.Linear("a8", N, K), M, r, 1)
    g = {k: v.cuda() for k, v in d.items()}
    W, s = q.quantize_weight(g["W"]), 16.0 / r
    U = g["X"].float() @ g["A"].float().t()
    x8 = q.act8_quantize(g["X"])
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    dX, dA, dB = q.qlora_linear_bwd_act8(g["dY"], x8, U, W, g["A"], g["B"], s, dx_dtype=dt, status=status)
    assert int(status[0]) == 0
    _check(d["dY"], x8, U, q.nf4_dequantize(W.codes, W.c8, W.s2, N * K).view(N, K), [N], d["A"], d["B"], s,
           (dX, dA, dB))
    again = q.qlora_linear_bwd_act8(g["dY"], x8, U, W, g["A"], g["B"], s, dx_dtype=dt)
    for a, b in zip(again, (dX, dA, dB)):
        assert _same(a, b)


def _check(dY, x8, U, Wd, members, A, B, s, got):
    """Against the formulas in fp64 on the GPU (the oracle's values as inputs)."""
    x = torch.from_numpy(act8.dequantize(x8.codes.cpu().numpy(), x8.exps.cpu().numpy())).cuda()
    dY, A, B, U, Wd = (v.double().cuda() for v in (dY, A, B, U, Wd))
    r = A.shape[0] // len(members)
    dX, dA, dB, n0 = 0, [], [], 0
    for i, n in enumerate(members):
        dYg, Bg, j = dY[:, n0:n0 + n], B[n0:n0 + n], slice(i * r, (i + 1) * r)
        dU = s * (dYg @ Bg)
        dX = dX + dYg @ Wd[n0:n0 + n] + dU @ A[j]
        dA.append(dU.t() @ x)
        dB.append(s * (dYg.t() @ U[:, j]))
        n0 += n
    for a, ref, tol in zip(got, (dX, torch.cat(dA), torch.cat(dB)), (2e-3, 4e-6, 4e-6)):
        assert float((a.double() - ref).norm() / ref.norm()) <= tol


@pytest.mark.parametrize("M,members,K,r", [(333, (256, 128), 512, 16), (1030, (512, 512, 256), 768, 64),
                                           (40, (128, 128, 128, 128), 192, 32), (512, (320,), 256, 128)])
def test_group_bwd_act8(M, members, K, r):
    G, N = len(members), sum(members)
    gen = torch.Generator().manual_seed(M)
    def rnd(*s, std=1.0):
        return (torch.randn(*s, generator=gen) * std).to(torch.bfloat16).cuda()
    W = q.quantize_weight(rnd(N, K, std=0.02))
    A, B, X, dY = rnd(G * r, K, std=K ** -0.5), rnd(N, r, std=0.1), rnd(M, K), rnd(M, N)
    U = X.float() @ A.float().t()
    x8 = q.act8_quantize(X)
    got = q.qlora_group_bwd_act8(dY, x8, U, W, members, A, B, 0.5)
    _check(dY, x8, U, q.nf4_dequantize(W.codes, W.c8, W.s2, N * K).view(N, K), members, A, B, 0.5, got)


@pytest.mark.parametrize("M,N,K,r,p", [(200, 512, 640, 32, 0.05), (600, 512, 768, 64, 0.5), (150, 384, 448, 144, 0.1)])
def test_dropout_bwd_act8(M, N, K, r, p):
    d = synth.linear_inputs(synth.Linear("a8d", N, K), M, r, 2)
    g = {k: v.cuda() for k, v in d.items()}
    W = q.quantize_weight(g["W"])
    Y, U, Xd = q.qlora_linear_fwd_dropout(g["X"], W, g["A"], g["B"], 0.25, p, 11)
    x8 = q.act8_quantize(Xd)
    back = q.act8_dequantize(x8)
    assert bool((back[Xd == 0] == 0).all())
    got = q.qlora_linear_bwd_dropout_act8(g["dY"], x8, U, W, g["A"], g["B"], 0.25, p, 11)
    want = q.qlora_linear_bwd_dropout(g["dY"], back, U, W, g["A"], g["B"], 0.25, p, 11)
    for a, b, tol in zip(got, want, (2e-3, 1e-4, 1e-4)):  # the plain pass on the decoded input
        assert float((a.double() - b.double()).norm() / b.double().norm()) <= tol


def test_no_tokens_give_zero_gradients():
    W = q.quantize_weight(torch.randn(128, 128).to(torch.bfloat16).cuda())
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    A = torch.zeros(16, 128, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(128, 16, dtype=torch.bfloat16, device="cuda")
    dX, dA, dB = q.qlora_linear_bwd_act8(e, q.act8_quantize(e), torch.empty(0, 16, device="cuda"), W, A, B, 1.0)
    assert dX.shape == (0, 128) and not dA.any() and not dB.any()


def test_refusals_on_device_tensors():
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    x8 = q.act8_quantize(x)
    for bad in (x[:, :100], x.t(), torch.zeros(4, 132, dtype=torch.bfloat16, device="cuda")[:, :128],
                x[:1].expand(4, 128), torch.zeros(4, 136, dtype=torch.bfloat16, device="cuda")[:, 4:132]):
        with pytest.raises(q.QloraError):
            q.act8_quantize(bad)
    with pytest.raises(q.QloraError):
        q.act8_dequantize(q.Act8(x8.codes, x8.exps[:, :1]))
    with pytest.raises(q.QloraError):
        q.act8_dequantize(x8, out=torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda"))
    W = q.quantize_weight(torch.zeros(128, 128, dtype=torch.bfloat16, device="cuda"))
    A = torch.zeros(16, 128, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(128, 16, dtype=torch.bfloat16, device="cuda")
    dY, U = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 16, device="cuda")
    for args in ((dY.float(), x8, U, W, A, B), (dY, x8, U[:3], W, A, B), (dY, x8, U, W, A[:, :64], B),
                 (dY, q.Act8(x8.codes[:2], x8.exps), U, W, A, B), (dY.t().contiguous().t(), x8, U, W, A, B)):
        with pytest.raises(q.QloraError):
            q.qlora_linear_bwd_act8(*args, 1.0)


@pytest.mark.parametrize("M,N,K,r,p,centred", [(16, 320, 512, 16, 0.05, False), (600, 512, 768, 64, 0.5, True),
                                               (150, 384, 448, 144, 0.1, False), (1153, 768, 256, 256, 0.3, True)])
def test_dropout_bwd_act8_against_the_formulas(M, N, K, r, p, centred):
    """dA = dU^T X_drop', dB = s dY^T U, dX = dY W' + keep / (1 - p) (dU A), dU = s dY B."""
    d = synth.linear_inputs(synth.Linear("a8f", N, K), M, r, 4)
    g = {k: v.cuda() for k, v in d.items()}
    W = (q.quantize_weight_centered if centred else q.quantize_weight)(g["W"])
    dense = (q.nf4_dequantize_centered(W.codes, W.c8, W.s2, W.mean, N * K) if centred
             else q.nf4_dequantize(W.codes, W.c8, W.s2, N * K)).view(N, K).double()
    _, U, Xd = q.qlora_linear_fwd_dropout(g["X"], W, g["A"], g["B"], 0.25, p, 12)
    x8 = q.act8_quantize(Xd)
    got = q.qlora_linear_bwd_dropout_act8(g["dY"], x8, U, W, g["A"], g["B"], 0.25, p, 12)
    x = torch.from_numpy(act8.dequantize(x8.codes.cpu().numpy(), x8.exps.cpu().numpy())).cuda()
    dY, A, B = (g[k].double() for k in ("dY", "A", "B"))
    dU = 0.25 * (dY @ B)
    keep = ((Xd != 0) | (g["X"] == 0)).double()
    want = (dY @ dense + keep / (1 - p) * (dU @ A), dU.t() @ x, 0.25 * (dY.t() @ U.double()))
    for a, ref, tol in zip(got, want, (2e-3, 4e-6, 4e-6)):
        assert float((a.double() - ref).norm() / ref.norm()) <= tol


@pytest.mark.parametrize("M,members,K,r", [(40, (320,), 192, 16), (700, (512,), 768, 64), (1030, (512, 256), 768, 32)])
def test_bwd_act8_of_a_centred_weight(M, members, K, r):
    G, N = len(members), sum(members)
    gen = torch.Generator().manual_seed(M)

    def rnd(*s, std=1.0):
        return (torch.randn(*s, generator=gen) * std).to(torch.bfloat16).cuda()
    W = q.quantize_weight_centered(rnd(N, K, std=0.02))
    A, B, X, dY = rnd(G * r, K, std=K ** -0.5), rnd(N, r, std=0.1), rnd(M, K), rnd(M, N)
    U = X.float() @ A.float().t()
    x8 = q.act8_quantize(X)
    got = (q.qlora_group_bwd_act8(dY, x8, U, W, members, A, B, 0.5) if G > 1
           else q.qlora_linear_bwd_act8(dY, x8, U, W, A, B, 0.5))
    _check(dY, x8, U, q.nf4_dequantize_centered(W.codes, W.c8, W.s2, W.mean, N * K).view(N, K), members, A, B, 0.5, got)


@pytest.mark.parametrize("M,N,K,r", [(64, 512, 512, 16), (1000, 384, 448, 64), (4096, 1024, 256, 64)])
def test_sums_that_cancel(M, N, K, r):
    """Tokens in pairs whose terms of dA and dB nearly cancel: the errors stay within
    4e-6 of the sums of the terms' absolute values (the derivation at the top)."""
    gen = torch.Generator().manual_seed(M)

    def rnd(*s, std=1.0):
        return torch.randn(*s, generator=gen) * std
    X, dY = rnd(M, K), rnd(M, N)
    X[1::2] = X[::2]
    dY[1::2] = -dY[::2] * (1 + 2.0 ** -6 * (rnd(M // 2, 1) > 0))
    X, dY, A, B = (t.to(torch.bfloat16).cuda() for t in (X, dY, rnd(r, K, std=K ** -0.5), rnd(N, r, std=0.1)))
    W = q.quantize_weight(rnd(N, K, std=0.02).to(torch.bfloat16).cuda())
    U = X.float() @ A.float().t()
    x8 = q.act8_quantize(X)
    _, dA, dB = q.qlora_linear_bwd_act8(dY, x8, U, W, A, B, 0.5)
    x = torch.from_numpy(act8.dequantize(x8.codes.cpu().numpy(), x8.exps.cpu().numpy())).cuda()
    dY, B, U = dY.double(), B.double(), U.double()
    for a, ref, size in ((dA, (0.5 * (dY @ B)).t() @ x, 0.5 * (dY.abs() @ B.abs()).t() @ x.abs()),
                         (dB, 0.5 * (dY.t() @ U), 0.5 * (dY.abs().t() @ U.abs()))):
        assert float(ref.norm()) < 0.1 * float(size.norm())
        assert bool(((a.double() - ref).abs() <= 4e-6 * size).all())
