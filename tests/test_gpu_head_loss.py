"""GPU parity of the loss head against the fp64 oracle on the exact bf16 inputs.

Tolerances, per element and derived:

* a logit is a sum of dim exact products in fp32, in any order: off by at most
  d_tv = 2 dim 2^-24 sum_d |h_td w_vd| (2^-24 half a step, twice for a sum that
  truncates), and d_t is the largest over v;
* lse is a weighted mean away from the logits' errors: off by d_t plus the
  fp32 exponentials (relative 2^-22, and the argument's rounding, 2^-23 of the
  largest |l| log2 e) and its own rounding: d_t + 2^-21 (4 + max|l|);
* the loss by that and the label logit's error: 2 d_t + 2^-21 (4 + 2 max|l|);
* dH: a probability is off by rel = 2 d_t + 2^-20 (4 + max|l|) relative.  At the
  label p - 1 = expm1(l - lse) is taken in fp32 first, so its error is that of
  p, rel p, and not rel (1 - p): with V = 1, where p = 1 and the gradient is 0,
  an lse half an ulp off gives rel.  Then G = p - onehot is rounded to bf16
  (2^-8 relative; twice where the step rescales a row) and the output once
  more: |g_t| sum_v (rel p_tv + 2^-8 |G_tv|) |W_vd| + 2^-8 |dH_td|.
"""

import math

import numpy as np
import pytest
import torch

import bit_nf4_quantized_26_b200 as q
from oracle import head_loss as hl
from oracle import nf4
from tests._util import bits

pytestmark = pytest.mark.gpu


def _case(T, V, D, seed=0, scale=1.0, ignored=0.25, lean=0.0):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, D, generator=g) * 0.02).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g)
    h = torch.randn(T, D, generator=g) * scale
    if lean:
        h = h + lean * torch.rand(T, 1, generator=g) * w[y].float() / (4e-4 * D)
    out = torch.rand(T, generator=g) < ignored
    return h.to(torch.bfloat16), w, torch.where(out, torch.full_like(y, -100), y)


class Ref:
    """The oracle's answers and the bounds above."""

    def __init__(self, h, w, y):
        hb, wb, self.y = bits(h), bits(w), y.numpy()
        H, W = hl._f64(hb), hl._f64(wb)
        D = H.shape[1]
        self.loss, self.lse, self.mean, self.count = hl.fwd(hb, wb, self.y)
        d = 2 * D * 2.0 ** -24 * (np.abs(H) @ np.abs(W).T).max(1)
        top = np.abs(H @ W.T).max(1)
        self.lse_tol = d + 2.0 ** -21 * (4 + top)
        self.loss_tol = 2 * d + 2.0 ** -21 * (4 + 2 * top)
        self.p = hl.probabilities(hb, wb, self.y)
        self.W, self.rel = W, 2 * d + 2.0 ** -20 * (4 + top)
        self.soft = np.exp(H @ W.T - self.lse[:, None])

    def check_loss(self, loss, lse, stats):
        loss, lse, stats = (v.double().cpu().numpy() for v in (loss, lse, stats))
        assert np.all(np.abs(lse - self.lse) <= self.lse_tol)
        assert np.all(np.abs(loss - self.loss) <= self.loss_tol)
        assert not loss[self.y == -100].any()
        assert stats[1] == self.count
        assert abs(stats[0] - self.mean) <= self.loss_tol.mean() * self.y.size / max(self.count, 1) + 2.0 ** -23 * abs(
            self.mean)

    def check_grad(self, dH, g, roundings=1):
        dH = dH.double().cpu().numpy()
        c = hl.counted(self.y, self.W.shape[0])
        g = np.where(c, np.asarray(g, dtype=np.float64), 0.0)
        ref = (self.p * g[:, None]) @ self.W
        off = (roundings * 2.0 ** -8 * 1.01 * np.abs(self.p) + self.rel[:, None] * self.soft) * np.abs(g)[:, None]
        tol = off @ np.abs(self.W) + 2.0 ** -8 * np.abs(ref) + 1e-37
        assert np.all(np.abs(dH - ref) <= tol)
        assert not dH[~c].any()
        if self.rel.max() < 1e-3 and self.W.shape[0] > 1:  # and as a whole, well inside
            assert np.linalg.norm(dH - ref) <= 5e-3 * np.linalg.norm(ref)


# tokens, vocabulary, width: one of each, odd ones, tile borders, widths that end inside a stage
SHAPES = [(1, 1, 8), (1, 1000, 64), (3, 257, 72), (129, 256, 256), (200, 1003, 520), (256, 512, 64), (257, 255, 192),
          (700, 3001, 1024), (60, 33000, 256), (128, 4000, 328), (16, 40001, 640), (380, 20000, 512), (300, 9000, 320),
          (2000, 9000, 1304)]  # the last: 48 tiles of dH on 74 pairs, each in two parts


@pytest.mark.parametrize("T,V,D", SHAPES)
def test_loss_and_gradient_match_oracle(T, V, D):
    h, w, y = _case(T, V, D, seed=T)
    y[-1] = V - 1
    r = Ref(h, w, y)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    H, W, Y = h.cuda(), w.cuda(), y.cuda()
    loss, lse, stats = q.qlora_head_loss_fwd(H, W, Y, status=status)
    r.check_loss(loss, lse, stats)
    g = torch.linspace(-1, 2, T)
    dH = q.qlora_head_loss_bwd(H, W, Y, lse, g.cuda(), status=status)
    r.check_grad(dH, g.numpy())
    up = torch.tensor([3.0], device="cuda")
    r.check_grad(q.qlora_head_loss_bwd(H, W, Y, lse, up, stats=stats), np.full(T, 3.0 / max(r.count, 1)))
    got = q.qlora_head_loss_step(H, W, Y, scale=2.0, status=status)
    r.check_loss(*got[:3])
    r.check_grad(got[3], np.full(T, 2.0 / max(r.count, 1)))
    got = q.qlora_head_loss_step(H, W, Y, weight=g.cuda(), scale=0.5, status=status)
    r.check_grad(got[3], 0.5 * g.numpy())
    assert int(status[0]) == 0
    again = q.qlora_head_loss_step(H, W, Y, weight=g.cuda(), scale=0.5)
    for a, b in zip(got, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))




@pytest.mark.parametrize("T,V,D", [(16500, 4500, 64), (33000, 2500, 128), (1000, 70000, 64), (2048, 36000, 336)])
def test_several_pieces(T, V, D):
    """Sizes at which the vocabulary runs in more than one piece: the fp32 sum
    carried between pieces (whole tiles', and parts' whose last piece is shorter)."""
    assert q.qlora_head_loss_workspace_size(T, V, D, False, q.HEAD_BWD) < 2 * T * V  # not the whole operand
    h, w, y = _case(T, V, D, seed=1, lean=10.0)
    rows = np.unique(np.linspace(0, T - 1, 400).astype(int))
    r = Ref(h[rows], w, y[rows])
    H, W, Y = h.cuda(), w.cuda(), y.cuda()
    g = torch.linspace(-1, 2, T)
    loss, lse, stats = q.qlora_head_loss_fwd(H, W, Y)
    assert np.all(np.abs(loss.cpu().numpy()[rows] - r.loss) <= r.loss_tol)
    sel = torch.from_numpy(rows).cuda()
    r.check_grad(q.qlora_head_loss_bwd(H, W, Y, lse, g.cuda())[sel], g.numpy()[rows])
    l2, lse2, st2, dH = q.qlora_head_loss_step(H, W, Y, weight=g.cuda())
    assert np.all(np.abs(l2.cpu().numpy()[rows] - r.loss) <= r.loss_tol)
    assert np.all(np.abs(lse2.cpu().numpy()[rows] - r.lse) <= r.lse_tol)
    assert float(st2[1]) == float(stats[1]) == int((y != -100).sum())
    assert abs(float(st2[0]) - float(stats[0])) <= 2 * r.loss_tol.max()
    r.check_grad(dH[sel], g.numpy()[rows])


@pytest.mark.parametrize("scale", [30.0, 200.0])
@pytest.mark.parametrize("T,V,D", [(100, 2000, 256), (16500, 4500, 64), (1000, 70000, 64)])
def test_large_logits_take_other_references(T, V, D, scale):
    """Logits of some hundreds, of either sign and far apart between tiles and
    pieces: rows whose tiles have different references, a row far below zero."""
    h, w, y = _case(T, V, D, seed=2, scale=scale)
    h, w = h.float(), w.float() * 4
    w[:256, 0] += 1.0
    w[1000:1256, 0] -= 1.0
    h[3] = 0
    w[:, 1] = 1.0
    h[3, 1] = -300.0        # every logit of the row at -300
    h[4] = 0
    h[4, 1] = 300.0
    h, w = h.to(torch.bfloat16), w.to(torch.bfloat16)
    y[3], y[4] = 5, V - 1
    rows = np.unique(np.concatenate([np.arange(60), np.linspace(0, T - 1, 100).astype(int)]))
    r = Ref(h[rows], w, y[rows])
    H, W, Y = h.cuda(), w.cuda(), y.cuda()
    sel = torch.from_numpy(rows).cuda()
    loss, lse, stats = q.qlora_head_loss_fwd(H, W, Y)
    assert np.all(np.abs(lse.cpu().numpy()[rows] - r.lse) <= r.lse_tol)
    g = torch.ones(T, device="cuda")
    r.check_grad(q.qlora_head_loss_bwd(H, W, Y, lse, g)[sel], np.ones(rows.size))
    l2, lse2, _, dH = q.qlora_head_loss_step(H, W, Y, weight=g)
    assert np.all(np.abs(l2.cpu().numpy()[rows] - r.loss) <= r.loss_tol)
    assert np.all(np.abs(lse2.cpu().numpy()[rows] - r.lse) <= r.lse_tol)
    r.check_grad(dH[sel], np.ones(rows.size), roundings=2)


# large enough that dH's products take the rows that count only: token tiles of
# both kinds, several pieces, a split contraction, NF4, logits with other references
COMPACT = [(300, 33000, 2560, False, 0.3, 1.0), (1153, 5000, 4400, True, 0.6, 1.0), (3000, 9000, 1024, False, 0.25, 1.0),
           (16500, 4500, 448, False, 0.5, 30.0), (2000, 12500, 1024, False, 0.999, 1.0),
           (2000, 12500, 1024, True, 0.0, 1.0)]


@pytest.mark.parametrize("T,V,D,nf4,ignored,scale", [c if not c[3] else (c[0], c[1], c[2] // 64 * 64) + c[3:]
                                                     for c in COMPACT])
def test_rows_that_count(T, V, D, nf4, ignored, scale):
    assert T > 256 and 4.0 * T * V * D >= 1e11
    h, w, y = _case(T, V, D, seed=12, ignored=ignored, scale=scale, lean=0.0 if scale > 1 else 5.0)
    y[T // 2] = V - 1                                     # one at least counts
    h[y == -100] = float("nan")
    H, Y, W = h.cuda(), y.cuda(), w.cuda()
    if nf4:
        W = q.quantize_weight(W)
        w = q.nf4_dequantize(W.codes, W.c8, W.s2, V * D).view(V, D).cpu()
    count = torch.nonzero(y != -100)[:, 0]
    rows = count[torch.linspace(0, count.numel() - 1, min(120, count.numel())).long()].unique()
    r = Ref(h[rows], w, y[rows])
    sel, gone = rows.cuda(), (y == -100).cuda()
    g = torch.linspace(-1, 2, T)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    _, lse, _ = q.qlora_head_loss_fwd(H, W, Y)
    buf = torch.full((T, D + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    for dH in (None, buf[:, 8:8 + D]):
        d = q.qlora_head_loss_bwd(H, W, Y, lse, g.cuda(), dH=dH, status=status)
        r.check_grad(d[sel], g.numpy()[rows], roundings=2)
        assert not d[gone].any()
    assert bool((buf[:, :8] == 5).all()) and bool((buf[:, 8 + D:] == 5).all())
    buf.fill_(5.0)
    for dH in (None, buf[:, 8:8 + D]):
        l2, lse2, st, d = q.qlora_head_loss_step(H, W, Y, weight=g.cuda(), dH=dH, status=status)
        r.check_grad(d[sel], g.numpy()[rows], roundings=2)
        assert not d[gone].any() and int(st[1]) == count.numel()
        assert np.all(np.abs(l2.cpu().numpy()[rows] - r.loss) <= r.loss_tol)
    assert bool((buf[:, :8] == 5).all()) and bool((buf[:, 8 + D:] == 5).all())
    assert int(status[0]) == 0
    again = H.clone()                                     # in place of the hidden states
    inplace = q.qlora_head_loss_step(again, W, Y, weight=g.cuda(), dH=again)[3]
    assert torch.equal(inplace, d)
    again = H.clone()
    want = q.qlora_head_loss_bwd(H, W, Y, lse, g.cuda())
    assert torch.equal(q.qlora_head_loss_bwd(again, W, Y, lse, g.cuda(), dH=again), want)


@pytest.mark.parametrize("case", ["none", "first", "last", "bad"])
def test_rows_that_count_at_the_ends(case):
    T, V, D = 3000, 9000, 1024
    h, w, y = _case(T, V, D, seed=13, ignored=0.0)
    k = {"none": [], "first": [0], "last": [T - 1], "bad": [5, 2500]}[case]
    z = torch.full_like(y, -100)
    z[k] = y[k]
    if case == "bad":
        z[7], z[2999], z[4] = V, -3, 1 << 40
    H, W, Y = h.cuda(), w.cuda(), z.cuda()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    loss, lse, stats, dH = q.qlora_head_loss_step(H, W, Y, scale=2.0, status=status)
    assert int(status[0]) == (q.DEV_LABEL if case == "bad" else 0) and int(stats[1]) == len(k)
    status.zero_()
    dB = q.qlora_head_loss_bwd(H, W, Y, lse, torch.full((1,), 2.0, device="cuda"), stats=stats, status=status)
    assert int(status[0]) == (q.DEV_LABEL if case == "bad" else 0)
    keep = torch.zeros(T, dtype=torch.bool)
    keep[k] = True
    for d in (dH, dB):
        assert not d[~keep.cuda()].any()
        if k:
            Ref(h[k], w, y[k]).check_grad(d[k], np.full(len(k), 2.0 / len(k)), roundings=2)


def test_rows_that_count_change_between_replays():
    """Captured once, replayed with other labels: the rows that count, their
    tiles and those tiles' parts are the replay's own."""
    T, V, D = 600, 20000, 2304
    assert 4.0 * T * V * D >= 1e11
    h, w, y = _case(T, V, D, seed=15, ignored=0.0)
    H, W, Y = h.cuda(), w.cuda(), y.cuda()
    g, buf = torch.linspace(-1, 1, T, device="cuda"), torch.empty(T, dtype=torch.int64, device="cuda")
    buf.copy_(Y)

    def call():
        step = q.qlora_head_loss_step(H, W, buf, weight=g)
        return (*step, q.qlora_head_loss_bwd(H, W, buf, step[1], g))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for keep in (1.0, 0.5, 0.0, 0.1, 0.9):
        buf.copy_(torch.where(torch.rand(T, generator=torch.Generator().manual_seed(int(10 * keep))) < keep, y,
                              torch.full_like(y, -100)))
        for o in outs:
            o.fill_(7.0)
        graph.replay()
        for got, want in zip(outs, call()):
            assert torch.equal(got, want)
        assert not outs[3][buf == -100].any() and not outs[4][buf == -100].any()


def test_well_predicted_tokens_keep_their_gradient():
    """p close to 1 at the label: the gradient is the small difference."""
    h, w, y = _case(64, 500, 256, seed=4, ignored=0.0)
    h = (h.float() + 25.0 * w[y].float() / (4e-4 * 256)).to(torch.bfloat16)
    r = Ref(h, w, y)
    assert r.loss.min() < 1e-4
    H, W, Y = h.cuda(), w.cuda(), y.cuda()
    loss, lse, stats = q.qlora_head_loss_fwd(H, W, Y)
    dH = q.qlora_head_loss_step(H, W, Y, weight=torch.ones(64, device="cuda"))[3].double().cpu().numpy()
    ref = r.p @ r.W
    err = np.linalg.norm(dH - ref, axis=1) / np.linalg.norm(ref, axis=1)
    # 1 - p is off by the lse's and label logit's fp32 errors over its size
    small = -np.take_along_axis(r.p, r.y[:, None], 1)[:, 0]
    assert np.all(err <= 2 * 2.0 ** -8 + r.loss_tol / small)


@pytest.mark.parametrize("T,V,D,sign", [(3, 500, 256, 1.0), (64, 3000, 256, 1.0), (300, 9000, 320, 1.0),
                                        (1000, 70000, 64, 1.0), (64, 3000, 256, -1.0)])
def test_losses_keep_their_digits(T, V, D, sign):
    """Losses from below 1e-7 to some tens, label logits far above the others (or far
    below).  With x = sum over the others of exp(l_v - l_label), loss =
    log1p(x): x is off by rel (the two logits' errors and the exponentials'),
    log1p by no more than that relative and its own 2^-22; the reference is one
    step of fp32 around.  The label's p - 1 = -x / (1 + x) likewise."""
    h, w, y = _case(T, V, D, seed=14, ignored=0.1)
    lead = torch.linspace(2.0, 38.0, T)[:, None]
    safe = y.clamp(min=0)
    unit = w[safe].float() / (w[safe].float() ** 2).sum(1, keepdim=True)
    h = (sign * lead * unit + 0.1 * h.float()).to(torch.bfloat16)
    rows = np.unique(np.linspace(0, T - 1, 200).astype(int))
    r = Ref(h[rows], w, y[rows])
    c = hl.counted(r.y, V)
    z = hl._f64(bits(h[rows])) @ hl._f64(bits(w)).T
    zy = z[np.arange(rows.size), np.where(c, r.y, 0)]
    others = np.exp(z - zy[:, None])
    others[np.arange(rows.size), np.where(c, r.y, 0)] = 0.0
    loss = np.where(c, np.log1p(others.sum(1)), 0.0)
    if sign > 0:
        assert loss[c].min() < 1e-7 and loss[c].max() > 1.0  # the oracle's: 1.3e-8 at 70000 x 64, far less elsewhere
    H, W, Y, sel = h.cuda(), w.cuda(), y.cuda(), torch.from_numpy(rows).cuda()
    tol = (r.rel + 2.0 ** -21) * loss
    got = q.qlora_head_loss_step(H, W, Y, weight=torch.ones(T, device="cuda"))
    for out in (q.qlora_head_loss_fwd(H, W, Y), got):
        assert np.all(np.abs(out[0][sel].double().cpu().numpy() - loss) <= tol)
        assert np.all(np.abs(out[1][sel].double().cpu().numpy() - r.lse) <= r.lse_tol)
    back = q.qlora_head_loss_bwd(H, W, Y, got[1], torch.ones(T, device="cuda"))
    r.check_grad(back[sel], np.ones(rows.size))
    g = np.abs(r.p)
    ref = r.p @ r.W
    bound = (r.rel[:, None] + 2.0 ** -21 + 2 * 2.0 ** -8 * 1.01) * g @ np.abs(r.W) + 2.0 ** -8 * np.abs(ref) + 1e-37
    assert np.all(np.abs(got[3][sel].double().cpu().numpy() - ref)[c] <= bound[c])


@pytest.mark.parametrize("T,V,D,centred", [(5, 1001, 64, False), (300, 2300, 512, True), (64, 40000, 2048, False),
                                           (17000, 4500, 128, True), (128, 300, 64, False), (129, 5000, 192, True),
                                           (512, 1000, 448, False), (127, 70001, 64, True), (3, 1, 64, False), (70, 63, 128, True), (380, 20000, 512, False), (1, 30000, 1024, False),
                                           (8, 6000, 20480, False)])
def test_nf4_head(T, V, D, centred):
    """An NF4 head is the bf16 head of its dequantised weight.  The logits are the
    same bits; the pieces, and so the order in which a row's exponentials are
    summed, are not: both losses lie within the bound of the exact one, so they
    differ by at most twice that."""
    h, w, y = _case(T, V, D, seed=5, lean=5.0)
    H, Y = h.cuda(), y.cuda()
    W = (q.quantize_weight_centered if centred else q.quantize_weight)(w.cuda())
    dense = (q.nf4_dequantize_centered(W.codes, W.c8, W.s2, W.mean, V * D) if centred
             else q.nf4_dequantize(W.codes, W.c8, W.s2, V * D)).view(V, D)
    a, b = q.qlora_head_loss_fwd(H, W, Y), q.qlora_head_loss_fwd(H, dense, Y)
    g = torch.linspace(-1, 1, T, device="cuda")
    n = min(T, 200)
    r = Ref(h[:n], dense.cpu(), y[:n])
    assert float(a[2][1]) == float(b[2][1])
    assert np.all(np.abs((a[0] - b[0]).cpu().numpy()[:n]) <= 2 * r.loss_tol)
    assert np.all(np.abs(a[0].cpu().numpy()[:n] - r.loss) <= r.loss_tol)
    r.check_grad(q.qlora_head_loss_bwd(H, W, Y, a[1], g)[:n], g.cpu().numpy()[:n])
    got = q.qlora_head_loss_step(H, W, Y, weight=g)
    r.check_grad(got[3][:n], g.cpu().numpy()[:n])
    assert np.all(np.abs(got[0].cpu().numpy()[:n] - r.loss) <= r.loss_tol)


def test_nf4_head_of_equal_constants():
    """Mean-centred constants that are all equal have scale 0: their value is the mean."""
    T, V, D = 20, 500, 128
    h, _, y = _case(T, V, D, seed=7)
    g = torch.Generator().manual_seed(3)
    w = torch.where(torch.rand(V, D, generator=g) < 0.5, 0.25, -0.25).to(torch.bfloat16)
    W = q.quantize_weight_centered(w.cuda())
    assert not W.s2.any() and float(W.mean) == 0.25
    r = Ref(h, w, y)
    got = q.qlora_head_loss_step(h.cuda(), W, y.cuda(), weight=torch.ones(T, device="cuda"))
    r.check_loss(*got[:3])
    r.check_grad(got[3], np.ones(T))


def test_ignored_rows_may_hold_anything():
    h, w, y = _case(300, 700, 128, seed=6, ignored=0.0)
    y[5], y[6], y[200], y[299] = -100, -100, -100, -100
    clean = h.clone()
    h[5], h[6, 3], h[200] = float("nan"), float("inf"), torch.finfo(torch.bfloat16).min
    H, C, W, Y = h.cuda(), clean.cuda(), w.cuda(), y.cuda()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    keep = torch.tensor([i for i in range(300) if i not in (5, 6, 200, 299)], device="cuda")
    a, b = (q.qlora_head_loss_fwd(x, W, Y, status=status) for x in (H, C))
    g = torch.ones(300, device="cuda")
    g[5], g[200] = float("nan"), float("inf")  # nor are their gradients read
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]) and torch.equal(a[1][keep], b[1][keep])
    da, db = q.qlora_head_loss_bwd(H, W, Y, a[1], g, status=status), q.qlora_head_loss_bwd(C, W, Y, b[1], g)
    sa, sb = q.qlora_head_loss_step(H, W, Y, status=status), q.qlora_head_loss_step(C, W, Y)
    wa, wb = q.qlora_head_loss_step(H, W, Y, weight=g, status=status), q.qlora_head_loss_step(C, W, Y, weight=g)
    for x, z in ((da, db), (wa[3], wb[3]), (sa[3], sb[3]), (sa[0], sb[0]), (sa[2], sb[2])):
        assert torch.equal(x, z)
    assert not da[5].any() and not sa[3][200].any()
    assert int(status[0]) == 0
    # a counted token's NaN stays with its row and is reported
    g = torch.ones(300, device="cuda")
    y2 = Y.clone()
    y2[5] = 1
    s2 = q.qlora_head_loss_step(H, W, y2, weight=g, status=status)
    assert int(status[0]) == q.DEV_NONFINITE
    assert torch.isnan(s2[0][5]) and torch.isnan(s2[3][5]).all()
    ref = q.qlora_head_loss_step(C, W, Y, weight=g)
    assert torch.equal(s2[3][keep], ref[3][keep])


def test_no_token_counts():
    h, w, y = _case(40, 300, 64)
    y[:] = -100
    H, W, Y = h.cuda(), w.cuda(), y.cuda()
    loss, lse, stats = q.qlora_head_loss_fwd(H, W, Y)
    assert not loss.any() and stats.tolist() == [0.0, 0.0] and bool(torch.isfinite(lse).all())
    assert not q.qlora_head_loss_bwd(H, W, Y, lse, torch.ones(1, device="cuda"), stats=stats).any()
    got = q.qlora_head_loss_step(H, W, Y)
    assert not got[3].any() and got[2].tolist() == [0.0, 0.0]


def test_no_tokens():
    H, W = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(9, 64, dtype=torch.bfloat16).cuda()
    Y = torch.empty(0, dtype=torch.int64, device="cuda")
    stats = torch.full((2,), 5.0, device="cuda")
    loss, lse, st = q.qlora_head_loss_fwd(H, W, Y, stats=stats)
    assert loss.numel() == 0 and st.tolist() == [0.0, 0.0]
    e = torch.empty(0, device="cuda")
    assert q.qlora_head_loss_bwd(H, W, Y, e, e).shape == (0, 64)
    assert q.qlora_head_loss_step(H, W, Y)[3].shape == (0, 64)


@pytest.mark.parametrize("bad", [-1, 300, 1 << 40, -(1 << 62)])
def test_labels_out_of_range_are_reported_and_ignored(bad):
    h, w, y = _case(40, 300, 64, ignored=0.0)
    y2 = y.clone()
    y2[7], y[7] = bad, -100
    H, W = h.cuda(), w.cuda()
    g = torch.ones(40, device="cuda")
    lse = None
    for f in (lambda Y, st: q.qlora_head_loss_fwd(H, W, Y, status=st),
              lambda Y, st: q.qlora_head_loss_step(H, W, Y, status=st),
              lambda Y, st: (q.qlora_head_loss_bwd(H, W, Y, lse, g, status=st),)):
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        a, b = f(y2.cuda(), status), f(y.cuda(), None)
        assert int(status[0]) == q.DEV_LABEL
        for x, z in zip(a, b):
            assert torch.equal(x, z)
        lse = b[1] if len(b) > 1 else lse


def test_other_ignore_index():
    h, w, y = _case(40, 300, 64)
    y2 = torch.where(y == -100, torch.full_like(y, 17), torch.where(y == 17, torch.full_like(y, 18), y))
    y1 = torch.where(y2 == 17, torch.full_like(y, -100), y2)
    H, W = h.cuda(), w.cuda()
    a, b = q.qlora_head_loss_step(H, W, y2.cuda(), ignore_index=17), q.qlora_head_loss_step(H, W, y1.cuda())
    for x, z in zip(a, b):
        assert torch.equal(x, z)


def test_strided_rows_and_shifted_labels():
    T, V, D = 150, 600, 136
    h, w, y = _case(T, V, D, seed=8)
    buf = torch.full((T + 1, 200), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:T, 16:16 + D] = h.cuda()
    wbuf = torch.full((V, 160), float("nan"), dtype=torch.bfloat16, device="cuda")
    wbuf[:, 8:8 + D] = w.cuda()
    lab = torch.cat([torch.zeros(1, dtype=torch.int64), y]).cuda()
    H, W, Y = buf[:T, 16:16 + D], wbuf[:, 8:8 + D], lab[1:]
    g = torch.linspace(0, 1, T, device="cuda")
    dH = torch.full((T + 1, 152), 3.0, dtype=torch.bfloat16, device="cuda")
    a = q.qlora_head_loss_step(H, W, Y, weight=g, dH=dH[:T, 8:8 + D])
    b = q.qlora_head_loss_step(h.cuda(), w.cuda(), y.cuda(), weight=g)
    for x, z in zip(a, b):
        assert torch.equal(x, z)
    assert bool((dH[:, :8] == 3).all()) and bool((dH[:, 8 + D:] == 3).all()) and bool((dH[T] == 3).all())
    c = q.qlora_head_loss_bwd(H, W, Y, a[1], g, dH=dH[:T, 8:8 + D])
    assert torch.equal(c, q.qlora_head_loss_bwd(h.cuda(), w.cuda(), y.cuda(), b[1], g))


@pytest.mark.parametrize("T,V,D", [(40, 300, 64), (300, 700, 128), (16500, 4500, 64)])
def test_gradient_in_place_of_the_hidden_states(T, V, D):
    h, w, y = _case(T, V, D, seed=10)
    W, Y, g = w.cuda(), y.cuda(), torch.linspace(-1, 1, T, device="cuda")
    want = q.qlora_head_loss_step(h.cuda(), W, Y, weight=g)
    H = h.cuda()
    got = q.qlora_head_loss_step(H, W, Y, weight=g, dH=H)
    assert got[3].data_ptr() == H.data_ptr()
    for x, z in zip(got, want):
        assert torch.equal(x, z)
    H = h.cuda()
    dH = q.qlora_head_loss_bwd(H, W, Y, want[1], g, dH=H)
    assert torch.equal(dH, q.qlora_head_loss_bwd(h.cuda(), W, Y, want[1], g))


@pytest.mark.parametrize("T,nf4", [(40, True), (200, False), (200, True)])
def test_workspace_of_any_16_byte_alignment(T, nf4):
    h, w, y = _case(T, 700, 128, seed=11)
    H, Y, W = h.cuda(), y.cuda(), w.cuda()
    W = q.quantize_weight(W) if nf4 else W
    want = q.qlora_head_loss_step(H, W, Y)
    n = q.qlora_head_loss_workspace_size(T, 700, 128, nf4, q.HEAD_STEP)
    buf = torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda")
    for o in (16, 48, 240):
        got = q.qlora_head_loss_step(H, W, Y, ws=buf[o:o + n])
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert bool((buf[240 + n:] == 255).all())  # and nothing behind it


def test_gradient_against_differences_of_the_loss():
    """The gradient along a direction against the loss at two points on it."""
    h, w, y = _case(128, 700, 256, seed=9, lean=10.0)
    H, W, Y = h.float().cuda(), w.cuda(), y.cuda()
    dH = q.qlora_head_loss_step(h.cuda(), W, Y, weight=torch.ones(128, device="cuda"))[3].double()
    step = torch.sign(dH).float() * 0.0625
    up, down = (H + step).to(torch.bfloat16), (H - step).to(torch.bfloat16)
    lu, ld = (q.qlora_head_loss_fwd(x, W, Y)[0].double() for x in (up, down))
    moved = (up.double() - down.double())
    pred = (dH * moved).sum(1)
    # the second-order term cancels in a central difference; third order: |f'''| step^3 / 24 with
    # |l'| <= |W| |moved| / 2 summed over dim, and bf16 points are off the line by half a step of H
    reach = (moved.abs() @ W.double().abs().t()).amax(1) / 2
    skew = ((up.double() + down.double()) / 2 - H.double()).abs() @ W.double().abs().t()
    tol = reach ** 3 / 3 + 2 * reach * skew.amax(1) + 2.0 ** -7 * pred.abs() + 1e-5
    assert bool(((lu - ld - pred).abs() <= tol).all())


def test_refusals_on_device_tensors():
    h, w, y = _case(8, 50, 64)
    H, W, Y = h.cuda(), w.cuda(), y.cuda()
    g = torch.ones(8, device="cuda")
    N = q.quantize_weight(W)
    assert q.qlora_head_loss_fwd(H, N, Y)[0].shape == (8,)
    for bad in (N._replace(codes=N.codes[:-1]), N._replace(c8=N.c8[:-1]), N._replace(s2=N.s2[:0]),
                N._replace(n_out=51), N._replace(codes=N.codes.cpu()), N._replace(s2=N.s2.double())):
        with pytest.raises(q.QloraError):
            q.qlora_head_loss_fwd(H, bad, Y)
    for f in (lambda: q.qlora_head_loss_fwd(H, W[:, :56], Y), lambda: q.qlora_head_loss_fwd(H, W, Y[:7]),
              lambda: q.qlora_head_loss_fwd(H, W, Y.int()), lambda: q.qlora_head_loss_fwd(H, W, y),
              lambda: q.qlora_head_loss_fwd(H, W.float(), Y), lambda: q.qlora_head_loss_fwd(H.t(), W, Y),
              lambda: q.qlora_head_loss_fwd(H[:, :60], W[:, :60], Y),
              lambda: q.qlora_head_loss_bwd(H, W, Y, g, g[:1]), lambda: q.qlora_head_loss_bwd(H, W, Y, g.double(), g),
              lambda: q.qlora_head_loss_bwd(H, W, Y, g, g, stats=g[:2]),
              lambda: q.qlora_head_loss_step(H, W, Y, weight=g[:4]),
              lambda: q.qlora_head_loss_step(H, W, Y, dH=torch.zeros(8, 32, dtype=torch.bfloat16, device="cuda")),
              lambda: q.qlora_head_loss_step(H, W, Y, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(q.QloraError):
            f()


@pytest.mark.parametrize("T,V,D", [(40, 3000, 64), (300, 9000, 320)])
def test_label_logits_far_above_others_near_forty(T, V, D):
    """The others' logits 39 each, the label's 85 to 120: their share of the sum
    is 1e-17 to 1e-32, which fp32 and bf16 hold, and it is all there is of the
    gradient.  Every logit is exact, so x = (V - 1) exp(39 - l_label) is off by the
    exponential's argument (2^-23 of it, below 128 in two halves) and a few
    roundings, below 2^-15; the operand's and dH's roundings are 2^-8 each."""
    g = torch.Generator().manual_seed(16)
    w = torch.randn(V, D, generator=g) * 0.5
    w[:, 0], w[:, 1], w[V // 2, 1] = 1.0, 0.0, 1.0
    w = w.to(torch.bfloat16)
    h = torch.zeros(T, D)
    top = torch.linspace(85, 120, T).round()
    h[:, 0], h[:, 1] = 39.0, top - 39.0
    y = torch.full((T,), V // 2)
    share = np.exp(39.0 - top.double().numpy())
    others = w.double().numpy().sum(0) - w[V // 2].double().numpy()
    loss = np.log1p((V - 1) * share)
    ref = share[:, None] * (others - (V - 1) * w[V // 2].double().numpy()) / (1 + (V - 1) * share)[:, None]
    size = share[:, None] * (np.abs(w.double().numpy()).sum(0) + V * np.abs(w[V // 2].double().numpy()))
    H, W, Y = h.to(torch.bfloat16).cuda(), w.cuda(), y.cuda()
    got = q.qlora_head_loss_step(H, W, Y, weight=torch.ones(T, device="cuda"))
    for out in (q.qlora_head_loss_fwd(H, W, Y), got):
        assert np.all(np.abs(out[0].double().cpu().numpy() - loss) <= 2.0 ** -15 * loss)
    err = np.abs(got[3].double().cpu().numpy() - ref)
    assert np.all(err <= (2.0 ** -8 * 1.01 + 2.0 ** -14) * size + 2.0 ** -8 * np.abs(ref))


@pytest.mark.parametrize("T,V,D,nf4,std", [(64, 3000, 256, False, 2.0), (300, 9000, 320, False, 2.0),
                                           (1000, 70000, 64, False, 2.0), (2000, 12500, 1024, False, 2.0),
                                           (64, 3000, 256, False, 15.0), (2000, 12500, 1024, False, 15.0),
                                           (64, 3000, 256, True, 2.0), (520, 5000, 256, True, 2.0)])
def test_what_the_heads_rows_share_cancels(T, V, D, nf4, std):
    """Rows of W with a common part of 30 times their own: the coefficients of a
    row of dH sum to zero, rounded or not, so an error of p_v, whatever its cause,
    moves dH by W_v - W_label.  H has 8 columns, so a logit is off by at most
    d = 2 8 2^-24 sum |h w| (the others add zeros), p relatively by rel = 2 d +
    2^-20 (4 + max|l|), and by its rounding, 2^-8 (twice for a rescaled row).  What
    does not cancel: the fp32 sum over the vocabulary, at most 2^-23 of it a step of
    16 columns, and in the backward the error of expm1(l - lse), rel."""
    g = torch.Generator().manual_seed(17)
    w = 0.6 * torch.randn(D, generator=g) + 0.02 * torch.randn(V, D, generator=g)
    w[:, :8] = torch.randn(V, 8, generator=g)
    h = torch.zeros(T, D)
    h[:, :8] = std * torch.randn(T, 8, generator=g)
    H, W = h.to(torch.bfloat16).cuda(), w.to(torch.bfloat16).cuda()
    if nf4:
        N = q.quantize_weight(W)
        W = q.nf4_dequantize(N.codes, N.c8, N.s2, V * D).view(V, D)
    y = torch.topk(H.double() @ W.double().t(), 4, dim=1)[1][:, 1].clone()  # a likely token
    y[::4] = torch.randint(0, V, (T,), generator=g)[::4].cuda()
    y[1::8] = -100
    gr = torch.linspace(-1, 2, T, device="cuda")
    lse = q.qlora_head_loss_fwd(H, N if nf4 else W, y)[1]
    back = q.qlora_head_loss_bwd(H, N if nf4 else W, y, lse, gr)
    step = q.qlora_head_loss_step(H, N if nf4 else W, y, weight=gr)[3]

    rows = torch.nonzero(y != -100)[:, 0]
    rows = rows[torch.linspace(0, rows.numel() - 1, min(150, rows.numel()), device="cuda").long()]
    x, v, t = H[rows].double(), W.double(), gr[rows].double()[:, None]
    z = x @ v.t()
    p = torch.softmax(z, 1).scatter(1, y[rows, None], 0.0)
    wy = v[y[rows]]
    ref = t * (p @ v - p.sum(1, keepdim=True) * wy)
    apart = torch.stack([(p[i, :, None] * (v - wy[i]).abs()).sum(0) for i in range(len(rows))])
    size = p @ v.abs() + p.sum(1, keepdim=True) * wy.abs()
    rel = 2 * 16 * 2.0 ** -24 * (x.abs() @ v.abs().t()).amax(1) + 2.0 ** -20 * (4 + z.abs().amax(1))
    for d, rounds, leak in ((back, 1, rel[:, None] * wy.abs()), (step, 2 if std > 2 else 1, 0)):
        tol = t.abs() * ((rounds * 2.0 ** -8 * 1.01 + 2 * rel[:, None]) * apart + (V / 16 + 8) * 2.0 ** -23 * size
                         + leak) + 2.0 ** -8 * ref.abs() + 1e-37
        assert bool(((d[rows].double() - ref).abs() <= tol).all())
        assert not d[y == -100].any()


@pytest.mark.parametrize("T,V,D", [(40, 300, 64), (300, 5000, 128), (600, 20000, 2304)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_backward_reports_a_non_finite_lse(T, V, D, bad):
    """Of a token that counts; its row only is lost.  The last size lists its rows."""
    h, w, y = _case(T, V, D, seed=18, ignored=0.0)
    y[5] = -100
    H, W, Y, g = h.cuda(), w.cuda(), y.cuda(), torch.ones(T, device="cuda")
    lse = q.qlora_head_loss_fwd(H, W, Y)[1]
    want = q.qlora_head_loss_bwd(H, W, Y, lse, g)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    lse[5] = bad                                          # an ignored token's is not read
    assert torch.equal(q.qlora_head_loss_bwd(H, W, Y, lse, g, status=status), want) and int(status[0]) == 0
    lse[T - 2] = bad
    got = q.qlora_head_loss_bwd(H, W, Y, lse, g, status=status)
    assert int(status[0]) == q.DEV_NONFINITE
    keep = torch.arange(T, device="cuda") != T - 2
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("T,V,D", [(40, 300, 64), (600, 20000, 2304)])
def test_gradients_of_the_losses_as_autograd_gives_them(T, V, D):
    """Of a sum (one element expanded), of a mean (no dimension), and a column of a
    matrix; the loss as a node of autograd."""
    h, w, y = _case(T, V, D, seed=19)
    H, W, Y = h.cuda(), w.cuda(), y.cuda()
    loss, lse, stats = q.qlora_head_loss_fwd(H, W, Y)
    two = torch.full((1,), 2.0, device="cuda")
    want = q.qlora_head_loss_bwd(H, W, Y, lse, two.repeat(T))
    assert torch.equal(q.qlora_head_loss_bwd(H, W, Y, lse, two.expand(T)), want)
    g = torch.rand(T, 3, device="cuda")
    assert torch.equal(q.qlora_head_loss_bwd(H, W, Y, lse, g[:, 1]),
                       q.qlora_head_loss_bwd(H, W, Y, lse, g[:, 1].contiguous()))
    mean = q.qlora_head_loss_bwd(H, W, Y, lse, two, stats=stats)
    assert torch.equal(q.qlora_head_loss_bwd(H, W, Y, lse, two[0], stats=stats), mean)

    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, reduce):
            loss, lse, stats = q.qlora_head_loss_fwd(x, W, Y)
            ctx.save_for_backward(x, lse, stats)
            ctx.reduce = reduce
            return stats[0].clone() if reduce else loss

        @staticmethod
        def backward(ctx, grad):
            x, lse, stats = ctx.saved_tensors
            return q.qlora_head_loss_bwd(x, W, Y, lse, grad, stats=stats if ctx.reduce else None), None

    for reduce, ref in ((False, want), (True, mean)):
        x = H.clone().requires_grad_()
        (2 * Loss.apply(x, reduce).sum()).backward()
        assert torch.equal(x.grad, ref)
    for bad in (two.expand(T + 1), two[0], two.double().expand(T), two.cpu().expand(T)):
        with pytest.raises(q.QloraError):
            q.qlora_head_loss_bwd(H, W, Y, lse, bad)
    for bad in (two.repeat(2), two.view(1, 1), two[0].double()):
        with pytest.raises(q.QloraError):
            q.qlora_head_loss_bwd(H, W, Y, lse, bad, stats=stats)


@pytest.mark.parametrize("T,V,D,nf4", [(600, 20000, 2304, False), (2000, 12500, 1024, False), (1153, 5000, 4416, True)])
def test_rows_that_count_are_rounded_once(T, V, D, nf4):
    """Logits within +-40: no exponential is rescaled, in the backward none ever."""
    assert T > 256 and 4.0 * T * V * D >= 1e11
    h, w, y = _case(T, V, D, seed=20, lean=5.0)
    H, Y, W = h.cuda(), y.cuda(), w.cuda()
    if nf4:
        W = q.quantize_weight(W)
        w = q.nf4_dequantize(W.codes, W.c8, W.s2, V * D).view(V, D).cpu()
    count = torch.nonzero(y != -100)[:, 0]
    rows = count[torch.linspace(0, count.numel() - 1, 100).long()]
    r, sel, g = Ref(h[rows], w, y[rows]), rows.cuda(), torch.linspace(-1, 2, T)
    _, lse, _, dH = q.qlora_head_loss_step(H, W, Y, weight=g.cuda())
    r.check_grad(dH[sel], g.numpy()[rows], roundings=1)
    r.check_grad(q.qlora_head_loss_bwd(H, W, Y, lse, g.cuda())[sel], g.numpy()[rows], roundings=1)


@pytest.mark.parametrize("T,V,D", [(5, 600001, 64), (130, 300000, 128)])
def test_few_tokens_and_a_large_vocabulary(T, V, D):
    """A contraction over several hundred thousand columns."""
    h, w, y = _case(T, V, D, seed=21, lean=10.0)
    n = min(T, 40)
    r = Ref(h[:n], w, y[:n])
    H, W, Y, g = h.cuda(), w.cuda(), y.cuda(), torch.linspace(-1, 2, T)
    loss, lse, _, dH = q.qlora_head_loss_step(H, W, Y, weight=g.cuda())
    assert np.all(np.abs(loss[:n].cpu().numpy() - r.loss) <= r.loss_tol)
    r.check_grad(dH[:n], g.numpy()[:n])
    r.check_grad(q.qlora_head_loss_bwd(H, W, Y, lse, g.cuda())[:n], g.numpy()[:n])


@pytest.mark.parametrize("T,V,D", [(40, 300, 64), (600, 20000, 2304)])
def test_label_logit_that_overflows(T, V, D):
    """lse - l of infinities is no number: neither is the loss, nor the row of dH."""
    h, w, y = _case(T, V, D, seed=22, ignored=0.0)
    h[3], w[7], y[3] = 0.0, 0.0, 7
    y[y == 7], y[3] = 8, 7
    H, W, Y, g = h.cuda(), w.cuda(), y.cuda(), torch.ones(T, device="cuda")
    want = q.qlora_head_loss_step(H, W, Y, weight=g)
    H[3, 1] = W[7, 1] = 1e30
    W[:7, 1], W[8:, 1] = 0.0, 0.0
    H[torch.arange(T, device="cuda") != 3, 1] = 0.0
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    step = q.qlora_head_loss_step(H, W, Y, weight=g, status=status)
    assert int(status[0]) == q.DEV_NONFINITE
    loss, lse, stats = q.qlora_head_loss_fwd(H, W, Y)
    for v in (step[0][3], step[1][3], step[2][0], loss[3], lse[3], stats[0]):
        assert not torch.isfinite(v)
    assert torch.isnan(step[0][3]) and torch.isnan(loss[3]) and torch.isnan(step[3][3]).all()
    keep = torch.arange(T, device="cuda") != 3
    assert bool(torch.isfinite(step[0][keep]).all()) and bool(torch.isfinite(step[3][keep].float()).all())
    assert bool(torch.isfinite(want[0]).all())
