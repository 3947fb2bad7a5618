"""The training-step operators together, as a user runs them: an adapted NF4
linear, its input kept in 8 bits, the loss head's loss and gradient, the
backward pass from the checkpoint and the 8-bit AdamW step; eagerly, captured
and replayed, on another stream, and two at once."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_26_b200 as q
from oracle import head_loss as hl
from tests._util import bits

pytestmark = pytest.mark.gpu


class Step:
    """One projection under a loss head, with every buffer of its own."""

    def __init__(self, M, K, D, V, r, nf4, seed):
        g = torch.Generator().manual_seed(seed)

        def rnd(*shape, std=1.0):
            return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()

        self.M, self.K, self.D, self.V, self.r, self.s = M, K, D, V, r, 16.0 / r
        self.X = rnd(M, K)
        self.W = q.quantize_weight(rnd(D, K, std=K ** -0.5))
        self.A, self.B = rnd(r, K, std=K ** -0.5), rnd(D, r, std=0.02)
        head = rnd(V, D, std=0.02)
        self.head = q.quantize_weight(head) if nf4 else head
        self.dense = q.nf4_dequantize(self.head.codes, self.head.c8, self.head.s2, V * D).view(V, D) if nf4 else head
        y = torch.randint(0, V, (M,), generator=g)
        self.y = torch.where(torch.rand(M, generator=g) < 0.3, torch.full_like(y, -100), y).cuda()
        e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        b16, u8 = torch.bfloat16, torch.uint8
        self.Y, self.U = e(M, D, dt=b16), e(M, r)
        self.x8 = q.Act8(e(M, K, dt=u8), e(M, K // 64, dt=u8))
        self.loss, self.lse, self.stats, self.dY = e(M), e(M), e(2), e(M, D, dt=b16)
        self.dX, self.dA, self.dB = e(M, K, dt=b16), e(r, K), e(D, r)
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        size = max(q.qlora_fwd_workspace_size(M, D, K, r), q.qlora_bwd_act8_workspace_size(M, D, K, 1, r),
                   q.qlora_head_loss_workspace_size(M, V, D, nf4, q.HEAD_STEP), 16)
        self.ws = e(size, dt=u8)

    def run(self, stream=None):
        k = dict(ws=self.ws, status=self.status, stream=stream)
        q.qlora_linear_fwd(self.X, self.W, self.A, self.B, self.s, Y=self.Y, U=self.U, **k)
        q.act8_quantize(self.X, *self.x8, status=self.status, stream=stream)
        q.qlora_head_loss_step(self.Y, self.head, self.y, loss=self.loss, lse=self.lse, stats=self.stats, dH=self.dY,
                               **k)
        q.qlora_linear_bwd_act8(self.dY, self.x8, self.U, self.W, self.A, self.B, self.s, dX=self.dX, dA=self.dA,
                                dB=self.dB, **k)

    def outputs(self):
        return {n: getattr(self, n).clone() for n in ("Y", "U", "loss", "lse", "stats", "dY", "dX", "dA", "dB")}

    def clear(self):
        for n in ("Y", "U", "loss", "lse", "stats", "dY", "dX", "dA", "dB"):
            getattr(self, n).fill_(-7)


def _same(a, b):
    return all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)


SIZES = [(40, 256, 512, 1000, 16), (333, 320, 256, 3001, 64)]


@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("M,K,D,V,r", SIZES)
def test_chain_matches_oracle(M, K, D, V, r, nf4):
    """Each link against fp64 on the values that the link before it gave."""
    st = Step(M, K, D, V, r, nf4, 1)
    st.run()
    out = st.outputs()
    assert int(st.status[0]) == 0
    y = st.y.cpu().numpy()
    loss, lse, mean, n = hl.fwd(bits(out["Y"]), bits(st.dense), y)
    assert np.abs(out["loss"].cpu().numpy() - loss).max() <= 1e-4 and int(out["stats"][1]) == n
    assert abs(float(out["stats"][0]) - mean) <= 1e-5 * mean
    ref = hl.bwd(bits(out["Y"]), bits(st.dense), y, np.full(M, 1.0 / n))
    assert np.linalg.norm(out["dY"].double().cpu().numpy() - ref) <= 5e-3 * np.linalg.norm(ref)
    dY, B = out["dY"].double(), st.B.double()
    dU = st.s * (dY @ B)
    x = q.act8_dequantize(st.x8).double()
    for got, want in ((out["dA"], dU.t() @ x), (out["dB"], st.s * (dY.t() @ out["U"].double()))):
        assert float((got.double() - want).norm() / want.norm()) <= 4e-6
    assert not out["dX"][st.y == -100].any()
    # what the 8-bit input costs dA: E4M3's half step, 2^-4 relative an element, averaged over the tokens
    full = dU.t() @ st.X.double()
    assert float((out["dA"].double() - full).norm() / full.norm()) <= 2.0 ** -4


def test_ten_steps_with_the_optimizer():
    """Ten steps with the optimizer: finite, and the adapters move."""
    st = Step(128, 256, 256, 500, 16, False, 2)
    A0 = st.A.clone()
    flat = st.A.view(-1)
    opt = q.AdamW8State(flat.numel(), paged=False)
    for i in range(10):
        st.run()
        q.qlora_adamw8_step(flat, st.dA.view(-1), opt, lr=1e-3, step=i + 1, status=st.status)
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0 and bool(torch.isfinite(st.loss).all()) and not torch.equal(st.A, A0)


@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("M,K,D,V,r", SIZES)
def test_captured_and_replayed(M, K, D, V, r, nf4):
    st = Step(M, K, D, V, r, nf4, 3)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        st.run()
    torch.cuda.synchronize()
    want = st.outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        st.run()
    for _ in range(2):
        st.clear()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(st.outputs(), want)
    # other data in the same buffers
    st.X.copy_(st.X.flip(0))
    st.y.copy_(st.y.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    got = st.outputs()
    st.clear()
    st.run()
    assert _same(got, st.outputs())


def test_two_graphs_share_a_workspace():
    a, b = Step(40, 256, 512, 1000, 16, False, 4), Step(333, 320, 256, 3001, 64, True, 5)
    a.ws = b.ws = max(a.ws, b.ws, key=lambda t: t.numel())
    want, graphs = [], []
    stream = torch.cuda.Stream()
    for st in (a, b):
        with torch.cuda.stream(stream):
            st.run()
        torch.cuda.synchronize()
        want.append(st.outputs())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            st.run()
        graphs.append(graph)
    for st in (a, b):
        st.clear()
    b.ws.fill_(255)
    for k in (0, 1, 1, 0, 1):
        graphs[k].replay()
    torch.cuda.synchronize()
    assert _same(a.outputs(), want[0]) and _same(b.outputs(), want[1])


def test_two_at_once():
    """Two steps in flight on two streams, each with its own workspace."""
    steps = [Step(333, 320, 256, 3001, 64, False, 6), Step(100, 256, 512, 9000, 16, True, 7)]
    want = []
    for st in steps:
        st.run()
        torch.cuda.synchronize()
        want.append(st.outputs())
        st.clear()
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, s in zip(steps, streams):
            st.run(stream=s)
    torch.cuda.synchronize()
    for st, w in zip(steps, want):
        assert _same(st.outputs(), w)


def test_outputs_of_a_call_on_another_stream():
    """Outputs and workspace that the call allocates belong to the stream it runs on."""
    st = Step(333, 320, 256, 3001, 64, True, 8)
    st.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = q.qlora_head_loss_step(st.Y, st.head, st.y, stream=side)
    x8 = q.act8_quantize(st.X, stream=side)
    bwd = q.qlora_linear_bwd_act8(got[3], x8, st.U, st.W, st.A, st.B, st.s, stream=side)
    junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(8)]  # this stream's allocations meanwhile
    side.synchronize()
    assert torch.equal(got[3], st.dY) and torch.equal(x8.codes, st.x8.codes)
    assert torch.equal(bwd[1], st.dA) and torch.equal(bwd[2], st.dB)
    del junk


def test_shared_dirty_workspace_and_order_of_calls():
    """Results do not depend on what the workspace held."""
    st = Step(333, 320, 256, 3001, 64, False, 9)
    st.run()
    torch.cuda.synchronize()
    want = st.outputs()
    for fill in (0, 255, 127):
        st.ws.fill_(fill)
        st.clear()
        st.run()
        torch.cuda.synchronize()
        assert _same(st.outputs(), want)


@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("M,K,D,V,r", SIZES)
def test_chain_gradients_against_differences(M, K, D, V, r, nf4):
    """dA, dB and dX of the chain along a direction E against the mean loss in fp64
    at two points Y +- h (dY/dparameter E) around the chain's own Y.  Off by dY's
    errors, of which an element's is at most 2^-8 of itself and 2^-8 of g sum p_v
    |W_v - W_label|; by dX's own rounding, 2^-8, dU's bf16 pair and the GEMM's sum
    (2^-16 each at most); and the difference's third-order term, below 1e-5 as h
    moves a logit by 2e-3 at most."""
    st = Step(M, K, D, V, r, nf4, 10)
    st.run()
    out = st.outputs()
    Y, head, y = out["Y"].double(), st.dense.double(), st.y
    c = torch.nonzero(y != -100)[:, 0]

    def mean_loss(Y):
        z = Y @ head.t()
        return (torch.logsumexp(z[c], 1) - z[c, y[c]]).mean()
    z = Y[c] @ head.t()
    p = torch.softmax(z, 1)
    ref = (p.scatter_add(1, y[c, None], -torch.ones_like(p[:, :1])) @ head) / len(c)
    apart = torch.stack([(p[i, :, None] * (head - head[y[t]]).abs()).sum(0) for i, t in enumerate(c)]) / len(c)
    off = torch.zeros_like(Y)
    off[c] = 2.0 ** -8 * 1.02 * (ref.abs() + apart)
    W = q.nf4_dequantize(st.W.codes, st.W.c8, st.W.s2, D * K).view(D, K).double()
    A, B, U, x = st.A.double(), st.B.double(), out["U"].double(), q.act8_dequantize(st.x8).double()
    for grad, own, move in ((out["dA"], 1e-5, lambda E: st.s * (x @ E.t()) @ B.t()),
                            (out["dB"], 1e-5, lambda E: st.s * U @ E.t()),
                            (out["dX"], 2.0 ** -8 * 1.02, lambda E: E @ W.t() + st.s * (E @ A.t()) @ B.t())):
        E = torch.sign(grad.double())
        dy = move(E)
        h = 1e-3 / float((dy.abs() @ head.abs().t()).max())
        slope = float(mean_loss(Y + h * dy) - mean_loss(Y - h * dy)) / (2 * h)
        pred = float((grad.double() * E).sum())
        tol = float((off * dy.abs()).sum()) + (own + 1e-5) * pred
        assert abs(pred - slope) <= tol and tol < 0.2 * pred
