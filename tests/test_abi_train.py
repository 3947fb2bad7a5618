"""Host-only checks of include/qlora_train.h: exported symbols, workspace sizes,
and every refusal of the C ABI and of the binding, before a device is touched.
No GPU needed; no test here enqueues device work."""

import ctypes
import os
import re

import pytest
import torch

import bit_nf4_quantized_26_b200 as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, WS, DTYPE = 0, 1, 2, 3, 4, 9
FAKE = 1 << 20  # a 16-byte aligned non-null value; never dereferenced


def test_header_declarations_are_exported():
    text = open(os.path.join(ROOT, "include", "qlora_train.h")).read()
    names = sorted(set(re.findall(r"QLORA_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)))
    assert sorted(q.EXPORTED_TRAIN) == names and len(names) == 10
    for n in names:
        assert hasattr(q.raw(), n), n


def _quant(X=FAKE, M=4, K=128, ld=128, codes=FAKE, exps=FAKE, status=None):
    return q.raw().act8_quantize(X, M, K, ld, codes, exps, status, None)


def _dequant(codes=FAKE, exps=FAKE, M=4, K=128, X=FAKE, ld=128):
    return q.raw().act8_dequantize(codes, exps, M, K, X, ld, None)


@pytest.mark.parametrize("f", [_quant, _dequant])
def test_act8_refusals(f):
    assert f(M=-1) == SHAPE and f(M=1 << 31) == SHAPE
    assert f(K=0) == SHAPE and f(K=96) == SHAPE and f(K=32) == SHAPE
    assert f(ld=120) == SHAPE and f(ld=132) == SHAPE and f(ld=1 << 31) == SHAPE
    assert f(M=1 << 30, K=1024, ld=1024) == SHAPE
    assert f(X=None) == NULL and f(codes=None) == NULL and f(exps=None) == NULL
    assert f(X=FAKE + 8) == ALIGN and f(codes=FAKE + 4) == ALIGN and f(exps=FAKE + 1) == ALIGN
    assert f(M=0, X=None, codes=None, exps=None) == OK
    assert f(M=0, K=65) == SHAPE


def _w(n=4096, k=4096):
    return q._NF4Weight(FAKE, FAKE, FAKE, n, k)


def _bwd(codes=FAKE, exps=FAKE, M=64, W=None, r=64, dX=FAKE, dt=0, wsb=1 << 40, dA=FAKE):
    return q.raw().qlora_linear_bwd_act8(FAKE, codes, exps, FAKE, M, _w() if W is None else W, FAKE, FAKE, r, 0.25, dX,
                                         dt, dA, FAKE, FAKE, wsb, None, None)


def test_bwd_act8_refusals_are_the_backwards():
    assert _bwd(codes=None) == NULL and _bwd(exps=None) == NULL and _bwd(dX=None) == NULL
    assert _bwd(codes=FAKE + 8) == ALIGN and _bwd(exps=FAKE + 8) == ALIGN and _bwd(dA=FAKE + 4) == ALIGN
    assert _bwd(r=8) == SHAPE and _bwd(r=272) == SHAPE and _bwd(W=_w(k=100)) == SHAPE and _bwd(M=-1) == SHAPE
    assert _bwd(dt=3) == DTYPE and _bwd(wsb=16) == WS
    assert _bwd(M=0, codes=None) == OK
    members = ctypes.cast((ctypes.c_int64 * 2)(4096, 4096), ctypes.c_void_p)

    def group(G=2, nm=members, r=64, codes=FAKE, wsb=1 << 40):
        return q.raw().qlora_group_bwd_act8(FAKE, codes, FAKE, FAKE, 64, _w(n=8192), G, nm, FAKE, FAKE, r, 0.25, FAKE,
                                            0, FAKE, FAKE, FAKE, wsb, None, None)

    assert group(G=0) == SHAPE and group(G=5) == SHAPE and group(nm=None) == NULL and group(r=128) == SHAPE
    assert group(codes=None) == NULL and group(wsb=0) == WS

    def drop(p, codes=FAKE):
        return q.raw().qlora_linear_bwd_dropout_act8(FAKE, codes, FAKE, FAKE, 64, _w(), FAKE, FAKE, 64, 0.25, p, 7,
                                                     FAKE, 0, FAKE, FAKE, FAKE, 16, None, None)

    assert drop(1.0) == SHAPE and drop(-0.5) == SHAPE and drop(float("nan")) == SHAPE
    assert drop(0.5, codes=None) == NULL and drop(0.5) == WS


def test_bwd_act8_workspace_size():
    f, g = q.qlora_bwd_act8_workspace_size, q.qlora_group_bwd_workspace_size
    assert f(0, 4096, 4096, 1, 64) == 0 and f(64, 4096, 4096, 0, 64) == 0 and f(64, 4096, 4096, 5, 64) == 0
    assert f(4096, 4096, 4096, 1, 64) == q.qlora_bwd_workspace_size(4096, 4096, 4096, 64) + 8 * 4096 * 64
    assert f(1000, 8192, 512, 2, 16) <= g(1000, 8192, 512, 2, 16) + 8 * 1000 * 2 * 16 + 512
    assert f(64, 512, 256, 1, 16, True) == f(64, 512, 256, 1, 16) + 64 * 256 * 4
    assert _bwd(wsb=f(64, 4096, 4096, 1, 64) - 1) == WS


def _h(w=FAKE, ld=512, V=1000, D=512, codes=None, c8=None, s2=None, mean=None):
    return q._Head(w, ld, codes, c8, s2, mean, V, D)


def _nf4(V=1000, D=512, codes=FAKE, c8=FAKE, s2=FAKE, mean=None):
    return q._Head(None, 0, codes, c8, s2, mean, V, D)


def _lf(H=FAKE, ldh=512, T=10, head=None, labels=FAKE, loss=FAKE, lse=FAKE, stats=FAKE, ws=FAKE, wsb=1 << 40,
        status=None):
    return q.raw().qlora_head_loss_fwd(H, ldh, T, _h() if head is None else head, labels, -100, loss, lse, stats, ws,
                                       wsb, status, None)


def _lb(H=FAKE, ldh=512, T=10, head=None, labels=FAKE, lse=FAKE, dloss=FAKE, stats=None, dH=FAKE, lddh=512, ws=FAKE,
        wsb=1 << 40, status=None):
    return q.raw().qlora_head_loss_bwd(H, ldh, T, _h() if head is None else head, labels, -100, lse, dloss, stats, dH,
                                       lddh, ws, wsb, status, None)


def _ls(H=FAKE, ldh=512, T=10, head=None, labels=FAKE, weight=None, loss=FAKE, lse=FAKE, stats=FAKE, dH=FAKE,
        lddh=512, ws=FAKE, wsb=1 << 40, status=None):
    return q.raw().qlora_head_loss_step(H, ldh, T, _h() if head is None else head, labels, -100, weight, 1.0, loss,
                                        lse, stats, dH, lddh, ws, wsb, status, None)


@pytest.mark.parametrize("f", [_lf, _lb, _ls])
def test_head_loss_refusals(f):
    assert f(T=-1) == SHAPE and f(T=1 << 31) == SHAPE
    assert f(head=_h(V=0)) == SHAPE and f(head=_h(V=1 << 31)) == SHAPE
    assert f(head=_h(D=4)) == SHAPE and f(head=_h(D=508)) == SHAPE and f(head=_h(D=1 << 21, ld=1 << 21)) == SHAPE
    assert f(head=_nf4(D=520)) == SHAPE                       # NF4 blocks never cross rows
    assert f(head=_h(ld=504)) == SHAPE and f(head=_h(ld=516)) == SHAPE
    assert f(ldh=504) == SHAPE and f(ldh=516) == SHAPE
    assert f(T=1 << 30, head=_h(V=1 << 30)) == SHAPE          # more tiles than are counted
    assert f(H=None) == NULL and f(labels=None) == NULL and f(lse=None) == NULL
    assert f(head=_nf4(codes=None)) == NULL and f(head=_nf4(c8=None)) == NULL and f(head=_nf4(s2=None)) == NULL
    assert f(H=FAKE + 8) == ALIGN and f(head=_h(w=FAKE + 8)) == ALIGN and f(labels=FAKE + 4) == ALIGN
    assert f(lse=FAKE + 2) == ALIGN and f(head=_nf4(mean=FAKE + 4)) == ALIGN and f(status=FAKE + 4) == ALIGN
    assert f(ws=None) == WS and f(wsb=64) == WS and f(ws=FAKE + 8) == ALIGN
    assert f(labels=FAKE + 8, wsb=64) == WS                   # a shifted view of the labels is fine


def test_head_loss_refusals_of_single_operators():
    assert _lf(loss=None) == NULL and _lf(stats=None) == NULL and _lf(stats=FAKE + 1) == ALIGN
    assert _lb(dloss=None) == NULL and _lb(dH=None) == NULL and _lb(dH=FAKE + 8) == ALIGN and _lb(lddh=504) == SHAPE
    assert _ls(dH=None) == NULL and _ls(lddh=500) == SHAPE and _ls(weight=FAKE + 2) == ALIGN
    assert _lb(T=0, H=None, labels=None, dH=None) == OK
    assert _lf(T=0, stats=None) == NULL


def test_head_loss_workspace_sizes():
    f = q.qlora_head_loss_workspace_size
    assert f(0, 1000, 512, False, q.HEAD_FWD) == 0 and f(10, 1000, 512, False, 3) == 0
    assert f(10, 1000, 520, True, q.HEAD_FWD) == 0            # a shape the calls refuse
    # forward: 8 bytes per 128 logits and per-token words, no logits
    T, V = 8192, 128000
    assert 8 * T * V // 128 <= f(T, V, 4096, False, q.HEAD_FWD) <= 8 * T * V // 128 + 16 * T + 4096
    # backward and step: bounded in the vocabulary
    for op in (q.HEAD_BWD, q.HEAD_STEP):
        rows = 2 * T * 4096 if op == q.HEAD_BWD else 0       # the rows that count
        parts = 74 * 4 * 256 * 256                           # one tile's sums more per CTA pair
        # piece, sum, statistics
        assert f(T, V, 4096, False, op) <= (1 << 27) + 4 * T * 4096 + parts + rows + (1 << 23)
        assert f(T, 4 * V, 4096, False, op) <= f(T, V, 4096, False, op) + (1 << 20)
    assert f(T, V, 4096, True, q.HEAD_BWD) - f(T, V, 4096, False, q.HEAD_BWD) <= 1 << 27


# ------------------------------------------------------------- the binding


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_wrong_tensors():
    with pytest.raises(q.QloraError, match="float32") as e:
        q.act8_quantize(_cpu(4, 64, dtype=torch.float32))
    assert e.value.code == DTYPE
    for bad in (_cpu(4, 64), _cpu(64)):                       # on the CPU; one dimension
        with pytest.raises(q.QloraError) as e:
            q.act8_quantize(bad)
        assert e.value.code == SHAPE
    with pytest.raises(q.QloraError):
        q.act8_dequantize(q.Act8(_cpu(4, 64, dtype=torch.uint8), _cpu(4, 1, dtype=torch.uint8)))
    H, W, y = _cpu(4, 64), _cpu(100, 64), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: q.qlora_head_loss_fwd(H, W, y), lambda: q.qlora_head_loss_step(H.float(), W, y),
                 lambda: q.qlora_head_loss_bwd(H, W, y, None, None)):
        with pytest.raises(q.QloraError):
            call()


@pytest.mark.parametrize("dY", [_cpu(64), torch.zeros((), dtype=torch.bfloat16), _cpu(2, 4, 64), _cpu(4, 64)])
def test_binding_refuses_other_gradients(dY):
    """Not a matrix, or not on a GPU: an error of the library, not Python's."""
    class W:
        n_out, k_in = 64, 64
    X8 = q.Act8(_cpu(4, 64, dtype=torch.uint8), _cpu(4, 1, dtype=torch.uint8))
    for f, more in ((q.qlora_linear_bwd_act8, ()), (q.qlora_linear_bwd_dropout_act8, (0.1, 3))):
        with pytest.raises(q.QloraError) as e:
            f(dY, X8, _cpu(4, 8, dtype=torch.float32), W, _cpu(8, 64), _cpu(64, 8), 1.0, *more)
        assert e.value.code == SHAPE
