"""Python binding of ``libqlora_nf4.so`` (the C ABI in ``include/qlora_nf4.h``,
``include/qlora_optim.h`` and ``include/qlora_train.h``).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  PyTorch provides device memory and the current
stream.  There is no CPU fallback: if the shared library is missing the
import fails, and every non-OK status raises :class:`QloraError`.

Functions keep the C names:

* :func:`nf4_quantize` / :func:`nf4_dequantize`
* :func:`qlora_linear_fwd` / :func:`qlora_linear_bwd`
* :func:`qlora_fwd_workspace_size` / :func:`qlora_bwd_workspace_size`
* :func:`nf4_levels`, :func:`qlora_strerror`
* :func:`qlora_adamw8_step` with :class:`AdamW8State` (``include/qlora_optim.h``)
* :func:`qlora_head_loss_fwd` / :func:`qlora_head_loss_bwd` /
  :func:`qlora_head_loss_step`, :func:`act8_quantize` / :func:`act8_dequantize`
  and the ``*_bwd_act8`` backward passes (``include/qlora_train.h``)
"""

import ctypes
import os
from collections import namedtuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora_nf4.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python bit_nf4_quantized_26_b200/build.py`")

_lib = ctypes.CDLL(LIB_PATH)

DTYPE_BF16 = 0
DTYPE_F32 = 1
DEV_NONFINITE = 1
DEV_TIMEOUT = 2

STATUS = {0: "QLORA_OK", 1: "QLORA_ERR_NULL", 2: "QLORA_ERR_SHAPE", 3: "QLORA_ERR_ALIGN",
          4: "QLORA_ERR_WORKSPACE", 5: "QLORA_ERR_NONFINITE", 6: "QLORA_ERR_TIMEOUT",
          7: "QLORA_ERR_CUDA", 8: "QLORA_ERR_ARCH", 9: "QLORA_ERR_DTYPE", 10: "QLORA_ERR_INTERNAL"}


class QloraError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)} ({qlora_strerror(code)})")


class _NF4Weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("c8", ctypes.c_void_p), ("s2", ctypes.c_void_p),
                ("n_out", ctypes.c_int64), ("k_in", ctypes.c_int64), ("mean", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t

_lib.nf4_quantize.argtypes = [_P, _I64, _P, _P, _P, _P, _P]
_lib.nf4_quantize.restype = ctypes.c_int
_lib.nf4_dequantize.argtypes = [_P, _P, _P, _I64, _P, _P]
_lib.nf4_dequantize.restype = ctypes.c_int
_lib.qlora_linear_fwd.argtypes = [_P, _I64, _NF4Weight, _P, _P, _I32, ctypes.c_float, _P, _I32, _P, _P, _SZ,
                                  _P, _P]
_lib.qlora_linear_fwd.restype = ctypes.c_int
_lib.qlora_linear_bwd.argtypes = [_P, _P, _P, _I64, _NF4Weight, _P, _P, _I32, ctypes.c_float, _P, _I32, _P, _P,
                                  _P, _SZ, _P, _P]
_lib.qlora_linear_bwd.restype = ctypes.c_int
_lib.qlora_fwd_workspace_size.argtypes = [_I64, _I64, _I64, _I32]
_lib.qlora_fwd_workspace_size.restype = _SZ
_lib.qlora_bwd_workspace_size.argtypes = [_I64, _I64, _I64, _I32]
_lib.qlora_bwd_workspace_size.restype = _SZ
_lib.nf4_levels.argtypes = [_P]
_lib.nf4_levels.restype = None
_lib.qlora_strerror.argtypes = [ctypes.c_int]
_lib.qlora_strerror.restype = ctypes.c_char_p
_lib.qlora_linear_fwd_noalloc.argtypes = [_P, _I64, _NF4Weight, _P, _P, _I32, ctypes.c_float, _P, _I32, _P, _P,
                                          _P]
_lib.qlora_linear_fwd_noalloc.restype = ctypes.c_int
_lib.qlora_profile_enable.argtypes = [_I32]
_lib.qlora_profile_enable.restype = None
_lib.qlora_profile_collect.argtypes = [_P, _P, _I32]
_lib.qlora_profile_collect.restype = _I32
_lib.qlora_kernel_name.argtypes = [_I32]
_lib.qlora_kernel_name.restype = ctypes.c_char_p

EXPORTED = ("nf4_quantize", "nf4_dequantize", "qlora_linear_fwd", "qlora_linear_bwd",
            "qlora_fwd_workspace_size", "qlora_bwd_workspace_size", "nf4_levels", "qlora_strerror",
            "qlora_profile_enable", "qlora_profile_collect", "qlora_kernel_name", "qlora_linear_fwd_noalloc")

# mean: None for the plain double quantisation, or the 1-element fp32 device
# tensor of a weight quantised with nf4_quantize_centered.
NF4Weight = namedtuple("NF4Weight", "codes c8 s2 n_out k_in mean", defaults=(None,))


def qlora_strerror(code):
    return _lib.qlora_strerror(int(code)).decode()


def nf4_levels():
    """The 16 fp32 NF4 levels the library's kernels use (host-only query)."""
    buf = (ctypes.c_float * 16)()
    _lib.nf4_levels(ctypes.cast(buf, _P))
    return [float(v) for v in buf]


def qlora_fwd_workspace_size(M, N, K, r):
    return int(_lib.qlora_fwd_workspace_size(M, N, K, r))


def qlora_bwd_workspace_size(M, N, K, r):
    return int(_lib.qlora_bwd_workspace_size(M, N, K, r))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(code, where):
    if code != 0:
        raise QloraError(code, where)


def _weight(W):
    mean = getattr(W, "mean", None)
    return _NF4Weight(W.codes.data_ptr(), W.c8.data_ptr(), W.s2.data_ptr(), int(W.n_out), int(W.k_in),
                      None if mean is None else mean.data_ptr())


def nf4_sizes(numel):
    """(codes bytes, c8 bytes, s2 floats) of the NF4 storage of ``numel`` elements."""
    nb = -(-numel // 64)
    return nb * 32, nb, -(-nb // 256)


def nf4_quantize(w, codes=None, c8=None, s2=None, status=None, stream=None):
    """Quantise a bf16 CUDA tensor; returns ``(codes, c8, s2)`` (allocated if not given)."""
    assert w.dtype == torch.bfloat16 and w.is_cuda and w.is_contiguous()
    numel = w.numel()
    nc, nb, ns = nf4_sizes(numel)
    dev = w.device
    codes = torch.empty(nc, dtype=torch.uint8, device=dev) if codes is None else codes
    c8 = torch.empty(nb, dtype=torch.uint8, device=dev) if c8 is None else c8
    s2 = torch.empty(ns, dtype=torch.float32, device=dev) if s2 is None else s2
    _check(_lib.nf4_quantize(_ptr(w), numel, _ptr(codes), _ptr(c8), _ptr(s2), _ptr(status), _stream(stream)),
           "nf4_quantize")
    return codes, c8, s2


def quantize_weight(w, stream=None):
    """NF4-quantise a bf16 weight [n_out, k_in]; returns an :class:`NF4Weight`."""
    codes, c8, s2 = nf4_quantize(w, stream=stream)
    return NF4Weight(codes, c8, s2, w.shape[0], w.shape[1])


def nf4_dequantize(codes, c8, s2, numel, out=None, stream=None):
    """bf16 tensor of ``numel`` dequantised values."""
    out = torch.empty(numel, dtype=torch.bfloat16, device=codes.device) if out is None else out
    _check(_lib.nf4_dequantize(_ptr(codes), _ptr(c8), _ptr(s2), numel, _ptr(out), _stream(stream)),
           "nf4_dequantize")
    return out


def qlora_linear_fwd(X, W, A, B, s, y_dtype=DTYPE_BF16, Y=None, U=None, ws=None, status=None, stream=None):
    """Forward of the adapter-augmented NF4 linear; returns ``(Y, U)``."""
    M = X.shape[0]
    N, K, r = int(W.n_out), int(W.k_in), A.shape[0]
    dev = X.device
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32 if y_dtype == DTYPE_F32 else torch.bfloat16, device=dev)
    if U is None:
        U = torch.empty((M, r), dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.empty(max(qlora_fwd_workspace_size(M, N, K, r), 16), dtype=torch.uint8, device=dev)
    _check(_lib.qlora_linear_fwd(_ptr(X), M, _weight(W), _ptr(A), _ptr(B), r, float(s), _ptr(Y), y_dtype,
                                 _ptr(U), _ptr(ws), ws.numel(), _ptr(status), _stream(stream)),
           "qlora_linear_fwd")
    return Y, U


def qlora_linear_fwd_noalloc(X, W, A, B, s, y_dtype=DTYPE_BF16, Y=None, U=None, status=None, stream=None):
    """Forward without a workspace, for callers that cannot allocate device
    memory at call time (the library keeps a fixed 16 MiB scratch array per
    device; problems that need more are rejected).  Returns ``(Y, U)``.  The
    output tensors are allocated here only when not given."""
    M = X.shape[0]
    N, r = int(W.n_out), A.shape[0]
    dev = X.device
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32 if y_dtype == DTYPE_F32 else torch.bfloat16, device=dev)
    if U is None:
        U = torch.empty((M, r), dtype=torch.float32, device=dev)
    _check(_lib.qlora_linear_fwd_noalloc(_ptr(X), M, _weight(W), _ptr(A), _ptr(B), r, float(s), _ptr(Y), y_dtype,
                                         _ptr(U), _ptr(status), _stream(stream)),
           "qlora_linear_fwd_noalloc")
    return Y, U


def qlora_linear_bwd(dY, X, U, W, A, B, s, dx_dtype=DTYPE_BF16, dX=None, dA=None, dB=None, ws=None,
                     status=None, stream=None):
    """Backward through the frozen NF4 weight; returns ``(dX, dA, dB)``."""
    M = X.shape[0]
    N, K, r = int(W.n_out), int(W.k_in), A.shape[0]
    dev = X.device
    if dX is None:
        dX = torch.empty((M, K), dtype=torch.float32 if dx_dtype == DTYPE_F32 else torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty((r, K), dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty((N, r), dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.empty(max(qlora_bwd_workspace_size(M, N, K, r), 16), dtype=torch.uint8, device=dev)
    _check(_lib.qlora_linear_bwd(_ptr(dY), _ptr(X), _ptr(U), M, _weight(W), _ptr(A), _ptr(B), r, float(s),
                                 _ptr(dX), dx_dtype, _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(), _ptr(status),
                                 _stream(stream)),
           "qlora_linear_bwd")
    return dX, dA, dB


def profile_enable(on=True):
    """Bracket every library kernel launch with CUDA events (diagnostics)."""
    _lib.qlora_profile_enable(1 if on else 0)


def profile_collect(capacity=1 << 16):
    """[(kernel name, ms)] of the launches recorded since the last collect."""
    ids = (ctypes.c_int32 * capacity)()
    ms = (ctypes.c_float * capacity)()
    n = _lib.qlora_profile_collect(ctypes.cast(ids, _P), ctypes.cast(ms, _P), capacity)
    if n < 0:
        raise QloraError(7, "qlora_profile_collect")
    return [(_lib.qlora_kernel_name(ids[i]).decode(), float(ms[i])) for i in range(min(n, capacity))]


def raw():
    """The loaded ``ctypes.CDLL`` (for callers that pass raw pointers)."""
    return _lib


# ------------------------------------------------------------ optimizer step
# (include/qlora_optim.h: AdamW with 8-bit states in paged memory)

_F = ctypes.c_float
_lib.qlora_adamw8_step.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _F, _F, _F, _F, _F, _I64, _P, _P]
_lib.qlora_adamw8_step.restype = ctypes.c_int
_lib.qlora_paged_alloc.argtypes = [ctypes.POINTER(ctypes.c_void_p), _SZ]
_lib.qlora_paged_alloc.restype = ctypes.c_int
_lib.qlora_paged_prefetch.argtypes = [_P, _SZ, _I32, _P]
_lib.qlora_paged_prefetch.restype = ctypes.c_int
_lib.qlora_paged_free.argtypes = [_P]
_lib.qlora_paged_free.restype = ctypes.c_int

EXPORTED = EXPORTED + ("qlora_adamw8_step", "qlora_paged_alloc", "qlora_paged_prefetch", "qlora_paged_free")

STATE_BLOCK = 256  # parameters per fp32 state scale


def _al(b):
    return (b + 255) & ~255


class AdamW8State:
    """8-bit AdamW state of an ``n``-parameter tensor: E4M3 codes of m and of
    sqrt(v) (one byte each per parameter) and one fp32 scale per 256
    parameters for each.  ``paged=True`` puts all four arrays in one CUDA
    managed allocation (``qlora_paged_alloc``: resident in HBM, evicted to
    host RAM under memory pressure, migrated back when touched); otherwise
    they live in a torch device tensor.  A fresh state is all zeros."""

    def __init__(self, n, paged=True, device=None):
        self.n = int(n)
        self.nb = -(-self.n // STATE_BLOCK)
        self._offs = (0, _al(self.n), 2 * _al(self.n), 2 * _al(self.n) + _al(4 * self.nb))
        self.bytes = self._offs[3] + _al(4 * self.nb)
        self.paged = paged
        self._buf = None
        self._base = None
        if paged:
            ptr = ctypes.c_void_p()
            _check(_lib.qlora_paged_alloc(ctypes.byref(ptr), self.bytes), "qlora_paged_alloc")
            self._base = ptr.value
        else:
            self._buf = torch.zeros(self.bytes, dtype=torch.uint8, device=device or "cuda")
            self._base = self._buf.data_ptr()

    def pointers(self):
        """Device-usable addresses of (m8, u8, m_scale, u_scale)."""
        return tuple(self._base + o for o in self._offs)

    def prefetch(self, to_host=False, stream=None):
        """Migrate a paged state to the device (or to host RAM) on ``stream``."""
        if self.paged:
            _check(_lib.qlora_paged_prefetch(ctypes.c_void_p(self._base), self.bytes, 1 if to_host else 0,
                                             _stream(stream)), "qlora_paged_prefetch")

    def host_arrays(self):
        """Copies of (m8, u8, m_scale, u_scale) as numpy arrays (synchronises)."""
        import numpy as np
        torch.cuda.synchronize()
        if self.paged:
            def grab(off, n, ct, dt):
                return np.ctypeslib.as_array((ct * n).from_address(self._base + off)).astype(dt, copy=True)
            return (grab(self._offs[0], self.n, ctypes.c_uint8, np.uint8),
                    grab(self._offs[1], self.n, ctypes.c_uint8, np.uint8),
                    grab(self._offs[2], self.nb, ctypes.c_float, np.float32),
                    grab(self._offs[3], self.nb, ctypes.c_float, np.float32))
        b = self._buf.cpu().numpy()
        o = self._offs
        return (b[o[0]:o[0] + self.n].copy(), b[o[1]:o[1] + self.n].copy(),
                b[o[2]:o[2] + 4 * self.nb].view(np.float32).copy(), b[o[3]:o[3] + 4 * self.nb].view(np.float32).copy())

    def close(self):
        if self.paged and self._base is not None:
            torch.cuda.synchronize()
            _check(_lib.qlora_paged_free(ctypes.c_void_p(self._base)), "qlora_paged_free")
        self._base = None
        self._buf = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def qlora_adamw8_step(p, grad, state, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1,
                      status=None, stream=None):
    """One AdamW step in place on the bf16 parameter tensor ``p`` with fp32
    gradient ``grad`` and the 8-bit :class:`AdamW8State` ``state``."""
    assert p.dtype == torch.bfloat16 and grad.dtype == torch.float32
    assert p.is_contiguous() and grad.is_contiguous() and p.numel() == grad.numel() == state.n
    m8, u8, ms, us = state.pointers()
    _check(_lib.qlora_adamw8_step(_ptr(p), _ptr(grad), ctypes.c_void_p(m8), ctypes.c_void_p(u8),
                                  ctypes.c_void_p(ms), ctypes.c_void_p(us), state.n, lr, beta1, beta2, eps,
                                  weight_decay, int(step), _ptr(status), _stream(stream)), "qlora_adamw8_step")
    return p


# ------------------------------------------------------------ LoRA dropout
# (include/qlora_nf4.h: dropout on the adapter input, Philox-4x32-10 mask)

_U64 = ctypes.c_uint64
_lib.qlora_bwd_dropout_workspace_size.argtypes = [_I64, _I64, _I64, _I32]
_lib.qlora_bwd_dropout_workspace_size.restype = _SZ
_lib.qlora_linear_fwd_dropout.argtypes = [_P, _I64, _NF4Weight, _P, _P, _I32, ctypes.c_float, ctypes.c_float, _U64,
                                          _P, _P, _I32, _P, _P, _SZ, _P, _P]
_lib.qlora_linear_fwd_dropout.restype = ctypes.c_int
_lib.qlora_linear_bwd_dropout.argtypes = [_P, _P, _P, _I64, _NF4Weight, _P, _P, _I32, ctypes.c_float, ctypes.c_float,
                                          _U64, _P, _I32, _P, _P, _P, _SZ, _P, _P]
_lib.qlora_linear_bwd_dropout.restype = ctypes.c_int

EXPORTED = EXPORTED + ("qlora_bwd_dropout_workspace_size", "qlora_linear_fwd_dropout", "qlora_linear_bwd_dropout")


def qlora_bwd_dropout_workspace_size(M, N, K, r):
    return int(_lib.qlora_bwd_dropout_workspace_size(M, N, K, r))


def qlora_linear_fwd_dropout(X, W, A, B, s, p, seed, y_dtype=DTYPE_BF16, Y=None, U=None, X_drop=None, ws=None,
                             status=None, stream=None):
    """Forward with dropout (probability ``p``, Philox ``seed``) on the adapter
    input; returns ``(Y, U, X_drop)`` (keep X_drop for the backward)."""
    M = X.shape[0]
    N, K, r = int(W.n_out), int(W.k_in), A.shape[0]
    dev = X.device
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32 if y_dtype == DTYPE_F32 else torch.bfloat16, device=dev)
    if U is None:
        U = torch.empty((M, r), dtype=torch.float32, device=dev)
    if X_drop is None:
        X_drop = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = torch.empty(max(qlora_fwd_workspace_size(M, N, K, r), 16), dtype=torch.uint8, device=dev)
    _check(_lib.qlora_linear_fwd_dropout(_ptr(X), M, _weight(W), _ptr(A), _ptr(B), r, float(s), float(p), int(seed),
                                         _ptr(X_drop), _ptr(Y), y_dtype, _ptr(U), _ptr(ws), ws.numel(), _ptr(status),
                                         _stream(stream)),
           "qlora_linear_fwd_dropout")
    return Y, U, X_drop


def qlora_linear_bwd_dropout(dY, X_drop, U, W, A, B, s, p, seed, dx_dtype=DTYPE_BF16, dX=None, dA=None, dB=None,
                             ws=None, status=None, stream=None):
    """Backward of :func:`qlora_linear_fwd_dropout` (same ``p`` and ``seed``);
    returns ``(dX, dA, dB)``."""
    M = X_drop.shape[0]
    N, K, r = int(W.n_out), int(W.k_in), A.shape[0]
    dev = X_drop.device
    if dX is None:
        dX = torch.empty((M, K), dtype=torch.float32 if dx_dtype == DTYPE_F32 else torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty((r, K), dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty((N, r), dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.empty(max(qlora_bwd_dropout_workspace_size(M, N, K, r), 16), dtype=torch.uint8, device=dev)
    _check(_lib.qlora_linear_bwd_dropout(_ptr(dY), _ptr(X_drop), _ptr(U), M, _weight(W), _ptr(A), _ptr(B), r,
                                         float(s), float(p), int(seed), _ptr(dX), dx_dtype, _ptr(dA), _ptr(dB),
                                         _ptr(ws), ws.numel(), _ptr(status), _stream(stream)),
           "qlora_linear_bwd_dropout")
    return dX, dA, dB


# ------------------------------------------------------ bounded-wait self-test

_lib.qlora_selftest_timeout.argtypes = [_P, _I64, _P]
_lib.qlora_selftest_timeout.restype = ctypes.c_int
EXPORTED = EXPORTED + ("qlora_selftest_timeout",)


def qlora_selftest_timeout(status, limit_ns, stream=None):
    """Run the kernels' bounded wait against a barrier nothing completes, with
    a ``limit_ns`` limit; sets DEV_TIMEOUT in the int32 device tensor ``status``."""
    _check(_lib.qlora_selftest_timeout(_ptr(status), int(limit_ns), _stream(stream)), "qlora_selftest_timeout")


# ------------------------------------------------------ few-token kernel choice

_lib.qlora_set_few_token_threshold.argtypes = [_I64]
_lib.qlora_set_few_token_threshold.restype = _I64
EXPORTED = EXPORTED + ("qlora_set_few_token_threshold",)
DEFAULT_FEW_TOKEN_THRESHOLD = 1 << 26


def qlora_set_few_token_threshold(min_weight_elems):
    """Weights of at least this many elements run the few-token kernel for
    M <= 16 tokens (0: always, a huge value: never); returns the previous value."""
    return int(_lib.qlora_set_few_token_threshold(int(min_weight_elems)))


# ------------------------------------------------------ grouped projections
# (include/qlora_nf4.h: linears sharing one input, stacked along the outputs)

_lib.qlora_group_fwd_workspace_size.argtypes = [_I64, _I64, _I64, _I32, _I32]
_lib.qlora_group_fwd_workspace_size.restype = _SZ
_lib.qlora_group_bwd_workspace_size.argtypes = [_I64, _I64, _I64, _I32, _I32]
_lib.qlora_group_bwd_workspace_size.restype = _SZ
_lib.qlora_group_fwd.argtypes = [_P, _I64, _NF4Weight, _I32, _P, _P, _P, _I32, ctypes.c_float, _P, _I32, _P, _P,
                                 _SZ, _P, _P]
_lib.qlora_group_fwd.restype = ctypes.c_int
_lib.qlora_group_bwd.argtypes = [_P, _P, _P, _I64, _NF4Weight, _I32, _P, _P, _P, _I32, ctypes.c_float, _P, _I32,
                                 _P, _P, _P, _SZ, _P, _P]
_lib.qlora_group_bwd.restype = ctypes.c_int

EXPORTED = EXPORTED + ("qlora_group_fwd_workspace_size", "qlora_group_bwd_workspace_size", "qlora_group_fwd",
                       "qlora_group_bwd")


def qlora_group_fwd_workspace_size(M, N, K, members, r):
    return int(_lib.qlora_group_fwd_workspace_size(M, N, K, members, r))


def qlora_group_bwd_workspace_size(M, N, K, members, r):
    return int(_lib.qlora_group_bwd_workspace_size(M, N, K, members, r))


def _members(n_member):
    arr = (ctypes.c_int64 * len(n_member))(*[int(n) for n in n_member])
    return len(n_member), arr


def quantize_group(weights, stream=None):
    """NF4-quantise the members of a group (bf16 [n_g, K] each) as one stacked
    weight; returns ``(NF4Weight [sum n_g, K], [n_g ...])``."""
    stacked = torch.cat([w.reshape(w.shape[0], -1) for w in weights], 0).contiguous()
    return quantize_weight(stacked, stream=stream), [int(w.shape[0]) for w in weights]


def qlora_group_fwd(X, W, n_member, A, B, s, y_dtype=DTYPE_BF16, Y=None, U=None, ws=None, status=None, stream=None):
    """Forward of a group of linears sharing ``X``: W stacked [N, K], A [G r, K],
    B [N, r]; returns ``(Y [M, N], U [M, G r])``."""
    M = X.shape[0]
    G, arr = _members(n_member)
    N, K, r = int(W.n_out), int(W.k_in), A.shape[0] // G
    dev = X.device
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32 if y_dtype == DTYPE_F32 else torch.bfloat16, device=dev)
    if U is None:
        U = torch.empty((M, G * r), dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.empty(max(qlora_group_fwd_workspace_size(M, N, K, G, r), 16), dtype=torch.uint8, device=dev)
    _check(_lib.qlora_group_fwd(_ptr(X), M, _weight(W), G, ctypes.cast(arr, _P), _ptr(A), _ptr(B), r, float(s),
                                _ptr(Y), y_dtype, _ptr(U), _ptr(ws), ws.numel(), _ptr(status), _stream(stream)),
           "qlora_group_fwd")
    return Y, U


def qlora_group_bwd(dY, X, U, W, n_member, A, B, s, dx_dtype=DTYPE_BF16, dX=None, dA=None, dB=None, ws=None,
                    status=None, stream=None):
    """Backward of :func:`qlora_group_fwd`; returns ``(dX [M, K] summed over the
    members, dA [G r, K], dB [N, r])``."""
    M = X.shape[0]
    G, arr = _members(n_member)
    N, K, r = int(W.n_out), int(W.k_in), A.shape[0] // G
    dev = X.device
    if dX is None:
        dX = torch.empty((M, K), dtype=torch.float32 if dx_dtype == DTYPE_F32 else torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty((G * r, K), dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty((N, r), dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.empty(max(qlora_group_bwd_workspace_size(M, N, K, G, r), 16), dtype=torch.uint8, device=dev)
    _check(_lib.qlora_group_bwd(_ptr(dY), _ptr(X), _ptr(U), M, _weight(W), G, ctypes.cast(arr, _P), _ptr(A),
                                _ptr(B), r, float(s), _ptr(dX), dx_dtype, _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(),
                                _ptr(status), _stream(stream)),
           "qlora_group_bwd")
    return dX, dA, dB


# ------------------------------------------ mean-centred double quantisation

_lib.nf4_centered_workspace_size.argtypes = [_I64]
_lib.nf4_centered_workspace_size.restype = _SZ
_lib.nf4_quantize_centered.argtypes = [_P, _I64, _P, _P, _P, _P, _P, _SZ, _P, _P]
_lib.nf4_quantize_centered.restype = ctypes.c_int
_lib.nf4_dequantize_centered.argtypes = [_P, _P, _P, _P, _I64, _P, _P]
_lib.nf4_dequantize_centered.restype = ctypes.c_int

EXPORTED = EXPORTED + ("nf4_centered_workspace_size", "nf4_quantize_centered", "nf4_dequantize_centered")


def nf4_centered_workspace_size(numel):
    return int(_lib.nf4_centered_workspace_size(numel))


def nf4_quantize_centered(w, codes=None, c8=None, s2=None, mean=None, ws=None, status=None, stream=None):
    """Quantise a bf16 CUDA tensor with mean-centred constants; returns
    ``(codes, c8, s2, mean)`` (allocated if not given; mean is fp32 [1])."""
    assert w.dtype == torch.bfloat16 and w.is_cuda and w.is_contiguous()
    numel = w.numel()
    nc, nb, ns = nf4_sizes(numel)
    dev = w.device
    codes = torch.empty(nc, dtype=torch.uint8, device=dev) if codes is None else codes
    c8 = torch.empty(nb, dtype=torch.uint8, device=dev) if c8 is None else c8
    s2 = torch.empty(ns, dtype=torch.float32, device=dev) if s2 is None else s2
    mean = torch.empty(4, dtype=torch.float32, device=dev)[:1] if mean is None else mean
    if ws is None:
        ws = torch.empty(max(nf4_centered_workspace_size(numel), 16), dtype=torch.uint8, device=dev)
    _check(_lib.nf4_quantize_centered(_ptr(w), numel, _ptr(codes), _ptr(c8), _ptr(s2), _ptr(mean), _ptr(ws),
                                      ws.numel(), _ptr(status), _stream(stream)), "nf4_quantize_centered")
    return codes, c8, s2, mean


def quantize_weight_centered(w, stream=None):
    """NF4-quantise a bf16 weight [n_out, k_in] with mean-centred constants;
    returns an :class:`NF4Weight` whose ``mean`` is set."""
    codes, c8, s2, mean = nf4_quantize_centered(w, stream=stream)
    return NF4Weight(codes, c8, s2, w.shape[0], w.shape[1], mean)


def nf4_dequantize_centered(codes, c8, s2, mean, numel, out=None, stream=None):
    """bf16 tensor of ``numel`` values dequantised with mean-centred constants."""
    out = torch.empty(numel, dtype=torch.bfloat16, device=codes.device) if out is None else out
    _check(_lib.nf4_dequantize_centered(_ptr(codes), _ptr(c8), _ptr(s2), _ptr(mean), numel, _ptr(out),
                                        _stream(stream)), "nf4_dequantize_centered")
    return out


# ------------------------------------------------ 8-bit activation checkpoints
# (include/qlora_train.h: E4M3 codes with a power of two per 64 elements)

_lib.act8_quantize.argtypes = [_P, _I64, _I64, _I64, _P, _P, _P, _P]
_lib.act8_quantize.restype = ctypes.c_int
_lib.act8_dequantize.argtypes = [_P, _P, _I64, _I64, _P, _I64, _P]
_lib.act8_dequantize.restype = ctypes.c_int
_lib.qlora_linear_bwd_act8.argtypes = [_P, _P, _P, _P, _I64, _NF4Weight, _P, _P, _I32, _F, _P, _I32, _P, _P, _P, _SZ,
                                       _P, _P]
_lib.qlora_linear_bwd_act8.restype = ctypes.c_int
_lib.qlora_group_bwd_act8.argtypes = [_P, _P, _P, _P, _I64, _NF4Weight, _I32, _P, _P, _P, _I32, _F, _P, _I32, _P, _P,
                                      _P, _SZ, _P, _P]
_lib.qlora_group_bwd_act8.restype = ctypes.c_int
_lib.qlora_linear_bwd_dropout_act8.argtypes = [_P, _P, _P, _P, _I64, _NF4Weight, _P, _P, _I32, _F, _F, _U64, _P, _I32,
                                               _P, _P, _P, _SZ, _P, _P]
_lib.qlora_linear_bwd_dropout_act8.restype = ctypes.c_int

_lib.qlora_bwd_act8_workspace_size.argtypes = [_I64, _I64, _I64, _I32, _I32, _I32]
_lib.qlora_bwd_act8_workspace_size.restype = _SZ

EXPORTED_TRAIN = ("act8_quantize", "act8_dequantize", "qlora_bwd_act8_workspace_size", "qlora_linear_bwd_act8",
                  "qlora_group_bwd_act8", "qlora_linear_bwd_dropout_act8")

DEV_LABEL = 4
ERR_SHAPE = 2
ERR_DTYPE = 9

#: 8-bit checkpoint of X [M, K]: ``codes`` uint8 [M, K], ``exps`` uint8 [M, K / 64].
Act8 = namedtuple("Act8", "codes exps")


def _run(dev, stream, call):
    """``call(stream handle)`` with ``dev`` current, on ``stream`` or ``dev``'s
    current stream; what it allocates belongs to that stream."""
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _run(dev, stream, call)
    if stream is None:
        return call(torch._C._cuda_getCurrentRawStream(dev.index))
    if stream.device != dev:
        _refuse(ERR_SHAPE, "stream", f"is on {stream.device}, the tensors on {dev}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _refuse(code, where, what):
    raise QloraError(code, f"{where}: {what}")


def _tensor(t, dtype, shape, dev, where, name, dense=True):
    """A tensor of this type and shape on this device, contiguous if ``dense``."""
    if t.dtype != dtype:
        _refuse(ERR_DTYPE, where, f"{name} is {t.dtype}, not {dtype}")
    if t.shape != shape:
        _refuse(ERR_SHAPE, where, f"{name} is {tuple(t.shape)}, not {shape}")
    if t.device != dev:
        _refuse(ERR_SHAPE, where, f"{name} is on {t.device}, not {dev}")
    if dense and not t.is_contiguous():
        _refuse(ERR_SHAPE, where, f"{name} is not contiguous")
    return t


def _out(t, like, shape, where, name):
    """``t``, or a new tensor of ``like``'s type on its device (the cheapest way to
    one: small problems take no longer on the GPU)."""
    return like.new_empty(shape) if t is None else _tensor(t, like.dtype, shape, like.device, where, name)


def _rows(t, where, name, cols=None, rows=None, dev=None):
    """(rows, columns, row stride) of a bf16 CUDA matrix whose rows are contiguous."""
    if t.dtype != torch.bfloat16:
        _refuse(ERR_DTYPE, where, f"{name} is {t.dtype}, not torch.bfloat16")
    if t.dim() != 2:
        _refuse(ERR_SHAPE, where, f"{name} has {t.dim()} dimensions, not 2")
    if not t.is_cuda or (dev is not None and t.device != dev):
        _refuse(ERR_SHAPE, where, f"{name} is on {t.device}")
    M, K = t.shape
    if (cols is not None and K != cols) or (rows is not None and M != rows):
        _refuse(ERR_SHAPE, where, f"{name} is {(M, K)}, not {(M if rows is None else rows, cols)}")
    ld, inner = t.stride()
    if K > 1 and M > 0 and inner != 1:
        _refuse(ERR_SHAPE, where, f"{name}'s rows are not contiguous")
    return M, K, ld if M > 1 else K


def _word(status, dev, where):
    """Address of the optional device status word."""
    if status is None:
        return None
    if status.dtype != torch.int32 or status.numel() < 1 or status.device != dev:
        _refuse(ERR_DTYPE, where, "status is not an int32 word on the call's device")
    return status.data_ptr()


def _nf4(W, dev, where, name):
    """An NF4 storage of the sizes its shape has, on this device."""
    nc, nb, ns = nf4_sizes(int(W.n_out) * int(W.k_in))
    for t, dtype, n in ((W.codes, torch.uint8, nc), (W.c8, torch.uint8, nb), (W.s2, torch.float32, ns)):
        if t.dtype != dtype or t.numel() != n or t.device != dev or not t.is_contiguous():
            _refuse(ERR_SHAPE, where, f"{name} is no NF4 storage of {int(W.n_out)} x {int(W.k_in)} on {dev}")
    mean = getattr(W, "mean", None)
    if mean is not None and (mean.dtype != torch.float32 or mean.numel() < 1 or mean.device != dev):
        _refuse(ERR_SHAPE, where, f"{name}'s mean is no fp32 word on {dev}")


def _workspace(ws, size, like, where):
    """(address, bytes, tensor) of the workspace, allocated on ``like``'s device if not given."""
    if ws is None:
        ws = like.new_empty(max(size(), 16), dtype=torch.uint8)
    elif ws.device != like.device or not ws.is_contiguous():
        _refuse(ERR_SHAPE, where, f"ws is on {ws.device}, or not contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def act8_quantize(X, codes=None, exps=None, status=None, stream=None):
    """8-bit checkpoint of a bf16 CUDA matrix X [M, K] (K % 64 == 0, rows may be
    strided); returns an :class:`Act8` (its tensors allocated if not given)."""
    where = "act8_quantize"
    M, K, ld = _rows(X, where, "X")
    dev = X.device

    def call(st):
        c = (X.new_empty((M, K), dtype=torch.uint8) if codes is None
             else _tensor(codes, torch.uint8, (M, K), dev, where, "codes"))
        e = c.new_empty((M, K // 64)) if exps is None else _tensor(exps, torch.uint8, (M, K // 64), dev, where, "exps")
        _check(_lib.act8_quantize(X.data_ptr(), M, K, ld, c.data_ptr(), e.data_ptr(), _word(status, dev, where), st),
               where)
        return Act8(c, e)
    return _run(dev, stream, call)


def act8_dequantize(X8, out=None, stream=None):
    """The bf16 values [M, K] an :class:`Act8` stands for (``out`` may have strided rows)."""
    where = "act8_dequantize"
    codes, exps = X8
    if codes.dim() != 2 or not codes.is_cuda:
        _refuse(ERR_SHAPE, where, "codes is not a CUDA matrix")
    M, K = codes.shape
    dev = codes.device
    _act8(X8, M, K, dev, where)
    ld = K if out is None else _rows(out, where, "out", K, M, dev)[2]

    def call(st):
        x = codes.new_empty((M, K), dtype=torch.bfloat16) if out is None else out
        _check(_lib.act8_dequantize(codes.data_ptr(), exps.data_ptr(), M, K, x.data_ptr(), ld, st), where)
        return x
    return _run(dev, stream, call)


def _act8(X8, M, K, dev, where):
    codes, exps = X8
    _tensor(codes, torch.uint8, (M, K), dev, where, "codes")
    _tensor(exps, torch.uint8, (M, K // 64), dev, where, "exps")


def qlora_bwd_act8_workspace_size(M, N, K, members, r, dropout=False):
    return int(_lib.qlora_bwd_act8_workspace_size(M, N, K, members, r, 1 if dropout else 0))


def _bwd_act8(where, dY, X8, U, W, G, A, B, dx_dtype, dX, dA, dB, drop, ws, status, stream, run):
    """Checks, outputs and workspace shared by the ``*_bwd_act8`` passes."""
    N, K = int(W.n_out), int(W.k_in)
    if dY.dim() != 2:
        _refuse(ERR_SHAPE, where, f"dY has {dY.dim()} dimensions, not 2")
    M = dY.shape[0]
    dev = dY.device
    if dx_dtype not in (DTYPE_BF16, DTYPE_F32):
        _refuse(ERR_DTYPE, where, f"dx_dtype is {dx_dtype}")
    if not dY.is_cuda:
        _refuse(ERR_SHAPE, where, f"dY is on {dev}")
    if A.dim() != 2 or A.shape[0] % G != 0:
        _refuse(ERR_SHAPE, where, f"A is {tuple(A.shape)} for {G} members")
    r = A.shape[0] // G
    _tensor(dY, torch.bfloat16, (M, N), dev, where, "dY")
    _act8(X8, M, K, dev, where)
    _tensor(U, torch.float32, (M, G * r), dev, where, "U")
    _tensor(A, torch.bfloat16, (G * r, K), dev, where, "A")
    _tensor(B, torch.bfloat16, (N, r), dev, where, "B")
    _nf4(W, dev, where, "W")

    def call(st):
        x = _out(dX, U if dx_dtype == DTYPE_F32 else dY, (M, K), where, "dX")
        a = _out(dA, U, (G * r, K), where, "dA")
        b = _out(dB, U, (N, r), where, "dB")
        if M == 0:  # nothing to sum; the library's call is a no-op
            a.zero_()
            b.zero_()
        at, size_, keep = _workspace(ws, lambda: qlora_bwd_act8_workspace_size(M, N, K, G, r, drop), U, where)
        _check(run(M, r, x.data_ptr(), a.data_ptr(), b.data_ptr(), at, size_, _word(status, dev, where), st), where)
        return x, a, b
    return _run(dev, stream, call)


def qlora_linear_bwd_act8(dY, X8, U, W, A, B, s, dx_dtype=DTYPE_BF16, dX=None, dA=None, dB=None, ws=None,
                          status=None, stream=None):
    """:func:`qlora_linear_bwd` with the input as its 8-bit checkpoint ``X8``;
    returns ``(dX, dA, dB)``."""
    def call(M, r, dX, dA, dB, ws, size, status, st):
        return _lib.qlora_linear_bwd_act8(dY.data_ptr(), X8[0].data_ptr(), X8[1].data_ptr(), U.data_ptr(), M,
                                          _weight(W), A.data_ptr(), B.data_ptr(), r, float(s), dX, dx_dtype, dA, dB,
                                          ws, size, status, st)
    return _bwd_act8("qlora_linear_bwd_act8", dY, X8, U, W, 1, A, B, dx_dtype, dX, dA, dB, False, ws, status, stream,
                     call)


def qlora_group_bwd_act8(dY, X8, U, W, n_member, A, B, s, dx_dtype=DTYPE_BF16, dX=None, dA=None, dB=None, ws=None,
                         status=None, stream=None):
    """:func:`qlora_group_bwd` with the shared input as its 8-bit checkpoint ``X8``."""
    G, arr = _members(n_member)

    def call(M, r, dX, dA, dB, ws, size, status, st):
        return _lib.qlora_group_bwd_act8(dY.data_ptr(), X8[0].data_ptr(), X8[1].data_ptr(), U.data_ptr(), M,
                                         _weight(W), G, ctypes.cast(arr, _P), A.data_ptr(), B.data_ptr(), r, float(s),
                                         dX, dx_dtype, dA, dB, ws, size, status, st)
    return _bwd_act8("qlora_group_bwd_act8", dY, X8, U, W, G, A, B, dx_dtype, dX, dA, dB, False, ws, status, stream,
                     call)


def qlora_linear_bwd_dropout_act8(dY, X8_drop, U, W, A, B, s, p, seed, dx_dtype=DTYPE_BF16, dX=None, dA=None,
                                  dB=None, ws=None, status=None, stream=None):
    """:func:`qlora_linear_bwd_dropout` with X_drop as its 8-bit checkpoint (same
    ``p`` and ``seed`` as the forward)."""
    def call(M, r, dX, dA, dB, ws, size, status, st):
        return _lib.qlora_linear_bwd_dropout_act8(dY.data_ptr(), X8_drop[0].data_ptr(), X8_drop[1].data_ptr(),
                                                  U.data_ptr(), M, _weight(W), A.data_ptr(), B.data_ptr(), r, float(s),
                                                  float(p), int(seed), dX, dx_dtype, dA, dB, ws, size, status, st)
    return _bwd_act8("qlora_linear_bwd_dropout_act8", dY, X8_drop, U, W, 1, A, B, dx_dtype, dX, dA, dB, True, ws,
                     status, stream, call)


# ------------------------------------------------------------------ loss head
# (include/qlora_train.h: softmax cross entropy in pieces of the vocabulary)


class _Head(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("ld", ctypes.c_int64), ("codes", ctypes.c_void_p), ("c8", ctypes.c_void_p),
                ("s2", ctypes.c_void_p), ("mean", ctypes.c_void_p), ("vocab", ctypes.c_int64),
                ("dim", ctypes.c_int64)]


_lib.qlora_head_loss_workspace_size.argtypes = [_I64, _I64, _I64, _I32, _I32]
_lib.qlora_head_loss_workspace_size.restype = _SZ
_lib.qlora_head_loss_fwd.argtypes = [_P, _I64, _I64, _Head, _P, _I64, _P, _P, _P, _P, _SZ, _P, _P]
_lib.qlora_head_loss_fwd.restype = ctypes.c_int
_lib.qlora_head_loss_bwd.argtypes = [_P, _I64, _I64, _Head, _P, _I64, _P, _P, _P, _P, _I64, _P, _SZ, _P, _P]
_lib.qlora_head_loss_bwd.restype = ctypes.c_int
_lib.qlora_head_loss_step.argtypes = [_P, _I64, _I64, _Head, _P, _I64, _P, _F, _P, _P, _P, _P, _I64, _P, _SZ, _P, _P]
_lib.qlora_head_loss_step.restype = ctypes.c_int

EXPORTED_TRAIN = EXPORTED_TRAIN + ("qlora_head_loss_workspace_size", "qlora_head_loss_fwd", "qlora_head_loss_bwd",
                                   "qlora_head_loss_step")

HEAD_FWD, HEAD_BWD, HEAD_STEP = 0, 1, 2
IGNORE_INDEX = -100


def qlora_head_loss_workspace_size(T, vocab, dim, nf4, op):
    """Workspace bytes of a loss-head call (``op`` one of HEAD_FWD, HEAD_BWD, HEAD_STEP)."""
    return int(_lib.qlora_head_loss_workspace_size(T, vocab, dim, 1 if nf4 else 0, op))


def _head(head, dev, where):
    """(C struct, vocab, dim, nf4) of a bf16 matrix [vocab, dim] or an :class:`NF4Weight`."""
    if isinstance(head, torch.Tensor):
        V, D, ld = _rows(head, where, "head", dev=dev)
        return _Head(head.data_ptr(), ld, None, None, None, None, V, D), V, D, False
    V, D = int(head.n_out), int(head.k_in)
    mean = getattr(head, "mean", None)
    _nf4(head, dev, where, "head")
    return _Head(None, 0, head.codes.data_ptr(), head.c8.data_ptr(), head.s2.data_ptr(),
                 None if mean is None else mean.data_ptr(), V, D), V, D, True


def _head_call(where, op, H, head, labels):
    """The checked problem: tokens, width, H's row stride, device, head, workspace query."""
    T, D, ldh = _rows(H, where, "H")
    dev = H.device
    h, V, dim, nf4 = _head(head, dev, where)
    if dim != D:
        _refuse(ERR_SHAPE, where, f"H has {D} columns, the head {dim}")
    _tensor(labels, torch.int64, (T,), dev, where, "labels")
    return T, D, ldh, dev, h, lambda: qlora_head_loss_workspace_size(T, V, D, nf4, op)


def _loss_out(H, loss, lse, stats, T, dev, where):
    """The losses', log-sum-exps' and statistics' tensors."""
    loss = (H.new_empty((T,), dtype=torch.float32) if loss is None
            else _tensor(loss, torch.float32, (T,), dev, where, "loss"))
    lse = torch.empty_like(loss) if lse is None else _tensor(lse, torch.float32, (T,), dev, where, "lse")
    stats = loss.new_empty(2) if stats is None else _tensor(stats, torch.float32, (2,), dev, where, "stats")
    return loss, lse, stats


def _grad_out(H, dH, T, D, dev, where):
    """(row stride of dH, maker of dH)."""
    if dH is None:
        return D, lambda: H.new_empty((T, D))
    return _rows(dH, where, "dH", D, T, dev)[2], lambda: dH


def qlora_head_loss_fwd(H, head, labels, ignore_index=IGNORE_INDEX, loss=None, lse=None, stats=None, ws=None,
                        status=None, stream=None):
    """Cross entropy of ``H @ head.T`` against ``labels`` (int64 [T]) without the
    logits; ``head`` is a bf16 matrix [vocab, dim] or an :class:`NF4Weight`.
    Returns ``(loss [T], lse [T], stats [2])``: per-token losses (0 where the
    label is ``ignore_index``), log-sum-exps (keep them for the backward), and
    the mean over the tokens that count with their number."""
    where = "qlora_head_loss_fwd"
    T, D, ldh, dev, h, size = _head_call(where, HEAD_FWD, H, head, labels)

    def call(st):
        lo, ls, sm = _loss_out(H, loss, lse, stats, T, dev, where)
        at, bytes_, keep = _workspace(ws, size, H, where)
        _check(_lib.qlora_head_loss_fwd(H.data_ptr(), ldh, T, h, labels.data_ptr(), int(ignore_index), lo.data_ptr(),
                                        ls.data_ptr(), sm.data_ptr(), at, bytes_, _word(status, dev, where), st),
               where)
        return lo, ls, sm
    return _run(dev, stream, call)


def qlora_head_loss_bwd(H, head, labels, lse, dloss, stats=None, ignore_index=IGNORE_INDEX, dH=None, ws=None,
                        status=None, stream=None):
    """Gradient of the losses of :func:`qlora_head_loss_fwd` towards ``H`` (bf16
    [T, dim]): ``dloss`` [T] holds the gradient of every token's loss, or, with
    the forward's ``stats`` given, ``dloss`` (one element, of no or one dimension)
    the gradient of the mean.  It may have any strides, as autograd hands over
    the gradient of a sum (one element expanded): a dense copy is made then."""
    where = "qlora_head_loss_bwd"
    T, D, ldh, dev, h, size = _head_call(where, HEAD_BWD, H, head, labels)
    _tensor(lse, torch.float32, (T,), dev, where, "lse")
    if stats is not None and dloss.dim() == 0:
        dloss = dloss.view(1)
    _tensor(dloss, torch.float32, (T if stats is None else 1,), dev, where, "dloss", dense=False)
    if stats is not None:
        _tensor(stats, torch.float32, (2,), dev, where, "stats")
    ldd, grad = _grad_out(H, dH, T, D, dev, where)

    def call(st):
        g, dl = grad(), dloss.contiguous()
        at, bytes_, keep = _workspace(ws, size, H, where)
        _check(_lib.qlora_head_loss_bwd(H.data_ptr(), ldh, T, h, labels.data_ptr(), int(ignore_index), lse.data_ptr(),
                                        dl.data_ptr(), None if stats is None else stats.data_ptr(), g.data_ptr(),
                                        ldd, at, bytes_, _word(status, dev, where), st), where)
        return g
    return _run(dev, stream, call)


def qlora_head_loss_step(H, head, labels, weight=None, scale=1.0, ignore_index=IGNORE_INDEX, loss=None, lse=None,
                         stats=None, dH=None, ws=None, status=None, stream=None):
    """The losses and their gradient in one call; returns ``(loss, lse, stats,
    dH)``.  ``dH`` is the gradient of ``scale`` times the mean loss, or, with
    ``weight`` (fp32 [T]), of ``scale * sum(weight * loss)``."""
    where = "qlora_head_loss_step"
    T, D, ldh, dev, h, size = _head_call(where, HEAD_STEP, H, head, labels)
    if weight is not None:
        _tensor(weight, torch.float32, (T,), dev, where, "weight")
    ldd, grad = _grad_out(H, dH, T, D, dev, where)

    def call(st):
        lo, ls, sm = _loss_out(H, loss, lse, stats, T, dev, where)
        g = grad()
        at, bytes_, keep = _workspace(ws, size, H, where)
        _check(_lib.qlora_head_loss_step(H.data_ptr(), ldh, T, h, labels.data_ptr(), int(ignore_index),
                                         None if weight is None else weight.data_ptr(), float(scale), lo.data_ptr(),
                                         ls.data_ptr(), sm.data_ptr(), g.data_ptr(), ldd, at, bytes_,
                                         _word(status, dev, where), st), where)
        return lo, ls, sm, g
    return _run(dev, stream, call)
