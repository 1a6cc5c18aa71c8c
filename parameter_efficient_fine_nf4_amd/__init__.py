"""Python binding of libqlora: the gfx950 QLoRA adapted linear.

Argument marshalling only.  Every step of the layer runs in the HIP kernels
of ``libqlora.so`` (built in-tree by ``parameter_efficient_fine_nf4_amd/build.py``);
torch provides device memory and the current stream.  Importing this module
fails loudly when the library has not been built.

The calls mirror include/qlora.h:

* ``quantize(W0)``                     -> ``NF4Weight``
* ``forward(X, w, A, B, alpha)``       -> ``Y`` (and ``T_save``)
* ``backward(dY, X, w, A, B, alpha)``  -> ``dX, dA, dB``
* ``merge(w, A, B, alpha)``            -> bf16 ``W``
* ``unmerge(W, A, B, alpha)``          -> bf16 ``W0``
* ``token_logprobs(logits, labels)``   -> fp32 ``logp`` (and row statistics)
* ``preference_loss(logp, ...)``, ``policy_loss(logits, ...)`` -> losses and gradients
* ``token_scores(logits, tokens, top)`` -> log-probabilities, entropy, best words
* ``checkpoint_save(X)``, ``forward_checkpoint``, ``backward_checkpoint`` -> the
  layer with its input kept at 8 bits
* ``adam_step``, ``muon_step``         -> the adapters' optimiser steps
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# QLORA_LIB_PATH selects another build of the same library (the host-side
# sanitizer build that build.py --sanitize writes under _build/).
LIB_PATH = os.environ.get("QLORA_LIB_PATH") or os.path.join(_HERE, "libqlora.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with "
        "`python parameter_efficient_fine_nf4_amd/build.py` (hipcc, gfx950)")

_lib = ctypes.CDLL(LIB_PATH)

_i64, _i32, _f32, _sz, _vp = (ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                              ctypes.c_size_t, ctypes.c_void_p)


class _Nf4Desc(ctypes.Structure):
    _fields_ = [("d", _i64), ("k", _i64), ("codes", _vp), ("absmax_q", _vp),
                ("absmax_scale", _vp), ("absmax_mean", _vp)]


_P = ctypes.POINTER(_Nf4Desc)
_sigs = {
    "qlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "qlora_version": (ctypes.c_int, []),
    "qlora_nf4_levels": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float)]),
    "qlora_nf4_sizes": (ctypes.c_int, [_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz),
                                       ctypes.POINTER(_sz), ctypes.POINTER(_sz)]),
    "qlora_quantize_workspace_bytes": (_sz, [_i64, _i64]),
    "nf4_quantize": (ctypes.c_int, [_vp, _i64, _i64, _P, _vp, _sz, _vp]),
    "qlora_tsave_bytes": (_sz, [_i64, _i32]),
    "qlora_forward_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32]),
    "qlora_forward": (ctypes.c_int, [_vp, _i64, _P, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _sz, _vp]),
    "qlora_backward_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32]),
    "qlora_backward": (ctypes.c_int, [_vp, _vp, _i64, _P, _vp, _vp, _i32, _f32, _vp, _vp, _vp,
                                      _vp, _vp, _sz, _vp]),
    "qlora_backward_noalloc": (ctypes.c_int, [_vp, _vp, _i64, _P, _vp, _vp, _i32, _f32, _vp, _vp, _vp,
                                              _vp, _vp]),
    "qlora_forward_sections": (ctypes.c_int, [_vp, _i64, _P, _i32, _vp, _vp, _i32, _f32, _vp, _vp, _vp,
                                              _sz, _vp]),
    "qlora_backward_sections": (ctypes.c_int, [_vp, _vp, _i64, _P, _i32, _vp, _vp, _i32, _f32, _vp,
                                               _vp, _vp, _vp, _vp, _sz, _vp]),
    "qlora_forward_dropout_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32]),
    "qlora_backward_dropout_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32]),
    "qlora_forward_dropout": (ctypes.c_int, [_vp, _i64, _P, _vp, _vp, _i32, _f32, _vp, _f32, _vp, _vp, _vp,
                                             _vp, _sz, _vp]),
    "qlora_backward_dropout": (ctypes.c_int, [_vp, _vp, _i64, _P, _vp, _vp, _i32, _f32, _vp, _f32, _vp, _vp,
                                              _vp, _vp, _vp, _vp, _sz, _vp]),
    "qlora_forward_multi_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32, _i32]),
    "qlora_forward_multi": (ctypes.c_int, [_vp, _i64, _P, _i32, _vp, _vp, _vp, _i32, _f32, _vp, _vp,
                                           _sz, _vp]),
    "qlora_adam_step": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _f32, _f32, _f32, _f32, _f32, _i64, _vp]),
    "qlora_token_logprobs": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i64, _vp, _f32, _vp, _vp, _vp]),
    "qlora_token_logprobs_backward": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i64, _i64, _vp, _f32, _vp, _vp, _i64,
                                                     _vp]),
    "qlora_preference_loss": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _vp, _i64, _i32, _i32, _f32, _f32, _f32, _vp,
                                             _vp, _vp, _vp, _vp]),
    "qlora_policy_loss": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i64, _vp, _f32, _vp, _vp, _vp, _vp, _f32, _f32, _f32,
                                         _vp, _vp, _vp, _vp, _i64, _vp]),
    "qlora_checkpoint_sizes": (ctypes.c_int, [_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)]),
    "qlora_checkpoint_save": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "qlora_checkpoint_load": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp]),
    "qlora_forward_checkpoint": (ctypes.c_int, [_vp, _i64, _P, _i32, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _vp, _vp,
                                                _sz, _vp]),
    "qlora_backward_checkpoint": (ctypes.c_int, [_vp, _vp, _vp, _i64, _P, _i32, _vp, _vp, _i32, _f32, _vp, _f32, _vp,
                                                 _vp, _vp, _vp, _vp, _sz, _vp]),
    "qlora_token_scores": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i64, _vp, _i32, _i32, _f32, _vp, _vp, _vp, _vp, _vp,
                                          _vp]),
    "qlora_token_scores_backward": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _f32, _vp, _vp,
                                                   _i64, _vp]),
    "qlora_muon_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "qlora_muon_step": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _f32, _f32, _i32, _f32, _f32, _f32, _i32,
                                       ctypes.POINTER(ctypes.c_float), _vp, _sz, _vp]),
    "lora_merge": (ctypes.c_int, [_P, _vp, _vp, _i32, _f32, _vp, _vp]),
    "lora_unmerge": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _i32, _f32, _vp, _vp]),
    "qlora_timing_enable": (ctypes.c_int, [ctypes.c_int]),
    "qlora_timing_collect": (ctypes.c_int, []),
    "qlora_timing_query": (ctypes.c_int, [ctypes.c_char_p, ctypes.POINTER(ctypes.c_double),
                                          ctypes.POINTER(_i64)]),
    "qlora_timing_reset": (ctypes.c_int, []),
}
for _name, (_res, _args) in _sigs.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_sigs)
STATUS = {0: "QLORA_OK", 1: "QLORA_ERR_NULL", 2: "QLORA_ERR_SHAPE", 3: "QLORA_ERR_RANK",
          4: "QLORA_ERR_ALIGN", 5: "QLORA_ERR_WORKSPACE", 6: "QLORA_ERR_ALPHA",
          7: "QLORA_ERR_ALIAS", 8: "QLORA_ERR_HIP", 9: "QLORA_ERR_TYPE"}


class QloraError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        msg = _lib.qlora_status_string(status).decode()
        super().__init__(f"{call} failed: {STATUS.get(status, status)} ({msg})")


def _check(status: int, call: str) -> None:
    if status != 0:
        raise QloraError(status, call)


def lib() -> ctypes.CDLL:
    """The loaded ctypes library (raw C ABI)."""
    return _lib


def nf4_levels() -> list:
    """The library's 16 NF4 levels (host computation)."""
    buf = (ctypes.c_float * 16)()
    _check(_lib.qlora_nf4_levels(buf), "qlora_nf4_levels")
    return list(buf)


def nf4_sizes(d: int, k: int) -> dict:
    out = [_sz() for _ in range(4)]
    _check(_lib.qlora_nf4_sizes(d, k, *[ctypes.byref(o) for o in out]), "qlora_nf4_sizes")
    return dict(zip(("codes", "absmax_q", "absmax_scale", "absmax_mean"), (o.value for o in out)))


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    """Raw handle of the current stream of ``device`` (torch's C accessor:
    a few microseconds cheaper per call than building a Stream object)."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    return torch._C._cuda_getCurrentRawStream(idx)


def _workspace(nbytes: int, device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


@dataclass
class NF4Weight:
    """Device buffers of one NF4-quantised d x k weight (caller-owned).

    With ``nsec`` > 1 the rows stack nsec weights of d/nsec rows each,
    quantised one by one (see ``quantize_sections``), and ``absmax_mean``
    holds their nsec means."""
    d: int
    k: int
    codes: torch.Tensor         # uint8 [d*k/2]
    absmax_q: torch.Tensor      # uint8 [d*k/64]   (FP8 E4M3FN)
    absmax_scale: torch.Tensor  # float32 [ceil(n_b/256)]
    absmax_mean: torch.Tensor   # float32 [nsec]
    nsec: int = 1

    @staticmethod
    def empty(d: int, k: int, device, nsec: int = 1) -> "NF4Weight":
        sz = nf4_sizes(d, k)
        return NF4Weight(d, k,
                         torch.empty(sz["codes"], dtype=torch.uint8, device=device),
                         torch.empty(sz["absmax_q"], dtype=torch.uint8, device=device),
                         torch.empty(sz["absmax_scale"] // 4, dtype=torch.float32, device=device),
                         torch.empty(nsec, dtype=torch.float32, device=device), nsec)

    def section(self, p: int) -> "NF4Weight":
        """Section p as a single-weight view of the same buffers (its rows
        are whole second-level groups, so every array slices cleanly)."""
        ds = self.d // self.nsec
        nb = ds * self.k // 64
        assert self.nsec == 1 or nb % 256 == 0
        return NF4Weight(ds, self.k, self.codes[p * ds * self.k // 2:(p + 1) * ds * self.k // 2],
                         self.absmax_q[p * nb:(p + 1) * nb],
                         self.absmax_scale[p * (nb // 256):(p + 1) * (nb // 256)] if self.nsec > 1
                         else self.absmax_scale,
                         self.absmax_mean[p:p + 1])

    def desc(self) -> _Nf4Desc:
        return _Nf4Desc(self.d, self.k, self.codes.data_ptr(), self.absmax_q.data_ptr(),
                        self.absmax_scale.data_ptr(), self.absmax_mean.data_ptr())

    @property
    def device(self):
        return self.codes.device


def quantize(W0: torch.Tensor, out: NF4Weight | None = None) -> NF4Weight:
    """NF4 + double-quantised absmax of a d x k fp32 device tensor."""
    assert W0.dtype == torch.float32 and W0.dim() == 2 and W0.is_contiguous()
    d, k = W0.shape
    w = out if out is not None else NF4Weight.empty(d, k, W0.device)
    ws = _workspace(_lib.qlora_quantize_workspace_bytes(d, k), W0.device)
    desc = w.desc()
    _check(_lib.nf4_quantize(W0.data_ptr(), d, k, ctypes.byref(desc), _ptr(ws),
                             0 if ws is None else ws.numel(), _stream(W0.device)), "nf4_quantize")
    return w


def quantize_sections(W0s) -> NF4Weight:
    """Row-stacked NF4 storage of several d_p x k fp32 weights of one shape
    (e.g. a layer's q, k and v projections), each quantised on its own."""
    n = len(W0s)
    d, k = W0s[0].shape
    assert all(W.shape == (d, k) for W in W0s)
    w = NF4Weight.empty(n * d, k, W0s[0].device, nsec=n)
    for p, W in enumerate(W0s):
        quantize(W, out=w.section(p))
    return w


def _rank(A):
    return 0 if A is None else int(A.shape[0])


def forward(X: torch.Tensor, w: NF4Weight, A=None, B=None, alpha: float = 0.0,
            save_t: bool = False, out: torch.Tensor | None = None):
    """Y = X w~^T + (alpha/r) (X A^T) B^T (bf16).  With ``save_t`` also
    returns the saved T^T buffer for ``backward``."""
    assert w.nsec == 1, "a weight with row sections goes through forward_sections"
    M = X.shape[0]
    r = _rank(A)
    dev = X.device
    Y = out if out is not None else torch.empty((M, w.d), dtype=torch.bfloat16, device=dev)
    T = None
    if save_t and r > 0:
        T = torch.empty(max(1, _lib.qlora_tsave_bytes(M, r) // 2), dtype=torch.bfloat16, device=dev)
    ws = _workspace(_lib.qlora_forward_workspace_bytes(M, w.d, w.k, r), dev)
    desc = w.desc()
    _check(_lib.qlora_forward(X.data_ptr(), M, ctypes.byref(desc), _ptr(A), _ptr(B), r,
                              float(alpha), Y.data_ptr(), _ptr(T), _ptr(ws),
                              0 if ws is None else ws.numel(), _stream(dev)), "qlora_forward")
    return (Y, T) if save_t else Y


def backward(dY: torch.Tensor, X: torch.Tensor, w: NF4Weight, A=None, B=None,
             alpha: float = 0.0, T_saved=None, need_dx: bool = True):
    """(dX, dA, dB) of the adapted linear; dX is None when ``need_dx`` is
    False; dA/dB are None when r == 0."""
    assert w.nsec == 1, "a weight with row sections goes through backward_sections"
    M = X.shape[0]
    r = _rank(A)
    dev = X.device
    dX = torch.empty((M, w.k), dtype=torch.bfloat16, device=dev) if need_dx else None
    dA = torch.empty((r, w.k), dtype=torch.bfloat16, device=dev) if r else None
    dB = torch.empty((w.d, r), dtype=torch.bfloat16, device=dev) if r else None
    ws = _workspace(_lib.qlora_backward_workspace_bytes(M, w.d, w.k, r), dev)
    desc = w.desc()
    _check(_lib.qlora_backward(dY.data_ptr(), X.data_ptr(), M, ctypes.byref(desc), _ptr(A),
                               _ptr(B), r, float(alpha), _ptr(T_saved), _ptr(dX), _ptr(dA),
                               _ptr(dB), _ptr(ws), 0 if ws is None else ws.numel(),
                               _stream(dev)), "qlora_backward")
    return dX, dA, dB


def backward_noalloc(dY: torch.Tensor, X: torch.Tensor, w: NF4Weight, A=None, B=None,
                     alpha: float = 0.0, T_saved=None, out=None):
    """``backward`` through qlora_backward_noalloc: no workspace; the library
    uses its static per-GPU scratch array.  ``out`` = (dX, dA, dB) to write
    into preallocated tensors (dX may be None to skip it)."""
    assert w.nsec == 1
    M = X.shape[0]
    r = _rank(A)
    dev = X.device
    if out is None:
        out = (torch.empty((M, w.k), dtype=torch.bfloat16, device=dev),
               torch.empty((r, w.k), dtype=torch.bfloat16, device=dev) if r else None,
               torch.empty((w.d, r), dtype=torch.bfloat16, device=dev) if r else None)
    dX, dA, dB = out
    desc = w.desc()
    _check(_lib.qlora_backward_noalloc(dY.data_ptr(), X.data_ptr(), M, ctypes.byref(desc), _ptr(A),
                                       _ptr(B), r, float(alpha), _ptr(T_saved), _ptr(dX), _ptr(dA),
                                       _ptr(dB), _stream(dev)), "qlora_backward_noalloc")
    return dX, dA, dB


def forward_sections(X: torch.Tensor, w: NF4Weight, A=None, B=None, alpha: float = 0.0,
                     save_t: bool = False, out: torch.Tensor | None = None):
    """Y (M x d) of the w.nsec projections stacked in ``w`` that share the
    input X: section p's columns are X w~_p^T + (alpha/r) (X A_p^T) B_p^T,
    with A = [A_0; A_1; ...] ((nsec*r) x k) and B = [B_0; B_1; ...] (d x r)."""
    M = X.shape[0]
    rt = _rank(A)
    r = rt // w.nsec
    dev = X.device
    Y = out if out is not None else torch.empty((M, w.d), dtype=torch.bfloat16, device=dev)
    T = None
    if save_t and r > 0:
        T = torch.empty(max(1, _lib.qlora_tsave_bytes(M, rt) // 2), dtype=torch.bfloat16, device=dev)
    ws = _workspace(_lib.qlora_forward_workspace_bytes(M, w.d, w.k, rt), dev)
    desc = w.desc()
    _check(_lib.qlora_forward_sections(X.data_ptr(), M, ctypes.byref(desc), w.nsec, _ptr(A), _ptr(B),
                                       r, float(alpha), Y.data_ptr(), _ptr(T), _ptr(ws),
                                       0 if ws is None else ws.numel(), _stream(dev)),
           "qlora_forward_sections")
    return (Y, T) if save_t else Y


def forward_dropout(X: torch.Tensor, w: NF4Weight, A, B, alpha: float, keep: torch.Tensor, p: float,
                    save_t: bool = False, out: torch.Tensor | None = None, xd_out: torch.Tensor | None = None):
    """``forward`` with LoRA dropout on the adapter path's input: keep is an
    M x k uint8 mask (nonzero = kept), p the dropout probability.  With
    ``xd_out`` (M x k bf16) the dropped input is kept there for
    ``backward_dropout(..., Xd_saved=xd_out)``."""
    assert w.nsec == 1 and keep.dtype == torch.uint8 and keep.is_contiguous()
    M = X.shape[0]
    r = _rank(A)
    dev = X.device
    Y = out if out is not None else torch.empty((M, w.d), dtype=torch.bfloat16, device=dev)
    T = None
    if save_t and r > 0:
        T = torch.empty(max(1, _lib.qlora_tsave_bytes(M, r) // 2), dtype=torch.bfloat16, device=dev)
    ws = _workspace(_lib.qlora_forward_dropout_workspace_bytes(M, w.d, w.k, r), dev)
    desc = w.desc()
    _check(_lib.qlora_forward_dropout(X.data_ptr(), M, ctypes.byref(desc), _ptr(A), _ptr(B), r, float(alpha),
                                      keep.data_ptr(), float(p), Y.data_ptr(), _ptr(T), _ptr(xd_out), _ptr(ws),
                                      0 if ws is None else ws.numel(), _stream(dev)), "qlora_forward_dropout")
    return (Y, T) if save_t else Y


def backward_dropout(dY: torch.Tensor, X: torch.Tensor, w: NF4Weight, A, B, alpha: float,
                     keep: torch.Tensor, p: float, T_saved=None, need_dx: bool = True, Xd_saved=None):
    """``backward`` for ``forward_dropout`` (the same mask and p)."""
    assert w.nsec == 1 and keep.dtype == torch.uint8 and keep.is_contiguous()
    M = X.shape[0]
    r = _rank(A)
    dev = X.device
    dX = torch.empty((M, w.k), dtype=torch.bfloat16, device=dev) if need_dx else None
    dA = torch.empty((r, w.k), dtype=torch.bfloat16, device=dev) if r else None
    dB = torch.empty((w.d, r), dtype=torch.bfloat16, device=dev) if r else None
    ws = _workspace(_lib.qlora_backward_dropout_workspace_bytes(M, w.d, w.k, r), dev)
    desc = w.desc()
    _check(_lib.qlora_backward_dropout(dY.data_ptr(), X.data_ptr(), M, ctypes.byref(desc), _ptr(A), _ptr(B), r,
                                       float(alpha), keep.data_ptr(), float(p), _ptr(T_saved), _ptr(Xd_saved),
                                       _ptr(dX),
                                       _ptr(dA), _ptr(dB), _ptr(ws), 0 if ws is None else ws.numel(),
                                       _stream(dev)), "qlora_backward_dropout")
    return dX, dA, dB


def forward_multi(X: torch.Tensor, w: NF4Weight, A, B, idx: torch.Tensor, alpha: float,
                  out: torch.Tensor | None = None):
    """Y (M x d) with a per-token adapter: token m adds (alpha/r) (X[m]
    A_a^T) B_a^T for a = idx[m] in [0, nad), nothing otherwise.  A is
    (nad*r) x k, B is (nad*d) x r (blocks B_0, B_1, ...), idx int32 [M]."""
    assert w.nsec == 1 and idx.dtype == torch.int32 and idx.is_contiguous()
    M = X.shape[0]
    nad = B.shape[0] // w.d
    r = A.shape[0] // nad
    dev = X.device
    Y = out if out is not None else torch.empty((M, w.d), dtype=torch.bfloat16, device=dev)
    ws = _workspace(_lib.qlora_forward_multi_workspace_bytes(M, w.d, w.k, nad, r), dev)
    desc = w.desc()
    _check(_lib.qlora_forward_multi(X.data_ptr(), M, ctypes.byref(desc), nad, A.data_ptr(), B.data_ptr(),
                                    idx.data_ptr(), r, float(alpha), Y.data_ptr(), _ptr(ws),
                                    0 if ws is None else ws.numel(), _stream(dev)), "qlora_forward_multi")
    return Y


def backward_sections(dY: torch.Tensor, X: torch.Tensor, w: NF4Weight, A=None, B=None,
                      alpha: float = 0.0, T_saved=None, need_dx: bool = True):
    """(dX, dA, dB) for ``forward_sections``: dA stacks the sections' dA_p
    like A, dB their dB_p like B."""
    M = X.shape[0]
    rt = _rank(A)
    r = rt // w.nsec
    dev = X.device
    dX = torch.empty((M, w.k), dtype=torch.bfloat16, device=dev) if need_dx else None
    dA = torch.empty((rt, w.k), dtype=torch.bfloat16, device=dev) if rt else None
    dB = torch.empty((w.d, r), dtype=torch.bfloat16, device=dev) if rt else None
    ws = _workspace(_lib.qlora_backward_workspace_bytes(M, w.d, w.k, rt), dev)
    desc = w.desc()
    _check(_lib.qlora_backward_sections(dY.data_ptr(), X.data_ptr(), M, ctypes.byref(desc), w.nsec,
                                        _ptr(A), _ptr(B), r, float(alpha), _ptr(T_saved), _ptr(dX),
                                        _ptr(dA), _ptr(dB), _ptr(ws), 0 if ws is None else ws.numel(),
                                        _stream(dev)), "qlora_backward_sections")
    return dX, dA, dB


# ------------------------------------------- 8-bit activation checkpoints ----

@dataclass
class Checkpoint:
    """An M x k bf16 activation kept at 8 bits (caller-owned device buffers).

    Column block b of 64 columns has one constant per token, in ``absmax[b]``
    (bf16; rows of M rounded up to 64, the padding unspecified)."""
    M: int
    k: int
    codes: torch.Tensor   # int8 [M, k]
    absmax: torch.Tensor  # bfloat16 [k/64, roundup(M, 64)]

    @staticmethod
    def empty(M: int, k: int, device) -> "Checkpoint":
        if M < 0 or k < 64 or k % 64:
            raise ValueError("a checkpoint has M >= 0 tokens of k columns, a multiple of 64")
        return Checkpoint(M, k, torch.empty((M, k), dtype=torch.int8, device=device),
                          torch.empty((k // 64, (M + 63) // 64 * 64), dtype=torch.bfloat16, device=device))

    def check(self, M: int, k: int, device) -> None:
        """Raise unless this is the checkpoint of an M x k tensor on ``device``."""
        if self.M != M or self.k != k:
            raise ValueError(f"the checkpoint is of {self.M} x {self.k}, not {M} x {k}")
        _dense("codes", self.codes, torch.int8, (M, k), device)
        _dense("absmax", self.absmax, torch.bfloat16, (k // 64, (M + 63) // 64 * 64), device)


def _dense(name: str, t: torch.Tensor, dtype, shape, device) -> None:
    """Raise unless t is a contiguous tensor of that type and shape on ``device``."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} is contiguous, {dtype}, of shape {tuple(shape)}, on {device}")


def _activation(name: str, t: torch.Tensor) -> torch.device:
    """The GPU of a contiguous bf16 matrix."""
    if t.dtype is not torch.bfloat16 or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} is a contiguous bfloat16 matrix")
    return _on_gpu(t)


def _new_checkpoint(X: torch.Tensor, M: int, k: int) -> Checkpoint:
    if k < 64 or k % 64:
        raise ValueError("a checkpoint's columns are a multiple of 64")
    return Checkpoint(M, k, torch.empty_like(X, dtype=torch.int8), X.new_empty(k // 64, (M + 63) // 64 * 64))


def checkpoint_save(X: torch.Tensor, out: Checkpoint | None = None) -> Checkpoint:
    """X (M x k bf16, k a multiple of 64) at 8 bits: int8 codes and a bf16
    constant for every 64 columns of a token."""
    dev = _activation("X", X)
    M, k = X.shape
    if out is None:
        out = _new_checkpoint(X, M, k)
    else:
        out.check(M, k, dev)
    _run("qlora_checkpoint_save", dev, X.data_ptr(), M, k, out.codes.data_ptr(), out.absmax.data_ptr())
    return out


def checkpoint_load(ck: Checkpoint, out: torch.Tensor | None = None) -> torch.Tensor:
    """What the checkpoint stands for (M x k bf16)."""
    dev = _on_gpu(ck.codes)
    ck.check(ck.M, ck.k, dev)
    if out is None:
        out = torch.empty_like(ck.codes, dtype=torch.bfloat16)
    else:
        _dense("out", out, torch.bfloat16, (ck.M, ck.k), dev)
    _run("qlora_checkpoint_load", dev, ck.codes.data_ptr(), ck.absmax.data_ptr(), ck.M, ck.k, out.data_ptr())
    return out


def _adapter(w: NF4Weight, A, B, device) -> int:
    """Ranks of each of w's sections."""
    if A is None and B is None:
        return 0
    if A is None or B is None:
        raise ValueError("A and B come together")
    rt, nsec = A.shape[0], w.nsec
    if rt % nsec:
        raise ValueError("A holds the same number of ranks for every section")
    _dense("A", A, torch.bfloat16, (rt, w.k), device)
    _dense("B", B, torch.bfloat16, (w.d, rt // nsec), device)
    return rt // nsec


def forward_checkpoint(X: torch.Tensor, w: NF4Weight, A=None, B=None, alpha: float = 0.0,
                       out: torch.Tensor | None = None, ck: Checkpoint | None = None):
    """(Y, T, checkpoint): ``forward`` (``forward_sections`` for a weight with
    sections) that keeps what ``backward_checkpoint`` needs: T and, in place
    of X, its checkpoint (written into ``ck`` if given).  T is None without an
    adapter."""
    dev = _activation("X", X)
    M, k = X.shape
    if k != w.k or w.codes.device != dev:
        raise ValueError(f"X and the weight have the same {w.k} columns and are on one GPU")
    r = _adapter(w, A, B, dev)
    rt = r * w.nsec
    if out is None:
        out = X.new_empty(M, w.d)
    else:
        _dense("out", out, torch.bfloat16, (M, w.d), dev)
    T = X.new_empty(rt, (M + 63) // 64 * 64) if r > 0 else None
    if ck is None:
        ck = _new_checkpoint(X, M, k)
    else:
        ck.check(M, k, dev)
    if M == 0:  # empty tensors have no address
        return out, T, ck
    nws = _lib.qlora_forward_workspace_bytes(M, w.d, k, rt)
    ws = _workspace(nws, dev)
    desc = w.desc()
    _run("qlora_forward_checkpoint", dev, X.data_ptr(), M, ctypes.byref(desc), w.nsec, _ptr(A), _ptr(B), r,
         float(alpha), out.data_ptr(), _ptr(T), ck.codes.data_ptr(), ck.absmax.data_ptr(), _ptr(ws), nws)
    return out, T, ck


def backward_checkpoint(dY: torch.Tensor, ck: Checkpoint, w: NF4Weight, A=None, B=None, alpha: float = 0.0,
                        T_saved: torch.Tensor | None = None, need_dx: bool = True, keep: torch.Tensor | None = None,
                        p: float = 0.0):
    """(dX, dA, dB) of ``forward_checkpoint``: dA from what the checkpoint
    stands for, dX and dB as ``backward`` gives them.  T_saved is required
    with an adapter.  With ``keep`` and ``p`` the gradients are
    ``backward_dropout``'s, ck being the checkpoint of the dropped input
    (``forward_dropout``'s xd_out)."""
    dev = _activation("dY", dY)
    M, k, d = dY.shape[0], w.k, w.d
    if dY.shape[1] != d or w.codes.device != dev:
        raise ValueError(f"dY has the weight's {d} columns and is on its GPU")
    r = _adapter(w, A, B, dev)
    rt = r * w.nsec
    codes = absmax = mask = dA = dB = T = None
    if r > 0:
        if ck is None:
            raise ValueError("an adapter's gradients need the checkpoint")
        ck.check(M, k, dev)
        codes, absmax, T = ck.codes.data_ptr(), ck.absmax.data_ptr(), T_saved
        ldt = (M + 63) // 64 * 64  # a T of another M has other rows: ranks would be read from wrong places
        if T is None or T.dtype is not torch.bfloat16 or not T.is_contiguous() or T.device != dev \
                or M > 0 and T.shape != (rt, ldt) and T.shape != (rt * ldt,):
            raise ValueError(f"T_saved is the T that the forward returned: {rt} x {ldt}, torch.bfloat16, on {dev}")
        if keep is not None:
            _dense("keep", keep, torch.uint8, (M, k), dev)
            mask = keep.data_ptr()
        new = dY.new_empty if M else dY.new_zeros  # without a token the sums are empty and nothing is launched
        dA, dB = new(rt, k), new(d, r)
    dX = dY.new_empty(M, k) if need_dx else None
    if M == 0:
        return dX, dA, dB
    nws = _lib.qlora_backward_workspace_bytes(M, d, k, rt)
    ws = _workspace(nws, dev)
    desc = w.desc()
    _run("qlora_backward_checkpoint", dev, dY.data_ptr(), codes, absmax, M, ctypes.byref(desc), w.nsec, _ptr(A),
         _ptr(B), r, float(alpha), mask, float(p), _ptr(T), _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws), nws)
    return dX, dA, dB


def adam_step(P: torch.Tensor, W: torch.Tensor, G: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
              lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
              weight_decay: float = 0.0) -> None:
    """One Adam step: W, m, v (fp32) in place, P = bf16(W); G bf16 gradients."""
    n = P.numel()
    assert P.dtype == torch.bfloat16 and G.dtype == torch.bfloat16 and G.numel() == n
    assert W.dtype == m.dtype == v.dtype == torch.float32 and W.numel() == m.numel() == v.numel() == n
    _check(_lib.qlora_adam_step(P.data_ptr(), W.data_ptr(), G.data_ptr(), m.data_ptr(), v.data_ptr(), n,
                                float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                                int(step), _stream(P.device)), "qlora_adam_step")


# ------------------------------------------------ losses on the logits ----

_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_KINDS = {"sigmoid": 0, "hinge": 1, "squared": 2}


def _on_gpu(t: torch.Tensor):
    if t.device.type != "cuda":
        raise ValueError("the tensors have to be on a GPU")
    return t.device


def _run(call: str, dev, *args) -> None:
    """The C call with the tensors' GPU current: a default stream is a GPU's
    own only while that GPU is."""
    if torch._C._cuda_getDevice() == dev.index:
        _check(getattr(_lib, call)(*args, _stream(dev)), call)
    else:
        with torch.cuda.device(dev):
            _check(getattr(_lib, call)(*args, _stream(dev)), call)


def _room(t: torch.Tensor) -> int:
    """Elements from t's first to the end of its storage."""
    return t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()


def _own_stride(t: torch.Tensor):
    """The longest row stride of t whose gaps are t's own, by the tensor that t
    is a view of: that tensor's row, where t starts with one.  None where there
    is no such row (a flat buffer, or a tensor of its own)."""
    V, base = t.shape[1], t._base
    if base is None:  # views are not known of in inference mode: less than another row of V
        return 2 * V - 1 if t.is_inference() else None
    steps = sorted(s for n, s in zip(base.shape, base.stride()) if n > 1)
    if base.dim() < 2 or steps[:1] != [1]:
        return None
    size = t.element_size()
    row = (steps[1] if len(steps) > 1 else base.numel()) * base.element_size() // size
    first = t.storage_offset() - base.storage_offset() * base.element_size() // size
    if row < V:  # a buffer's shape
        return None
    return row if first % row == 0 else V


def _row_stride(t: torch.Tensor) -> int:
    """Row stride of a T x V tensor.  A single row has none of its own: that of
    the padded matrix that it was sliced from, or says nothing."""
    (T, V), ld = t.shape, t.stride(0)
    if T > 1 or ld == V:
        return ld
    own = _own_stride(t)
    if own is not None and t._base is not None:
        ld = own
    return ld if V <= ld <= min(_room(t), 2 * V - 1 if own is None else own) else V


def _rows(logits: torch.Tensor):
    """(T, V, row stride) of logits whose rows are contiguous."""
    if logits.dim() != 2 or logits.dtype not in _DTYPES:
        raise TypeError("logits are a T x V tensor of bfloat16 or float32")
    T, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("the logits of one token have to be contiguous")
    return T, V, _row_stride(logits)


def _per(name: str, t, n: int, dtype, device):
    """Pointer of an optional contiguous vector of n values on ``device``."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != (n,) or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} is a contiguous vector of {n} {dtype} on {device}")
    return t.data_ptr()


def _grad_rows(logits: torch.Tensor, out, T: int, V: int, ld: int):
    """The tensor that receives dlogits and its row stride.  Rows are written
    to their whole stride, so the storage has to hold them."""
    if out is None:
        # a padded head's gradient keeps the padding (as zeros), with rows
        # that start where the logits' rows do
        ldd = ld if ld - V < 256 else V
        rows = logits.new_empty(T, ldd)
        return (rows if ldd == V else rows.narrow(1, 0, V)), ldd
    if out.shape != logits.shape or out.dtype != logits.dtype or out.device != logits.device:
        raise ValueError("out has the shape, type and device of the logits")
    if V > 1 and out.stride(1) != 1:
        raise ValueError("the gradient of one token has to be contiguous")
    ldd = _row_stride(out)
    own = _own_stride(out) if T > 1 and ldd > V else None
    if own is not None and ldd > own:
        raise ValueError("between out's rows lie other rows or columns of its tensor: the rows are written whole")
    if T * ldd > _room(out):
        raise ValueError("out's last row ends before its stride: the rows are written whole")
    return out, ldd


def token_logprobs(logits: torch.Tensor, labels: torch.Tensor, inv_temperature: float = 1.0,
                   save_stats: bool = False):
    """Log-probability of each token's label (fp32 [T]) under T x V logits
    (bf16 or fp32; rows may be a slice of a wider matrix).  A label (int32)
    outside [0, V) gives 0.  With ``save_stats`` also returns the rows'
    statistics for ``token_logprobs_backward``."""
    T, V, ld = _rows(logits)
    dev = logits.device
    y = _per("labels", labels, T, torch.int32, dev)
    logp = torch.empty(T, dtype=torch.float32, device=_on_gpu(logits))
    stats = torch.empty((T, 2), dtype=torch.float32, device=dev) if save_stats else None
    _run("qlora_token_logprobs", dev, logits.data_ptr(), _DTYPES[logits.dtype], T, V, ld, y, float(inv_temperature),
         logp.data_ptr(), _ptr(stats))
    return (logp, stats) if save_stats else logp


def token_logprobs_backward(dlogp: torch.Tensor, logits: torch.Tensor, labels: torch.Tensor, stats: torch.Tensor,
                            inv_temperature: float = 1.0, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient in the logits for ``dlogp`` = d loss / d logp (fp32 [T]).
    ``out`` may be the logits themselves.  Rows of ``out`` are written to
    their whole stride: of a slice ``dY[:, :V]`` the columns from V on get
    zeros, so dY is ready for the head's backward.  A slice between whose rows
    others of its tensor lie (``d[:, 0]`` of B x S x V, ``d[::2]``) is refused
    for that; a single row has no stride and leaves its neighbours."""
    T, V, ld = _rows(logits)
    dev = logits.device
    g = _per("dlogp", dlogp, T, torch.float32, dev)
    y = _per("labels", labels, T, torch.int32, dev)
    if stats.shape != (T, 2) or stats.dtype != torch.float32 or not stats.is_contiguous() or stats.device != dev:
        raise ValueError("stats are the T x 2 values that token_logprobs returned")
    out, ldd = _grad_rows(logits, out, T, V, ld)
    _on_gpu(logits)
    _run("qlora_token_logprobs_backward", dev, g, logits.data_ptr(), _DTYPES[logits.dtype], T, V, ld, y,
         float(inv_temperature), stats.data_ptr(), out.data_ptr(), ldd)
    return out


def preference_loss(logp: torch.Tensor, labels: torch.Tensor, vocab: int, cu_seqlens: torch.Tensor, beta: float,
                    ref_logp: torch.Tensor | None = None, kind: str = "sigmoid", average: bool = False,
                    label_smoothing: float = 0.0, margin: float = 0.0, weight: torch.Tensor | None = None,
                    need_grad: bool = True):
    """(loss [P], reward [2P], dlogp [T]) of P pairs of sequences at offsets
    ``cu_seqlens`` (int32 [2P + 1]; the P chosen ones first, then the P
    rejected ones), from the tokens' log-probabilities under the policy and,
    optionally, a reference.  ``kind`` is "sigmoid", "hinge" or "squared";
    ``weight`` [P] weights the pairs in dlogp.  dlogp is None without
    ``need_grad``."""
    if kind not in _KINDS:
        raise ValueError(f"kind is one of {sorted(_KINDS)}")
    if logp.dim() != 1 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] % 2 != 1:
        raise ValueError("logp is a vector and cu_seqlens holds 2P + 1 offsets")
    T, P, dev = logp.shape[0], cu_seqlens.shape[0] // 2, logp.device
    lp = _per("logp", logp, T, torch.float32, dev)
    y = _per("labels", labels, T, torch.int32, dev)
    cu = _per("cu_seqlens", cu_seqlens, 2 * P + 1, torch.int32, dev)
    ref = _per("ref_logp", ref_logp, T, torch.float32, dev)
    wt = _per("weight", weight, P, torch.float32, dev)
    loss = torch.empty(P, dtype=torch.float32, device=_on_gpu(logp))
    reward = torch.empty(2 * P, dtype=torch.float32, device=dev)
    dlogp = None
    if need_grad:  # without a pair there is no loss and nothing is launched
        dlogp = (torch.empty if P else torch.zeros)(T, dtype=torch.float32, device=dev)
    _run("qlora_preference_loss", dev, lp, ref, y, T, int(vocab), cu, P, _KINDS[kind], int(average), float(beta),
         float(label_smoothing), float(margin), wt, loss.data_ptr(), reward.data_ptr(), _ptr(dlogp))
    return loss, reward, dlogp


def policy_loss(logits: torch.Tensor, labels: torch.Tensor, advantages: torch.Tensor,
                old_logp: torch.Tensor | None = None, ref_logp: torch.Tensor | None = None,
                weight: torch.Tensor | None = None, clip_low: float = 0.2, clip_high: float = 0.2,
                kl_coef: float = 0.0, inv_temperature: float = 1.0, need_grad: bool = True,
                out: torch.Tensor | None = None):
    """(loss [T], kl [T], logp [T], dlogits) of the clipped policy loss with a
    KL term, per token; dlogits is the gradient of sum(weight * loss) and is
    None without ``need_grad``.  ``out`` as in ``token_logprobs_backward``
    (it may be the logits)."""
    T, V, ld = _rows(logits)
    dev = logits.device
    y = _per("labels", labels, T, torch.int32, dev)
    vec = [_per(n, t, T, torch.float32, dev) for n, t in (("advantages", advantages), ("old_logp", old_logp),
                                                          ("ref_logp", ref_logp), ("weight", weight))]
    loss, kl, logp = torch.empty((3, T), dtype=torch.float32, device=_on_gpu(logits)).unbind(0)
    dlogits, ldd = _grad_rows(logits, out, T, V, ld) if need_grad else (None, 0)
    _run("qlora_policy_loss", dev, logits.data_ptr(), _DTYPES[logits.dtype], T, V, ld, y, float(inv_temperature), *vec,
         float(clip_low), float(clip_high), float(kl_coef), loss.data_ptr(), kl.data_ptr(), logp.data_ptr(),
         _ptr(dlogits), ldd)
    return loss, kl, logp, dlogits


def _tokens(tokens, T: int, dev):
    """(pointer, number of tokens a row, whether they came as a vector)."""
    if tokens is None:
        return None, 0, False
    if tokens.dtype != torch.int32 or tokens.dim() not in (1, 2) or tokens.shape[0] != T \
            or not tokens.is_contiguous() or tokens.device != dev:
        raise ValueError(f"tokens are a contiguous vector of {T}, or matrix of {T} rows, of torch.int32 on {dev}")
    return (tokens.data_ptr(), 1, True) if tokens.dim() == 1 else (tokens.data_ptr(), tokens.shape[1], False)


def token_scores(logits: torch.Tensor, tokens: torch.Tensor | None = None, top: int = 0,
                 inv_temperature: float = 1.0, save_stats: bool = False):
    """(logp, entropy [T], top_ids [T, top], top_logp [T, top]) of T x V logits
    (bf16 or fp32; rows may be a slice of a wider matrix): the
    log-probabilities of the given tokens (int32 [T] or [T, m], logp of their
    shape, None without tokens), the distribution's entropy, and its ``top``
    (up to 64) best words, the lowest index first among equal logits (both
    None for top = 0).  A token
    outside [0, V) does not count and gives 0; of a row without one that
    counts nothing is read (entropy 0, ids -1 at -inf).  Masked words (-inf)
    are no alternatives: past the last finite one ids are -1 at -inf.  With
    ``save_stats`` also returns the rows' statistics for
    ``token_scores_backward``."""
    T, V, ld = _rows(logits)
    dev = logits.device
    y, m, flat = _tokens(tokens, T, dev)
    if not 0 <= top <= 64 or top > V or m > 64:
        raise ValueError("up to 64 tokens a row and 64 alternatives, no more than there are words")
    entropy = torch.empty(T, dtype=torch.float32, device=_on_gpu(logits))
    logp = None if tokens is None else torch.empty_like(tokens, dtype=torch.float32)
    ids = best = stats = None
    if top:
        best = entropy.new_empty(T, top)
        ids = torch.empty_like(best, dtype=torch.int32)
    if save_stats:
        stats = entropy.new_empty(T, 3)
    _run("qlora_token_scores", dev, logits.data_ptr(), _DTYPES[logits.dtype], T, V, ld, y, m, int(top),
         float(inv_temperature), _ptr(logp), entropy.data_ptr(), _ptr(ids), _ptr(best), _ptr(stats))
    return (logp, entropy, ids, best, stats) if save_stats else (logp, entropy, ids, best)


def token_scores_backward(dlogp: torch.Tensor | None, dentropy: torch.Tensor | None, logits: torch.Tensor,
                          tokens: torch.Tensor | None, stats: torch.Tensor, inv_temperature: float = 1.0,
                          out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient in the logits for ``dlogp`` = d loss / d logp (fp32, of the
    tokens' shape; None without tokens) and ``dentropy`` = d loss / d entropy
    (fp32 [T], None for a loss without it).  ``out`` as in
    ``token_logprobs_backward`` (it may be the logits).  A loss on the top
    alternatives gives their ids as tokens: an id of -1 does not count, and
    one that is there twice gets both gradients.  A row of which the forward
    read nothing has no statistics: a token that counts there makes its
    gradient NaN."""
    T, V, ld = _rows(logits)
    dev = logits.device
    y, m, _ = _tokens(tokens, T, dev)
    if m > 64:
        raise ValueError("up to 64 tokens a row")
    if (dlogp is None) != (tokens is None):
        raise ValueError("dlogp and tokens come together")
    if dlogp is not None and (dlogp.dtype != torch.float32 or dlogp.shape != tokens.shape
                              or not dlogp.is_contiguous() or dlogp.device != dev):
        raise ValueError(f"dlogp is contiguous, torch.float32, of the tokens' shape, on {dev}")
    ge = _per("dentropy", dentropy, T, torch.float32, dev)
    if stats.shape != (T, 3) or stats.dtype != torch.float32 or not stats.is_contiguous() or stats.device != dev:
        raise ValueError("stats are the T x 3 values that token_scores returned")
    out, ldd = _grad_rows(logits, out, T, V, ld)
    _on_gpu(logits)
    _run("qlora_token_scores_backward", dev, _ptr(dlogp), ge, logits.data_ptr(), _DTYPES[logits.dtype], T, V, ld, y, m,
         float(inv_temperature), stats.data_ptr(), out.data_ptr(), ldd)
    return out


def muon_step(P: torch.Tensor, W: torch.Tensor, G: torch.Tensor, m: torch.Tensor, lr: float, momentum: float = 0.95,
              nesterov: bool = True, weight_decay: float = 0.0, ns_steps: int = 5, scale: float | None = None,
              coefficients=None, eps: float = 1e-7) -> None:
    """One step of momentum with an orthogonalised update on one adapter
    factor (rows x cols) or a stack of them (n x rows x cols, as the A or B
    of several sections): W and m (fp32) in place, P = bf16(W); G bf16
    gradients.  ``scale`` is the update's size in units of lr, by default
    sqrt(max(1, rows / cols)); ``coefficients`` is one (a, b, c) for every
    step or a sequence of ns_steps of them."""
    if W.dim() not in (2, 3):
        raise ValueError("W is rows x cols or n x rows x cols")
    rows, cols = W.shape[-2:]
    nmat = W.shape[0] if W.dim() == 3 else 1
    for name, t, dtype in (("P", P, torch.bfloat16), ("W", W, torch.float32), ("G", G, torch.bfloat16),
                           ("m", m, torch.float32)):
        if t.dtype != dtype or t.shape != W.shape or not t.is_contiguous():
            raise ValueError(f"{name} is contiguous, {dtype}, of shape {tuple(W.shape)}")
    if scale is None:
        scale = max(1.0, rows / max(1, cols)) ** 0.5
    coef = None
    if coefficients is not None:
        c = [list(t) for t in coefficients] if isinstance(coefficients[0], (list, tuple)) \
            else [list(coefficients)] * ns_steps
        if len(c) != ns_steps or any(len(t) != 3 for t in c):
            raise ValueError("coefficients: (a, b, c), or ns_steps of them")
        coef = (ctypes.c_float * (3 * ns_steps))(*[v for t in c for v in t])
    dev = _on_gpu(P)
    # like adam_step's, the fp32 state may be paged out to pinned host memory
    if G.device != dev or any(t.device != dev and not t.is_pinned() for t in (W, m)):
        raise ValueError(f"P and G have to be on one GPU ({dev}), W and m there or in pinned host memory")
    ws = _workspace(_lib.qlora_muon_workspace_bytes(nmat, rows, cols), dev)
    _run("qlora_muon_step", dev, P.data_ptr(), W.data_ptr(), G.data_ptr(), m.data_ptr(), nmat, rows, cols, float(lr),
         float(momentum), int(nesterov), float(weight_decay), float(scale), float(eps), int(ns_steps), coef, _ptr(ws),
         0 if ws is None else ws.numel())


def merge(w: NF4Weight, A=None, B=None, alpha: float = 0.0, out=None) -> torch.Tensor:
    """W = bf16(w~ + (alpha/r) B A), d x k bf16 (one section at a time:
    ``merge(w.section(p), A_p, B_p, alpha)``)."""
    assert w.nsec == 1, "merge the sections one at a time through NF4Weight.section"
    r = _rank(A)
    W = out if out is not None else torch.empty((w.d, w.k), dtype=torch.bfloat16, device=w.device)
    desc = w.desc()
    _check(_lib.lora_merge(ctypes.byref(desc), _ptr(A), _ptr(B), r, float(alpha), W.data_ptr(),
                           _stream(w.device)), "lora_merge")
    return W


def unmerge(W: torch.Tensor, A=None, B=None, alpha: float = 0.0, out=None) -> torch.Tensor:
    """W0 = bf16(W - (alpha/r) B A); ``out`` may be ``W`` itself."""
    r = _rank(A)
    d, k = W.shape
    O = out if out is not None else torch.empty_like(W)
    _check(_lib.lora_unmerge(W.data_ptr(), d, k, _ptr(A), _ptr(B), r, float(alpha), O.data_ptr(),
                             _stream(W.device)), "lora_unmerge")
    return O


class kernel_timing:
    """Context manager: per-kernel HIP-event timing of every launch made by
    the library inside the block.  ``totals()`` -> {name: (total_ms, n)}."""

    NAMES = ("quant_blocks", "quant_group_sums", "quant_mean", "quant_dq", "merge", "unmerge",
             "prep_adapters", "lora_proj", "lora_proj_finish", "token_reduce",
             "token_reduce_finish", "fwd_decode", "fwd_decode_finish", "fwd_rich", "dx", "drop_input", "adam",
             "fwd_sum_splits", "dx_sum_splits", "logprob", "logprob_grad", "preference", "policy", "muon_gram",
             "muon_sum", "muon_poly", "muon_apply", "muon_whole", "ck_save", "ck_load", "token_reduce_ck", "scores",
             "scores_grad")

    def __enter__(self):
        _check(_lib.qlora_timing_reset(), "qlora_timing_reset")
        _check(_lib.qlora_timing_enable(1), "qlora_timing_enable")
        return self

    def __exit__(self, *exc):
        _lib.qlora_timing_enable(0)
        _check(_lib.qlora_timing_collect(), "qlora_timing_collect")
        return False

    @staticmethod
    def totals() -> dict:
        out = {}
        for n in kernel_timing.NAMES:
            ms, cnt = ctypes.c_double(), _i64()
            _check(_lib.qlora_timing_query(n.encode(), ctypes.byref(ms), ctypes.byref(cnt)),
                   "qlora_timing_query")
            if cnt.value:
                out[n] = (ms.value, cnt.value)
        return out


__all__ = ["kernel_timing", "NF4Weight", "QloraError", "quantize", "forward", "backward", "merge", "unmerge",
           "quantize_sections", "forward_sections", "backward_sections", "forward_multi", "forward_dropout",
           "backward_dropout", "backward_noalloc", "adam_step", "token_logprobs", "token_logprobs_backward",
           "preference_loss", "policy_loss", "Checkpoint", "checkpoint_save", "checkpoint_load", "forward_checkpoint",
           "backward_checkpoint", "token_scores", "token_scores_backward", "muon_step", "nf4_levels", "nf4_sizes", "lib", "EXPORTED", "LIB_PATH"]
