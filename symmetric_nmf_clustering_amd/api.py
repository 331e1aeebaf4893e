"""Python binding of libsymnmf (argument marshalling only).

Each function takes and returns torch tensors on the current HIP device and
passes raw device pointers, sizes and torch's current stream to the C ABI of
include/symnmf.h. Every step of the path runs in the library's kernels; torch
only supplies device memory and the stream.
"""
from __future__ import annotations

import ctypes
import functools
import math
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

from . import _lib as L

_KINDS = {"abscorr": L.ABSCORR, "corr": L.ABSCORR, "tpdm": L.TPDM}
_SOLVERS = {"auto": L.AUTO, "full": L.FULL, "block_svrg": L.BLOCK_SVRG, "svrg": L.BLOCK_SVRG}
_INITS = {"uniform": L.INIT_UNIFORM, "scale_matched": L.INIT_SCALE_MATCHED, "caller": L.INIT_CALLER}


def _stream_ptr() -> int:
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _require_cuda(t: torch.Tensor, name: str, dtype=torch.float32):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a HIP device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")


def _S_layout(S: torch.Tensor):
    _require_cuda(S, "S")
    if S.dim() != 2 or S.shape[0] != S.shape[1] or S.stride(1) != 1:
        raise ValueError("S must be an n x n row-major view (unit column stride)")
    n = S.shape[0]
    lds = S.stride(0)
    if lds % 4 or S.data_ptr() % 16:
        raise ValueError("S needs a leading dimension that is a multiple of 4 and 16-byte "
                         "alignment; use alloc_S(n) or pad_S(S)")
    return n, lds


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A caller-owned workspace buffer (torch allocations are 256-byte aligned)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8,
                       device=device or torch.device("cuda"))


def workspace_bytes(op: int, n: int, k_or_p: int, T: int = 0, params: Optional[L.FitParams] = None) -> int:
    lib = L.load()
    b = lib.symnmf_workspace_bytes(op, n, k_or_p, T, ctypes.byref(params) if params else None)
    if b == 0:
        raise ValueError("invalid sizes for workspace query")
    return int(b)


def alloc_S(n: int, device=None) -> torch.Tensor:
    """An uninitialised n x n fp32 view with leading dimension round_up(n, 4)."""
    lds = (n + 3) // 4 * 4
    buf = torch.empty((n, lds), dtype=torch.float32, device=device or torch.device("cuda"))
    return buf[:, :n]


def pad_S(S: torch.Tensor) -> torch.Tensor:
    out = alloc_S(S.shape[0], S.device)
    out.copy_(S)
    return out


# ---------------------------------------------------------------------------
def build_S(X: torch.Tensor, kind: str = "abscorr", tail_frac: float = 0.05,
            out: Optional[torch.Tensor] = None):
    """S (n x n fp32) from a T x n returns window X. Returns (S, ||S||_F^2)."""
    _require_cuda(X, "X")
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be T x n row-major")
    T, n = X.shape
    S = alloc_S(n, X.device) if out is None else out
    n_s, lds = _S_layout(S)
    if n_s != n:
        raise ValueError("out has the wrong size")
    lib = L.load()
    ws = workspace(workspace_bytes(L.OP_BUILD_S, n, 1, T), X.device)
    fro = ctypes.c_double(0.0)
    st = lib.symnmf_build_S(_KINDS[kind], _ptr(X), T, n, X.stride(0), float(tail_frac), _ptr(S),
                            lds, ctypes.byref(fro), _ptr(ws), ws.numel(), ctypes.c_void_p(_stream_ptr()))
    L.check(st, "symnmf_build_S")
    return S, fro.value


def spectral_probe(S: torch.Tensor, p: int = 64, max_iters: int = 300, tol: float = 1e-6,
                   seed: int = 0):
    """Top-p eigenvalues of S by magnitude (sign kept). Returns (eigvals, iters, converged)."""
    n, lds = _S_layout(S)
    lib = L.load()
    ws = workspace(workspace_bytes(L.OP_PROBE, n, p), S.device)
    ev = (ctypes.c_double * p)()
    its = ctypes.c_int32(0)
    st = lib.symnmf_spectral_probe(_ptr(S), n, lds, p, max_iters, float(tol), int(seed), ev,
                                   ctypes.byref(its), _ptr(ws), ws.numel(),
                                   ctypes.c_void_p(_stream_ptr()))
    L.check(st, "symnmf_spectral_probe")
    return np.array(ev[:], dtype=np.float64), int(its.value), st == L.OK


def sh(S: torch.Tensor, H: torch.Tensor):
    """One S.H pass: returns (P = S H, tr(H^T S H))."""
    n, lds = _S_layout(S)
    _require_cuda(H, "H")
    if H.dim() != 2 or H.shape[0] != n or not H.is_contiguous():
        raise ValueError("H must be a contiguous n x k tensor")
    k = H.shape[1]
    P = torch.empty_like(H)
    lib = L.load()
    ws = workspace(workspace_bytes(L.OP_SH, n, k), S.device)
    tr = ctypes.c_double(0.0)
    st = lib.symnmf_sh(_ptr(S), n, lds, _ptr(H), k, _ptr(P), ctypes.byref(tr), _ptr(ws),
                       ws.numel(), ctypes.c_void_p(_stream_ptr()))
    L.check(st, "symnmf_sh")
    return P, tr.value


def sh_noalloc(S: torch.Tensor, H: torch.Tensor, out: Optional[torch.Tensor] = None,
               tr_out: Optional[torch.Tensor] = None):
    """The S.H pass on the library's static scratch (no workspace, no device
    allocation inside the call): returns (P, tr) with tr a one-element float64
    device tensor. ``out`` and ``tr_out`` let the caller own every buffer."""
    n, lds = _S_layout(S)
    _require_cuda(H, "H")
    if H.dim() != 2 or H.shape[0] != n or not H.is_contiguous():
        raise ValueError("H must be a contiguous n x k tensor")
    k = H.shape[1]
    P = torch.empty_like(H) if out is None else out
    tr = torch.empty(1, dtype=torch.float64, device=S.device) if tr_out is None else tr_out
    st = L.load().symnmf_sh_noalloc(_ptr(S), n, lds, _ptr(H), k, _ptr(P), _ptr(tr),
                                    ctypes.c_void_p(_stream_ptr()))
    L.check(st, "symnmf_sh_noalloc")
    return P, tr


def sh_sym(S: torch.Tensor, H: torch.Tensor):
    """The S.H pass from the upper triangle of a symmetric S (each block on or
    above the diagonal read once, bf16 matrix cores with split operands):
    returns (P = S H, tr(H^T S H)); k <= 32."""
    n, lds = _S_layout(S)
    _require_cuda(H, "H")
    if H.dim() != 2 or H.shape[0] != n or not H.is_contiguous() or H.dtype != torch.float32:
        raise ValueError("H must be a contiguous float32 n x k tensor")
    k = H.shape[1]
    P = torch.empty_like(H)
    lib = L.load()
    ws = workspace(workspace_bytes(L.OP_SH_SYM, n, k), S.device)
    tr = ctypes.c_double(0.0)
    st = lib.symnmf_sh_sym(_ptr(S), n, lds, _ptr(H), k, _ptr(P), ctypes.byref(tr), _ptr(ws),
                           ws.numel(), ctypes.c_void_p(_stream_ptr()))
    L.check(st, "symnmf_sh_sym")
    return P, tr.value


def sq(S: torch.Tensor, Q: torch.Tensor) -> torch.Tensor:
    """The probe's product Y = S Q on the bf16 matrix cores (three-part split
    operands, fp32 accumulation)."""
    n, lds = _S_layout(S)
    _require_cuda(Q, "Q")
    if Q.dim() != 2 or Q.shape[0] != n or not Q.is_contiguous() or Q.dtype != torch.float32:
        raise ValueError("Q must be a contiguous float32 n x w tensor")
    w = Q.shape[1]
    Y = torch.empty_like(Q)
    lib = L.load()
    ws = workspace(workspace_bytes(L.OP_SQ, n, w), S.device)
    st = lib.symnmf_sq(_ptr(S), n, lds, _ptr(Q), w, _ptr(Y), _ptr(ws), ws.numel(),
                       ctypes.c_void_p(_stream_ptr()))
    L.check(st, "symnmf_sq")
    return Y


@dataclass
class FitState:
    """The AdaptGrow controller state at a returned H: pass it back with that H
    and G (``fit(..., H0=H, G0=G, state=...)``) to continue the run exactly."""
    iter: int
    blocks: int
    anchor_iter: int
    f_prev_valid: int
    f_anchor: float
    f_prev: float
    H_anchor: torch.Tensor
    P_anchor: torch.Tensor


@dataclass
class FitResult:
    H: torch.Tensor
    G: Optional[torch.Tensor]
    report: dict
    f_trace: np.ndarray
    status: int
    state: Optional[FitState] = None

    @property
    def converged(self) -> bool:
        return bool(self.report["converged"])


def fit_params(**kw) -> L.FitParams:
    lib = L.load()
    p = L.FitParams()
    lib.symnmf_fit_params_default(ctypes.byref(p))
    for key, val in kw.items():
        if key == "solver" and isinstance(val, str):
            val = _SOLVERS[val]
        if key == "init" and isinstance(val, str):
            val = _INITS[val]
        if key == "sh_pass" and isinstance(val, str):
            val = {"rows": L.SH_ROWS, "upper": L.SH_UPPER}[val]
        if not hasattr(p, key):
            raise TypeError(f"unknown fit parameter {key}")
        setattr(p, key, val)
    return p


def fit(S: torch.Tensor, k: int, *, eigvals=None, H0: Optional[torch.Tensor] = None,
        G0: Optional[torch.Tensor] = None, return_G: bool = False,
        trace_cap: Optional[int] = None, ws: Optional[torch.Tensor] = None,
        state: Optional[FitState] = None, return_state: bool = False, **params) -> FitResult:
    """SymNMF fit S ~ H H^T with projected AdaGrad / Block-SVRG AdaptGrow.

    ``params`` are the fields of symnmf_fit_params (solver, max_iters, lr, eps,
    block_rows, init, phi0, gap_threshold, tol_rel, stall_tol, init_scale,
    seed, check_every, rms_decay, sh_pass, obj_floor, start_iter). H0 sets
    init='caller'; G0 sets resume=1. ``state`` (a previous result's state,
    with its H as H0 and G as G0) restores the controller and sets start_iter;
    ``return_state`` asks for the state of the returned H."""
    n, lds = _S_layout(S)
    if H0 is not None:
        if params.setdefault("init", L.INIT_CALLER) not in (L.INIT_CALLER, "caller"):
            raise ValueError("H0 given with an init other than 'caller'")
    if G0 is not None:
        params["resume"] = 1
    if state is not None:
        if G0 is None:
            raise ValueError("resuming from a state needs G0")
        params["start_iter"] = state.iter
    p = fit_params(**params)
    H = torch.empty((n, k), dtype=torch.float32, device=S.device)
    if H0 is not None:
        _require_cuda(H0, "H0")
        H.copy_(H0)
    G = None
    if return_G or G0 is not None:
        G = torch.empty((n, k), dtype=torch.float32, device=S.device)
        if G0 is not None:
            G.copy_(G0)
    cap = p.max_iters if trace_cap is None else int(trace_cap)
    trace = (ctypes.c_double * max(cap, 1))()
    ev = None
    n_eig = 0
    if eigvals is not None:
        eig = np.ascontiguousarray(eigvals, dtype=np.float64)
        ev = eig.ctypes.data_as(ctypes.POINTER(ctypes.c_double))
        n_eig = eig.size
    rep = L.FitReport()
    lib = L.load()
    need = workspace_bytes(L.OP_FIT, n, k, 0, p)
    if ws is None or ws.numel() < need:
        ws = workspace(need, S.device)
    cst = None
    Ha_out = Pa_out = None
    if state is not None or return_state:
        Ha_out = torch.empty((n, k), dtype=torch.float32, device=S.device)
        Pa_out = torch.empty((n, k), dtype=torch.float32, device=S.device)
        cst = L.FitState()
        if state is not None:
            for name in ("iter", "blocks", "anchor_iter", "f_prev_valid", "f_anchor", "f_prev"):
                setattr(cst, name, getattr(state, name))
            Ha_out.copy_(state.H_anchor)
            Pa_out.copy_(state.P_anchor)
        cst.H_anchor = Ha_out.data_ptr()
        cst.P_anchor = Pa_out.data_ptr()
    st = lib.symnmf_fit(_ptr(S), n, lds, k, ctypes.byref(p), ev, n_eig, _ptr(H), _ptr(G),
                        trace if cap > 0 else None, cap, ctypes.byref(rep),
                        ctypes.byref(cst) if cst is not None else None, _ptr(ws), ws.numel(),
                        ctypes.c_void_p(_stream_ptr()))
    L.check(st, "symnmf_fit")
    r = rep.as_dict()
    ncopy = min(cap, r["iterations"] + (1 if r["converged"] else 0))
    out_state = None
    if cst is not None:
        out_state = FitState(cst.iter, cst.blocks, cst.anchor_iter, cst.f_prev_valid,
                             cst.f_anchor, cst.f_prev, Ha_out, Pa_out)
    return FitResult(H, G, r, np.array(trace[:ncopy], dtype=np.float64), st, out_state)


def labels(H: torch.Tensor) -> torch.Tensor:
    """Row-wise argmax of H (lowest index on ties) as int32."""
    _require_cuda(H, "H")
    if H.dim() != 2 or not H.is_contiguous():
        raise ValueError("H must be a contiguous n x k tensor")
    n, k = H.shape
    out = torch.empty(n, dtype=torch.int32, device=H.device)
    st = L.load().symnmf_labels(_ptr(H), n, k, _ptr(out), ctypes.c_void_p(_stream_ptr()))
    L.check(st, "symnmf_labels")
    return out


@dataclass
class KmeansResult:
    labels: torch.Tensor
    centroids: Optional[torch.Tensor]
    iterations: int
    converged: bool
    objective: float
    status: int


def spherical_kmeans(S: torch.Tensor, k: int, *, max_iters: int = 100, seed: int = 0,
                     return_centroids: bool = False) -> KmeansResult:
    """Spherical k-means on the L2-normalised rows of S (the hard-clustering
    baseline). Returns labels (n int32), optionally the centroids (n x k, column
    j = centroid j), the number of centroid updates, whether the last
    assignment moved no row, and sum_i <x_i, c_label(i)>."""
    n, lds = _S_layout(S)
    lab = torch.empty(n, dtype=torch.int32, device=S.device)
    C = torch.empty((n, k), dtype=torch.float32, device=S.device) if return_centroids else None
    ws = workspace(workspace_bytes(L.OP_KMEANS, n, k), S.device)
    it = ctypes.c_int32(0)
    conv = ctypes.c_int32(0)
    obj = ctypes.c_double(0.0)
    st = L.load().symnmf_spherical_kmeans(_ptr(S), n, lds, k, max_iters, seed, _ptr(lab), _ptr(C),
                                          ctypes.byref(it), ctypes.byref(conv), ctypes.byref(obj),
                                          _ptr(ws), ws.numel(), ctypes.c_void_p(_stream_ptr()))
    L.check(st, "symnmf_spherical_kmeans")
    return KmeansResult(lab, C, it.value, bool(conv.value), obj.value, st)


# ---- sequence operators ------------------------------------------------------
_DTYPES = {torch.float32: L.F32, torch.bfloat16: L.BF16, torch.float16: L.F16}
_INDEX = {torch.int32: L.I32, torch.int64: L.I64}


def _seq_tensor(t, name: str, types=_DTYPES, dtype=None, shape=None, device=None) -> int:
    """Checks a device tensor of a sequence operator and returns its type code."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a HIP device tensor")
    if t.dtype not in types or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype or ' or '.join(str(d) for d in types)}, "
                         f"not {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, not {t.device}")
    return types[t.dtype]


def _here(device):
    """The stream to launch on: torch's current one, of the tensors' device. The
    raw handle (0.1 us) rather than a Stream object made for the call (2.7 us,
    a quarter of a small call)."""
    index = torch._C._cuda_getDevice()
    if device.index != index:
        raise ValueError(f"the tensors are on {device}, which is not the current device")
    return torch._C._cuda_getCurrentRawStream(index)


def _rows_out(n: int, width: int, dtype, device) -> torch.Tensor:
    # a dense n x width output (empty_strided: the cheapest allocation call)
    return torch.empty_strided((n, width), (width, 1), dtype=dtype, device=device)


def _steps_out(batch: int, steps: int, width: int, dtype, device) -> torch.Tensor:
    return torch.empty_strided((batch, steps, width), (steps * width, width, 1), dtype=dtype,
                               device=device)


_no_scratch: dict = {}


@functools.lru_cache(maxsize=4096)
def _scratch_bytes(op: int, n: int, k: int, T: int) -> int:
    # the sizes decide alone, so a loop's calls ask once
    return workspace_bytes(op, n, k, T)


def _scratch(op: int, n: int, k: int, T: int, device) -> torch.Tensor:
    """Workspace of a call. One of the least size is never touched (the query's
    answer for "none"), so all such calls of a device share one."""
    nbytes = _scratch_bytes(op, n, k, T)
    if nbytes > 256:
        return torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=device)
    ws = _no_scratch.get(device)
    if ws is None:
        ws = _no_scratch[device] = workspace(256, device)
    return ws


def _rows_ld(t: torch.Tensor, name: str) -> int:
    """Leading dimension of a 2-D tensor of rows with unit column stride."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.numel() and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if ld < t.shape[1]:
        raise ValueError(f"{name} has overlapping rows")
    return ld


def embed(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
          dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """scale * table[ids] (rows x width table of float32, bfloat16 or float16;
    int32 or int64 ids of any shape), of shape ids.shape + (width,) in ``dtype``
    (default: the table's). A negative id is an empty slot (a row of zeros); an
    id past the table gives a row of NaN."""
    tt = _seq_tensor(table, "table")
    it = _seq_tensor(ids, "ids", _INDEX, device=table.device)
    ld = _rows_ld(table, "table")
    rows, width = table.shape
    if rows < 1 or width < 1:
        raise ValueError("table must not be empty")
    out = torch.empty((*ids.shape, width), dtype=dtype or table.dtype, device=table.device)
    ot = _seq_tensor(out, "out")
    ids = ids.contiguous()
    st = L.load().symnmf_embed(table.data_ptr(), tt, rows, width, ld, ids.data_ptr(), it,
                               ids.numel(), scale, out.data_ptr(), ot, width,
                               _here(table.device))
    L.check(st, "symnmf_embed")
    return out


def embed_grad(dout: torch.Tensor, ids: torch.Tensor, rows: int, scale: float = 1.0,
               dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
               accumulate: bool = False) -> torch.Tensor:
    """Gradient of ``embed`` at its table: scale * the sum of dout's rows by id
    (dout of shape ids.shape + (width,)), a rows x width tensor of ``dtype`` or
    ``out`` itself (accumulate=True adds to what ``out`` holds). dout may be an
    expanded view. Summed in float32 in a fixed order. Ids outside the table
    give nothing."""
    dt = _seq_tensor(dout, "dout")
    it = _seq_tensor(ids, "ids", _INDEX, device=dout.device)
    if dout.dim() < 1 or tuple(dout.shape[:-1]) != tuple(ids.shape):
        raise ValueError("dout must have the shape of ids and one more dimension")
    width = dout.shape[-1]
    if rows < 1 or width < 1:
        raise ValueError("the table must not be empty")
    if accumulate and out is None:
        raise ValueError("accumulate=True needs out")
    if out is None:
        out = _rows_out(rows, width, dtype, dout.device)
    ot = _seq_tensor(out, "out", shape=(rows, width), device=dout.device)
    ldo = _rows_ld(out, "out")
    flat = dout.reshape(-1, width)
    if (width > 1 and flat.stride(1) != 1) or (flat.shape[0] > 1 and flat.stride(0) < width):
        flat = flat.contiguous()  # an expanded dout (a sum's gradient) among them
    ldd = _rows_ld(flat, "dout") if flat.shape[0] else width
    ids = ids.contiguous()
    ws = _scratch(L.OP_EMBED_GRAD, rows, width, ids.numel(), dout.device)
    st = L.load().symnmf_embed_grad(flat.data_ptr(), dt, ids.numel(), width, ldd, ids.data_ptr(), it,
                                    scale, int(accumulate), out.data_ptr(), ot, rows, ldo,
                                    ws.data_ptr(), ws.numel(), _here(dout.device))
    L.check(st, "symnmf_embed_grad")
    return out


def _scan_view(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None):
    """(batch stride, step stride) of a batch x steps x width tensor."""
    if like is None:
        _seq_tensor(t, name)
        if t.dim() != 3:
            raise ValueError(f"{name} must be batch x steps x width")
    else:
        _seq_tensor(t, name, dtype=like.dtype, shape=like.shape, device=like.device)
    if t.numel() == 0:
        return 0, 0
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} needs unit channel stride")
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)


def _state_ptr(t: Optional[torch.Tensor], name: str, shape, device):
    if t is None:
        return None
    _seq_tensor(t, name, dtype=torch.float32, shape=shape, device=device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _lengths_ptr(lengths: Optional[torch.Tensor], batch: int, device):
    if lengths is None:
        return None
    _seq_tensor(lengths, "lengths", {torch.int32: 0}, shape=(batch,), device=device)
    if not lengths.is_contiguous():
        raise ValueError("lengths must be contiguous")
    return lengths.data_ptr()


def gated_scan(x: torch.Tensor, gate: torch.Tensor, h0: Optional[torch.Tensor] = None,
               lengths: Optional[torch.Tensor] = None, return_states: bool = False):
    """h_t = a_t h_{t-1} + (1 - a_t) x_t over the steps of x (batch x steps x
    width), a = sigmoid(gate), from the state ``h0`` (batch x width float32;
    default zeros). ``gate`` has x's shape and type; an expanded view (one decay
    per channel, say) is read as it is. Steps at and past ``lengths[b]`` (int32)
    are masked: h is 0 there and the state passes. Returns (h, the last state in
    float32), and with ``return_states`` the states ``gated_scan_grad`` needs.
    Batches past 65535 rows take a library call for each 65535."""
    x_b, x_t = _scan_view(x, "x")
    g_b, g_t = _scan_view(gate, "gate", x)
    batch, steps, width = x.shape
    h = _steps_out(batch, steps, width, x.dtype, x.device)
    states = None
    if return_states:
        states = _steps_out(batch, -(-steps // L.SCAN_CHUNK), width, torch.float32, x.device)
    last = _scan_call(x, gate, (batch, steps, width), (x_b, x_t, g_b, g_t), lengths, h0, h, states)
    return (h, last, states) if return_states else (h, last)


def _batch_rows(batch: int, *tensors):
    """The batch rows of each tensor (None stays None), as many at a time as a
    library call takes."""
    for lo in range(0, batch, L.MAX_BATCH):
        yield [None if t is None else t[lo:lo + L.MAX_BATCH] for t in tensors]


def _scan_call(x, gate, sizes, strides, lengths, h0, h, states, last=None):
    batch, steps, width = sizes
    x_b, x_t, g_b, g_t = strides
    dev = x.device
    if batch < 1 or width < 1:
        raise ValueError("x must have at least one batch row and one channel")
    lengths_p = _lengths_ptr(lengths, batch, dev)
    h0_p = _state_ptr(h0, "h0", (batch, width), dev)
    if last is None:
        last = _rows_out(batch, width, torch.float32, dev)
    if batch > L.MAX_BATCH:
        for xs, gs, ns, ss, hs, sts, ls in _batch_rows(batch, x, gate, lengths, h0, h, states, last):
            _scan_call(xs, gs, (xs.shape[0], steps, width), strides, ns, ss, hs, sts, ls)
        return last
    ws = _scratch(L.OP_GATED_SCAN, width, batch, steps, dev)
    st = L.load().symnmf_gated_scan(
        _DTYPES[x.dtype], batch, steps, width, x.data_ptr(), x_b, x_t, gate.data_ptr(), g_b, g_t,
        lengths_p, h0_p, h.data_ptr(), last.data_ptr(),
        None if states is None else states.data_ptr(), ws.data_ptr(), ws.numel(), _here(dev))
    L.check(st, "symnmf_gated_scan")
    return last


def gated_step(x: torch.Tensor, gate: torch.Tensor, state: torch.Tensor):
    """One step of ``gated_scan`` for live streams: x and gate batch x width,
    state batch x width float32. Returns (h in x's type, the new state)."""
    _seq_tensor(x, "x")
    _seq_tensor(gate, "gate", dtype=x.dtype, shape=x.shape, device=x.device)
    if x.dim() != 2 or (x.shape[1] > 1 and (x.stride(1) != 1 or gate.stride(1) != 1)):
        raise ValueError("x and gate must be batch x width with unit channel stride")
    batch, width = x.shape
    h = _rows_out(batch, width, x.dtype, x.device)
    strides = (x.stride(0), 0, gate.stride(0), 0) if batch > 1 else (0, 0, 0, 0)
    return h, _scan_call(x, gate, (batch, 1, width), strides, None, state, h, None)


def gated_scan_grad(x: torch.Tensor, gate: torch.Tensor, states: torch.Tensor, dh: torch.Tensor,
                    dh_last: Optional[torch.Tensor] = None,
                    lengths: Optional[torch.Tensor] = None):
    """Gradient of ``gated_scan`` from dh (at h) and ``dh_last`` (at the last
    state), with the forward's ``states``. Returns (dx, dgate, dh0): dx and
    dgate per element in x's type, dh0 batch x width float32. The gradient of
    an expanded gate is dgate's sum over the expanded dimensions."""
    return _scan_grad_call(x, gate, states, dh, dh_last, lengths)


def _scan_grad_call(x, gate, states, dh, dh_last, lengths, dx=None, dgate=None, dh0=None):
    x_b, x_t = _scan_view(x, "x")
    g_b, g_t = _scan_view(gate, "gate", x)
    d_b, d_t = _scan_view(dh, "dh", x)
    batch, steps, width = x.shape
    dev = x.device
    if batch < 1 or width < 1:
        raise ValueError("x must have at least one batch row and one channel")
    lengths_p = _lengths_ptr(lengths, batch, dev)
    states_p = _state_ptr(states, "states", (batch, -(-steps // L.SCAN_CHUNK), width), dev)
    last_p = _state_ptr(dh_last, "dh_last", (batch, width), dev)
    if dx is None:
        dx = _steps_out(batch, steps, width, x.dtype, dev)
        dgate = torch.empty_like(dx)
        dh0 = _rows_out(batch, width, torch.float32, dev)
    if batch > L.MAX_BATCH:
        for part in _batch_rows(batch, x, gate, states, dh, dh_last, lengths, dx, dgate, dh0):
            _scan_grad_call(*part)
        return dx, dgate, dh0
    ws = _scratch(L.OP_GATED_SCAN, width, batch, steps, dev)
    st = L.load().symnmf_gated_scan_grad(
        _DTYPES[x.dtype], batch, steps, width, x.data_ptr(), x_b, x_t, gate.data_ptr(), g_b, g_t,
        lengths_p, states_p, dh.data_ptr(), d_b, d_t, last_p, dx.data_ptr(), dgate.data_ptr(),
        dh0.data_ptr(), ws.data_ptr(), ws.numel(), _here(dev))
    L.check(st, "symnmf_gated_scan_grad")
    return dx, dgate, dh0


@dataclass
class TokenLogprobs:
    logp: torch.Tensor
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logp: Optional[torch.Tensor]
    top_ids: Optional[torch.Tensor]


def _tokens(tokens: torch.Tensor, n: int, device):
    it = _seq_tensor(tokens, "tokens", _INDEX, shape=(n,), device=device)
    return tokens.contiguous(), it


def _row_values(t: Optional[torch.Tensor], name: str, n: int, device):
    if t is None:
        return None
    _seq_tensor(t, name, dtype=torch.float32, shape=(n,), device=device)
    return t.contiguous()


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0,
                   scale: float = 1.0) -> TokenLogprobs:
    """Per row of logits (count x vocab float32, bfloat16 or float16), under
    softmax(scale * logits): the log probability of the row's token, the
    entropy, the log of the normaliser and the ``top`` (at most 32) most likely
    columns with their log probabilities (equal logits: lowest column first).
    All float32, ids int32. Logits of -inf are excluded columns; a negative
    token stands for none (logp 0)."""
    lt = _seq_tensor(logits, "logits")
    ld = _rows_ld(logits, "logits")
    n, vocab = logits.shape
    dev = logits.device
    if vocab < 1 or not 0 <= top <= L.MAX_TOP:
        raise ValueError(f"logits need a column, and top must be 0 to {L.MAX_TOP}")
    if not (scale > 0 and math.isfinite(scale)):
        raise ValueError("scale must be positive and finite")
    tokens, it = _tokens(tokens, n, dev)
    logp = torch.empty_strided((n,), (1,), dtype=torch.float32, device=dev)
    entropy, lse = torch.empty_like(logp), torch.empty_like(logp)
    top_logp = top_ids = None
    if top:
        top_logp = _rows_out(n, top, torch.float32, dev)
        top_ids = _rows_out(n, top, torch.int32, dev)
    ws = _scratch(L.OP_TOKEN_LOGPROBS, vocab, top, n, dev)
    st = L.load().symnmf_token_logprobs(
        logits.data_ptr(), lt, n, vocab, ld, tokens.data_ptr(), it, scale, logp.data_ptr(),
        entropy.data_ptr(), lse.data_ptr(), top, top_logp.data_ptr() if top else None,
        top_ids.data_ptr() if top else None, ws.data_ptr(), ws.numel(), _here(dev))
    L.check(st, "symnmf_token_logprobs")
    return TokenLogprobs(logp, entropy, lse, top_logp, top_ids)


def token_logprobs_grad(logits: torch.Tensor, tokens: torch.Tensor, lse: torch.Tensor,
                        entropy: Optional[torch.Tensor], dlogp: torch.Tensor,
                        dentropy: Optional[torch.Tensor] = None, scale: float = 1.0,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient at the logits from the gradients at ``token_logprobs``'s logp
    and (optionally) entropy, with its lse and entropy. In the logits' type;
    ``out`` may be the logits themselves. Rows far from zero (|lse| > 64) are
    read twice, for the bits that lse's rounding took."""
    lt = _seq_tensor(logits, "logits")
    ld = _rows_ld(logits, "logits")
    n, vocab = logits.shape
    dev = logits.device
    if vocab < 1:
        raise ValueError("logits need a column")
    if not (scale > 0 and math.isfinite(scale)):
        raise ValueError("scale must be positive and finite")
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs the entropy")
    tokens, it = _tokens(tokens, n, dev)
    if lse is None or dlogp is None:
        raise ValueError("lse and dlogp are needed")
    lse = _row_values(lse, "lse", n, dev)
    entropy = _row_values(entropy, "entropy", n, dev)
    dlogp = _row_values(dlogp, "dlogp", n, dev)
    dentropy = _row_values(dentropy, "dentropy", n, dev)
    if out is None:
        out = _rows_out(n, vocab, logits.dtype, dev)
    _seq_tensor(out, "out", dtype=logits.dtype, shape=logits.shape, device=dev)
    ldd = _rows_ld(out, "out")
    if out.data_ptr() == logits.data_ptr() and ldd != ld:
        raise ValueError("out shares the logits' memory in another layout")
    st = L.load().symnmf_token_logprobs_grad(
        logits.data_ptr(), lt, n, vocab, ld, tokens.data_ptr(), it, scale, lse.data_ptr(),
        None if entropy is None else entropy.data_ptr(), dlogp.data_ptr(),
        None if dentropy is None else dentropy.data_ptr(), out.data_ptr(), ldd, _here(dev))
    L.check(st, "symnmf_token_logprobs_grad")
    return out


# ---- kernel timing ---------------------------------------------------------
def profile_enable(on: bool = True):
    L.load().symnmf_profile_enable(1 if on else 0)


def profile_reset():
    L.load().symnmf_profile_reset()


def profile_read(which: int):
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    by = ctypes.c_double(0.0)
    L.check(L.load().symnmf_profile_read(which, ctypes.byref(n), ctypes.byref(ms), ctypes.byref(by)),
            "symnmf_profile_read")
    return {"launches": int(n.value), "ms": ms.value, "bytes": by.value}
