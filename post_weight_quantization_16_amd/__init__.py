"""GPTQ layer quantization on MI355X (gfx950): Python binding.

Thin wrapper over the C ABI of ``libgptq_mi355x.so`` (include/gptq.h).
Every step of the path runs in the library's HIP kernels; this module only
checks tensor placement, passes device pointers and the current HIP stream,
and allocates outputs/workspaces with torch (PyTorch is used for device
memory and streams only).

    H = torch.zeros(d, d, device="cuda")
    hessian_accumulate(H, X)                      # H += 2 XᵀX, X token-major
    prep = prepare_hinv(H, params)                # U, perm, dead
    out = quantize_layer(W, prep, params)         # qweight, scales, zeros, ...

8-bit floating point (block-scaled e4m3 matrices, Fp8Matrix): fp8_quantize,
rmsnorm_fp8, fp8_gemm, fp8_linear (bias, activation, residual), fp8_gated_gemm;
and for blocks of experts (Fp8Experts, Routing): moe_route, moe_plan,
fp8_quantize_experts, fp8_expert_gated_gemm, fp8_expert_gemm.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools

from . import _native

__all__ = [
    "GPTQParams", "GPTQError", "NotPositiveDefinite", "hessian_accumulate",
    "hessian_accumulate_noalloc", "prepare_hinv",
    "quantize_layer", "quantize", "workspace_bytes", "version", "Prepared", "Quantized",
    "Exported", "export", "quantize_layers", "obq_layer", "timing", "timing_read", "w4a16_gemm",
    "Fp8Matrix", "Normed", "fp8_quantize", "rmsnorm_fp8", "fp8_gemm", "fp8_gated_gemm",
    "fp8_linear", "Fp8Experts", "Routing", "moe_route", "moe_plan", "fp8_quantize_experts",
    "fp8_expert_gated_gemm", "fp8_expert_gemm", "expert_workspace_bytes",
]


class GPTQError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class NotPositiveDefinite(GPTQError):
    def __init__(self, code, msg, pivot):
        super().__init__(code, msg)
        self.pivot = pivot


@dataclasses.dataclass(frozen=True)
class GPTQParams:
    bits: int = 4
    group_size: int = 128
    block_size: int = 128
    percdamp: float = 0.01
    act_order: bool = False
    sym: bool = False

    def c(self) -> _native.Params:
        return _native.Params(self.bits, self.group_size, self.block_size, self.percdamp,
                              int(self.act_order), int(self.sym))

    def n_groups(self, d_in: int) -> int:
        g = d_in if self.group_size <= 0 or self.group_size >= d_in else self.group_size
        return (d_in + g - 1) // g


@dataclasses.dataclass
class Prepared:
    U: "object"        # [d, d] fp32 upper factor of H_d⁻¹ (quantization order)
    perm: "object"     # [d] int32 quantization order
    dead: "object"     # [d] uint8 dead-channel mask (original order)
    natural: bool = False   # perm is the identity (prepared without act-order)
    status: "object" = None   # prepare_hinv(sync=False): pinned host status words
    event: "object" = None    # ... and the event recorded after their copy

    def check(self) -> "Prepared":
        """For prepare_hinv(sync=False): wait for the status words and raise
        as prepare_hinv would have; a no-op for a synchronous preparation."""
        if self.status is None:
            return self
        self.event.synchronize()
        info = ctypes.c_int64(-1)
        rc = _native.lib().gptq_prepare_status(ctypes.c_void_p(self.status.data_ptr()),
                                               self.U.shape[0], ctypes.byref(info))
        if rc == _native.ERR_NOT_SPD:
            raise NotPositiveDefinite(rc, _native.last_error(), info.value)
        _check(rc)
        self.status = self.event = None
        return self


@dataclasses.dataclass
class Quantized:
    qweight: "object"  # [d_out, ceil(d_in/8)] int32 (bits <= 4) or [d_out, ceil(d_in/4)] (8-bit)
    scales: "object"   # [d_out, n_groups] fp32, groups in quantization order
    zeros: "object"    # [d_out, n_groups] uint8
    W_hat: "object"    # [d_out, d_in] fp32, original column order (or None)
    g_idx: "object"    # [d_in] int32
    row_loss: "object"  # [d_out] fp32, ½Σerr² per row


def _check(rc: int):
    if rc != _native.OK:
        raise GPTQError(rc, _native.last_error())


def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    m = {torch.float32: _native.F32, torch.bfloat16: _native.BF16, torch.float16: _native.F16}
    if t.dtype not in m:
        raise ValueError(f"unsupported dtype {t.dtype} (float32, bfloat16 or float16)")
    return m[t.dtype]


def _require(t, name, dtype, shape, device=None):
    """Dense tensor of the given dtype and shape (on `device` when given):
    the library reads and writes it as a plain row-major buffer."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _matrix_rows(t, name):
    """2-D with unit column stride (rows may be padded: the row stride is passed)."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must be 2-D with unit column stride")


def _dev(t, name):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return ctypes.c_void_p(t.data_ptr())


def _ws_check(ws, device):
    torch = _torch()
    if ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("a workspace must be a contiguous uint8 tensor")
    if ws.device != device:
        raise ValueError(f"workspace is on {ws.device}, expected {device}")


def _stream(device):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _workspace(nbytes: int, device):
    torch = _torch()
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def version() -> str:
    return _native.lib().gptq_version().decode()


def workspace_bytes(which: int, d_out: int, d_in: int, n_tok: int = 0,
                    params: GPTQParams | None = None) -> int:
    p = (params or GPTQParams()).c()
    return int(_native.lib().gptq_workspace_bytes(which, d_out, d_in, n_tok, ctypes.byref(p)))


def hessian_accumulate(H, X, ws=None):
    """H += 2·XᵀX (X token-major [n_tok, d_in]; row stride X.stride(0))."""
    torch = _torch()
    _matrix_rows(X, "X")
    n_tok, d = X.shape
    xdt = _dtype_code(X)
    _require(H, "H", torch.float32, (d, d), X.device)
    L = _native.lib()
    if ws is None:
        ws = _workspace(L.gptq_workspace_bytes(_native.WS_HESSIAN, 0, d, n_tok, None), X.device)
    _ws_check(ws, X.device)
    _check(L.gptq_hessian_accumulate(_dev(H, "H"), d, _dev(X, "X"), xdt, n_tok,
                                     X.stride(0), _dev(ws, "ws"), ws.numel(), _stream(X.device)))
    return H


def hessian(H, X, ws=None):
    """H = 2·XᵀX (X token-major [n_tok, d_in]): hessian_accumulate on a zeroed
    H in one call, without reading H."""
    torch = _torch()
    _matrix_rows(X, "X")
    n_tok, d = X.shape
    xdt = _dtype_code(X)
    _require(H, "H", torch.float32, (d, d), X.device)
    L = _native.lib()
    if ws is None:
        ws = _workspace(L.gptq_workspace_bytes(_native.WS_HESSIAN, 0, d, n_tok, None), X.device)
    _ws_check(ws, X.device)
    _check(L.gptq_hessian(_dev(H, "H"), d, _dev(X, "X"), xdt, n_tok, X.stride(0), _dev(ws, "ws"),
                          ws.numel(), _stream(X.device)))
    return H


def hessian_accumulate_noalloc(H, X):
    """H += 2·XᵀX without a workspace: the library's static device scratch
    (for callers that cannot allocate; d_in <= 4096; calls that overlap on
    one GPU race)."""
    torch = _torch()
    _matrix_rows(X, "X")
    n_tok, d = X.shape
    xdt = _dtype_code(X)
    _require(H, "H", torch.float32, (d, d), X.device)
    _check(_native.lib().gptq_hessian_accumulate_noalloc(_dev(H, "H"), d, _dev(X, "X"), xdt, n_tok,
                                                         X.stride(0), _stream(X.device)))
    return H


def prepare_hinv(H, params: GPTQParams, ws=None, sync: bool = True) -> Prepared:
    """Dead fix, damping, act-order and U (H is overwritten with H_d).

    sync=False returns at once (gptq_prepare_hinv_async): the work, and the
    quantization queued behind it, run while the host goes on; call
    ``Prepared.check()`` later for the factorization's outcome."""
    torch = _torch()
    if H.dim() != 2:
        raise ValueError("H must be a square matrix")
    d = H.shape[0]
    _require(H, "H", torch.float32, (d, d))
    L = _native.lib()
    p = params.c()
    dev = H.device
    U = torch.empty(d, d, dtype=torch.float32, device=dev)
    perm = torch.empty(d, dtype=torch.int32, device=dev)
    dead = torch.empty(d, dtype=torch.uint8, device=dev)
    if ws is None:
        ws = _workspace(L.gptq_workspace_bytes(_native.WS_PREPARE, 0, d, 0, ctypes.byref(p)), dev)
    _ws_check(ws, dev)
    if not sync:
        status = torch.empty(2, dtype=torch.int32, pin_memory=True)
        _check(L.gptq_prepare_hinv_async(_dev(H, "H"), d, ctypes.byref(p), _dev(U, "U"),
                                         _dev(perm, "perm"), _dev(dead, "dead"), _dev(ws, "ws"),
                                         ws.numel(), ctypes.c_void_p(status.data_ptr()),
                                         _stream(dev)))
        ev = torch.cuda.Event()
        ev.record(torch.cuda.current_stream(dev))
        return Prepared(U, perm, dead, natural=not params.act_order, status=status, event=ev)
    info = ctypes.c_int64(-1)
    rc = L.gptq_prepare_hinv(_dev(H, "H"), d, ctypes.byref(p), _dev(U, "U"), _dev(perm, "perm"),
                             _dev(dead, "dead"), _dev(ws, "ws"), ws.numel(), ctypes.byref(info),
                             _stream(dev))
    if rc == _native.ERR_NOT_SPD:
        raise NotPositiveDefinite(rc, _native.last_error(), info.value)
    _check(rc)
    return Prepared(U, perm, dead, natural=not params.act_order)


def quantize_layer(W, prep: Prepared, params: GPTQParams, want_what: bool = True,
                   ws=None) -> Quantized:
    """Run the sweep on W [d_out, d_in] with the factor from prepare_hinv."""
    torch = _torch()
    _matrix_rows(W, "W")
    m, d = W.shape
    wdt = _dtype_code(W)
    dev = W.device
    _require(prep.U, "U", torch.float32, (d, d), dev)
    if params.act_order and prep.natural:
        raise ValueError("act_order needs a Prepared from prepare_hinv with act_order")
    if not prep.natural:
        _require(prep.perm, "perm", torch.int32, (d,), dev)
    if prep.dead is not None:
        _require(prep.dead, "dead", torch.uint8, (d,), dev)
    L = _native.lib()
    p = params.c()
    cpw = 8 if params.bits <= 4 else 4
    ng = params.n_groups(d)
    qweight = torch.empty(m, (d + cpw - 1) // cpw, dtype=torch.int32, device=dev)
    scales = torch.empty(m, ng, dtype=torch.float32, device=dev)
    zeros = torch.empty(m, ng, dtype=torch.uint8, device=dev)
    W_hat = torch.empty(m, d, dtype=torch.float32, device=dev) if want_what else None
    g_idx = torch.empty(d, dtype=torch.int32, device=dev)
    row_loss = torch.empty(m, dtype=torch.float32, device=dev)
    if ws is None:
        ws = _workspace(L.gptq_workspace_bytes(_native.WS_QUANTIZE, m, d, 0, ctypes.byref(p)), dev)
    _ws_check(ws, dev)
    _check(L.gptq_quantize_layer(
        _dev(W, "W"), wdt, m, d, W.stride(0), _dev(prep.U, "U"),
        None if prep.natural else _dev(prep.perm, "perm"),
        _dev(prep.dead, "dead"), ctypes.byref(p), _dev(qweight, "qweight"), _dev(scales, "scales"),
        _dev(zeros, "zeros"), _dev(W_hat, "W_hat"), _dev(g_idx, "g_idx"), _dev(row_loss, "row_loss"),
        _dev(ws, "ws"), ws.numel(), _stream(dev)))
    return Quantized(qweight, scales, zeros, W_hat, g_idx, row_loss)


def quantize_layers(Ws, prep: Prepared, params: GPTQParams, want_what: bool = True,
                    ws=None) -> list:
    """Several layers with the same inputs (one H, one factor): one Quantized
    per W, bitwise what quantize_layer gives for each alone."""
    torch = _torch()
    if not Ws:
        raise ValueError("no layers")
    d = Ws[0].shape[1]
    dev = Ws[0].device
    _require(prep.U, "U", torch.float32, (d, d), dev)
    if params.act_order and prep.natural:
        raise ValueError("act_order needs a Prepared from prepare_hinv with act_order")
    if not prep.natural:
        _require(prep.perm, "perm", torch.int32, (d,), dev)
    if prep.dead is not None:
        _require(prep.dead, "dead", torch.uint8, (d,), dev)
    p = params.c()
    cpw = 8 if params.bits <= 4 else 4
    ng = params.n_groups(d)
    outs, descs = [], (_native.Layer * len(Ws))()
    for i, W in enumerate(Ws):
        _matrix_rows(W, f"W[{i}]")
        if W.shape[1] != d or W.device != dev:
            raise ValueError(f"W[{i}] must have {d} columns and live on {dev}")
        m = W.shape[0]
        o = Quantized(torch.empty(m, (d + cpw - 1) // cpw, dtype=torch.int32, device=dev),
                      torch.empty(m, ng, dtype=torch.float32, device=dev),
                      torch.empty(m, ng, dtype=torch.uint8, device=dev),
                      torch.empty(m, d, dtype=torch.float32, device=dev) if want_what else None,
                      None, torch.empty(m, dtype=torch.float32, device=dev))
        outs.append(o)
        descs[i] = _native.Layer(_dev(W, "W"), _dtype_code(W), 0, m, W.stride(0),
                                 _dev(o.qweight, "qweight"), _dev(o.scales, "scales"),
                                 _dev(o.zeros, "zeros"), _dev(o.W_hat, "W_hat"),
                                 _dev(o.row_loss, "row_loss"))
    g_idx = torch.empty(d, dtype=torch.int32, device=dev)
    L = _native.lib()
    total = sum(W.shape[0] for W in Ws)
    if ws is None:
        ws = _workspace(L.gptq_workspace_bytes(_native.WS_QUANTIZE, total, d, 0, ctypes.byref(p)), dev)
    _ws_check(ws, dev)
    _check(L.gptq_quantize_layers(len(Ws), descs, d, _dev(prep.U, "U"),
                                  None if prep.natural else _dev(prep.perm, "perm"),
                                  _dev(prep.dead, "dead"), ctypes.byref(p), _dev(g_idx, "g_idx"),
                                  _dev(ws, "ws"), ws.numel(), _stream(dev)))
    for o in outs:
        o.g_idx = g_idx
    return outs


def quantize_independent(layers, params: GPTQParams, want_what: bool = True, ws=None) -> list:
    """Independent layers, each with its own inputs: ``layers`` is a list of
    (W, X) device tensors (W [d_out, d_in], X [n_tok, d_in] token-major).
    Every layer gets a fresh H = 2·XᵀX, its own factor and its quantization;
    the library runs the layers concurrently and synchronizes once.  Returns
    one (Quantized, Prepared, H_d) per layer, bitwise what hessian_accumulate,
    prepare_hinv and quantize_layer give for that layer alone.  ``ws``: None,
    or one workspace per layer (GPTQ_WS_LAYER bytes each).  Raises like
    prepare_hinv when a layer's factorization fails (the first such layer);
    the exception's ``statuses`` and ``results`` give every layer's status
    and outputs (valid for the layers that succeeded)."""
    torch = _torch()
    if not layers:
        raise ValueError("no layers")
    if ws is not None and len(ws) != len(layers):
        raise ValueError("ws must hold one workspace per layer")
    L = _native.lib()
    p = params.c()
    cpw = 8 if params.bits <= 4 else 4
    jobs = (_native.LayerJob * len(layers))()
    out, keep = [], []
    dev0 = layers[0][0].device
    for i, (W, X) in enumerate(layers):
        _matrix_rows(W, f"W[{i}]")
        _matrix_rows(X, f"X[{i}]")
        m, d = W.shape
        n_tok = X.shape[0]
        dev = W.device
        if dev != dev0:
            raise ValueError(f"W[{i}] is on {dev}; every layer must live on {dev0}")
        if X.shape[1] != d or X.device != dev:
            raise ValueError(f"X[{i}] must have {d} columns and live on {dev}")
        ng = params.n_groups(d)
        H = torch.zeros(d, d, dtype=torch.float32, device=dev)
        prep = Prepared(torch.empty(d, d, dtype=torch.float32, device=dev),
                        torch.empty(d, dtype=torch.int32, device=dev),
                        torch.empty(d, dtype=torch.uint8, device=dev),
                        natural=not params.act_order)
        q = Quantized(torch.empty(m, (d + cpw - 1) // cpw, dtype=torch.int32, device=dev),
                      torch.empty(m, ng, dtype=torch.float32, device=dev),
                      torch.empty(m, ng, dtype=torch.uint8, device=dev),
                      torch.empty(m, d, dtype=torch.float32, device=dev) if want_what else None,
                      torch.empty(d, dtype=torch.int32, device=dev),
                      torch.empty(m, dtype=torch.float32, device=dev))
        w = ws[i] if ws is not None else _workspace(
            L.gptq_workspace_bytes(_native.WS_LAYER, m, d, n_tok, ctypes.byref(p)), dev)
        _ws_check(w, dev)
        keep.append(w)
        jobs[i] = _native.LayerJob(
            _dev(X, "X"), _dtype_code(X), _dtype_code(W), n_tok, X.stride(0), _dev(W, "W"), m, d,
            W.stride(0), _dev(H, "H"), _dev(prep.U, "U"), _dev(prep.perm, "perm"),
            _dev(prep.dead, "dead"), _dev(q.qweight, "qweight"), _dev(q.scales, "scales"),
            _dev(q.zeros, "zeros"), _dev(q.W_hat, "W_hat"), _dev(q.g_idx, "g_idx"),
            _dev(q.row_loss, "row_loss"), _dev(w, "ws"), w.numel(), 0, 0, -1)
        out.append((q, prep, H))
    with _torch().cuda.device(dev0):   # the library runs the jobs on the current device
        rc = L.gptq_quantize_independent(len(layers), jobs, ctypes.byref(p), _stream(dev0))
    if rc != _native.OK:
        if rc == _native.ERR_NOT_SPD:
            bad = next(j for j in jobs if j.status == _native.ERR_NOT_SPD)
            err = NotPositiveDefinite(rc, _native.last_error(), bad.info)
        else:
            err = GPTQError(rc, _native.last_error())
        # per-layer statuses and results: the layers that succeeded are valid
        err.statuses = [j.status for j in jobs]
        err.results = out
        raise err
    return out


def obq_layer(W, H, params: GPTQParams, ws=None):
    """OBQ (greedy order per row) of a tiny layer against the fp32 Hessian H.

    Returns (Quantized, order [d_out, d_in] int32).  params.group_size must
    be -1 (one grid per row) and act_order False; d_in <= 128.
    """
    torch = _torch()
    _matrix_rows(W, "W")
    m, d = W.shape
    wdt = _dtype_code(W)
    dev = W.device
    _require(H, "H", torch.float32, (d, d), dev)
    p = params.c()
    cpw = 8 if params.bits <= 4 else 4
    qweight = torch.empty(m, (d + cpw - 1) // cpw, dtype=torch.int32, device=dev)
    scales = torch.empty(m, 1, dtype=torch.float32, device=dev)
    zeros = torch.empty(m, 1, dtype=torch.uint8, device=dev)
    W_hat = torch.empty(m, d, dtype=torch.float32, device=dev)
    order = torch.empty(m, d, dtype=torch.int32, device=dev)
    row_loss = torch.empty(m, dtype=torch.float32, device=dev)
    L = _native.lib()
    if ws is None:
        ws = _workspace(L.gptq_workspace_bytes(_native.WS_OBQ, m, d, 0, ctypes.byref(p)), dev)
    _ws_check(ws, dev)
    rc = L.gptq_obq_layer(_dev(W, "W"), wdt, m, d, W.stride(0), _dev(H, "H"), ctypes.byref(p),
                          _dev(qweight, "qweight"), _dev(scales, "scales"), _dev(zeros, "zeros"),
                          _dev(W_hat, "W_hat"), _dev(order, "order"), _dev(row_loss, "row_loss"),
                          _dev(ws, "ws"), ws.numel(), _stream(dev))
    if rc == _native.ERR_NOT_SPD:
        raise NotPositiveDefinite(rc, _native.last_error(), -1)
    _check(rc)
    return Quantized(qweight, scales, zeros, W_hat, None, row_loss), order


TIMED_STAGES = ("block_update", "sweep", "cholesky", "inverse", "hessian", "lead_panel")


def timing(enable: bool) -> None:
    """Start (clearing earlier records) or stop per-stage event timing."""
    _native.lib().gptq_timing(1 if enable else 0)


def timing_read() -> dict:
    """Milliseconds per timed stage since timing was enabled (or last read)."""
    buf = (ctypes.c_float * len(TIMED_STAGES))()
    _check(_native.lib().gptq_timing_read(buf, len(TIMED_STAGES)))
    return {k: float(v) for k, v in zip(TIMED_STAGES, buf)}


@dataclasses.dataclass
class Exported:
    qweight: "object"     # [d_out, ceil(d_in·bits/32)] int32, dense little-endian bit stream per row
    scales_f16: "object"  # [d_out, n_groups] float16
    zeros_f16: "object"   # [d_out, n_groups] float16


def export(q: Quantized, params: GPTQParams, d_in: int) -> Exported:
    """Dense b-bit codes and 16-bit scales/zeros from a quantize_layer result."""
    torch = _torch()
    m = q.scales.shape[0]
    ng = q.scales.shape[1]
    dev = q.scales.device
    cpw = 8 if params.bits <= 4 else 4
    _require(q.qweight, "qweight", torch.int32, (m, (d_in + cpw - 1) // cpw), dev)
    _require(q.scales, "scales", torch.float32, (m, ng), dev)
    _require(q.zeros, "zeros", torch.uint8, (m, ng), dev)
    qd = torch.empty(m, (d_in * params.bits + 31) // 32, dtype=torch.int32, device=dev)
    s16 = torch.empty(m, ng, dtype=torch.float16, device=dev)
    z16 = torch.empty(m, ng, dtype=torch.float16, device=dev)
    _check(_native.lib().gptq_export(params.bits, m, d_in, ng, _dev(q.qweight, "qweight"),
                                     _dev(q.scales, "scales"), _dev(q.zeros, "zeros"),
                                     _dev(qd, "qweight_dense"), _dev(s16, "scales_f16"),
                                     _dev(z16, "zeros_f16"), _stream(dev)))
    return Exported(qd, s16, z16)


def w4a16_gemm(A, ex: Exported, bits: int, group_size: int, g_idx=None, out=None, ws=None):
    """C = A·Ŵᵀ from an export: A [M, K] float16/bfloat16, C [M, N] float32.
    ws: the split-K workspace (allocated here when None; pass one to reuse)."""
    torch = _torch()
    _matrix_rows(A, "A")
    M, K = A.shape
    dev = A.device
    if A.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("A must be float16 or bfloat16")
    N, ng = ex.scales_f16.shape
    _require(ex.qweight, "qweight", torch.int32, (N, (K * bits + 31) // 32), dev)
    _require(ex.scales_f16, "scales_f16", torch.float16, (N, ng), dev)
    _require(ex.zeros_f16, "zeros_f16", torch.float16, (N, ng), dev)
    if g_idx is not None:
        _require(g_idx, "g_idx", torch.int32, (K,), dev)
    C = out if out is not None else torch.empty(M, N, dtype=torch.float32, device=dev)
    _require(C, "C", torch.float32, (M, N), dev)
    L = _native.lib()
    if ws is None:
        ws = _workspace(L.gptq_workspace_bytes(_native.WS_W4A16, N, K, M, None), dev)
    _ws_check(ws, dev)
    _check(L.gptq_w4a16_gemm(
        _dev(A, "A"), _dtype_code(A), M, K, A.stride(0), _dev(ex.qweight, "qweight"), bits,
        _dev(ex.scales_f16, "scales_f16"), _dev(ex.zeros_f16, "zeros_f16"),
        _dev(g_idx, "g_idx"), group_size, ng, N, _dev(C, "C"), N, _dev(ws, "ws"), ws.numel(),
        _stream(dev)))
    return C


# ---------------------------------------------------------------- 8-bit floating point
FP8_BLOCK = 128


@dataclasses.dataclass(slots=True)
class Fp8Matrix:
    """A block-scaled matrix: value = code·scale."""
    codes: "object"      # [rows, cols] float8_e4m3fn, unit column stride
    scales: "object"     # [ceil(rows/block_rows), ceil(cols/128)] float32
    block_rows: int = 1  # 1 (activations) or 128 (weights)


@dataclasses.dataclass(slots=True)
class Normed:
    q: "object"          # Fp8Matrix of y, or None
    h: "object"          # [rows, cols] x + residual in x's type (x itself without a residual)
    y: "object"          # [rows, cols] y in x's type, or None


_T = None   # what the 8-bit calls need of torch, looked up once


def _t8():
    global _T
    if _T is None:
        torch = _torch()
        if torch.cuda.is_available():
            torch.cuda.init()   # the two look-ups below take it for granted
        _T = (torch.empty, torch.float8_e4m3fn, torch.float32, torch._C._cuda_getDevice,
              torch._C._cuda_getCurrentRawStream,
              {torch.float32: _native.F32, torch.bfloat16: _native.BF16, torch.float16: _native.F16})
    return _T


def _fp8_new(rows: int, cols: int, block_rows: int, device) -> tuple:
    """(Fp8Matrix, row stride) to be filled.  Its rows start at multiples of
    16 bytes (what the products' wide copies need); the bytes behind a row's
    end are not written."""
    empty, e4m3, f32 = _t8()[:3]
    ld = (cols + 15) // 16 * 16
    c = empty((rows, ld), dtype=e4m3, device=device)
    s = empty(((rows + block_rows - 1) // block_rows, (cols + FP8_BLOCK - 1) // FP8_BLOCK), dtype=f32,
              device=device)
    return Fp8Matrix(c if ld == cols else c[:, :cols], s, block_rows), ld


def _fp8_arg(m: Fp8Matrix, name, block_rows, device=None):
    """(rows, cols, row stride, device) of a block-scaled argument after its checks."""
    if m.block_rows != block_rows:
        raise ValueError(f"{name} must have block_rows {block_rows} (got {m.block_rows})")
    c, s = m.codes, m.scales
    _, e4m3, f32, _, _, _ = _t8()
    if c.dtype != e4m3:
        raise ValueError(f"{name}.codes must be float8_e4m3fn (got {c.dtype})")
    ld = _fp8_rows(c, name)
    rows, cols = c.shape
    dev = c.device
    want = ((rows + block_rows - 1) // block_rows, (cols + FP8_BLOCK - 1) // FP8_BLOCK)
    if s.dtype != f32 or s.shape != want or not s.is_contiguous():
        raise ValueError(f"{name}.scales must be contiguous float32 of shape {want} "
                         f"(got {s.dtype}, {tuple(s.shape)})")
    if s.device != dev or (device is not None and dev != device):
        raise ValueError(f"{name} is on {dev} (scales on {s.device}), expected {device or dev}")
    return rows, cols, ld, dev


def _fp8_rows(t, name) -> int:
    """Row stride of a 2-D tensor with unit column stride (a single row's own
    stride says nothing: its length is taken)."""
    st = t.stride()
    if len(st) == 2:
        rows, cols = t.shape
        if st[1] == 1 or cols <= 1:
            if rows <= 1:
                return cols
            if st[0] >= cols:
                return st[0]
    raise ValueError(f"{name} must be 2-D with unit column stride")


def _fp8_dtype(t, name) -> int:
    code = _t8()[5].get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: unsupported dtype {t.dtype} (float32, bfloat16 or float16)")
    return code


def _fp8_out(t, name, dtype, shape, device) -> int:
    if t.dtype != dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be {dtype} of shape {shape} on {device}")
    return _fp8_rows(t, name)


def _launch(device, fn, *args):
    """Call an entry point with the device current and its stream last."""
    if device.type != "cuda":
        raise ValueError("the tensors must be device tensors")
    i = device.index
    _, _, _, current, raw_stream, _ = _t8()
    if current() == i:
        rc = fn(*args, raw_stream(i))
    else:
        with _torch().cuda.device(i):
            rc = fn(*args, raw_stream(i))
    if rc != _native.OK:
        _check(rc)


def fp8_quantize(X, block_rows: int = 1, out: Fp8Matrix | None = None) -> Fp8Matrix:
    """X [rows, cols] (float32/bfloat16/float16) in e4m3 with one scale per
    block of block_rows x 128: 1 for activations, 128 for weights."""
    xdt = _fp8_dtype(X, "X")
    ld_x = _fp8_rows(X, "X")
    rows, cols = X.shape
    dev = X.device
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError(f"block_rows must be 1 or {FP8_BLOCK} (got {block_rows})")
    if out is None:
        out, ld_c = _fp8_new(rows, cols, block_rows, dev)
    else:
        r, c, ld_c, _ = _fp8_arg(out, "out", block_rows, dev)
        if (r, c) != (rows, cols):
            raise ValueError(f"out must have shape {(rows, cols)} (got {(r, c)})")
    _launch(dev, _native.lib().gptq_fp8_quantize, X.data_ptr(), xdt, rows, cols, ld_x, block_rows,
            out.codes.data_ptr(), ld_c, out.scales.data_ptr())
    return out


def rmsnorm_fp8(X, gamma, eps: float = 1e-6, residual=None, want_q: bool = True,
                want_y: bool = False, h_out=None) -> Normed:
    """h = X + residual (rounded to X's type), y = h·gamma/sqrt(mean(h²) + eps)
    per row, quantized in 1 x 128 blocks (want_q) and/or rounded to X's type
    (want_y).  h_out: where h goes (X or residual itself for an update in
    place); without a residual h is X and nothing is written."""
    empty, _, f32 = _t8()[:3]
    xdt = _fp8_dtype(X, "X")
    ld_x = _fp8_rows(X, "X")
    rows, cols = X.shape
    dev = X.device
    dt = X.dtype
    if gamma.dtype != dt and gamma.dtype != f32:
        raise ValueError(f"gamma must be {dt} or float32 (got {gamma.dtype})")
    if gamma.shape != (cols,) or not gamma.is_contiguous() or gamma.device != dev:
        raise ValueError(f"gamma must be contiguous of shape {(cols,)} on {dev}")
    if not (want_q or want_y):
        raise ValueError("want_q or want_y must be set")
    h, ld_r, ld_h, hp = X, 0, 0, None
    if residual is not None:
        ld_r = _fp8_out(residual, "residual", dt, (rows, cols), dev)
        if h_out is None:
            h, ld_h = empty((rows, cols), dtype=dt, device=dev), cols
        else:
            h, ld_h = h_out, _fp8_out(h_out, "h_out", dt, (rows, cols), dev)
        hp = h.data_ptr()
    elif h_out is not None:
        raise ValueError("h_out needs a residual")
    y = empty((rows, cols), dtype=dt, device=dev) if want_y else None
    q, qc, qs, ld_c = None, None, None, 0
    if want_q:
        q, ld_c = _fp8_new(rows, cols, 1, dev)
        qc, qs = q.codes.data_ptr(), q.scales.data_ptr()
    _launch(dev, _native.lib().gptq_rmsnorm_fp8, X.data_ptr(), ld_x,
            None if residual is None else residual.data_ptr(), ld_r, xdt, gamma.data_ptr(),
            xdt if gamma.dtype == dt else _native.F32, rows, cols, eps, hp, ld_h,
            y.data_ptr() if want_y else None, cols, qc, ld_c, qs)
    return Normed(q, h, y)


@functools.lru_cache(maxsize=4096)
def _fp8_bytes(which, M, N, K):
    return _native.lib().gptq_workspace_bytes(which, N, K, M, None)


def _fp8_workspace(which, M, N, K, ws, dev):
    """(address, bytes, tensor to keep) of the split-K workspace; sizes that
    need none (the library says 256) get none."""
    if ws is None:
        need = _fp8_bytes(which, M, N, K)
        if need <= 256:
            return None, 0, None
        ws = _workspace(need, dev)
    else:
        _ws_check(ws, dev)
    return ws.data_ptr(), ws.numel(), ws


def fp8_gemm(A: Fp8Matrix, B: Fp8Matrix, out_dtype=None, out=None, ws=None):
    """C = A·Bᵀ: A [M, K] with block_rows 1, B [N, K] with block_rows 128,
    C [M, N] in out_dtype (bfloat16 unless given, or `out`'s type).  float32
    has exact products and fp32 sums; the 16-bit types take the fp8 matrix
    instruction, twice as fast, whose sums are off by 1.5e-5 to 6e-5 of the
    result's norm (values whose sum cancels: by more than their own rounding).
    ws: the split-K workspace (allocated here when None; pass one to reuse)."""
    M, K, lda, dev = _fp8_arg(A, "A", 1)
    N, kb, ldb, _ = _fp8_arg(B, "B", FP8_BLOCK, dev)
    if kb != K:
        raise ValueError(f"A has {K} columns, B has {kb}")
    if out is None:
        out = _t8()[0]((M, N), dtype=out_dtype or _torch().bfloat16, device=dev)
        ldc = N
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out must be {out_dtype} (got {out.dtype})")
        ldc = _fp8_out(out, "out", out.dtype, (M, N), dev)
    cdt = _fp8_dtype(out, "out")
    wp, wn, ws = _fp8_workspace(_native.WS_FP8_GEMM, M, N, K, ws, dev)
    _launch(dev, _native.lib().gptq_fp8_gemm, A.codes.data_ptr(), A.scales.data_ptr(), M, K, lda,
            B.codes.data_ptr(), B.scales.data_ptr(), N, ldb, out.data_ptr(), cdt, ldc, wp, wn)
    return out


_ACTIVATIONS = {"silu": _native.ACT_SILU, "gelu": _native.ACT_GELU,
                "gelu_tanh": _native.ACT_GELU_TANH}


def fp8_gated_gemm(A: Fp8Matrix, gate: Fp8Matrix, up: Fp8Matrix, activation: str = "silu",
                   out_dtype=None, out=None, ws=None):
    """act(A·gateᵀ)·(A·upᵀ): A [M, K] with block_rows 1, gate and up [N, K]
    with block_rows 128.  Returns an Fp8Matrix [M, N] with block_rows 1, or a
    tensor of out_dtype where that is given; `out` is either, to be filled.
    ws: the split-K workspace (allocated here when None; pass one to reuse)."""
    M, K, lda, dev = _fp8_arg(A, "A", 1)
    N, kg, ldg, _ = _fp8_arg(gate, "gate", FP8_BLOCK, dev)
    nu, ku, ldu, _ = _fp8_arg(up, "up", FP8_BLOCK, dev)
    if kg != K or ku != K or nu != N:
        raise ValueError(f"A has {K} columns; gate {(N, kg)} and up {(nu, ku)} do not fit")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)} (got {activation!r})")
    cp, cdt, ldc, qc, ldq, qs = None, 0, 0, None, 0, None
    if out is None and out_dtype is None:
        out, ldq = _fp8_new(M, N, 1, dev)
        qc, qs = out.codes.data_ptr(), out.scales.data_ptr()
    elif isinstance(out, Fp8Matrix):
        if out_dtype is not None:
            raise ValueError("an Fp8Matrix out has no out_dtype")
        mo, no, ldq, _ = _fp8_arg(out, "out", 1, dev)
        if (mo, no) != (M, N):
            raise ValueError(f"out must have shape {(M, N)} (got {(mo, no)})")
        qc, qs = out.codes.data_ptr(), out.scales.data_ptr()
    else:
        if out is None:
            out = _t8()[0]((M, N), dtype=out_dtype, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out must be {out_dtype} (got {out.dtype})")
        cdt = _fp8_dtype(out, "out")
        ldc = _fp8_out(out, "out", out.dtype, (M, N), dev)
        cp = out.data_ptr()
    wp, wn, ws = _fp8_workspace(_native.WS_FP8_GATED, M, N, K, ws, dev)
    _launch(dev, _native.lib().gptq_fp8_gated_gemm, A.codes.data_ptr(), A.scales.data_ptr(), M, K,
            lda, gate.codes.data_ptr(), gate.scales.data_ptr(), ldg, up.codes.data_ptr(),
            up.scales.data_ptr(), ldu, N, act, cp, cdt, ldc, qc, ldq, qs, wp, wn)
    return out


def fp8_linear(A: Fp8Matrix, B: Fp8Matrix, bias=None, activation: str | None = None, residual=None,
               out_dtype=None, out=None, ws=None):
    """act(A·Bᵀ + bias) + residual: A [M, K] with block_rows 1, B [N, K] with
    block_rows 128, bias [N] (float32/bfloat16/float16), residual [M, N] of
    the result's type.  Returns [M, N] in out_dtype (bfloat16 unless given, or
    `out`'s type), rounded once; with out_dtype torch.float8_e4m3fn (or an
    Fp8Matrix `out`) an Fp8Matrix with block_rows 1, without a residual.
    Products and sums are fp8_gemm's; out may be residual itself.
    ws: the split-K workspace (allocated here when None; pass one to reuse)."""
    M, K, lda, dev = _fp8_arg(A, "A", 1)
    N, kb, ldb, _ = _fp8_arg(B, "B", FP8_BLOCK, dev)
    empty, e4m3 = _t8()[:2]
    if kb != K:
        raise ValueError(f"A has {K} columns, B has {kb}")
    act = -1
    if activation is not None:
        act = _ACTIVATIONS.get(activation)
        if act is None:
            raise ValueError(f"activation must be None or one of {sorted(_ACTIVATIONS)} (got {activation!r})")
    bp, bdt = None, 0
    if bias is not None:
        bdt = _fp8_dtype(bias, "bias")
        if bias.shape != (N,) or not bias.is_contiguous() or bias.device != dev:
            raise ValueError(f"bias must be contiguous of shape {(N,)} on {dev}")
        bp = bias.data_ptr()
    cp, cdt, ldc, qc, ldq, qs, rp, ldr = None, 0, 0, None, 0, None, None, 0
    if isinstance(out, Fp8Matrix) or (out is None and out_dtype is e4m3):
        if residual is not None:
            raise ValueError("a residual needs a tensor result, not an Fp8Matrix")
        if out is None:
            out, ldq = _fp8_new(M, N, 1, dev)
        else:
            if out_dtype is not None and out_dtype is not e4m3:
                raise ValueError(f"an Fp8Matrix out is {e4m3} (got {out_dtype})")
            mo, no, ldq, _ = _fp8_arg(out, "out", 1, dev)
            if (mo, no) != (M, N):
                raise ValueError(f"out must have shape {(M, N)} (got {(mo, no)})")
        qc, qs = out.codes.data_ptr(), out.scales.data_ptr()
    else:
        if out is None:
            out = empty((M, N), dtype=out_dtype or _torch().bfloat16, device=dev)
            ldc = N
        else:
            if out_dtype is not None and out.dtype != out_dtype:
                raise ValueError(f"out must be {out_dtype} (got {out.dtype})")
            ldc = _fp8_out(out, "out", out.dtype, (M, N), dev)
        cdt = _fp8_dtype(out, "out")
        cp = out.data_ptr()
        if residual is not None:
            ldr = _fp8_out(residual, "residual", out.dtype, (M, N), dev)
            rp = residual.data_ptr()
    wp, wn, ws = _fp8_workspace(_native.WS_FP8_LINEAR, M, N, K, ws, dev)
    _launch(dev, _native.lib().gptq_fp8_linear, A.codes.data_ptr(), A.scales.data_ptr(), M, K, lda,
            B.codes.data_ptr(), B.scales.data_ptr(), N, ldb, bp, bdt, act, rp, ldr, cp, cdt, ldc, qc,
            ldq, qs, wp, wn)
    return out


# ---------------------------------------------------------------- experts
@dataclasses.dataclass(slots=True)
class Fp8Experts:
    """One block-scaled weight matrix for each expert: value = code·scale."""
    codes: "object"      # [E, N, K] float8_e4m3fn, unit column stride
    scales: "object"     # [E, ceil(N/128), ceil(K/128)] float32

    def expert(self, e: int) -> Fp8Matrix:
        """The weights of expert e, as fp8_gemm takes them (a view)."""
        return Fp8Matrix(self.codes[e], self.scales[e], FP8_BLOCK)


@dataclasses.dataclass(slots=True)
class Routing:
    """Which experts each token takes, and the slots token·top_k + j by expert."""
    ids: "object"        # [T, top_k] int32; -1: none
    weights: "object"    # [T, top_k] float32
    offsets: "object"    # [E + 1] int32: expert e's positions in order
    order: "object"      # [T·top_k] int32: slots sorted by expert, -1 behind the last


_SCORES = {"softmax": _native.SCORE_SOFTMAX, "sigmoid": _native.SCORE_SIGMOID}


def expert_workspace_bytes(which: int, T: int, top_k: int, n_experts: int, N: int = 0, K: int = 0) -> int:
    return int(_native.lib().gptq_expert_workspace_bytes(which, T, top_k, n_experts, N, K))


@functools.lru_cache(maxsize=4096)
def _expert_bytes(which, T, k, E, N, K):
    return _native.lib().gptq_expert_workspace_bytes(which, T, k, E, N, K)


def _expert_workspace(which, T, k, E, N, K, ws, dev):
    """(address, bytes, tensor to keep) of an experts' call's workspace."""
    if ws is None:
        need = _expert_bytes(which, T, k, E, N, K)
        if need <= 256:
            return None, 0, None
        ws = _workspace(need, dev)
    else:
        _ws_check(ws, dev)
    return ws.data_ptr(), ws.numel(), ws


def moe_route(logits, top_k: int, scores: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
              group_top: int = 1, renormalize: bool = True, scale: float = 1.0, mask=None,
              ws=None) -> Routing:
    """Each token's top_k experts of logits [T, E] (float32/bfloat16/float16).

    p = softmax or sigmoid of the logits; the choice goes by c = p + bias
    (bias [E] float32; without one by the logits), among the top_groups of
    `groups` groups of neighbouring experts with the largest sum of their
    group_top (1 or 2) best c; ties to the lowest index.  weights = p of the
    chosen, over their sum with renormalize, times scale.  A logit of -inf
    excludes its expert; mask [T] bool: False for tokens that take none
    (padding).  Slots without an expert have id -1 and weight 0.
    ws: the workspace (allocated here when None; pass one to reuse)."""
    empty, _, f32 = _t8()[:3]
    i32 = _torch().int32
    dt = _fp8_dtype(logits, "logits")
    ld = _fp8_rows(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    sc = _SCORES.get(scores)
    if sc is None:
        raise ValueError(f"scores must be one of {sorted(_SCORES)} (got {scores!r})")
    bp, mp = None, None
    if bias is not None:
        if bias.dtype != f32 or bias.shape != (E,) or not bias.is_contiguous() or bias.device != dev:
            raise ValueError(f"bias must be contiguous float32 of shape {(E,)} on {dev}")
        bp = bias.data_ptr()
    if mask is not None:
        if mask.dtype != _torch().bool or mask.shape != (T,) or not mask.is_contiguous() or mask.device != dev:
            raise ValueError(f"mask must be contiguous bool of shape {(T,)} on {dev}")
        mp = mask.data_ptr()
    wp, wn, ws = _expert_workspace(_native.WS_MOE, T, top_k, E, 0, 0, ws, dev)
    k = max(int(top_k), 0)   # a bad top_k is the library's to refuse
    r = Routing(empty((T, k), dtype=i32, device=dev), empty((T, k), dtype=f32, device=dev),
                empty(E + 1, dtype=i32, device=dev), empty(T * k, dtype=i32, device=dev))
    _launch(dev, _native.lib().gptq_moe_route, logits.data_ptr(), dt, T, E, ld, bp, mp, sc, top_k,
            groups, top_groups, group_top, 1 if renormalize else 0, scale, r.ids.data_ptr(),
            r.weights.data_ptr(), r.offsets.data_ptr(), r.order.data_ptr(), wp, wn)
    return r


def moe_plan(ids, weights, n_experts: int, ws=None) -> Routing:
    """A Routing of experts that were chosen elsewhere: ids [T, top_k] int32
    (below 0 or from n_experts on: none), weights [T, top_k] float32."""
    empty, _, f32 = _t8()[:3]
    i32 = _torch().int32
    if ids.dim() != 2:
        raise ValueError("ids must be [T, top_k]")
    T, k = ids.shape
    dev = ids.device
    _require(ids, "ids", i32, (T, k))
    _require(weights, "weights", f32, (T, k), dev)
    wp, wn, ws = _expert_workspace(_native.WS_MOE, T, k, n_experts, 0, 0, ws, dev)
    r = Routing(ids, weights, empty(max(n_experts, 0) + 1, dtype=i32, device=dev),
                empty(T * k, dtype=i32, device=dev))
    _launch(dev, _native.lib().gptq_moe_plan, ids.data_ptr(), T, k, n_experts, r.offsets.data_ptr(),
            r.order.data_ptr(), wp, wn)
    return r


def fp8_quantize_experts(W, out: Fp8Experts | None = None) -> Fp8Experts:
    """W [E, N, K] (float32/bfloat16/float16) in e4m3, each expert's matrix as
    fp8_quantize(W[e], 128) gives it, one call for each.  out: to be filled; its
    experts lie apart."""
    if W.dim() != 3:
        raise ValueError("W must be [E, N, K]")
    empty, e4m3, f32 = _t8()[:3]
    E, N, K = W.shape
    if out is None:
        ld = (K + 15) // 16 * 16
        out = Fp8Experts(empty((E, N, ld), dtype=e4m3, device=W.device)[:, :, :K],
                         empty((E, (N + FP8_BLOCK - 1) // FP8_BLOCK, (K + FP8_BLOCK - 1) // FP8_BLOCK),
                               dtype=f32, device=W.device))
    elif out.codes.shape != W.shape or out.codes.device != W.device:
        raise ValueError(f"out must have shape {tuple(W.shape)} on {W.device}")
    _, _, _, ld, next_ = _experts_arg(out, "out", W.device)
    if _experts_overlap(E, N, K, ld, next_):
        raise ValueError("out's experts overlap in memory")
    for e in range(E):
        fp8_quantize(W[e], FP8_BLOCK, out=out.expert(e))
    return out


def _experts_overlap(E, N, K, ld, next_) -> bool:
    """Whether rows of two experts share bytes (one's rows lie apart: ld >= K)."""
    for e in range(1, E):
        n = e * next_ // max(ld, 1)   # the other's rows next to this one's first
        if any(abs(e * next_ - min(i, N - 1) * ld) < K for i in (n, n + 1)):
            return True
    return False


def _experts_arg(m: Fp8Experts, name, device):
    """(E, N, K, row stride, expert stride) of the experts' weights after their checks."""
    c, s = m.codes, m.scales
    _, e4m3, f32, _, _, _ = _t8()
    if c.dtype != e4m3:
        raise ValueError(f"{name}.codes must be float8_e4m3fn (got {c.dtype})")
    if c.dim() != 3:
        raise ValueError(f"{name}.codes must be [E, N, K]")
    E, N, K = c.shape
    next_, ld, one = c.stride()
    if N <= 1:
        ld = K
    if E <= 1:
        next_ = 0
    if (one != 1 and K > 1) or ld < K or next_ < 0:
        raise ValueError(f"{name}.codes must have unit column stride")
    want = (E, (N + FP8_BLOCK - 1) // FP8_BLOCK, (K + FP8_BLOCK - 1) // FP8_BLOCK)
    if s.dtype != f32 or s.shape != want or not s.is_contiguous():
        raise ValueError(f"{name}.scales must be contiguous float32 of shape {want} "
                         f"(got {s.dtype}, {tuple(s.shape)})")
    if c.device != device or s.device != device:
        raise ValueError(f"{name} is on {c.device} (scales on {s.device}), expected {device}")
    return E, N, K, ld, next_


def _routing_arg(r: Routing, E, device):
    """(T, top_k) of a routing over E experts after its checks."""
    _, _, f32, _, _, _ = _t8()
    i32 = _torch().int32
    if r.ids.dim() != 2:
        raise ValueError("routing.ids must be [T, top_k]")
    T, k = r.ids.shape
    for t, name, dtype, shape in ((r.ids, "ids", i32, (T, k)), (r.weights, "weights", f32, (T, k)),
                                  (r.offsets, "offsets", i32, (E + 1,)), (r.order, "order", i32, (T * k,))):
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
            raise ValueError(f"routing.{name} must be contiguous {dtype} of shape {shape} on {device} "
                             f"(got {t.dtype}, {tuple(t.shape)} on {t.device})")
    return T, k


def fp8_expert_gated_gemm(A: Fp8Matrix, routing: Routing, gate: Fp8Experts, up: Fp8Experts,
                          activation: str = "silu", out_dtype=None, out=None, ws=None):
    """act(x·gate_eᵀ)·(x·up_eᵀ) of each token x of A [T, K] and each of its
    experts e, rows in the order of routing.order: an Fp8Matrix [T·top_k, N]
    with block_rows 1, or a tensor of out_dtype where that is given; `out` is
    either, to be filled.  Rows behind the last that has an expert are left as
    they were.  ws: as for fp8_gated_gemm."""
    T, K, lda, dev = _fp8_arg(A, "A", 1)
    E, N, kg, ldg, next_g = _experts_arg(gate, "gate", dev)
    eu, nu, ku, ldu, next_u = _experts_arg(up, "up", dev)
    if kg != K or ku != K or nu != N or eu != E:
        raise ValueError(f"A has {K} columns; gate {(E, N, kg)} and up {(eu, nu, ku)} do not fit")
    tr, k = _routing_arg(routing, E, dev)
    if tr != T:
        raise ValueError(f"A has {T} rows, the routing {tr} tokens")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)} (got {activation!r})")
    M = T * k
    cp, cdt, ldc, qc, ldq, qs = None, 0, 0, None, 0, None
    if out is None and out_dtype is None:
        out, ldq = _fp8_new(M, N, 1, dev)
        qc, qs = out.codes.data_ptr(), out.scales.data_ptr()
    elif isinstance(out, Fp8Matrix):
        if out_dtype is not None:
            raise ValueError("an Fp8Matrix out has no out_dtype")
        mo, no, ldq, _ = _fp8_arg(out, "out", 1, dev)
        if (mo, no) != (M, N):
            raise ValueError(f"out must have shape {(M, N)} (got {(mo, no)})")
        qc, qs = out.codes.data_ptr(), out.scales.data_ptr()
    else:
        if out is None:
            out = _t8()[0]((M, N), dtype=out_dtype, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out must be {out_dtype} (got {out.dtype})")
        cdt = _fp8_dtype(out, "out")
        ldc = _fp8_out(out, "out", out.dtype, (M, N), dev)
        cp = out.data_ptr()
    wp, wn, ws = _expert_workspace(_native.WS_EXPERT_GATED, T, k, E, N, K, ws, dev)
    _launch(dev, _native.lib().gptq_fp8_expert_gated_gemm, A.codes.data_ptr(), A.scales.data_ptr(), T,
            K, lda, k, routing.offsets.data_ptr(), routing.order.data_ptr(), E, gate.codes.data_ptr(),
            gate.scales.data_ptr(), ldg, next_g, up.codes.data_ptr(), up.scales.data_ptr(), ldu, next_u,
            N, act, cp, cdt, ldc, qc, ldq, qs, wp, wn)
    return out


def fp8_expert_gemm(H: Fp8Matrix, routing: Routing, down: Fp8Experts, residual=None, out_dtype=None,
                    out=None, ws=None):
    """Σ_j weights[t, j]·(h·down_eᵀ) + residual[t]: H [T·top_k, K] in the order
    of routing.order, as fp8_expert_gated_gemm gives it; the result [T, N] in
    out_dtype (bfloat16 unless given, or `out`'s type), rounded once.
    residual [T, N] of that type; out may be residual itself.
    ws: the workspace (allocated here when None; pass one to reuse)."""
    M, K, ldh, dev = _fp8_arg(H, "H", 1)
    E, N, kd, ldd, next_d = _experts_arg(down, "down", dev)
    if kd != K:
        raise ValueError(f"H has {K} columns, down has {kd}")
    T, k = _routing_arg(routing, E, dev)
    if T * k != M:
        raise ValueError(f"H has {M} rows, the routing {T} tokens of {k} slots")
    if out is None:
        out = _t8()[0]((T, N), dtype=out_dtype or _torch().bfloat16, device=dev)
        ldc = N
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out must be {out_dtype} (got {out.dtype})")
        ldc = _fp8_out(out, "out", out.dtype, (T, N), dev)
    cdt = _fp8_dtype(out, "out")
    rp, ldr = None, 0
    if residual is not None:
        ldr = _fp8_out(residual, "residual", out.dtype, (T, N), dev)
        rp = residual.data_ptr()
    wp, wn, ws = _expert_workspace(_native.WS_EXPERT_GEMM, T, k, E, N, K, ws, dev)
    _launch(dev, _native.lib().gptq_fp8_expert_gemm, H.codes.data_ptr(), H.scales.data_ptr(), T, K, ldh,
            k, routing.ids.data_ptr(), routing.weights.data_ptr(), routing.offsets.data_ptr(),
            routing.order.data_ptr(), E, down.codes.data_ptr(), down.scales.data_ptr(), ldd, next_d, N,
            rp, ldr, out.data_ptr(), cdt, ldc, wp, wn)
    return out


def quantize(W, X, params: GPTQParams = GPTQParams()):
    """Whole layer: H from X, prepare, sweep.  Returns (Quantized, Prepared, H_d)."""
    torch = _torch()
    d = W.shape[1]
    H = torch.zeros(d, d, dtype=torch.float32, device=W.device)
    hessian_accumulate(H, X)
    prep = prepare_hinv(H, params)
    return quantize_layer(W, prep, params), prep, H
