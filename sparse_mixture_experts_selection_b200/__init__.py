"""B200 (sm_100a) forward pass of one sparse Mixture-of-Experts layer.

Thin Python binding of the C ABI in include/moe.h (libmoe.so): argument
marshalling only.  Every step of the layer runs in the library's CUDA kernels;
there is no CPU or PyTorch fallback -- importing this package fails loudly when
the library is missing or does not load.

PyTorch provides the device memory and the stream: tensors are passed by
pointer (``tensor.data_ptr()``) and work is enqueued on
``torch.cuda.current_stream()`` unless a stream is given.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

from ._build import LIB_PATH

__all__ = [
    "MoeConfig", "MoeError", "lib", "config_for", "moe_workspace_size", "moe_route", "moe_permute",
    "moe_expert_ffn", "moe_expert_ffn_workspace_size", "moe_combine", "moe_bias_update",
    "moe_layer_forward", "moe_get_device_error", "moe_clear_device_error", "alloc_workspace",
    "moe_router_stats", "moe_router_stats_workspace_size", "ROUTER_STATS", "moe_permute_noalloc",
    "moe_quantized_bytes", "moe_quantize_rows", "DTYPE_BF16_E4M3", "moe_layer_backward", "moe_gather_rows",
    "moe_set_phase_events", "moe_selftest_bounded_wait", "moe_ep_plan", "moe_expert_ffn_tile_rows",
    "moe_layer_norm", "moe_layer_norm_backward", "moe_layer_norm_backward_workspace_size", "moe_dropout_add",
    "moe_dropout_backward", "moe_quantize_tiles", "moe_quantize_blocks", "moe_block_matmul",
    "moe_block_matmul_workspace_size", "moe_block_ffn", "moe_block_ffn_workspace_size", "NORM_LAYER", "NORM_RMS",
    "SCORE_SIGMOID", "SCORE_SOFTMAX", "DTYPE_F32", "DTYPE_BF16",
]

SCORE_SIGMOID, SCORE_SOFTMAX = 0, 1
DTYPE_F32, DTYPE_BF16, DTYPE_BF16_E4M3 = 0, 1, 2
NORM_LAYER, NORM_RMS = 0, 1
DEVERR_NONE, DEVERR_WAIT_TIMEOUT, DEVERR_INDEX, DEVERR_RANGE = 0, 1, 2, 3
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE"}


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("E_r", ctypes.c_int32),
                ("E_s", ctypes.c_int32), ("K", ctypes.c_int32), ("d_ffn", ctypes.c_int32),
                ("d_ffn_shared", ctypes.c_int32), ("score_fn", ctypes.c_int32),
                ("n_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_topn", ctypes.c_int32), ("capacity_factor", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("add_residual", ctypes.c_int32),
                ("train", ctypes.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status


_lib = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32

# (name, restype, argtypes) of every exported symbol of include/moe.h
SIGNATURES = {
    "moe_abi_version": (ctypes.c_int32, []),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_last_error_detail": (ctypes.c_char_p, []),
    "moe_workspace_size": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_expert_ffn_workspace_size": (ctypes.c_int, [_P, _I32, _I32, _I32, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_expert_ffn_tile_rows": (ctypes.c_int, [_P, _I32, _I32, ctypes.POINTER(ctypes.c_int32)]),
    "moe_route": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_permute": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_expert_ffn": (ctypes.c_int, [_P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P,
                                      ctypes.c_size_t, _P]),
    "moe_combine": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P]),
    "moe_bias_update": (ctypes.c_int, [_P, _P, ctypes.c_float, _P, _P, _P]),
    "moe_layer_forward": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                         _P, _P, _P, _P, _I32, ctypes.c_float, _P, _P,
                                         ctypes.c_size_t, _P]),
    "moe_router_stats_workspace_size": (ctypes.c_int, [_P, _I32, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_quantized_bytes": (ctypes.c_int, [ctypes.c_int64, _I32, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_layer_backward": (ctypes.c_int, [_P] * 20 + [_P, ctypes.c_size_t, _P]),
    "moe_quantize_rows": (ctypes.c_int, [_P, _I32, ctypes.c_int64, _I32, _P, _P]),
    "moe_gather_rows": (ctypes.c_int, [_P, ctypes.c_int64, _I32, _P, ctypes.c_int64, _P, _P]),
    "moe_ep_plan": (ctypes.c_int, [_P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P]),
    "moe_router_stats": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, ctypes.c_float, ctypes.c_float,
                                        ctypes.c_float, _P, _P, ctypes.c_size_t, _P]),
    "moe_get_device_error": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int32)]),
    "moe_clear_device_error": (ctypes.c_int, [_P, _P]),
    "moe_set_phase_events": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), _I32]),
    "moe_permute_noalloc": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_layer_norm": (ctypes.c_int, [_P, _I32, ctypes.c_int64, _I32, _I32, _P, _P, ctypes.c_float] + [_P] * 6),
    "moe_layer_norm_backward_workspace_size": (ctypes.c_int, [ctypes.c_int64, _I32, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_layer_norm_backward": (ctypes.c_int, [_P, _P, _I32, ctypes.c_int64, _I32, _I32] + [_P] * 8
                                + [ctypes.c_size_t, _P]),
    "moe_dropout_add": (ctypes.c_int, [_P, _P, _I32, ctypes.c_int64, ctypes.c_double, _P, _P, _P]),
    "moe_dropout_backward": (ctypes.c_int, [_P, _I32, ctypes.c_int64, ctypes.c_double, _P, _P, _P]),
    "moe_quantize_tiles": (ctypes.c_int, [_P, _I32, ctypes.c_int64, _I32, _P, _P, _P]),
    "moe_quantize_blocks": (ctypes.c_int, [_P, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "moe_block_matmul_workspace_size": (ctypes.c_int, [_I32] * 4 + [ctypes.POINTER(ctypes.c_size_t)]),
    "moe_block_matmul": (ctypes.c_int, [_I32] * 4 + [_P] * 6 + [_I32, _P, _P, ctypes.c_size_t, _P]),
    "moe_block_ffn_workspace_size": (ctypes.c_int, [_I32] * 4 + [ctypes.POINTER(ctypes.c_size_t)]),
    "moe_block_ffn": (ctypes.c_int, [_I32] * 4 + [_P] * 10 + [_I32, _P, _P, ctypes.c_size_t, _P]),
    "moe_selftest_bounded_wait": (ctypes.c_int, [_P, ctypes.c_int64, _P]),
}

# phases of moe_layer_forward marked by moe_set_phase_events (between marks i and i+1)
PHASES = ["route", "dispatch", "ffn_groups", "ffn_gate_up", "ffn_down", "combine", "bias_step"]


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m sparse_mixture_experts_selection_b200._build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != 0:
        raise MoeError(status, lib().moe_last_error_detail().decode())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current_stream = None


def _stream(stream) -> Optional[int]:
    global _current_stream
    if stream is None:
        if _current_stream is None:
            import torch
            # the handle alone: making a Stream object takes as long as a launch
            raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
            _current_stream = (lambda: raw(device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
        return _current_stream()
    return stream if isinstance(stream, int) else stream.cuda_stream


def config_for(w, **overrides) -> MoeConfig:
    """MoeConfig of a ``moe_inputs.Workload`` (or any object with the same fields)."""
    c = MoeConfig(T=w.T, d_model=w.d_model, E_r=w.E_r, E_s=w.E_s, K=w.K, d_ffn=w.d_ffn,
                  d_ffn_shared=w.d_ffn_shared, score_fn=w.score_fn, n_groups=w.n_groups,
                  topk_groups=w.topk_groups, group_topn=w.group_topn,
                  capacity_factor=w.capacity_factor,
                  dtype={"bf16": DTYPE_BF16, "bf16_e4m3": DTYPE_BF16_E4M3}.get(w.dtype, DTYPE_F32),
                  add_residual=w.add_residual)
    for k, v in overrides.items():
        setattr(c, k, v)
    return c


def moe_workspace_size(cfg: MoeConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def moe_expert_ffn_workspace_size(cfg: MoeConfig, n_experts: int, d_ffn: int, max_rows: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_expert_ffn_workspace_size(ctypes.byref(cfg), n_experts, d_ffn, max_rows, ctypes.byref(n)))
    return n.value


def moe_expert_ffn_tile_rows(cfg: MoeConfig, n_experts: int, max_rows: int) -> int:
    """Row-tile height of the GEMMs moe_expert_ffn runs for these arguments:
    256 on CTA pairs, 128 single-CTA tensor-core, the CUDA-core tile for fp32."""
    n = ctypes.c_int32(0)
    _check(lib().moe_expert_ffn_tile_rows(ctypes.byref(cfg), n_experts, max_rows, ctypes.byref(n)))
    return n.value


def alloc_workspace(nbytes: int, device="cuda"):
    """A zeroed uint8 device tensor usable as a workspace (torch allocations are
    at least 256-byte aligned)."""
    import torch
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def moe_route(cfg, h, e, b, s_in, s_out, idx, gates, counts, ws, stream=None, z_out=None):
    _check(lib().moe_route(ctypes.byref(cfg), _ptr(h), _ptr(e), _ptr(b), _ptr(s_in), _ptr(s_out),
                           _ptr(z_out), _ptr(idx), _ptr(gates), _ptr(counts), _ptr(ws), ws.numel(),
                           _stream(stream)))


def moe_router_stats_workspace_size(cfg: MoeConfig, seq_len: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_router_stats_workspace_size(ctypes.byref(cfg), int(seq_len), ctypes.byref(n)))
    return n.value


def moe_gather_rows(src, n_src: int, row_bytes: int, map_, n_rows: int, dst, stream=None):
    """dst[r] = src[map_[r]] row by row (zero where map_[r] < 0)."""
    _check(lib().moe_gather_rows(_ptr(src), int(n_src), int(row_bytes), _ptr(map_), int(n_rows), _ptr(dst),
                                 _stream(stream)))


def moe_quantized_bytes(n_rows: int, cols: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_quantized_bytes(int(n_rows), int(cols), ctypes.byref(n)))
    return n.value


def moe_quantize_rows(src, src_dtype: int, n_rows: int, cols: int, dst, stream=None):
    _check(lib().moe_quantize_rows(_ptr(src), int(src_dtype), int(n_rows), int(cols), _ptr(dst),
                                   _stream(stream)))


def moe_layer_backward(cfg, h, e, s, idx, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, dy, dh, de,
                       dw_gate, dw_up, dw_down, dws_gate, dws_up, dws_down, ws, stream=None):
    """Gradients of the last moe_layer_forward (cfg.train = 1, same workspace)."""
    _check(lib().moe_layer_backward(
        ctypes.byref(cfg), _ptr(h), _ptr(e), _ptr(s), _ptr(idx), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
        _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(dy), _ptr(dh), _ptr(de), _ptr(dw_gate), _ptr(dw_up),
        _ptr(dw_down), _ptr(dws_gate), _ptr(dws_up), _ptr(dws_down), _ptr(ws), ws.numel(), _stream(stream)))


# order of the values moe_router_stats writes
ROUTER_STATS = ["aux_loss", "z_loss", "seq_balance_loss", "load_entropy", "max_vio", "dropped_rate"]


def moe_router_stats(cfg, s, z, idx, kept, stats, ws, seq_len=0, alpha_aux=0.01, c_z=1e-3,
                     alpha_seq=1e-4, stream=None):
    _check(lib().moe_router_stats(ctypes.byref(cfg), _ptr(s), _ptr(z), _ptr(idx), _ptr(kept),
                                  int(seq_len), float(alpha_aux), float(c_z), float(alpha_seq),
                                  _ptr(stats), _ptr(ws), ws.numel(), _stream(stream)))


def moe_permute(cfg, idx, gates, h, offsets, perm_tok, row_of, kept, row_gate, x_perm, ws, stream=None):
    _check(lib().moe_permute(ctypes.byref(cfg), _ptr(idx), _ptr(gates), _ptr(h), _ptr(offsets),
                             _ptr(perm_tok), _ptr(row_of), _ptr(kept), _ptr(row_gate), _ptr(x_perm),
                             _ptr(ws), ws.numel(), _stream(stream)))


def moe_permute_noalloc(cfg, idx, gates, h, offsets, perm_tok, row_of, kept, row_gate, x_perm,
                        dev_error=None, stream=None):
    """moe_permute with no workspace: for callers that cannot allocate device
    memory (see include/moe.h); scratch is a fixed array inside the library."""
    _check(lib().moe_permute_noalloc(ctypes.byref(cfg), _ptr(idx), _ptr(gates), _ptr(h), _ptr(offsets),
                                     _ptr(perm_tok), _ptr(row_of), _ptr(kept), _ptr(row_gate),
                                     _ptr(x_perm), _ptr(dev_error), _stream(stream)))


def moe_ep_plan(offsets_all, world, rank, E_r, max_recv, splits, local_offsets, regroup, inverse,
                dev_error=None, stream=None):
    """Exchange plan of an expert-parallel layer on the device (see include/moe.h)."""
    _check(lib().moe_ep_plan(_ptr(offsets_all), world, rank, E_r, max_recv, _ptr(splits), _ptr(local_offsets),
                             _ptr(regroup), _ptr(inverse), _ptr(dev_error), _stream(stream)))


def moe_expert_ffn(cfg, n_experts, d_ffn, max_rows, offsets, x, w_gate, w_up, w_down, row_scale,
                   out, ws, stream=None):
    _check(lib().moe_expert_ffn(ctypes.byref(cfg), n_experts, d_ffn, max_rows, _ptr(offsets), _ptr(x),
                                _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(row_scale), _ptr(out),
                                _ptr(ws), ws.numel(), _stream(stream)))


def moe_combine(cfg, h, slot, shared_out, row_of, y, stream=None):
    _check(lib().moe_combine(ctypes.byref(cfg), _ptr(h), _ptr(slot), _ptr(shared_out), _ptr(row_of),
                             _ptr(y), _stream(stream)))


def moe_bias_update(cfg, counts, gamma, b, max_vio, stream=None):
    _check(lib().moe_bias_update(ctypes.byref(cfg), _ptr(counts), float(gamma), _ptr(b), _ptr(max_vio),
                                 _stream(stream)))


def moe_layer_forward(cfg, h, e, b, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, y, ws, *,
                      s_in=None, idx_out=None, gates_out=None, counts_out=None, kept_out=None,
                      s_out=None, z_out=None, update_bias=False, gamma=0.0, max_vio_out=None,
                      stream=None):
    _check(lib().moe_layer_forward(
        ctypes.byref(cfg), _ptr(h), _ptr(e), _ptr(b), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
        _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(s_in), _ptr(y), _ptr(idx_out), _ptr(gates_out),
        _ptr(counts_out), _ptr(kept_out), _ptr(s_out), _ptr(z_out), int(bool(update_bias)), float(gamma),
        _ptr(max_vio_out), _ptr(ws), ws.numel(), _stream(stream)))


def moe_get_device_error(ws) -> int:
    code = ctypes.c_int32(0)
    st = lib().moe_get_device_error(_ptr(ws), ctypes.byref(code))
    if st not in (0, 5):
        _check(st)
    return code.value


def moe_set_phase_events(events) -> None:
    """Record these torch.cuda.Event objects (up to 8) at the phase boundaries of
    every later moe_layer_forward call in this thread; [] turns it off."""
    arr = (ctypes.c_void_p * max(1, len(events)))(*[ev.cuda_event for ev in events])
    _check(lib().moe_set_phase_events(arr, len(events)))


def moe_selftest_bounded_wait(ws, limit_ns: int = 50_000_000, stream=None) -> None:
    """Enqueue the failure-detection self-test (see include/moe.h)."""
    _check(lib().moe_selftest_bounded_wait(_ptr(ws), int(limit_ns), _stream(stream)))


def moe_clear_device_error(ws, stream=None) -> None:
    _check(lib().moe_clear_device_error(_ptr(ws), _stream(stream)))


# ---------------------------------------------------------------------------
# around and inside a sublayer x + dropout(MoE(norm(x)))
# ---------------------------------------------------------------------------
class _Types:
    """The types that a tensor may have, by torch's names (torch is imported with
    the first call)."""
    __slots__ = ("names", "dtypes")

    def __init__(self, *names):
        self.names, self.dtypes = names, None

    def load(self):
        import torch
        self.dtypes = tuple(getattr(torch, k) for k in self.names)
        return self.dtypes


_F32, _I32S, _BF16S = _Types("float32"), _Types("int32"), _Types("bfloat16")
_CODES, _RNG, _BYTES = _Types("uint8", "float8_e4m3fn"), _Types("int64", "uint64"), _Types("uint8")
_ACT = {DTYPE_F32: _F32, DTYPE_BF16: _BF16S}
_UNKNOWN = _Types("bool")          # an unknown dtype code: the library would refuse it too
_torch = None


def _refuse(name, t, types, n):
    if t.dtype not in types.dtypes:
        raise MoeError(1, f"{name} has type {t.dtype}, not {' or '.join(types.names)}")
    if not t.is_contiguous():
        raise MoeError(1, f"{name} is not contiguous")
    raise MoeError(1, f"{name} has {t.numel()} values, {n} are needed")


def _pointers(*checks):
    """The addresses of a call's tensors and the device they are on, after a check
    of each (name, tensor, types, number of values).  The kernels take dense
    arrays by pointer, so a strided view, another type, a short tensor or one of
    another device is refused here.  None and plain addresses pass (a workspace's
    size is asked for apart, by _room)."""
    out, device, other = [], None, None
    for name, t, types, n in checks:
        if t is None or t.__class__ is int:
            out.append(t)
            continue
        if t.dtype not in (types.dtypes or types.load()) or not t.is_contiguous() or t.numel() < n:
            _refuse(name, t, types, n)
        at = t.get_device()
        if at != device:
            if device is not None:
                other = name
            device = at
        out.append(t.data_ptr())
    if other is not None or (device is not None and device < 0):
        raise MoeError(1, "the tensors are not on one GPU" + (f" ({other} is on another device)" if other else ""))
    out.append(device)
    return out


def _room(ws) -> int:
    """Bytes of a workspace.  An address alone does not say how many there are."""
    if ws.__class__ is int:
        raise MoeError(3, "ws is a plain address, which has no size: pass the tensor")
    return 0 if ws is None else ws.numel()


def _enqueue(fn, device, stream, *args) -> None:
    """Make the call on the tensors' device and stream."""
    global _torch
    if _torch is None:
        import torch as _torch
    if device is None or device == _torch.cuda.current_device():
        status = fn(*args, _stream(stream))
    else:
        with _torch.cuda.device(device):
            status = fn(*args, _stream(stream))
    if status != 0:
        raise MoeError(status, lib().moe_last_error_detail().decode())


def _blocks(n: int) -> int:
    return (n + 127) // 128


def moe_layer_norm(x, dtype: int, n_rows: int, d: int, kind: int, gamma, beta, eps: float, out, mean=None, rstd=None,
                   codes=None, scales=None, stream=None):
    """Norm of n_rows rows of d values (NORM_LAYER or NORM_RMS); with codes and
    scales the output once more in e4m3 tiles of 1 x 128 (see include/moe.h)."""
    n, act = n_rows * d, _ACT.get(dtype, _UNKNOWN)
    (p_x, p_gamma, p_beta, p_out, p_mean, p_rstd, p_codes, p_scales, device) = _pointers(
        ("x", x, act, n), ("gamma", gamma, _F32, d), ("beta", beta, _F32, d), ("out", out, act, n),
        ("mean", mean, _F32, n_rows), ("rstd", rstd, _F32, n_rows), ("codes", codes, _CODES, n),
        ("scales", scales, _F32, n_rows * _blocks(d)))
    _enqueue(lib().moe_layer_norm, device, stream, p_x, dtype, n_rows, d, kind, p_gamma, p_beta, eps, p_out, p_mean,
             p_rstd, p_codes, p_scales)


def moe_layer_norm_backward_workspace_size(n_rows: int, d: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_layer_norm_backward_workspace_size(int(n_rows), int(d), ctypes.byref(n)))
    return n.value


def moe_layer_norm_backward(dy, x, dtype: int, n_rows: int, d: int, kind: int, gamma, mean, rstd, dres, dx, dgamma,
                            dbeta, ws, stream=None):
    """Gradients of moe_layer_norm; dres is added to dx (see include/moe.h)."""
    n, act = n_rows * d, _ACT.get(dtype, _UNKNOWN)
    (p_dy, p_x, p_gamma, p_mean, p_rstd, p_dres, p_dx, p_dgamma, p_dbeta, p_ws, device) = _pointers(
        ("dy", dy, act, n), ("x", x, act, n), ("gamma", gamma, _F32, d), ("mean", mean, _F32, n_rows),
        ("rstd", rstd, _F32, n_rows), ("dres", dres, act, n), ("dx", dx, act, n), ("dgamma", dgamma, _F32, d),
        ("dbeta", dbeta, _F32, d), ("ws", ws, _BYTES, 0))
    _enqueue(lib().moe_layer_norm_backward, device, stream, p_dy, p_x, dtype, n_rows, d, kind, p_gamma, p_mean,
             p_rstd, p_dres, p_dx, p_dgamma, p_dbeta, p_ws, _room(ws))


def moe_dropout_add(x, res, dtype: int, n: int, p: float, rng, out, stream=None):
    """out = res + dropout(x) over n values; rng: int64 [2] on the device, the
    seed and the number of this draw (see include/moe.h)."""
    act = _ACT.get(dtype, _UNKNOWN)
    (p_x, p_res, p_rng, p_out, device) = _pointers(
        ("x", x, act, n), ("res", res, act, n), ("rng", rng, _RNG, 2), ("out", out, act, n))
    _enqueue(lib().moe_dropout_add, device, stream, p_x, p_res, dtype, n, p, p_rng, p_out)


def moe_dropout_backward(dy, dtype: int, n: int, p: float, rng, dx, stream=None):
    """dx = dy through the mask that moe_dropout_add drew with the same rng, p and n."""
    act = _ACT.get(dtype, _UNKNOWN)
    (p_dy, p_rng, p_dx, device) = _pointers(
        ("dy", dy, act, n), ("rng", rng, _RNG, 2), ("dx", dx, act, n))
    _enqueue(lib().moe_dropout_backward, device, stream, p_dy, dtype, n, p, p_rng, p_dx)


def moe_quantize_tiles(src, src_dtype: int, n_rows: int, cols: int, codes, scales, stream=None):
    """e4m3 codes and one power-of-two scale for each 1 x 128 tile of the rows."""
    (p_src, p_codes, p_scales, device) = _pointers(
        ("src", src, _ACT.get(src_dtype, _UNKNOWN), n_rows * cols), ("codes", codes, _CODES, n_rows * cols),
        ("scales", scales, _F32, n_rows * _blocks(cols)))
    _enqueue(lib().moe_quantize_tiles, device, stream, p_src, src_dtype, n_rows, cols, p_codes, p_scales)


def moe_quantize_blocks(src, src_dtype: int, n_mats: int, rows: int, cols: int, codes, scales, stream=None):
    """e4m3 codes and one power-of-two scale for each 128 x 128 block of the matrices."""
    n = n_mats * rows * cols
    (p_src, p_codes, p_scales, device) = _pointers(
        ("src", src, _ACT.get(src_dtype, _UNKNOWN), n), ("codes", codes, _CODES, n),
        ("scales", scales, _F32, n_mats * _blocks(rows) * _blocks(cols)))
    _enqueue(lib().moe_quantize_blocks, device, stream, p_src, src_dtype, n_mats, rows, cols, p_codes, p_scales)


def moe_block_matmul_workspace_size(n_groups: int, n_cols: int, k: int, max_rows: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_block_matmul_workspace_size(int(n_groups), int(n_cols), int(k), int(max_rows), ctypes.byref(n)))
    return n.value


def moe_block_matmul(n_groups: int, n_cols: int, k: int, max_rows: int, offsets, x, x_scale, w, w_scale, row_scale,
                     out_dtype: int, out, ws, stream=None):
    """Grouped product of block-scaled e4m3 operands (see include/moe.h); offsets
    None with one group takes all max_rows rows."""
    (p_offsets, p_x, p_x_scale, p_w, p_w_scale, p_row_scale, p_out, p_ws, device) = _pointers(
        ("offsets", offsets, _I32S, n_groups + 1), ("x", x, _CODES, max_rows * k),
        ("x_scale", x_scale, _F32, max_rows * _blocks(k)), ("w", w, _CODES, n_groups * n_cols * k),
        ("w_scale", w_scale, _F32, n_groups * _blocks(n_cols) * _blocks(k)),
        ("row_scale", row_scale, _F32, max_rows), ("out", out, _ACT.get(out_dtype, _UNKNOWN), max_rows * n_cols),
        ("ws", ws, _BYTES, 0))
    _enqueue(lib().moe_block_matmul, device, stream, n_groups, n_cols, k, max_rows, p_offsets, p_x, p_x_scale, p_w,
             p_w_scale, p_row_scale, out_dtype, p_out, p_ws, _room(ws))


def moe_block_ffn_workspace_size(n_experts: int, d_model: int, d_ffn: int, max_rows: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_block_ffn_workspace_size(int(n_experts), int(d_model), int(d_ffn), int(max_rows),
                                              ctypes.byref(n)))
    return n.value


def moe_block_ffn(n_experts: int, d_model: int, d_ffn: int, max_rows: int, offsets, x, x_scale, w_gate, s_gate, w_up,
                  s_up, w_down, s_down, row_scale, out_dtype: int, out, ws, stream=None):
    """Grouped SwiGLU experts on block-scaled e4m3 weights (see include/moe.h)."""
    n = n_experts * d_model * d_ffn
    nb = n_experts * _blocks(d_model) * _blocks(d_ffn)
    (p_offsets, p_x, p_x_scale, p_w_gate, p_s_gate, p_w_up, p_s_up, p_w_down, p_s_down, p_row_scale, p_out, p_ws,
     device) = _pointers(
        ("offsets", offsets, _I32S, n_experts + 1), ("x", x, _CODES, max_rows * d_model),
        ("x_scale", x_scale, _F32, max_rows * _blocks(d_model)), ("w_gate", w_gate, _CODES, n),
        ("s_gate", s_gate, _F32, nb), ("w_up", w_up, _CODES, n), ("s_up", s_up, _F32, nb),
        ("w_down", w_down, _CODES, n), ("s_down", s_down, _F32, nb), ("row_scale", row_scale, _F32, max_rows),
        ("out", out, _ACT.get(out_dtype, _UNKNOWN), max_rows * d_model), ("ws", ws, _BYTES, 0))
    _enqueue(lib().moe_block_ffn, device, stream, n_experts, d_model, d_ffn, max_rows, p_offsets, p_x, p_x_scale,
             p_w_gate, p_s_gate, p_w_up, p_s_up, p_w_down, p_s_down, p_row_scale, out_dtype, p_out, p_ws, _room(ws))
