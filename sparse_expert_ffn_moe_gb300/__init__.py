"""Python binding of libmoe, the GB300 (sm_103a) sparse MoE FFN layer forward.

Argument marshalling only: every step of the layer runs in the CUDA kernels of
libmoe.so (built from csrc/ by ``_build.build``).  The functions have the names
and argument order of the C ABI in include/moe.h; tensors are torch CUDA
tensors (or None for a NULL pointer), ``stream`` defaults to torch's current
stream.  A non-OK status raises MoeError.  There is no CPU path: importing the
binding without the built library raises ImportError.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE = 0, 1, 2, 3
MOE_ERR_CUDA, MOE_ERR_TIMEOUT, MOE_ERR_BOUNDS = 4, 5, 6
MOE_F32, MOE_BF16 = 0, 1
MOE_ROUTER_SOFTMAX, MOE_ROUTER_SIGMOID = 0, 1

EXPORTED = ("moe_status_string", "moe_workspace_bytes", "moe_route", "moe_permute",
            "moe_permute_noalloc", "moe_expert_ffn", "moe_combine", "moe_forward",
            "moe_quantize_fp8_rows", "moe_expert_ffn_fp8", "moe_forward_fp8",
            "moe_quantize_fp8_blocks", "moe_expert_ffn_fp8_blocks", "moe_forward_fp8_blocks",
            "moe_expert_ffn_w8a8", "moe_forward_w8a8", "moe_expert_ffn_w8a8_blocks",
            "moe_forward_w8a8_blocks", "moe_forward_w8a8_codes", "moe_forward_w8a8_blocks_codes",
            "moe_balance_workspace_bytes", "moe_balance_loss",
            "moe_route_backward", "moe_dropout", "moe_combine_dropout", "moe_combine_backward",
            "moe_few_workspace_bytes", "moe_forward_few", "moe_forward_few_fp8",
            "moe_forward_few_fp8_blocks",
            "moe_rmsnorm", "moe_rmsnorm_workspace_bytes", "moe_rmsnorm_backward",
            "moe_get_device_error")
FP8_BLOCK = 128  # side of the square weight-scale blocks of the *_fp8_blocks calls


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class moe_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("inter_shared", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("router", ctypes.c_int32)]


class moe_fp8_experts(ctypes.Structure):
    """E4M3 expert weight codes (uint8) and fp32 scales (per row, or per 128 x 128
    block for the *_fp8_blocks calls): device pointers."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down",
        "ws_gate", "ws_up", "ws_down", "ss_gate", "ss_up", "ss_down")]


def _load_lib() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libmoe.so is not built ({LIB_PATH}); run sparse_expert_ffn_moe_gb300._build.build() "
            "-- there is no CPU fallback")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    sp = ctypes.POINTER(moe_shape)
    lib.moe_status_string.argtypes = [i32]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_workspace_bytes.argtypes = [sp]
    lib.moe_workspace_bytes.restype = sz
    lib.moe_route.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_permute.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_permute_noalloc.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_expert_ffn.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_combine.argtypes = [sp, vp, vp, vp, vp, vp, vp]
    lib.moe_forward.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    fp = ctypes.POINTER(moe_fp8_experts)
    lib.moe_quantize_fp8_rows.argtypes = [ctypes.c_int64, ctypes.c_int64, i32, vp, vp, vp, vp]
    lib.moe_expert_ffn_fp8.argtypes = [sp, vp, vp, fp, vp, vp, sz, vp]
    lib.moe_forward_fp8.argtypes = [sp, vp, vp, vp, fp, vp, vp, sz, vp]
    lib.moe_quantize_fp8_blocks.argtypes = lib.moe_quantize_fp8_rows.argtypes
    lib.moe_expert_ffn_fp8_blocks.argtypes = lib.moe_expert_ffn_fp8.argtypes
    lib.moe_forward_fp8_blocks.argtypes = lib.moe_forward_fp8.argtypes
    lib.moe_expert_ffn_w8a8.argtypes = [sp, vp, vp, fp, vp, vp, sz, vp]
    lib.moe_forward_w8a8.argtypes = [sp, vp, vp, vp, fp, vp, vp, sz, vp]
    lib.moe_expert_ffn_w8a8_blocks.argtypes = lib.moe_expert_ffn_w8a8.argtypes
    lib.moe_forward_w8a8_blocks.argtypes = lib.moe_forward_w8a8.argtypes
    lib.moe_forward_w8a8_codes.argtypes = [sp, vp, vp, vp, vp, vp, fp, vp, vp, sz, vp]
    lib.moe_forward_w8a8_blocks_codes.argtypes = lib.moe_forward_w8a8_codes.argtypes
    f64, f32 = ctypes.c_double, ctypes.c_float
    lib.moe_balance_workspace_bytes.argtypes = [sp, i32]
    lib.moe_balance_workspace_bytes.restype = sz
    lib.moe_balance_loss.argtypes = [sp, vp, vp, vp, vp, i32, f32, vp, vp, vp, vp, sz, vp]
    lib.moe_route_backward.argtypes = [sp, vp, vp, vp, vp, vp, i32, f32, vp, vp, vp, vp]
    lib.moe_dropout.argtypes = [ctypes.c_int64, i32, vp, vp, f64, vp, vp, vp]
    lib.moe_combine_dropout.argtypes = [sp, vp, vp, vp, vp, vp, f64, vp, vp, vp]
    lib.moe_combine_backward.argtypes = [sp, vp, vp, vp, vp, f64, vp, vp, vp, vp, vp]
    lib.moe_few_workspace_bytes.argtypes = [sp]
    lib.moe_few_workspace_bytes.restype = sz
    lib.moe_forward_few.argtypes = [sp] + [vp] * 12 + [sz, vp]
    lib.moe_forward_few_fp8.argtypes = [sp, vp, vp, vp, fp, vp, vp, vp, sz, vp]
    lib.moe_forward_few_fp8_blocks.argtypes = lib.moe_forward_few_fp8.argtypes
    i64 = ctypes.c_int64
    lib.moe_rmsnorm.argtypes = [i64, i64, i32, vp, vp, vp, f32, vp, vp, vp, vp, vp]
    lib.moe_rmsnorm_workspace_bytes.argtypes = [i64, i64]
    lib.moe_rmsnorm_workspace_bytes.restype = sz
    lib.moe_rmsnorm_backward.argtypes = [i64, i64, i32, vp, vp, vp, f32, vp, vp, vp, vp, sz, vp]
    lib.moe_get_device_error.argtypes = [vp, ctypes.POINTER(i32)]
    for f in ("moe_route", "moe_permute", "moe_permute_noalloc", "moe_expert_ffn", "moe_combine",
              "moe_forward", "moe_quantize_fp8_rows", "moe_expert_ffn_fp8", "moe_forward_fp8",
              "moe_quantize_fp8_blocks", "moe_expert_ffn_fp8_blocks", "moe_forward_fp8_blocks",
              "moe_expert_ffn_w8a8", "moe_forward_w8a8", "moe_expert_ffn_w8a8_blocks",
              "moe_forward_w8a8_blocks", "moe_forward_w8a8_codes", "moe_forward_w8a8_blocks_codes",
              "moe_balance_loss", "moe_route_backward", "moe_dropout",
              "moe_combine_dropout", "moe_combine_backward", "moe_forward_few",
              "moe_forward_few_fp8", "moe_forward_few_fp8_blocks", "moe_rmsnorm", "moe_rmsnorm_backward",
              "moe_get_device_error"):
        getattr(lib, f).restype = i32
    return lib


_lib = _load_lib()


def library() -> ctypes.CDLL:
    return _lib


def status_string(status: int) -> str:
    return _lib.moe_status_string(int(status)).decode()


def make_shape(T: int, d: int, E: int, K: int, inter: int, inter_shared: int = 0,
               dtype: str | int = "bf16", router: str | int = "softmax") -> moe_shape:
    if isinstance(dtype, str):
        dtype = {"bf16": MOE_BF16, "f32": MOE_F32}[dtype]
    if isinstance(router, str):
        router = {"softmax": MOE_ROUTER_SOFTMAX, "sigmoid": MOE_ROUTER_SIGMOID}[router]
    return moe_shape(T, d, E, K, inter, inter_shared, dtype, router)


def _p(t):
    """Device pointer of a tensor (None -> NULL).  Host tensors are refused."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("libmoe takes device tensors only")
    return t.data_ptr()


# the current stream's handle without a Stream object (2.9 us -> 0.3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where)


def _ws(workspace):
    if workspace is None:
        return None, 0
    return _p(workspace), workspace.numel() * workspace.element_size()


def moe_workspace_bytes(shape: moe_shape) -> int:
    return int(_lib.moe_workspace_bytes(ctypes.byref(shape)))


def alloc_workspace(shape: moe_shape, device=None) -> torch.Tensor:
    n = moe_workspace_bytes(shape)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def moe_route(shape, x, w_g, bias, logits_in, logits_out, topk_idx, topk_w, workspace,
              stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_route(ctypes.byref(shape), _p(x), _p(w_g), _p(bias), _p(logits_in),
                          _p(logits_out), _p(topk_idx), _p(topk_w), ws, nws, _stream(stream)),
           "moe_route")


def moe_permute(shape, topk_idx, x, counts, offsets, perm, inv_perm, x_perm, workspace,
                stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_permute(ctypes.byref(shape), _p(topk_idx), _p(x), _p(counts), _p(offsets),
                            _p(perm), _p(inv_perm), _p(x_perm), ws, nws, _stream(stream)),
           "moe_permute")


def moe_permute_noalloc(shape, topk_idx, x, counts, offsets, perm, inv_perm, x_perm,
                        stream=None):
    """moe_permute without a workspace: its scratch is a fixed array inside the
    library, for callers that cannot allocate device memory."""
    _check(_lib.moe_permute_noalloc(ctypes.byref(shape), _p(topk_idx), _p(x), _p(counts),
                                    _p(offsets), _p(perm), _p(inv_perm), _p(x_perm),
                                    _stream(stream)), "moe_permute_noalloc")


def moe_expert_ffn(shape, x_perm, offsets, w_gate, w_up, w_down, y_perm, workspace, stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_expert_ffn(ctypes.byref(shape), _p(x_perm), _p(offsets), _p(w_gate),
                               _p(w_up), _p(w_down), _p(y_perm), ws, nws, _stream(stream)),
           "moe_expert_ffn")


def moe_combine(shape, y_perm, inv_perm, topk_w, y_shared, y, stream=None):
    _check(_lib.moe_combine(ctypes.byref(shape), _p(y_perm), _p(inv_perm), _p(topk_w),
                            _p(y_shared), _p(y), _stream(stream)), "moe_combine")


def moe_forward(shape, x, w_g, bias, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, y,
                workspace, stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_forward(ctypes.byref(shape), _p(x), _p(w_g), _p(bias), _p(w_gate), _p(w_up),
                            _p(w_down), _p(ws_gate), _p(ws_up), _p(ws_down), _p(y), ws, nws,
                            _stream(stream)), "moe_forward")


def moe_quantize_fp8_rows(w, codes, scales, stream=None):
    """Per-row E4M3 quantisation of the last dimension of w (bf16 or fp32):
    codes (uint8, w's shape) and scales (fp32, w's leading shape)."""
    dtype = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}[w.dtype]
    cols = w.shape[-1]
    rows = w.numel() // cols if cols else 0
    _check(_lib.moe_quantize_fp8_rows(rows, cols, dtype, _p(w), _p(codes), _p(scales),
                                      _stream(stream)), "moe_quantize_fp8_rows")


def moe_quantize_fp8_blocks(w, codes, scales, stream=None):
    """Block-scaled E4M3 quantisation of w (bf16 or fp32) taken as one stacked
    [rows][cols] matrix (rows = the product of the leading sizes): codes (uint8,
    w's shape) and scales (fp32, [ceil(rows/128)][ceil(cols/128)])."""
    dtype = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}[w.dtype]
    cols = w.shape[-1]
    rows = w.numel() // cols if cols else 0
    _check(_lib.moe_quantize_fp8_blocks(rows, cols, dtype, _p(w), _p(codes), _p(scales),
                                        _stream(stream)), "moe_quantize_fp8_blocks")


def make_fp8_experts(q: dict) -> moe_fp8_experts:
    """A moe_fp8_experts from a dict of device tensors (w_gate, w_up, w_down codes,
    s_gate, s_up, s_down scales; ws_* / ss_* for the shared expert, optional).
    The caller keeps the tensors alive while the struct is in use."""
    return moe_fp8_experts(*[_p(q.get(n)) for n, _ in moe_fp8_experts._fields_])


def moe_expert_ffn_fp8(shape, x_perm, offsets, w: moe_fp8_experts, y_perm, workspace,
                       stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_expert_ffn_fp8(ctypes.byref(shape), _p(x_perm), _p(offsets), ctypes.byref(w),
                                   _p(y_perm), ws, nws, _stream(stream)), "moe_expert_ffn_fp8")


def moe_forward_fp8(shape, x, w_g, bias, w: moe_fp8_experts, y, workspace, stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_forward_fp8(ctypes.byref(shape), _p(x), _p(w_g), _p(bias), ctypes.byref(w),
                                _p(y), ws, nws, _stream(stream)), "moe_forward_fp8")


def moe_expert_ffn_fp8_blocks(shape, x_perm, offsets, w: moe_fp8_experts, y_perm, workspace,
                              stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_expert_ffn_fp8_blocks(ctypes.byref(shape), _p(x_perm), _p(offsets),
                                          ctypes.byref(w), _p(y_perm), ws, nws, _stream(stream)),
           "moe_expert_ffn_fp8_blocks")


def moe_forward_fp8_blocks(shape, x, w_g, bias, w: moe_fp8_experts, y, workspace, stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_forward_fp8_blocks(ctypes.byref(shape), _p(x), _p(w_g), _p(bias),
                                       ctypes.byref(w), _p(y), ws, nws, _stream(stream)),
           "moe_forward_fp8_blocks")


def moe_expert_ffn_w8a8(shape, x_perm, offsets, w: moe_fp8_experts, y_perm, workspace,
                        stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_expert_ffn_w8a8(ctypes.byref(shape), _p(x_perm), _p(offsets),
                                    ctypes.byref(w), _p(y_perm), ws, nws, _stream(stream)),
           "moe_expert_ffn_w8a8")


def moe_forward_w8a8(shape, x, w_g, bias, w: moe_fp8_experts, y, workspace, stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_forward_w8a8(ctypes.byref(shape), _p(x), _p(w_g), _p(bias), ctypes.byref(w),
                                 _p(y), ws, nws, _stream(stream)), "moe_forward_w8a8")


def moe_expert_ffn_w8a8_blocks(shape, x_perm, offsets, w: moe_fp8_experts, y_perm, workspace,
                               stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_expert_ffn_w8a8_blocks(ctypes.byref(shape), _p(x_perm), _p(offsets),
                                           ctypes.byref(w), _p(y_perm), ws, nws, _stream(stream)),
           "moe_expert_ffn_w8a8_blocks")


def moe_forward_w8a8_blocks(shape, x, w_g, bias, w: moe_fp8_experts, y, workspace, stream=None):
    ws, nws = _ws(workspace)
    _check(_lib.moe_forward_w8a8_blocks(ctypes.byref(shape), _p(x), _p(w_g), _p(bias),
                                        ctypes.byref(w), _p(y), ws, nws, _stream(stream)),
           "moe_forward_w8a8_blocks")


def _arg(t, name: str, dtype, n: int, optional: bool = False):
    """Device pointer of a contiguous tensor of n elements of `dtype`."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is missing")
    if t.is_cuda and t.dtype == dtype and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError("libmoe takes device tensors only")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, not {t.numel()}")
    raise ValueError(f"{name} must be contiguous")


def _row_dtype(shape: moe_shape):
    return torch.bfloat16 if shape.dtype == MOE_BF16 else torch.float32


def _seqs(seq_offsets):
    """(pointer, number of sequences) of seq_offsets, an int32 [n_seq + 1] tensor or None."""
    if seq_offsets is None:
        return None, 1
    n = seq_offsets.numel()
    return _arg(seq_offsets, "seq_offsets", torch.int32, n), n - 1


def _mask(token_mask, T):
    """token_mask: a byte a token, or truth values (torch.bool, the same bytes); or None."""
    truth = token_mask is not None and token_mask.dtype == torch.bool
    return _arg(token_mask, "token_mask", torch.bool if truth else torch.uint8, T, True)


def _rng(rng):
    """rng {seed, offset}: an int64 (or uint64) device tensor; None where nothing is drawn."""
    if rng is None:
        return None
    return _arg(rng, "rng", torch.uint64 if rng.dtype == torch.uint64 else torch.int64, 2)


def _w8a8_codes(call, name, s, x, x_codes, x_scales, w_g, bias, w, y, workspace, stream):
    bf = torch.bfloat16
    ws, nws = _ws(workspace)
    _check(call(ctypes.byref(s), _arg(x, "x", bf, s.T * s.d),
                _arg(x_codes, "x_codes", torch.uint8, s.T * s.d),
                _arg(x_scales, "x_scales", torch.float32, s.T), _arg(w_g, "w_g", bf, s.E * s.d),
                _arg(bias, "bias", torch.float32, s.E, True), ctypes.byref(w),
                _arg(y, "y", bf, s.T * s.d), ws, nws, _stream(stream)), name)


def moe_forward_w8a8_codes(shape, x, x_codes, x_scales, w_g, bias, w: moe_fp8_experts, y, workspace,
                           stream=None):
    """moe_forward_w8a8 on rows that are in 8 bits already (codes uint8 [T][d], scales [T]);
    x (bf16) is the router's."""
    _w8a8_codes(_lib.moe_forward_w8a8_codes, "moe_forward_w8a8_codes", shape, x, x_codes, x_scales,
                w_g, bias, w, y, workspace, stream)


def moe_forward_w8a8_blocks_codes(shape, x, x_codes, x_scales, w_g, bias, w: moe_fp8_experts, y,
                                  workspace, stream=None):
    """moe_forward_w8a8_blocks on rows that are in 8 bits already."""
    _w8a8_codes(_lib.moe_forward_w8a8_blocks_codes, "moe_forward_w8a8_blocks_codes", shape, x,
                x_codes, x_scales, w_g, bias, w, y, workspace, stream)


def moe_balance_workspace_bytes(shape: moe_shape, n_seq: int = 1) -> int:
    return int(_lib.moe_balance_workspace_bytes(ctypes.byref(shape), n_seq))


def alloc_balance_workspace(shape: moe_shape, n_seq: int = 1, device=None) -> torch.Tensor:
    n = moe_balance_workspace_bytes(shape, n_seq)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_balance_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def moe_balance_loss(shape, logits, topk_idx, token_mask, seq_offsets, alpha, counts, mean_probs,
                     loss, workspace, stream=None):
    """Balance loss [1] (fp32), per-expert counts [n_seq][E] (int32) and mean
    probabilities [n_seq][E] (fp32) of the router's logits [T][E] and picks [T][K]."""
    T, E, K = shape.T, shape.E, shape.K
    seqs, n = _seqs(seq_offsets)
    ws, nws = _ws(workspace)
    _check(_lib.moe_balance_loss(
        ctypes.byref(shape), _arg(logits, "logits", torch.float32, T * E),
        _arg(topk_idx, "topk_idx", torch.int32, T * K),
        _mask(token_mask, T), seqs, n, alpha,
        _arg(counts, "counts", torch.int32, n * E),
        _arg(mean_probs, "mean_probs", torch.float32, n * E),
        _arg(loss, "loss", torch.float32, 1), ws, nws, _stream(stream)), "moe_balance_loss")


def moe_route_backward(shape, logits, topk_idx, d_topk_w, token_mask, seq_offsets, alpha, counts,
                       d_loss, d_logits, stream=None):
    """Gradient of the logits: the routing weights' (d_topk_w, or None) and the
    balance loss's (counts as moe_balance_loss wrote them, or None) together."""
    T, E, K = shape.T, shape.E, shape.K
    seqs, n = _seqs(seq_offsets)
    _check(_lib.moe_route_backward(
        ctypes.byref(shape), _arg(logits, "logits", torch.float32, T * E),
        _arg(topk_idx, "topk_idx", torch.int32, T * K, True),
        _arg(d_topk_w, "d_topk_w", torch.float32, T * K, True),
        _mask(token_mask, T), seqs, n, alpha,
        _arg(counts, "counts", torch.int32, n * E, True),
        _arg(d_loss, "d_loss", torch.float32, 1, True),
        _arg(d_logits, "d_logits", torch.float32, T * E), _stream(stream)), "moe_route_backward")


def moe_dropout(x, residual, p, rng, y, stream=None):
    """y = residual + dropout(x), x of any shape (bf16 or fp32); rng an int64
    device tensor {seed, offset}.  The same call on the output's gradient, with
    the same rng and no residual, gives x's gradient."""
    dtype = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}.get(x.dtype)
    if dtype is None:
        raise ValueError(f"x must be torch.bfloat16 or torch.float32, not {x.dtype}")
    n = x.numel()
    _check(_lib.moe_dropout(n, dtype, _arg(x, "x", x.dtype, n),
                            _arg(residual, "residual", x.dtype, n, True), p, _rng(rng),
                            _arg(y, "y", x.dtype, n), _stream(stream)), "moe_dropout")


def moe_combine_dropout(shape, y_perm, inv_perm, topk_w, y_shared, residual, p, rng, y,
                        stream=None):
    """moe_combine with dropout on its sum and the residual added."""
    dt, n, row = _row_dtype(shape), shape.T * shape.K, shape.T * shape.d
    _check(_lib.moe_combine_dropout(
        ctypes.byref(shape), _arg(y_perm, "y_perm", dt, n * shape.d),
        _arg(inv_perm, "inv_perm", torch.int32, n), _arg(topk_w, "topk_w", torch.float32, n),
        _arg(y_shared, "y_shared", dt, row, True), _arg(residual, "residual", dt, row, True), p,
        _rng(rng), _arg(y, "y", dt, row), _stream(stream)), "moe_combine_dropout")


def moe_combine_backward(shape, d_y, y_perm, inv_perm, topk_w, p, rng, d_y_perm, d_topk_w,
                         d_shared, stream=None):
    """Gradients of moe_combine_dropout from d_y: of the expert rows (d_y_perm), the
    routing weights (d_topk_w, fp32) and the shared expert's rows (d_shared), each or None."""
    dt, n, row = _row_dtype(shape), shape.T * shape.K, shape.T * shape.d
    _check(_lib.moe_combine_backward(
        ctypes.byref(shape), _arg(d_y, "d_y", dt, row),
        _arg(y_perm, "y_perm", dt, n * shape.d, True), _arg(inv_perm, "inv_perm", torch.int32, n),
        _arg(topk_w, "topk_w", torch.float32, n, True), p, _rng(rng),
        _arg(d_y_perm, "d_y_perm", dt, n * shape.d, True),
        _arg(d_topk_w, "d_topk_w", torch.float32, n, True),
        _arg(d_shared, "d_shared", dt, row, True), _stream(stream)), "moe_combine_backward")


def moe_few_workspace_bytes(shape: moe_shape) -> int:
    return int(_lib.moe_few_workspace_bytes(ctypes.byref(shape)))


def alloc_few_workspace(shape: moe_shape, device=None) -> torch.Tensor:
    n = moe_few_workspace_bytes(shape)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_few_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def moe_forward_few(shape, x, w_g, bias, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, residual,
                    y, workspace, stream=None):
    """moe_forward for at most 16 tokens in two launches, y = residual + layer(x) (residual or
    None); bf16 weights, workspace from alloc_few_workspace."""
    s, bf = shape, torch.bfloat16
    ws, nws = _ws(workspace)
    one, sh = s.E * s.inter * s.d, s.inter_shared * s.d
    _check(_lib.moe_forward_few(
        ctypes.byref(s), _arg(x, "x", bf, s.T * s.d), _arg(w_g, "w_g", bf, s.E * s.d),
        _arg(bias, "bias", torch.float32, s.E, True), _arg(w_gate, "w_gate", bf, one),
        _arg(w_up, "w_up", bf, one), _arg(w_down, "w_down", bf, one),
        _arg(ws_gate, "ws_gate", bf, sh, True), _arg(ws_up, "ws_up", bf, sh, True),
        _arg(ws_down, "ws_down", bf, sh, True), _arg(residual, "residual", bf, s.T * s.d, True),
        _arg(y, "y", bf, s.T * s.d), ws, nws, _stream(stream)), "moe_forward_few")


def _few_fp8(call, name, s, x, w_g, bias, w, residual, y, workspace, stream):
    bf = torch.bfloat16
    ws, nws = _ws(workspace)
    _check(call(ctypes.byref(s), _arg(x, "x", bf, s.T * s.d), _arg(w_g, "w_g", bf, s.E * s.d),
                _arg(bias, "bias", torch.float32, s.E, True), ctypes.byref(w),
                _arg(residual, "residual", bf, s.T * s.d, True), _arg(y, "y", bf, s.T * s.d), ws,
                nws, _stream(stream)), name)


def moe_forward_few_fp8(shape, x, w_g, bias, w: moe_fp8_experts, residual, y, workspace,
                        stream=None):
    """moe_forward_fp8 for at most 16 tokens in two launches, y = residual + layer(x)."""
    _few_fp8(_lib.moe_forward_few_fp8, "moe_forward_few_fp8", shape, x, w_g, bias, w, residual, y,
             workspace, stream)


def moe_forward_few_fp8_blocks(shape, x, w_g, bias, w: moe_fp8_experts, residual, y, workspace,
                               stream=None):
    """moe_forward_fp8_blocks for at most 16 tokens in two launches, y = residual + layer(x)."""
    _few_fp8(_lib.moe_forward_few_fp8_blocks, "moe_forward_few_fp8_blocks", shape, x, w_g, bias, w,
             residual, y, workspace, stream)


_ROW_DTYPES = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}


def _norm_dtype(x, name: str):
    dtype = _ROW_DTYPES.get(x.dtype)
    if dtype is None:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, not {x.dtype}")
    return dtype


def moe_rmsnorm(x, residual, weight, eps, s, y, codes, scales, stream=None):
    """RMS norm of the rows of x (bf16 or fp32, the last dimension) after the residual's
    addition: the sum s, the normalised rows y, and y as E4M3 codes (uint8, x's shape)
    with a scale a row (fp32); residual, s, y and (codes, scales) may each be None."""
    dtype = _norm_dtype(x, "x")
    t, n, cols = x.dtype, x.numel(), x.shape[-1]
    rows = n // cols if cols else 0
    _check(_lib.moe_rmsnorm(
        rows, cols, dtype, _arg(x, "x", t, n), _arg(residual, "residual", t, n, True),
        _arg(weight, "weight", t, cols), eps, _arg(s, "s", t, n, True), _arg(y, "y", t, n, True),
        _arg(codes, "codes", torch.uint8, n, True),
        _arg(scales, "scales", torch.float32, rows, True), _stream(stream)), "moe_rmsnorm")


def moe_rmsnorm_workspace_bytes(rows: int, cols: int) -> int:
    return int(_lib.moe_rmsnorm_workspace_bytes(rows, cols))


def alloc_rmsnorm_workspace(rows: int, cols: int, device=None) -> torch.Tensor:
    n = moe_rmsnorm_workspace_bytes(rows, cols)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_rmsnorm_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def moe_rmsnorm_backward(d_y, s, weight, eps, d_s, d_x, d_weight, workspace, stream=None):
    """Gradients of moe_rmsnorm from y's gradient d_y, on the rows s that it normalised:
    d_x (with d_s, the residual stream's own gradient, added; or None) and d_weight
    (fp32, or None; it alone needs the workspace)."""
    dtype = _norm_dtype(s, "s")
    t, n, cols = s.dtype, s.numel(), s.shape[-1]
    rows = n // cols if cols else 0
    ws, nws = _ws(workspace)
    _check(_lib.moe_rmsnorm_backward(
        rows, cols, dtype, _arg(d_y, "d_y", t, n), _arg(s, "s", t, n),
        _arg(weight, "weight", t, cols), eps, _arg(d_s, "d_s", t, n, True),
        _arg(d_x, "d_x", t, n, True), _arg(d_weight, "d_weight", torch.float32, cols, True),
        ws, nws, _stream(stream)), "moe_rmsnorm_backward")


def moe_get_device_error(workspace) -> int:
    code = ctypes.c_int32(0)
    _check(_lib.moe_get_device_error(_p(workspace), ctypes.byref(code)), "moe_get_device_error")
    return int(code.value)
