"""ctypes binding of ``libmoe_mi355x.so``: the C entry points under the same
names, taking torch tensors.  Argument marshalling only -- every step of the
layer runs in the library's HIP kernels; there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_HIP = 4
MOE_WFMT_BF16 = 0
MOE_WFMT_Q3G128 = 1
MOE_WFMT_BF16_PAIRS = 2
MOE_WFMT_FP8_B128 = 4

DEFAULT_FAT_THRESHOLD = 32

EXPORTS = ("moe_status_string", "moe_version", "moe_workspace_size", "moe_route_topk", "moe_router_topk",
           "moe_permute", "moe_grouped_ffn", "moe_ffn_plan", "moe_ffn_gate_up", "moe_ffn_down",
           "moe_combine", "moe_grouped_ffn_noalloc", "moe_route_permute_plan", "moe_pack_bf16_pairs",
           "moe_quantize_fp8", "moe_balance_workspace_size", "moe_balance_loss", "moe_route_backward",
           "moe_combine_backward")

NOALLOC_SCRATCH_BYTES = 64 << 20

_lib = None


class MoEError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {lib().moe_status_string(status).decode()} (status {status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load the built library (fails loudly if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(f"{LIB} is missing: build it with `python -m routed_expert_ffn_03_amd.build`")
        L = ctypes.CDLL(LIB)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [i32]
        L.moe_version.restype = ctypes.c_char_p
        L.moe_version.argtypes = []
        L.moe_workspace_size.restype = sz
        L.moe_workspace_size.argtypes = [i32] * 6
        L.moe_route_topk.restype = i32
        L.moe_route_topk.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
        L.moe_router_topk.restype = i32
        L.moe_router_topk.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_permute.restype = i32
        L.moe_permute.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]
        L.moe_grouped_ffn.restype = i32
        L.moe_grouped_ffn.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                      i32, i32, i32, i32, i32, i32, vp, vp, sz, vp]
        L.moe_ffn_plan.restype = i32
        L.moe_ffn_plan.argtypes = [vp, i32, i32, i32, i32, i32, i32, i32, vp, sz, vp]
        L.moe_ffn_gate_up.restype = i32
        L.moe_ffn_gate_up.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, sz, vp]
        L.moe_ffn_down.restype = i32
        L.moe_ffn_down.argtypes = [i32, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, sz, vp]
        L.moe_grouped_ffn_noalloc.restype = i32
        L.moe_grouped_ffn_noalloc.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                              i32, i32, i32, i32, i32, i32, vp, vp]
        L.moe_route_permute_plan.restype = i32
        L.moe_route_permute_plan.argtypes = [vp, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_combine.restype = i32
        L.moe_combine.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
        L.moe_pack_bf16_pairs.restype = i32
        L.moe_pack_bf16_pairs.argtypes = [vp, vp, ctypes.c_int64, i32, i32, i32, vp]
        L.moe_quantize_fp8.restype = i32
        L.moe_quantize_fp8.argtypes = [vp, ctypes.c_int64, i32, i32, i32, vp, vp, vp]
        L.moe_balance_workspace_size.restype = sz
        L.moe_balance_workspace_size.argtypes = [i32] * 3
        L.moe_balance_loss.restype = i32
        L.moe_balance_loss.argtypes = [vp, vp, vp, i32, i32, i32, i32, ctypes.c_float, vp, vp, vp, vp, vp, sz, vp]
        L.moe_route_backward.restype = i32
        L.moe_route_backward.argtypes = [vp] * 8 + [i32] * 4 + [vp, vp]
        L.moe_combine_backward.restype = i32
        L.moe_combine_backward.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, vp]
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the current stream's handle without a Stream object around it, where torch has the call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoEError(status, what)


def _dev(t: torch.Tensor, dtype, name: str):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor on the GPU")


_CODES = (torch.uint8, torch.float8_e4m3fn)


def _current(t, name: str) -> int:
    """The current device's index, once ``t`` is known to be a GPU tensor."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError(f"{name}: expected a tensor on the GPU")
    return torch.cuda.current_device()


def _arg(t, name: str, dtypes, shape, dev: int):
    """The address of a contiguous tensor of one of ``dtypes`` and of ``shape`` on device ``dev``, the current one
    (the launch and the default stream are there)."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor, got {type(t).__name__}")
    raise ValueError(f"{name}: expected a contiguous tensor of {' or '.join(str(d) for d in dtypes)} and shape "
                     f"{tuple(shape)} on the current device (cuda:{dev}), got {t.dtype} {tuple(t.shape)} on {t.device}"
                     + ("" if t.is_contiguous() else ", not contiguous"))


_F32, _I32, _U8, _F16 = (torch.float32,), (torch.int32,), (torch.uint8,), (torch.float16, torch.int16)
_BF16, _MASK = (torch.bfloat16, torch.int16), (torch.uint8, torch.bool)


def _fp8_experts(E, H, I, gate_up=None, down=None, **others):
    """Types and shapes of e4m3 expert weights and their fp32 scales per 128 x 128 block; they and the ``others``
    lie on the current device."""
    if H % 128 or I % 128:
        raise ValueError(f"e4m3 experts: H = {H} and I = {I} must be multiples of 128")
    if gate_up is not None:
        w_gate, w_up, s_gate, s_up = gate_up
        dev = _current(w_gate, "w_gate")
        _arg(w_gate, "w_gate", _CODES, (E, I, H), dev)
        _arg(w_up, "w_up", _CODES, (E, I, H), dev)
        _arg(s_gate, "s_gate", _F32, (E, I // 128, H // 128), dev)
        _arg(s_up, "s_up", _F32, (E, I // 128, H // 128), dev)
    if down is not None:
        w_down, s_down = down
        dev = _current(w_down, "w_down")
        _arg(w_down, "w_down", _CODES, (E, H, I), dev)
        _arg(s_down, "s_down", _F32, (E, H // 128, I // 128), dev)
    for name, t in others.items():
        if t.get_device() != dev:
            raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")


def moe_workspace_size(T: int, E: int, k: int, H: int, I: int, wfmt: int = MOE_WFMT_BF16) -> int:
    return int(lib().moe_workspace_size(T, E, k, H, I, wfmt))


def moe_route_topk(logits, k, topk_ids, topk_w, expert_counts, stream=None):
    _dev(logits, torch.float32, "logits")
    T, E = logits.shape
    for t, dt, n, shp in ((topk_ids, torch.int32, "topk_ids", (T, k)), (topk_w, torch.float32, "topk_w", (T, k)),
                          (expert_counts, torch.int32, "expert_counts", (E,))):
        _dev(t, dt, n)
        if tuple(t.shape) != shp:
            raise ValueError(f"{n}: shape {tuple(t.shape)} != {shp}")
    _check(lib().moe_route_topk(_ptr(logits), T, E, k, _ptr(topk_ids), _ptr(topk_w), _ptr(expert_counts),
                                _stream(stream)), "moe_route_topk")


def moe_router_topk(x, w_router, k, topk_ids, topk_w, expert_counts, logits=None, workspace=None, stream=None):
    """Router GEMM (x [T, H] bf16 bits . w_router [E, H] bf16 bits) fused with the top-k gate;
    ``logits`` (fp32 [T, E]) is written only when given; ``workspace`` (uint8, >= T * E * 4
    bytes) lets a batch of at most 32 tokens spread the GEMM over E / 32 blocks without it."""
    T, H = x.shape
    E = w_router.shape[0]
    if x.dtype not in (torch.int16, torch.bfloat16) or w_router.dtype not in (torch.int16, torch.bfloat16):
        raise ValueError("x and w_router: bf16 bit patterns (int16 or bfloat16 tensors)")
    for t, name in ((x, "x"), (w_router, "w_router")):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError(f"{name}: expected a contiguous tensor on the GPU")
    if w_router.shape[1] != H:
        raise ValueError("w_router must be [E, H]")
    _dev(topk_ids, torch.int32, "topk_ids")
    _dev(topk_w, torch.float32, "topk_w")
    _dev(expert_counts, torch.int32, "expert_counts")
    if logits is not None:
        _dev(logits, torch.float32, "logits")
    ws_bytes = 0
    if workspace is not None:
        _dev(workspace, torch.uint8, "workspace")
        ws_bytes = workspace.numel()
    _check(lib().moe_router_topk(_ptr(x), _ptr(w_router), T, E, H, k, _ptr(topk_ids), _ptr(topk_w),
                                 _ptr(expert_counts), _ptr(logits), _ptr(workspace), ws_bytes, _stream(stream)),
           "moe_router_topk")


def moe_permute(topk_ids, E, expert_offsets, sorted_pair, pair_to_sorted, workspace, stream=None):
    _dev(topk_ids, torch.int32, "topk_ids")
    T, k = topk_ids.shape
    for t, n, shp in ((expert_offsets, "expert_offsets", (E + 1,)), (sorted_pair, "sorted_pair", (T * k,)),
                      (pair_to_sorted, "pair_to_sorted", (T * k,))):
        _dev(t, torch.int32, n)
        if tuple(t.shape) != shp:
            raise ValueError(f"{n}: shape {tuple(t.shape)} != {shp}")
    _dev(workspace, torch.uint8, "workspace")
    _check(lib().moe_permute(_ptr(topk_ids), T, E, k, _ptr(expert_offsets), _ptr(sorted_pair),
                             _ptr(pair_to_sorted), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_permute")


def moe_grouped_ffn(x, w_gate, w_up, w_down, expert_offsets, sorted_pair, k, y_sorted, workspace,
                    s_gate=None, s_up=None, s_down=None, fat_threshold=DEFAULT_FAT_THRESHOLD,
                    wfmt=MOE_WFMT_BF16, stream=None):
    """x, weights and y_sorted hold bf16/fp16 bit patterns (torch.bfloat16 /
    torch.float16 / int16 tensors are all accepted; 3-bit words are int32;
    e4m3 codes are uint8 or float8_e4m3fn with fp32 scales per 128 x 128 block)."""
    T, H = x.shape
    E = expert_offsets.numel() - 1
    I = w_gate.shape[1]          # [E, I, H] bf16 or [E, I, H/128, 13] 3-bit words
    for t, n in ((x, "x"), (y_sorted, "y_sorted"), (w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down"),
                 (expert_offsets, "expert_offsets"), (sorted_pair, "sorted_pair"), (workspace, "workspace")):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError(f"{n}: expected a contiguous GPU tensor")
    if x.element_size() != 2 or y_sorted.element_size() != 2:
        raise ValueError("x and y_sorted must have 16-bit elements")
    if tuple(y_sorted.shape) != (T * k, H):
        raise ValueError(f"y_sorted: shape {tuple(y_sorted.shape)} != {(T * k, H)}")
    if wfmt == MOE_WFMT_FP8_B128:
        _fp8_experts(E, H, I, (w_gate, w_up, s_gate, s_up), (w_down, s_down), x=x, y_sorted=y_sorted,
                     expert_offsets=expert_offsets, sorted_pair=sorted_pair, workspace=workspace)
    _check(lib().moe_grouped_ffn(_ptr(x), wfmt, _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(s_gate),
                                 _ptr(s_up), _ptr(s_down), _ptr(expert_offsets), _ptr(sorted_pair), T, E, k, H, I,
                                 fat_threshold, _ptr(y_sorted), _ptr(workspace), workspace.numel(),
                                 _stream(stream)), "moe_grouped_ffn")


def moe_route_permute_plan(logits, k, H, I, topk_ids, topk_w, expert_counts, expert_offsets, sorted_pair,
                           pair_to_sorted, workspace, fat_threshold=DEFAULT_FAT_THRESHOLD, wfmt=MOE_WFMT_BF16,
                           stream=None):
    """moe_route_topk + moe_permute + moe_ffn_plan (one launch for T <= 64)."""
    _dev(logits, torch.float32, "logits")
    T, E = logits.shape
    for t, dt, n, shp in ((topk_ids, torch.int32, "topk_ids", (T, k)), (topk_w, torch.float32, "topk_w", (T, k)),
                          (expert_counts, torch.int32, "expert_counts", (E,)),
                          (expert_offsets, torch.int32, "expert_offsets", (E + 1,)),
                          (sorted_pair, torch.int32, "sorted_pair", (T * k,)),
                          (pair_to_sorted, torch.int32, "pair_to_sorted", (T * k,))):
        _dev(t, dt, n)
        if tuple(t.shape) != shp:
            raise ValueError(f"{n}: shape {tuple(t.shape)} != {shp}")
    _dev(workspace, torch.uint8, "workspace")
    _check(lib().moe_route_permute_plan(_ptr(logits), T, E, k, H, I, wfmt, fat_threshold, _ptr(topk_ids),
                                        _ptr(topk_w), _ptr(expert_counts), _ptr(expert_offsets), _ptr(sorted_pair),
                                        _ptr(pair_to_sorted), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_route_permute_plan")


def moe_grouped_ffn_noalloc(x, w_gate, w_up, w_down, expert_offsets, sorted_pair, k, y_sorted, s_gate=None,
                            s_up=None, s_down=None, fat_threshold=DEFAULT_FAT_THRESHOLD, wfmt=MOE_WFMT_BF16,
                            stream=None):
    """moe_grouped_ffn with the library's own per-GPU scratch array as its
    workspace (no allocation; calls that overlap on one GPU race)."""
    T, H = x.shape
    E = expert_offsets.numel() - 1
    I = w_gate.shape[1]
    for t, n in ((x, "x"), (y_sorted, "y_sorted"), (w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down"),
                 (expert_offsets, "expert_offsets"), (sorted_pair, "sorted_pair")):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError(f"{n}: expected a contiguous GPU tensor")
    if x.element_size() != 2 or y_sorted.element_size() != 2:
        raise ValueError("x and y_sorted must have 16-bit elements")
    if tuple(y_sorted.shape) != (T * k, H):
        raise ValueError(f"y_sorted: shape {tuple(y_sorted.shape)} != {(T * k, H)}")
    if wfmt == MOE_WFMT_FP8_B128:
        _fp8_experts(E, H, I, (w_gate, w_up, s_gate, s_up), (w_down, s_down), x=x, y_sorted=y_sorted,
                     expert_offsets=expert_offsets, sorted_pair=sorted_pair)
    _check(lib().moe_grouped_ffn_noalloc(_ptr(x), wfmt, _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(s_gate),
                                         _ptr(s_up), _ptr(s_down), _ptr(expert_offsets), _ptr(sorted_pair), T, E,
                                         k, H, I, fat_threshold, _ptr(y_sorted), _stream(stream)),
           "moe_grouped_ffn_noalloc")


def moe_ffn_plan(expert_offsets, T, k, H, I, workspace, fat_threshold=DEFAULT_FAT_THRESHOLD,
                 wfmt=MOE_WFMT_BF16, stream=None):
    E = expert_offsets.numel() - 1
    _dev(expert_offsets, torch.int32, "expert_offsets")
    _dev(workspace, torch.uint8, "workspace")
    _check(lib().moe_ffn_plan(_ptr(expert_offsets), T, E, k, H, I, wfmt, fat_threshold, _ptr(workspace),
                              workspace.numel(), _stream(stream)), "moe_ffn_plan")


def moe_ffn_gate_up(x, w_gate, w_up, sorted_pair, E, k, workspace, s_gate=None, s_up=None,
                    fat_threshold=DEFAULT_FAT_THRESHOLD, wfmt=MOE_WFMT_BF16, stream=None):
    T, H = x.shape
    I = w_gate.shape[1]
    if wfmt == MOE_WFMT_FP8_B128:
        _fp8_experts(E, H, I, gate_up=(w_gate, w_up, s_gate, s_up), x=x, sorted_pair=sorted_pair, workspace=workspace)
    _check(lib().moe_ffn_gate_up(_ptr(x), wfmt, _ptr(w_gate), _ptr(w_up), _ptr(s_gate), _ptr(s_up),
                                 _ptr(sorted_pair), T, E, k, H, I, fat_threshold, _ptr(workspace),
                                 workspace.numel(), _stream(stream)), "moe_ffn_gate_up")


def moe_ffn_down(w_down, T, E, k, I, y_sorted, workspace, s_down=None, fat_threshold=DEFAULT_FAT_THRESHOLD,
                 wfmt=MOE_WFMT_BF16, stream=None):
    H = y_sorted.shape[1]
    if wfmt == MOE_WFMT_FP8_B128:
        _fp8_experts(E, H, I, down=(w_down, s_down), y_sorted=y_sorted, workspace=workspace)
    _check(lib().moe_ffn_down(wfmt, _ptr(w_down), _ptr(s_down), T, E, k, H, I, fat_threshold, _ptr(y_sorted),
                              _ptr(workspace), workspace.numel(), _stream(stream)), "moe_ffn_down")


def moe_combine(y_sorted, topk_w, pair_to_sorted, out, stream=None):
    T, k = topk_w.shape
    H = out.shape[1]
    _dev(topk_w, torch.float32, "topk_w")
    _dev(pair_to_sorted, torch.int32, "pair_to_sorted")
    _dev(out, torch.float32, "out")
    if not (y_sorted.is_cuda and y_sorted.is_contiguous() and y_sorted.element_size() == 2):
        raise ValueError("y_sorted: expected a contiguous 16-bit GPU tensor")
    _check(lib().moe_combine(_ptr(y_sorted), _ptr(topk_w), _ptr(pair_to_sorted), T, k, H, _ptr(out),
                             _stream(stream)), "moe_combine")


def moe_pack_bf16_pairs(src, dst, to_fp16=False, stream=None):
    """Copy bf16 matrices ``src`` [..., rows, cols] into ``dst`` (same shape) in the row-pair layout
    that ``MOE_WFMT_BF16_PAIRS`` reads: rows 2p and 2p+1 alternate every 32 columns; with
    ``to_fp16`` the values are converted to fp16 toward zero (that format's W_down)."""
    for t, name in ((src, "src"), (dst, "dst")):
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous() and t.element_size() == 2):
            raise ValueError(f"{name}: expected a contiguous 16-bit GPU tensor")
    if src.dim() < 2 or tuple(src.shape) != tuple(dst.shape):
        raise ValueError(f"src {tuple(src.shape)} and dst {tuple(dst.shape)}: same shape [..., rows, cols] expected")
    rows, cols = int(src.shape[-2]), int(src.shape[-1])
    mats = src.numel() // (rows * cols) if rows * cols else 0
    _check(lib().moe_pack_bf16_pairs(_ptr(src), _ptr(dst), mats, rows, cols, int(bool(to_fp16)), _stream(stream)),
           "moe_pack_bf16_pairs")


def moe_quantize_fp8(src, codes, scales, block_rows=1, stream=None):
    """e4m3 ``codes`` (uint8 or float8_e4m3fn, the shape of ``src``) and fp32 ``scales``
    [..., rows / block_rows, cols / 128] of bf16 ``src`` [..., rows, cols]; ``block_rows`` 1 for
    activations, 128 for the weights of ``MOE_WFMT_FP8_B128``."""
    dev = _current(src, "src")
    shape = src.shape
    n = src.numel()
    if len(shape) < 2 or n == 0:
        raise ValueError(f"src: shape {tuple(shape)}: [..., rows, cols] with at least one value expected")
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows {block_rows}: 1 or 128")
    rows, cols = shape[-2], shape[-1]
    if cols % 128 or rows % block_rows:
        raise ValueError(f"src: {rows} x {cols} is not a whole number of {block_rows} x 128 blocks")
    _check(lib().moe_quantize_fp8(
        _arg(src, "src", _BF16, shape, dev), n // (rows * cols), rows, cols, block_rows,
        _arg(codes, "codes", _CODES, shape, dev),
        _arg(scales, "scales", _F32, (*shape[:-2], rows // block_rows, cols // 128), dev),
        _stream(stream)), "moe_quantize_fp8")


def moe_balance_workspace_size(T: int, E: int, groups: int = 1) -> int:
    return int(lib().moe_balance_workspace_size(T, E, groups))


def _matrix(t, name: str):
    """(rows, columns) of a two-dimensional tensor."""
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a matrix, got shape {tuple(t.shape)}")
    return t.shape


def moe_balance_loss(logits, topk_ids, expert_counts, prob_mean, group_scale, loss, workspace, token_mask=None,
                     coef=1.0, stream=None):
    """The balance loss and per-expert counts of ``logits`` [T, E] routed to ``topk_ids`` [T, k];
    ``expert_counts`` (int32) and ``prob_mean`` [G, E] fix the number of groups G, ``group_scale``
    [G] goes to ``moe_route_backward``; ``loss`` [1]; masked tokens (0) are not counted."""
    dev = _current(logits, "logits")
    T, E = _matrix(logits, "logits")
    k = _matrix(topk_ids, "topk_ids")[1]
    G = _matrix(expert_counts, "expert_counts")[0]
    _check(lib().moe_balance_loss(
        _arg(logits, "logits", _F32, (T, E), dev), _arg(topk_ids, "topk_ids", _I32, (T, k), dev),
        None if token_mask is None else _arg(token_mask, "token_mask", _MASK, (T,), dev), T, E, k, G, coef,
        _arg(expert_counts, "expert_counts", _I32, (G, E), dev), _arg(prob_mean, "prob_mean", _F32, (G, E), dev),
        _arg(group_scale, "group_scale", _F32, (G,), dev), _arg(loss, "loss", _F32, (1,), dev),
        _arg(workspace, "workspace", _U8, workspace.shape, dev), workspace.numel(), _stream(stream)),
        "moe_balance_loss")


def moe_route_backward(logits, topk_ids, topk_w, d_logits, d_topk_w=None, expert_counts=None, group_scale=None,
                       d_loss=None, token_mask=None, stream=None):
    """``d_logits`` [T, E] of the gate weights (``d_topk_w`` [T, k], or none) and of the balance loss
    (``expert_counts`` [G, E] and ``group_scale`` [G] from ``moe_balance_loss``, ``d_loss`` [1]; or none
    of the three)."""
    dev = _current(d_logits, "d_logits")
    T, E = _matrix(d_logits, "d_logits")
    k = _matrix(topk_ids, "topk_ids")[1]
    G = 1 if expert_counts is None else _matrix(expert_counts, "expert_counts")[0]
    _check(lib().moe_route_backward(
        _arg(logits, "logits", _F32, (T, E), dev), _arg(topk_ids, "topk_ids", _I32, (T, k), dev),
        _arg(topk_w, "topk_w", _F32, (T, k), dev),
        None if d_topk_w is None else _arg(d_topk_w, "d_topk_w", _F32, (T, k), dev),
        None if expert_counts is None else _arg(expert_counts, "expert_counts", _I32, (G, E), dev),
        None if group_scale is None else _arg(group_scale, "group_scale", _F32, (G,), dev),
        None if d_loss is None else _arg(d_loss, "d_loss", _F32, (1,), dev),
        None if token_mask is None else _arg(token_mask, "token_mask", _MASK, (T,), dev), T, E, k, G,
        _arg(d_logits, "d_logits", _F32, (T, E), dev), _stream(stream)), "moe_route_backward")


def moe_combine_backward(d_out, y_sorted, topk_w, pair_to_sorted, d_y_sorted=None, d_topk_w=None, stream=None):
    """Gradient of ``moe_combine``: ``d_y_sorted`` (fp16, the shape of ``y_sorted``) and ``d_topk_w``
    (fp32 [T, k]), either may be None."""
    dev = _current(d_out, "d_out")
    T, H = _matrix(d_out, "d_out")
    k = _matrix(topk_w, "topk_w")[1]
    _check(lib().moe_combine_backward(
        _arg(d_out, "d_out", _F32, (T, H), dev),
        None if y_sorted is None else _arg(y_sorted, "y_sorted", _F16, (T * k, H), dev),
        _arg(topk_w, "topk_w", _F32, (T, k), dev), _arg(pair_to_sorted, "pair_to_sorted", _I32, (T * k,), dev), T, k, H,
        None if d_y_sorted is None else _arg(d_y_sorted, "d_y_sorted", _F16, (T * k, H), dev),
        None if d_topk_w is None else _arg(d_topk_w, "d_topk_w", _F32, (T, k), dev), _stream(stream)),
        "moe_combine_backward")
