"""MI355X (gfx950) fused Mixture-of-Experts layer.

Thin ctypes binding over libmoe_mi355x.so, the C ABI in include/moe.h.  The
functions here only check tensor shapes/dtypes/devices and marshal pointers;
every step of the layer runs in the library's HIP kernels.  PyTorch provides
device memory and the current stream.  There is no fallback: if the library
is not built, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

__all__ = [
    "MoEError", "load", "LIB_PATH", "route_topk", "router_logits", "align_capacity", "align", "quant_e4m3",
    "workspace_size", "fused_align_shape", "fused_forward", "Tuning", "STATUS", "NUM_STAGES", "STAGE_NAMES",
    "NOALLOC_SCRATCH_BYTES", "fused_path", "PATH_NAMES", "grouped_gemm", "grouped_gemm_dgrad", "grouped_gemm_wgrad",
    "grouped_gemm_w4", "swiglu_checkpoint", "swiglu_checkpoint_grad", "CHECKPOINT_GROUP", "W4_GROUP",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_mi355x.so")

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE_TOO_SMALL",
          4: "MOE_ERR_DEVICE"}
DTYPE_BF16, DTYPE_FP8 = 0, 1
NUM_STAGES = 5
NOALLOC_SCRATCH_BYTES = 64 << 20  # MOE_NOALLOC_SCRATCH_BYTES
CHECKPOINT_GROUP = 32  # values per scale of an 8-bit activation checkpoint
W4_GROUP = {"mxfp4": 32, "int4": 128}  # weights per scale along K of the 4-bit formats
STAGE_NAMES = ("route", "align", "gate_up", "down", "finalize")
# moe_fused_path's MOE_PATH_* values, in order
PATH_NAMES = ("none", "prefill", "decode", "decode_token_down", "two_launches", "single_launch")


class MoEError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__("%s failed: %s (%d)" % (fn, STATUS.get(code, "?"), code))
        self.code = code


class Tuning(ctypes.Structure):
    _fields_ = [("gemm1_ksplit", ctypes.c_int32), ("gemm2_ksplit", ctypes.c_int32),
                ("token_tiles", ctypes.c_int32), ("unroll", ctypes.c_int32),
                ("gemm2_wave_ksplit", ctypes.c_int32), ("gemm1_stream_tiles", ctypes.c_int32),
                ("gemm2_stream_tiles", ctypes.c_int32), ("reverse_order", ctypes.c_int32),
                ("single_launch", ctypes.c_int32), ("down_per_token", ctypes.c_int32),
                ("routing_in_gate_up", ctypes.c_int32), ("gemm1_feature_tiles", ctypes.c_int32),
                ("gemm2_row_tiles", ctypes.c_int32)]


class _FusedArgs(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int32), ("E", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
        ("top_k", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("logits", ctypes.c_void_p), ("w13", ctypes.c_void_p), ("w2", ctypes.c_void_p),
        ("w13_scale", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p), ("x_scale", ctypes.c_void_p),
        ("h_scale", ctypes.c_void_p), ("y", ctypes.c_void_p), ("topk_ids", ctypes.c_void_p),
        ("topk_weights", ctypes.c_void_p), ("expert_counts", ctypes.c_void_p), ("scales_out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("tuning", ctypes.POINTER(Tuning)),
        ("weight_scale_mode", ctypes.c_int32),
        ("router_w", ctypes.c_void_p), ("logits_out", ctypes.c_void_p),
        ("n_shared", ctypes.c_int32),
        ("expert_offsets", ctypes.c_void_p), ("sorted_ids", ctypes.c_void_p), ("block_expert", ctypes.c_void_p),
        ("num_padded", ctypes.c_void_p),
        ("deterministic", ctypes.c_int32),
    ]


class _Rows(ctypes.Structure):  # moe_rows_t
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64), ("rows", ctypes.c_int32),
                ("div", ctypes.c_int32), ("ids", ctypes.c_void_p)]


class _GroupedArgs(ctypes.Structure):  # moe_grouped_args_t
    _fields_ = [("R", ctypes.c_int32), ("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("offsets", ctypes.c_void_p), ("in_", _Rows), ("weight", ctypes.c_int32), ("w", ctypes.c_void_p),
                ("w_scale", ctypes.c_void_p), ("out", _Rows), ("out_type", ctypes.c_int32)]


class _GroupedWgradArgs(ctypes.Structure):  # moe_grouped_wgrad_args_t
    _fields_ = [("R", ctypes.c_int32), ("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("offsets", ctypes.c_void_p), ("dy", _Rows), ("in_", _Rows), ("dw", ctypes.c_void_p),
                ("out_type", ctypes.c_int32), ("accumulate", ctypes.c_int32)]


_lib = None
_ABI = 15  # moe_abi_version() of the library whose moe_fused_args_t _FusedArgs mirrors


def load():
    """Load the built library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libmoe_mi355x.so is not built (run `python -c 'import __graft_entry__ as g; g.build()'`)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_abi_version.restype = i32
    lib.moe_route_topk.restype = ctypes.c_int
    lib.moe_route_topk.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    lib.moe_align_capacity.restype = sz
    lib.moe_align_capacity.argtypes = [i32, i32, i32, i32]
    lib.moe_align.restype = ctypes.c_int
    lib.moe_align.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    lib.moe_router_logits.restype = ctypes.c_int
    lib.moe_router_logits.argtypes = [vp, vp, i32, i32, i32, vp, vp]
    lib.moe_quant_e4m3.restype = ctypes.c_int
    lib.moe_quant_e4m3.argtypes = [vp, i64, vp, vp, vp]
    lib.moe_fused_workspace_size.restype = sz
    lib.moe_fused_workspace_size.argtypes = [i32, i32, i32, i32, i32, ctypes.c_int]
    lib.moe_fused_align_shape.restype = ctypes.c_int
    lib.moe_fused_align_shape.argtypes = [i32, i32, i32, i32, i32, ctypes.c_int, i32, i32, vp, vp]
    lib.moe_fused_forward.restype = ctypes.c_int
    lib.moe_fused_forward.argtypes = [ctypes.POINTER(_FusedArgs), vp]
    lib.moe_fused_forward_profiled.restype = ctypes.c_int
    lib.moe_fused_forward_profiled.argtypes = [ctypes.POINTER(_FusedArgs), vp, vp]
    lib.moe_fused_forward_noalloc.restype = ctypes.c_int
    lib.moe_fused_path.restype = ctypes.c_int
    lib.moe_fused_path.argtypes = [ctypes.POINTER(_FusedArgs), ctypes.POINTER(i32)]
    lib.moe_fused_forward_noalloc.argtypes = [ctypes.POINTER(_FusedArgs), vp]
    lib.moe_grouped_gemm.restype = ctypes.c_int
    lib.moe_grouped_gemm.argtypes = [ctypes.POINTER(_GroupedArgs), vp]
    lib.moe_grouped_gemm_dgrad.restype = ctypes.c_int
    lib.moe_grouped_gemm_dgrad.argtypes = [ctypes.POINTER(_GroupedArgs), vp]
    lib.moe_grouped_gemm_wgrad.restype = ctypes.c_int
    lib.moe_grouped_gemm_wgrad.argtypes = [ctypes.POINTER(_GroupedWgradArgs), vp]
    lib.moe_swiglu_checkpoint.restype = ctypes.c_int
    lib.moe_swiglu_checkpoint.argtypes = [vp, i64, vp, i32, i32, vp, vp, vp, vp, vp]
    lib.moe_swiglu_checkpoint_grad.restype = ctypes.c_int
    lib.moe_swiglu_checkpoint_grad.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp]
    if lib.moe_abi_version() != _ABI:
        raise RuntimeError("libmoe_mi355x.so has ABI version %d, this binding expects %d: rebuild it"
                           % (lib.moe_abi_version(), _ABI))
    _lib = lib
    return lib


def _check(fn: str, code: int):
    if code != 0:
        raise MoEError(fn, code)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype, index: int, stream, scratch: bool = False) -> torch.Tensor:
    """A tensor on GPU `index` for a call on `stream` (None: the current one) to
    write.  For another stream than the current one it comes from that stream's
    own memory: a block that was freed on the current stream may still be read by
    work queued there, which the call does not wait for.  The current stream,
    where the caller goes on to use it, is recorded on it, unless it is scratch
    memory that the call alone uses."""
    dev = torch.device("cuda", index)
    if stream is None or _stream(stream) == torch._C._cuda_getCurrentRawStream(index):
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if not scratch:
        t.record_stream(torch.cuda.current_stream(dev))
    return t


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype, shape: Sequence[int]):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be on the GPU" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def route_topk(logits: torch.Tensor, top_k: int, ids: Optional[torch.Tensor] = None,
               weights: Optional[torch.Tensor] = None, stream=None):
    """Top-k experts per token and their softmax weights (moe_route_topk)."""
    M, E = logits.shape
    _need(logits, "logits", torch.float32, (M, E))
    if ids is None:
        ids = _empty((M, top_k), torch.int32, logits.get_device(), stream)
    if weights is None:
        weights = _empty((M, top_k), torch.float32, logits.get_device(), stream)
    _need(ids, "ids", torch.int32, (M, top_k))
    _need(weights, "weights", torch.float32, (M, top_k))
    _check("moe_route_topk", load().moe_route_topk(_ptr(logits), M, E, top_k, _ptr(ids), _ptr(weights),
                                                   _stream(stream)))
    return ids, weights


def router_logits(x: torch.Tensor, router_w: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None):
    """logits = x . router_w^T (moe_router_logits): x bf16 [M,H], router_w bf16
    [E,H] -> fp32 [M,E]."""
    M, H = x.shape
    E = router_w.shape[0]
    _need(x, "x", torch.bfloat16, (M, H))
    _need(router_w, "router_w", torch.bfloat16, (E, H))
    if out is None:
        out = _empty((M, E), torch.float32, x.get_device(), stream)
    _need(out, "out", torch.float32, (M, E))
    _check("moe_router_logits", load().moe_router_logits(_ptr(x), _ptr(router_w), M, E, H, _ptr(out), _stream(stream)))
    return out


def align_capacity(M: int, top_k: int, E: int, block: int) -> int:
    return int(load().moe_align_capacity(M, top_k, E, block))


def align(ids: torch.Tensor, E: int, block: int, stream=None):
    """Sort-and-pad of the (token, slot) pairs by expert (moe_align)."""
    M, k = ids.shape
    _need(ids, "ids", torch.int32, (M, k))
    cap = align_capacity(M, k, E, block)
    counts, offsets, sorted_ids, block_expert, num = (
        _empty((n,), torch.int32, ids.get_device(), stream) for n in (E, E + 1, max(cap, 1), max(cap // block, 1), 1))
    _check("moe_align", load().moe_align(_ptr(ids), M, k, E, block, _ptr(counts), _ptr(offsets), _ptr(sorted_ids),
                                         _ptr(block_expert), _ptr(num), _stream(stream)))
    return dict(counts=counts, offsets=offsets, sorted_ids=sorted_ids[:cap], block_expert=block_expert[:cap // block],
                num_padded=num)


def quant_e4m3(x: torch.Tensor, scale: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None):
    """e4m3 codes of fp32 data with a per-tensor scale (moe_quant_e4m3)."""
    _need(x, "x", torch.float32, x.shape)
    _need(scale, "scale", torch.float32, (1,))
    if out is None:
        out = _empty(x.shape, torch.uint8, x.get_device(), stream)
    _need(out, "out", torch.uint8, x.shape)
    _check("moe_quant_e4m3", load().moe_quant_e4m3(_ptr(x), x.numel(), _ptr(scale), _ptr(out), _stream(stream)))
    return out


def workspace_size(M: int, E: int, H: int, I: int, top_k: int, dtype: str) -> int:
    return int(load().moe_fused_workspace_size(M, E, H, I, top_k, DTYPE_FP8 if dtype == "fp8" else DTYPE_BF16))


def fused_align_shape(M: int, E: int, H: int, I: int, top_k: int, dtype: str, deterministic: bool = False,
                      weight_scale_mode: int = 0):
    """(block, capacity) of the fused call's sort-and-pad step
    (moe_fused_align_shape); E and top_k count the shared experts."""
    b, c = ctypes.c_int32(0), ctypes.c_int64(0)
    _check("moe_fused_align_shape", load().moe_fused_align_shape(
        M, E, H, I, top_k, DTYPE_FP8 if dtype == "fp8" else DTYPE_BF16, int(bool(deterministic)),
        int(weight_scale_mode), ctypes.byref(b), ctypes.byref(c)))
    return int(b.value), int(c.value)


def fused_path(M: int, E: int, H: int, I: int, top_k: int, dtype: str = "bf16", n_shared: int = 0,
               weight_scale_mode: int = 0, static_x_scale: bool = False, static_h_scale: bool = False,
               router_w: bool = False, deterministic: bool = False, tuning: Optional[Tuning] = None) -> str:
    """Name (PATH_NAMES) of the launch sequence fused_forward takes on a call
    of this shape (moe_fused_path; host only, no GPU needed).  E and top_k
    count the routed experts; static_x_scale/static_h_scale: fp8 scales given
    by the caller; router_w: logits computed in the layer."""
    fp8 = dtype == "fp8"
    fake = 1 << 20  # moe_fused_path reads no memory through the pointers
    args = _FusedArgs(
        M=M, E=E, H=H, I=I, top_k=top_k, dtype=DTYPE_FP8 if fp8 else DTYPE_BF16, x=fake, w13=fake, w2=fake,
        logits=None if router_w else fake, router_w=fake if router_w else None,
        w13_scale=fake if fp8 else None, w2_scale=fake if fp8 else None,
        x_scale=fake if static_x_scale else None, h_scale=fake if static_h_scale else None,
        tuning=ctypes.pointer(tuning) if tuning is not None else None, weight_scale_mode=int(weight_scale_mode),
        n_shared=int(n_shared), deterministic=int(bool(deterministic)))
    p = ctypes.c_int32(-1)
    _check("moe_fused_path", load().moe_fused_path(ctypes.byref(args), ctypes.byref(p)))
    return PATH_NAMES[p.value]


def fused_forward(x: torch.Tensor, logits: Optional[torch.Tensor], w13: torch.Tensor, w2: torch.Tensor, top_k: int,
                  dtype: str = "bf16", w13_scale: Optional[torch.Tensor] = None,
                  w2_scale: Optional[torch.Tensor] = None, x_scale: Optional[torch.Tensor] = None,
                  h_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, topk_ids: Optional[torch.Tensor] = None,
                  topk_weights: Optional[torch.Tensor] = None, expert_counts: Optional[torch.Tensor] = None,
                  scales_out: Optional[torch.Tensor] = None, tuning: Optional[Tuning] = None, stream=None,
                  events=None, router_w: Optional[torch.Tensor] = None,
                  logits_out: Optional[torch.Tensor] = None, n_shared: int = 0,
                  align_out: Optional[dict] = None, deterministic: bool = False,
                  noalloc: bool = False) -> torch.Tensor:
    """The fused layer (moe_fused_forward).

    x bf16 [M,H]; logits fp32 [M,E]; w13 [E,2I,H] and w2 [E,H,I] as bf16
    (dtype "bf16") or uint8 e4m3fn codes (dtype "fp8") with fp32 device
    scales, either one per tensor ([1] each), one per weight row (w13_scale
    [E,2I], w2_scale [E,H]) or one per expert ([E] each), or uint8 E8M0 codes
    one per 128 x 128 block (w13_scale [E,2I/128,H/128], w2_scale
    [E,H/128,I/128]: block-scaled mode, activations scaled per 128 elements);
    x_scale/h_scale: static fp8 activation scales or None (dynamic).  logits may be None when router_w (bf16 [E,H]) is given:
    the layer then computes them (into logits_out fp32 [M,E] when given).
    n_shared: S shared experts stacked after the E routed ones (w13 [E+S,2I,H],
    w2 [E+S,H,I], per-row scales [E+S,..]), each taken by every token with
    weight one; topk_ids/topk_weights are then [M,top_k+S], expert_counts [E+S].
    events: optional list of 2*NUM_STAGES hipEvent_t handles (ints) recorded
    around the stages on the stream.
    align_out: optional dict of int32 GPU tensors receiving the call's
    sort-and-pad outputs: "offsets" [E+S+1], "sorted_ids" [capacity],
    "block_expert" [capacity/block], "num_padded" [1] (block and capacity
    from fused_align_shape; any subset of the keys).
    deterministic: batch-invariant mode (fp8 needs x_scale and h_scale).
    noalloc: call moe_fused_forward_noalloc, whose workspace is the library's
    own scratch array (no workspace may be given; `out` must be given, so
    that the call allocates nothing here either).
    """
    M, H = x.shape
    if (logits is None) == (router_w is None):
        raise ValueError("give exactly one of logits and router_w")
    E = logits.shape[1] if logits is not None else router_w.shape[0]
    fp8 = dtype == "fp8"
    I = w2.shape[2]
    S = int(n_shared)
    ES, KS = E + S, top_k + S
    wdt = torch.uint8 if fp8 else torch.bfloat16
    _need(x, "x", torch.bfloat16, (M, H))
    if logits is not None:
        _need(logits, "logits", torch.float32, (M, E))
    else:
        _need(router_w, "router_w", torch.bfloat16, (E, H))
        if logits_out is not None:
            _need(logits_out, "logits_out", torch.float32, (M, E))
    _need(w13, "w13", wdt, (ES, 2 * I, H))
    _need(w2, "w2", wdt, (ES, H, I))
    # weight scale mode from the scale shapes: uint8 E8M0 codes
    # [E+S,2I/128,H/128] one per 128 x 128 block (3), [E+S,rows] one per row
    # (1), [E+S] with E+S > 1 one per expert (2), [1] one per tensor (0)
    mode = 0
    if w13_scale is not None and w13_scale.dtype == torch.uint8:
        mode = 3
        _need(w13_scale, "w13_scale", torch.uint8, (ES, 2 * I // 128, H // 128))
        _need(w2_scale, "w2_scale", torch.uint8, (ES, H // 128, I // 128))
    elif w13_scale is not None and w13_scale.dim() == 2:
        mode = 1
        _need(w13_scale, "w13_scale", torch.float32, (ES, 2 * I))
        _need(w2_scale, "w2_scale", torch.float32, (ES, H))
    elif w13_scale is not None and ES > 1 and w13_scale.numel() == ES:
        mode = 2
        _need(w13_scale, "w13_scale", torch.float32, (ES,))
        _need(w2_scale, "w2_scale", torch.float32, (ES,))
    for name, s in (("w13_scale", None if mode else w13_scale), ("w2_scale", None if mode else w2_scale),
                    ("x_scale", x_scale), ("h_scale", h_scale)):
        if s is not None:
            _need(s, name, torch.float32, (1,))
    if out is None:
        if noalloc:
            raise ValueError("the no-alloc call needs `out`")
        out = _empty((M, H), torch.bfloat16, x.get_device(), stream)
    _need(out, "out", torch.bfloat16, (M, H))
    if topk_ids is not None:
        _need(topk_ids, "topk_ids", torch.int32, (M, KS))
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, (M, KS))
    if expert_counts is not None:
        _need(expert_counts, "expert_counts", torch.int32, (ES,))
    if scales_out is not None:
        _need(scales_out, "scales_out", torch.float32, (2,))
    al = dict(align_out or {})
    if set(al) - {"offsets", "sorted_ids", "block_expert", "num_padded"}:
        raise ValueError("unknown align_out keys: %s" % sorted(set(al) - {"offsets", "sorted_ids", "block_expert",
                                                                            "num_padded"}))
    if al:
        blk, cap = fused_align_shape(M, ES, H, I, KS, dtype, deterministic, mode)
        for key, shape in (("offsets", (ES + 1,)), ("sorted_ids", (cap,)), ("block_expert", (cap // blk,)),
                           ("num_padded", (1,))):
            if key in al:
                _need(al[key], "align_out[%s]" % key, torch.int32, shape)
    lib = load()
    if noalloc:
        if workspace is not None:
            raise ValueError("the no-alloc call takes no workspace")
    else:
        need = int(lib.moe_fused_workspace_size(M, ES, H, I, KS, DTYPE_FP8 if fp8 else DTYPE_BF16))
        if workspace is None:
            workspace = _empty((max(need, 256),), torch.uint8, x.get_device(), stream, scratch=True)
        if workspace.dtype != torch.uint8 or workspace.device.type != "cuda" or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 GPU tensor")
    args = _FusedArgs(
        M=M, E=E, H=H, I=I, top_k=top_k, dtype=DTYPE_FP8 if fp8 else DTYPE_BF16,
        x=_ptr(x), logits=_ptr(logits), w13=_ptr(w13), w2=_ptr(w2),
        w13_scale=_ptr(w13_scale), w2_scale=_ptr(w2_scale), x_scale=_ptr(x_scale), h_scale=_ptr(h_scale),
        y=_ptr(out), topk_ids=_ptr(topk_ids), topk_weights=_ptr(topk_weights),
        expert_counts=_ptr(expert_counts), scales_out=_ptr(scales_out),
        workspace=_ptr(workspace), workspace_bytes=0 if workspace is None else workspace.numel(),
        tuning=ctypes.pointer(tuning) if tuning is not None else None,
        weight_scale_mode=mode,
        router_w=_ptr(router_w), logits_out=_ptr(logits_out), n_shared=S,
        expert_offsets=_ptr(al.get("offsets")), sorted_ids=_ptr(al.get("sorted_ids")),
        block_expert=_ptr(al.get("block_expert")), num_padded=_ptr(al.get("num_padded")),
        deterministic=int(bool(deterministic)),
    )
    if noalloc:
        if events is not None:
            raise ValueError("the no-alloc call records no stage events")
        _check("moe_fused_forward_noalloc", lib.moe_fused_forward_noalloc(ctypes.byref(args), _stream(stream)))
    elif events is None:
        _check("moe_fused_forward", lib.moe_fused_forward(ctypes.byref(args), _stream(stream)))
    else:
        if len(events) != 2 * NUM_STAGES:
            raise ValueError("events must hold %d hipEvent_t handles" % (2 * NUM_STAGES))
        arr = (ctypes.c_void_p * len(events))(*events)
        _check("moe_fused_forward_profiled",
               lib.moe_fused_forward_profiled(ctypes.byref(args), _stream(stream), ctypes.cast(arr, ctypes.c_void_p)))
    return out


# ------------------------------------------------------------------ grouped products and the checkpointed activation
class _Call:
    """The tensors of one call: all on one GPU, whose current stream (or
    `stream`) it runs on; outputs made here are from that stream's memory.  A
    decode-sized call takes about ten microseconds on the GPU, so the checks are
    written for few Python steps."""

    __slots__ = ("index", "given", "stream")

    def __init__(self, like: torch.Tensor, stream):
        if not isinstance(like, torch.Tensor) or not like.is_cuda:
            raise ValueError("the operands must be GPU tensors")
        self.index, self.given = like.get_device(), stream
        self.stream = torch._C._cuda_getCurrentRawStream(self.index) if stream is None else _stream(stream)

    def need(self, t, name, dtype, shape):
        """Pointer of a contiguous tensor of this type and shape."""
        if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            _need(t, name, dtype, shape)  # says what is wrong
        if t.get_device() != self.index:
            self.elsewhere(t, name)
        return t.data_ptr()

    def elsewhere(self, t, name):
        raise ValueError("%s is on %s, the other operands on cuda:%d" % (name, t.device, self.index))

    def empty(self, shape, dtype):
        return _empty(shape, dtype, self.index, self.given)

    def vector(self, t, name, dtype, n):
        return None if t is None else self.need(t, name, dtype, (n,))

    def rows(self, t, name, dtype, width, ids, div, R) -> _Rows:
        """A [rows, width] operand whose rows may be strided, as moe_rows_t."""
        if not isinstance(t, torch.Tensor) or t.get_device() != self.index:
            raise ValueError("%s must be a tensor on cuda:%d" % (name, self.index))
        if t.dtype is not dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        shape = t.shape
        if len(shape) != 2 or shape[1] != width:
            raise ValueError("%s must have shape (rows, %d), got %s" % (name, width, tuple(shape)))
        step = t.stride()
        if step[1] != 1 and width > 1:
            raise ValueError("%s's rows must be contiguous" % name)
        ptr = None
        if ids is not None:
            ptr = self.need(ids, name + "'s row ids", torch.int32, (R,)) or None
        if shape[0] >> 31:
            _sizes(shape[0])
        # one row has no stride of its own, no row at all no address
        return _Rows(t.data_ptr() or 16, step[0] if shape[0] > 1 else width, shape[0], div if ptr else 1, ptr)

    def run(self, fn, *args):
        call = getattr(_lib or load(), fn)
        if torch._C._cuda_getDevice() == self.index:
            code = call(*args, self.stream)
        else:
            with torch.cuda.device(self.index):
                code = call(*args, self.stream)
        if code:
            raise MoEError(fn, code)


def _sizes(bits: int):
    """`bits`: the bitwise or of what the library takes as int32, sizes and at
    most one divisor; ctypes would drop the bits above."""
    if bits >> 31 not in (0, -1):
        raise ValueError("a size, or a divisor, does not fit 32 bits")


_OUT_TYPE = {torch.bfloat16: 0, torch.float32: 1}


def _out_type(dtype, name) -> int:
    if dtype not in _OUT_TYPE:
        raise TypeError("%s must be torch.bfloat16 or torch.float32, got %s" % (name, dtype))
    return _OUT_TYPE[dtype]


def _grouped(fn, call, a, w, E, N, K, offsets, out, in_rows, in_div, out_rows, out_dtype, weight=0, scales=None):
    src, dst = (N, K) if fn == "moe_grouped_gemm_dgrad" else (K, N)
    off = call.need(offsets, "offsets", torch.int32, (E + 1,))
    R = a.shape[0] if in_rows is None else in_rows.numel()
    _sizes(R | E | N | K | in_div)
    if out is None:
        out_type = _out_type(out_dtype, "out_dtype")
        out = call.empty((R, dst), out_dtype)
    elif isinstance(out, torch.Tensor):
        out_type = _out_type(out.dtype, "out")
    else:
        raise ValueError("out must be a GPU tensor")
    args = _GroupedArgs(R, E, N, K, off, call.rows(a, "input", torch.bfloat16, src, in_rows, in_div, R), weight, w,
                        scales, call.rows(out, "out", out.dtype, dst, out_rows, 1, R), out_type)
    call.run(fn, ctypes.byref(args))
    return out


def _bf16_product(fn, a, w, offsets, out, in_rows, in_div, out_rows, out_dtype, stream):
    call = _Call(a, stream)
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("the weights must be a tensor [E, N, K]")
    E, N, K = w.shape
    return _grouped(fn, call, a, call.need(w, "w", torch.bfloat16, (E, N, K)), E, N, K, offsets, out, in_rows, in_div,
                    out_rows, out_dtype)


def grouped_gemm(a: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None, *,
                 a_rows: Optional[torch.Tensor] = None, a_div: int = 1, out_rows: Optional[torch.Tensor] = None,
                 out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """out[i] = w[e] a[i] for the rows i of every expert e (moe_grouped_gemm):
    offsets[e] <= i < offsets[e+1], int32 [E+1] on the GPU.

    a bf16 [R,K] (rows may be strided); w bf16 [E,N,K]; out bf16 or fp32
    [R,N], made here as out_dtype when not given (rows at or beyond offsets[E]
    are not written).  a_rows int32 [R]: row i is row a_rows[i] // a_div of a,
    zeros outside it (a_rows = align's sorted_ids, a_div = top_k: the tokens
    themselves).  out_rows int32 [R]: row i goes to row out_rows[i] of out, and
    nowhere outside it (without `out`, a result of R rows is made)."""
    return _bf16_product("moe_grouped_gemm", a, w, offsets, out, a_rows, a_div, out_rows, out_dtype, stream)


def grouped_gemm_dgrad(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
                       *, dy_rows: Optional[torch.Tensor] = None, dy_div: int = 1,
                       out_rows: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                       stream=None) -> torch.Tensor:
    """Gradient of grouped_gemm's input, out[i] = w[e]^T dy[i]
    (moe_grouped_gemm_dgrad): dy bf16 [R,N] -> out [R,K]; the rest as there."""
    return _bf16_product("moe_grouped_gemm_dgrad", dy, w, offsets, out, dy_rows, dy_div, out_rows, out_dtype, stream)


def grouped_gemm_wgrad(dy: torch.Tensor, a: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
                       *, dy_rows: Optional[torch.Tensor] = None, dy_div: int = 1,
                       a_rows: Optional[torch.Tensor] = None, a_div: int = 1, accumulate: bool = False,
                       out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """Gradient of grouped_gemm's weights, out[e] = sum of dy[i] a[i]^T over
    expert e's rows (moe_grouped_gemm_wgrad), zeros for an expert without rows:
    dy bf16 [R,N], a bf16 [R,K] -> out [E,N,K] fp32 or bf16.  accumulate: add
    to `out` (fp32) instead.  Rows may be gathered as in grouped_gemm: R is then
    the number of ids, and an operand without ids holds at least R rows."""
    call = _Call(dy, stream)
    if not isinstance(a, torch.Tensor) or dy.dim() != 2 or a.dim() != 2:
        raise ValueError("dy and a must be [rows, width] tensors")
    E, N, K = offsets.numel() - 1, dy.shape[1], a.shape[1]
    off = call.need(offsets, "offsets", torch.int32, (E + 1,))
    ids = dy_rows if dy_rows is not None else a_rows
    R = dy.shape[0] if ids is None else ids.numel()
    if ids is None and a.shape[0] != R:
        raise ValueError("without row ids dy and a must have the same number of rows, got %d and %d" % (R, a.shape[0]))
    _sizes(R | E | N | K | dy_div)
    _sizes(a_div)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs `out`")
        _out_type(out_dtype, "out_dtype")
        out = call.empty((E, N, K), out_dtype)
    elif not isinstance(out, torch.Tensor):
        raise ValueError("out must be a GPU tensor")
    args = _GroupedWgradArgs(R, E, N, K, off, call.rows(dy, "dy", torch.bfloat16, N, dy_rows, dy_div, R),
                             call.rows(a, "a", torch.bfloat16, K, a_rows, a_div, R),
                             call.need(out, "out", out.dtype, (E, N, K)), _out_type(out.dtype, "out"),
                             int(bool(accumulate)))
    call.run("moe_grouped_gemm_wgrad", ctypes.byref(args))
    return out


def grouped_gemm_w4(a: torch.Tensor, w4: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor,
                    out: Optional[torch.Tensor] = None, *, a_rows: Optional[torch.Tensor] = None, a_div: int = 1,
                    out_rows: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """grouped_gemm with 4-bit weights, streamed for a few rows per expert:
    w4 uint8 [E,N,K/2], two codes per byte along K (low nibble first).  scales
    uint8 [E,N,K/32]: OCP MXFP4 (e2m1 codes, E8M0 scales; a scale of 255 is NaN,
    weights of 2^128 and more are infinities); scales bf16 [E,N,K/128]:
    integers 0..15 standing for -8..7, for rows of elements below 2^116."""
    if not isinstance(w4, torch.Tensor) or w4.dim() != 3:
        raise ValueError("the weights must be a tensor [E, N, K/2]")
    if not isinstance(scales, torch.Tensor) or scales.dtype not in (torch.uint8, torch.bfloat16):
        raise TypeError("scales must be uint8 (MXFP4) or bfloat16 (int4)")
    call = _Call(a, stream)
    E, N, K = w4.shape[0], w4.shape[1], 2 * w4.shape[2]
    fmt, group = (1, W4_GROUP["mxfp4"]) if scales.dtype is torch.uint8 else (2, W4_GROUP["int4"])
    return _grouped("moe_grouped_gemm", call, a, call.need(w4, "w4", torch.uint8, (E, N, K // 2)), E, N, K, offsets,
                    out, a_rows, a_div, out_rows, out_dtype, fmt,
                    call.need(scales, "scales", scales.dtype, (E, N, K // group)))


def swiglu_checkpoint(gu: torch.Tensor, row_weight: Optional[torch.Tensor] = None, *, checkpoint: bool = True,
                      num_rows: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                      codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, stream=None):
    """h = row_weight * SiLU(gate) * up of gu bf16 [R,2I] (gate columns first;
    rows may be strided), and gu kept in 8 bits (moe_swiglu_checkpoint).

    Returns (h bf16 [R,I], codes uint8 e4m3 [R,2I], scales uint8 E8M0
    [R,2,ceil(I/32)]); the last two are None with checkpoint=False.  num_rows
    int32 [1] on the GPU (offsets[E:]): rows at or beyond it are left alone."""
    call = _Call(gu, stream)
    if gu.dim() != 2 or gu.shape[1] % 2:
        raise ValueError("gu must have shape (rows, 2*I), got %s" % (tuple(gu.shape),))
    R, I = gu.shape[0], gu.shape[1] // 2
    _sizes(R | I)
    src = call.rows(gu, "gu", torch.bfloat16, 2 * I, None, 1, R)
    if h is None:
        h = call.empty((R, I), torch.bfloat16)
    G = -(-I // CHECKPOINT_GROUP)
    if checkpoint:
        codes = call.empty((R, 2 * I), torch.uint8) if codes is None else codes
        scales = call.empty((R, 2, G), torch.uint8) if scales is None else scales
    elif codes is not None or scales is not None:
        raise ValueError("codes and scales need checkpoint=True")
    call.run("moe_swiglu_checkpoint", src.data, src.stride, call.vector(row_weight, "row_weight", torch.float32, R),
             R, I, call.vector(num_rows, "num_rows", torch.int32, 1), call.need(h, "h", torch.bfloat16, (R, I)),
             call.need(codes, "codes", torch.uint8, (R, 2 * I)) if checkpoint else None,
             call.need(scales, "scales", torch.uint8, (R, 2, G)) if checkpoint else None)
    return h, codes, scales


def swiglu_checkpoint_grad(codes: torch.Tensor, scales: torch.Tensor, dh: torch.Tensor,
                           row_weight: Optional[torch.Tensor] = None, *, num_rows: Optional[torch.Tensor] = None,
                           dgu: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                           dweight: Optional[torch.Tensor] = None, stream=None):
    """Gradient of swiglu_checkpoint from its codes and scales and dh bf16
    [R,I] (moe_swiglu_checkpoint_grad): returns (dgu bf16 [R,2I], h bf16 [R,I]
    recomputed from the checkpoint and weighted, dweight fp32 [R])."""
    call = _Call(dh, stream)
    if dh.dim() != 2:
        raise ValueError("dh must have shape (rows, I), got %s" % (tuple(dh.shape),))
    R, I = dh.shape
    _sizes(R | I)
    if dgu is None:
        dgu = call.empty((R, 2 * I), torch.bfloat16)
    if h is None:
        h = call.empty((R, I), torch.bfloat16)
    if dweight is None:
        dweight = call.empty((R,), torch.float32)
    call.run("moe_swiglu_checkpoint_grad", call.need(codes, "codes", torch.uint8, (R, 2 * I)),
             call.need(scales, "scales", torch.uint8, (R, 2, -(-I // CHECKPOINT_GROUP))),
             call.need(dh, "dh", torch.bfloat16, (R, I)), call.vector(row_weight, "row_weight", torch.float32, R), R, I,
             call.vector(num_rows, "num_rows", torch.int32, 1), call.need(dgu, "dgu", torch.bfloat16, (R, 2 * I)),
             call.need(h, "h", torch.bfloat16, (R, I)), call.need(dweight, "dweight", torch.float32, (R,)))
    return dgu, h, dweight
