"""Python binding of libmoe.so, the MI355X fused Mixture-of-Experts layer.

The binding only marshals arguments: every step of the layer runs in the
HIP kernels of libmoe.so (see include/moe.h).  PyTorch provides device
memory and streams.  There is no fallback path: if the library is missing
or cannot be loaded, importing this module raises.

Functions carry the C names:

    moe_pack_weights(w, dtype)                          -> PackedWeight (packed copy + descriptor, one-time)
    moe_routing_layout(T, k, E, H, I, dtype)            -> dict (host only)
    moe_workspace_layout(T, k, E, H, I, dtype)          -> dict (host only)
    moe_router_split_weights(w)                         -> split fp32 router weight pair (one-time)
    moe_router_gemm(x, w_pair, N)                       -> fp32 router scores
    moe_router_gemm_topk(x, w_pair, E, k, ...)          -> (topk_ids, topk_w[, scores])
    moe_router_topk(logits, k, renormalize, n_shared)    -> (topk_ids, topk_w)
    moe_build_routing_bf16(topk_ids, E, H, I, routing)  -> None
    moe_build_routing_fp8(topk_ids, E, H, I, routing)   -> None
    moe_forward_bf16(x, topk_w, routing, w1, w2, workspace, out) -> out
    moe_forward_fp8(x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out) -> out
    moe_build_routing_mxfp8 / moe_forward_mxfp8 (as the fp8 pair, e8m0 block-scale codes)
    moe_build_routing_int8 / moe_forward_int8   (as the fp8 pair, int8 codes)
    moe_build_routing_int4 / moe_forward_int4   (int4 weights + group scales, bf16 activations)
    moe_build_routing_fp8_block / moe_forward_fp8_block (128x128 weight blocks, 1x128 token groups)
    moe_build_routing_int8_w8a16 / moe_forward_int8_w8a16 (int8 weights + row scales, bf16 activations)
    moe_quantize_mxfp4(x) / moe_dequantize_mxfp4(codes, scales) -> MXFP4 codes and scale codes / values
    moe_pack_weights_mxfp4(codes, scales)               -> PackedWeight (one-time)
    moe_build_routing_mxfp4 / moe_forward_mxfp4         (as the bf16 pair, MXFP4 weights and activations)
    moe_dispatch(x, routing, k, E, topk_w)              -> rows in expert order
    moe_combine(y, routing, k, E, topk_w)               -> rows in token order
    moe_dispatch_grad / moe_combine_grad                (gradients of the rows and of topk_w)
    moe_router_topk_grad(logits, topk_ids, topk_w, dtopk_w) -> gradient of the router scores
    moe_grouped_linear(xs, w, routing, k, ...) / moe_linear(x, w, ...)
                                                        -> act(x w^T + bias) + residual, by expert / of plain rows
    moe_grouped_linear_grad_x / moe_linear_grad_x       (gradient of the rows, or of the pre-activation before them)
    moe_grouped_linear_grad_w / moe_linear_grad_w       (gradients of the matrices and biases)
    moe_grouped_act_grad / moe_act_grad                 (gradient of an activation by itself)

plus allocation helpers (alloc_routing, alloc_workspace), pack_weights() for a
whole weight dict, and a convenience moe_layer() that runs routing + forward
with freshly allocated buffers.  The forward calls take W1/W2 packed by
moe_pack_weights (a one-time byte permutation into MFMA-fragment order).
A size that does not fit the library's C int raises ctypes.ArgumentError.
"""
from __future__ import annotations

import ctypes
import operator
import os

import torch  # loads the HIP runtime that libmoe.so binds to

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_DTYPE_BF16 = 0
MOE_DTYPE_FP8_W8A8 = 1
MOE_DTYPE_MXFP8 = 2
MOE_DTYPE_INT8_W8A8 = 3
MOE_DTYPE_INT4_W4A16 = 4
MOE_DTYPE_FP8_BLOCK = 5
MOE_DTYPE_INT8_W8A16 = 6
MOE_DTYPE_MXFP4 = 8
DTYPES = {"bf16": MOE_DTYPE_BF16, "fp8": MOE_DTYPE_FP8_W8A8, "mxfp8": MOE_DTYPE_MXFP8,
          "int8": MOE_DTYPE_INT8_W8A8, "int4": MOE_DTYPE_INT4_W4A16, "fp8b": MOE_DTYPE_FP8_BLOCK,
          "int8w": MOE_DTYPE_INT8_W8A16, "mxfp4": MOE_DTYPE_MXFP4}
ROW_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ACTS = {"none": 0, "silu": 1, "gelu": 2, "swiglu": 3}


class MoeError(RuntimeError):
    def __init__(self, name, status):
        self.status = status
        super().__init__(f"{name} failed: {status} ({status_string(status)})")


class RoutingLayout(ctypes.Structure):
    _fields_ = [("header", ctypes.c_size_t), ("expert_offsets", ctypes.c_size_t),
                ("sorted_pairs", ctypes.c_size_t), ("pair_pos", ctypes.c_size_t),
                ("tasks", ctypes.c_size_t), ("scratch", ctypes.c_size_t),
                ("total_bytes", ctypes.c_size_t),
                ("block_m", ctypes.c_int32), ("max_tasks", ctypes.c_int32)]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [("xq", ctypes.c_size_t), ("x_scale", ctypes.c_size_t),
                ("x_scale_rows", ctypes.c_size_t), ("g", ctypes.c_size_t),
                ("h", ctypes.c_size_t), ("h_scale", ctypes.c_size_t), ("y", ctypes.c_size_t),
                ("total_bytes", ctypes.c_size_t), ("split_k1", ctypes.c_int32),
                ("split_k2", ctypes.c_int32), ("tiling", ctypes.c_int32)]


class PackedWeightsDesc(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("check", ctypes.c_uint64)]


class PackedWeight:
    """A weight tensor packed by moe_pack_weights together with the
    library's descriptor of it, which the forward calls take.  `tensor` is
    the packed device tensor (same shape and dtype as the row-major one; MXFP4:
    uint8 [E][rows][cols / 2 + cols / 32], codes and scale codes)."""

    def __init__(self, tensor, desc):
        self.tensor = tensor
        self.desc = desc

    shape = property(lambda self: self.tensor.shape)
    dtype = property(lambda self: self.tensor.dtype)
    device = property(lambda self: self.tensor.device)

    def clone(self):
        """A device copy of the packed bytes, with its own descriptor."""
        return moe_describe_packed_weights(self.tensor.clone(), self.desc.dtype)

    def numel(self):
        return self.tensor.numel()

    def element_size(self):
        return self.tensor.element_size()


EXPORTS = ("moe_status_string", "moe_pack_weights", "moe_describe_packed_weights", "moe_routing_layout",
           "moe_workspace_layout",
           "moe_router_topk", "moe_router_pair_bytes", "moe_router_split_weights",
           "moe_router_workspace_bytes", "moe_router_gemm", "moe_router_gemm_topk",
           "moe_build_routing_bf16", "moe_build_routing_fp8", "moe_build_routing_mxfp8",
           "moe_build_routing_int8", "moe_build_routing_int4", "moe_forward_bf16",
           "moe_forward_fp8", "moe_forward_mxfp8", "moe_forward_int8", "moe_forward_int4",
           "moe_build_routing_fp8_block", "moe_forward_fp8_block",
           "moe_build_routing_int8_w8a16", "moe_forward_int8_w8a16", "moe_set_stage_events", "moe_device_cu_count",
           "moe_stream_read", "moe_forward_fp8_noalloc", "moe_route_forward_bf16", "moe_route_forward_fp8",
           "moe_route_forward_int8", "moe_route_forward_fp8_block", "moe_route_forward_mxfp8",
           "moe_route_forward_int4", "moe_route_forward_int8_w8a16", "moe_tile_copy_read",
           "moe_quantize_mxfp4", "moe_dequantize_mxfp4", "moe_pack_weights_mxfp4", "moe_build_routing_mxfp4",
           "moe_forward_mxfp4", "moe_route_forward_mxfp4", "moe_dispatch", "moe_combine", "moe_dispatch_grad",
           "moe_combine_grad", "moe_router_topk_grad", "moe_grouped_linear", "moe_grouped_linear_grad_x",
           "moe_grouped_linear_grad_w", "moe_grouped_act_grad", "moe_linear", "moe_linear_grad_x", "moe_linear_grad_w",
           "moe_act_grad")


class _CInt:
    """A C int argument.  ctypes.c_int would keep the low 32 bits of a larger
    number, and the library would check and run that size."""

    @staticmethod
    def from_param(value):
        if value.__class__ is not int:
            value = operator.index(value)
        if -0x80000000 <= value <= 0x7fffffff:
            return value
        raise ValueError(f"{value} does not fit the library's 32-bit sizes")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python mixture_experts_layer_lds_amd/build.py` (or __graft_entry__.build())")
    L = ctypes.CDLL(LIB_PATH)
    i, r, P, sz = _CInt, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_status_string.argtypes = [i]
    L.moe_pack_weights.restype = r
    L.moe_pack_weights.argtypes = [P, i, i, i, i, P, ctypes.POINTER(PackedWeightsDesc), P]
    L.moe_describe_packed_weights.restype = r
    L.moe_describe_packed_weights.argtypes = [P, i, i, i, i, ctypes.POINTER(PackedWeightsDesc)]
    L.moe_routing_layout.restype = r
    L.moe_routing_layout.argtypes = [i, i, i, i, i, i, ctypes.POINTER(RoutingLayout)]
    L.moe_workspace_layout.restype = r
    L.moe_workspace_layout.argtypes = [i, i, i, i, i, i, ctypes.POINTER(WorkspaceLayout)]
    for n in ("moe_build_routing_bf16", "moe_build_routing_fp8"):
        f = getattr(L, n)
        f.restype = r
        f.argtypes = [P, i, i, i, i, i, P, sz, P]
    L.moe_router_topk.restype = r
    L.moe_router_pair_bytes.restype = r
    L.moe_router_pair_bytes.argtypes = [i, i, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_router_split_weights.restype = r
    L.moe_router_split_weights.argtypes = [P, i, i, P, sz, P]
    L.moe_router_workspace_bytes.restype = r
    L.moe_router_workspace_bytes.argtypes = [i, i, i, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_router_gemm.restype = r
    L.moe_router_gemm.argtypes = [P, P, i, i, i, P, sz, P, P]
    L.moe_router_gemm_topk.restype = r
    L.moe_router_gemm_topk.argtypes = [P, P, i, i, i, i, i, i, P, sz, P, P, P, P]
    L.moe_router_topk.argtypes = [P, i, i, i, i, i, P, P, P]
    L.moe_forward_bf16.restype = r
    D = ctypes.POINTER(PackedWeightsDesc)
    L.moe_forward_bf16.argtypes = [P, P, P, D, D, i, i, i, i, i, P, sz, P, P]
    L.moe_forward_fp8.restype = r
    L.moe_forward_fp8.argtypes = [P, P, P, D, P, D, P, i, i, i, i, i, P, sz, P, P]
    L.moe_forward_mxfp8.restype = r
    L.moe_forward_mxfp8.argtypes = [P, P, P, D, P, D, P, i, i, i, i, i, P, sz, P, P]
    L.moe_forward_fp8_block.restype = r
    L.moe_forward_fp8_block.argtypes = [P, P, P, D, P, D, P, i, i, i, i, i, P, sz, P, P]
    L.moe_forward_int4.restype = r
    L.moe_forward_int4.argtypes = [P, P, P, D, P, D, P, i, i, i, i, i, P, sz, P, P]
    L.moe_forward_int8.restype = r
    L.moe_forward_int8.argtypes = [P, P, P, D, P, D, P, i, i, i, i, i, P, sz, P, P]
    L.moe_forward_int8_w8a16.restype = r
    L.moe_forward_int8_w8a16.argtypes = [P, P, P, D, P, D, P, i, i, i, i, i, P, sz, P, P]
    L.moe_set_stage_events.restype = r
    L.moe_set_stage_events.argtypes = [ctypes.POINTER(P), i]
    L.moe_device_cu_count.restype = r
    L.moe_device_cu_count.argtypes = []
    L.moe_forward_fp8_noalloc.restype = r
    L.moe_forward_fp8_noalloc.argtypes = [P, P, P, D, P, D, P, i, i, i, i, i, P, P]
    L.moe_stream_read.restype = r
    L.moe_stream_read.argtypes = [P, sz, P, sz, P]
    L.moe_tile_copy_read.restype = r
    L.moe_tile_copy_read.argtypes = [i, P, sz, i, i, P, sz, P]
    L.moe_route_forward_bf16.restype = r
    L.moe_route_forward_bf16.argtypes = [P, P, P, P, sz, D, D, i, i, i, i, i, P, sz, P, P]
    L.moe_route_forward_fp8.restype = r
    L.moe_route_forward_fp8.argtypes = [P, P, P, P, sz, D, P, D, P, i, i, i, i, i, P, sz, P, P]
    for f in (L.moe_route_forward_int8, L.moe_route_forward_fp8_block, L.moe_route_forward_mxfp8,
              L.moe_route_forward_int4, L.moe_route_forward_int8_w8a16):
        f.restype = r
        f.argtypes = [P, P, P, P, sz, D, P, D, P, i, i, i, i, i, P, sz, P, P]
    i64 = ctypes.c_int64
    for n, args in (("moe_quantize_mxfp4", [P, i, i64, i, i64, P, P, P]),
                    ("moe_dequantize_mxfp4", [P, P, i64, i, i, P, P]),
                    ("moe_pack_weights_mxfp4", [P, P, i, i, i, P, D, P]),
                    ("moe_build_routing_mxfp4", [P, i, i, i, i, i, P, sz, P]),
                    ("moe_forward_mxfp4", [P, P, P, D, D, i, i, i, i, i, P, sz, P, P]),
                    ("moe_route_forward_mxfp4", [P, P, P, P, sz, D, D, i, i, i, i, i, P, sz, P, P]),
                    ("moe_dispatch", [P, i, P, P, sz, i, i, i, i, P, P]),
                    ("moe_combine", [P, i, P, P, sz, i, i, i, i, P, P]),
                    ("moe_dispatch_grad", [P, P, i, P, P, sz, i, i, i, i, P, P, P]),
                    ("moe_combine_grad", [P, P, i, P, P, sz, i, i, i, i, P, P, P]),
                    ("moe_router_topk_grad", [P, P, P, P, i, i, i, i, i, P, P]),
                    ("moe_grouped_linear", [P, P, P, P, i, i, P, sz, i, i, i, i, i, P, P, P]),
                    ("moe_grouped_linear_grad_x", [P, P, P, i, i, P, sz, i, i, i, i, i, P, P]),
                    ("moe_grouped_linear_grad_w", [P, P, i, i, i, P, sz, i, i, i, i, i, P, P, P]),
                    ("moe_grouped_act_grad", [P, P, i, i, P, sz, i, i, i, i, P, P]),
                    ("moe_linear", [P, P, P, P, i, i, i, i, i, P, P, P]),
                    ("moe_linear_grad_x", [P, P, P, i, i, i, i, i, P, P]),
                    ("moe_linear_grad_w", [P, P, i, i, i, i, i, i, P, P, P]),
                    ("moe_act_grad", [P, P, i, i, i, i, P, P])):
        f = getattr(L, n)
        f.restype = r
        f.argtypes = args
    return L


_lib = _load()


def status_string(status: int) -> str:
    return _lib.moe_status_string(int(status)).decode()


def _check(name, rc):
    if rc != 0:
        raise MoeError(name, rc)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def moe_pack_weights(w, dtype="bf16", out=None, stream=None):
    """Packed copy of a row-major [E][rows][cols] weight tensor (bf16; uint8
    e4m3 codes for dtype "fp8", "fp8b" and "mxfp8"; int8 codes for "int8"; uint8 bytes
    of two int4 codes for "int4", whose K length is twice the byte count), as a
    PackedWeight (the packed tensor and its descriptor for the forward calls)."""
    want = {"bf16": torch.bfloat16, "int8": torch.int8, "int8w": torch.int8}.get(dtype, torch.uint8)
    if w.dtype != want or w.dim() != 3 or not w.is_contiguous():
        raise ValueError(f"moe_pack_weights: expected contiguous {want} [E][rows][cols]")
    E, rows, cols = w.shape
    if dtype == "int4":
        cols *= 2
    if out is None:
        out = torch.empty_like(w)
    desc = PackedWeightsDesc()
    _check("moe_pack_weights", _lib.moe_pack_weights(_ptr(w), E, rows, cols, DTYPES[dtype],
                                                     _ptr(out), ctypes.byref(desc), _stream(stream)))
    return PackedWeight(out, desc)


def moe_describe_packed_weights(packed, dtype):
    """PackedWeight for a tensor that already holds packed bytes (a copy of a
    packed tensor, or packed weights loaded from storage); dtype is a name of
    DTYPES or its code."""
    code = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    E, rows, cols = packed.shape
    if code == MOE_DTYPE_INT4_W4A16:
        cols *= 2
    elif code == MOE_DTYPE_MXFP4:
        if cols % 17 or not packed.is_contiguous() or packed.element_size() != 1:
            raise ValueError("moe_describe_packed_weights: packed MXFP4 rows hold cols / 2 + cols / 32 contiguous bytes")
        cols = cols // 17 * 32
    desc = PackedWeightsDesc()
    _check("moe_describe_packed_weights",
           _lib.moe_describe_packed_weights(_ptr(packed), E, rows, cols, code, ctypes.byref(desc)))
    return PackedWeight(packed, desc)


def pack_weights(weights, dtype="bf16", stream=None):
    """Weight dict with w1/w2 packed for the forward calls (scales copied by
    reference; MXFP4: packed with the codes and left out)."""
    out = dict(weights)
    if dtype == "mxfp4":
        for n in ("w1", "w2"):
            out[n] = moe_pack_weights_mxfp4(weights[n], out.pop(n + "_scale"), stream=stream)
        return out
    out["w1"] = moe_pack_weights(weights["w1"], dtype, stream=stream)
    out["w2"] = moe_pack_weights(weights["w2"], dtype, stream=stream)
    return out


def moe_routing_layout(T, k, E, H, I, dtype="bf16") -> dict:
    L = RoutingLayout()
    _check("moe_routing_layout", _lib.moe_routing_layout(T, k, E, H, I, DTYPES[dtype], ctypes.byref(L)))
    return {f: getattr(L, f) for f, _ in RoutingLayout._fields_}


def moe_workspace_layout(T, k, E, H, I, dtype="bf16") -> dict:
    W = WorkspaceLayout()
    _check("moe_workspace_layout", _lib.moe_workspace_layout(T, k, E, H, I, DTYPES[dtype], ctypes.byref(W)))
    return {f: getattr(W, f) for f, _ in WorkspaceLayout._fields_}


def alloc_routing(T, k, E, H, I, dtype="bf16", device="cuda"):
    n = moe_routing_layout(T, k, E, H, I, dtype)["total_bytes"]
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def alloc_workspace(T, k, E, H, I, dtype="bf16", device="cuda"):
    n = moe_workspace_layout(T, k, E, H, I, dtype)["total_bytes"]
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def moe_router_topk(logits, k, renormalize=True, n_shared=0, topk_ids=None, topk_w=None,
                    stream=None):
    """Router top-k of fp32 logits [T][E] into (topk_ids int32, topk_w fp32),
    both [T][k + n_shared]; the last n_shared columns are the fused shared
    experts (ids E.., weight 1)."""
    if logits.dtype != torch.float32 or logits.dim() != 2 or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous fp32 [T][E] tensor")
    T, E = logits.shape
    ncol = k + n_shared
    if topk_ids is None:
        topk_ids = torch.empty(T, ncol, dtype=torch.int32, device=logits.device)
    if topk_w is None:
        topk_w = torch.empty(T, ncol, dtype=torch.float32, device=logits.device)
    _check_tensor("topk_ids", topk_ids, torch.int32, (T, ncol))
    _check_tensor("topk_w", topk_w, torch.float32, (T, ncol))
    _check("moe_router_topk", _lib.moe_router_topk(
        _ptr(logits), T, E, k, int(bool(renormalize)), n_shared, _ptr(topk_ids), _ptr(topk_w),
        _stream(stream)))
    return topk_ids, topk_w


def moe_router_pair_bytes(N, K) -> int:
    n = ctypes.c_size_t()
    _check("moe_router_pair_bytes", _lib.moe_router_pair_bytes(N, K, ctypes.byref(n)))
    return n.value


def moe_router_workspace_bytes(T, N, K) -> int:
    n = ctypes.c_size_t()
    _check("moe_router_workspace_bytes", _lib.moe_router_workspace_bytes(T, N, K, ctypes.byref(n)))
    return n.value


def moe_router_split_weights(w, out=None, stream=None):
    """Split pair (uint8 tensor of moe_router_pair_bytes) of fp32 router weights [N][K]."""
    if w.dtype != torch.float32 or w.dim() != 2 or not w.is_contiguous():
        raise ValueError("w must be a contiguous fp32 [N][K] tensor")
    N, K = w.shape
    nbytes = moe_router_pair_bytes(N, K)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    _check("moe_router_split_weights", _lib.moe_router_split_weights(
        _ptr(w), N, K, _ptr(out), out.numel() * out.element_size(), _stream(stream)))
    return out


def _router_ws(T, N, K, workspace, device):
    n = moe_router_workspace_bytes(T, N, K)
    if workspace is None:
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=device)
    return workspace


def moe_router_gemm(x, w_pair, N, scores=None, workspace=None, stream=None):
    """fp32 scores [T][N] of bf16 x [T][K] against a split router weight pair."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 [T][K] tensor")
    T, K = x.shape
    workspace = _router_ws(T, N, K, workspace, x.device)
    if scores is None:
        scores = torch.empty(T, N, dtype=torch.float32, device=x.device)
    _check_tensor("scores", scores, torch.float32, (T, N))
    _check("moe_router_gemm", _lib.moe_router_gemm(
        _ptr(x), _ptr(w_pair), T, N, K, _ptr(workspace), workspace.numel(), _ptr(scores),
        _stream(stream)))
    return scores


def moe_router_gemm_topk(x, w_pair, E, k, renormalize=True, n_shared=0, want_scores=False,
                         topk_ids=None, topk_w=None, scores=None, workspace=None, stream=None):
    """Router GEMM + top-k: (topk_ids, topk_w) [T][k + n_shared], plus the fp32
    scores [T][E] when want_scores (or a scores tensor is given)."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 [T][K] tensor")
    T, K = x.shape
    ncol = k + n_shared
    workspace = _router_ws(T, E, K, workspace, x.device)
    if topk_ids is None:
        topk_ids = torch.empty(T, ncol, dtype=torch.int32, device=x.device)
    if topk_w is None:
        topk_w = torch.empty(T, ncol, dtype=torch.float32, device=x.device)
    if scores is None and want_scores:
        scores = torch.empty(T, E, dtype=torch.float32, device=x.device)
    if scores is not None:
        _check_tensor("scores", scores, torch.float32, (T, E))
    _check_tensor("topk_ids", topk_ids, torch.int32, (T, ncol))
    _check_tensor("topk_w", topk_w, torch.float32, (T, ncol))
    _check("moe_router_gemm_topk", _lib.moe_router_gemm_topk(
        _ptr(x), _ptr(w_pair), T, E, K, k, int(bool(renormalize)), n_shared, _ptr(workspace),
        workspace.numel(), _ptr(scores), _ptr(topk_ids), _ptr(topk_w), _stream(stream)))
    return (topk_ids, topk_w, scores) if scores is not None else (topk_ids, topk_w)


def _shape_tk(topk_ids):
    if topk_ids.dim() != 2 or topk_ids.dtype != torch.int32 or not topk_ids.is_contiguous():
        raise ValueError("topk_ids must be a contiguous int32 [T][k] tensor")
    return topk_ids.shape


def _build_routing(fn, name, topk_ids, E, H, I, routing, stream):
    T, k = _shape_tk(topk_ids)
    _check(name, fn(_ptr(topk_ids), T, k, E, H, I, _ptr(routing), routing.numel(), _stream(stream)))


def moe_build_routing_bf16(topk_ids, E, H, I, routing, stream=None):
    _build_routing(_lib.moe_build_routing_bf16, "moe_build_routing_bf16", topk_ids, E, H, I, routing, stream)


def moe_build_routing_fp8(topk_ids, E, H, I, routing, stream=None):
    _build_routing(_lib.moe_build_routing_fp8, "moe_build_routing_fp8", topk_ids, E, H, I, routing, stream)


def moe_build_routing_mxfp8(topk_ids, E, H, I, routing, stream=None):
    _build_routing(_lib.moe_build_routing_mxfp8, "moe_build_routing_mxfp8", topk_ids, E, H, I, routing,
                   stream)


def moe_build_routing_int8(topk_ids, E, H, I, routing, stream=None):
    _build_routing(_lib.moe_build_routing_int8, "moe_build_routing_int8", topk_ids, E, H, I, routing,
                   stream)


def moe_build_routing_int4(topk_ids, E, H, I, routing, stream=None):
    _build_routing(_lib.moe_build_routing_int4, "moe_build_routing_int4", topk_ids, E, H, I, routing,
                   stream)


def moe_build_routing_int8_w8a16(topk_ids, E, H, I, routing, stream=None):
    _build_routing(_lib.moe_build_routing_int8_w8a16, "moe_build_routing_int8_w8a16", topk_ids, E, H, I,
                   routing, stream)


def moe_build_routing_fp8_block(topk_ids, E, H, I, routing, stream=None):
    _build_routing(_lib.moe_build_routing_fp8_block, "moe_build_routing_fp8_block", topk_ids, E, H, I,
                   routing, stream)


def build_routing(topk_ids, E, H, I, routing, dtype="bf16", stream=None):
    """The routing build of the given dtype's forward."""
    {"bf16": moe_build_routing_bf16, "fp8": moe_build_routing_fp8,
     "mxfp8": moe_build_routing_mxfp8, "int8": moe_build_routing_int8,
     "int4": moe_build_routing_int4, "fp8b": moe_build_routing_fp8_block,
     "int8w": moe_build_routing_int8_w8a16, "mxfp4": moe_build_routing_mxfp4}[dtype](
        topk_ids, E, H, I, routing, stream)


def _check_tensor(name, t, dtype, shape):
    if isinstance(t, PackedWeight):
        t = t.tensor
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _desc(name, w):
    """The library descriptor of a packed weight (forward calls take nothing else)."""
    if not isinstance(w, PackedWeight):
        raise TypeError(f"{name}: expected a PackedWeight from moe_pack_weights / pack_weights, "
                        f"got {type(w).__name__} (the forward calls take packed weights only)")
    return ctypes.byref(w.desc)


def moe_forward_bf16(x, topk_w, routing, w1, w2, workspace, out, stream=None):
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2, _ = w1.shape
    I = I2 // 2
    _check_tensor("x", x, torch.bfloat16, (T, H))
    _check_tensor("topk_w", topk_w, torch.float32, (T, k))
    _check_tensor("w1", w1, torch.bfloat16, (E, 2 * I, H))
    _check_tensor("w2", w2, torch.bfloat16, (E, H, I))
    _check_tensor("out", out, torch.bfloat16, (T, H))
    _check("moe_forward_bf16", _lib.moe_forward_bf16(
        _ptr(x), _ptr(topk_w), _ptr(routing), _desc("w1", w1), _desc("w2", w2), T, k, E, H, I,
        _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream)))
    return out


def moe_forward_fp8(x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out, stream=None):
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2, _ = w1.shape
    I = I2 // 2
    _check_tensor("x", x, torch.bfloat16, (T, H))
    _check_tensor("topk_w", topk_w, torch.float32, (T, k))
    _check_tensor("w1", w1, torch.uint8, (E, 2 * I, H))
    _check_tensor("w1_scale", w1_scale, torch.float32, (E, 2 * I))
    _check_tensor("w2", w2, torch.uint8, (E, H, I))
    _check_tensor("w2_scale", w2_scale, torch.float32, (E, H))
    _check_tensor("out", out, torch.bfloat16, (T, H))
    _check("moe_forward_fp8", _lib.moe_forward_fp8(
        _ptr(x), _ptr(topk_w), _ptr(routing), _desc("w1", w1), _ptr(w1_scale), _desc("w2", w2), _ptr(w2_scale),
        T, k, E, H, I, _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream)))
    return out


def moe_route_forward_bf16(topk_ids, x, topk_w, routing, w1, w2, workspace, out, stream=None):
    """moe_build_routing_bf16 + moe_forward_bf16 in one call (one token:
    the routing build runs inside the gate-up launch)."""
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2, _ = w1.shape
    I = I2 // 2
    _check_tensor("topk_ids", topk_ids, torch.int32, (T, k))
    _check_tensor("x", x, torch.bfloat16, (T, H))
    _check_tensor("topk_w", topk_w, torch.float32, (T, k))
    _check_tensor("w1", w1, torch.bfloat16, (E, 2 * I, H))
    _check_tensor("w2", w2, torch.bfloat16, (E, H, I))
    _check_tensor("out", out, torch.bfloat16, (T, H))
    _check("moe_route_forward_bf16", _lib.moe_route_forward_bf16(
        _ptr(topk_ids), _ptr(x), _ptr(topk_w), _ptr(routing), routing.numel(), _desc("w1", w1), _desc("w2", w2),
        T, k, E, H, I, _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream)))
    return out


def moe_route_forward_fp8(topk_ids, x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out,
                          stream=None):
    """moe_build_routing_fp8 + moe_forward_fp8 in one call (one token: the
    routing build runs inside the x-quantisation launch)."""
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2, _ = w1.shape
    I = I2 // 2
    _check_tensor("topk_ids", topk_ids, torch.int32, (T, k))
    _check_tensor("x", x, torch.bfloat16, (T, H))
    _check_tensor("topk_w", topk_w, torch.float32, (T, k))
    _check_tensor("w1", w1, torch.uint8, (E, 2 * I, H))
    _check_tensor("w1_scale", w1_scale, torch.float32, (E, 2 * I))
    _check_tensor("w2", w2, torch.uint8, (E, H, I))
    _check_tensor("w2_scale", w2_scale, torch.float32, (E, H))
    _check_tensor("out", out, torch.bfloat16, (T, H))
    _check("moe_route_forward_fp8", _lib.moe_route_forward_fp8(
        _ptr(topk_ids), _ptr(x), _ptr(topk_w), _ptr(routing), routing.numel(), _desc("w1", w1), _ptr(w1_scale),
        _desc("w2", w2), _ptr(w2_scale), T, k, E, H, I, _ptr(workspace), workspace.numel(), _ptr(out),
        _stream(stream)))
    return out


def _route_forward_q(fn, name, topk_ids, x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out,
                     stream, scale_dtype, scale_shape):
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2, _ = w1.shape
    I = I2 // 2
    _check_tensor("topk_ids", topk_ids, torch.int32, (T, k))
    _check_tensor("x", x, torch.bfloat16, (T, H))
    _check_tensor("topk_w", topk_w, torch.float32, (T, k))
    _check_tensor("w1_scale", w1_scale, scale_dtype, scale_shape(E, 2 * I, H))
    _check_tensor("w2_scale", w2_scale, scale_dtype, scale_shape(E, H, I))
    _check_tensor("out", out, torch.bfloat16, (T, H))
    _check(name, fn(_ptr(topk_ids), _ptr(x), _ptr(topk_w), _ptr(routing), routing.numel(), _desc("w1", w1),
                    _ptr(w1_scale), _desc("w2", w2), _ptr(w2_scale), T, k, E, H, I, _ptr(workspace),
                    workspace.numel(), _ptr(out), _stream(stream)))
    return out


def moe_route_forward_int8(topk_ids, x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out,
                           stream=None):
    """moe_build_routing_int8 + moe_forward_int8 in one call."""
    return _route_forward_q(_lib.moe_route_forward_int8, "moe_route_forward_int8", topk_ids, x, topk_w, routing,
                            w1, w1_scale, w2, w2_scale, workspace, out, stream, torch.float32,
                            lambda E, N, K: (E, N))


def moe_route_forward_fp8_block(topk_ids, x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out,
                                stream=None):
    """moe_build_routing_fp8_block + moe_forward_fp8_block in one call."""
    return _route_forward_q(_lib.moe_route_forward_fp8_block, "moe_route_forward_fp8_block", topk_ids, x, topk_w,
                            routing, w1, w1_scale, w2, w2_scale, workspace, out, stream, torch.float32,
                            lambda E, N, K: (E, N // 128, K // 128))


def moe_route_forward_mxfp8(topk_ids, x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out,
                            stream=None):
    """moe_build_routing_mxfp8 + moe_forward_mxfp8 in one call."""
    return _route_forward_q(_lib.moe_route_forward_mxfp8, "moe_route_forward_mxfp8", topk_ids, x, topk_w,
                            routing, w1, w1_scale, w2, w2_scale, workspace, out, stream, torch.uint8,
                            lambda E, N, K: (E, N, K // 32))


def moe_route_forward_int4(topk_ids, x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out,
                           stream=None):
    """moe_build_routing_int4 + moe_forward_int4 in one call."""
    return _route_forward_q(_lib.moe_route_forward_int4, "moe_route_forward_int4", topk_ids, x, topk_w, routing,
                            w1, w1_scale, w2, w2_scale, workspace, out, stream, torch.float32,
                            lambda E, N, K: (E, N, K // 128))


def moe_route_forward_int8_w8a16(topk_ids, x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out,
                                 stream=None):
    """moe_build_routing_int8_w8a16 + moe_forward_int8_w8a16 in one call."""
    return _route_forward_q(_lib.moe_route_forward_int8_w8a16, "moe_route_forward_int8_w8a16", topk_ids, x,
                            topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out, stream, torch.float32,
                            lambda E, N, K: (E, N))


def route_forward(topk_ids, x, topk_w, routing, weights, workspace, out, dtype="bf16", stream=None):
    """Routing build + forward in one library call, any dtype."""
    W = weights
    if dtype == "bf16":
        return moe_route_forward_bf16(topk_ids, x, topk_w, routing, W["w1"], W["w2"], workspace, out, stream)
    if dtype == "mxfp4":
        return moe_route_forward_mxfp4(topk_ids, x, topk_w, routing, W["w1"], W["w2"], workspace, out, stream)
    fn = {"fp8": moe_route_forward_fp8, "int8": moe_route_forward_int8, "fp8b": moe_route_forward_fp8_block,
          "mxfp8": moe_route_forward_mxfp8, "int4": moe_route_forward_int4,
          "int8w": moe_route_forward_int8_w8a16}[dtype]
    return fn(topk_ids, x, topk_w, routing, W["w1"], W["w1_scale"], W["w2"], W["w2_scale"], workspace, out, stream)


STATIC_WORKSPACE_BYTES = 64 << 20


def moe_forward_fp8_noalloc(x, topk_w, routing, w1, w1_scale, w2, w2_scale, out, stream=None):
    """moe_forward_fp8 on the library's fixed per-GPU workspace (no workspace
    argument, nothing allocated); sizes whose workspace exceeds
    STATIC_WORKSPACE_BYTES raise MoeError (MOE_ERR_BUFFER_TOO_SMALL)."""
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2, _ = w1.shape
    I = I2 // 2
    _check_tensor("x", x, torch.bfloat16, (T, H))
    _check_tensor("topk_w", topk_w, torch.float32, (T, k))
    _check_tensor("w1", w1, torch.uint8, (E, 2 * I, H))
    _check_tensor("w1_scale", w1_scale, torch.float32, (E, 2 * I))
    _check_tensor("w2", w2, torch.uint8, (E, H, I))
    _check_tensor("w2_scale", w2_scale, torch.float32, (E, H))
    _check_tensor("out", out, torch.bfloat16, (T, H))
    _check("moe_forward_fp8_noalloc", _lib.moe_forward_fp8_noalloc(
        _ptr(x), _ptr(topk_w), _ptr(routing), _desc("w1", w1), _ptr(w1_scale), _desc("w2", w2),
        _ptr(w2_scale), T, k, E, H, I, _ptr(out), _stream(stream)))
    return out


def moe_forward_mxfp8(x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out, stream=None):
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2, _ = w1.shape
    I = I2 // 2
    _check_tensor("x", x, torch.bfloat16, (T, H))
    _check_tensor("topk_w", topk_w, torch.float32, (T, k))
    _check_tensor("w1", w1, torch.uint8, (E, 2 * I, H))
    _check_tensor("w1_scale", w1_scale, torch.uint8, (E, 2 * I, H // 32))
    _check_tensor("w2", w2, torch.uint8, (E, H, I))
    _check_tensor("w2_scale", w2_scale, torch.uint8, (E, H, I // 32))
    _check_tensor("out", out, torch.bfloat16, (T, H))
    _check("moe_forward_mxfp8", _lib.moe_forward_mxfp8(
        _ptr(x), _ptr(topk_w), _ptr(routing), _desc("w1", w1), _ptr(w1_scale), _desc("w2", w2), _ptr(w2_scale),
        T, k, E, H, I, _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream)))
    return out


def moe_forward_fp8_block(x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out, stream=None):
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2, _ = w1.shape
    I = I2 // 2
    _check_tensor("x", x, torch.bfloat16, (T, H))
    _check_tensor("topk_w", topk_w, torch.float32, (T, k))
    _check_tensor("w1", w1, torch.uint8, (E, 2 * I, H))
    _check_tensor("w1_scale", w1_scale, torch.float32, (E, 2 * I // 128, H // 128))
    _check_tensor("w2", w2, torch.uint8, (E, H, I))
    _check_tensor("w2_scale", w2_scale, torch.float32, (E, H // 128, I // 128))
    _check_tensor("out", out, torch.bfloat16, (T, H))
    _check("moe_forward_fp8_block", _lib.moe_forward_fp8_block(
        _ptr(x), _ptr(topk_w), _ptr(routing), _desc("w1", w1), _ptr(w1_scale), _desc("w2", w2), _ptr(w2_scale),
        T, k, E, H, I, _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream)))
    return out


def moe_forward_int8_w8a16(x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out, stream=None):
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2, _ = w1.shape
    I = I2 // 2
    _check_tensor("x", x, torch.bfloat16, (T, H))
    _check_tensor("topk_w", topk_w, torch.float32, (T, k))
    _check_tensor("w1", w1, torch.int8, (E, 2 * I, H))
    _check_tensor("w1_scale", w1_scale, torch.float32, (E, 2 * I))
    _check_tensor("w2", w2, torch.int8, (E, H, I))
    _check_tensor("w2_scale", w2_scale, torch.float32, (E, H))
    _check_tensor("out", out, torch.bfloat16, (T, H))
    _check("moe_forward_int8_w8a16", _lib.moe_forward_int8_w8a16(
        _ptr(x), _ptr(topk_w), _ptr(routing), _desc("w1", w1), _ptr(w1_scale), _desc("w2", w2), _ptr(w2_scale),
        T, k, E, H, I, _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream)))
    return out


def moe_forward_int4(x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out, stream=None):
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2, _ = w1.shape
    I = I2 // 2
    _check_tensor("x", x, torch.bfloat16, (T, H))
    _check_tensor("topk_w", topk_w, torch.float32, (T, k))
    _check_tensor("w1", w1, torch.uint8, (E, 2 * I, H // 2))
    _check_tensor("w1_scale", w1_scale, torch.float32, (E, 2 * I, H // 128))
    _check_tensor("w2", w2, torch.uint8, (E, H, I // 2))
    _check_tensor("w2_scale", w2_scale, torch.float32, (E, H, I // 128))
    _check_tensor("out", out, torch.bfloat16, (T, H))
    _check("moe_forward_int4", _lib.moe_forward_int4(
        _ptr(x), _ptr(topk_w), _ptr(routing), _desc("w1", w1), _ptr(w1_scale), _desc("w2", w2), _ptr(w2_scale),
        T, k, E, H, I, _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream)))
    return out


def moe_forward_int8(x, topk_w, routing, w1, w1_scale, w2, w2_scale, workspace, out, stream=None):
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2, _ = w1.shape
    I = I2 // 2
    _check_tensor("x", x, torch.bfloat16, (T, H))
    _check_tensor("topk_w", topk_w, torch.float32, (T, k))
    _check_tensor("w1", w1, torch.int8, (E, 2 * I, H))
    _check_tensor("w1_scale", w1_scale, torch.float32, (E, 2 * I))
    _check_tensor("w2", w2, torch.int8, (E, H, I))
    _check_tensor("w2_scale", w2_scale, torch.float32, (E, H))
    _check_tensor("out", out, torch.bfloat16, (T, H))
    _check("moe_forward_int8", _lib.moe_forward_int8(
        _ptr(x), _ptr(topk_w), _ptr(routing), _desc("w1", w1), _ptr(w1_scale), _desc("w2", w2), _ptr(w2_scale),
        T, k, E, H, I, _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream)))
    return out


def _check_device(*tensors):
    """Every given tensor (None: left out) is on the current GPU: a kernel
    cannot take host memory, and a launch goes to the current device's streams."""
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else 0
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"expected tensors on the current GPU, got one of shape {tuple(t.shape)} on {t.device}")
    return dev


def _bytes(name, t):
    """Bytes of a routing buffer or workspace, which the library takes as one run."""
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous buffer, got strides {t.stride()}")
    return t.nbytes


def _here(dev, stream):
    """The hipStream_t of `stream`, which has to be device dev's, or of its current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream: expected one of GPU {dev}, got one of GPU {stream.device_index}")
    return stream.cuda_stream


def _is(name, t, dtype, shape):
    """_check_tensor for the short calls: no conversions where all is well."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _check_tensor(name, t, dtype, shape)


def _at(t):
    return None if t is None else t.data_ptr()


def _empty(like, shape, dtype, stream):
    """An output beside `like`, allocated for use on `stream` (None: the current stream)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _output(name, t, like, shape, dtype, stream):
    """The caller's output t, checked, or a new one."""
    if t is None:
        return _empty(like, shape, dtype, stream)
    _is(name, t, dtype, shape)
    return t


def _row_type(name, t):
    if t.dtype not in ROW_TYPES:
        raise ValueError(f"{name}: expected bf16, fp16 or fp32 rows, got {t.dtype}")
    return ROW_TYPES[t.dtype]


def moe_quantize_mxfp4(x, codes=None, scales=None, stream=None):
    """MXFP4 of rows x [..., cols] (bf16, fp16 or fp32; contiguous, or 2-D with
    contiguous rows apart by x.stride(0)): (codes uint8 [..., cols / 2], scales
    uint8 [..., cols / 32]).  A block that holds Inf or NaN becomes NaN."""
    kind = _row_type("x", x)
    *lead, cols = x.shape or (0,)
    if cols % 32 or cols == 0:
        raise ValueError(f"x: expected rows of a multiple of 32 values, got {tuple(x.shape)}")
    stride = cols
    if not x.is_contiguous():
        if x.dim() != 2 or x.stride(1) != 1 or x.stride(0) < cols:
            raise ValueError(f"x: expected contiguous rows, got strides {x.stride()}")
        stride = x.stride(0)
    dev = _check_device(x, codes, scales)
    codes = _output("codes", codes, x, (*lead, cols // 2), torch.uint8, stream)
    scales = _output("scales", scales, x, (*lead, cols // 32), torch.uint8, stream)
    _check("moe_quantize_mxfp4", _lib.moe_quantize_mxfp4(
        x.data_ptr(), kind, x.numel() // cols, cols, stride, codes.data_ptr(), scales.data_ptr(), _here(dev, stream)))
    return codes, scales


def moe_dequantize_mxfp4(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """Values [..., cols] (bf16, fp16 or fp32) of MXFP4 codes [..., cols / 2] and
    scale codes [..., cols / 32]."""
    if codes.dim() < 1 or codes.shape[-1] % 16 or codes.shape[-1] == 0:
        raise ValueError(f"codes: expected rows of a multiple of 16 bytes, got {tuple(codes.shape)}")
    *lead, half = codes.shape
    cols = 2 * half
    _is("codes", codes, torch.uint8, codes.shape)
    _is("scales", scales, torch.uint8, (*lead, cols // 32))
    dev = _check_device(codes, scales, out)
    out = _output("out", out, codes, (*lead, cols), dtype if out is None else out.dtype, stream)
    kind = _row_type("out", out)
    _check("moe_dequantize_mxfp4", _lib.moe_dequantize_mxfp4(
        codes.data_ptr(), scales.data_ptr(), out.numel() // cols, cols, kind, out.data_ptr(), _here(dev, stream)))
    return out


def moe_pack_weights_mxfp4(codes, scales, out=None, stream=None):
    """PackedWeight of row-major MXFP4 weights: codes uint8 [E][rows][cols / 2]
    and scale codes uint8 [E][rows][cols / 32]."""
    if codes.dim() != 3:
        raise ValueError(f"codes: expected [E][rows][cols / 2], got {tuple(codes.shape)}")
    E, rows, cols = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
    _check_tensor("codes", codes, torch.uint8, (E, rows, cols // 2))
    _check_tensor("scales", scales, torch.uint8, (E, rows, cols // 32))
    if out is None:
        out = _empty(codes, (E, rows, cols // 2 + cols // 32), torch.uint8, stream)
    _check_tensor("out", out, torch.uint8, (E, rows, cols // 2 + cols // 32))
    dev = _check_device(codes, scales, out)
    desc = PackedWeightsDesc()
    _check("moe_pack_weights_mxfp4", _lib.moe_pack_weights_mxfp4(
        _ptr(codes), _ptr(scales), E, rows, cols, _ptr(out), ctypes.byref(desc), _here(dev, stream)))
    return PackedWeight(out, desc)


def moe_build_routing_mxfp4(topk_ids, E, H, I, routing, stream=None):
    _here(_check_device(topk_ids, routing), stream)
    _bytes("routing", routing)
    _build_routing(_lib.moe_build_routing_mxfp4, "moe_build_routing_mxfp4", topk_ids, E, H, I, routing, stream)


def _mxfp4_sizes(x, topk_w, w1, w2, routing, workspace, out, topk_ids=None):
    """(T, k, E, H, I), the weights' descriptors and the device of an MXFP4
    forward call, its tensors checked."""
    T, H = x.shape
    k = topk_w.shape[1]
    E, I2 = w1.shape[:2]
    I = I2 // 2
    d1, d2 = _desc("w1", w1), _desc("w2", w2)
    _is("x", x, torch.bfloat16, (T, H))
    _is("topk_w", topk_w, torch.float32, (T, k))
    _is("w1", w1.tensor, torch.uint8, (E, 2 * I, H // 2 + H // 32))
    _is("w2", w2.tensor, torch.uint8, (E, H, I // 2 + I // 32))
    _is("out", out, torch.bfloat16, (T, H))
    dev = _check_device(x, topk_w, w1.tensor, w2.tensor, routing, workspace, out, topk_ids)
    return (T, k, E, H, I), (d1, d2), dev


def moe_forward_mxfp4(x, topk_w, routing, w1, w2, workspace, out, stream=None):
    sizes, desc, dev = _mxfp4_sizes(x, topk_w, w1, w2, routing, workspace, out)
    _check("moe_forward_mxfp4", _lib.moe_forward_mxfp4(
        x.data_ptr(), topk_w.data_ptr(), routing.data_ptr(), *desc, *sizes, workspace.data_ptr(),
        _bytes("workspace", workspace), out.data_ptr(), _here(dev, stream)))
    return out


def moe_route_forward_mxfp4(topk_ids, x, topk_w, routing, w1, w2, workspace, out, stream=None):
    """moe_build_routing_mxfp4 + moe_forward_mxfp4 in one call."""
    sizes, desc, dev = _mxfp4_sizes(x, topk_w, w1, w2, routing, workspace, out, topk_ids)
    _is("topk_ids", topk_ids, torch.int32, sizes[:2])
    _check("moe_route_forward_mxfp4", _lib.moe_route_forward_mxfp4(
        topk_ids.data_ptr(), x.data_ptr(), topk_w.data_ptr(), routing.data_ptr(),
        _bytes("routing", routing), *desc, *sizes, workspace.data_ptr(), _bytes("workspace", workspace),
        out.data_ptr(), _here(dev, stream)))
    return out


def _rows(name, t, k, sorted_rows):
    """(T, H) of token rows [T][H], or of sorted rows [T * k][H]."""
    if k < 1 or t.dim() != 2 or (sorted_rows and t.shape[0] % k):
        raise ValueError(f"{name}: expected {'[T * k]' if sorted_rows else '[T]'}[H] rows, got {tuple(t.shape)}, k = {k}")
    return (t.shape[0] // k if sorted_rows else t.shape[0]), t.shape[1]


def _move(name, fn, src, src_name, sorted_src, routing, k, E, topk_w, out, out_name, stream):
    kind = _row_type(src_name, src)
    T, H = _rows(src_name, src, k, sorted_src)
    _is(src_name, src, src.dtype, src.shape)
    if topk_w is not None:
        _is("topk_w", topk_w, torch.float32, (T, k))
    dev = _check_device(src, out, topk_w, routing)
    out = _output(out_name, out, src, (T, H) if sorted_src else (T * k, H), src.dtype, stream)
    _check(name, fn(src.data_ptr(), kind, _at(topk_w), routing.data_ptr(), _bytes("routing", routing),
                    T, k, E, H, out.data_ptr(), _here(dev, stream)))
    return out


def moe_dispatch(x, routing, k, E, topk_w=None, out=None, stream=None):
    """Token rows x [T][H] (bf16, fp16 or fp32) to expert order: out [T * k][H],
    row r the (weighted) token of the pair sorted there.  Rows behind the last
    valid pair are not written."""
    return _move("moe_dispatch", _lib.moe_dispatch, x, "x", False, routing, k, E, topk_w, out, "out", stream)


def moe_combine(y, routing, k, E, topk_w=None, out=None, stream=None):
    """Rows y [T * k][H] in expert order back to token order: out [T][H], the
    (weighted) sum of each token's valid pairs."""
    return _move("moe_combine", _lib.moe_combine, y, "y", True, routing, k, E, topk_w, out, "out", stream)


def _move_grad(name, fn, grad, grad_name, sorted_grad, other, other_name, routing, k, E, topk_w, out, out_name, dw, stream):
    if dw is not None and other is None:
        raise ValueError(f"{name}: dtopk_w needs {other_name}")
    if other is not None and topk_w is None:
        raise ValueError(f"{name}: the gradient of topk_w needs topk_w")
    kind = _row_type(grad_name, grad)
    T, H = _rows(grad_name, grad, k, sorted_grad)
    shape = (T, H) if sorted_grad else (T * k, H)
    _is(grad_name, grad, grad.dtype, grad.shape)
    if topk_w is not None:
        _is("topk_w", topk_w, torch.float32, (T, k))
    if other is not None:
        _is(other_name, other, grad.dtype, shape)
    dev = _check_device(grad, out, other, topk_w, dw, routing)
    out = _output(out_name, out, grad, shape, grad.dtype, stream)
    if other is not None:
        dw = _output("dtopk_w", dw, grad, (T, k), torch.float32, stream)
    _check(name, fn(grad.data_ptr(), _at(other), kind, _at(topk_w), routing.data_ptr(),
                    _bytes("routing", routing), T, k, E, H, out.data_ptr(), _at(dw), _here(dev, stream)))
    return out if dw is None else (out, dw)


def moe_dispatch_grad(dxs, routing, k, E, x=None, topk_w=None, dx=None, dtopk_w=None, stream=None):
    """Gradient of moe_dispatch: dx [T][H] from dxs [T * k][H] (topk_w as in the
    forward call); with the forward's x also the weights' gradient: (dx, dtopk_w)."""
    return _move_grad("moe_dispatch_grad", _lib.moe_dispatch_grad, dxs, "dxs", True, x, "x", routing, k, E, topk_w, dx,
                      "dx", dtopk_w, stream)


def moe_combine_grad(dout, routing, k, E, y=None, topk_w=None, dy=None, dtopk_w=None, stream=None):
    """Gradient of moe_combine: dy [T * k][H] from dout [T][H] (topk_w as in the
    forward call; rows behind the last valid pair are not written); with the
    forward's y also the weights' gradient: (dy, dtopk_w)."""
    return _move_grad("moe_combine_grad", _lib.moe_combine_grad, dout, "dout", False, y, "y", routing, k, E, topk_w, dy,
                      "dy", dtopk_w, stream)


def moe_router_topk_grad(logits, topk_ids, topk_w, dtopk_w, renormalize=True, n_shared=0, dlogits=None, stream=None):
    """Gradient of moe_router_topk's scores, fp32 [T][E], from that of its
    weights (topk_ids, topk_w, dtopk_w: [T][k + n_shared])."""
    if logits.dim() != 2 or topk_ids.dim() != 2:
        raise ValueError("logits must be [T][E], topk_ids [T][k + n_shared]")
    T, E = logits.shape
    pairs = topk_ids.shape
    _is("logits", logits, torch.float32, logits.shape)
    _is("topk_ids", topk_ids, torch.int32, pairs)
    if pairs[0] != T:
        raise ValueError(f"topk_ids: expected {T} tokens, got {pairs[0]}")
    _is("topk_w", topk_w, torch.float32, pairs)
    _is("dtopk_w", dtopk_w, torch.float32, pairs)
    dev = _check_device(logits, topk_ids, topk_w, dtopk_w, dlogits)
    dlogits = _output("dlogits", dlogits, logits, logits.shape, torch.float32, stream)
    _check("moe_router_topk_grad", _lib.moe_router_topk_grad(
        logits.data_ptr(), topk_ids.data_ptr(), topk_w.data_ptr(), dtopk_w.data_ptr(), T, E, pairs[1] - n_shared,
        1 if renormalize else 0, n_shared, dlogits.data_ptr(), _here(dev, stream)))
    return dlogits


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act: expected one of {', '.join(ACTS)}, got {act!r}")
    return ACTS[act]


def _linear_type(name, t):
    """Row type of a linear layer's rows: bf16 or fp16."""
    kind = ROW_TYPES.get(t.dtype, 2)
    if kind == 2:
        raise ValueError(f"{name}: expected bf16 or fp16 rows, got {t.dtype}")
    return kind


def _two(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected [rows][values], got {tuple(t.shape)}")
    return t.shape


def _matrices(w, grouped):
    """(E, N, K) of the experts' matrices, or of the one of plain rows."""
    if w.dim() != (3 if grouped else 2):
        raise ValueError(f"w: expected {'[E][N][K]' if grouped else '[N][K]'}, got {tuple(w.shape)}")
    return w.shape if grouped else (1, *w.shape)


def _groups(R, k, routing):
    """The routing arguments of a grouped call up to T and k; none for plain rows."""
    if routing is None:
        return ()
    if k < 1 or R % k:
        raise ValueError(f"expected T * k rows, got {R} with k = {k}")
    return routing.data_ptr(), _bytes("routing", routing), R // k, k


def _linear(name, fn, x, x_name, w, routing, k, bias, act, residual, want_z, z, out, stream):
    code, kind = _act(act), _linear_type(x_name, x)
    E, N, K = _matrices(w, routing is not None)
    R = _two(x_name, x)[0]
    M = N // 2 if code == 3 else N
    _is(x_name, x, x.dtype, (R, K))
    _is("w", w, x.dtype, w.shape)
    if bias is not None:
        _is("bias", bias, x.dtype, w.shape[:-1])
    if residual is not None:
        _is("residual", residual, x.dtype, (R, M))
    dev = _check_device(x, w, bias, residual, z, out, routing)
    groups = _groups(R, k, routing)
    out = _output("out", out, x, (R, M), x.dtype, stream)
    if want_z or z is not None:
        z = _output("z", z, x, (R, N), x.dtype, stream)
    sizes = (*groups, E, N, K) if groups else (R, N, K)
    _check(name, fn(x.data_ptr(), w.data_ptr(), _at(bias), _at(residual), kind, code, *sizes, _at(z), out.data_ptr(),
                    _here(dev, stream)))
    return out if z is None else (out, z)


def moe_grouped_linear(xs, w, routing, k, bias=None, act="none", residual=None, want_z=False, z=None, out=None,
                       stream=None):
    """residual + act(xs w^T + bias) of rows xs [T * k][K] in expert order (bf16 or
    fp16) with their experts' matrices w [E][N][K] and biases [E][N]: [T * k][N]
    (act "swiglu": [T * k][N / 2]).  With want_z or z also the sums before the
    activation, [T * k][N], which the gradients take: (out, z).  Rows behind the last
    valid pair are not written; residual may be out."""
    return _linear("moe_grouped_linear", _lib.moe_grouped_linear, xs, "xs", w, routing, k, bias, act, residual, want_z,
                   z, out, stream)


def moe_linear(x, w, bias=None, act="none", residual=None, want_z=False, z=None, out=None, stream=None):
    """moe_grouped_linear of plain rows x [rows][K] with one matrix w [N][K] (bias [N])."""
    return _linear("moe_linear", _lib.moe_linear, x, "x", w, None, 1, bias, act, residual, want_z, z, out, stream)


def _linear_grad_x(name, fn, dy, w, routing, k, z, act, dx, stream):
    code, kind = _act(act), _linear_type("dy", dy)
    E, N, K = _matrices(w, routing is not None)
    R = _two("dy", dy)[0]
    Z = 2 * K if code == 3 else K
    _is("dy", dy, dy.dtype, (R, N))
    _is("w", w, dy.dtype, w.shape)
    if (z is None) != (code == 0):
        raise ValueError(f"{name}: z goes with an activation, got act {act!r} {'without' if z is None else 'and'} z")
    if z is not None:
        _is("z", z, dy.dtype, (R, Z))
    dev = _check_device(dy, w, z, dx, routing)
    groups = _groups(R, k, routing)
    dx = _output("dx", dx, dy, (R, Z), dy.dtype, stream)
    sizes = (*groups, E, N, K) if groups else (R, N, K)
    _check(name, fn(dy.data_ptr(), w.data_ptr(), _at(z), kind, code, *sizes, dx.data_ptr(), _here(dev, stream)))
    return dx


def moe_grouped_linear_grad_x(dy, w, routing, k, z=None, act="none", dx=None, stream=None):
    """Gradient of moe_grouped_linear's rows, dx [T * k][K], from dy [T * k][N], the
    gradient of its sums.  With act and z, the pre-activation of the product whose
    output those rows were: the gradient of that z ([T * k][K], "swiglu": [T * k][2K])."""
    return _linear_grad_x("moe_grouped_linear_grad_x", _lib.moe_grouped_linear_grad_x, dy, w, routing, k, z, act, dx, stream)


def moe_linear_grad_x(dy, w, z=None, act="none", dx=None, stream=None):
    """moe_grouped_linear_grad_x of plain rows with one matrix w [N][K]."""
    return _linear_grad_x("moe_linear_grad_x", _lib.moe_linear_grad_x, dy, w, None, 1, z, act, dx, stream)


def _linear_grad_w(name, fn, dy, x, x_name, routing, k, E, want_bias, dw, dbias, dtype, accumulate, stream):
    kind = _linear_type("dy", dy)
    (R, N), K = _two("dy", dy), _two(x_name, x)[1]
    _is("dy", dy, dy.dtype, dy.shape)
    _is(x_name, x, dy.dtype, (R, K))
    if dtype is None:
        dtype = dw.dtype if dw is not None else dy.dtype
    if dtype not in (dy.dtype, torch.float32):
        raise ValueError(f"dtype: expected {dy.dtype} or torch.float32, got {dtype}")
    want_bias = want_bias or dbias is not None
    if accumulate and (dw is None or (want_bias and dbias is None)):
        raise ValueError(f"{name}: accumulate adds to the dw and dbias that it is given")
    lead = () if routing is None else (E,)
    dev = _check_device(dy, x, dw, dbias, routing)
    groups = _groups(R, k, routing)
    dw = _output("dw", dw, dy, (*lead, N, K), dtype, stream)
    if want_bias:
        dbias = _output("dbias", dbias, dy, (*lead, N), dtype, stream)
    sizes = (*groups, E, N, K) if groups else (R, N, K)
    _check(name, fn(dy.data_ptr(), x.data_ptr(), kind, ROW_TYPES[dtype], 1 if accumulate else 0, *sizes, dw.data_ptr(),
                    _at(dbias), _here(dev, stream)))
    return dw if dbias is None else (dw, dbias)


def moe_grouped_linear_grad_w(dy, xs, routing, k, E, want_bias=False, dw=None, dbias=None, dtype=None, accumulate=False,
                              stream=None):
    """Gradient of moe_grouped_linear's matrices, dw [E][N][K], from dy [T * k][N] and
    the rows xs [T * k][K]; with want_bias or dbias also the biases': (dw, dbias).
    dtype: the rows' own (or dw's) or torch.float32; accumulate adds to dw and dbias."""
    return _linear_grad_w("moe_grouped_linear_grad_w", _lib.moe_grouped_linear_grad_w, dy, xs, "xs", routing, k, E,
                          want_bias, dw, dbias, dtype, accumulate, stream)


def moe_linear_grad_w(dy, x, want_bias=False, dw=None, dbias=None, dtype=None, accumulate=False, stream=None):
    """moe_grouped_linear_grad_w of plain rows: dw [N][K], dbias [N]."""
    return _linear_grad_w("moe_linear_grad_w", _lib.moe_linear_grad_w, dy, x, "x", None, 1, 1, want_bias, dw, dbias,
                          dtype, accumulate, stream)


def _act_grad(name, fn, dy, z, routing, k, E, act, dz, stream):
    code, kind = _act(act), _linear_type("dy", dy)
    R, M = _two("dy", dy)
    shape = (R, 2 * M if code == 3 else M)
    _is("dy", dy, dy.dtype, dy.shape)
    _is("z", z, dy.dtype, shape)
    dev = _check_device(dy, z, dz, routing)
    groups = _groups(R, k, routing)
    dz = _output("dz", dz, dy, shape, dy.dtype, stream)
    sizes = (*groups, E, M) if groups else (R, M)
    _check(name, fn(dy.data_ptr(), z.data_ptr(), kind, code, *sizes, dz.data_ptr(), _here(dev, stream)))
    return dz


def moe_grouped_act_grad(dy, z, routing, k, E, act, dz=None, stream=None):
    """Gradient of an activation's argument z from that of its value, dy [T * k][M];
    z and dz [T * k][M] ("swiglu": [T * k][2M]).  Rows behind the last valid pair are
    not written."""
    return _act_grad("moe_grouped_act_grad", _lib.moe_grouped_act_grad, dy, z, routing, k, E, act, dz, stream)


def moe_act_grad(dy, z, act, dz=None, stream=None):
    """moe_grouped_act_grad of plain rows."""
    return _act_grad("moe_act_grad", _lib.moe_act_grad, dy, z, None, 1, 1, act, dz, stream)


def moe_set_stage_events(events):
    """events: list of 10 entries, each a torch.cuda.Event(enable_timing=True)
    (already recorded once) or None (stage s is recorded when entries 2s and
    2s+1 are events), or None to switch the hook off."""
    if events is None:
        _check("moe_set_stage_events", _lib.moe_set_stage_events(None, 0))
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event if e is not None else None
                                             for e in events])
    _check("moe_set_stage_events", _lib.moe_set_stage_events(arr, len(events)))


def moe_device_cu_count() -> int:
    n = _lib.moe_device_cu_count()
    if n < 0:
        raise MoeError("moe_device_cu_count", n)
    return n


def moe_stream_read(buf, sink, stream=None):
    """Measurement aid: one streaming read of the device tensor `buf` (its
    whole storage) into per-workgroup words of the uint32/int32 tensor `sink`."""
    nbytes = buf.numel() * buf.element_size()
    _check("moe_stream_read", _lib.moe_stream_read(_ptr(buf), nbytes, _ptr(sink), sink.numel(),
                                                   _stream(stream)))


def moe_tile_copy_read(pattern, buf, row_bytes, reps, sink, stream=None):
    """Measurement aid: token-tile copies into LDS in one of three lane
    patterns (0 contiguous, 1 MFMA lane order, 2 a row per lane quad) from the
    device tensor `buf` (its whole storage); one word per workgroup into the
    uint32/int32 tensor `sink`."""
    nbytes = buf.numel() * buf.element_size()
    _check("moe_tile_copy_read", _lib.moe_tile_copy_read(pattern, _ptr(buf), nbytes, row_bytes, reps, _ptr(sink),
                                                         sink.numel(), _stream(stream)))


def moe_layer(x, topk_ids, topk_w, weights, dtype="bf16", out=None, stream=None):
    """Routing + forward with freshly allocated routing buffer and workspace.

    weights: {"w1", "w2"} (bf16, mxfp4) or {"w1", "w1_scale", "w2", "w2_scale"} (fp8),
    with w1/w2 already packed (pack_weights).  Returns (out, routing, workspace)."""
    T, H = x.shape
    k = topk_ids.shape[1]
    E, I2, _ = weights["w1"].shape
    I = I2 // 2
    routing = alloc_routing(T, k, E, H, I, dtype, x.device)
    ws = alloc_workspace(T, k, E, H, I, dtype, x.device)
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
    build_routing(topk_ids, E, H, I, routing, dtype, stream)
    if dtype == "bf16":
        moe_forward_bf16(x, topk_w, routing, weights["w1"], weights["w2"], ws, out, stream)
    elif dtype == "mxfp4":
        moe_forward_mxfp4(x, topk_w, routing, weights["w1"], weights["w2"], ws, out, stream)
    else:
        fwd = {"fp8": moe_forward_fp8, "mxfp8": moe_forward_mxfp8, "int8": moe_forward_int8,
               "int4": moe_forward_int4, "fp8b": moe_forward_fp8_block,
               "int8w": moe_forward_int8_w8a16}[dtype]
        fwd(x, topk_w, routing, weights["w1"], weights["w1_scale"], weights["w2"],
            weights["w2_scale"], ws, out, stream)
    return out, routing, ws


def read_routing(routing, T, k, E, H, I, dtype="bf16") -> dict:
    """Copy a routing buffer's parts to host int32 tensors (for tests and tools)."""
    L = moe_routing_layout(T, k, E, H, I, dtype)
    b = routing.cpu()
    P = T * k

    def part(off, n):
        return b[off:off + 4 * n].view(torch.int32).clone()

    hdr = part(L["header"], 16)
    nt = int(hdr[0])
    return {"header": hdr, "num_tasks": nt, "num_dropped": int(hdr[1]), "block_m": int(hdr[2]),
            "offsets": part(L["expert_offsets"], E + 1), "sorted": part(L["sorted_pairs"], P),
            "pos": part(L["pair_pos"], P), "tasks": part(L["tasks"], 4 * nt).view(nt, 4),
            "layout": L}
