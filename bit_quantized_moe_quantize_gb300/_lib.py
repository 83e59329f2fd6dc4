"""ctypes binding of libft_moe.so: argument marshalling only.

Every function here checks tensor dtypes, devices and shapes, then passes raw
device pointers and the current CUDA stream to the C ABI declared in
``include/ft_moe.h``.  No arithmetic of the routed matmul happens in Python,
and there is no fallback: if the library is missing or was built from other
sources, loading raises.
"""

from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libft_moe.so")

FT_OK, FT_ERR_ARG, FT_ERR_SIZE, FT_ERR_ALIGN, FT_ERR_LAUNCH, FT_ERR_WORKSPACE, FT_ERR_CUDA, FT_ERR_DEVICE_FLAG = range(8)
STATUS_NAMES = {0: "FT_OK", 1: "FT_ERR_ARG", 2: "FT_ERR_SIZE", 3: "FT_ERR_ALIGN", 4: "FT_ERR_LAUNCH",
                5: "FT_ERR_WORKSPACE", 6: "FT_ERR_CUDA", 7: "FT_ERR_DEVICE_FLAG"}
FT_DEVERR_BAD_EXPERT_ID = 0x1
FT_DEVERR_WAIT_TIMEOUT = 0x2
FT_DEVERR_WORKSPACE_GUARD = 0x4
FT_PATH_AUTO, FT_PATH_GEMV, FT_PATH_GEMM, FT_PATH_GEMV_DP4A = 0, 1, 2, 3
PATHS = {"auto": FT_PATH_AUTO, "gemv": FT_PATH_GEMV, "gemm": FT_PATH_GEMM, "gemv_dp4a": FT_PATH_GEMV_DP4A}

EXPORTS = ("ft_quantize_q8_1", "ft_moe_route_offsets", "ft_moe_q4_0_q8_1", "ft_moe_workspace_bytes",
           "ft_moe_reserve", "ft_moe_release", "ft_moe_read_device_error", "ft_moe_set_path",
           "ft_moe_selected_path", "ft_moe_gguf_selected_path", "ft_moe_block_dots", "ft_last_error", "ft_abi_version", "ft_profile_enable",
           "ft_profile_read", "ft_moe_route_offsets_noalloc", "ft_moe_q4_0_q8_1_slots",
           "ft_moe_q4_0_q8_1_ep", "ft_act_mul_quantize_q8_1", "ft_moe_ffn_q4_0_q8_1", "ft_moe_gguf_q8_1",
           "ft_repack_q4_0_soa", "ft_debug_wait_timeout", "ft_moe_q4_0_q8_1_act", "ft_moe_ffn_reserve",
           "ft_moe_q4_0_fp16", "ft_debug_stream_read", "ft_moe_gate", "ft_quantize_fp8", "ft_act_mul_quantize_fp8",
           "ft_moe_fp8_workspace_bytes", "ft_moe_fp8_fp8", "ft_moe_fp8_fp8_slots", "ft_matmul_fp8_fp8",
           "ft_moe_combine", "ft_moe_layer_fp8_workspace_bytes", "ft_moe_layer_fp8",
           "ft_moe_balance_workspace_bytes", "ft_moe_balance_loss", "ft_moe_gate_backward", "ft_moe_combine_backward",
           "ft_lora_workspace_bytes", "ft_lora_add", "ft_lora_backward")


class FtError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.message = message


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library, refusing a build whose source hash is stale."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        from . import build as _build
        if not os.path.exists(path):
            raise FtError(FT_ERR_CUDA, f"{path} is missing: run bit_quantized_moe_quantize_gb300.build.build()")
        if path == LIB_PATH and not _build.is_current():
            raise FtError(FT_ERR_CUDA, f"{path} was built from other sources: rebuild it")
        L = ctypes.CDLL(path)
        i64, i32, vp, u32p = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)
        L.ft_quantize_q8_1.argtypes = [vp, vp, i64, i64, vp]
        L.ft_moe_route_offsets.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, vp]
        L.ft_moe_route_offsets_noalloc.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, vp]
        L.ft_moe_q4_0_q8_1.argtypes = [vp, vp, vp, vp, i64, i32, i32, i64, i64, vp]
        L.ft_moe_q4_0_q8_1_slots.argtypes = [vp, vp, vp, vp, i64, i32, i32, i64, i64, vp]
        L.ft_moe_q4_0_fp16.argtypes = [vp, vp, vp, vp, i64, i32, i32, i64, i64, vp]
        L.ft_moe_q4_0_q8_1_ep.argtypes = [vp, vp, vp, vp, i64, i32, i32, i32, i32, i64, i64, vp]
        L.ft_moe_block_dots.argtypes = [vp, vp, vp, vp, i64, i32, i32, i64, i64, vp]
        L.ft_act_mul_quantize_q8_1.argtypes = [vp, vp, i64, i64, i32, vp]
        L.ft_moe_gguf_q8_1.argtypes = [i32, vp, vp, vp, vp, i64, i32, i32, i64, i64, vp]
        L.ft_repack_q4_0_soa.argtypes = [vp, vp, vp, i64, vp]
        L.ft_debug_wait_timeout.argtypes = [i64, vp]
        L.ft_debug_stream_read.argtypes = [vp, i64, vp]
        L.ft_moe_ffn_q4_0_q8_1.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i64, i64, i32, vp]
        L.ft_moe_q4_0_q8_1_act.argtypes = [vp, vp, vp, vp, i64, i32, i32, i64, i64, i32, vp]
        L.ft_moe_ffn_reserve.argtypes = [i64, i32, i32, i64, i64]
        L.ft_moe_workspace_bytes.argtypes = [i64, i32, i32, i64, i64]
        L.ft_moe_workspace_bytes.restype = ctypes.c_size_t
        L.ft_moe_reserve.argtypes = [i64, i32, i32, i64, i64]
        L.ft_moe_release.argtypes = []
        L.ft_moe_read_device_error.argtypes = [vp, u32p]
        L.ft_moe_set_path.argtypes = [i32]
        L.ft_moe_selected_path.argtypes = [i64, i32, i32, i64, i64]
        L.ft_moe_gguf_selected_path.argtypes = [i32, i64, i32, i32, i64, i64]
        L.ft_last_error.argtypes = []
        L.ft_last_error.restype = ctypes.c_char_p
        L.ft_abi_version.argtypes = []
        L.ft_profile_enable.argtypes = [i32]
        dp, lp = ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)
        L.ft_profile_read.argtypes = [dp, dp, dp, lp, lp]
        sz, f32 = ctypes.c_size_t, ctypes.c_float
        L.ft_moe_gate.argtypes = [vp, i32, i64, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, i32, f32, vp]
        L.ft_quantize_fp8.argtypes = [vp, i32, vp, vp, i64, i64, vp]
        L.ft_act_mul_quantize_fp8.argtypes = [vp, i32, vp, vp, i64, i64, i32, vp]
        L.ft_moe_fp8_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i64, i64, vp, sz, vp]
        L.ft_moe_fp8_fp8_slots.argtypes = L.ft_moe_fp8_fp8.argtypes
        L.ft_matmul_fp8_fp8.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]
        L.ft_moe_combine.argtypes = [vp, i32, vp, vp, vp, i32, i64, i32, i64, vp]
        L.ft_moe_layer_fp8.argtypes = [vp, i32, vp, i32, i64, vp, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i64, i64,
                                       i32, i32, i32, i32, i32, f32, i32, vp, sz, vp]
        L.ft_moe_fp8_workspace_bytes.argtypes = [i64, i32, i32, i64]
        L.ft_moe_fp8_workspace_bytes.restype = sz
        L.ft_moe_layer_fp8_workspace_bytes.argtypes = [i64, i32, i32, i64, i64]
        L.ft_moe_layer_fp8_workspace_bytes.restype = sz
        L.ft_moe_balance_workspace_bytes.argtypes = [i64, i32, i32]
        L.ft_moe_balance_workspace_bytes.restype = sz
        L.ft_moe_balance_loss.argtypes = [vp, i32, i64, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, vp, sz, vp]
        L.ft_moe_gate_backward.argtypes = [vp, i32, i64, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, f32, i32, vp]
        L.ft_moe_combine_backward.argtypes = [vp, i32, vp, i32, vp, vp, vp, i64, i32, i64, vp]
        L.ft_lora_workspace_bytes.argtypes = [i64, i32, i32, i32, i64, i64, i32]
        L.ft_lora_workspace_bytes.restype = sz
        L.ft_lora_add.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, i64, i64, vp, sz, vp]
        L.ft_lora_backward.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, i64, i64, vp, sz, vp]
        for name in EXPORTS:
            getattr(L, name).restype = getattr(L, name).restype or ctypes.c_int
        L.ft_moe_workspace_bytes.restype = ctypes.c_size_t
        L.ft_last_error.restype = ctypes.c_char_p
        _lib = L
        return L


def last_error() -> str:
    return load().ft_last_error().decode()


def _check(status: int):
    if status != FT_OK:
        raise FtError(status, last_error())


# ------------------------------------------------------------------ tensors
def _torch():
    import torch
    return torch


def _current_device():
    return _torch().cuda.current_device()


def _refuse_device(index):
    """The library works on the current device: tensors of another one would be read and written from there."""
    raise ValueError(f"the tensors are on cuda:{index}, the current device is cuda:{_current_device()}")


def _stream(t):
    if t.get_device() != _current_device():
        _refuse_device(t.get_device())
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dev(t, dtype, name, ndim=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


def quantize_q8_1(x, out=None):
    """fp16 [T, K] -> Q8_1 uint8 [T, K/32, 36] (ft_quantize_q8_1)."""
    torch = _torch()
    px = _dev(x, torch.float16, "x", 2)
    T, K = x.shape
    if out is None:
        out = torch.empty((T, K // 32, 36), dtype=torch.uint8, device=x.device)
    po = _dev(out, torch.uint8, "out")
    _check(load().ft_quantize_q8_1(px, po, T, K, _stream(x)))
    return out


def route_offsets(topk_ids, n_experts, counts=None, offsets=None, perm=None, dev_err=None):
    """int32 [T, k] -> (counts [E], offsets [E+1], perm [T*k]) (ft_moe_route_offsets)."""
    torch = _torch()
    pid = _dev(topk_ids, torch.int32, "topk_ids", 2)
    T, k = topk_ids.shape
    dev = topk_ids.device
    counts = torch.empty(n_experts, dtype=torch.int32, device=dev) if counts is None else counts
    offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev) if offsets is None else offsets
    perm = torch.empty(T * k, dtype=torch.int32, device=dev) if perm is None else perm
    pe = ctypes.c_void_p(0) if dev_err is None else _dev(dev_err, torch.int32, "dev_err")
    _check(load().ft_moe_route_offsets(pid, T, k, n_experts, _dev(counts, torch.int32, "counts"),
                                       _dev(offsets, torch.int32, "offsets"), _dev(perm, torch.int32, "perm"),
                                       pe, _stream(topk_ids)))
    return counts, offsets, perm


def _matmul_shape(weights, act, topk_ids):
    torch = _torch()
    _dev(weights, torch.uint8, "weights", 4)
    _dev(act, torch.uint8, "act", 3)
    _dev(topk_ids, torch.int32, "topk_ids", 2)
    E, N, nb, wb = weights.shape
    T, nb2, ab = act.shape
    if wb != 18 or ab != 36 or nb != nb2 or topk_ids.shape[0] != T:
        raise ValueError(f"shape mismatch: weights {tuple(weights.shape)} act {tuple(act.shape)} "
                         f"topk_ids {tuple(topk_ids.shape)}")
    return E, N, nb * 32, T, topk_ids.shape[1]


def moe_q4_0_q8_1(weights, act, topk_ids, out=None):
    """Routed matmul: Q4_0 [E,N,K/32,18] x Q8_1 [T,K/32,36] -> fp32 [T, k, N] (ft_moe_q4_0_q8_1)."""
    torch = _torch()
    E, N, K, T, k = _matmul_shape(weights, act, topk_ids)
    if out is None:
        out = torch.empty((T, k, N), dtype=torch.float32, device=weights.device)
    po = _dev(out, torch.float32, "out")
    _check(load().ft_moe_q4_0_q8_1(ctypes.c_void_p(weights.data_ptr()), ctypes.c_void_p(act.data_ptr()),
                                   ctypes.c_void_p(topk_ids.data_ptr()), po, T, k, E, N, K, _stream(weights)))
    return out


def moe_q4_0_q8_1_slots(weights, act_slots, topk_ids, out=None):
    """Routed matmul with one activation row per slot: Q4_0 [E,N,K/32,18] x
    Q8_1 [T*k,K/32,36] (row s for slot s = t*k + j) -> fp32 [T, k, N]
    (ft_moe_q4_0_q8_1_slots)."""
    torch = _torch()
    _dev(weights, torch.uint8, "weights", 4)
    _dev(act_slots, torch.uint8, "act_slots", 3)
    _dev(topk_ids, torch.int32, "topk_ids", 2)
    E, N, nb, wb = weights.shape
    S, nb2, ab = act_slots.shape
    T, k = topk_ids.shape
    if wb != 18 or ab != 36 or nb != nb2 or S != T * k:
        raise ValueError(f"shape mismatch: weights {tuple(weights.shape)} act_slots {tuple(act_slots.shape)} "
                         f"topk_ids {tuple(topk_ids.shape)}")
    if out is None:
        out = torch.empty((T, k, N), dtype=torch.float32, device=weights.device)
    po = _dev(out, torch.float32, "out")
    _check(load().ft_moe_q4_0_q8_1_slots(ctypes.c_void_p(weights.data_ptr()), ctypes.c_void_p(act_slots.data_ptr()),
                                         ctypes.c_void_p(topk_ids.data_ptr()), po, T, k, E, N, nb * 32,
                                         _stream(weights)))
    return out


def moe_q4_0_q8_1_ep(weights_local, act, topk_ids, n_experts_global, expert_start, out=None):
    """Routed matmul on an expert-parallel shard (ft_moe_q4_0_q8_1_ep):
    weights_local Q4_0 [E_local,N,K/32,18] holds experts [expert_start,
    expert_start + E_local) of n_experts_global; topk_ids hold global ids;
    rows of slots routed elsewhere are 0."""
    torch = _torch()
    E_local, N, K, T, k = _matmul_shape(weights_local, act, topk_ids)
    if out is None:
        out = torch.empty((T, k, N), dtype=torch.float32, device=weights_local.device)
    po = _dev(out, torch.float32, "out")
    _check(load().ft_moe_q4_0_q8_1_ep(ctypes.c_void_p(weights_local.data_ptr()), ctypes.c_void_p(act.data_ptr()),
                                      ctypes.c_void_p(topk_ids.data_ptr()), po, T, k, int(n_experts_global),
                                      int(expert_start), E_local, N, K, _stream(weights_local)))
    return out


# GGUF weight types: GGML type number, bytes per stored block, weights per block
WEIGHT_TYPES = {"q4_0": (2, 18, 32), "q4_1": (3, 20, 32), "q5_0": (6, 22, 32), "q5_1": (7, 24, 32),
                "q8_0": (8, 34, 32), "q4_k": (12, 144, 256), "q5_k": (13, 176, 256),
                "q6_k": (14, 210, 256), "q2_k": (10, 84, 256), "q3_k": (11, 110, 256)}


def moe_gguf_q8_1(wtype, weights, act, topk_ids, out=None):
    """Routed matmul with weights of a GGUF type (ft_moe_gguf_q8_1): weights uint8
    [E, N, K/32 (K/256 for the K-quants), bytes of the type] x Q8_1 [T, K/32, 36]
    -> fp32 [T, k, N]."""
    torch = _torch()
    tid, bb, per = WEIGHT_TYPES[wtype]
    _dev(weights, torch.uint8, "weights", 4)
    _dev(act, torch.uint8, "act", 3)
    _dev(topk_ids, torch.int32, "topk_ids", 2)
    E, N, nb, wb = weights.shape
    T, nb2, ab = act.shape
    if wb != bb or ab != 36 or nb * per != nb2 * 32 or topk_ids.shape[0] != T:
        raise ValueError(f"shape mismatch for {wtype}: weights {tuple(weights.shape)} act {tuple(act.shape)} "
                         f"topk_ids {tuple(topk_ids.shape)}")
    k = topk_ids.shape[1]
    if out is None:
        out = torch.empty((T, k, N), dtype=torch.float32, device=weights.device)
    po = _dev(out, torch.float32, "out")
    _check(load().ft_moe_gguf_q8_1(tid, ctypes.c_void_p(weights.data_ptr()), ctypes.c_void_p(act.data_ptr()),
                                   ctypes.c_void_p(topk_ids.data_ptr()), po, T, k, E, N, nb * per, _stream(weights)))
    return out


def repack_q4_0_soa(weights, qs=None, d=None):
    """Q4_0 blocks uint8 [..., 18] -> (nibble bytes uint8 [n, 16], fp16 scales [n])
    (ft_repack_q4_0_soa)."""
    torch = _torch()
    _dev(weights, torch.uint8, "weights")
    if weights.shape[-1] != 18:
        raise ValueError(f"weights must end in 18-byte Q4_0 blocks, got {tuple(weights.shape)}")
    n = weights.numel() // 18
    qs = torch.empty((n, 16), dtype=torch.uint8, device=weights.device) if qs is None else qs
    d = torch.empty(n, dtype=torch.float16, device=weights.device) if d is None else d
    _check(load().ft_repack_q4_0_soa(ctypes.c_void_p(weights.data_ptr()), _dev(qs, torch.uint8, "qs"),
                                     _dev(d, torch.float16, "d"), n, _stream(weights)))
    return qs, d


ACT_SILU = 0
ACT_GELU_TANH = 1


def act_mul_quantize_q8_1(h, act_kind, out=None):
    """fp32 [..., 2I] (gate | up) -> Q8_1 uint8 [rows, I/32, 36] of act(gate) * up,
    rows = h.numel() / 2I (ft_act_mul_quantize_q8_1)."""
    torch = _torch()
    ph = _dev(h, torch.float32, "h")
    two_i = h.shape[-1]
    if two_i % 64:
        raise ValueError(f"the last dim of h must be 2 * n_inter with n_inter % 32 == 0 (got {two_i})")
    rows = h.numel() // two_i
    if out is None:
        out = torch.empty((rows, two_i // 64, 36), dtype=torch.uint8, device=h.device)
    po = _dev(out, torch.uint8, "out")
    if out.numel() != rows * (two_i // 64) * 36:
        raise ValueError(f"out must hold {rows} x {two_i // 64} Q8_1 blocks")
    _check(load().ft_act_mul_quantize_q8_1(ph, po, rows, two_i // 2, int(act_kind), _stream(h)))
    return out


def moe_q4_0_fp16(weights, x, topk_ids, out=None):
    """The whole hot path from fp16 rows (ft_moe_q4_0_fp16): Q4_0 [E, N, K/32, 18]
    x fp16 [T, K] -> fp32 [T, k, N]; one launch for decode-sized batches."""
    torch = _torch()
    _dev(weights, torch.uint8, "weights", 4)
    px = _dev(x, torch.float16, "x", 2)
    _dev(topk_ids, torch.int32, "topk_ids", 2)
    E, N, nb, wb = weights.shape
    T, K = x.shape
    if wb != 18 or nb * 32 != K or topk_ids.shape[0] != T:
        raise ValueError(f"shape mismatch: weights {tuple(weights.shape)} x {tuple(x.shape)} "
                         f"topk_ids {tuple(topk_ids.shape)}")
    k = topk_ids.shape[1]
    if out is None:
        out = torch.empty((T, k, N), dtype=torch.float32, device=weights.device)
    po = _dev(out, torch.float32, "out")
    _check(load().ft_moe_q4_0_fp16(ctypes.c_void_p(weights.data_ptr()), px, ctypes.c_void_p(topk_ids.data_ptr()),
                                   po, T, k, E, N, K, _stream(weights)))
    return out


def moe_q4_0_q8_1_act(w13, act, topk_ids, act_kind, out=None):
    """Layer 1 with the gated activation fused (ft_moe_q4_0_q8_1_act): w13 Q4_0
    [E, 2I, H/32, 18] (gate rows, then up rows), act Q8_1 [T, H/32, 36] ->
    Q8_1 uint8 [T*k, I/32, 36] of act(gate) * up per slot."""
    torch = _torch()
    E, two_i, H, T, k = _matmul_shape(w13, act, topk_ids)
    if two_i % 64:
        raise ValueError(f"w13 must hold 2 * n_inter rows with n_inter % 32 == 0 (got {two_i})")
    I = two_i // 2
    if out is None:
        out = torch.empty((T * k, I // 32, 36), dtype=torch.uint8, device=w13.device)
    po = _dev(out, torch.uint8, "out")
    if out.numel() != T * k * (I // 32) * 36:
        raise ValueError(f"out must hold {T * k} x {I // 32} Q8_1 blocks")
    _check(load().ft_moe_q4_0_q8_1_act(ctypes.c_void_p(w13.data_ptr()), ctypes.c_void_p(act.data_ptr()),
                                       ctypes.c_void_p(topk_ids.data_ptr()), po, T, k, E, I, H, int(act_kind),
                                       _stream(w13)))
    return out


def moe_ffn_q4_0_q8_1(w13, w2, act, topk_ids, act_kind, out=None, h=None, act_mid=None, keep_h=True):
    """Both expert layers per slot (ft_moe_ffn_q4_0_q8_1): w13 Q4_0 [E, 2I, H/32, 18]
    (gate rows, then up rows), w2 Q4_0 [E, H, I/32, 18], act Q8_1 [T, H/32, 36]
    -> out fp32 [T, k, H]; returns (out, h [T, k, 2I] fp32, act_mid [T*k, I/32, 36]).
    keep_h=False (and h None): layer 1 with the activation fused, h is None."""
    torch = _torch()
    E, two_i, H, T, k = _matmul_shape(w13, act, topk_ids)
    _dev(w2, torch.uint8, "w2", 4)
    if w2.shape[0] != E or w2.shape[1] != H or w2.shape[3] != 18 or 2 * w2.shape[2] * 32 != two_i:
        raise ValueError(f"shape mismatch: w13 {tuple(w13.shape)} w2 {tuple(w2.shape)}")
    I = two_i // 2
    dev = w13.device
    out = torch.empty((T, k, H), dtype=torch.float32, device=dev) if out is None else out
    if h is None and keep_h:
        h = torch.empty((T, k, two_i), dtype=torch.float32, device=dev)
    act_mid = torch.empty((T * k, I // 32, 36), dtype=torch.uint8, device=dev) if act_mid is None else act_mid
    ph = ctypes.c_void_p(0) if h is None else _dev(h, torch.float32, "h")
    _check(load().ft_moe_ffn_q4_0_q8_1(ctypes.c_void_p(w13.data_ptr()), ctypes.c_void_p(w2.data_ptr()),
                                       ctypes.c_void_p(act.data_ptr()), ctypes.c_void_p(topk_ids.data_ptr()),
                                       ph, _dev(act_mid, torch.uint8, "act_mid"),
                                       _dev(out, torch.float32, "out"), T, k, E, H, I, int(act_kind),
                                       _stream(w13)))
    return out, h, act_mid


def ffn_reserve(max_tokens, max_top_k, n_experts, hidden, n_inter):
    """Workspace for both expert layers up to these sizes (ft_moe_ffn_reserve)."""
    _check(load().ft_moe_ffn_reserve(max_tokens, max_top_k, n_experts, hidden, n_inter))


def block_dots(weights, act, topk_ids, out=None):
    """Diagnostic: int32 [T*k, N, K/32] per-block integer dots (ft_moe_block_dots)."""
    torch = _torch()
    E, N, K, T, k = _matmul_shape(weights, act, topk_ids)
    if out is None:
        out = torch.empty((T * k, N, K // 32), dtype=torch.int32, device=weights.device)
    po = _dev(out, torch.int32, "out")
    _check(load().ft_moe_block_dots(ctypes.c_void_p(weights.data_ptr()), ctypes.c_void_p(act.data_ptr()),
                                    ctypes.c_void_p(topk_ids.data_ptr()), po, T, k, E, N, K, _stream(weights)))
    return out


# ------------------------------------------------- FP8 expert-layer operators
# A decoded token's calls take the GPU a few microseconds: the checks below stay cheap
# (one attribute at a time, device indices instead of device objects).
SCORES = {"softmax": 0, "sigmoid": 1}
F32, F16, BF16 = 0, 1, 2
_DTYPES: dict = {}       # torch dtype -> FT_DTYPE_*
_CODES: tuple = ()       # torch dtypes that hold e4m3 codes
_i32 = _f32 = _e4m3 = None
_Tensor = _empty_strided = _raw_stream = None


def _ready():
    """The library, with the torch names that the checks use."""
    global _CODES, _i32, _f32, _e4m3, _Tensor, _empty_strided, _raw_stream, _current_device
    torch = _torch()
    if not _CODES:
        _DTYPES.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
        _i32, _f32, _e4m3 = torch.int32, torch.float32, torch.float8_e4m3fn
        _Tensor, _empty_strided = torch.Tensor, torch.empty_strided
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", _current_device)      # without a check for a first use
        _CODES = (torch.float8_e4m3fn, torch.uint8)
    return load()


def _stream_of(index):
    """The current stream of device `index`, which has to be the current device."""
    if index != _current_device():
        _refuse_device(index)
    return _raw_stream(index)


def _lib_ready():
    return _lib if _CODES and _lib is not None else _ready()


def _bad_dtype(name, allowed, dt):
    names = ", ".join(str(t).replace("torch.", "") for t, c in _DTYPES.items() if c in allowed)
    raise TypeError(f"{name} must be one of {names}, got {dt}")


def _dtype_code(dt, name, allowed=(F32, F16, BF16)):
    """FT_DTYPE_* of a torch dtype, one of `allowed`."""
    code = _DTYPES.get(dt)
    if code is None or code not in allowed:
        _bad_dtype(name, allowed, dt)
    return code


def _ptr(t, name, ndim, dev=None):
    """Data pointer of a contiguous CUDA tensor with `ndim` dims on device `dev`."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    return t.data_ptr()


def _codes_ptr(t, name, ndim, dev=None):
    p = _ptr(t, name, ndim, dev)
    if t.dtype not in _CODES:
        raise TypeError(f"{name} must hold e4m3 codes (torch.float8_e4m3fn or uint8), got {t.dtype}")
    return p


def _typed_ptr(t, name, dtype, shape, dev):
    p = _ptr(t, name, len(shape), dev)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return p


def _empty(shape, dtype, device):
    """A new contiguous tensor of up to three dims; with its strides given torch makes it sooner (1.4 us of a call's 15)."""
    n = len(shape)
    stride = (shape[1], 1) if n == 2 else (shape[1] * shape[2], shape[2], 1) if n == 3 else (1,) * n
    return _empty_strided(shape, stride, dtype=dtype, device=device)


def _out(out, name, shape, dtype, like, dev):
    """`out` checked, or a new tensor beside `like`."""
    if out is None:
        return _empty(shape, dtype, like.device)
    _ptr(out, name, len(shape), dev)
    if out.dtype != dtype or out.shape != shape:
        raise ValueError(f"{name} must be {dtype} {shape}, got {out.dtype} {tuple(out.shape)}")
    return out


def _workspace(n, like):
    """(tensor, pointer) of n bytes; the caching allocator hands them out in stream order."""
    if not n:
        return None, None
    t = _empty((n,), _CODES[1], like.device)
    return t, t.data_ptr()


def _b(n):
    return (n + 127) // 128


def _logits_of(logits):
    """(tokens, experts, row stride, device index) of router logits, whose rows may lie apart."""
    if not isinstance(logits, _Tensor) or not logits.is_cuda:
        raise TypeError("logits must be a CUDA tensor")
    if logits.dim() != 2:
        raise ValueError(f"logits must have 2 dims, got {tuple(logits.shape)}")
    T, E = logits.shape
    stride, step = logits.stride()
    if E > 1 and step != 1:
        raise ValueError("the elements of a row of logits must be neighbours")
    if T <= 1:
        stride = E
    elif stride < E:
        raise ValueError("rows of logits must not overlap")
    return T, E, stride, logits.get_device()


def _score_code(score):
    code = SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return code


def moe_gate(logits, top_k, score="softmax", bias=None, n_groups=1, topk_groups=1, group_top=1, renormalize=True,
             scale=1.0, topk_ids=None, topk_weights=None):
    """Router (ft_moe_gate): logits [T, E] fp32 / fp16 / bf16 (rows may lie apart) ->
    (topk_ids int32 [T, k], topk_weights fp32 [T, k]); id -1, weight 0 where no expert is left."""
    L = _lib_ready()
    T, E, stride, dev = _logits_of(logits)
    code = _dtype_code(logits.dtype, "logits")
    pb = None if bias is None else _typed_ptr(bias, "bias", _f32, (E,), dev)
    shape = (T, max(int(top_k), 0))
    topk_ids = _out(topk_ids, "topk_ids", shape, _i32, logits, dev)
    topk_weights = _out(topk_weights, "topk_weights", shape, _f32, logits, dev)
    st = L.ft_moe_gate(logits.data_ptr(), code, stride, pb, topk_ids.data_ptr(), topk_weights.data_ptr(), T, E, top_k,
                       _score_code(score), n_groups, topk_groups, group_top, 1 if renormalize else 0, scale,
                       _stream_of(dev))
    if st:
        _check(st)
    return topk_ids, topk_weights


def quantize_fp8(x, codes=None, scales=None):
    """[R, K] fp32 / fp16 / bf16 -> (e4m3 codes [R, K], fp32 scales [R, ceil(K/128)]) (ft_quantize_fp8)."""
    L = _lib_ready()
    px = _ptr(x, "x", 2)
    R, K = x.shape
    dev = x.get_device()
    code = _dtype_code(x.dtype, "x")
    codes = _out(codes, "codes", (R, K), _e4m3, x, dev)
    scales = _out(scales, "scales", (R, _b(K)), _f32, x, dev)
    st = L.ft_quantize_fp8(px, code, codes.data_ptr(), scales.data_ptr(), R, K, _stream_of(dev))
    if st:
        _check(st)
    return codes, scales


def act_mul_quantize_fp8(h, act_kind, codes=None, scales=None):
    """[R, 2I] (gate | up) fp32 / fp16 / bf16 -> (e4m3 codes [R, I], fp32 scales [R, ceil(I/128)])
    of act(gate) * up (ft_act_mul_quantize_fp8)."""
    L = _lib_ready()
    ph = _ptr(h, "h", 2)
    R, two_i = h.shape
    if two_i % 2:
        raise ValueError(f"h must hold gate and up values, got rows of {two_i}")
    I = two_i // 2
    dev = h.get_device()
    code = _dtype_code(h.dtype, "h")
    codes = _out(codes, "codes", (R, I), _e4m3, h, dev)
    scales = _out(scales, "scales", (R, _b(I)), _f32, h, dev)
    st = L.ft_act_mul_quantize_fp8(ph, code, codes.data_ptr(), scales.data_ptr(), R, I, int(act_kind), _stream_of(dev))
    if st:
        _check(st)
    return codes, scales


def _moe_fp8(per_slot, weights, w_scales, act, act_scales, topk_ids, out, out_dtype):
    L = _lib_ready()
    pw = _codes_ptr(weights, "weights", 3)
    E, N, K = weights.shape
    dev = weights.get_device()
    pi = _ptr(topk_ids, "topk_ids", 2, dev)
    if topk_ids.dtype != _i32:
        raise TypeError(f"topk_ids must be {_i32}, got {topk_ids.dtype}")
    T, k = topk_ids.shape
    rows = T * k if per_slot else T
    pa = _codes_ptr(act, "act", 2, dev)
    if act.shape != (rows, K):
        raise ValueError(f"act must have shape {(rows, K)}, got {tuple(act.shape)}")
    nb = _b(K)
    ps = _typed_ptr(w_scales, "w_scales", _f32, (E, _b(N), nb), dev)
    pt = _typed_ptr(act_scales, "act_scales", _f32, (rows, nb), dev)
    out_dtype = (out_dtype or _f32) if out is None else out.dtype
    code = _dtype_code(out_dtype, "out_dtype", (F32, BF16))
    out = _out(out, "out", (T, k, N), out_dtype, weights, dev)
    n = L.ft_moe_fp8_workspace_bytes(T, k, E, K)
    ws, pws = _workspace(n, weights)
    st = (L.ft_moe_fp8_fp8_slots if per_slot else L.ft_moe_fp8_fp8)(
        pw, ps, pa, pt, pi, out.data_ptr(), code, T, k, E, N, K, pws, n, _stream_of(dev))
    if st:
        _check(st)
    return out


def moe_fp8_fp8(weights, w_scales, act, act_scales, topk_ids, out=None, out_dtype=None):
    """Routed product (ft_moe_fp8_fp8): e4m3 weights [E, N, K] with scales [E, ceil(N/128), ceil(K/128)] x
    e4m3 rows [T, K] with scales [T, ceil(K/128)] -> [T, k, N] fp32 (default) or bf16.
    Slots whose id is -1 have no expert: their rows are 0."""
    return _moe_fp8(False, weights, w_scales, act, act_scales, topk_ids, out, out_dtype)


def moe_fp8_fp8_slots(weights, w_scales, act_slots, act_scales, topk_ids, out=None, out_dtype=None):
    """moe_fp8_fp8 with one activation row per routed slot, act_slots [T*k, K] (ft_moe_fp8_fp8_slots)."""
    return _moe_fp8(True, weights, w_scales, act_slots, act_scales, topk_ids, out, out_dtype)


def matmul_fp8_fp8(weights, w_scales, act, act_scales, out=None, out_dtype=None):
    """Product with one dense matrix (ft_matmul_fp8_fp8): weights [N, K] x rows [M, K] -> [M, N]
    fp32 (default) or bf16."""
    L = _lib_ready()
    pw = _codes_ptr(weights, "weights", 2)
    N, K = weights.shape
    dev = weights.get_device()
    pa = _codes_ptr(act, "act", 2, dev)
    M = act.shape[0]
    if act.shape[1] != K:
        raise ValueError(f"act must have {K} columns, got {tuple(act.shape)}")
    nb = _b(K)
    ps = _typed_ptr(w_scales, "w_scales", _f32, (_b(N), nb), dev)
    pt = _typed_ptr(act_scales, "act_scales", _f32, (M, nb), dev)
    out_dtype = (out_dtype or _f32) if out is None else out.dtype
    code = _dtype_code(out_dtype, "out_dtype", (F32, BF16))
    out = _out(out, "out", (M, N), out_dtype, weights, dev)
    st = L.ft_matmul_fp8_fp8(pw, ps, pa, pt, out.data_ptr(), code, M, N, K, _stream_of(dev))
    if st:
        _check(st)
    return out


def moe_combine(rows, topk_weights, add=None, out=None, out_dtype=None):
    """Weighted sum of each token's expert rows (ft_moe_combine): rows [T, k, N] fp32 / bf16, topk_weights
    fp32 [T, k], add [T, N] or None -> [T, N] of out_dtype (default: rows' type).  Rows with weight 0 are not read."""
    L = _lib_ready()
    pr = _ptr(rows, "rows", 3)
    T, k, N = rows.shape
    dev = rows.get_device()
    pw = _typed_ptr(topk_weights, "topk_weights", _f32, (T, k), dev)
    code = _dtype_code(rows.dtype, "rows", (F32, BF16))
    out_dtype = (out_dtype or rows.dtype) if out is None else out.dtype
    ocode = _dtype_code(out_dtype, "out_dtype")
    out = _out(out, "out", (T, N), out_dtype, rows, dev)
    pa = None if add is None else _typed_ptr(add, "add", out_dtype, (T, N), dev)
    st = L.ft_moe_combine(pr, code, pw, pa, out.data_ptr(), ocode, T, k, N, _stream_of(dev))
    if st:
        _check(st)
    return out


def moe_layer_fp8(x, logits, w13, s13, w2, s2, top_k, act_kind=0, score="softmax", bias=None, n_groups=1,
                  topk_groups=1, group_top=1, renormalize=True, scale=1.0, out=None):
    """A whole expert layer (ft_moe_layer_fp8): x [T, H] fp16 / bf16, router logits [T, E], e4m3 w13 [E, 2I, H]
    (gate rows, then up rows) and w2 [E, H, I] with their scales -> (y [T, H], topk_ids, topk_weights)."""
    L = _lib_ready()
    px = _ptr(x, "x", 2)
    T, H = x.shape
    xcode = _dtype_code(x.dtype, "x", (F16, BF16))
    T2, E, stride, dev = _logits_of(logits)
    if T2 != T or x.get_device() != dev:
        raise ValueError(f"logits must be [{T}, E] on {x.device}, got {tuple(logits.shape)} on {logits.device}")
    lcode = _dtype_code(logits.dtype, "logits")
    pw13, pw2 = _codes_ptr(w13, "w13", 3, dev), _codes_ptr(w2, "w2", 3, dev)
    two_i = w13.shape[1]
    I = two_i // 2
    if two_i % 2 or w13.shape != (E, two_i, H) or w2.shape != (E, H, I):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)} logits {tuple(logits.shape)} w13 {tuple(w13.shape)} "
                         f"w2 {tuple(w2.shape)}")
    nbh = _b(H)
    ps13 = _typed_ptr(s13, "s13", _f32, (E, _b(two_i), nbh), dev)
    ps2 = _typed_ptr(s2, "s2", _f32, (E, nbh, _b(I)), dev)
    pb = None if bias is None else _typed_ptr(bias, "bias", _f32, (E,), dev)
    out = _out(out, "out", (T, H), x.dtype, x, dev)
    device, shape = x.device, (T, max(int(top_k), 0))
    ids = _empty(shape, _i32, device)
    weights = _empty(shape, _f32, device)
    n = L.ft_moe_layer_fp8_workspace_bytes(T, top_k, E, H, I)
    ws, pws = _workspace(n, x)
    st = L.ft_moe_layer_fp8(px, xcode, logits.data_ptr(), lcode, stride, pb, pw13, ps13, pw2, ps2, out.data_ptr(),
                            ids.data_ptr(), weights.data_ptr(), T, E, top_k, H, I, _score_code(score), n_groups,
                            topk_groups, group_top, 1 if renormalize else 0, scale, int(act_kind), pws, n,
                            _stream_of(dev))
    if st:
        _check(st)
    return out, ids, weights


# ------------------------------------------------- adapting a layer of experts
def _offsets_of(seq_offsets, dev):
    """(pointer, number of sequences) of the offsets of packed sequences, None: one sequence of all rows."""
    if seq_offsets is None:
        return None, 1
    p = _ptr(seq_offsets, "seq_offsets", 1, dev)
    if seq_offsets.dtype != _i32:
        raise TypeError(f"seq_offsets must be {_i32}, got {seq_offsets.dtype}")
    n = seq_offsets.shape[0] - 1
    if n < 1:
        raise ValueError("seq_offsets must hold the start of every sequence and the end of the last")
    return p, n


def _ids_of(topk_ids, tokens, dev):
    """(pointer, top_k) of the chosen experts of `tokens` rows."""
    p = _ptr(topk_ids, "topk_ids", 2, dev)
    if topk_ids.dtype != _i32:
        raise TypeError(f"topk_ids must be {_i32}, got {topk_ids.dtype}")
    if topk_ids.shape[0] != tokens:
        raise ValueError(f"topk_ids must have {tokens} rows, got {tuple(topk_ids.shape)}")
    return p, topk_ids.shape[1]


def moe_balance_loss(logits, topk_ids, score="softmax", seq_offsets=None):
    """Load-balance loss of a router (ft_moe_balance_loss): logits [T, E] (rows may lie apart) and the chosen
    topk_ids [T, k] -> (loss fp32 [], counts int32 [S, E], seq_scale fp32 [S]).  seq_offsets int32 [S + 1]: where
    each packed sequence starts, and where the last ends; None: one sequence.  counts and seq_scale are what
    moe_gate_backward needs for the loss' gradient."""
    L = _lib_ready()
    T, E, stride, dev = _logits_of(logits)
    code = _dtype_code(logits.dtype, "logits")
    pi, k = _ids_of(topk_ids, T, dev)
    po, S = _offsets_of(seq_offsets, dev)
    device = logits.device
    loss = _empty((), _f32, device)
    counts = _empty((S, E), _i32, device)
    seq_scale = _empty((S,), _f32, device)
    n = L.ft_moe_balance_workspace_bytes(T, E, S)
    ws, pws = _workspace(n, logits)
    st = L.ft_moe_balance_loss(logits.data_ptr(), code, stride, pi, po, loss.data_ptr(), counts.data_ptr(),
                               seq_scale.data_ptr(), T, E, k, _score_code(score), S, pws, n, _stream_of(dev))
    if st:
        _check(st)
    return loss, counts, seq_scale


def moe_gate_backward(logits, topk_ids, grad_weights=None, score="softmax", renormalize=True, scale=1.0, counts=None,
                      seq_scale=None, grad_loss=None, seq_offsets=None, grad_logits=None):
    """Gradient of the router (ft_moe_gate_backward) -> grad_logits [T, E] of the logits' type: of moe_gate's
    weights (grad_weights fp32 [T, k]), of moe_balance_loss (its counts and seq_scale, and grad_loss fp32 of
    one element), or of both at once.  score, renormalize, scale: as moe_gate had them."""
    L = _lib_ready()
    T, E, stride, dev = _logits_of(logits)
    code = _dtype_code(logits.dtype, "logits")
    pi, k = _ids_of(topk_ids, T, dev)
    pw = None if grad_weights is None else _typed_ptr(grad_weights, "grad_weights", _f32, (T, k), dev)
    pc = ps = pl = po = None
    S = 1
    if counts is not None or seq_scale is not None or grad_loss is not None:
        if counts is None or seq_scale is None or grad_loss is None:
            raise ValueError("counts, seq_scale and grad_loss come together")
        po, S = _offsets_of(seq_offsets, dev)
        pc = _typed_ptr(counts, "counts", _i32, (S, E), dev)
        ps = _typed_ptr(seq_scale, "seq_scale", _f32, (S,), dev)
        pl = _typed_ptr(grad_loss, "grad_loss", _f32, (1,) if getattr(grad_loss, "ndim", 0) else (), dev)
    grad_logits = _out(grad_logits, "grad_logits", (T, E), logits.dtype, logits, dev)
    st = L.ft_moe_gate_backward(logits.data_ptr(), code, stride, pi, pw, pc, ps, pl, po, grad_logits.data_ptr(), T, E, k,
                                _score_code(score), 1 if renormalize else 0, scale, S, _stream_of(dev))
    if st:
        _check(st)
    return grad_logits


def moe_combine_backward(grad_out, rows, topk_weights, need_rows=True, need_weights=True, grad_rows=None,
                         grad_weights=None):
    """Gradients of moe_combine (ft_moe_combine_backward): grad_out [T, N] fp32 / fp16 / bf16, rows [T, k, N] fp32 /
    bf16 and topk_weights fp32 [T, k] as it had them -> (grad_rows [T, k, N] of the rows' type, grad_weights fp32
    [T, k]); None where not needed."""
    L = _lib_ready()
    pr = _ptr(rows, "rows", 3)
    T, k, N = rows.shape
    dev = rows.get_device()
    code = _dtype_code(rows.dtype, "rows", (F32, BF16))
    pw = _typed_ptr(topk_weights, "topk_weights", _f32, (T, k), dev)
    pg = _ptr(grad_out, "grad_out", 2, dev)
    gcode = _dtype_code(grad_out.dtype, "grad_out")
    if grad_out.shape != (T, N):
        raise ValueError(f"grad_out must have shape {(T, N)}, got {tuple(grad_out.shape)}")
    if need_rows or grad_rows is not None:
        grad_rows = _out(grad_rows, "grad_rows", (T, k, N), rows.dtype, rows, dev)
    if need_weights or grad_weights is not None:
        grad_weights = _out(grad_weights, "grad_weights", (T, k), _f32, rows, dev)
    st = L.ft_moe_combine_backward(pg, gcode, pr, code, pw, None if grad_rows is None else grad_rows.data_ptr(),
                                   None if grad_weights is None else grad_weights.data_ptr(), T, k, N, _stream_of(dev))
    if st:
        _check(st)
    return grad_rows, grad_weights


def _lora_args(x, a, b, ids, scales):
    """Checked: (pointers of x, a, b, ids, scales, type code, device, T, k, per_slot, L, R, K, N, shape of the slots)."""
    px = _ptr(x, "x", 2)
    rows, K = x.shape
    dev = x.get_device()
    code = _dtype_code(x.dtype, "x", (F16, BF16))
    pa, pb = _ptr(a, "a", 3, dev), _ptr(b, "b", 3, dev)
    L, R, _ = a.shape
    N = b.shape[1]
    if a.dtype != x.dtype or b.dtype != x.dtype:
        raise TypeError(f"x, a and b must have one type, got {x.dtype}, {a.dtype} and {b.dtype}")
    if a.shape != (L, R, K) or b.shape != (L, N, R):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)} a {tuple(a.shape)} b {tuple(b.shape)}")
    pi = _ptr(ids, "ids", 1 if ids.dim() == 1 else 2, dev)
    if ids.dtype != _i32:
        raise TypeError(f"ids must be {_i32}, got {ids.dtype}")
    lead = tuple(ids.shape)
    T, k = lead if len(lead) == 2 else (lead[0], 1)
    if rows != T and rows != T * k:
        raise ValueError(f"x must have a row per token ({T}) or per slot ({T * k}), got {rows}")
    ps = None if scales is None else _typed_ptr(scales, "scales", _f32, (L,), dev)
    return px, pa, pb, pi, ps, code, dev, T, k, 1 if rows != T or k == 1 else 0, L, R, K, N, lead


def lora_add(x, a, b, ids, scales=None, add=None, out=None, out_dtype=None):
    """Low-rank adapters beside a product (ft_lora_add): rows x [T, K], or [T*k, K] per slot, fp16 / bf16; adapters a
    [L, R, K] and b [L, N, R]; ids int32 [T] or [T, k], -1: none; scales fp32 [L] or None -> add + scale * b (a x),
    [T, N] or [T, k, N], of out_dtype (fp32 or x's type; default: add's type, else x's).  out may be add."""
    lib = _lib_ready()
    px, pa, pb, pi, ps, code, dev, T, k, per_slot, L, R, K, N, lead = _lora_args(x, a, b, ids, scales)
    out_dtype = (out_dtype or (x.dtype if add is None else add.dtype)) if out is None else out.dtype
    ocode = _dtype_code(out_dtype, "out_dtype", (F32, code))
    padd = None if add is None else _typed_ptr(add, "add", out_dtype, (*lead, N), dev)
    out = _out(out, "out", (*lead, N), out_dtype, x, dev)
    n = lib.ft_lora_workspace_bytes(T, k, L, R, K, N, 0)
    ws, pws = _workspace(n, x)
    st = lib.ft_lora_add(px, code, pa, pb, ps, pi, padd, out.data_ptr(), ocode, T, k, per_slot, L, R, K, N, pws, n,
                         _stream_of(dev))
    if st:
        _check(st)
    return out


def lora_backward(grad_out, x, a, b, ids, scales=None, add=None, need_x=True, need_a=True, need_b=True, grad_x=None,
                  grad_a=None, grad_b=None):
    """Gradients of lora_add (ft_lora_backward): grad_out [T, N] or [T, k, N] of x's type, the other arguments as it
    had them, add of x's shape or None -> (grad_x = add + the gradient, of x's shape and type, summed over a token's slots where
    they share a row; grad_a fp32 [L, R, K]; grad_b fp32 [L, N, R]); None where not needed."""
    lib = _lib_ready()
    px, pa, pb, pi, ps, code, dev, T, k, per_slot, L, R, K, N, lead = _lora_args(x, a, b, ids, scales)
    pg = _typed_ptr(grad_out, "grad_out", x.dtype, (*lead, N), dev)
    padd = None if add is None else _typed_ptr(add, "add", x.dtype, x.shape, dev)
    if need_x or grad_x is not None:
        grad_x = _out(grad_x, "grad_x", tuple(x.shape), x.dtype, x, dev)
    if need_a or grad_a is not None:
        grad_a = _out(grad_a, "grad_a", (L, R, K), _f32, x, dev)
    if need_b or grad_b is not None:
        grad_b = _out(grad_b, "grad_b", (L, N, R), _f32, x, dev)
    n = lib.ft_lora_workspace_bytes(T, k, L, R, K, N, 1)
    ws, pws = _workspace(n, x)
    st = lib.ft_lora_backward(pg, px, code, pa, pb, ps, pi, padd, None if grad_x is None else grad_x.data_ptr(),
                              None if grad_a is None else grad_a.data_ptr(), None if grad_b is None else grad_b.data_ptr(),
                              T, k, per_slot, L, R, K, N, pws, n, _stream_of(dev))
    if st:
        _check(st)
    return grad_x, grad_a, grad_b


def workspace_bytes(tokens, top_k, n_experts, nrows, ncols) -> int:
    return int(load().ft_moe_workspace_bytes(tokens, top_k, n_experts, nrows, ncols))


def reserve(max_tokens, max_top_k, n_experts, nrows, ncols):
    _check(load().ft_moe_reserve(max_tokens, max_top_k, n_experts, nrows, ncols))


def release():
    _check(load().ft_moe_release())


def read_device_error(stream=None) -> int:
    """Synchronize, return and clear the library's device error word (no raise)."""
    torch = _torch()
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream if stream is None else stream)
    flags = ctypes.c_uint32(0)
    st = load().ft_moe_read_device_error(s, ctypes.byref(flags))
    if st not in (FT_OK, FT_ERR_DEVICE_FLAG):
        raise FtError(st, last_error())
    return int(flags.value)


def debug_stream_read(buf, nbytes=None, stream=None):
    """Measurement hook (ft_debug_stream_read): stream the first nbytes (default:
    all, rounded down to 16) of a CUDA tensor through the SMs, nothing written."""
    torch = _torch()
    if not isinstance(buf, torch.Tensor) or not buf.is_cuda or not buf.is_contiguous():
        raise TypeError("buf must be a contiguous CUDA tensor")
    n = buf.numel() * buf.element_size() if nbytes is None else int(nbytes)
    n -= n % 16
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream if stream is None else stream)
    _check(load().ft_debug_stream_read(ctypes.c_void_p(buf.data_ptr()), n, s))


def debug_wait_timeout(limit_ns: int, stream=None):
    """Test hook (ft_debug_wait_timeout): a kernel whose bounded wait gives up
    after limit_ns; the flag it raises is read with read_device_error()."""
    torch = _torch()
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream if stream is None else stream)
    _check(load().ft_debug_wait_timeout(int(limit_ns), s))


def set_path(path) -> int:
    p = PATHS[path] if isinstance(path, str) else int(path)
    prev = load().ft_moe_set_path(p)
    if prev < 0:
        raise ValueError(f"unknown path {path!r}")
    return prev


def selected_path(tokens, top_k, n_experts, nrows, ncols, wtype="q4_0") -> int:
    """The path (FT_PATH_GEMV / FT_PATH_GEMM) the matmul would take for this shape
    and weight type under the current setting, or -1."""
    if wtype == "q4_0":
        return int(load().ft_moe_selected_path(tokens, top_k, n_experts, nrows, ncols))
    return int(load().ft_moe_gguf_selected_path(WEIGHT_TYPES[wtype][0], tokens, top_k, n_experts, nrows, ncols))


def profile_enable(max_calls: int):
    """Record CUDA events around this library's kernels for the next max_calls calls (0 stops)."""
    _check(load().ft_profile_enable(int(max_calls)))


def profile_read() -> dict:
    """Synchronize on the recorded events; summed kernel times (ms), calls and launches; resets."""
    q, r, m = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
    n, nl = ctypes.c_int64(), ctypes.c_int64()
    _check(load().ft_profile_read(ctypes.byref(q), ctypes.byref(r), ctypes.byref(m), ctypes.byref(n),
                                  ctypes.byref(nl)))
    return {"quantize_ms": q.value, "route_ms": r.value, "matmul_ms": m.value, "calls": n.value,
            "launches": nl.value}
