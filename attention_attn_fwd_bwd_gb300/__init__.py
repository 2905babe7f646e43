"""attnfuse-gb300: fused RoPE + variant attention for NVIDIA GB300 (sm_103a).

Thin Python binding over the C ABI declared in ``include/attnfuse.h`` (ctypes; argument
marshalling only — every step of the computation runs in the library's CUDA kernels).
PyTorch supplies device memory and streams. There is no CPU fallback: every call raises
if ``libattnfuse.so`` is missing or fails to load.

Low-level functions carry the C names (``attnfuse_fwd`` ...) and take raw pointers; the
torch-level helpers ``fwd``, ``bwd``, ``decode``, ``rope_prerotate`` and, on a ``PagedCache``,
``paged_append``, ``paged_gather`` and ``paged_decode`` allocate outputs and workspace with torch
and call them on the current CUDA stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import operator
import os
import struct
import threading

__all__ = [
    "ROPE_NONE", "ROPE_FUSED", "ROPE_PREROTATE", "MASK_FULL", "MASK_CAUSAL", "MASK_WINDOW",
    "MASK_BLOCK_SPARSE", "BIAS_NONE", "BIAS_ALIBI", "BIAS_ADDITIVE", "AttnfuseError", "Variant",
    "load", "library_path", "fwd", "bwd", "decode", "rope_prerotate", "device_status",
    "fwd_workspace_size", "bwd_workspace_size", "decode_workspace_size",
    "CACHE_BF16", "CACHE_Q4", "PagedCache", "paged_append", "paged_gather", "paged_decode",
    "paged_decode_workspace_size",
]

ROPE_NONE, ROPE_FUSED, ROPE_PREROTATE, ROPE_AUTO = 0, 1, 2, 3
ROPE_REUSE_TABLE = 0x100
MASK_FULL, MASK_CAUSAL, MASK_WINDOW, MASK_BLOCK_SPARSE = 0, 1, 2, 3
BIAS_NONE, BIAS_ALIBI, BIAS_ADDITIVE = 0, 1, 2
NORM_SOFTMAX, NORM_RELU = 0, 1
CACHE_BF16, CACHE_Q4 = 0, 1
_STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "WORKSPACE_TOO_SMALL",
           4: "CUDA_ERROR", 5: "TIMEOUT", 6: "FP16_RANGE", 7: "PAGE_RANGE"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_lib", "libattnfuse.so")
_lock = threading.Lock()
_lib = None


class AttnfuseError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"attnfuse error {code} ({_STATUS.get(code, '?')}): {msg}")
        self.code = code


class CVariant(ctypes.Structure):
    """Mirror of the C struct attnfuse_variant."""
    _fields_ = [
        ("mask", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("bs_block", ctypes.c_int32),
        ("bs_row_ptr", ctypes.c_void_p),
        ("bs_col_idx", ctypes.c_void_p),
        ("bias", ctypes.c_int32),
        ("add_bias_is_bf16", ctypes.c_int32),
        ("alibi_slopes", ctypes.c_void_p),
        ("add_bias", ctypes.c_void_p),
        ("add_bias_strides", ctypes.c_int64 * 4),
        ("tile_visits", ctypes.c_void_p),
        ("dbias", ctypes.c_void_p),
        ("dbias_strides", ctypes.c_int64 * 4),
        ("normalizer", ctypes.c_int32),
        ("bwd_dq_visits", ctypes.c_void_p),
        ("bwd_dkdv_visits", ctypes.c_void_p),
    ]


class CPagedCache(ctypes.Structure):
    """Mirror of the C struct attnfuse_paged_cache."""
    _fields_ = [
        ("format", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("B", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_strides", ctypes.c_int64 * 4),
        ("v_strides", ctypes.c_int64 * 4),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
        ("k_scale_strides", ctypes.c_int64 * 4),
        ("v_scale_strides", ctypes.c_int64 * 4),
        ("page_table", ctypes.c_void_p),
        ("page_table_stride", ctypes.c_int64),
    ]


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libattnfuse.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise AttnfuseError(4, f"{_LIB_PATH} not built; run __graft_entry__.build() or "
                                   f"python -m attention_attn_fwd_bwd_gb300._build")
        lib = ctypes.CDLL(_LIB_PATH)
        P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        ST = ctypes.POINTER(ctypes.c_int64)
        VP = ctypes.POINTER(CVariant)
        sig = {
            "attnfuse_last_error": ([], ctypes.c_char_p),
            "attnfuse_version": ([], I),
            "attnfuse_device_status": ([P, I, ctypes.POINTER(I)], I),
            "attnfuse_fwd_workspace_size": ([I, I, I, I, I, I, ctypes.POINTER(S)], I),
            "attnfuse_fwd": ([P, ST, P, ST, P, ST, P, ST, P, I, I, I, I, I, F, F, I, VP, P, S, P], I),
            "attnfuse_bwd_workspace_size": ([I, I, I, I, I, I, ctypes.POINTER(S)], I),
            "attnfuse_bwd": ([P, ST, P, ST, P, ST, P, ST, P, P, ST, P, ST, P, ST, P, ST,
                              I, I, I, I, I, F, F, I, VP, P, S, P], I),
            "attnfuse_decode_workspace_size": ([I, I, I, I, I, I, ctypes.POINTER(S)], I),
            "attnfuse_decode": ([P, ST, P, ST, P, ST, P, ST, P, I, I, I, I, I, I, F, F, I, I,
                                 P, S, P], I),
            "attnfuse_decode_auto_splits": ([I, I, I, ctypes.POINTER(I)], I),
            "attnfuse_decode_noalloc": ([P, ST, P, ST, P, ST, P, ST, P, I, I, I, I, I, I, F, F, I,
                                         I, P], I),
            "attnfuse_paged_append": ([P, P, P, P, P, P, P, I, F, I, P], I),
            "attnfuse_paged_gather": ([P, P, P, P, P, P, P, I, P], I),
            "attnfuse_paged_decode_workspace_size": ([I, I, I, I, ctypes.POINTER(S)], I),
            "attnfuse_paged_decode": ([P, P, P, P, P, P, P, I, F, F, I, I, P, P, S, P], I),
            "attnfuse_rope_prerotate": ([P, ST, P, I, I, I, I, F, P, S, P], I),
            "attnfuse_debug_wait_timeout": ([ctypes.c_uint64, P], I),
            "attnfuse_rope_table": ([P, S, I, I, F, P], I),
            "attnfuse_rope_auto_mode": ([I, I, I, ctypes.POINTER(I)], I),
            "attnfuse_fwd_fp8_workspace_size": ([I, I, I, I, I, ctypes.POINTER(S)], I),
            "attnfuse_fwd_host_workspace_size": ([I, I, I, I, I, I, I, ctypes.POINTER(S)], I),
            "attnfuse_fwd_host": ([P, P, P, P, P, I, I, I, I, I, F, F, I, VP, I, P, S, P], I),
            "attnfuse_fwd_fp8": ([P, ST, P, ST, P, ST, P, ST, P, I, I, I, I, I, F, F, F, F, VP,
                                  P, S, P], I),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _check(rc):
    if rc != 0:
        raise AttnfuseError(rc, load().attnfuse_last_error().decode())


def _strides(t, n):
    arr = (ctypes.c_int64 * n)(*t.stride())
    return arr


def _launch_context(device, stream=None):
    """(context manager, stream handle) for a call whose tensors live on `device`.

    The C ABI works on the current CUDA device (its status word, tensor maps and launches), so
    every call runs with the tensors' device made current and, unless the caller passes one,
    on that device's current stream. A stream of another device is rejected."""
    import torch

    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.device(device), ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t, name, dtypes, shape=None, device=None, contiguous=False, ndim=None, dims=""):
    """Reject what the C ABI cannot see through a bare pointer: a tensor that is not on the
    CUDA device of the call (its address would reach a kernel), of another element type, of
    another shape, or (where the call takes no strides) not contiguous."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {dims}, got shape {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(x) for x in dtypes)}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device.type != "cuda" or (device is not None and t.device != device):
        raise ValueError(f"{name}: on {t.device}, expected {device or 'a CUDA device'}")


# ------------------------------------------------------------------------------------------
# C names (raw pointers)
# ------------------------------------------------------------------------------------------
def __getattr__(name):
    if name.startswith("attnfuse_"):
        return getattr(load(), name)
    raise AttributeError(name)


# ------------------------------------------------------------------------------------------
# torch-level helpers
# ------------------------------------------------------------------------------------------
class Variant:
    """Combinator set (paper §3.1). Tensors must live on the device of the attention inputs.

    mask: MASK_*; causal: also require n <= m; window: W for MASK_WINDOW; bs_row_ptr /
    bs_col_idx: int32 CSR block layout (block edge bs_block, 64 or 128); bias: BIAS_*;
    alibi_slopes: fp32 [Hq]; add_bias: fp32 or bf16 tensor broadcastable to [B, Hq, N, N];
    tile_visits: uint8 [B, Hq, ceil(N/128), ceil(N/128)] (debug record of computed tiles);
    bwd_dq_visits / bwd_dkdv_visits: the backward's records, uint8 [B, Hq, ceil(N/128),
    ceil(N/128)] (dQ kernel) and [B, Hq, ceil(N/64), ceil(N/128)] (dK/dV kernel, 64-row blocks);
    dbias: fp32 [B, Hq, N, N] output of the backward with an additive bias (its gradient before
    any broadcast is summed out); norm: NORM_SOFTMAX or NORM_RELU (relu_attention: O_m =
    (1/N) sum_n max(s_mn, 0) v_n, forward only, no LSE).
    """

    def __init__(self, mask=MASK_CAUSAL, causal=False, window=0, bs_block=64, bs_row_ptr=None,
                 bs_col_idx=None, bias=BIAS_NONE, alibi_slopes=None, add_bias=None,
                 tile_visits=None, dbias=None, norm=NORM_SOFTMAX, bwd_dq_visits=None,
                 bwd_dkdv_visits=None):
        self.norm = norm
        self.bwd_dq_visits, self.bwd_dkdv_visits = bwd_dq_visits, bwd_dkdv_visits
        self.mask, self.causal, self.window, self.bs_block = mask, causal, window, bs_block
        self.bs_row_ptr, self.bs_col_idx = bs_row_ptr, bs_col_idx
        self.bias, self.alibi_slopes, self.add_bias = bias, alibi_slopes, add_bias
        self.tile_visits = tile_visits
        self.dbias = dbias

    def check(self, device, B, Hq, N):
        """Validate the variant's tensors for a call on `device` with B, Hq and N (lengths
        the kernels index by; the values of a block-sparse layout are the caller's to keep in
        range, since reading them here would synchronise the stream)."""
        import torch

        if self.mask == MASK_BLOCK_SPARSE:
            if self.bs_row_ptr is None or self.bs_col_idx is None:
                raise ValueError("block-sparse variant: bs_row_ptr and bs_col_idx are required")
            if self.bs_block in (64, 128):
                rows = -(-N // self.bs_block)
                if self.bs_row_ptr.numel() < rows + 1:
                    raise ValueError(f"bs_row_ptr: {self.bs_row_ptr.numel()} entries, "
                                     f"the layout has {rows} block rows (needs {rows + 1})")
            _need(self.bs_row_ptr, "bs_row_ptr", (torch.int32,), device=device, contiguous=True)
            _need(self.bs_col_idx, "bs_col_idx", (torch.int32,), device=device, contiguous=True)
        if self.alibi_slopes is not None:
            if self.alibi_slopes.numel() < Hq:
                raise ValueError(f"alibi_slopes: {self.alibi_slopes.numel()} entries for {Hq} heads")
            _need(self.alibi_slopes, "alibi_slopes", (torch.float32,), device=device, contiguous=True)
        if self.add_bias is not None:
            if self.add_bias.dim() > 4:
                raise ValueError("add_bias: at most 4 dimensions ([B, Hq, N, N])")
            full = (B, Hq, N, N)[4 - self.add_bias.dim():]
            for have, want in zip(self.add_bias.shape, full):
                if have not in (1, want):
                    raise ValueError(f"add_bias: shape {tuple(self.add_bias.shape)} does not "
                                     f"broadcast to {(B, Hq, N, N)}")
            _need(self.add_bias, "add_bias", (torch.float32, torch.bfloat16), device=device)
        if self.tile_visits is not None:
            t = -(-N // 128)
            _need(self.tile_visits, "tile_visits", (torch.uint8,), (B, Hq, t, t), device, True)
        if self.dbias is not None:
            _need(self.dbias, "dbias", (torch.float32,), (B, Hq, N, N), device)
        if self.bwd_dq_visits is not None:
            t = -(-N // 128)
            _need(self.bwd_dq_visits, "bwd_dq_visits", (torch.uint8,), (B, Hq, t, t), device, True)
        if self.bwd_dkdv_visits is not None:
            _need(self.bwd_dkdv_visits, "bwd_dkdv_visits", (torch.uint8,),
                  (B, Hq, -(-N // 64), -(-N // 128)), device, True)

    def c_struct(self):
        v = CVariant()
        v.mask, v.causal, v.window, v.bs_block = self.mask, int(bool(self.causal)), self.window, self.bs_block
        if self.bs_row_ptr is not None:
            v.bs_row_ptr, v.bs_col_idx = self.bs_row_ptr.data_ptr(), self.bs_col_idx.data_ptr()
        v.bias = self.bias
        v.normalizer = self.norm
        if self.alibi_slopes is not None:
            v.alibi_slopes = self.alibi_slopes.data_ptr()
        if self.add_bias is not None:
            import torch

            ab = self.add_bias
            while ab.dim() < 4:
                ab = ab.unsqueeze(0)
            v.add_bias = ab.data_ptr()
            v.add_bias_is_bf16 = int(ab.dtype == torch.bfloat16)
            for i in range(4):
                v.add_bias_strides[i] = ab.stride(i) if ab.size(i) > 1 else 0
        if self.tile_visits is not None:
            v.tile_visits = self.tile_visits.data_ptr()
        if self.bwd_dq_visits is not None:
            v.bwd_dq_visits = self.bwd_dq_visits.data_ptr()
        if self.bwd_dkdv_visits is not None:
            v.bwd_dkdv_visits = self.bwd_dkdv_visits.data_ptr()
        if self.dbias is not None:
            v.dbias = self.dbias.data_ptr()
            for i in range(4):
                v.dbias_strides[i] = self.dbias.stride(i)
        return v


def rope_auto_mode(N, d, backward=False):
    """The mode ROPE_AUTO resolves to (ROPE_FUSED or ROPE_PREROTATE) for N and head dim d."""
    m = ctypes.c_int()
    _check(load().attnfuse_rope_auto_mode(N, d, int(bool(backward)), ctypes.byref(m)))
    return m.value


def fwd_workspace_size(B, Hq, Hkv, N, d, rope_mode):
    n = ctypes.c_size_t()
    _check(load().attnfuse_fwd_workspace_size(B, Hq, Hkv, N, d, rope_mode, ctypes.byref(n)))
    return n.value


def fwd_fp8_workspace_size(B, Hq, Hkv, N, d):
    n = ctypes.c_size_t()
    _check(load().attnfuse_fwd_fp8_workspace_size(B, Hq, Hkv, N, d, ctypes.byref(n)))
    return n.value


def bwd_workspace_size(B, Hq, Hkv, N, d, rope_mode):
    n = ctypes.c_size_t()
    _check(load().attnfuse_bwd_workspace_size(B, Hq, Hkv, N, d, rope_mode, ctypes.byref(n)))
    return n.value


def decode_workspace_size(B, Hq, Hkv, L, d, num_splits):
    n = ctypes.c_size_t()
    _check(load().attnfuse_decode_workspace_size(B, Hq, Hkv, L, d, num_splits, ctypes.byref(n)))
    return n.value


def _workspace(nbytes, device, workspace=None, reuse_table=False):
    """The caller's workspace if it holds nbytes, else a new one. With ROPE_REUSE_TABLE the
    (cos, sin) table must already sit in the caller's workspace, so a missing or too small one
    is an error (a new buffer would hold no table)."""
    import torch

    have = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if have and not workspace.is_contiguous():  # an expanded view has less memory than elements
        have = min(have, workspace.untyped_storage().nbytes() - workspace.storage_offset() * workspace.element_size())
    if reuse_table and (workspace is None or have < nbytes):
        raise ValueError(f"ROPE_REUSE_TABLE needs the workspace that holds the table "
                         f"({nbytes} bytes); got {'none' if workspace is None else f'{have} bytes'}")
    if nbytes == 0:
        return None
    if workspace is not None:
        _need(workspace, "workspace", (workspace.dtype,), device=device)
        if have >= nbytes:
            return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def fwd(q, k, v, scale=None, rope_theta=10000.0, rope_mode=ROPE_FUSED, variant=None,
        out=None, lse=None, with_lse=True, workspace=None, stream=None):
    """Forward: q [B,Hq,N,d], k/v [B,Hkv,N,d] bf16 CUDA tensors -> (out, lse)."""
    import torch

    bf16, f32 = (torch.bfloat16,), (torch.float32,)
    _need(q, "q", bf16, ndim=4, dims="[B, Hq, N, d]")
    B, Hq, N, d = q.shape
    dev = q.device
    _need(k, "k", bf16, ndim=4, dims="[B, Hkv, N, d]")
    Hkv = k.shape[1]
    _need(k, "k", bf16, (B, Hkv, N, d), dev)
    _need(v, "v", bf16, (B, Hkv, N, d), dev)
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", bf16, (B, Hq, N, d), dev)
    relu = variant is not None and variant.norm == NORM_RELU
    if relu and lse is not None:
        raise ValueError("relu_attention has no LSE: pass lse=None")
    if with_lse and lse is None and not relu:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", f32, (B, Hq, N), dev, contiguous=True)
    if variant is not None:
        variant.check(dev, B, Hq, N)
    ws_n = fwd_workspace_size(B, Hq, Hkv, N, d, rope_mode & 0xFF)
    ws = _workspace(ws_n, dev, workspace, bool(rope_mode & ROPE_REUSE_TABLE))
    cv = (variant or Variant()).c_struct()
    ctx, st = _launch_context(dev, stream)
    with ctx:
        _check(load().attnfuse_fwd(
            _ptr(q), _strides(q, 4), _ptr(k), _strides(k, 4), _ptr(v), _strides(v, 4),
            _ptr(out), _strides(out, 4), _ptr(lse), B, Hq, Hkv, N, d, float(scale),
            float(rope_theta), rope_mode, ctypes.byref(cv), _ptr(ws), ws_n, st))
    return out, lse


def fwd_host_workspace_size(B, Hq, Hkv, N, d, rope_mode, chunk_b):
    n = ctypes.c_size_t()
    _check(load().attnfuse_fwd_host_workspace_size(B, Hq, Hkv, N, d, rope_mode, chunk_b,
                                                   ctypes.byref(n)))
    return n.value


def fwd_host(q, k, v, scale=None, rope_theta=10000.0, rope_mode=ROPE_FUSED, variant=None,
             out=None, lse=None, with_lse=True, chunk_b=1, workspace=None, device=None,
             stream=None, sync=True):
    """Forward on CPU tensors (contiguous bf16; pinned memory lets the copies overlap): the
    batch is copied in, attended and copied out in chunks of chunk_b elements, the copies of
    one chunk overlapping the forward of the next. Returns CPU (out, lse); with sync=False the
    results are valid once the device stream has reached this point."""
    import torch

    bf16, f32 = (torch.bfloat16,), (torch.float32,)
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
            raise ValueError(f"{name}: expected a CPU tensor")
        if t.dtype not in bf16:
            raise TypeError(f"{name}: dtype {t.dtype}, expected torch.bfloat16")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous [B, H, N, d] tensor")
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (B, Hkv, N, d) or tuple(v.shape) != (B, Hkv, N, d):
        raise ValueError("k, v: expected [B, Hkv, N, d] matching q")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if scale is None:
        scale = d ** -0.5
    pin = q.is_pinned()
    if out is None:
        out = torch.empty((B, Hq, N, d), dtype=torch.bfloat16, pin_memory=pin)
    relu = variant is not None and variant.norm == NORM_RELU
    if with_lse and lse is None and not relu:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, pin_memory=pin)
    for t, name, dt, shape in ((out, "out", bf16, (B, Hq, N, d)), (lse, "lse", f32, (B, Hq, N))):
        if t is None:
            continue
        if t.device.type != "cpu" or t.dtype not in dt or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous CPU {dt[0]} tensor of shape {shape}")
    if variant is not None:
        variant.check(dev, B, Hq, N)
    ws_n = fwd_host_workspace_size(B, Hq, Hkv, N, d, rope_mode, chunk_b)
    ws = _workspace(ws_n, dev, workspace)
    cv = (variant or Variant()).c_struct()
    ctx, st = _launch_context(dev, stream)
    with ctx:
        _check(load().attnfuse_fwd_host(
            _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, N, d, float(scale),
            float(rope_theta), rope_mode, ctypes.byref(cv), int(chunk_b), _ptr(ws), ws_n, st))
        if sync:
            torch.cuda.current_stream(dev).synchronize() if stream is None else stream.synchronize()
    return out, lse


def fwd_fp8(q, k, v, q_scale, k_scale, v_scale, scale=None, variant=None, out=None, lse=None,
            with_lse=True, workspace=None, stream=None):
    """e4m3 forward (head dim 128): q [B,Hq,N,128], k/v [B,Hkv,N,128] as torch.uint8 (raw
    e4m3 bytes) or torch.float8_e4m3fn CUDA tensors; attends over q_scale*q, k_scale*k and
    v_scale*v; returns (out bf16, lse fp32). No RoPE: q and k are used as given."""
    import torch

    f8 = tuple(t for t in (torch.uint8, getattr(torch, "float8_e4m3fn", None)) if t is not None)
    bf16, f32 = (torch.bfloat16,), (torch.float32,)
    _need(q, "q", f8, ndim=4, dims="[B, Hq, N, d]")
    B, Hq, N, d = q.shape
    dev = q.device
    _need(k, "k", f8, ndim=4, dims="[B, Hkv, N, d]")
    Hkv = k.shape[1]
    _need(k, "k", f8, (B, Hkv, N, d), dev)
    _need(v, "v", f8, (B, Hkv, N, d), dev)
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty((B, Hq, N, d), dtype=torch.bfloat16, device=dev)
    _need(out, "out", bf16, (B, Hq, N, d), dev)
    relu = variant is not None and variant.norm == NORM_RELU
    if relu and lse is not None:
        raise ValueError("relu_attention has no LSE: pass lse=None")
    if with_lse and lse is None and not relu:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=dev)
    if lse is not None:
        _need(lse, "lse", f32, (B, Hq, N), dev, contiguous=True)
    if variant is not None:
        variant.check(dev, B, Hq, N)
    ws_n = fwd_fp8_workspace_size(B, Hq, Hkv, N, d)
    ws = _workspace(ws_n, dev, workspace)
    cv = (variant or Variant()).c_struct()
    ctx, st = _launch_context(dev, stream)
    with ctx:
        _check(load().attnfuse_fwd_fp8(
            _ptr(q), _strides(q, 4), _ptr(k), _strides(k, 4), _ptr(v), _strides(v, 4),
            _ptr(out), _strides(out, 4), _ptr(lse), B, Hq, Hkv, N, d, float(scale),
            float(q_scale), float(k_scale), float(v_scale), ctypes.byref(cv), _ptr(ws), ws_n, st))
    return out, lse


def bwd(q, k, v, out, lse, dout, scale=None, rope_theta=10000.0, rope_mode=ROPE_FUSED,
        variant=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward (paper §4.4): returns (dq, dk, dv) w.r.t. the un-rotated q, k and v."""
    import torch

    bf16, f32 = (torch.bfloat16,), (torch.float32,)
    _need(q, "q", bf16, ndim=4, dims="[B, Hq, N, d]")
    B, Hq, N, d = q.shape
    dev = q.device
    _need(k, "k", bf16, ndim=4, dims="[B, Hkv, N, d]")
    Hkv = k.shape[1]
    _need(k, "k", bf16, (B, Hkv, N, d), dev)
    _need(v, "v", bf16, (B, Hkv, N, d), dev)
    _need(out, "out", bf16, (B, Hq, N, d), dev)
    _need(lse, "lse", f32, (B, Hq, N), dev, contiguous=True)
    _need(dout, "dout", bf16, (B, Hq, N, d), dev)
    if scale is None:
        scale = d ** -0.5
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _need(dq, "dq", bf16, (B, Hq, N, d), dev)
    _need(dk, "dk", bf16, (B, Hkv, N, d), dev)
    _need(dv, "dv", bf16, (B, Hkv, N, d), dev)
    if variant is not None:
        variant.check(dev, B, Hq, N)
    ws_n = bwd_workspace_size(B, Hq, Hkv, N, d, rope_mode & 0xFF)
    ws = _workspace(ws_n, dev, workspace, bool(rope_mode & ROPE_REUSE_TABLE))
    cv = (variant or Variant()).c_struct()
    ctx, st = _launch_context(dev, stream)
    with ctx:
        _check(load().attnfuse_bwd(
            _ptr(q), _strides(q, 4), _ptr(k), _strides(k, 4), _ptr(v), _strides(v, 4),
            _ptr(out), _strides(out, 4), _ptr(lse), _ptr(dout), _strides(dout, 4),
            _ptr(dq), _strides(dq, 4), _ptr(dk), _strides(dk, 4), _ptr(dv), _strides(dv, 4),
            B, Hq, Hkv, N, d, float(scale), float(rope_theta), rope_mode, ctypes.byref(cv),
            _ptr(ws), ws_n, st))
    return dq, dk, dv


def decode(q, k_cache, v_cache, q_pos, scale=None, rope_theta=10000.0, rope_mode=ROPE_FUSED,
           num_splits=0, out=None, lse=None, with_lse=True, workspace=None, stream=None):
    """Split-KV decode (paper §4.2): q [B,Hq,d], caches [B,Hkv,L,d] -> (out [B,Hq,d], lse)."""
    import torch

    bf16 = (torch.bfloat16,)
    _need(q, "q", bf16, ndim=3, dims="[B, Hq, d]")
    B, Hq, d = q.shape
    dev = q.device
    _need(k_cache, "k_cache", bf16, ndim=4, dims="[B, Hkv, L, d]")
    Hkv, L = k_cache.shape[1], k_cache.shape[2]
    _need(k_cache, "k_cache", bf16, (B, Hkv, L, d), dev)
    _need(v_cache, "v_cache", bf16, (B, Hkv, L, d), dev)
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", bf16, (B, Hq, d), dev)
    if with_lse and lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", (torch.float32,), (B, Hq), dev, contiguous=True)
    ws_n = decode_workspace_size(B, Hq, Hkv, L, d, num_splits)
    ws = _workspace(ws_n, dev, workspace)
    ctx, st = _launch_context(dev, stream)
    with ctx:
        _check(load().attnfuse_decode(
            _ptr(q), _strides(q, 3), _ptr(k_cache), _strides(k_cache, 4), _ptr(v_cache),
            _strides(v_cache, 4), _ptr(out), _strides(out, 3), _ptr(lse), B, Hq, Hkv, L, d,
            int(q_pos), float(scale), float(rope_theta), rope_mode, int(num_splits), _ptr(ws),
            ws_n, st))
    return out, lse


def decode_auto_splits(B, Hkv, L):
    n = ctypes.c_int()
    _check(load().attnfuse_decode_auto_splits(B, Hkv, L, ctypes.byref(n)))
    return n.value


def rope_prerotate(x, rope_theta, out=None, workspace=None, stream=None):
    """x [B,H,N,d] bf16 -> R_n x (contiguous)."""
    import torch

    _need(x, "x", (torch.bfloat16,), ndim=4, dims="[B, H, N, d]")
    B, H, N, d = x.shape
    out = torch.empty((B, H, N, d), dtype=x.dtype, device=x.device) if out is None else out
    _need(out, "out", (torch.bfloat16,), (B, H, N, d), x.device, contiguous=True)
    ws_n = fwd_workspace_size(B, H, H, N, d, ROPE_FUSED)
    ws = _workspace(ws_n, x.device, workspace)
    ctx, st = _launch_context(x.device, stream)
    with ctx:
        _check(load().attnfuse_rope_prerotate(_ptr(x), _strides(x, 4), _ptr(out), B, H, N, d,
                                              float(rope_theta), _ptr(ws), ws_n, st))
    return out


# Paged caches. A decode step on a small batch is a few microseconds on the GPU, so the binding's
# own cost counts here: checks that pass touch each tensor once (_need runs for the message of
# one that does not), and what goes to the C ABI by address is packed into bytes: a cache's struct
# once, strides per call.
_S3, _S4 = struct.Struct("@3q").pack, struct.Struct("@4q").pack
_CACHE = struct.Struct("@7i2P8q2P8qPq")  # the fields of CPagedCache
assert _CACHE.size == ctypes.sizeof(CPagedCache)


def _live_strides(t):
    """Element strides with those of one-element dimensions, which address nothing and may hold
    any value, replaced by what a contiguous tensor would have."""
    st, shape = t.stride(), t.shape
    if 1 in shape:
        st = list(st)
        inner = 1
        for i in range(len(st) - 1, -1, -1):
            if shape[i] == 1:
                st[i] = inner
            elif st[i] * shape[i] > inner:
                inner = st[i] * shape[i]
    return st


def _want(t, name, dtype, shape, device, contiguous=False):
    if not (getattr(t, "dtype", None) is dtype and t.shape == shape and t.device == device
            and (not contiguous or t.is_contiguous())):
        _need(t, name, (dtype,), shape, device, contiguous)


_CURRENT = contextlib.nullcontext()


def _on(stream, device):
    """Context for allocations that a call on `stream` uses: made on another stream, their memory
    could be handed to that stream's work again while the call still runs."""
    import torch

    if stream is None:
        return _CURRENT
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _launch(fn, args, device, stream):
    """fn(*args, stream) on `device`: as in _launch_context, but without making the device current
    where it is."""
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if stream is None and raw is not None and device.index == torch._C._cuda_getDevice():
        rc = fn(*args, raw(device.index))
        if rc:
            _check(rc)
        return
    ctx, st = _launch_context(device, stream)
    with ctx:
        _check(fn(*args, st))


class PagedCache:
    """A key/value cache in pages (attnfuse_paged_cache): pools, and a table of pages per sequence.

    k, v: bf16 [num_pages, Hkv, page_size, d], or for the 4-bit format uint8 [num_pages, Hkv,
    page_size, d/2] with k_scales, v_scales bf16 [num_pages, Hkv, page_size, d/32]. page_table:
    int32 [B, max_pages]; position p of sequence b is slot p % page_size of page
    page_table[b, p // page_size]. The object holds references only, and its tensors cannot be
    exchanged: the caller allocates pages, fills the table in place (or makes another PagedCache
    over the same pools) and keeps the lengths. page_size: a multiple of 16.
    """

    __slots__ = ("_tensors", "_c", "q4", "format", "device", "num_pages", "Hkv", "page_size", "d", "B", "max_pages")

    def __init__(self, k, v, page_table, k_scales=None, v_scales=None):
        import torch

        bf16 = torch.bfloat16
        dt = getattr(k, "dtype", None)
        q4 = dt is torch.uint8
        if not (q4 or dt is bf16) or k.dim() != 4 or not k.is_cuda:
            _need(k, "cache k", (torch.uint8,) if q4 else (bf16, torch.uint8), ndim=4,
                  dims="[num_pages, Hkv, page_size, d/2]" if q4 else "[num_pages, Hkv, page_size, d]")
        shape, dev = k.shape, k.device
        P, H, S, d = shape
        _want(v, "cache v", dt, shape, dev)
        if q4:
            d *= 2
            steps = (P, H, S, d // 32)
            _want(k_scales, "cache k_scales", bf16, steps, dev)
            _want(v_scales, "cache v_scales", bf16, steps, dev)
            scales = (k_scales.data_ptr(), v_scales.data_ptr(), *_live_strides(k_scales), *_live_strides(v_scales))
        elif k_scales is not None or v_scales is not None:
            raise ValueError("k_scales, v_scales belong to the 4-bit format (uint8 pools)")
        else:
            scales = _NO_SCALES
        if getattr(page_table, "dtype", None) is not torch.int32 or page_table.dim() != 2 or page_table.device != dev:
            _need(page_table, "page_table", (torch.int32,), ndim=2, dims="[B, max_pages]", device=dev)
        B, max_pages = page_table.shape
        row, one = page_table.stride()
        if max_pages > 1 and one != 1:
            raise ValueError("page_table: rows must be contiguous")
        self._tensors = (k, v, page_table, k_scales, v_scales)
        self.q4, self.device = q4, dev
        self.format = fmt = CACHE_Q4 if q4 else CACHE_BF16
        self.num_pages, self.Hkv, self.page_size, self.d, self.B, self.max_pages = P, H, S, d, B, max_pages
        self._c = _CACHE.pack(fmt, P, H, S, d, B, max_pages, k.data_ptr(), v.data_ptr(), *_live_strides(k), *_live_strides(v),
                              *scales, page_table.data_ptr(), row)

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    page_table = property(lambda self: self._tensors[2])
    k_scales = property(lambda self: self._tensors[3])
    v_scales = property(lambda self: self._tensors[4])

    @classmethod
    def empty(cls, num_pages, Hkv, page_size, d, page_table, q4=False):
        """A cache with newly allocated (uninitialised) pools on page_table's device."""
        import torch

        dev = page_table.device
        new = lambda row, dt: torch.empty((num_pages, Hkv, page_size, row), dtype=dt, device=dev)  # noqa: E731
        if not q4:
            return cls(new(d, torch.bfloat16), new(d, torch.bfloat16), page_table)
        return cls(new(d // 2, torch.uint8), new(d // 2, torch.uint8), page_table,
                   new(d // 32, torch.bfloat16), new(d // 32, torch.bfloat16))


_NO_SCALES = (0,) * 10


def _need_cache(cache):
    raise TypeError(f"cache: expected a PagedCache, got {type(cache).__name__}")


def _index(t, name, cache):
    """Address of an int32 [B] tensor, or None."""
    import torch

    if t is None:
        return None
    _want(t, name, torch.int32, (cache.B,), cache.device, contiguous=True)
    return t.data_ptr()


def paged_append(cache, k, v, start, count=None, rope_theta=10000.0, rope_mode=ROPE_FUSED, stream=None):
    """Write rows into the cache: k, v [B, Hkv, N, d] bf16; row n < count[b] of sequence b becomes
    position start[b] + n (start, count: int32 [B] device tensors; count None: all N). K is
    rotated at its position on the way (rope_mode ROPE_FUSED) or taken as it is (ROPE_NONE)."""
    import torch

    if not isinstance(cache, PagedCache):
        _need_cache(cache)
    bf16, dev = torch.bfloat16, cache.device
    if getattr(k, "dtype", None) is not bf16 or k.dim() != 4:
        _need(k, "k", (bf16,), ndim=4, dims="[B, Hkv, N, d]")
    N = k.shape[2]
    shape = (cache.B, cache.Hkv, N, cache.d)
    _want(k, "k", bf16, shape, dev)
    _want(v, "v", bf16, shape, dev)
    if start is None:
        raise TypeError("start: expected an int32 [B] tensor")
    _launch(load().attnfuse_paged_append,
            (cache._c, k.data_ptr(), _S4(*_live_strides(k)), v.data_ptr(), _S4(*_live_strides(v)),
             _index(start, "start", cache), _index(count, "count", cache), N, rope_theta, rope_mode), dev, stream)


def paged_gather(cache, start, count, N, k=None, v=None, stream=None):
    """Read rows back: positions start[b] .. start[b] + count[b] - 1 (start None: from 0; count None:
    N rows) into rows 0 .. of k, v [B, Hkv, N, d] bf16, zeros behind. Returns (k, v)."""
    import torch

    if not isinstance(cache, PagedCache):
        _need_cache(cache)
    bf16, dev, N = torch.bfloat16, cache.device, operator.index(N)
    shape = (cache.B, cache.Hkv, N, cache.d)
    dense = N * cache.d
    ks = vs = _S4(cache.Hkv * dense, dense, cache.d, 1)
    if k is not None:
        _want(k, "k", bf16, shape, dev)
        ks = _S4(*_live_strides(k))
    if v is not None:
        _want(v, "v", bf16, shape, dev)
        vs = _S4(*_live_strides(v))
    with _on(stream, dev):
        k = torch.empty(shape, dtype=bf16, device=dev) if k is None else k
        v = torch.empty(shape, dtype=bf16, device=dev) if v is None else v
    _launch(load().attnfuse_paged_gather,
            (cache._c, _index(start, "start", cache), _index(count, "count", cache), k.data_ptr(), ks, v.data_ptr(), vs, N),
            dev, stream)
    return k, v


def paged_decode_workspace_size(Hq, Hkv, d, cache_format):
    """Bytes of workspace for paged_decode on the current device (independent of the lengths and of
    B; the two cache formats need different ones)."""
    n = ctypes.c_size_t()
    _check(load().attnfuse_paged_decode_workspace_size(Hq, Hkv, d, cache_format, ctypes.byref(n)))
    return n.value


_paged_sizes = {}  # (device index, Hq, Hkv, d, format) -> workspace bytes


def _paged_workspace_size(device, *key):
    import torch

    with torch.cuda.device(device):
        n = _paged_sizes[(device.index,) + key] = paged_decode_workspace_size(*key)
    return n


def paged_decode(q, cache, lens, scale=None, rope_theta=10000.0, rope_mode=ROPE_FUSED, window=0,
                 alibi_slopes=None, out=None, lse=None, with_lse=True, workspace=None, stream=None):
    """Decode over a paged cache: q [B, Hq, d] bf16 at position lens[b] - 1 against positions
    n < lens[b] (window > 0: the last `window` of them) -> (out [B, Hq, d], lse [B, Hq]).
    lens: int32 [B] device tensor (0: out 0, lse -inf); alibi_slopes: fp32 [Hq], adds
    slope_h (n - (lens[b] - 1)) to the scores. With a stream, what the call allocates belongs to
    that stream."""
    import torch

    if not isinstance(cache, PagedCache):
        _need_cache(cache)
    bf16, f32, dev, B, d = torch.bfloat16, torch.float32, cache.device, cache.B, cache.d
    if getattr(q, "dtype", None) is not bf16 or q.dim() != 3:
        _need(q, "q", (bf16,), ndim=3, dims="[B, Hq, d]")
    Hq = q.shape[1]
    shape = (B, Hq, d)
    _want(q, "q", bf16, shape, dev)
    if lens is None:
        raise TypeError("lens: expected an int32 [B] tensor")
    if alibi_slopes is not None:
        _want(alibi_slopes, "alibi_slopes", f32, (Hq,), dev, contiguous=True)
        alibi_slopes = alibi_slopes.data_ptr()
    os_ = _S3(Hq * d, d, 1)
    if out is not None:
        _want(out, "out", bf16, shape, dev)
        os_ = _S3(*_live_strides(out))
    if lse is not None:
        _want(lse, "lse", f32, (B, Hq), dev, contiguous=True)
    ws_n = _paged_sizes.get((dev.index, Hq, cache.Hkv, d, cache.format))
    if ws_n is None:
        ws_n = _paged_workspace_size(dev, Hq, cache.Hkv, d, cache.format)
    with _on(stream, dev):
        if out is None:
            out = torch.empty(shape, dtype=bf16, device=dev)
        if lse is None and with_lse:
            lse = torch.empty((B, Hq), dtype=f32, device=dev)
        if workspace is None:
            workspace = torch.empty(ws_n, dtype=torch.uint8, device=dev)
        else:
            workspace = _workspace(ws_n, dev, workspace)
    _launch(load().attnfuse_paged_decode,
            (cache._c, q.data_ptr(), _S3(*_live_strides(q)), _index(lens, "lens", cache), out.data_ptr(), os_,
             None if lse is None else lse.data_ptr(), Hq, d ** -0.5 if scale is None else scale, rope_theta, rope_mode,
             max(-1, min(window, 0x7FFFFFFF)), alibi_slopes, workspace.data_ptr(), ws_n), dev, stream)
    return out, lse


def device_status(clear=True, stream=None, device=None):
    """Synchronise and return the device status of `device` (default: the stream's device,
    else the current device): 0 OK, 5 TIMEOUT (a kernel gave up waiting), 6 FP16_RANGE (a
    rotating-mode forward saturated an fp16 Q' / K' element or met a non-finite input), 7 PAGE_RANGE
    (a paged-cache call skipped rows on a page, or with a start, length or count, out of range)."""
    import torch

    if device is None:
        device = stream.device if stream is not None else torch.device("cuda", torch.cuda.current_device())
    code = ctypes.c_int()
    ctx, st = _launch_context(device, stream)
    with ctx:
        _check(load().attnfuse_device_status(st, int(clear), ctypes.byref(code)))
    return code.value
