"""Python binding of the wlq C ABI (include/wlq.h): argument marshalling only.

Every step of the quantization and of the Linear runs in the CUDA library
``libwlq.so`` (sm_100a); this module only turns torch tensors into pointers,
sizes and the current stream.  PyTorch provides device memory and streams.
There is no fallback: if the library is missing or fails to load, importing
this package raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libwlq.so")

OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_NONFINITE, ERR_WORKSPACE, ERR_TIMEOUT, ERR_CUDA, \
    ERR_INDEX = range(10)
OUT_BF16, OUT_F32 = 0, 1
STATUS_NAMES = {
    OK: "WLQ_OK", ERR_INVALID_ARG: "WLQ_ERR_INVALID_ARG", ERR_SHAPE: "WLQ_ERR_SHAPE",
    ERR_ALIGN: "WLQ_ERR_ALIGN", ERR_UNSUPPORTED: "WLQ_ERR_UNSUPPORTED",
    ERR_NONFINITE: "WLQ_ERR_NONFINITE", ERR_WORKSPACE: "WLQ_ERR_WORKSPACE",
    ERR_TIMEOUT: "WLQ_ERR_TIMEOUT", ERR_CUDA: "WLQ_ERR_CUDA", ERR_INDEX: "WLQ_ERR_INDEX",
}
EXPORTS = ("wlq_quantize", "wlq_quantize_pack", "wlq_quantize_ex", "wlq_quantize_fp8", "wlq_packed_bytes",
           "wlq_pack", "wlq_unpack", "wlq_linear_workspace", "wlq_linear", "wlq_linear_noalloc",
           "wlq_lowrank_workspace", "wlq_lowrank_split", "wlq_lowrank_residual", "wlq_nvfp4_scales_bytes",
           "wlq_nvfp4_quantize", "wlq_nvfp4_linear_workspace", "wlq_nvfp4_linear", "wlq_w4a4_workspace",
           "wlq_w4a4_linear", "wlq_qk_norm_rope", "wlq_kv4_append", "wlq_kv4_read", "wlq_kv4_attention",
           "wlq_int8_linear", "wlq_w8a8_linear", "wlq_get_status",
           "wlq_probe_wait_timeout", "wlq_set_grid_limit", "wlq_last_error", "wlq_version")

if not os.path.exists(LIB_PATH):
    raise ImportError("libwlq.so is not built; run `python weight_only_quantized_rtn_b200/_build.py`")

lib = ctypes.CDLL(LIB_PATH)
_i64, _i32, _vp, _sz, _u64 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint64
_f64 = ctypes.c_double
lib.wlq_quantize.argtypes = [_vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp]
lib.wlq_packed_bytes.argtypes = [_i64, _i64, _i32, _i32]
lib.wlq_packed_bytes.restype = _sz
lib.wlq_pack.argtypes = [_vp, _vp, _i64, _i64, _i32, _i32, _vp, _vp]
lib.wlq_unpack.argtypes = [_vp, _i64, _i64, _i32, _i32, _vp, _vp]
lib.wlq_quantize_pack.argtypes = [_vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp]
lib.wlq_quantize_ex.argtypes = [_vp, _i32, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _vp]
lib.wlq_quantize_fp8.argtypes = [_vp, _i32, _i64, _i64, _i32, _vp, _vp, _vp]
lib.wlq_linear_workspace.argtypes = [_i64, _i64, _i64, _i32, _i32, _i32]
lib.wlq_linear_workspace.restype = _sz
lib.wlq_linear.argtypes = [_vp, _i64, _vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _sz, _vp]
lib.wlq_linear_noalloc.argtypes = [_vp, _i64, _vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _vp]
lib.wlq_lowrank_workspace.argtypes = [_i64, _i64, _i32, _i32]
lib.wlq_lowrank_workspace.restype = _sz
lib.wlq_lowrank_split.argtypes = [_vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
lib.wlq_lowrank_residual.argtypes = [_vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp]
lib.wlq_nvfp4_scales_bytes.argtypes = [_i64, _i64]
lib.wlq_nvfp4_scales_bytes.restype = _sz
lib.wlq_nvfp4_quantize.argtypes = [_vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp]
lib.wlq_nvfp4_linear_workspace.argtypes = [_i64, _i64, _i64, _i32]
lib.wlq_nvfp4_linear_workspace.restype = _sz
lib.wlq_nvfp4_linear.argtypes = [_vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _i32,
                                 _vp, _sz, _vp]
lib.wlq_w4a4_workspace.argtypes = [_i64, _i64, _i64, _i32]
lib.wlq_w4a4_workspace.restype = _sz
lib.wlq_w4a4_linear.argtypes = [_vp, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _sz, _vp]
lib.wlq_qk_norm_rope.argtypes = [_vp, _i64, _i32, _vp, _i64, _i32, _i64, _i32, _vp, _vp, _f64, _vp, _i32, _vp, _i32, _vp,
                                 _i32, _vp, _i64, _vp, _i64, _vp]
lib.wlq_kv4_append.argtypes = [_vp, _i64, _vp, _i64, _i64, _i32, _i32, _vp, _f64, _vp, _i32, _vp, _i32, _vp, _i32,
                               _vp, _vp, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _vp]
lib.wlq_kv4_read.argtypes = [_vp, _vp, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i64, _i32, _i32,
                             _vp, _vp, _vp]
lib.wlq_kv4_attention_workspace.argtypes = [_i64, _i32, _i32, _i64, _i32, _i32, _i32]
lib.wlq_kv4_attention_workspace.restype = _sz
lib.wlq_kv4_attention.argtypes = [_vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _i32, _i32, _i64, _vp, _i64, _vp, _vp, _vp, _vp,
                                  _i64, _i32, _i32, ctypes.c_float, _i32, _i32, _vp, _vp, _vp, _sz, _vp]
lib.wlq_int8_linear.argtypes = [_vp, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _i32, _vp]
lib.wlq_w8a8_workspace.argtypes = [_i64, _i64]
lib.wlq_w8a8_workspace.restype = _sz
lib.wlq_w8a8_linear.argtypes = [_vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _i32, _vp, _sz, _vp]
lib.wlq_get_status.argtypes = [_vp]
lib.wlq_probe_wait_timeout.argtypes = [_u64, _vp]
lib.wlq_set_grid_limit.argtypes = [_i32]
lib.wlq_set_grid_limit.restype = None
lib.wlq_last_error.restype = ctypes.c_char_p
lib.wlq_version.restype = ctypes.c_char_p
for _f in ("wlq_quantize", "wlq_quantize_pack", "wlq_quantize_ex", "wlq_quantize_fp8", "wlq_pack", "wlq_unpack", "wlq_linear",
           "wlq_linear_noalloc", "wlq_lowrank_split", "wlq_lowrank_residual", "wlq_nvfp4_quantize", "wlq_nvfp4_linear",
           "wlq_w4a4_linear", "wlq_qk_norm_rope", "wlq_kv4_append", "wlq_kv4_read", "wlq_kv4_attention",
           "wlq_int8_linear", "wlq_w8a8_linear", "wlq_get_status",
           "wlq_probe_wait_timeout"):
    getattr(lib, _f).restype = ctypes.c_int


class WlqError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, status), msg))
        self.status = status


def _check(rc: int):
    if rc != OK:
        raise WlqError(rc, lib.wlq_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if not torch.cuda.is_initialized():
        torch.cuda.init()
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())  # torch.cuda.current_stream(), without the object


def groups(K: int, group: int) -> int:
    return 1 if group == 0 else K // group


def quantize(W: torch.Tensor, bits: int, group: int, stream=None):
    """RTN symmetric quantization of fp32 W [N, K] -> (codes int8 [N,K], scales fp32 [N,G])."""
    assert W.dtype == torch.float32 and W.is_cuda and W.is_contiguous()
    N, K = W.shape
    codes = torch.empty((N, K), dtype=torch.int8, device=W.device)
    scales = torch.empty((N, groups(K, group)), dtype=torch.float32, device=W.device)
    _check(lib.wlq_quantize(_ptr(W), N, K, bits, group, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


SCALE_F32, SCALE_F16, SCALE_BF16 = 0, 1, 2
_SCALE_TORCH = {SCALE_F32: torch.float32, SCALE_F16: torch.float16, SCALE_BF16: torch.bfloat16}


def _in_dtype(W: torch.Tensor) -> int:
    if W.dtype == torch.float32:
        return 0
    if W.dtype == torch.bfloat16:
        return 1
    raise WlqError(ERR_UNSUPPORTED, "input must be fp32 or bf16")


def quantize_ex(W: torch.Tensor, bits: int, group: int, scale_dtype: int = SCALE_F32, stream=None):
    """RTN for 2..8 bits from fp32 or bf16 W [N, K] -> (codes int8 [N,K], scales [N,G] in scale_dtype)."""
    assert W.is_cuda and W.is_contiguous()
    N, K = W.shape
    codes = torch.empty((N, K), dtype=torch.int8, device=W.device)
    scales = torch.empty((N, groups(K, group)), dtype=_SCALE_TORCH[scale_dtype], device=W.device)
    _check(lib.wlq_quantize_ex(_ptr(W), _in_dtype(W), N, K, bits, group, scale_dtype, _ptr(codes), _ptr(scales),
                               _stream(stream)))
    return codes, scales


def quantize_fp8(W: torch.Tensor, group: int, stream=None):
    """fp8 e4m3 block quantization of fp32 or bf16 W [N, K] -> (codes uint8 [N,K], scales fp32 [N,G])."""
    assert W.is_cuda and W.is_contiguous()
    N, K = W.shape
    codes = torch.empty((N, K), dtype=torch.uint8, device=W.device)
    scales = torch.empty((N, groups(K, group)), dtype=torch.float32, device=W.device)
    _check(lib.wlq_quantize_fp8(_ptr(W), _in_dtype(W), N, K, group, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def packed_bytes(N: int, K: int, bits: int, group: int) -> int:
    return int(lib.wlq_packed_bytes(N, K, bits, group))


def pack(codes: torch.Tensor, scales: torch.Tensor, bits: int, group: int, stream=None) -> torch.Tensor:
    N, K = codes.shape
    nbytes = packed_bytes(N, K, bits, group)
    if nbytes == 0:
        raise WlqError(ERR_UNSUPPORTED, "no packed layout for bits=%d group=%d K=%d" % (bits, group, K))
    out = torch.empty(nbytes, dtype=torch.uint8, device=codes.device)
    _check(lib.wlq_pack(_ptr(codes), _ptr(scales), N, K, bits, group, _ptr(out), _stream(stream)))
    return out


def quantize_pack(W: torch.Tensor, bits: int, group: int, stream=None):
    """quantize then pack in one pass: fp32 W [N, K] -> (scales fp32 [N,G], packed uint8)."""
    assert W.dtype == torch.float32 and W.is_cuda and W.is_contiguous()
    N, K = W.shape
    nbytes = packed_bytes(N, K, bits, group)
    if nbytes == 0:
        raise WlqError(ERR_UNSUPPORTED, "no packed layout for bits=%d group=%d K=%d" % (bits, group, K))
    scales = torch.empty((N, groups(K, group)), dtype=torch.float32, device=W.device)
    out = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    _check(lib.wlq_quantize_pack(_ptr(W), N, K, bits, group, _ptr(scales), _ptr(out), _stream(stream)))
    return scales, out


def unpack(packed: torch.Tensor, N: int, K: int, bits: int, group: int, stream=None) -> torch.Tensor:
    codes = torch.empty((N, K), dtype=torch.int8, device=packed.device)
    _check(lib.wlq_unpack(_ptr(packed), N, K, bits, group, _ptr(codes), _stream(stream)))
    return codes


def workspace_bytes(M: int, N: int, K: int, bits: int, group: int, r: int = 0) -> int:
    return int(lib.wlq_linear_workspace(M, N, K, bits, group, r))


def new_workspace(M, N, K, bits, group, r=0, device="cuda"):
    """A zero-filled workspace of the size wlq_linear needs (None when it needs none)."""
    n = workspace_bytes(M, N, K, bits, group, r)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def linear_into(y, x, packed, N, K, bits, group, bias=None, L1=None, L2=None, workspace=None, stream=None):
    """y = x deq(W)^T [+ (x L1) L2] [+ b] into a preallocated y (bf16 or fp32 [M, N])."""
    M = x.shape[0]
    r = 0 if L1 is None else L1.shape[1]
    out = OUT_F32 if y.dtype == torch.float32 else OUT_BF16
    ws_n = 0 if workspace is None else workspace.numel()
    _check(lib.wlq_linear(_ptr(x), M, _ptr(packed), N, K, bits, group, _ptr(bias), _ptr(L1), _ptr(L2), r,
                          _ptr(y), out, _ptr(workspace), ws_n, _stream(stream)))
    return y


def linear(x, packed, N, K, bits, group, bias=None, L1=None, L2=None, out_dtype=torch.bfloat16,
           workspace=None, stream=None):
    assert x.dtype == torch.bfloat16 and x.is_contiguous()
    M = x.shape[0]
    y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    r = 0 if L1 is None else L1.shape[1]
    if workspace is None:
        workspace = new_workspace(M, N, K, bits, group, r, device=x.device)
    return linear_into(y, x, packed, N, K, bits, group, bias, L1, L2, workspace, stream)


def linear_noalloc_into(y, x, packed, N, K, bits, group, bias=None, L1=None, L2=None, stream=None):
    """wlq_linear_noalloc: like linear_into, with the library's built-in scratch."""
    M = x.shape[0]
    r = 0 if L1 is None else L1.shape[1]
    out = OUT_F32 if y.dtype == torch.float32 else OUT_BF16
    _check(lib.wlq_linear_noalloc(_ptr(x), M, _ptr(packed), N, K, bits, group, _ptr(bias), _ptr(L1), _ptr(L2), r,
                                  _ptr(y), out, _stream(stream)))
    return y


def lowrank_split(W: torch.Tensor, r: int, omega: torch.Tensor, power_iters: int = 2, stream=None):
    """Top-r split of W's transpose for the low-rank branch: fp32 W [N, K] and a
    caller-drawn test matrix omega fp32 [N, l] -> (L1 bf16 [K, r], L2 bf16
    [r, N], sigma fp32 [r])."""
    assert W.dtype == torch.float32 and W.is_cuda and W.is_contiguous()
    N, K = W.shape
    l = omega.shape[1]
    L1 = torch.empty((K, r), dtype=torch.bfloat16, device=W.device)
    L2 = torch.empty((r, N), dtype=torch.bfloat16, device=W.device)
    sigma = torch.empty(r, dtype=torch.float32, device=W.device)
    n = int(lib.wlq_lowrank_workspace(N, K, r, l))
    if n == 0:
        raise WlqError(ERR_SHAPE, "no low-rank split for N=%d K=%d r=%d l=%d" % (N, K, r, l))
    ws = torch.empty(n, dtype=torch.uint8, device=W.device)
    _check(lib.wlq_lowrank_split(_ptr(W), N, K, r, l, power_iters, _ptr(omega), _ptr(L1), _ptr(L2), _ptr(sigma),
                                 _ptr(ws), n, _stream(stream)))
    return L1, L2, sigma


def lowrank_residual(W: torch.Tensor, L1: torch.Tensor, L2: torch.Tensor, stream=None) -> torch.Tensor:
    """R = fp32(W - (L1 L2)^T), the part left for quantization."""
    N, K = W.shape
    r = L1.shape[1]
    R = torch.empty_like(W)
    _check(lib.wlq_lowrank_residual(_ptr(W), _ptr(L1), _ptr(L2), N, K, r, _ptr(R), _stream(stream)))
    return R


def nvfp4_scales_bytes(rows: int, K: int) -> int:
    return int(lib.wlq_nvfp4_scales_bytes(rows, K))


def nvfp4_quantize(X: torch.Tensor, stream=None):
    """NVFP4 quantization of fp32 or bf16 X [rows, K] -> (codes uint8 [rows, K/2]
    (two E2M1 codes a byte, low nibble first), scales uint8 (E4M3, the MMA's
    512-byte atom layout), gscale fp32 [2] = (tensor scale, amax))."""
    assert X.is_cuda and X.is_contiguous()
    rows, K = X.shape
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=X.device)
    scales = torch.empty(max(nvfp4_scales_bytes(rows, K), 16), dtype=torch.uint8, device=X.device)
    gscale = torch.empty(2, dtype=torch.float32, device=X.device)
    _check(lib.wlq_nvfp4_quantize(_ptr(X), _in_dtype(X), rows, K, _ptr(codes), _ptr(scales), _ptr(gscale),
                                  _stream(stream)))
    return codes, scales, gscale


def nvfp4_linear_into(y, xq, xs, xg, wq, ws, wg, N, K, x=None, bias=None, L1=None, L2=None, workspace=None,
                      stream=None):
    """y = deq(xq) deq(wq)^T [+ (x L1) L2] [+ b] (NVFP4 operands from nvfp4_quantize)."""
    M = xq.shape[0]
    r = 0 if L1 is None else L1.shape[1]
    out = OUT_F32 if y.dtype == torch.float32 else OUT_BF16
    if workspace is None:
        n = int(lib.wlq_nvfp4_linear_workspace(M, N, K, r))
        workspace = torch.empty(n, dtype=torch.uint8, device=y.device) if n else None
    ws_n = 0 if workspace is None else workspace.numel()
    _check(lib.wlq_nvfp4_linear(_ptr(xq), _ptr(xs), _ptr(xg), _ptr(x), M, _ptr(wq), _ptr(ws), _ptr(wg), N, K,
                                _ptr(bias), _ptr(L1), _ptr(L2), r, _ptr(y), out, _ptr(workspace), ws_n,
                                _stream(stream)))
    return y


def w4a4_workspace(M: int, N: int, K: int, r: int = 0, device="cuda"):
    n = int(lib.wlq_w4a4_workspace(M, N, K, r))
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def w4a4_linear_into(y, x, wq, ws, wg, N, K, bias=None, L1=None, L2=None, workspace=None, stream=None):
    """The W4A4 forward from bf16 x [M, K]: x quantized to NVFP4 in the
    workspace, then y = deq(xq) deq(wq)^T [+ (x L1) L2] [+ b]."""
    M = x.shape[0]
    r = 0 if L1 is None else L1.shape[1]
    out = OUT_F32 if y.dtype == torch.float32 else OUT_BF16
    if workspace is None:
        workspace = w4a4_workspace(M, N, K, r, device=x.device)
    ws_n = 0 if workspace is None else workspace.numel()
    _check(lib.wlq_w4a4_linear(_ptr(x), M, _ptr(wq), _ptr(ws), _ptr(wg), N, K, _ptr(bias), _ptr(L1), _ptr(L2), r,
                               _ptr(y), out, _ptr(workspace), ws_n, _stream(stream)))
    return y


# ------------------------------------------------- the attention layer's steps
class Kv4Cache(tuple):
    """A paged 4-bit KV cache: the tensors (k_codes, k_scales, v_codes, v_scales),
    codes uint8 [pages, heads, page_size, head_dim / 2], scales fp16 [pages,
    heads, page_size, head_dim / group].  Any 4-tuple of such tensors serves."""

    def __new__(cls, num_pages: int, heads: int, page_size: int, head_dim: int, group: int, device="cuda"):
        shapes = ((head_dim // 2, torch.uint8), (head_dim // group, torch.float16)) * 2
        return super().__new__(cls, (torch.zeros((num_pages, heads, page_size, n), dtype=t, device=device)
                                     for n, t in shapes))

    def __reduce__(self):  # copies and saved caches are plain tuples
        return tuple, (tuple(self),)


def _want(ok: bool, what: str):
    if not ok:
        raise WlqError(ERR_INVALID_ARG, what)


def _on(*tensors):
    """Every tensor on the current CUDA device, where the launch goes."""
    cur = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != cur:  # -1 on the host
            raise WlqError(ERR_INVALID_ARG, "tensors must be on the current CUDA device (cuda:%d)" % cur)


def _ws_bytes(workspace) -> int:
    if workspace is None:
        return 0
    _want(workspace.is_contiguous(), "workspace must be contiguous")
    return workspace.numel() * workspace.element_size()


def _head_rows(name: str, x, head_dim: int):
    """(pointer, token stride, heads) of bf16 x [tokens, heads, head_dim], heads contiguous within a token."""
    if x.dim() != 3:
        raise WlqError(ERR_INVALID_ARG, name + " must be [tokens, heads, head_dim]")
    T, H, D = x.shape
    st, sh, sd = x.stride()
    if x.dtype is not torch.bfloat16:
        raise WlqError(ERR_INVALID_ARG, name + " must be bf16")
    if D != head_dim or sd != 1 or (sh != D and H > 1):
        raise WlqError(ERR_INVALID_ARG, name + ": a token's heads must be contiguous")
    return x.data_ptr(), st if T > 1 else H * D, H


def _weight(name: str, w, head_dim: int):
    if w is None:
        return None
    if w.dtype is not torch.bfloat16 or w.numel() != head_dim or not w.is_contiguous():
        raise WlqError(ERR_INVALID_ARG, name + " must be contiguous bf16 [head_dim]")
    return w.data_ptr()


_SECTIONS = {}


def _rope(positions, inv_freq, sections, tokens: int):
    """(positions, axes, inv_freq, rotary_dim, sections) for the C call."""
    if positions is None:
        return None, 0, None, 0, None
    if inv_freq is None or inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise WlqError(ERR_INVALID_ARG, "positions need inv_freq, contiguous fp32 [pairs]")
    shape = positions.shape
    axes = shape[1] if len(shape) == 2 else 1
    if positions.dtype is not torch.int32 or not positions.is_contiguous() or len(shape) > 2 or shape[0] != tokens:
        raise WlqError(ERR_INVALID_ARG, "positions must be contiguous int32 [tokens] or [tokens, axes]")
    pairs = inv_freq.shape[0]
    sections = (pairs,) if sections is None else tuple(sections)
    if len(sections) != axes:
        raise WlqError(ERR_INVALID_ARG, "one section for each axis")
    arr = _SECTIONS.get(sections)
    if arr is None:
        arr = _SECTIONS[sections] = (ctypes.c_int32 * axes)(*sections)
    return positions.data_ptr(), axes, inv_freq.data_ptr(), 2 * pairs, arr


def qk_norm_rope(q, k, positions=None, inv_freq=None, sections=None, interleaved: bool = True, q_weight=None,
                 k_weight=None, eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """Norm of each head's queries and keys (RMS, times the weight; none without a
    weight) and rotation by the positions, one pass -> (q_out, k_out), bf16.

    q [tokens, q_heads, head_dim] and k [tokens, k_heads, head_dim]: bf16,
    token stride free (views of a fused projection); either may be None.
    positions int32 [tokens] or [tokens, axes], inv_freq fp32 [rotary_dim / 2],
    sections: the pairs that turn by each axis.  interleaved: pairs (2 i,
    2 i + 1), else (i, i + rotary_dim / 2).  q_out / k_out may be q / k."""
    if stream is not None:  # what is allocated here belongs to that stream, too
        with torch.cuda.stream(stream):
            return qk_norm_rope(q, k, positions, inv_freq, sections, interleaved, q_weight, k_weight, eps, q_out, k_out)
    some = q if q is not None else k
    _want(some is not None, "q or k is needed")
    _want(some.dim() == 3, "q and k must be [tokens, heads, head_dim]")
    T, _, D = some.shape
    _on(q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out)
    qp = kp = qo = ko = None
    qs = ks = qos = kos = hq = hk = 0
    if q is not None:
        qp, qs, hq = _head_rows("q", q, D)
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
            qo, qos = q_out.data_ptr(), hq * D
        else:
            _want(q_out.shape == q.shape, "q_out must have q's shape")
            qo, qos, _ = _head_rows("q_out", q_out, D)
    if k is not None:
        _want(k.shape[0] == T, "q and k need the same tokens")
        kp, ks, hk = _head_rows("k", k, D)
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
            ko, kos = k_out.data_ptr(), hk * D
        else:
            _want(k_out.shape == k.shape, "k_out must have k's shape")
            ko, kos, _ = _head_rows("k_out", k_out, D)
    _check(lib.wlq_qk_norm_rope(qp, qs, hq, kp, ks, hk, T, D, _weight("q_weight", q_weight, D),
                                _weight("k_weight", k_weight, D), eps, *_rope(positions, inv_freq, sections, T),
                                int(interleaved), qo, qos, ko, kos, _stream()))
    return q_out, k_out


def _pool(cache):
    """(pointers..., num_pages, page_size, group), heads, head_dim of a 4-bit cache."""
    kc, ks, vc, vs = cache
    shape, scales = kc.shape, ks.shape
    if len(shape) != 4 or len(scales) != 4:
        raise WlqError(ERR_INVALID_ARG, "cache: four arrays of four dimensions")
    pages, H, P, half = shape
    groups = scales[3]
    if (kc.dtype is not torch.uint8 or vc.dtype is not torch.uint8 or ks.dtype is not torch.float16 or vs.dtype is not torch.float16
            or vc.shape != shape or vs.shape != scales or scales != (pages, H, P, groups) or groups == 0):
        raise WlqError(ERR_INVALID_ARG, "cache: uint8 codes [pages, heads, page_size, head_dim / 2] and fp16 scales "
                                        "[pages, heads, page_size, head_dim / group], the same for keys and values")
    if not (kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()):
        raise WlqError(ERR_INVALID_ARG, "cache: contiguous arrays")
    return (kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), pages, P, 2 * half // groups), H, 2 * half


def _batch(cu_seqlens, kv_lens, block_table, max_q: int):
    if block_table.dim() != 2:
        raise WlqError(ERR_INVALID_ARG, "block_table must be [batch, width]")
    n, width = block_table.shape
    i32 = torch.int32
    if (cu_seqlens.dtype is not i32 or kv_lens.dtype is not i32 or block_table.dtype is not i32 or cu_seqlens.numel() != n + 1
            or kv_lens.numel() != n or not (cu_seqlens.is_contiguous() and kv_lens.is_contiguous() and block_table.is_contiguous())):
        raise WlqError(ERR_INVALID_ARG, "contiguous int32 cu_seqlens [batch + 1], kv_lens [batch], block_table [batch, width]")
    if max_q >> 31:  # ctypes would pass its lower 32 bits
        raise WlqError(ERR_INVALID_ARG, "max_q must be 0 .. 2^31 - 1")
    return cu_seqlens.data_ptr(), kv_lens.data_ptr(), n, max_q, block_table.data_ptr(), width


def kv4_append(cache, k, v, cu_seqlens, kv_lens, block_table, max_q: int, positions=None, inv_freq=None, sections=None,
               interleaved: bool = True, k_weight=None, eps: float = 1e-6, stream=None):
    """Keys (normed and rotated by qk_norm_rope's formula) and values rounded to 4
    bits into the paged cache.  k, v: bf16 [tokens, heads, head_dim], token stride
    free.  Sequence b's tokens cu_seqlens[b] .. cu_seqlens[b + 1] become the
    last of its kv_lens[b] cached ones, on pages block_table[b]; max_q: an upper
    bound of the sequences' token counts."""
    if stream is not None:  # what is allocated here belongs to that stream, too
        with torch.cuda.stream(stream):
            return kv4_append(cache, k, v, cu_seqlens, kv_lens, block_table, max_q, positions, inv_freq, sections, interleaved, k_weight, eps)
    ptrs, H, D = _pool(cache)
    T = k.shape[0]
    _on(k, v, *cache, cu_seqlens, kv_lens, block_table, positions, inv_freq, k_weight)
    kp, kst, hk = _head_rows("k", k, D)
    vp, vst, hv = _head_rows("v", v, D)
    if hk != H or hv != H or v.shape[0] != T:
        raise WlqError(ERR_INVALID_ARG, "k and v must be [tokens, the cache's heads, head_dim]")
    _check(lib.wlq_kv4_append(kp, kst, vp, vst, T, H, D, _weight("k_weight", k_weight, D), eps,
                              *_rope(positions, inv_freq, sections, T), int(interleaved),
                              *_batch(cu_seqlens, kv_lens, block_table, max_q), *ptrs, _stream()))


def kv4_read(cache, cu_seqlens, kv_lens, block_table, max_q: int, tokens: int, stream=None):
    """The cached rows of the call's tokens as bf16 -> (k, v) [tokens, heads,
    head_dim] (rows of no sequence stay uninitialised)."""
    if stream is not None:  # what is allocated here belongs to that stream, too
        with torch.cuda.stream(stream):
            return kv4_read(cache, cu_seqlens, kv_lens, block_table, max_q, tokens)
    ptrs, H, D = _pool(cache)
    _on(*cache, cu_seqlens, kv_lens, block_table)
    k = torch.empty((tokens, H, D), dtype=torch.bfloat16, device=cache[0].device)
    v = torch.empty_like(k)
    _check(lib.wlq_kv4_read(*_batch(cu_seqlens, kv_lens, block_table, max_q), *ptrs, tokens, H, D, k.data_ptr(),
                            v.data_ptr(), _stream()))
    return k, v


def kv4_attention_workspace(tokens: int, batch: int, max_q: int, max_kv: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    """Workspace bytes of kv4_attention (0: none needed)."""
    return int(lib.wlq_kv4_attention_workspace(tokens, batch, max_q, max_kv, q_heads, kv_heads, head_dim))


def kv4_attention(q, cache, cu_seqlens, kv_lens, block_table, max_q: int, max_kv: int, scale=None, causal: bool = True,
                  window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Attention of bf16 q [tokens, q_heads, head_dim] (token stride free) over the
    paged 4-bit cache -> out, bf16 [tokens, q_heads, head_dim].

    Sequence b's queries cu_seqlens[b] .. cu_seqlens[b + 1] are the last of its
    kv_lens[b] cached tokens; causal queries see up to themselves, with a
    window only the last `window` of those.  A query that sees nothing gets 0.
    max_q, max_kv: upper bounds of the lengths.  scale: 1 / sqrt(head_dim) by
    default.  lse: fp32 [tokens, q_heads] to be filled, or None.  Rows of no
    sequence are left as they were (uninitialised without out).  workspace: of
    kv4_attention_workspace bytes; allocated here if None."""
    if stream is not None:  # what is allocated here belongs to that stream, too
        with torch.cuda.stream(stream):
            return kv4_attention(q, cache, cu_seqlens, kv_lens, block_table, max_q, max_kv, scale, causal, window, out, lse, workspace)
    ptrs, H, D = _pool(cache)
    _want(q.dim() == 3 and q.shape[2] == D, "q must be [tokens, q_heads, the cache's head_dim]")
    T, Hq, _ = q.shape
    _on(q, *cache, cu_seqlens, kv_lens, block_table, out, lse, workspace)
    qp, qs, _ = _head_rows("q", q, D)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _want(out.shape == q.shape and out.dtype is torch.bfloat16 and out.is_contiguous(), "out must be contiguous bf16 of q's shape")
    _want(lse is None or (lse.shape == (T, Hq) and lse.dtype is torch.float32 and lse.is_contiguous()),
          "lse must be contiguous fp32 [tokens, q_heads]")
    batch = _batch(cu_seqlens, kv_lens, block_table, max_q)
    if window >> 31:
        raise WlqError(ERR_INVALID_ARG, "window must be 0 .. 2^31 - 1")
    if workspace is None:
        n = int(lib.wlq_kv4_attention_workspace(T, batch[2], batch[3], max_kv, Hq, H, D))
        workspace = out.new_empty((n + 1) // 2) if n else None  # bf16: two bytes each
    ws_n = _ws_bytes(workspace)
    _check(lib.wlq_kv4_attention(qp, qs, T, Hq, H, D, batch[0], batch[1], batch[2], batch[3], max_kv, batch[4], batch[5], *ptrs,
                                 D ** -0.5 if scale is None else scale, int(causal), window, out.data_ptr(),
                                 None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(), ws_n,
                                 _stream()))
    return out


def _int8_operands(y, wq, ws, bias, M: int, K: int):
    N, Kw = wq.shape
    if wq.dtype is not torch.int8 or Kw != K or not wq.is_contiguous():
        raise WlqError(ERR_INVALID_ARG, "wq must be contiguous int8 [N, K]")
    if ws.dtype is not torch.float32 or ws.numel() != N or not ws.is_contiguous():
        raise WlqError(ERR_INVALID_ARG, "ws must be contiguous fp32 [N]")
    if bias is not None and (bias.dtype is not torch.bfloat16 or bias.numel() != N or not bias.is_contiguous()):
        raise WlqError(ERR_INVALID_ARG, "bias must be contiguous bf16 [N]")
    dt = y.dtype
    if (dt is not torch.bfloat16 and dt is not torch.float32) or y.shape != (M, N) or not y.is_contiguous():
        raise WlqError(ERR_INVALID_ARG, "y must be contiguous bf16 or fp32 [M, N]")
    return N, OUT_F32 if dt is torch.float32 else OUT_BF16


def int8_linear_into(y, xq, xs, wq, ws, bias=None, stream=None):
    """y = xs ws (xq wq^T) + b from int8 codes xq [M, K], wq [N, K] and fp32 scales of
    each token and output channel (quantize_ex(x, 8, 0), quantize(W, 8, 0)); y bf16 or fp32."""
    if stream is not None:  # what is allocated here belongs to that stream, too
        with torch.cuda.stream(stream):
            return int8_linear_into(y, xq, xs, wq, ws, bias)
    _want(xq.dim() == 2 and wq.dim() == 2, "xq and wq must be [M, K] and [N, K]")
    M, K = xq.shape
    _on(y, xq, xs, wq, ws, bias)
    _want(xq.dtype == torch.int8 and xq.is_contiguous(), "xq must be contiguous int8 [M, K]")
    _want(xs.dtype == torch.float32 and xs.numel() == M and xs.is_contiguous(), "xs must be contiguous fp32 [M]")
    N, out = _int8_operands(y, wq, ws, bias, M, K)
    _check(lib.wlq_int8_linear(xq.data_ptr(), xs.data_ptr(), M, wq.data_ptr(), ws.data_ptr(), N, K,
                               None if bias is None else bias.data_ptr(), y.data_ptr(), out, _stream()))
    return y


def w8a8_workspace(M: int, K: int) -> int:
    """Workspace bytes of w8a8_linear."""
    return int(lib.wlq_w8a8_workspace(M, K))


def w8a8_linear_into(y, x, wq, ws, bias=None, workspace=None, stream=None):
    """The W8A8 forward from bf16 x [M, K]: x quantized token by token in the
    workspace, then y = xs ws (xq wq^T) + b (int8 wq [N, K], fp32 ws [N])."""
    if stream is not None:  # what is allocated here belongs to that stream, too
        with torch.cuda.stream(stream):
            return w8a8_linear_into(y, x, wq, ws, bias, workspace)
    _want(x.dim() == 2 and wq.dim() == 2, "x and wq must be [M, K] and [N, K]")
    M, K = x.shape
    _on(y, x, wq, ws, bias, workspace)
    _want(x.dtype == torch.bfloat16 and x.is_contiguous(), "x must be contiguous bf16 [M, K]")
    N, out = _int8_operands(y, wq, ws, bias, M, K)
    if workspace is None:
        n = int(lib.wlq_w8a8_workspace(M, K))
        workspace = x.new_empty((n + 1) // 2) if n else None  # bf16: two bytes each
    ws_n = _ws_bytes(workspace)
    _check(lib.wlq_w8a8_linear(x.data_ptr(), M, wq.data_ptr(), ws.data_ptr(), N, K, None if bias is None else bias.data_ptr(),
                               y.data_ptr(), out, None if workspace is None else workspace.data_ptr(), ws_n, _stream()))
    return y


def w8a8_linear(x, wq, ws, bias=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """w8a8_linear_into with a new y [M, N]."""
    if stream is not None:  # what is allocated here belongs to that stream, too
        with torch.cuda.stream(stream):
            return w8a8_linear(x, wq, ws, bias, out_dtype, workspace)
    y = torch.empty((x.shape[0], wq.shape[0]), dtype=out_dtype, device=x.device)
    return w8a8_linear_into(y, x, wq, ws, bias, workspace)


def get_status(stream=None) -> int:
    """Synchronise and return (and clear) the device error status as a code."""
    return int(lib.wlq_get_status(_stream(stream)))


def check_status(stream=None):
    _check(get_status(stream))


def probe_wait_timeout(timeout_ns: int, stream=None):
    _check(lib.wlq_probe_wait_timeout(timeout_ns, _stream(stream)))


def set_grid_limit(max_ctas: int):
    """Cap the CTAs of every later wlq_linear launch (0: no cap)."""
    lib.wlq_set_grid_limit(int(max_ctas))


def version() -> str:
    return lib.wlq_version().decode()
