"""Python binding of libfp8q.so -- W8A8 block-scaled FP8 projection on MI355X.

Argument marshalling only: every function takes torch tensors that already
live on the current GPU, passes their device pointers and the current torch
stream to the C ABI (include/fp8q.h) and raises on a non-OK status.  Every
step of the computation runs in the library's HIP kernels; there is no CPU
or PyTorch fallback: the first call raises if the library has not been built
(``python -m w8a8_fp8_block_amd.build``).

Names match the C entry points:

  fp8q_quant_act(x, q, scale_rm, variant=0)
  fp8q_quant_act_kmajor(x, q, scale_rm, scale_km, variant=0)
  fp8q_scale_to_kmajor(scale_rm, scale_km)
  fp8q_gemm_blockscaled(a, a_scale_km, w, w_scale, out, kernel=0)
  fp8q_proj(x, w, w_scale, out, act_q, act_scale, act_scale_km)
  fp8q_silu_mul_quant(gate, up, h, h_scale_km)
  fp8q_ffn_gate_up(x_q, x_scale_km, w_gate, w_gate_scale, w_up, w_up_scale, h, h_scale_km)
  fp8q_ffn(x, w_gate, w_gate_scale, w_up, w_up_scale, w_down, w_down_scale, out,
           workspace, variant=0)
  fp8q_moe_route(logits, ids, weights, order, pos, offsets, workspace, renormalize=True)
  fp8q_group_rows(ids, order, pos, offsets, workspace)
  fp8q_gemm_grouped(a, a_scale_km, w, w_scale, offsets, out, order=None, top_k=1, kernel=0)
  fp8q_moe_ffn(x, weights, order, pos, offsets, w_gate, w_gate_scale, w_up, w_up_scale,
               w_down, w_down_scale, out, workspace, variant=0)
  fp8q_moe_combine(y, weights, pos, offsets, out)
  fp8q_proj_lora(x, w, w_scale, lora_a, lora_b, lora_scale, adapter_ids, out, act_q, act_scale,
                 act_scale_km, workspace)
  fp8q_add_rmsnorm_quant(x, residual, weight, h, y, q, scale_rm, scale_km, rstd, eps=1e-6)
  fp8q_add_rmsnorm_grad(dy, dh, h, weight, rstd, dx, dweight, workspace)
  fp8q_quant_act_dual(x, q, scale_km, q_tok, exp_tok)
  fp8q_gemm_dgrad(dy, dy_scale_km, w, w_scale, dx, workspace)
  fp8q_gemm_wgrad(dy_tok, dy_exp, x_tok, x_exp, dw, workspace)
  fp8q_moe_balance(logits, ids, counts, prob, loss, workspace, coef=1.0)
  fp8q_moe_route_grad(logits, ids, dweights, counts, dloss, dlogits, renormalize=True, coef=1.0)
  fp8q_m_pad(m), fp8q_quant_select(M, K, cu_count), ...

Dtypes: bf16 tensors may be torch.bfloat16 or torch.uint16/int16 views;
e4m3 codes may be torch.uint8 or torch.float8_e4m3fn; scales float32.
"""
from __future__ import annotations

import ctypes
import os

# torch first: its libtorch_hip.so asks for "libamdhip64.so" while this
# library asks for "libamdhip64.so.7"; loading torch's runtime first lets the
# dynamic linker satisfy ours with the same object (matching soname), so one
# HIP runtime serves both.  The other order would load a second runtime.
import torch  # (device memory and streams)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8q.so")

_P = ctypes.c_void_p
_U = ctypes.c_uint32
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_F = ctypes.c_float


class SelectParams(ctypes.Structure):
    _fields_ = [("cu_count", ctypes.c_uint32), ("min_wg_per_cu", ctypes.c_uint32),
                ("b_groups_per_wg", ctypes.c_uint32), ("a_groups_per_wg", ctypes.c_uint32),
                ("requested", ctypes.c_int), ("b_present", ctypes.c_int),
                ("a_present", ctypes.c_int)]


_SIGS = {
    "fp8q_m_pad": (_U, [_U]),
    "fp8q_last_error": (ctypes.c_char_p, []),
    "fp8q_version": (ctypes.c_char_p, []),
    "fp8q_quant_act": (_I, [_P, _P, _P, _U, _U, _P]),
    "fp8q_quant_act_ex": (_I, [_P, _P, _P, _U, _U, _I, _P]),
    "fp8q_quant_act_kmajor": (_I, [_P, _P, _P, _P, _U, _U, _P]),
    "fp8q_quant_act_kmajor_ex": (_I, [_P, _P, _P, _P, _U, _U, _I, _P]),
    "fp8q_default_select_params": (SelectParams, [_U]),
    "fp8q_quant_select_with": (_I, [_U, _U, ctypes.POINTER(SelectParams),
                                    ctypes.POINTER(_U * 3), ctypes.POINTER(ctypes.c_char_p)]),
    "fp8q_quant_select": (_I, [_U, _U, _U, ctypes.POINTER(_U * 3),
                               ctypes.POINTER(ctypes.c_char_p)]),
    "fp8q_quant_b_min_m": (_U, [_U, ctypes.POINTER(SelectParams)]),
    "fp8q_quant_log_slot": (_I, [_I, ctypes.c_char_p, _I]),
    "fp8q_scale_to_kmajor": (_I, [_P, _P, _U, _U, _P]),
    "fp8q_gemm_select": (_I, [_U, _U, _U]),
    "fp8q_gemm_select_cus": (_I, [_U, _U, _U, _U]),
    "fp8q_proj_quant_fused": (_I, [_U, _U]),
    "fp8q_gemm_blockscaled": (_I, [_P, _P, _P, _P, _P, _U, _U, _U, _P]),
    "fp8q_gemm_blockscaled_ex": (_I, [_P, _P, _P, _P, _P, _U, _U, _U, _I, _P]),
    "fp8q_gemm_blockscaled_splitk": (_I, [_P, _P, _P, _P, _P, _P, _SZ, _U, _U, _U, _U, _P]),
    "fp8q_gemm_splitk_select": (_U, [_U, _U, _U]),
    "fp8q_gemm_splitk_select_cus": (_U, [_U, _U, _U, _U]),
    "fp8q_gemm_streamk_select": (_I, [_U, _U, _U]),
    "fp8q_gemm_streamk_select_cus": (_I, [_U, _U, _U, _U]),
    "fp8q_gemm_splitk_workspace_bytes": (_SZ, [_U, _U, _U, _U]),
    "fp8q_gemm_blockscaled_streamk": (_I, [_P, _P, _P, _P, _P, _P, _SZ, _U, _U, _U, _U, _P]),
    "fp8q_gemm_kernel_name": (ctypes.c_char_p, [_U, _U, _U, _I]),
    "fp8q_gemm_streamk_workspace_bytes": (_SZ, [_U]),
    "fp8q_gemm_blockscaled_splitk_noalloc": (_I, [_P, _P, _P, _P, _P, _U, _U, _U, _U, _P]),
    "fp8q_clock_stamp": (_I, [_P, _U, _P]),
    "fp8q_proj": (_I, [_P, _P, _P, _P, _P, _P, _P, _U, _U, _U, _P]),
    "fp8q_proj_splitk": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _SZ, _U, _U, _U, _P]),
    "fp8q_gemm_rowscaled": (_I, [_P, _P, _P, _P, _P, _U, _U, _U, _P]),
    "fp8q_gemm_rowscaled_ex": (_I, [_P, _P, _P, _P, _P, _U, _U, _U, _I, _P]),
    "fp8q_proj_rowscaled": (_I, [_P, _P, _P, _P, _P, _P, _P, _U, _U, _U, _P]),
    "fp8q_dequant_fp8_bf16": (_I, [_P, _P, _P, _U, _U, _I, _P]),
    "fp8q_gemm_bf16": (_I, [_P, _P, _P, _U, _U, _U, _P]),
    "fp8q_silu_mul_quant": (_I, [_P, _P, _P, _P, _U, _U, _P]),
    "fp8q_ffn_gate_up": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _U, _U, _U, _P]),
    "fp8q_ffn_select": (_I, [_U, _U, _U]),
    "fp8q_ffn_workspace_bytes": (ctypes.c_size_t, [_U, _U, _U, _I]),
    "fp8q_ffn": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _U, _U, _U, _I, _P]),
    "fp8q_moe_route": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _SZ, _U, _U, _U, _I, _P]),
    "fp8q_moe_route_workspace_bytes": (_SZ, [_U, _U, _U]),
    "fp8q_group_rows": (_I, [_P, _P, _P, _P, _P, _SZ, _U, _U, _P]),
    "fp8q_group_rows_workspace_bytes": (_SZ, [_U, _U]),
    "fp8q_moe_combine": (_I, [_P, _P, _P, _P, _P, _U, _U, _U, _U, _P]),
    "fp8q_gemm_grouped": (_I, [_P, _P, _P, _P, _P, _P, _P, _U, _U, _U, _U, _U, _U, _I, _P]),
    "fp8q_gemm_grouped_select": (_I, [_U, _U, _U]),
    "fp8q_moe_ffn": (_I, [_P] * 13 + [_SZ, _U, _U, _U, _U, _U, _I, _P]),
    "fp8q_moe_ffn_select": (_I, [_U, _U, _U, _U]),
    "fp8q_proj_lora": (_I, [_P] * 12 + [_SZ, _U, _U, _U, _U, _U, _P]),
    "fp8q_proj_lora_workspace_bytes": (_SZ, [_U, _U, _U, _U]),
    "fp8q_moe_ffn_workspace_bytes": (_SZ, [_U, _U, _U, _U, _U, _I]),
    "fp8q_add_rmsnorm_quant": (_I, [_P] * 9 + [_F, _U, _U, _P]),
    "fp8q_add_rmsnorm_grad": (_I, [_P] * 8 + [_SZ, _U, _U, _P]),
    "fp8q_add_rmsnorm_grad_workspace_bytes": (_SZ, [_U, _U]),
    "fp8q_quant_act_dual": (_I, [_P] * 5 + [_U, _U, _P]),
    "fp8q_gemm_dgrad": (_I, [_P] * 6 + [_SZ, _U, _U, _U, _P]),
    "fp8q_gemm_dgrad_workspace_bytes": (_SZ, [_U, _U, _U]),
    "fp8q_gemm_wgrad": (_I, [_P] * 6 + [_SZ, _U, _U, _U, _P]),
    "fp8q_gemm_wgrad_workspace_bytes": (_SZ, [_U, _U, _U]),
    "fp8q_moe_balance": (_I, [_P, _I] + [_P] * 5 + [_SZ, _F, _U, _U, _U, _P]),
    "fp8q_moe_balance_workspace_bytes": (_SZ, [_U, _U]),
    "fp8q_moe_route_grad": (_I, [_P, _I] + [_P] * 5 + [_F, _U, _U, _U, _I, _P]),
}

_lib = None


def lib():
    """The ctypes handle of libfp8q.so (raw C ABI), loaded on first use.
    Raises if the library has not been built: there is no fallback path."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python -m w8a8_fp8_block_amd.build` "
                "(the projection has no fallback path)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


STATUS = {0: "FP8Q_OK", 1: "FP8Q_ERR_NULL", 2: "FP8Q_ERR_SHAPE", 3: "FP8Q_ERR_ALIGN",
          4: "FP8Q_ERR_DEVICE", 5: "FP8Q_ERR_LAUNCH", 6: "FP8Q_ERR_VARIANT"}


class Fp8qError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


def _check(st: int):
    if st != 0:
        raise Fp8qError(st, lib().fp8q_last_error().decode())


def _ptr(t) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _optr(t) -> int:
    return 0 if t is None else _ptr(t)


_raw_stream = None


def _stream(stream=None) -> int:
    """The HIP stream handle to launch on: `stream`'s, else torch's current
    stream on the current device (read through torch's raw-handle query
    where the build has it: ~0.4 us against ~2.7 us for building a Stream
    object, per call, on the host)."""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        q = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        dev = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        torch.cuda.current_device()  # initialises torch's device state
        _raw_stream = ((lambda: q(dev())) if q is not None
                       else (lambda: torch.cuda.current_stream().cuda_stream))
    return _raw_stream()


def _dims(t, nd):
    shape = t.shape
    if len(shape) != nd:
        raise ValueError(f"expected a {nd}-d tensor, got shape {tuple(shape)}")
    return shape


# ------------------------------------------------------------------ API
def fp8q_m_pad(m: int) -> int:
    return int(lib().fp8q_m_pad(m))


def fp8q_version() -> str:
    return lib().fp8q_version().decode()


def fp8q_quant_act(x, q, scale_rm, variant: int = 0, stream=None):
    M, K = _dims(x, 2)
    _check(lib().fp8q_quant_act_ex(_ptr(x), _ptr(q), _ptr(scale_rm), M, K, variant,
                                  _stream(stream)))


def fp8q_quant_act_kmajor(x, q, scale_rm, scale_km, variant: int = 0, stream=None):
    M, K = _dims(x, 2)
    _check(lib().fp8q_quant_act_kmajor_ex(_ptr(x), _ptr(q), _optr(scale_rm), _ptr(scale_km), M,
                                         K, variant, _stream(stream)))


def fp8q_scale_to_kmajor(scale_rm, scale_km, stream=None):
    M, G = _dims(scale_rm, 2)
    _check(lib().fp8q_scale_to_kmajor(_ptr(scale_rm), _ptr(scale_km), M, G * 128,
                                     _stream(stream)))


def fp8q_gemm_blockscaled(a, a_scale_km, w, w_scale, out, kernel: int = 0, stream=None):
    M, K = _dims(a, 2)
    N, K2 = _dims(w, 2)
    if K2 != K:
        raise ValueError("a and w disagree on K")
    _check(lib().fp8q_gemm_blockscaled_ex(_ptr(a), _ptr(a_scale_km), _ptr(w), _ptr(w_scale),
                                         _ptr(out), M, N, K, kernel, _stream(stream)))


def fp8q_gemm_splitk_select(M: int, N: int, K: int, cu_count: int = None) -> int:
    """Split count fp8q_gemm_blockscaled_splitk takes with splits=0 (1 = no split)
    on the current device, or on a device with cu_count compute units."""
    if cu_count is not None:
        return int(lib().fp8q_gemm_splitk_select_cus(M, N, K, cu_count))
    return int(lib().fp8q_gemm_splitk_select(M, N, K))


def fp8q_gemm_streamk_select(M: int, N: int, K: int, cu_count: int = None) -> int:
    """1 if fp8q_gemm_blockscaled_splitk with splits=0 runs the stream-K form
    (on the current device, or one with cu_count compute units)."""
    if cu_count is not None:
        return int(lib().fp8q_gemm_streamk_select_cus(M, N, K, cu_count))
    return int(lib().fp8q_gemm_streamk_select(M, N, K))


def fp8q_gemm_splitk_workspace_bytes(M: int, N: int, K: int, splits: int = 0) -> int:
    return int(lib().fp8q_gemm_splitk_workspace_bytes(M, N, K, splits))


def fp8q_gemm_blockscaled_splitk(a, a_scale_km, w, w_scale, out, workspace, splits: int = 0,
                                 stream=None):
    """fp8q_gemm_blockscaled with the K blocks split over `splits` workgroups
    per tile (0 = automatic); workspace: a device tensor of at least
    fp8q_gemm_splitk_workspace_bytes(M, N, K, splits) bytes, or None when that is 0."""
    M, K = _dims(a, 2)
    N, K2 = _dims(w, 2)
    if K2 != K:
        raise ValueError("a and w disagree on K")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fp8q_gemm_blockscaled_splitk(_ptr(a), _ptr(a_scale_km), _ptr(w), _ptr(w_scale),
                                             _ptr(out), _optr(workspace), nbytes, M, N, K,
                                             splits, _stream(stream)))


def fp8q_gemm_streamk_workspace_bytes(workgroups: int = 0) -> int:
    return int(lib().fp8q_gemm_streamk_workspace_bytes(workgroups))


def fp8q_gemm_blockscaled_streamk(a, a_scale_km, w, w_scale, out, workspace, workgroups: int = 0,
                                  stream=None):
    """fp8q_gemm_blockscaled in its stream-K form on `workgroups` persistent
    workgroups (0 = the device's CU count); workspace: a device tensor of at
    least fp8q_gemm_streamk_workspace_bytes(workgroups) bytes."""
    M, K = _dims(a, 2)
    N, K2 = _dims(w, 2)
    if K2 != K:
        raise ValueError("a and w disagree on K")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fp8q_gemm_blockscaled_streamk(_ptr(a), _ptr(a_scale_km), _ptr(w), _ptr(w_scale),
                                              _ptr(out), _optr(workspace), nbytes, M, N, K,
                                              workgroups, _stream(stream)))


NOALLOC_SCRATCH_BYTES = 32 << 20  # FP8Q_NOALLOC_SCRATCH_BYTES


def fp8q_gemm_blockscaled_splitk_noalloc(a, a_scale_km, w, w_scale, out, splits: int = 0,
                                         stream=None):
    """fp8q_gemm_blockscaled_splitk with the partials in the library's static
    device scratch (no workspace; splits * M * N * 4 <= NOALLOC_SCRATCH_BYTES)."""
    M, K = _dims(a, 2)
    N, K2 = _dims(w, 2)
    if K2 != K:
        raise ValueError("a and w disagree on K")
    _check(lib().fp8q_gemm_blockscaled_splitk_noalloc(_ptr(a), _ptr(a_scale_km), _ptr(w),
                                                     _ptr(w_scale), _ptr(out), M, N, K, splits,
                                                     _stream(stream)))


def fp8q_proj(x, w, w_scale, out, act_q, act_scale, act_scale_km, stream=None):
    M, K = _dims(x, 2)
    N, K2 = _dims(w, 2)
    if K2 != K:
        raise ValueError("x and w disagree on K")
    _check(lib().fp8q_proj(_ptr(x), _ptr(w), _ptr(w_scale), _ptr(out), _ptr(act_q),
                          _ptr(act_scale), _ptr(act_scale_km), M, N, K, _stream(stream)))


def fp8q_proj_splitk(x, w, w_scale, out, act_q, act_scale, act_scale_km, workspace, stream=None):
    """fp8q_proj with the GEMM split over K where fp8q_gemm_splitk_select says
    so; workspace: a device tensor of at least
    fp8q_gemm_splitk_workspace_bytes(M, N, K) bytes, or None when that is 0."""
    M, K = _dims(x, 2)
    N, K2 = _dims(w, 2)
    if K2 != K:
        raise ValueError("x and w disagree on K")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fp8q_proj_splitk(_ptr(x), _ptr(w), _ptr(w_scale), _ptr(out), _ptr(act_q),
                                 _ptr(act_scale), _ptr(act_scale_km), _optr(workspace), nbytes,
                                 M, N, K, _stream(stream)))


def fp8q_gemm_rowscaled(a, a_scale_km, w, w_scale_row, out, kernel: int = 0, stream=None):
    """As fp8q_gemm_blockscaled with one fp32 weight scale per row, w_scale_row [N]."""
    M, K = _dims(a, 2)
    N, K2 = _dims(w, 2)
    if K2 != K:
        raise ValueError("a and w disagree on K")
    _check(lib().fp8q_gemm_rowscaled_ex(_ptr(a), _ptr(a_scale_km), _ptr(w), _ptr(w_scale_row),
                                       _ptr(out), M, N, K, kernel, _stream(stream)))


def fp8q_proj_rowscaled(x, w, w_scale_row, out, act_q, act_scale, act_scale_km, stream=None):
    M, K = _dims(x, 2)
    N, K2 = _dims(w, 2)
    if K2 != K:
        raise ValueError("x and w disagree on K")
    _check(lib().fp8q_proj_rowscaled(_ptr(x), _ptr(w), _ptr(w_scale_row), _ptr(out), _ptr(act_q),
                                    _ptr(act_scale), _ptr(act_scale_km), M, N, K, _stream(stream)))


def fp8q_dequant_fp8_bf16(w, scale, dst, per_row: bool, stream=None):
    """FP8 weights [N,K] -> bf16 [N,K] (dst), block-scaled or per-row scales."""
    N, K = _dims(w, 2)
    _check(lib().fp8q_dequant_fp8_bf16(_ptr(w), _ptr(scale), _ptr(dst), N, K, 1 if per_row else 0,
                                      _stream(stream)))


def fp8q_gemm_bf16(x, w, out, stream=None):
    """bf16 comparator GEMM: out[M,N] = bf16(x[M,K] . w[N,K]^T)."""
    M, K = _dims(x, 2)
    N, K2 = _dims(w, 2)
    if K2 != K:
        raise ValueError("x and w disagree on K")
    _check(lib().fp8q_gemm_bf16(_ptr(x), _ptr(w), _ptr(out), M, N, K, _stream(stream)))


def fp8q_silu_mul_quant(gate, up, h, h_scale_km, stream=None):
    """FFN intermediate h = bf16(silu(gate) * up) of bf16 gate/up [M,I],
    quantized: codes h [M,I], K-major scales h_scale_km [I/128, ceil16(M)]."""
    M, I = _dims(gate, 2)
    if _dims(up, 2) != (M, I):
        raise ValueError("gate and up differ in shape")
    _check(lib().fp8q_silu_mul_quant(_ptr(gate), _ptr(up), _ptr(h), _ptr(h_scale_km), M, I,
                                    _stream(stream)))


def fp8q_ffn_gate_up(x_q, x_scale_km, w_gate, w_gate_scale, w_up, w_up_scale, h, h_scale_km,
                     stream=None):
    """Fused gate/up projection of quantized x [M,H] with weights [I,H] to the
    quantized intermediate h [M,I] and its K-major scales."""
    M, H = _dims(x_q, 2)
    I, H2 = _dims(w_gate, 2)
    if H2 != H or _dims(w_up, 2) != (I, H):
        raise ValueError("x, w_gate and w_up disagree in shape")
    _check(lib().fp8q_ffn_gate_up(_ptr(x_q), _ptr(x_scale_km), _ptr(w_gate), _ptr(w_gate_scale),
                                 _ptr(w_up), _ptr(w_up_scale), _ptr(h), _ptr(h_scale_km), M, H, I,
                                 _stream(stream)))


def fp8q_ffn_select(M: int, H: int, I: int) -> int:
    """Variant fp8q_ffn runs with variant=0: 1 fused gate/up, 2 separate."""
    return int(lib().fp8q_ffn_select(M, H, I))


def fp8q_ffn_workspace_bytes(M: int, H: int, I: int, variant: int = 0) -> int:
    return int(lib().fp8q_ffn_workspace_bytes(M, H, I, variant))


def fp8q_ffn(x, w_gate, w_gate_scale, w_up, w_up_scale, w_down, w_down_scale, out, workspace,
             variant: int = 0, stream=None):
    """The dense FFN: out [M,H] = down(quant(bf16(silu(gate) * up))) of x [M,H];
    workspace: a device byte tensor of fp8q_ffn_workspace_bytes(M, H, I, variant)."""
    M, H = _dims(x, 2)
    I, H2 = _dims(w_gate, 2)
    if H2 != H or _dims(w_up, 2) != (I, H) or _dims(w_down, 2) != (H, I):
        raise ValueError("x and the weights disagree in shape")
    _check(lib().fp8q_ffn(_ptr(x), _ptr(w_gate), _ptr(w_gate_scale), _ptr(w_up), _ptr(w_up_scale),
                         _ptr(w_down), _ptr(w_down_scale), _ptr(out), _ptr(workspace),
                         workspace.numel() * workspace.element_size(), M, H, I, variant,
                         _stream(stream)))


def _of(t, dtype, n, what) -> int:
    """Pointer of a tensor of `dtype` with n elements."""
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{what} has {t.numel()} elements, {n} needed")
    return _ptr(t)


_BF16 = frozenset((torch.bfloat16, torch.int16, torch.uint16))
_E4M3 = frozenset((torch.uint8, torch.float8_e4m3fn))
_F32 = frozenset((torch.float32,))


def _wrong_type(**tensors):
    """Raises for the first of what=(tensor, its dtypes) of another type.  (The callers
    test the types first, in one expression: a call's host time counts at decode.)"""
    for what, (t, dtypes) in tensors.items():
        if t.dtype not in dtypes:
            raise TypeError(f"{what} must be {' or '.join(sorted(map(str, dtypes)))}, got {t.dtype}")


def _scratch(t, dtypes, n, what) -> int:
    """Pointer of a scratch tensor of n elements or more."""
    if t.dtype not in dtypes:
        _wrong_type(**{what: (t, dtypes)})
    if t.numel() < n:
        raise ValueError(f"{what} has {t.numel()} elements, {n} needed")
    return _ptr(t)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def fp8q_moe_route_workspace_bytes(T: int, E: int, top_k: int) -> int:
    return int(lib().fp8q_moe_route_workspace_bytes(T, E, top_k))


def fp8q_moe_route(logits, ids, weights, order, pos, offsets, workspace, renormalize: bool = True,
                   stream=None):
    """Top-k routing of logits [T,E] (float32 or bfloat16) and the grouping of
    the T*top_k slots by expert.  Out: ids [T,top_k] int32, weights [T,top_k]
    float32, order and pos [T*top_k] int32, offsets [E+1] int32; workspace: a
    device tensor of fp8q_moe_route_workspace_bytes(T, E, top_k) bytes, or
    None when that is 0."""
    T, E = _dims(logits, 2)
    k = _dims(ids, 2)[1]
    bf16 = logits.dtype is torch.bfloat16
    if not bf16 and logits.dtype is not torch.float32:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    if ids.shape != weights.shape:
        raise ValueError("ids and weights disagree in shape")
    R, i32 = T * k, torch.int32
    st = lib().fp8q_moe_route(_ptr(logits), bf16, _of(ids, i32, R, "ids"), _of(weights, torch.float32, R, "weights"),
                              _of(order, i32, R, "order"), _of(pos, i32, R, "pos"),
                              _of(offsets, i32, E + 1, "offsets"), _optr(workspace), _nbytes(workspace), T, E, k,
                              bool(renormalize), _stream(stream))
    if st:
        _check(st)


def fp8q_group_rows_workspace_bytes(n: int, groups: int) -> int:
    return int(lib().fp8q_group_rows_workspace_bytes(n, groups))


def fp8q_group_rows(ids, order, pos, offsets, workspace, stream=None):
    """The grouping of given ids (any shape, int32) into offsets.numel() - 1
    groups; ids outside them come last.  workspace: a device tensor of
    fp8q_group_rows_workspace_bytes(n, groups) bytes, or None when that is 0."""
    n, groups, i32 = ids.numel(), offsets.numel() - 1, torch.int32
    _check(lib().fp8q_group_rows(_of(ids, i32, n, "ids"), _of(order, i32, n, "order"), _of(pos, i32, n, "pos"),
                                _of(offsets, i32, groups + 1, "offsets"), _optr(workspace), _nbytes(workspace), n,
                                groups, _stream(stream)))


def fp8q_moe_combine(y, weights, pos, offsets, out, stream=None):
    """out [T,H] = the weighted sum of each token's rows of y [T*top_k,H]
    (sorted rows, bf16), weights [T,top_k] float32."""
    T, k = _dims(weights, 2)
    R, H = _dims(y, 2)
    if R != T * k or _dims(out, 2) != (T, H):
        raise ValueError("y, weights and out disagree in shape")
    E = offsets.numel() - 1
    if not (y.dtype in _BF16 and out.dtype in _BF16):
        _wrong_type(y=(y, _BF16), out=(out, _BF16))
    _check(lib().fp8q_moe_combine(_ptr(y), _of(weights, torch.float32, R, "weights"),
                                 _of(pos, torch.int32, R, "pos"), _of(offsets, torch.int32, E + 1, "offsets"),
                                 _ptr(out), T, E, k, H, _stream(stream)))


def fp8q_gemm_grouped_select(R: int, E: int, N: int) -> int:
    """Kernel fp8q_gemm_grouped runs with kernel=0 for R rows in E groups and N
    columns: 1 weight streaming, 2 128x128 tiles, 3 persistent 128x256 tiles."""
    return int(lib().fp8q_gemm_grouped_select(R, E, N))


def fp8q_gemm_grouped(a, a_scale_km, w, w_scale, offsets, out, order=None, top_k: int = 1,
                      kernel: int = 0, stream=None):
    """out [R,N] = each sorted row times its expert's weights w [E,N,K] (block
    scales [E,N/128,K/128]).  With order, sorted row p reads activation row
    order[p] // top_k of a [R/top_k,K]; without, row p of a [R,K].  a_scale_km:
    K-major scales of a's rows.  Rows past offsets[E] are left as they are."""
    rows, K = _dims(a, 2)
    E, N, K2 = _dims(w, 3)
    R, N2 = _dims(out, 2)
    if K2 != K or N2 != N:
        raise ValueError("a, w and out disagree in shape")
    if w_scale.shape != (E, N // 128, K // 128) or a_scale_km.shape != (K // 128, (rows + 15) // 16 * 16):
        raise ValueError("a scale tensor's shape does not match")
    if not (a.dtype in _E4M3 and a_scale_km.dtype in _F32 and w.dtype in _E4M3 and w_scale.dtype in _F32
            and out.dtype in _BF16):
        _wrong_type(a=(a, _E4M3), a_scale_km=(a_scale_km, _F32), w=(w, _E4M3), w_scale=(w_scale, _F32), out=(out, _BF16))
    _check(lib().fp8q_gemm_grouped(_ptr(a), _ptr(a_scale_km), _ptr(w), _ptr(w_scale),
                                  _of(offsets, torch.int32, E + 1, "offsets"),
                                  0 if order is None else _of(order, torch.int32, R, "order"), _ptr(out), rows,
                                  R, E, top_k, N, K, kernel, _stream(stream)))


def fp8q_moe_ffn_select(T: int, E: int, top_k: int, I: int) -> int:
    """Variant fp8q_moe_ffn runs with variant=0: 1 fused gate/up, 2 separate."""
    return int(lib().fp8q_moe_ffn_select(T, E, top_k, I))


def fp8q_moe_ffn_workspace_bytes(T: int, E: int, top_k: int, H: int, I: int, variant: int = 0) -> int:
    return int(lib().fp8q_moe_ffn_workspace_bytes(T, E, top_k, H, I, variant))


def fp8q_moe_ffn(x, weights, order, pos, offsets, w_gate, w_gate_scale, w_up, w_up_scale, w_down,
                 w_down_scale, out, workspace, variant: int = 0, stream=None):
    """The experts' FFN: out [T,H] = the weighted sum over each token's experts
    of down(quant(bf16(silu(gate) * up))) of x [T,H].  weights [T,top_k]
    float32 and the grouping as from fp8q_moe_route; w_gate, w_up [E,I,H],
    w_down [E,H,I]; workspace: a device byte tensor of
    fp8q_moe_ffn_workspace_bytes(T, E, top_k, H, I, variant)."""
    T, H = _dims(x, 2)
    T2, k = _dims(weights, 2)
    E, I, H2 = _dims(w_gate, 3)
    if T2 != T or H2 != H or _dims(w_up, 3) != (E, I, H) or _dims(w_down, 3) != (E, H, I) or _dims(out, 2) != (T, H):
        raise ValueError("x, the weights and out disagree in shape")
    if not (w_gate_scale.shape == w_up_scale.shape == (E, I // 128, H // 128)
            and w_down_scale.shape == (E, H // 128, I // 128)):
        raise ValueError("a scale tensor's shape does not match")
    if not (x.dtype in _BF16 and out.dtype in _BF16 and w_gate.dtype in _E4M3 and w_up.dtype in _E4M3
            and w_down.dtype in _E4M3 and w_gate_scale.dtype in _F32 and w_up_scale.dtype in _F32
            and w_down_scale.dtype in _F32):
        _wrong_type(x=(x, _BF16), w_gate=(w_gate, _E4M3), w_gate_scale=(w_gate_scale, _F32), w_up=(w_up, _E4M3),
                    w_up_scale=(w_up_scale, _F32), w_down=(w_down, _E4M3), w_down_scale=(w_down_scale, _F32),
                    out=(out, _BF16))
    R, i32 = T * k, torch.int32
    _check(lib().fp8q_moe_ffn(_ptr(x), _of(weights, torch.float32, R, "weights"), _of(order, i32, R, "order"),
                             _of(pos, i32, R, "pos"), _of(offsets, i32, E + 1, "offsets"), _ptr(w_gate),
                             _ptr(w_gate_scale), _ptr(w_up), _ptr(w_up_scale), _ptr(w_down), _ptr(w_down_scale),
                             _ptr(out), _optr(workspace), _nbytes(workspace), T, E, k, H, I, variant,
                             _stream(stream)))


def fp8q_proj_lora_workspace_bytes(M: int, N: int, K: int, rank: int) -> int:
    return int(lib().fp8q_proj_lora_workspace_bytes(M, N, K, rank))


def fp8q_proj_lora(x, w, w_scale, lora_a, lora_b, lora_scale, adapter_ids, out, act_q, act_scale,
                   act_scale_km, workspace, stream=None):
    """fp8q_proj plus each row's low-rank adapter: out[m] = proj(x)[m] +
    lora_scale[a] * (x[m] . lora_a[a]^T) . lora_b[a]^T, a = adapter_ids[m]
    (outside 0..n-1: none).  lora_a [n,rank,K], lora_b [n,N,rank] bf16,
    lora_scale [n] float32, adapter_ids [M] int32; act_q, act_scale, act_scale_km:
    alloc_proj_scratch(M, K), or larger; workspace: a device byte tensor of
    fp8q_proj_lora_workspace_bytes(M, N, K, rank)."""
    M, K = _dims(x, 2)
    N, K2 = _dims(w, 2)
    n, R, K3 = _dims(lora_a, 3)
    if K2 != K or K3 != K or _dims(lora_b, 3) != (n, N, R) or _dims(out, 2) != (M, N):
        raise ValueError("x, w, the adapters and out disagree in shape")
    G = K // 128
    if w_scale.shape != (N // 128, G):
        raise ValueError("w_scale's shape does not match")
    if not (x.dtype in _BF16 and w.dtype in _E4M3 and w_scale.dtype in _F32 and lora_a.dtype in _BF16
            and lora_b.dtype in _BF16 and out.dtype in _BF16):
        _wrong_type(x=(x, _BF16), w=(w, _E4M3), w_scale=(w_scale, _F32), lora_a=(lora_a, _BF16),
                    lora_b=(lora_b, _BF16), out=(out, _BF16))
    _check(lib().fp8q_proj_lora(_ptr(x), _ptr(w), _ptr(w_scale), _ptr(lora_a), _ptr(lora_b),
                               _of(lora_scale, torch.float32, n, "lora_scale"),
                               _of(adapter_ids, torch.int32, M, "adapter_ids"), _ptr(out),
                               _scratch(act_q, _E4M3, M * K, "act_q"), _scratch(act_scale, _F32, M * G, "act_scale"),
                               _scratch(act_scale_km, _F32, G * ((M + 15) // 16 * 16), "act_scale_km"),
                               _optr(workspace), _nbytes(workspace), M, N, K, n, R, _stream(stream)))


_I32 = frozenset((torch.int32,))
_U8 = frozenset((torch.uint8,))


def _device(t, what) -> int:
    """The device of a call's first tensor, which has to be the current one (the call goes
    to its stream)."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{what} must be on the current GPU, got {t.device}")
    return dev


def _arg(t, dtypes, shape, what, dev) -> int:
    """Pointer of a contiguous tensor of one of `dtypes`, of `shape` and on device `dev`."""
    if t.dtype not in dtypes or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, dtypes, shape, what, dev)
    return t.data_ptr()


def _refuse(t, dtypes, shape, what, dev):
    if t.dtype not in dtypes:
        _wrong_type(**{what: (t, dtypes)})
    if t.shape != shape:
        raise ValueError(f"{what} must be of shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{what} must be on the current GPU, cuda:{dev}, got {t.device}")
    raise ValueError(f"{what} must be contiguous")


def _oarg(t, dtypes, shape, what, dev) -> int:
    return 0 if t is None else _arg(t, dtypes, shape, what, dev)


def _work(t, dev):
    """(pointer, bytes) of a workspace."""
    return (0, 0) if t is None else (_arg(t, _U8, t.shape, "workspace", dev), t.numel())


def fp8q_add_rmsnorm_quant(x, residual, weight, h, y, q, scale_rm, scale_km, rstd, eps: float = 1e-6, stream=None):
    """h = x + residual (bf16, [M,K]); q, scale_rm [M,K/128] and scale_km
    [K/128, ceil16(M)] = the FP8 codes and scales of h * rstd * weight, y the same in
    bf16, rstd [M] float32 = 1 / sqrt(mean(h^2) + eps).  residual and h go together
    (None: h is x); y, rstd and one of the scales may be None."""
    M, K = shape = _dims(x, 2)
    dev = _device(x, "x")
    _check(lib().fp8q_add_rmsnorm_quant(
        _arg(x, _BF16, shape, "x", dev), _oarg(residual, _BF16, shape, "residual", dev),
        _arg(weight, _BF16, (K,), "weight", dev),
        _oarg(h, _BF16, shape, "h", dev), _oarg(y, _BF16, shape, "y", dev), _arg(q, _E4M3, shape, "q", dev),
        _oarg(scale_rm, _F32, (M, K // 128), "scale_rm", dev),
        _oarg(scale_km, _F32, (K // 128, (M + 15) // 16 * 16), "scale_km", dev),
        _oarg(rstd, _F32, (M,), "rstd", dev), eps, M, K, _stream(stream)))


def fp8q_add_rmsnorm_grad_workspace_bytes(M: int, K: int) -> int:
    return int(lib().fp8q_add_rmsnorm_grad_workspace_bytes(M, K))


def fp8q_add_rmsnorm_grad(dy, dh, h, weight, rstd, dx, dweight, workspace, stream=None):
    """The gradient of fp8q_add_rmsnorm_quant: dx [M,K] bf16 (of x and of the residual)
    from dy (of y) and dh (of h; None: none), dweight [K] float32; workspace: a uint8
    tensor of fp8q_add_rmsnorm_grad_workspace_bytes(M, K)."""
    M, K = shape = _dims(h, 2)
    dev = _device(h, "h")
    work, nbytes = _work(workspace, dev)
    _check(lib().fp8q_add_rmsnorm_grad(
        _arg(dy, _BF16, shape, "dy", dev), _oarg(dh, _BF16, shape, "dh", dev), _arg(h, _BF16, shape, "h", dev),
        _arg(weight, _BF16, (K,), "weight", dev), _arg(rstd, _F32, (M,), "rstd", dev),
        _arg(dx, _BF16, shape, "dx", dev),
        _arg(dweight, _F32, (K,), "dweight", dev), work, nbytes, M, K, _stream(stream)))


def fp8q_quant_act_dual(x, q, scale_km, q_tok, exp_tok, stream=None):
    """Codes of x [M,K] bf16 along its rows (q, scale_km as fp8q_quant_act_kmajor's;
    both None: not wanted) and along its tokens (q_tok [M,K], exp_tok
    [ceil(M/512),K,4] uint8)."""
    M, K = shape = _dims(x, 2)
    dev = _device(x, "x")
    _check(lib().fp8q_quant_act_dual(
        _arg(x, _BF16, shape, "x", dev), _oarg(q, _E4M3, shape, "q", dev),
        _oarg(scale_km, _F32, (K // 128, (M + 15) // 16 * 16), "scale_km", dev),
        _arg(q_tok, _E4M3, shape, "q_tok", dev),
        _arg(exp_tok, _U8, ((M + 511) // 512, K, 4), "exp_tok", dev), M, K, _stream(stream)))


def fp8q_gemm_dgrad_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().fp8q_gemm_dgrad_workspace_bytes(M, N, K))


def fp8q_gemm_dgrad(dy, dy_scale_km, w, w_scale, dx, workspace, stream=None):
    """dx [M,K] bf16 = dy [M,N] times w [N,K] (row codes of dy with K-major scales; w as
    the forward call reads it); workspace: a uint8 tensor of
    fp8q_gemm_dgrad_workspace_bytes(M, N, K), or None when that is 0."""
    M, N = shape = _dims(dy, 2)
    dev = _device(dy, "dy")
    K = _dims(w, 2)[1]
    work, nbytes = _work(workspace, dev)
    _check(lib().fp8q_gemm_dgrad(
        _arg(dy, _E4M3, shape, "dy", dev), _arg(dy_scale_km, _F32, (N // 128, (M + 15) // 16 * 16), "dy_scale_km", dev),
        _arg(w, _E4M3, (N, K), "w", dev), _arg(w_scale, _F32, (N // 128, K // 128), "w_scale", dev),
        _arg(dx, _BF16, (M, K), "dx", dev), work, nbytes, M, N, K, _stream(stream)))


def fp8q_gemm_wgrad_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().fp8q_gemm_wgrad_workspace_bytes(M, N, K))


def fp8q_gemm_wgrad(dy_tok, dy_exp, x_tok, x_exp, dw, workspace, stream=None):
    """dw [N,K] bf16 = the transpose of dy [M,N] times x [M,K], both as
    fp8q_quant_act_dual's token codes and bytes; workspace: a uint8 tensor of
    fp8q_gemm_wgrad_workspace_bytes(M, N, K), or None when that is 0."""
    M, N = shape = _dims(dy_tok, 2)
    dev = _device(dy_tok, "dy_tok")
    K = _dims(x_tok, 2)[1]
    packs = (M + 511) // 512
    work, nbytes = _work(workspace, dev)
    _check(lib().fp8q_gemm_wgrad(
        _arg(dy_tok, _E4M3, shape, "dy_tok", dev), _arg(dy_exp, _U8, (packs, N, 4), "dy_exp", dev),
        _arg(x_tok, _E4M3, (M, K), "x_tok", dev), _arg(x_exp, _U8, (packs, K, 4), "x_exp", dev),
        _arg(dw, _BF16, (N, K), "dw", dev),
        work, nbytes, M, N, K, _stream(stream)))


_LOGITS = frozenset((torch.float32, torch.bfloat16))


def fp8q_moe_balance_workspace_bytes(T: int, E: int) -> int:
    return int(lib().fp8q_moe_balance_workspace_bytes(T, E))


def fp8q_moe_balance(logits, ids, counts, prob, loss, workspace, coef: float = 1.0, stream=None):
    """Balance loss of router logits [T,E] (float32 or bfloat16) and choices ids
    [T,top_k] int32: counts [E+1] int32 (the last: tokens with an expert to choose),
    prob [E] and loss [1] float32; workspace: a uint8 tensor of
    fp8q_moe_balance_workspace_bytes(T, E), or None when that is 0."""
    T, E = shape = _dims(logits, 2)
    dev = _device(logits, "logits")
    k = _dims(ids, 2)[1]
    work, nbytes = _work(workspace, dev)
    _check(lib().fp8q_moe_balance(
        _arg(logits, _LOGITS, shape, "logits", dev), logits.dtype is torch.bfloat16,
        _arg(ids, _I32, (T, k), "ids", dev), _arg(counts, _I32, (E + 1,), "counts", dev),
        _arg(prob, _F32, (E,), "prob", dev), _arg(loss, _F32, (1,), "loss", dev), work, nbytes, coef, T, E, k,
        _stream(stream)))


def fp8q_moe_route_grad(logits, ids, dweights, counts, dloss, dlogits, renormalize: bool = True, coef: float = 1.0,
                        top_k: int = None, stream=None):
    """dlogits [T,E], of the logits' type, through the weights of fp8q_moe_route (ids and
    their gradients dweights [T,top_k] float32; both None: not) and the balance loss
    (counts [E+1] of fp8q_moe_balance, dloss [1] float32 or None for 1; counts None:
    not).  top_k: needed where ids is None."""
    T, E = shape = _dims(logits, 2)
    dev = _device(logits, "logits")
    k = top_k if ids is None else _dims(ids, 2)[1]
    if k is None:
        raise ValueError("top_k is needed without ids")
    _check(lib().fp8q_moe_route_grad(
        _arg(logits, _LOGITS, shape, "logits", dev), logits.dtype is torch.bfloat16,
        _oarg(ids, _I32, (T, k), "ids", dev), _oarg(dweights, _F32, (T, k), "dweights", dev),
        _oarg(counts, _I32, (E + 1,), "counts", dev), _oarg(dloss, _F32, (1,), "dloss", dev),
        _arg(dlogits, (logits.dtype,), shape, "dlogits", dev), coef, T, E, k, bool(renormalize), _stream(stream)))


def fp8q_default_select_params(cu_count: int) -> SelectParams:
    return lib().fp8q_default_select_params(cu_count)


def fp8q_quant_select_with(M: int, K: int, params: SelectParams):
    """-> (variant, grid tuple, reject reason or None); variant -1 on bad args."""
    grid = (_U * 3)()
    why = ctypes.c_char_p()
    v = lib().fp8q_quant_select_with(M, K, ctypes.byref(params), ctypes.byref(grid),
                                    ctypes.byref(why))
    return v, tuple(grid), (why.value.decode() if why.value else None)


def fp8q_quant_select(M: int, K: int, cu_count: int):
    grid = (_U * 3)()
    why = ctypes.c_char_p()
    v = lib().fp8q_quant_select(M, K, cu_count, ctypes.byref(grid), ctypes.byref(why))
    return v, tuple(grid), (why.value.decode() if why.value else None)


def fp8q_gemm_select(M: int, N: int, K: int, cu_count: int = None) -> int:
    """Kernel id the auto GEMM runs for this shape (see fp8q_gemm_blockscaled_ex)
    on the current device, or on a device with cu_count compute units."""
    if cu_count is not None:
        return int(lib().fp8q_gemm_select_cus(M, N, K, cu_count))
    return int(lib().fp8q_gemm_select(M, N, K))


def fp8q_proj_quant_fused(M: int, K: int) -> bool:
    """True if fp8q_proj writes the K-major scales from the quantizer itself."""
    return bool(lib().fp8q_proj_quant_fused(M, K))


def fp8q_gemm_kernel_name(M: int, N: int, K: int, kernel: int = 0) -> str:
    """Name (as a kernel trace shows it) of the kernel fp8q_gemm_blockscaled
    runs for this shape and kernel id (0 = automatic) on the current device."""
    return lib().fp8q_gemm_kernel_name(M, N, K, kernel).decode()


FFN_GATE_UP_KERNEL_NAME = "gemm_pp_kernel<3, false, true>"
SPLITK_KERNEL_NAMES = ("gemm_tiled_kernel<128, 128, 2, 2, 2, false, true>", "splitk_reduce_kernel")
STREAMK_KERNEL_NAME = "gemm_pp_sk_kernel<3>"


def fp8q_quant_b_min_m(K: int, params: SelectParams) -> int:
    return int(lib().fp8q_quant_b_min_m(K, ctypes.byref(params)))


def fp8q_quant_log_slot(variant: int, reject, requested: bool) -> int:
    r = None if reject is None else reject.encode()
    return int(lib().fp8q_quant_log_slot(variant, r, int(bool(requested))))


def fp8q_clock_stamp(stamps, stream=None):
    """Clock stamp into stamps (int64 device tensor [n, 4]): per one-wave
    workgroup {XCD id, HW_ID, shader clock counter, 100 MHz counter}."""
    n, four = _dims(stamps, 2)
    if four != 4:
        raise ValueError("stamps must be [n, 4]")
    _check(lib().fp8q_clock_stamp(_ptr(stamps), n, _stream(stream)))


def shader_clock_ghz(before, after):
    """Average shader clock per XCD between two clock stamps (host arrays
    [n, 4] from fp8q_clock_stamp), pairing the stamps of the same CU:
    ({xcd: median GHz over its CU pairs}, number of pairs)."""
    first = {}
    for r in before:
        first.setdefault((int(r[0]), (int(r[1]) >> 8) & 0xFF), r)
    per = {}
    for r in after:
        b = first.get((int(r[0]), (int(r[1]) >> 8) & 0xFF))
        if b is None or int(r[3]) <= int(b[3]):
            continue
        per.setdefault(int(r[0]), []).append((int(r[2]) - int(b[2])) / (int(r[3]) - int(b[3])) * 0.1)
    import statistics
    return {x: statistics.median(v) for x, v in per.items()}, sum(len(v) for v in per.values())


# ------------------------------------------------------- allocation helpers
def alloc_proj_scratch(M: int, K: int, device="cuda"):
    """(act_q [M,K] u8, act_scale [M,K/128] f32, act_scale_km [K/128, ceil16(M)] f32)."""
    import torch
    G = K // 128
    return (torch.empty((M, K), dtype=torch.uint8, device=device),
            torch.empty((M, G), dtype=torch.float32, device=device),
            torch.empty((G, fp8q_m_pad(M)), dtype=torch.float32, device=device))


def alloc_ffn_workspace(M: int, H: int, I: int, variant: int = 0, device="cuda"):
    """Device byte tensor sized for fp8q_ffn(M, H, I, variant)."""
    import torch
    n = fp8q_ffn_workspace_bytes(M, H, I, variant)
    if n == 0:
        raise ValueError("invalid FFN shape or variant")
    return torch.empty((n,), dtype=torch.uint8, device=device)
