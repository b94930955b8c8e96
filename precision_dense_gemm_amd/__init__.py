"""Python binding of libpdgemm: multi-precision dense GEMM on MI355X (gfx950).

Argument marshalling only.  Every GEMM runs in the HIP kernels of
libpdgemm.so, called through its C ABI (include/pdgemm.h) on the current
torch stream.  torch is used for device memory and streams; nothing here
computes.  If the library has not been built, importing this package fails.

Operands are torch tensors on the GPU whose rows are contiguous in K:

    A    (M, K) row-major; a column slice of a wider buffer is fine
         (lda = A.stride(0))
    Bt   (N, K): the column-major B of C = A*B, stored as the rows of its
         transpose (ldb = Bt.stride(0))
    out  (M, N) row-major (ldc = out.stride(0)); allocated when omitted

With the *_rowb functions B is instead a (K, N) row-major tensor
(ldb = B.stride(0)); INT4 packs it along N, (K, N/2) bytes.

INT4 operands are uint8 tensors of packed bytes, (rows, K/2), two signed
4-bit values per byte with the even k in the low nibble; K is passed
explicitly and the leading dimensions are counted in 4-bit elements.

The dequantizing variants of the integer GEMMs take float32 scale vectors
scale_a (M,) and scale_b (N,) and write ((float)sum * scale_a[i]) *
scale_b[j] as float32, or rounded to float16.

MXFP4 operands (microscaled 4-bit floating point) are a pair of uint8 tensors:
packed codes (rows, ceil(K/2)), two e2m1 values per byte with the even k in the
low nibble, and scales (ceil(K/32), rows), the e8m0 byte of each block of 32
values stored by block.  Rows of both start on multiples of 16 bytes; mxf4_quantize
allocates them so, and rows of more than 1 KB of codes on multiples of 128 bytes,
the faster stride.  Scales that a checkpoint keeps by row, (rows, K/32), are
transposed once into such rows:
    scales = torch.empty(K // 32, (rows + 15) // 16 * 16, dtype=torch.uint8, device="cuda")[:, :rows]
    scales.copy_(by_row.t())

Around the products: rms_norm, rms_norm_i8 (whose codes and scales are the A and scale_a of
gemm_i8_dequant) and rms_norm_backward; gemm_a16_i4, 16-bit activations times symmetric INT4
weights (signed codes, no zero points) with scales by group, (ceil(K/group), N), of consecutive k;
moe_route and moe_a16_i4, a mixture-of-experts layer of such weights.

No call here records a graph: a result carries no gradient, whatever its inputs ask for.
A layer that trains computes dX and dW by calls of its own (see mxf4_quantize_both), for
example from a torch.autograd.Function.
"""
from __future__ import annotations

import ctypes
import os

# torch first: in a process that opened a HIP library before importing torch,
# torch's later device set-up failed (every GPU call returned hipErrorNoDevice)
import torch  # noqa: E402

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_HERE, "libpdgemm.so")

PREC_F16, PREC_I8, PREC_I4 = 0, 1, 2
I4_MAX_K = 131071

if not os.path.exists(LIBRARY):
    raise ImportError(
        f"{LIBRARY} is missing: build the HIP library first "
        "(python precision_dense_gemm_amd/build.py, or __graft_entry__.build())")

lib = ctypes.CDLL(LIBRARY)
_i64, _p, _i = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
for _name in ("gemm_f16", "gemm_i8", "gemm_i4"):
    getattr(lib, _name).argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
    getattr(lib, _name).restype = _i
for _name in ("gemm_i8_dequant", "gemm_i4_dequant"):
    getattr(lib, _name).argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _i64, _i, _p]
    getattr(lib, _name).restype = _i
for _name in ("gemm_f16_rowb", "gemm_i8_rowb", "gemm_i4_rowb"):
    getattr(lib, _name).argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
    getattr(lib, _name).restype = _i
lib.pdgemm_gemm_rowb_cfg.argtypes = [_i, _i, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
lib.pdgemm_gemm_rowb_cfg.restype = _i
lib.pdgemm_dequant_cfg.argtypes = [_i, _i, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _i64,
                                   _i, _p]
lib.pdgemm_dequant_cfg.restype = _i
lib.pdgemm_gemm_cfg.argtypes = [_i, _i, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
lib.pdgemm_gemm_cfg.restype = _i
lib.pdgemm_gemm_splitk_cfg.argtypes = [_i, _i, _i, _i, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
lib.pdgemm_gemm_splitk_cfg.restype = _i
lib.pdgemm_pick_splits.argtypes = [_i, _i, _i64, _i64, _i64, ctypes.POINTER(_i)]
lib.pdgemm_pick_splits.restype = _i
lib.pdgemm_num_configs.argtypes = []
lib.pdgemm_num_configs.restype = _i
lib.pdgemm_pick_config.argtypes = [_i, _i64, _i64, _i64]
lib.pdgemm_pick_config.restype = _i
lib.pdgemm_config_info.argtypes = [_i] + [ctypes.POINTER(_i)] * 5
lib.pdgemm_config_info.restype = _i
lib.pdgemm_i4_workspace_size.argtypes = [_i64, _i64, _i64]
lib.pdgemm_i4_workspace_size.restype = _i64
lib.pdgemm_i4_f6_workspace_bytes.argtypes = [_i64, _i64, _i64]
lib.pdgemm_i4_f6_workspace_bytes.restype = _i64
lib.pdgemm_i4_f6_pick.argtypes = [_i64, _i64, _i64]
lib.pdgemm_i4_f6_pick.restype = _i
lib.pdgemm_i4_f6_num_configs.argtypes = []
lib.pdgemm_i4_f6_num_configs.restype = _i
for _name in ("gemm_i4_ws", "gemm_i4_rowb_ws"):
    getattr(lib, _name).argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
    getattr(lib, _name).restype = _i
lib.gemm_i4_dequant_ws.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _i64, _i, _p, _i64,
                                   _p]
lib.gemm_i4_dequant_ws.restype = _i
lib.pdgemm_i4_f6_cfg.argtypes = [_i, _i, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _i64, _i, _p,
                                 _i64, _p]
lib.pdgemm_i4_f6_cfg.restype = _i
lib.pdgemm_i4_f6_image_bytes.argtypes = [_i64, _i64]
lib.pdgemm_i4_f6_image_bytes.restype = _i64
lib.pdgemm_i4_f6_pack.argtypes = [_i64, _i64, _p, _i64, _i, _p, _i64, _p]
lib.pdgemm_i4_f6_pack.restype = _i
lib.gemm_i4_packed_b.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
lib.gemm_i4_packed_b.restype = _i
lib.gemm_i4_dequant_packed_b.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _i64, _i, _p,
                                         _i64, _p]
lib.gemm_i4_dequant_packed_b.restype = _i
lib.pdgemm_i4_packed_b_cfg.argtypes = [_i, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _i64, _i, _p,
                                       _i64, _p]
lib.pdgemm_i4_packed_b_cfg.restype = _i
lib.gemm_i4_noalloc.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
lib.gemm_i4_noalloc.restype = _i
lib.pdgemm_i4_noalloc_max_bytes.argtypes = []
lib.pdgemm_i4_noalloc_max_bytes.restype = _i64
lib.pdgemm_mxf4_quantize.argtypes = [_i64, _i64, _p, _i64, _i, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _i, _p]
lib.pdgemm_mxf4_quantize.restype = _i
lib.pdgemm_mxf4_dequantize.argtypes = [_i64, _i64, _p, _i64, _p, _i64, _p, _i64, _i, _p]
lib.pdgemm_mxf4_dequantize.restype = _i
lib.gemm_mxf4.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _i, _p]
lib.gemm_mxf4.restype = _i
lib.pdgemm_mxf4_cfg.argtypes = [_i] + lib.gemm_mxf4.argtypes
lib.pdgemm_mxf4_cfg.restype = _i
lib.pdgemm_mxf4_num_configs.argtypes = []
lib.pdgemm_mxf4_num_configs.restype = _i
lib.pdgemm_mxf4_pick.argtypes = [_i64, _i64, _i64]
lib.pdgemm_mxf4_pick.restype = _i
lib.gemm_a16_mxf4.argtypes = [_i64, _i64, _i64, _p, _i64, _i, _p, _i64, _p, _i64, _p, _i64, _i, _p]
lib.gemm_a16_mxf4.restype = _i
lib.pdgemm_a16_mxf4_cfg.argtypes = [_i] + lib.gemm_a16_mxf4.argtypes
lib.pdgemm_a16_mxf4_cfg.restype = _i
lib.pdgemm_a16_mxf4_num_configs.argtypes = []
lib.pdgemm_a16_mxf4_num_configs.restype = _i
lib.pdgemm_a16_mxf4_pick.argtypes = [_i, _i64, _i64, _i64]
lib.pdgemm_a16_mxf4_pick.restype = _i
lib.pdgemm_rms_norm.argtypes = [_i64, _i64, _p, _i64, _i, _p, _i64, _p, _i64, _p, _i, ctypes.c_float, _p, _i64, _i,
                                _p, _p]
lib.pdgemm_rms_norm.restype = _i
lib.pdgemm_rms_norm_backward_workspace_size.argtypes = [_i64, _i64]
lib.pdgemm_rms_norm_backward_workspace_size.restype = _i64
lib.pdgemm_rms_norm_backward.argtypes = [_i64, _i64, _p, _i64, _p, _i64, _p, _i64, _i, _p, _i, ctypes.c_float, _p,
                                         _i64, _p, _p, _i64, _p]
lib.pdgemm_rms_norm_backward.restype = _i
lib.gemm_a16_i4.argtypes = [_i64, _i64, _i64, _p, _i64, _i, _p, _i64, _p, _i64, _i, _i64, _p, _i64, _i, _p, _i64, _p]
lib.gemm_a16_i4.restype = _i
lib.pdgemm_a16_i4_cfg.argtypes = [_i] + lib.gemm_a16_i4.argtypes
lib.pdgemm_a16_i4_cfg.restype = _i
lib.pdgemm_a16_i4_workspace_size.argtypes = [_i64, _i64, _i64, _i64]
lib.pdgemm_a16_i4_workspace_size.restype = _i64
lib.pdgemm_a16_i4_cfg_workspace_size.argtypes = [_i, _i64, _i64, _i64]
lib.pdgemm_a16_i4_cfg_workspace_size.restype = _i64
lib.pdgemm_a16_i4_num_configs.argtypes = []
lib.pdgemm_a16_i4_num_configs.restype = _i
lib.pdgemm_a16_i4_pick.argtypes = [_i64, _i64, _i64, _i64]
lib.pdgemm_a16_i4_pick.restype = _i
lib.pdgemm_moe_route.argtypes = [_i64, _i64, _i64, _p, _i64, _i, _i, _p, _p, _p]
lib.pdgemm_moe_route.restype = _i
lib.pdgemm_moe_a16_i4_workspace_size.argtypes = [_i64] * 5
lib.pdgemm_moe_a16_i4_workspace_size.restype = _i64
lib.pdgemm_moe_a16_i4_wide_workspace_size.argtypes = [_i64] * 5
lib.pdgemm_moe_a16_i4_wide_workspace_size.restype = _i64
lib.pdgemm_moe_a16_i4.argtypes = ([_i64] * 5 + [_p, _i64, _i, _p, _p] + [_p, _i64, _i64] * 4
                                  + [_i, _i64, _p, _i64, _p, _i64, _p])
lib.pdgemm_moe_a16_i4.restype = _i
lib.pdgemm_strerror.argtypes = [_i]
lib.pdgemm_strerror.restype = ctypes.c_char_p
lib.pdgemm_version.argtypes = []
lib.pdgemm_version.restype = _i


class PdgemmError(RuntimeError):
    def __init__(self, code: int):
        self.code = code
        super().__init__(f"pdgemm error {code}: {strerror(code)}")


def strerror(code: int) -> str:
    return lib.pdgemm_strerror(code).decode()


def version() -> int:
    return lib.pdgemm_version()


def num_configs() -> int:
    return lib.pdgemm_num_configs()


def pick_config(prec: int, M: int, N: int, K: int) -> int:
    return lib.pdgemm_pick_config(prec, M, N, K)


def pick_splits(prec: int, M: int, N: int, K: int, rowb: bool = False) -> tuple[int, int]:
    """(ranges of K, tile configuration) the raw-sum entry points use for a shape;
    ranges == 1: no K split across workgroups."""
    cfg = _i()
    s = lib.pdgemm_pick_splits(prec, 1 if rowb else 0, M, N, K, ctypes.byref(cfg))
    return s, cfg.value


def config_info(cfg: int) -> dict:
    vals = [_i() for _ in range(5)]
    rc = lib.pdgemm_config_info(cfg, *[ctypes.byref(v) for v in vals])
    if rc:
        raise PdgemmError(rc)
    keys = ("block_m", "block_n", "wave_m", "wave_n", "threads")
    return {k: v.value for k, v in zip(keys, vals)}


def i4_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace the INT4 workspace entry points need for this shape
    (0 where they run the INT8-MFMA kernels)."""
    return lib.pdgemm_i4_workspace_size(M, N, K)


def i4_f6_workspace_bytes(M: int, N: int, K: int) -> int:
    """Bytes of workspace of the FP6 path for this shape, whichever tile it takes."""
    return lib.pdgemm_i4_f6_workspace_bytes(M, N, K)


def i4_f6_pick(M: int, N: int, K: int) -> int:
    """The FP6 tile the workspace entry points take for this shape (-1: INT8-MFMA kernels)."""
    return lib.pdgemm_i4_f6_pick(M, N, K)


def i4_f6_num_configs() -> int:
    return lib.pdgemm_i4_f6_num_configs()


def i4_workspace(M: int, N: int, K: int, device=None, f6: bool = False) -> torch.Tensor:
    """A workspace tensor for an INT4 GEMM of this shape (at least 256 bytes; with f6,
    sized for the FP6 path whatever the library would pick)."""
    n = i4_f6_workspace_bytes(M, N, K) if f6 else i4_workspace_size(M, N, K)
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _row_major_2d(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows (stride(1) == 1)")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _scale(t: torch.Tensor, n: int, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.dim() != 1:
        raise TypeError(f"{name} must be a 1-D float32 tensor")
    if t.shape[0] != n:
        raise ValueError(f"{name} must hold {n} values")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.data_ptr()


def _workspace(ws, device):
    """(pointer, bytes) of a workspace tensor (or (None, 0))."""
    if ws is None:
        return None, 0
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or not ws.is_contiguous():
        raise TypeError("workspace must be a contiguous GPU tensor")
    if ws.device != device:
        raise ValueError("workspace must be on the operands' GPU")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _marshal(prec, A, Bt, out, K, lda, ldb, stream, cfg, scales=None, N=None, rowb=False,
             workspace=None, f6cfg=None, splits=None):
    """The C function and its argument tuple for one GEMM (dequantizing when
    scales = (scale_a, scale_b) is given; B row-major when rowb, with N given;
    INT4 on the FP6 cores with a workspace, by the library's choice or with
    the FP6 tile f6cfg; K split over `splits` ranges across workgroups on the
    tile cfg)."""
    M = A.shape[0]
    N = Bt.shape[0] if N is None else N
    ldc = _row_major_2d(out, "out")
    tensors = [A, Bt, out] + ([] if scales is None else list(scales))
    if any(isinstance(t, torch.Tensor) and t.device != out.device for t in tensors):
        raise ValueError("operands, scales and out must be on the same GPU")
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must have shape {(M, N)}")
    if splits is not None:
        if cfg is None or scales is not None or workspace is not None or f6cfg is not None:
            raise ValueError("a K split across workgroups takes a tile cfg and no scales or workspace")
        return lib.pdgemm_gemm_splitk_cfg, (prec, cfg, 1 if rowb else 0, splits, M, N, K, A.data_ptr(), lda,
                                            Bt.data_ptr(), ldb, out.data_ptr(), ldc, _stream(stream))
    if workspace is not None or f6cfg is not None:
        if prec != PREC_I4:
            raise ValueError("a workspace serves the INT4 GEMM on the FP6 cores only")
        if cfg is not None:
            raise ValueError("cfg selects an INT8-MFMA tile; the FP6 tile is f6cfg")
        ws, ws_bytes = _workspace(workspace, out.device)
        sa = sb = None
        if scales is not None:
            if out.dtype not in (torch.float32, torch.float16):
                raise TypeError("a dequantizing GEMM writes float32 or float16")
            sa, sb = _scale(scales[0], M, "scale_a"), _scale(scales[1], N, "scale_b")
        half = 1 if out.dtype == torch.float16 else 0
        if f6cfg is not None:
            return lib.pdgemm_i4_f6_cfg, (f6cfg, 1 if rowb else 0, M, N, K, A.data_ptr(), lda,
                                          Bt.data_ptr(), ldb, sa, sb, out.data_ptr(), ldc, half, ws,
                                          ws_bytes, _stream(stream))
        if scales is not None:
            if rowb:
                raise ValueError("the dequantizing epilogue takes a column-major B")
            return lib.gemm_i4_dequant_ws, (M, N, K, A.data_ptr(), lda, Bt.data_ptr(), ldb, sa, sb,
                                            out.data_ptr(), ldc, half, ws, ws_bytes, _stream(stream))
        fn = lib.gemm_i4_rowb_ws if rowb else lib.gemm_i4_ws
        return fn, (M, N, K, A.data_ptr(), lda, Bt.data_ptr(), ldb, out.data_ptr(), ldc, ws, ws_bytes,
                    _stream(stream))
    if rowb:
        if scales is not None:
            raise ValueError("the dequantizing epilogue takes a column-major B")
        args = (M, N, K, A.data_ptr(), lda, Bt.data_ptr(), ldb, out.data_ptr(), ldc,
                _stream(stream))
        if cfg is None:
            return (lib.gemm_f16_rowb, lib.gemm_i8_rowb, lib.gemm_i4_rowb)[prec], args
        return lib.pdgemm_gemm_rowb_cfg, (prec, cfg) + args
    if scales is None:
        args = (M, N, K, A.data_ptr(), lda, Bt.data_ptr(), ldb, out.data_ptr(), ldc,
                _stream(stream))
        if cfg is None:
            return (lib.gemm_f16, lib.gemm_i8, lib.gemm_i4)[prec], args
        return lib.pdgemm_gemm_cfg, (prec, cfg) + args
    if prec == PREC_F16:
        raise ValueError("the dequantizing epilogue is for INT8 and INT4")
    if out.dtype not in (torch.float32, torch.float16):
        raise TypeError("a dequantizing GEMM writes float32 or float16")
    args = (M, N, K, A.data_ptr(), lda, Bt.data_ptr(), ldb, _scale(scales[0], M, "scale_a"),
            _scale(scales[1], N, "scale_b"), out.data_ptr(), ldc,
            1 if out.dtype == torch.float16 else 0, _stream(stream))
    if cfg is None:
        return (None, lib.gemm_i8_dequant, lib.gemm_i4_dequant)[prec], args
    return lib.pdgemm_dequant_cfg, (prec, cfg) + args


def _call(prec, A, Bt, out, K, lda, ldb, stream, cfg, scales=None, N=None, rowb=False, workspace=None,
          f6cfg=None, splits=None):
    fn, args = _marshal(prec, A, Bt, out, K, lda, ldb, stream, cfg, scales, N, rowb, workspace, f6cfg, splits)
    rc = fn(*args)
    if rc != 0:
        raise PdgemmError(rc)
    return out


def gemm_f16(A: torch.Tensor, Bt: torch.Tensor, out: torch.Tensor | None = None,
             stream=None, cfg: int | None = None, splits: int | None = None) -> torch.Tensor:
    """C = A * B for binary16 A (M, K) and Bt (N, K); fp32 accumulate, fp32 C (M, N)."""
    if A.dtype != torch.float16 or Bt.dtype != torch.float16:
        raise TypeError("gemm_f16 takes float16 operands")
    K = A.shape[1]
    if Bt.shape[1] != K:
        raise ValueError("A and Bt disagree on K")
    lda, ldb = _row_major_2d(A, "A"), _row_major_2d(Bt, "Bt")
    if out is None:
        out = torch.empty((A.shape[0], Bt.shape[0]), dtype=torch.float32, device=A.device)
    elif out.dtype != torch.float32:
        raise TypeError("gemm_f16 writes a float32 output")
    return _call(PREC_F16, A, Bt, out, K, lda, ldb, stream, cfg, splits=splits)


def gemm_i8(A: torch.Tensor, Bt: torch.Tensor, out: torch.Tensor | None = None,
            stream=None, cfg: int | None = None, splits: int | None = None) -> torch.Tensor:
    """C = A * B for int8 A (M, K) and Bt (N, K); int32 accumulate, int32 C (M, N)."""
    if A.dtype != torch.int8 or Bt.dtype != torch.int8:
        raise TypeError("gemm_i8 takes int8 operands")
    K = A.shape[1]
    if Bt.shape[1] != K:
        raise ValueError("A and Bt disagree on K")
    lda, ldb = _row_major_2d(A, "A"), _row_major_2d(Bt, "Bt")
    if out is None:
        out = torch.empty((A.shape[0], Bt.shape[0]), dtype=torch.int32, device=A.device)
    elif out.dtype != torch.int32:
        raise TypeError("gemm_i8 writes an int32 output")
    return _call(PREC_I8, A, Bt, out, K, lda, ldb, stream, cfg, splits=splits)


def gemm_i4(A: torch.Tensor, Bt: torch.Tensor, K: int | None = None,
            out: torch.Tensor | None = None, stream=None, cfg: int | None = None,
            workspace: torch.Tensor | None = None, f6cfg: int | None = None,
            splits: int | None = None) -> torch.Tensor:
    """C = A * B for packed INT4 A (M, K/2) and Bt (N, K/2) bytes; int32 C (M, N).
    With a workspace (see i4_workspace) the library may run it on the FP6 cores."""
    if A.dtype != torch.uint8 or Bt.dtype != torch.uint8:
        raise TypeError("gemm_i4 takes uint8 tensors of packed 4-bit values")
    if K is None:
        K = 2 * A.shape[1]
    if A.shape[1] * 2 < K or Bt.shape[1] * 2 < K:
        raise ValueError("packed operands hold fewer than K values per row")
    lda, ldb = 2 * _row_major_2d(A, "A"), 2 * _row_major_2d(Bt, "Bt")
    if out is None:
        out = torch.empty((A.shape[0], Bt.shape[0]), dtype=torch.int32, device=A.device)
    elif out.dtype != torch.int32:
        raise TypeError("gemm_i4 writes an int32 output")
    return _call(PREC_I4, A, Bt, out, K, lda, ldb, stream, cfg, workspace=workspace, f6cfg=f6cfg,
                 splits=splits)


def gemm_i4_noalloc(A: torch.Tensor, Bt: torch.Tensor, K: int | None = None,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gemm_i4 through the allocation-free entry point (the library's own fixed
    workspace; calls that overlap on one GPU race)."""
    if A.dtype != torch.uint8 or Bt.dtype != torch.uint8:
        raise TypeError("gemm_i4_noalloc takes uint8 tensors of packed 4-bit values")
    if K is None:
        K = 2 * A.shape[1]
    if A.shape[1] * 2 < K or Bt.shape[1] * 2 < K:
        raise ValueError("packed operands hold fewer than K values per row")
    lda, ldb = 2 * _row_major_2d(A, "A"), 2 * _row_major_2d(Bt, "Bt")
    if out is None:
        out = torch.empty((A.shape[0], Bt.shape[0]), dtype=torch.int32, device=A.device)
    elif out.dtype != torch.int32:
        raise TypeError("gemm_i4_noalloc writes an int32 output")
    M, N = A.shape[0], Bt.shape[0]
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must have shape {(M, N)}")
    if A.device != out.device or Bt.device != out.device:
        raise ValueError("operands and out must be on the same GPU")
    rc = lib.gemm_i4_noalloc(M, N, K, A.data_ptr(), lda, Bt.data_ptr(), ldb, out.data_ptr(),
                             _row_major_2d(out, "out"), _stream(stream))
    if rc != 0:
        raise PdgemmError(rc)
    return out


def i4_f6_image_bytes(rows: int, K: int) -> int:
    """Bytes of the FP6 image of an INT4 operand of `rows` rows of K values."""
    return int(lib.pdgemm_i4_f6_image_bytes(rows, K))


def i4_f6_pack(src: torch.Tensor, K: int | None = None, rowmajor: bool = False, N: int | None = None,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The FP6 image (a uint8 tensor) of an INT4 operand, for gemm_i4_packed_b:
    src (rows, K/2) packed along K (A, or a column-major B as Bt), or with
    rowmajor a row-major B (K, N/2) packed along N (N defaults to 2 * src.shape[1])."""
    if src.dtype != torch.uint8:
        raise TypeError("i4_f6_pack takes a uint8 tensor of packed 4-bit values")
    ld = 2 * _row_major_2d(src, "src")
    if rowmajor:
        K = src.shape[0] if K is None else K
        rows = 2 * src.shape[1] if N is None else N
        if src.shape[0] < K or 2 * src.shape[1] < rows:
            raise ValueError("src holds fewer than K rows of N values")
    else:
        K = 2 * src.shape[1] if K is None else K
        rows = src.shape[0]
        if 2 * src.shape[1] < K:
            raise ValueError("src holds fewer than K values per row")
    need = i4_f6_image_bytes(rows, K)
    if out is None:
        out = torch.empty(max(need, 16), dtype=torch.uint8, device=src.device)
    ptr, nbytes = _workspace(out, src.device)
    rc = lib.pdgemm_i4_f6_pack(rows, K, src.data_ptr(), ld, 1 if rowmajor else 0, ptr, nbytes, _stream(stream))
    if rc != 0:
        raise PdgemmError(rc)
    return out


def gemm_i4_packed_b(A: torch.Tensor, image_b: torch.Tensor, K: int, N: int, out: torch.Tensor | None = None,
                     scales=None, workspace: torch.Tensor | None = None, f6cfg: int | None = None,
                     stream=None) -> torch.Tensor:
    """C = A * B with B given as its FP6 image (i4_f6_pack of N rows, same K): int32 C,
    or with scales = (scale_a, scale_b) the dequantized float32 / float16 C."""
    if A.dtype != torch.uint8:
        raise TypeError("gemm_i4_packed_b takes a uint8 A of packed 4-bit values")
    if 2 * A.shape[1] < K:
        raise ValueError("A holds fewer than K values per row")
    M = A.shape[0]
    lda = 2 * _row_major_2d(A, "A")
    if out is None:
        out = torch.empty((M, N), dtype=torch.int32 if scales is None else torch.float32, device=A.device)
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must have shape {(M, N)}")
    if scales is None and out.dtype != torch.int32:
        raise TypeError("gemm_i4_packed_b writes an int32 output")
    if scales is not None and out.dtype not in (torch.float32, torch.float16):
        raise TypeError("a dequantizing GEMM writes float32 or float16")
    if A.device != out.device:
        raise ValueError("A and out must be on the same GPU")
    if workspace is None:
        workspace = torch.empty(max(i4_f6_image_bytes(M, K), 16), dtype=torch.uint8, device=A.device)
    ws, ws_bytes = _workspace(workspace, out.device)
    img, img_bytes = _workspace(image_b, out.device)
    ldc = _row_major_2d(out, "out")
    sa = sb = None
    if scales is not None:
        sa, sb = _scale(scales[0], M, "scale_a"), _scale(scales[1], N, "scale_b")
    half = 1 if out.dtype == torch.float16 else 0
    if f6cfg is not None:
        rc = lib.pdgemm_i4_packed_b_cfg(f6cfg, M, N, K, A.data_ptr(), lda, img, img_bytes, sa, sb,
                                        out.data_ptr(), ldc, half, ws, ws_bytes, _stream(stream))
    elif scales is not None:
        rc = lib.gemm_i4_dequant_packed_b(M, N, K, A.data_ptr(), lda, img, img_bytes, sa, sb, out.data_ptr(),
                                          ldc, half, ws, ws_bytes, _stream(stream))
    else:
        rc = lib.gemm_i4_packed_b(M, N, K, A.data_ptr(), lda, img, img_bytes, out.data_ptr(), ldc, ws,
                                  ws_bytes, _stream(stream))
    if rc != 0:
        raise PdgemmError(rc)
    return out


_DTYPES = {"f16": (torch.float16, torch.float32, PREC_F16), "i8": (torch.int8, torch.int32, PREC_I8),
           "i4": (torch.uint8, torch.int32, PREC_I4)}


def _gemm_rowb(prec, A, B, K, N, out, stream, cfg, workspace=None, f6cfg=None, splits=None):
    in_t, out_t, p = _DTYPES[prec]
    if A.dtype != in_t or B.dtype != in_t:
        raise TypeError(f"{prec} with row-major B takes {in_t} operands")
    per = 2 if prec == "i4" else 1
    K = per * A.shape[1] if K is None else K
    N = per * B.shape[1] if N is None else N
    if per * A.shape[1] < K or B.shape[0] < K or per * B.shape[1] < N:
        raise ValueError("operands hold fewer than K values per row of A, K rows of B or N columns")
    lda, ldb = per * _row_major_2d(A, "A"), per * _row_major_2d(B, "B")
    if out is None:
        out = torch.empty((A.shape[0], N), dtype=out_t, device=A.device)
    elif out.dtype != out_t:
        raise TypeError(f"{prec} writes a {out_t} output")
    return _call(p, A, B, out, K, lda, ldb, stream, cfg, N=N, rowb=True, workspace=workspace,
                 f6cfg=f6cfg, splits=splits)


def gemm_f16_rowb(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor | None = None,
                  stream=None, cfg: int | None = None, splits: int | None = None) -> torch.Tensor:
    """C = A * B for binary16 A (M, K) and row-major B (K, N); fp32 C (M, N)."""
    return _gemm_rowb("f16", A, B, None, None, out, stream, cfg, splits=splits)


def gemm_i8_rowb(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor | None = None,
                 stream=None, cfg: int | None = None, splits: int | None = None) -> torch.Tensor:
    """C = A * B for int8 A (M, K) and row-major B (K, N); int32 C (M, N)."""
    return _gemm_rowb("i8", A, B, None, None, out, stream, cfg, splits=splits)


def gemm_i4_rowb(A: torch.Tensor, B: torch.Tensor, K: int | None = None, N: int | None = None,
                 out: torch.Tensor | None = None, stream=None, cfg: int | None = None,
                 workspace: torch.Tensor | None = None, f6cfg: int | None = None,
                 splits: int | None = None) -> torch.Tensor:
    """C = A * B for packed INT4 A (M, K/2) and row-major B (K, N/2 bytes, packed along N)."""
    return _gemm_rowb("i4", A, B, K, N, out, stream, cfg, workspace, f6cfg, splits)


def gemm_i8_dequant(A: torch.Tensor, Bt: torch.Tensor, scale_a: torch.Tensor,
                    scale_b: torch.Tensor, out: torch.Tensor | None = None,
                    out_dtype: torch.dtype = torch.float32, stream=None,
                    cfg: int | None = None) -> torch.Tensor:
    """INT8 GEMM, then C[i][j] = ((float)sum * scale_a[i]) * scale_b[j] in binary32,
    stored as float32 or rounded to float16 (out's dtype, else out_dtype)."""
    if A.dtype != torch.int8 or Bt.dtype != torch.int8:
        raise TypeError("gemm_i8_dequant takes int8 operands")
    K = A.shape[1]
    if Bt.shape[1] != K:
        raise ValueError("A and Bt disagree on K")
    lda, ldb = _row_major_2d(A, "A"), _row_major_2d(Bt, "Bt")
    if out is None:
        out = torch.empty((A.shape[0], Bt.shape[0]), dtype=out_dtype, device=A.device)
    return _call(PREC_I8, A, Bt, out, K, lda, ldb, stream, cfg, (scale_a, scale_b))


def gemm_i4_dequant(A: torch.Tensor, Bt: torch.Tensor, scale_a: torch.Tensor,
                    scale_b: torch.Tensor, K: int | None = None,
                    out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
                    stream=None, cfg: int | None = None, workspace: torch.Tensor | None = None,
                    f6cfg: int | None = None) -> torch.Tensor:
    """Packed INT4 GEMM with the dequantizing epilogue of gemm_i8_dequant."""
    if A.dtype != torch.uint8 or Bt.dtype != torch.uint8:
        raise TypeError("gemm_i4_dequant takes uint8 tensors of packed 4-bit values")
    if K is None:
        K = 2 * A.shape[1]
    if A.shape[1] * 2 < K or Bt.shape[1] * 2 < K:
        raise ValueError("packed operands hold fewer than K values per row")
    lda, ldb = 2 * _row_major_2d(A, "A"), 2 * _row_major_2d(Bt, "Bt")
    if out is None:
        out = torch.empty((A.shape[0], Bt.shape[0]), dtype=out_dtype, device=A.device)
    return _call(PREC_I4, A, Bt, out, K, lda, ldb, stream, cfg, (scale_a, scale_b), workspace=workspace,
                 f6cfg=f6cfg)


# ---- MXFP4 ----

MX_BLOCK = 32
_MX_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_MX_RULES = {"floor": 0, "fit": 1}


def _round_up(x: int, m: int) -> int:
    return (x + m - 1) // m * m


def _mx_type(dtype, name: str) -> int:
    kind = _MX_TYPES.get(dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16")
    return kind


# The calls these serve can be shorter than their checks, so the checks are few and cheap:
# one look at a tensor's shape and stride, device indices rather than device objects, and
# the current stream's handle without a Stream object around it.

def _mx_rows(t: torch.Tensor, name: str) -> tuple[int, int, int]:
    """(rows, columns, row stride) of a 2-D tensor with contiguous rows.  A single row's stride
    says nothing (the last token of a sequence, h[:, -1, :], has the whole sequence's) and may pass
    the longest row the library takes, so its length stands for it."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows (stride(1) == 1)")
    return rows, cols, (ld if rows > 1 else cols)


def _mx_operand(codes: torch.Tensor, scales: torch.Tensor, K: int | None, name: str):
    """(rows, K, ld in values, scale row stride) of an MXFP4 operand.  The stride of a single
    row is its length, up to the next multiple the library accepts."""
    if not isinstance(codes, torch.Tensor) or codes.dtype is not torch.uint8:
        raise TypeError(f"{name}'s codes must be a uint8 tensor")
    if not isinstance(scales, torch.Tensor) or scales.dtype is not torch.uint8:
        raise TypeError(f"{name}'s scales must be a uint8 tensor")
    rows, width, ld = _mx_rows(codes, name)
    have, cols, lds = _mx_rows(scales, name)
    if K is None:
        K = 2 * width
    elif K < 0 or 2 * width < K:
        raise ValueError(f"{name} holds fewer than K values per row")
    blocks = (K + MX_BLOCK - 1) // MX_BLOCK
    if width > blocks * (MX_BLOCK // 2):   # (bytes that only fill the last block may be part of it)
        raise ValueError(f"{name}'s codes and the call disagree on K")
    if have < blocks or cols < rows:
        raise ValueError(f"{name}'s scales must hold {blocks} blocks of {rows} rows")
    if rows <= 1:
        ld = _round_up(ld, 16)
    if have <= 1:
        lds = _round_up(lds, 16)
    return rows, K, 2 * ld, lds


def _mx_call(fn, args, tensors, stream):
    """Runs fn(*args, stream) for tensors of one GPU, with that GPU current: on `stream`, or
    on its current stream."""
    index = tensors[0].get_device()   # -1: not on a GPU
    for t in tensors:
        if t.get_device() != index or index < 0:
            raise ValueError("all tensors must be on the same GPU")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device_index == index:
        handle = stream.cuda_stream
    else:
        raise ValueError("stream must be on the tensors' GPU")
    if index == torch.cuda.current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc != 0:
        raise PdgemmError(rc)


def _mx_empty(rows, cols, dtype, device, stream):
    """A new tensor of the stream that will write it, so that its memory is not handed out
    again before that stream is done with it."""
    if stream is None:
        return torch.empty(rows, cols, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(rows, cols, dtype=dtype, device=device)


def _mx_new_form(rows, width, row, blocks, lds, device):
    """New codes (rows, width) in rows of `row` bytes, and scales (blocks, rows) in rows of
    `lds`: made with their strides, which costs less than half of making and slicing them.
    The codes' memory holds their last row whole, as the quantiser writes it; of the scales the
    last 16 bytes are only read whole, and an allocation is of whole 16-byte granules."""
    codes = torch.empty(rows, row, dtype=torch.uint8, device=device)
    if row != width:
        codes = codes.as_strided((rows, width), (row, 1))
    return codes, torch.empty_strided((blocks, rows), (lds, 1), dtype=torch.uint8, device=device)


def _mx_form(out, rows: int, K: int, device, stream, name: str):
    """An operand to write, `out` or a new one whose rows the library takes: its tensors, and its
    part of the C call's arguments."""
    if out is not None:
        codes, scales = out
        r, _, ld, lds = _mx_operand(codes, scales, K, name)
        if r != rows:
            raise ValueError(f"{name} must have {rows} rows")
        # the last row's last chunk is written whole: 16 bytes a block, wherever the view ends
        end = codes.storage_offset() + (rows - 1) * (ld // 2) + 16 * ((K + MX_BLOCK - 1) // MX_BLOCK)
        if rows and codes.untyped_storage().nbytes() < end:
            raise ValueError(f"{name}'s codes must have room for whole 16-byte blocks in every row")
        return (codes, scales), (codes.data_ptr(), ld, scales.data_ptr(), lds)
    blocks = (K + MX_BLOCK - 1) // MX_BLOCK
    lds = _round_up(rows, 16)
    row, width = 16 * blocks, (K + 1) // 2
    if row > 1024:
        # whole 128-byte lines, which the products copy: 2000 x 5000 x 7000 46 us and not 52
        row = _round_up(row, 128)
    if stream is None:
        codes, scales = _mx_new_form(rows, width, row, blocks, lds, device)
    else:
        with torch.cuda.stream(stream):
            codes, scales = _mx_new_form(rows, width, row, blocks, lds, device)
    return (codes, scales), (codes.data_ptr(), 2 * row, scales.data_ptr(), lds)


_MX_NO_FORM = (None, 0, None, 0)


def _mx_quantize(x, along_k: bool, along_rows: bool, scale_rule, out, out_t, stream):
    kind = _mx_type(x.dtype, "x")
    rule = _MX_RULES.get(scale_rule)
    if rule is None:
        raise ValueError(f"scale_rule must be one of {sorted(_MX_RULES)}")
    rows, K, ld = _mx_rows(x, "x")
    device = x.device
    q = qt = None
    args = args_t = _MX_NO_FORM
    if along_k:
        q, args = _mx_form(out, rows, K, device, stream, "out")
    if along_rows:
        qt, args_t = _mx_form(out_t, K, rows, device, stream, "the transposed out")
    if rows and K:
        tensors = (x,) + (() if out is None else q) + (() if out_t is None else qt)
        _mx_call(lib.pdgemm_mxf4_quantize, (rows, K, x.data_ptr(), ld, kind, *args, *args_t, rule), tensors, stream)
    return q, qt


def mxf4_quantize(x: torch.Tensor, transpose: bool = False, scale_rule: str = "floor", out=None, stream=None):
    """(codes, scales) of x (rows, K), float32, float16 or bfloat16, in MXFP4 along K; with
    transpose, of its transpose: K rows quantised along x's rows, for a product that contracts
    over them.  scale_rule "floor" is the rule of the MX specification (values above 6 times
    the scale saturate), "fit" takes the smallest scale at which none does.  A block that holds
    an infinity or a NaN becomes NaN.  out: a (codes, scales) pair to write."""
    if transpose:
        return _mx_quantize(x, False, True, scale_rule, None, out, stream)[1]
    return _mx_quantize(x, True, False, scale_rule, out, None, stream)[0]


def mxf4_quantize_both(x: torch.Tensor, scale_rule: str = "floor", out=None, stream=None):
    """((codes, scales), (codes_t, scales_t)): mxf4_quantize of x and of its transpose, from one
    read of x.  out: a pair of such pairs to write.

    A linear layer Y = X W^T takes both forms of X, W and G = dL/dY: Y contracts X and W along K,
    dX = G W takes G's rows and W's transpose, dW = G^T X both transposes."""
    first, second = (None, None) if out is None else out
    return _mx_quantize(x, True, True, scale_rule, first, second, stream)


def _mx_dense_out(out, rows, cols, out_dtype, device, stream):
    """(out or a new tensor, its row stride, its type)."""
    kind = _mx_type(out_dtype if out is None else out.dtype, "the output")
    if out is None:
        return _mx_empty(rows, cols, out_dtype, device, stream), cols, kind
    r, c, ld = _mx_rows(out, "out")
    if (r, c) != (rows, cols):
        raise ValueError(f"out must have shape {(rows, cols)}")
    return out, ld, kind


def mxf4_dequantize(codes: torch.Tensor, scales: torch.Tensor, K: int | None = None,
                    out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
                    stream=None) -> torch.Tensor:
    """The values (rows, K) of an MXFP4 operand, as out's dtype, else out_dtype (float32: exact)."""
    rows, K, ld, lds = _mx_operand(codes, scales, K, "the operand")
    out, ldd, kind = _mx_dense_out(out, rows, K, out_dtype, codes.device, stream)
    if rows and K:
        _mx_call(lib.pdgemm_mxf4_dequantize, (rows, K, codes.data_ptr(), ld, scales.data_ptr(), lds, out.data_ptr(),
                                              ldd, kind), (codes, scales, out), stream)
    return out


def gemm_mxf4(A: torch.Tensor, scale_a: torch.Tensor, Bt: torch.Tensor, scale_b: torch.Tensor, K: int | None = None,
              out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32, stream=None,
              cfg: int | None = None) -> torch.Tensor:
    """C = A * B of MXFP4 A (M rows) and Bt (N rows); binary32 sums, C (M, N) float32, float16
    or bfloat16 (out's dtype, else out_dtype).  cfg: an explicit tile configuration."""
    M, Ka, lda, ldsa = _mx_operand(A, scale_a, K, "A")
    N, Kb, ldb, ldsb = _mx_operand(Bt, scale_b, K, "Bt")
    if Ka != Kb:
        raise ValueError("A and Bt disagree on K")
    out, ldc, kind = _mx_dense_out(out, M, N, out_dtype, A.device, stream)
    args = (M, N, Ka, A.data_ptr(), lda, scale_a.data_ptr(), ldsa, Bt.data_ptr(), ldb, scale_b.data_ptr(), ldsb,
            out.data_ptr(), ldc, kind)
    fn, args = (lib.gemm_mxf4, args) if cfg is None else (lib.pdgemm_mxf4_cfg, (cfg,) + args)
    _mx_call(fn, args, (A, scale_a, Bt, scale_b, out), stream)
    return out


def mxf4_num_configs() -> int:
    return lib.pdgemm_mxf4_num_configs()


def mxf4_pick(M: int, N: int, K: int) -> int:
    """The tile configuration gemm_mxf4 takes for a shape."""
    return lib.pdgemm_mxf4_pick(M, N, K)


def gemm_a16_mxf4(A: torch.Tensor, Bt: torch.Tensor, scale_b: torch.Tensor, out: torch.Tensor | None = None,
                  out_dtype: torch.dtype = torch.float32, stream=None, cfg: int | None = None) -> torch.Tensor:
    """C = A * B of float16 or bfloat16 A (M, K), rows of a multiple of 16 bytes, and MXFP4 Bt
    (N rows of K values); binary32 sums, C (M, N) float32, float16 or bfloat16.  cfg: an
    explicit tile configuration."""
    if A.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("gemm_a16_mxf4 takes a float16 or bfloat16 A")
    M, K, lda = _mx_rows(A, "A")
    if M <= 1:
        lda = _round_up(lda, 8)
    N, K, ldb, ldsb = _mx_operand(Bt, scale_b, K, "Bt")
    out, ldc, kind = _mx_dense_out(out, M, N, out_dtype, A.device, stream)
    args = (M, N, K, A.data_ptr(), lda, _MX_TYPES[A.dtype], Bt.data_ptr(), ldb, scale_b.data_ptr(), ldsb,
            out.data_ptr(), ldc, kind)
    fn, args = (lib.gemm_a16_mxf4, args) if cfg is None else (lib.pdgemm_a16_mxf4_cfg, (cfg,) + args)
    _mx_call(fn, args, (A, Bt, scale_b, out), stream)
    return out


def a16_mxf4_num_configs() -> int:
    return lib.pdgemm_a16_mxf4_num_configs()


def a16_mxf4_pick(dtype: torch.dtype, M: int, N: int, K: int) -> int:
    """The tile configuration gemm_a16_mxf4 takes for activations of `dtype` and a shape."""
    return lib.pdgemm_a16_mxf4_pick(_MX_TYPES[dtype], M, N, K)


# ---- norms ----

_I8 = 3


def _like_x(t, x, name: str):
    """The row stride of a tensor of x's shape and type."""
    if not isinstance(t, torch.Tensor) or t.dtype is not x.dtype:
        raise TypeError(f"{name} must be a tensor of x's type")
    shape = t.shape
    if shape != x.shape:
        raise ValueError(f"{name} must have shape {tuple(x.shape)}")
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows (stride(1) == 1)")
    return ld if shape[0] > 1 else shape[1]


def _norm_weight(weight, cols: int) -> int:
    if not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a tensor")
    kind = _mx_type(weight.dtype, "weight")
    if weight.shape != (cols,):
        raise ValueError(f"weight must hold {cols} values")
    if cols > 1 and weight.stride() != (1,):
        raise ValueError("weight must be contiguous")
    return kind


def _new_vector(n, dtype, device, stream):
    if stream is None:
        return torch.empty(n, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=dtype, device=device)


def _rms_norm(x, rows, cols, ldx, weight, eps, residual, sum_out, out, ldo, out_kind, scale, stream):
    kind = _mx_type(x.dtype, "x")
    wkind = _norm_weight(weight, cols)
    tensors = (x, weight, out) if scale is None else (x, weight, out, scale)
    if residual is not None:
        ldr = _like_x(residual, x, "residual")
        if sum_out is None:
            sum_out, lds = _mx_empty(rows, cols, x.dtype, x.device, stream), cols
        else:
            lds = _like_x(sum_out, x, "sum_out")
        add = (residual.data_ptr(), ldr, sum_out.data_ptr(), lds)
        tensors += (residual, sum_out)
    elif sum_out is not None:
        raise ValueError("sum_out holds x + residual: it takes a residual")
    else:
        add = (None, 0, None, 0)
    _mx_call(lib.pdgemm_rms_norm, (rows, cols, x.data_ptr(), ldx, kind, *add, weight.data_ptr(), wkind, eps,
                                   out.data_ptr(), ldo, out_kind, None if scale is None else scale.data_ptr()),
             tensors, stream)
    return sum_out


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
             out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
             sum_out: torch.Tensor | None = None, stream=None):
    """y = h * weight / sqrt(mean(h^2) + eps) over the rows of h = x, or with a residual of h = x + residual
    (rounded to x's type), then (y, h).  x (rows, cols) float32, float16 or bfloat16, at most 32768 columns;
    y has out's dtype, else out_dtype, else x's.  sum_out takes h: it may be residual or x itself; out may be
    x itself too."""
    rows, cols, ldx = _mx_rows(x, "x")
    out, ldo, kind = _mx_dense_out(out, rows, cols, x.dtype if out_dtype is None else out_dtype, x.device, stream)
    h = _rms_norm(x, rows, cols, ldx, weight, eps, residual, sum_out, out, ldo, kind, None, stream)
    return out if h is None else (out, h)


def rms_norm_i8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                out=None, sum_out: torch.Tensor | None = None, stream=None):
    """(q, scale), with a residual (q, scale, h): rms_norm's rows as int8 codes of their largest magnitude over 127,
    and that scale, float32 (rows,): the A and scale_a of gemm_i8_dequant.  A row of zeros takes scale 0, a row that
    holds an infinity or a NaN codes 0 and scale NaN.  out: a (q, scale) pair to write; a new q has rows of a multiple
    of 16 bytes, as the products take them."""
    rows, cols, ldx = _mx_rows(x, "x")
    if out is None:
        ldo = _round_up(cols, 16)
        q = _mx_empty(rows, ldo, torch.int8, x.device, stream)
        if ldo != cols:
            q = q.as_strided((rows, cols), (ldo, 1))
        scale = _new_vector(rows, torch.float32, x.device, stream)
    else:
        q, scale = out
        if not isinstance(q, torch.Tensor) or q.dtype is not torch.int8:
            raise TypeError("out's codes must be an int8 tensor")
        r, c, ldo = _mx_rows(q, "out's codes")
        if (r, c) != (rows, cols):
            raise ValueError(f"out's codes must have shape {(rows, cols)}")
        _scale(scale, rows, "out's scale")
    h = _rms_norm(x, rows, cols, ldx, weight, eps, residual, sum_out, q, ldo, _I8, scale, stream)
    return (q, scale) if h is None else (q, scale, h)


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                      dh: torch.Tensor | None = None, out: torch.Tensor | None = None,
                      dweight: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """(dx, dweight) of y = rms_norm(h) for the gradient dy of y: dx, of h's type, is the gradient of x and of the
    residual alike, with dh, the gradient that h has from elsewhere, added; dweight is float32.  All matrices have
    h's type and shape; out may be dy or dh itself."""
    kind = _mx_type(h.dtype, "h")
    rows, cols, ldh = _mx_rows(h, "h")
    wkind = _norm_weight(weight, cols)
    lddy = _like_x(dy, h, "dy")
    lddh = 0 if dh is None else _like_x(dh, h, "dh")
    if out is None:
        out, lddx = _mx_empty(rows, cols, h.dtype, h.device, stream), cols
    else:
        lddx = _like_x(out, h, "out")
    if dweight is None:
        dweight = _new_vector(cols, torch.float32, h.device, stream)
        dw = dweight.data_ptr()
    else:
        dw = _scale(dweight, cols, "dweight")
    need = lib.pdgemm_rms_norm_backward_workspace_size(rows, cols)
    if workspace is None and need:
        workspace = _mx_empty(1, need, torch.uint8, h.device, stream)
        ws, ws_bytes = workspace.data_ptr(), need
    else:
        ws, ws_bytes = _workspace(workspace, h.device)
    _mx_call(lib.pdgemm_rms_norm_backward,
             (rows, cols, dy.data_ptr(), lddy, h.data_ptr(), ldh, None if dh is None else dh.data_ptr(), lddh, kind,
              weight.data_ptr(), wkind, eps, out.data_ptr(), lddx, dw, ws, ws_bytes),
             (h, dy, weight, out, dweight) + (() if dh is None else (dh,)), stream)
    return out, dweight


# ---- INT4 weights with group scales ----

def _i4_weights(codes: torch.Tensor, scales: torch.Tensor, K: int, group: int, name: str):
    """(rows, ld in values, scale row stride, scale type) of INT4 weights.  The stride of a single row is its
    length, up to the next multiple the library accepts."""
    if not isinstance(codes, torch.Tensor) or codes.dtype is not torch.uint8:
        raise TypeError(f"{name} must be a uint8 tensor of packed 4-bit values")
    if group <= 0 or group % MX_BLOCK:
        raise ValueError("group must be a positive multiple of 32")
    kind = _mx_type(scales.dtype, f"{name}'s scales") if isinstance(scales, torch.Tensor) else None
    if kind is None:
        raise TypeError(f"{name}'s scales must be a tensor")
    rows, width, ld = _mx_rows(codes, name)
    if width != (K + 1) // 2:
        raise ValueError(f"{name} must hold {(K + 1) // 2} bytes per row for K = {K}")
    groups, cols, lds = _mx_rows(scales, f"{name}'s scales")
    if groups != (K + group - 1) // group or cols != rows:
        raise ValueError(f"{name}'s scales must have shape {((K + group - 1) // group, rows)}")
    return rows, 2 * (_round_up(ld, 16) if rows <= 1 else ld), lds, kind


def gemm_a16_i4(A: torch.Tensor, Bt: torch.Tensor, scale_b: torch.Tensor, group: int, out: torch.Tensor | None = None,
                out_dtype: torch.dtype = torch.float32, workspace: torch.Tensor | None = None, stream=None,
                cfg: int | None = None) -> torch.Tensor:
    """C = A * B of float16 or bfloat16 A (M, K), rows of a multiple of 16 bytes, and INT4 weights: Bt (N, ceil(K/2))
    packed bytes as gemm_i4 takes them, and scale_b (ceil(K/group), N), float32, float16 or bfloat16, one scale per
    `group` (a multiple of 32) values of a row.  Binary32 sums, C (M, N) float32, float16 or bfloat16 (out's dtype,
    else out_dtype).  Scales that a checkpoint keeps by row, (N, K/group), are transposed once: scales.t().contiguous().
    workspace: a16_i4_workspace_size bytes, not shared by calls that overlap; allocated where it is needed and omitted.
    cfg: an explicit tile configuration."""
    if A.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("gemm_a16_i4 takes a float16 or bfloat16 A")
    M, K, lda = _mx_rows(A, "A")
    if M <= 1:
        lda = _round_up(lda, 8)
    N, ldb, ldsb, skind = _i4_weights(Bt, scale_b, K, group, "Bt")
    out, ldc, kind = _mx_dense_out(out, M, N, out_dtype, A.device, stream)
    args = (M, N, K, A.data_ptr(), lda, _MX_TYPES[A.dtype], Bt.data_ptr(), ldb, scale_b.data_ptr(), ldsb, skind, group,
            out.data_ptr(), ldc, kind)
    if workspace is not None:
        args += _workspace(workspace, out.device)
    else:
        need = a16_i4_workspace_size(M, N, K, group, cfg) if M > 16 or cfg is not None else 0
        if need:
            workspace = _mx_empty(1, need, torch.uint8, A.device, stream)
            args += (workspace.data_ptr(), need)
        else:
            args += (None, 0)
    fn, args = (lib.gemm_a16_i4, args) if cfg is None else (lib.pdgemm_a16_i4_cfg, (cfg,) + args)
    _mx_call(fn, args, (A, Bt, scale_b, out), stream)
    return out


def a16_i4_workspace_size(M: int, N: int, K: int, group: int, cfg: int | None = None) -> int:
    """Bytes of workspace gemm_a16_i4 needs for a shape (0: none)."""
    if cfg is None:
        return lib.pdgemm_a16_i4_workspace_size(M, N, K, group)
    return lib.pdgemm_a16_i4_cfg_workspace_size(cfg, M, N, K)


def a16_i4_num_configs() -> int:
    return lib.pdgemm_a16_i4_num_configs()


def a16_i4_pick(M: int, N: int, K: int, group: int) -> int:
    """The tile configuration gemm_a16_i4 takes for a shape."""
    return lib.pdgemm_a16_i4_pick(M, N, K, group)


def _moe_pairs(t, rows: int, dtype, name: str) -> int:
    """Columns of a dense (rows, top) tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape ({rows}, top_k)")
    return shape[1]


def moe_route(logits: torch.Tensor, top_k: int, normalize: bool = True, out=None, stream=None):
    """(ids, weights): int32 and float32 (T, top_k), the top_k largest of each row of logits (T, E) in falling order,
    ties to the lower index, and their softmax among themselves, or without normalize among all of the row.  An expert
    at -inf is not taken (id -1, weight 0).  out: a pair of contiguous tensors to write."""
    kind = _mx_type(logits.dtype, "logits")
    T, E, ld = _mx_rows(logits, "logits")
    if out is None:
        ids = _mx_empty(T, top_k, torch.int32, logits.device, stream)
        weights = _mx_empty(T, top_k, torch.float32, logits.device, stream)
    else:
        ids, weights = out
        if _moe_pairs(ids, T, torch.int32, "ids") != top_k or _moe_pairs(weights, T, torch.float32, "weights") != top_k:
            raise ValueError(f"ids and weights must have {top_k} columns")
    _mx_call(lib.pdgemm_moe_route, (T, E, top_k, logits.data_ptr(), ld, kind, 1 if normalize else 0, ids.data_ptr(),
                                    weights.data_ptr()), (logits, ids, weights), stream)
    return ids, weights


def _moe_weights(codes, scales, E: int, N: int, K: int, group: int, name: str):
    """The C call's (codes, ld, expert stride, scales, ld, expert stride) of E experts' weights."""
    if not isinstance(codes, torch.Tensor) or codes.dtype is not torch.uint8:
        raise TypeError(f"{name} must be a uint8 tensor of packed 4-bit values")
    if not isinstance(scales, torch.Tensor):
        raise TypeError(f"{name}'s scales must be a tensor")
    if codes.shape != (E, N, (K + 1) // 2):
        raise ValueError(f"{name} must have shape {(E, N, (K + 1) // 2)}")
    if scales.shape != (E, (K + group - 1) // group, N):
        raise ValueError(f"{name}'s scales must have shape {(E, (K + group - 1) // group, N)}")
    e, ld, step = codes.stride()
    es, lds, steps = scales.stride()
    if (step != 1 and codes.shape[2] > 1) or (steps != 1 and N > 1):
        raise ValueError(f"{name} and its scales must have contiguous rows")
    # strides that nothing is read by may be anything
    if N == 1:
        ld = _round_up(codes.shape[2], 16)
    if E == 1:
        e, es = 0, 0
    if scales.shape[1] == 1:
        lds = N
    return codes.data_ptr(), 2 * ld, 2 * e, scales.data_ptr(), lds, es


_EWORKSPACE = -7   # PDGEMM_EWORKSPACE


def moe_a16_i4_workspace_size(T: int, H: int, I: int, E: int, top_k: int) -> int:
    """Bytes of workspace moe_a16_i4 needs."""
    return lib.pdgemm_moe_a16_i4_wide_workspace_size(T, H, I, E, top_k)


def moe_a16_i4(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13: torch.Tensor, s13: torch.Tensor,
               w2: torch.Tensor, s2: torch.Tensor, group: int, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """A mixture-of-experts layer for a few tokens (T * top_k <= 4096; past 64 tokens its time grows with their square, and
    calls of 64 are faster from some 128 to 256 on): y (T, H), of x's type, with
        y[t] = sum over the slots s of weights[t, s] * W2[e] (silu(Wg[e] x[t]) * (Wu[e] x[t])),  e = ids[t, s].
    x (T, H) float16 or bfloat16, rows of a multiple of 16 bytes; ids int32 and weights float32 (T, top_k), as moe_route
    makes them; INT4 weights of E experts: w13 (E, 2 I, ceil(H/2)), the gate's rows and then the up projection's, w2
    (E, H, ceil(I/2)), and their scales s13 (E, ceil(H/group), 2 I), s2 (E, ceil(I/group), H), both of one type.  An id
    outside 0 .. E - 1 adds nothing.  The gated activations keep binary32's range, to 2^-16 of a value.  workspace:
    moe_a16_i4_workspace_size bytes, not shared by calls that overlap."""
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("moe_a16_i4 takes a float16 or bfloat16 x")
    T, H, ldx = _mx_rows(x, "x")
    if T <= 1:
        ldx = _round_up(ldx, 8)
    top = _moe_pairs(ids, T, torch.int32, "ids")
    if _moe_pairs(weights, T, torch.float32, "weights") != top:
        raise ValueError("ids and weights must have the same shape")
    if group <= 0 or group % MX_BLOCK:
        raise ValueError("group must be a positive multiple of 32")
    if not isinstance(w13, torch.Tensor) or w13.dim() != 3 or w13.shape[1] % 2:
        raise ValueError("w13 must have shape (E, 2 * I, ceil(H / 2))")
    E, I = w13.shape[0], w13.shape[1] // 2
    first = _moe_weights(w13, s13, E, 2 * I, H, group, "w13")
    second = _moe_weights(w2, s2, E, H, I, group, "w2")
    if s13.dtype is not s2.dtype:
        raise TypeError("s13 and s2 must have the same type")
    skind = _mx_type(s13.dtype, "the scales")
    if out is not None and out.dtype is not x.dtype:
        raise TypeError("out must be of x's type")
    out, ldy, kind = _mx_dense_out(out, T, H, x.dtype, x.device, stream)
    need = lib.pdgemm_moe_a16_i4_wide_workspace_size(T, H, I, E, top)
    if workspace is None:
        ws_bytes = max(need, 16)
        workspace = _new_vector(ws_bytes, torch.uint8, x.device, stream)
        ws = workspace.data_ptr()
    else:
        ws, ws_bytes = _workspace(workspace, x.device)
        if ws_bytes < need:   # (the C call takes less, and rounds what it keeps there to x's type)
            raise PdgemmError(_EWORKSPACE)
    _mx_call(lib.pdgemm_moe_a16_i4, (T, H, I, E, top, x.data_ptr(), ldx, kind, ids.data_ptr(), weights.data_ptr(), *first,
                                     *second, skind, group, out.data_ptr(), ldy, ws, ws_bytes),
             (x, ids, weights, w13, s13, w2, s2, out), stream)
    return out


def prepare(prec: str, A: torch.Tensor, Bt: torch.Tensor, out: torch.Tensor, K: int | None = None,
            stream=None, cfg: int | None = None, scales=None, rowb: bool = False,
            workspace: torch.Tensor | None = None, f6cfg: int | None = None):
    """Check and marshal one GEMM once; return a no-argument callable that
    enqueues it again (on the stream current now) through the C ABI.

    For repeated launches of the same operands, e.g. timing loops: the
    callable skips the per-call Python checks, so host time stays far below
    the kernel time even for small shapes.  The tensors must stay alive.
    With scales = (scale_a, scale_b) an INT8 / INT4 GEMM is the dequantizing
    one, and out is float32 or float16.  With rowb, Bt is a row-major B
    (K, N) instead (INT4: packed along N) and N is out's column count.  An
    INT4 GEMM with a workspace runs through the workspace entry points.
    """
    integer_out = (torch.int32,) if scales is None else (torch.float32, torch.float16)
    if prec == "f16":
        if A.dtype != torch.float16 or Bt.dtype != torch.float16 or out.dtype != torch.float32:
            raise TypeError("f16 takes float16 operands and a float32 output")
        K = A.shape[1] if K is None else K
        lda, ldb, p = _row_major_2d(A, "A"), _row_major_2d(Bt, "Bt"), PREC_F16
    elif prec == "i8":
        if A.dtype != torch.int8 or Bt.dtype != torch.int8 or out.dtype not in integer_out:
            raise TypeError("i8 takes int8 operands and an int32 (dequantizing: float) output")
        K = A.shape[1] if K is None else K
        lda, ldb, p = _row_major_2d(A, "A"), _row_major_2d(Bt, "Bt"), PREC_I8
    elif prec == "i4":
        if A.dtype != torch.uint8 or Bt.dtype != torch.uint8 or out.dtype not in integer_out:
            raise TypeError("i4 takes uint8 packed operands and an int32 (dequantizing: float) output")
        K = 2 * A.shape[1] if K is None else K
        lda, ldb, p = 2 * _row_major_2d(A, "A"), 2 * _row_major_2d(Bt, "Bt"), PREC_I4
    else:
        raise ValueError(f"unknown precision {prec!r}")
    per = 2 if prec == "i4" else 1
    N = out.shape[1]
    if rowb:
        if A.shape[1] * per < K or Bt.shape[0] < K or Bt.shape[1] * per < N:
            raise ValueError("operands hold fewer than K values per row of A, K rows of B or N columns")
    elif A.shape[1] * per < K or Bt.shape[1] * per < K:
        raise ValueError("operands hold fewer than K values per row")
    fn, args = _marshal(p, A, Bt, out, K, lda, ldb, stream, cfg, scales, N=N if rowb else None,
                        rowb=rowb, workspace=workspace, f6cfg=f6cfg)
    rc = fn(*args)  # validates the arguments once, and is a first launch
    if rc != 0:
        raise PdgemmError(rc)

    # the callable holds the tensors, so their memory outlives it
    keep = (A, Bt, out) + (tuple(scales) if scales is not None else ()) + (
        (workspace,) if workspace is not None else ())

    def launch():
        rc = fn(*args)
        if rc != 0:
            raise PdgemmError(rc)

    launch.tensors = keep
    return launch
