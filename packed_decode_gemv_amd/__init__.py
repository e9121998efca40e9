"""Thin Python binding of libvbq (packed mixed-bit GEMV for MI355X / gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libvbq.so`` behind the C ABI declared in ``include/vbq.h``.
PyTorch provides device memory and streams. There is no fallback: if the
library is not built, importing this package raises.

The C ABI takes plain pointers, so the sizes, dtypes and layouts of the
tensors are checked here, before anything is launched (a wrong tensor raises
``ValueError``).

Function names follow the C ABI: ``vbq_pack``, ``vbq_gemv``,
``vbq_gemv_batched``, ``vbq_gemv_batched_static``, ``vbq_gemv_levels``,
``vbq_gemv_cell8``, ``vbq_gemm``, ``cell_requant_verify``, ``cell_drift_bound``,
``cell8_encode``, ``cell8_decode``, ``vbq_residual_error``, and for the 4-bit
key/value cache (``Kv4Cache``) ``kv4_append``, ``kv4_read``, ``kv4_attention``.
For several continuations of one prompt: ``kv4_fork``, ``kv4_attention_shared``,
``head_norm_rotary`` (with a ``HeadRotary``) and ``token_logprobs``.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import os
import struct
import typing

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libvbq.so")

GROUP = 64
TILE_ROWS = 32
TILE_GROUPS = 64
MAX_BATCH = 8
MAX_LAUNCH_MATS = 32

STATUS = {0: "ok", 1: "invalid argument", 2: "bad shape", 3: "width not in {1,2,4,8}", 4: "misaligned buffer",
          5: "unsupported size", 6: "layout does not match its buffers", 7: "HIP runtime error"}


class VbqError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)} (status {status})")
        self.status = status


class vbq_matrix(C.Structure):
    _fields_ = [("n_rows", C.c_int32), ("n_cols", C.c_int32), ("n_tiles", C.c_int64), ("n_bytes16", C.c_int64),
                ("tiles", C.c_void_p), ("stream", C.c_void_p)]


class vbq_layout_sizes(C.Structure):
    _fields_ = [("n_tiles", C.c_int64), ("n_records", C.c_int64), ("n_bytes16", C.c_int64),
                ("max_tile_bytes16", C.c_int64), ("code_bits", C.c_int64), ("groups_by_width", C.c_int64 * 4)]


EXPORTS = ("vbq_abi_version", "vbq_status_string", "vbq_pack_query", "vbq_pack", "vbq_matrix_check",
           "vbq_gemv", "vbq_gemv_batched", "vbq_gemv_batched_static", "vbq_gemv_levels", "vbq_gemm",
           "cell_requant_verify", "cell_drift_bound", "vbq_residual_error", "vbq_gemv_cell8", "cell8_encode",
           "cell8_decode", "kv4_page_bytes", "kv4_append", "kv4_read", "kv4_attention_workspace", "kv4_attention",
           "head_norm_rotary", "kv4_fork_workspace", "kv4_fork",
           "kv4_attention_shared_workspace", "kv4_attention_shared", "token_logprobs_workspace", "token_logprobs")


class vbq_kv4(C.Structure):
    _fields_ = [("n_pages", C.c_int64), ("page_tokens", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("reserved", C.c_int32), ("data", C.c_void_p), ("flags", C.c_void_p)]


class vbq_kv4_range(C.Structure):
    _fields_ = [("batch", C.c_int32), ("table_width", C.c_int32), ("total_tokens", C.c_int32),
                ("max_tokens", C.c_int32), ("table", C.c_void_p), ("start", C.c_void_p), ("cu", C.c_void_p)]


class vbq_kv4_attn(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("batch", "table_width", "total_q", "max_q", "max_kv", "n_heads", "dtype",
                                         "causal", "window", "sinks")] + \
               [("scale", C.c_float), ("reserved", C.c_int32)] + \
               [(n, C.c_void_p) for n in ("table", "kv_lens", "cu_q", "q")] + \
               [("q_token_stride", C.c_int64), ("q_head_stride", C.c_int64)] + \
               [(n, C.c_void_p) for n in ("out", "lse", "workspace")] + [("workspace_bytes", C.c_int64)]


class vbq_head_rotary(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("head_dim", "rotary_dim", "axes", "interleaved")] + \
               [("eps", C.c_float), ("reserved", C.c_int32)] + \
               [(n, C.c_void_p) for n in ("inv_freq", "axis", "q_weight", "k_weight")]


class vbq_head_rows(C.Structure):
    _fields_ = [("in_", C.c_void_p), ("out", C.c_void_p)] + \
               [(n, C.c_int64) for n in ("in_token_stride", "in_head_stride", "out_token_stride", "out_head_stride")] + \
               [(n, C.c_int32) for n in ("heads", "in_dtype", "out_dtype", "reserved")]


class vbq_kv4_fork(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("batch_in", "batch_out", "table_width", "reserved")] + \
               [(n, C.c_void_p) for n in ("table_in", "lens_in", "refs_in", "parents", "reserve", "table_out",
                                          "lens_out", "refs_out", "workspace")] + [("workspace_bytes", C.c_int64)]


class vbq_kv4_groups(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_groups", "max_shared", "max_own", "max_group_q")] + \
               [("cu_groups", C.c_void_p), ("shared", C.c_void_p), ("reserved", C.c_int64)]


class vbq_logprobs(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("rows", "vocab", "dtype", "top")] + [("row_stride", C.c_int64)] + \
               [("logits", C.c_void_p), ("tokens", C.c_void_p), ("token_bytes", C.c_int32), ("reserved", C.c_int32)] + \
               [(n, C.c_void_p) for n in ("logprob", "rank", "entropy", "lse", "top_logprob", "top_index",
                                          "workspace")] + [("workspace_bytes", C.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libvbq.so is not built ({LIB_PATH}); run __graft_entry__.build() or "
                          "python packed_decode_gemv_amd/build.py")
    lib = C.CDLL(LIB_PATH)
    P, I32 = C.c_void_p, C.c_int32
    lib.vbq_abi_version.restype = C.c_int
    lib.vbq_abi_version.argtypes = []
    lib.vbq_status_string.restype = C.c_char_p
    lib.vbq_status_string.argtypes = [C.c_int]
    lib.vbq_pack_query.restype = C.c_int
    lib.vbq_pack_query.argtypes = [P, I32, I32, C.POINTER(vbq_layout_sizes)]
    lib.vbq_pack.restype = C.c_int
    lib.vbq_pack.argtypes = [P, P, C.POINTER(vbq_matrix), P]
    lib.vbq_matrix_check.restype = C.c_int
    lib.vbq_matrix_check.argtypes = [C.POINTER(vbq_matrix), P]
    lib.vbq_gemv.restype = C.c_int
    lib.vbq_gemv.argtypes = [C.POINTER(vbq_matrix), P, I32, P, P, P]
    lib.vbq_gemv_batched.restype = C.c_int
    lib.vbq_gemv_batched.argtypes = [I32, C.POINTER(vbq_matrix), C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), I32, P]
    lib.vbq_gemv_batched_static.restype = C.c_int
    lib.vbq_gemv_batched_static.argtypes = [I32, C.POINTER(vbq_matrix), C.POINTER(C.c_void_p),
                                            C.POINTER(C.c_void_p), I32, P]
    lib.vbq_gemv_levels.restype = C.c_int
    lib.vbq_gemv_levels.argtypes = [I32, C.POINTER(vbq_matrix), P, I32, P, P]
    lib.vbq_gemm.restype = C.c_int
    lib.vbq_gemm.argtypes = [C.POINTER(vbq_matrix), P, I32, P, P]
    lib.cell_requant_verify.restype = C.c_int
    lib.cell_requant_verify.argtypes = [C.POINTER(vbq_matrix), P, P, P, P]
    lib.cell_drift_bound.restype = C.c_int
    lib.cell_drift_bound.argtypes = [C.POINTER(vbq_matrix), P, I32, P, P]
    lib.vbq_residual_error.restype = C.c_int
    lib.vbq_residual_error.argtypes = [C.POINTER(vbq_matrix), P, P, P]
    lib.vbq_gemv_cell8.restype = C.c_int
    lib.vbq_gemv_cell8.argtypes = [C.POINTER(vbq_matrix), P, I32, P, P, P]
    lib.cell8_encode.restype = C.c_int
    lib.cell8_encode.argtypes = [C.POINTER(vbq_matrix), P, P, P]
    lib.cell8_decode.restype = C.c_int
    lib.cell8_decode.argtypes = [C.POINTER(vbq_matrix), P, P, P]
    I64 = C.c_int64
    lib.kv4_page_bytes.restype = I64
    lib.kv4_page_bytes.argtypes = [I32, I32, I32]
    lib.kv4_append.restype = C.c_int
    lib.kv4_append.argtypes = [C.POINTER(vbq_kv4), P, P, P, I32, I64, I64, I64, I64, P]
    lib.kv4_read.restype = C.c_int
    lib.kv4_read.argtypes = [C.POINTER(vbq_kv4), P, P, P, I32, P]
    lib.kv4_attention_workspace.restype = I64
    lib.kv4_attention_workspace.argtypes = [C.POINTER(vbq_kv4), P]
    lib.kv4_attention.restype = C.c_int
    lib.kv4_attention.argtypes = [C.POINTER(vbq_kv4), P, P]
    lib.head_norm_rotary.restype = C.c_int
    lib.head_norm_rotary.argtypes = [C.POINTER(vbq_head_rotary), P, P, P, I64, I32, P]
    lib.kv4_fork_workspace.restype = I64
    lib.kv4_fork_workspace.argtypes = [C.POINTER(vbq_kv4), I32, I32, I32]
    lib.kv4_fork.restype = C.c_int
    lib.kv4_fork.argtypes = [C.POINTER(vbq_kv4), P, P]
    lib.kv4_attention_shared_workspace.restype = I64
    lib.kv4_attention_shared_workspace.argtypes = [C.POINTER(vbq_kv4), P, P]
    lib.kv4_attention_shared.restype = C.c_int
    lib.kv4_attention_shared.argtypes = [C.POINTER(vbq_kv4), P, P, P]
    lib.token_logprobs_workspace.restype = I64
    lib.token_logprobs_workspace.argtypes = [I32, I32, I32]
    lib.token_logprobs.restype = C.c_int
    lib.token_logprobs.argtypes = [P, P]
    return lib


lib = _load()


def _check(st: int, what: str):
    if st != 0:
        raise VbqError(st, what)


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _need(t, what: str, dtype, shape, device=None):
    """Raises ValueError unless t is a contiguous tensor of this dtype and
    shape (on `device` when given, else on a GPU)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: not contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    if device is None and t.device.type != "cuda":
        raise ValueError(f"{what}: on {t.device}, expected a GPU tensor")


def _rows2(x):
    return x if x.dim() == 2 else x.view(1, -1)


def abi_version() -> int:
    return lib.vbq_abi_version()


def pack_query(widths) -> vbq_layout_sizes:
    """Host-only sizing of the layout for uint8 widths [N][K/64] (numpy)."""
    w = np.ascontiguousarray(widths, dtype=np.uint8)
    if w.ndim != 2:
        raise ValueError(f"widths: expected [N][K/64], got shape {w.shape}")
    N, G = w.shape
    out = vbq_layout_sizes()
    _check(lib.vbq_pack_query(w.ctypes.data_as(C.c_void_p), N, G * GROUP, C.byref(out)), "vbq_pack_query")
    return out


class PackedMatrix:
    """Device buffers of one packed matrix (owned by torch) and their descriptor."""

    def __init__(self, N: int, K: int, sizes: vbq_layout_sizes, device="cuda"):
        import torch
        self.N, self.K = int(N), int(K)
        self.sizes = sizes
        self.tiles = torch.empty(4 * (sizes.n_tiles + 1), dtype=torch.int32, device=device)
        self.stream = torch.empty(4 * sizes.n_bytes16, dtype=torch.int32, device=device)
        self.desc = vbq_matrix(self.N, self.K, sizes.n_tiles, sizes.n_bytes16,
                               self.tiles.data_ptr(), self.stream.data_ptr())

    @property
    def device(self):
        return self.stream.device

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.tiles, self.stream))

    def clone(self) -> "PackedMatrix":
        """A copy in new device buffers (same layout)."""
        pm = PackedMatrix(self.N, self.K, self.sizes, device=self.tiles.device)
        pm.tiles.copy_(self.tiles)
        pm.stream.copy_(self.stream)
        return pm

    def host_layout(self) -> dict:
        """The layout as numpy arrays (device-to-host copy), in the oracle's format."""
        return dict(tiles=self.tiles.cpu().numpy().view(np.uint32), stream=self.stream.cpu().numpy().view(np.uint32),
                    N=self.N, K=self.K)


def vbq_pack(W, widths, stream=None, check: bool = True) -> PackedMatrix:
    """Quantise W (torch float32 [N][K] on the GPU) with per-group widths
    (numpy or torch uint8 [N][K/64]) into a PackedMatrix."""
    import torch
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise ValueError("W: expected a 2-D torch tensor")
    N, K = W.shape
    _need(W, "W", torch.float32, (N, K))
    widths_np = widths.cpu().numpy() if isinstance(widths, torch.Tensor) else np.asarray(widths)
    widths_np = np.ascontiguousarray(widths_np, dtype=np.uint8)
    if K % GROUP or widths_np.shape != (N, K // GROUP):
        raise ValueError(f"widths: shape {widths_np.shape}, expected {(N, K // GROUP)} for W {tuple(W.shape)}")
    sizes = pack_query(widths_np)
    pm = PackedMatrix(N, K, sizes, device=W.device)
    wd = torch.from_numpy(widths_np).to(W.device)
    st = lib.vbq_pack(_ptr(W), _ptr(wd), C.byref(pm.desc), _stream(stream))
    _check(st, "vbq_pack")
    if check:
        _check(lib.vbq_matrix_check(C.byref(pm.desc), _stream(stream)), "vbq_matrix_check")
    pm._keep = (W, wd)
    return pm


def vbq_gemv(pm: PackedMatrix, x, residual=None, out=None, stream=None):
    """y [B][N] float32 = x [B][K] (fp16) . (dequant(W) + residual)^T."""
    import torch
    x2 = _rows2(x)
    B = x2.shape[0]
    _need(x2, "x", torch.float16, (B, pm.K), pm.device)
    if not 1 <= B <= MAX_BATCH:
        raise ValueError(f"x: batch {B} outside 1..{MAX_BATCH}")
    if residual is not None:
        _need(residual, "residual", torch.float16, (pm.N, pm.K), pm.device)
    if out is None:
        out = torch.empty(B, pm.N, dtype=torch.float32, device=x.device)
    _need(out, "out", torch.float32, (B, pm.N), pm.device)
    st = lib.vbq_gemv(C.byref(pm.desc), _ptr(x2), B, _ptr(residual), _ptr(out), _stream(stream))
    _check(st, "vbq_gemv")
    return out


def vbq_gemv_cell8(pm: PackedMatrix, x, cell, out=None, stream=None):
    """y [B][N] float32 = x [B][K] (fp16) . (dequant(W) + s * cell / 256)^T,
    cell int8 [N][K] (the compact in-cell residual)."""
    import torch
    x2 = _rows2(x)
    B = x2.shape[0]
    _need(x2, "x", torch.float16, (B, pm.K), pm.device)
    if not 1 <= B <= MAX_BATCH:
        raise ValueError(f"x: batch {B} outside 1..{MAX_BATCH}")
    _need(cell, "cell", torch.int8, (pm.N, pm.K), pm.device)
    if out is None:
        out = torch.empty(B, pm.N, dtype=torch.float32, device=x.device)
    _need(out, "out", torch.float32, (B, pm.N), pm.device)
    _check(lib.vbq_gemv_cell8(C.byref(pm.desc), _ptr(x2), B, _ptr(cell), _ptr(out), _stream(stream)),
           "vbq_gemv_cell8")
    return out


def cell8_encode(pm: PackedMatrix, residual, out=None, stream=None):
    """int8 [N][K] fractions f = clamp(rint(r / s * 256), -127, 127) of an fp16
    residual, with the scales of the packed matrix."""
    import torch
    _need(residual, "residual", torch.float16, (pm.N, pm.K), pm.device)
    if out is None:
        out = torch.empty(pm.N, pm.K, dtype=torch.int8, device=residual.device)
    _need(out, "out", torch.int8, (pm.N, pm.K), pm.device)
    _check(lib.cell8_encode(C.byref(pm.desc), _ptr(residual), _ptr(out), _stream(stream)), "cell8_encode")
    return out


def cell8_decode(pm: PackedMatrix, cell, out=None, stream=None):
    """fp16 [N][K] residual fp16(s * f / 256) of int8 fractions f."""
    import torch
    _need(cell, "cell", torch.int8, (pm.N, pm.K), pm.device)
    if out is None:
        out = torch.empty(pm.N, pm.K, dtype=torch.float16, device=cell.device)
    _need(out, "out", torch.float16, (pm.N, pm.K), pm.device)
    _check(lib.cell8_decode(C.byref(pm.desc), _ptr(cell), _ptr(out), _stream(stream)), "cell8_decode")
    return out


class CellUpdate:
    """An in-cell update served beside a frozen packed matrix (CellFill
    abstract: the release's codes and scales stay untouched, and dropping the
    residual revokes the update). Holds the matrix and the update's fraction
    bytes; gemv() calls vbq_gemv_cell8 while the update is applied and
    vbq_gemv (the release) once it is revoked. Nothing in the matrix changes
    either way, so revoke() and apply() can alternate freely."""

    def __init__(self, pm: PackedMatrix, cell):
        import torch
        _need(cell, "cell", torch.int8, (pm.N, pm.K), pm.device)
        self.pm, self.cell, self.applied = pm, cell, True

    @classmethod
    def from_residual(cls, pm: PackedMatrix, residual, stream=None) -> "CellUpdate":
        """Encodes an fp16 residual with the matrix's scales (cell8_encode)."""
        return cls(pm, cell8_encode(pm, residual, stream=stream))

    def revoke(self):
        self.applied = False

    def apply(self):
        self.applied = True

    def gemv(self, x, out=None, stream=None):
        if self.applied:
            return vbq_gemv_cell8(self.pm, x, self.cell, out=out, stream=stream)
        return vbq_gemv(self.pm, x, out=out, stream=stream)

    def residual(self, stream=None):
        """The fp16 residual the fraction bytes stand for (cell8_decode)."""
        return cell8_decode(self.pm, self.cell, stream=stream)

    def verify(self, stream=None):
        """cell_requant_verify of the decoded residual: (mismatches,
        out_of_cell, first_bad_index, None)."""
        return cell_requant_verify(self.pm, self.residual(stream=stream), stream=stream)


def vbq_gemv_batched(pms, xs, ys=None, stream=None, static=False):
    """One launch for several independent GEMVs (same batch size). With
    static=True it calls vbq_gemv_batched_static, which allocates nothing and
    gives every k-tile of a long matrix a workgroup of its own."""
    import torch
    name = "vbq_gemv_batched_static" if static else "vbq_gemv_batched"
    n = len(pms)
    if not 1 <= n <= MAX_LAUNCH_MATS or len(xs) != n or (ys is not None and len(ys) != n):
        raise ValueError(f"{name}: {n} matrices, {len(xs)} inputs (1..{MAX_LAUNCH_MATS} each)")
    x2s = [_rows2(x) for x in xs]
    B = x2s[0].shape[0]
    for pm, x in zip(pms, x2s):
        _need(x, "x", torch.float16, (B, pm.K), pm.device)
    if ys is None:
        ys = [torch.empty(B, pm.N, dtype=torch.float32, device=x.device) for pm, x in zip(pms, x2s)]
    for pm, y in zip(pms, ys):
        _need(y, "y", torch.float32, (B, pm.N), pm.device)
    descs = (vbq_matrix * n)(*[pm.desc for pm in pms])
    xp = (C.c_void_p * n)(*[x.data_ptr() for x in x2s])
    yp = (C.c_void_p * n)(*[y.data_ptr() for y in ys])
    _check(getattr(lib, name)(n, descs, xp, yp, B, _stream(stream)), name)
    return ys


class GemvPlan:
    """Pre-marshalled argument block of vbq_gemv_batched (or, with
    static=True, vbq_gemv_batched_static), for timing loops (the tensors are
    checked once, here)."""

    def __init__(self, pms, xs, ys, static=False):
        import torch
        n = len(pms)
        if not 1 <= n <= MAX_LAUNCH_MATS:
            raise ValueError(f"GemvPlan: {n} matrices (1..{MAX_LAUNCH_MATS})")
        self.n = n
        self.B = xs[0].shape[0]
        for pm, x, y in zip(pms, xs, ys):
            _need(x, "x", torch.float16, (self.B, pm.K), pm.device)
            _need(y, "y", torch.float32, (self.B, pm.N), pm.device)
        self.descs = (vbq_matrix * n)(*[pm.desc for pm in pms])
        self.xp = (C.c_void_p * n)(*[x.data_ptr() for x in xs])
        self.yp = (C.c_void_p * n)(*[y.data_ptr() for y in ys])
        self._keep = (pms, xs, ys)
        self.name = "vbq_gemv_batched_static" if static else "vbq_gemv_batched"
        self._fn = getattr(lib, self.name)

    def launch(self, stream_handle):
        st = self._fn(self.n, self.descs, self.xp, self.yp, self.B, stream_handle)
        if st != 0:
            raise VbqError(st, self.name)


def vbq_gemm(pm: PackedMatrix, x_bf16, out=None, stream=None):
    """y [M][N] float32 = x [M][K] (bf16) . bf16(dequant(W))^T on MFMA."""
    import torch
    if not isinstance(x_bf16, torch.Tensor) or x_bf16.dim() != 2:
        raise ValueError("x: expected a 2-D torch tensor")
    M = x_bf16.shape[0]
    _need(x_bf16, "x", torch.bfloat16, (M, pm.K), pm.device)
    if out is None:
        out = torch.empty(M, pm.N, dtype=torch.float32, device=x_bf16.device)
    _need(out, "out", torch.float32, (M, pm.N), pm.device)
    _check(lib.vbq_gemm(C.byref(pm.desc), _ptr(x_bf16), M, _ptr(out), _stream(stream)), "vbq_gemm")
    return out


def cell_requant_verify(pm: PackedMatrix, residual, requant_codes: bool = False, stream=None):
    """Returns (mismatches, out_of_cell, first_bad_index, re-quantised stream tensor or None)."""
    import torch
    _need(residual, "residual", torch.float16, (pm.N, pm.K), pm.device)
    res = torch.empty(3, dtype=torch.int64, device=residual.device)
    rq = torch.empty_like(pm.stream) if requant_codes else None
    _check(lib.cell_requant_verify(C.byref(pm.desc), _ptr(residual), _ptr(res), _ptr(rq), _stream(stream)),
           "cell_requant_verify")
    r = res.cpu().numpy().view(np.uint64)
    return int(r[0]), int(r[1]), int(r[2]), rq


def cell_drift_bound(pm: PackedMatrix, x, out=None, stream=None):
    """bound [B][N] float32 = 0.5 * sum_g s[n][g] * sum_{k in g} |x[b][k]|: no
    residual inside its cells moves y[b][n] further."""
    import torch
    x2 = _rows2(x)
    B = x2.shape[0]
    _need(x2, "x", torch.float16, (B, pm.K), pm.device)
    if not 1 <= B <= MAX_BATCH:
        raise ValueError(f"x: batch {B} outside 1..{MAX_BATCH}")
    if out is None:
        out = torch.empty(B, pm.N, dtype=torch.float32, device=x.device)
    _need(out, "out", torch.float32, (B, pm.N), pm.device)
    _check(lib.cell_drift_bound(C.byref(pm.desc), _ptr(x2), B, _ptr(out), _stream(stream)), "cell_drift_bound")
    return out


def vbq_residual_error(pm: PackedMatrix, E, out=None, stream=None):
    """E - dequant(W) in binary32 (N x K float32): what the next residual level quantises."""
    import torch
    _need(E, "E", torch.float32, (pm.N, pm.K), pm.device)
    if out is None:
        out = torch.empty_like(E)
    _need(out, "out", torch.float32, (pm.N, pm.K), pm.device)
    _check(lib.vbq_residual_error(C.byref(pm.desc), _ptr(E), _ptr(out), _stream(stream)), "vbq_residual_error")
    return out


def rrq_pack(W, n_levels: int, stream=None):
    """Recurrent residual levels of W: a 2-bit base and n_levels - 1 2-bit
    levels, each packed from the error the levels before it leave."""
    import torch
    _need(W, "W", torch.float32, tuple(W.shape))
    widths = np.full((W.shape[0], W.shape[1] // GROUP), 2, np.uint8)
    E = W
    levels = []
    for i in range(n_levels):
        pm = vbq_pack(E, widths, stream=stream)
        levels.append(pm)
        if i + 1 < n_levels:
            E = vbq_residual_error(pm, E, stream=stream)
    return levels


def vbq_gemv_levels(pms, x, out=None, stream=None):
    """y [B][N] float32 = sum over levels of x . dequant(W_i)^T, one launch."""
    import torch
    n = len(pms)
    if not 1 <= n <= MAX_LAUNCH_MATS:
        raise ValueError(f"vbq_gemv_levels: {n} levels (1..{MAX_LAUNCH_MATS})")
    x2 = _rows2(x)
    B = x2.shape[0]
    _need(x2, "x", torch.float16, (B, pms[0].K), pms[0].device)
    if any((pm.N, pm.K) != (pms[0].N, pms[0].K) for pm in pms):
        raise ValueError("vbq_gemv_levels: levels of different shapes")
    descs = (vbq_matrix * n)(*[pm.desc for pm in pms])
    if out is None:
        out = torch.empty(B, pms[0].N, dtype=torch.float32, device=x.device)
    _need(out, "out", torch.float32, (B, pms[0].N), pms[0].device)
    _check(lib.vbq_gemv_levels(n, descs, _ptr(x2), B, _ptr(out), _stream(stream)), "vbq_gemv_levels")
    return out


# ---- 4-bit key/value cache ---------------------------------------------------------
KV4_FLAG_PAGE, KV4_FLAG_LENGTH, KV4_FLAG_NAN, KV4_FLAG_FULL = 1, 2, 4, 8
KV4_COUNTERS = 2048


_KV4_DTYPES = {}       # torch dtype -> vbq_dtype
_KV4_RANGE = struct.Struct("@4i3P")                     # vbq_kv4_range
_KV4_ATTN = struct.Struct("@10ifi4P2q3Pq")              # vbq_kv4_attn
assert _KV4_RANGE.size == C.sizeof(vbq_kv4_range) and _KV4_ATTN.size == C.sizeof(vbq_kv4_attn)


def _kv4_dtype(dtype, what: str, most: int = 2) -> int:
    if not _KV4_DTYPES:
        import torch
        _KV4_DTYPES.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    dt = _KV4_DTYPES.get(dtype, 3)
    if dt > most:
        raise ValueError(f"{what}: dtype {dtype}, expected one of {', '.join(('float16', 'bfloat16', 'float32')[:most + 1])}")
    return dt


def _kv4_rows(t, what: str, heads: int, cache):
    """Raises ValueError unless t is [tokens][heads][head_dim] on the cache's
    device with contiguous channels and 16-byte aligned rows; returns its
    number of tokens, their stride and the heads'."""
    if getattr(t, "ndim", 0) != 3:
        raise ValueError(f"{what}: expected a torch tensor [tokens][{heads}][{cache.head_dim}]")
    T, H, D = t.shape
    if H != heads or D != cache.head_dim:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected (tokens, {heads}, {cache.head_dim})")
    if t.get_device() != cache.index:
        raise ValueError(f"{what}: on {t.device}, expected {cache.device}")
    ts, hs, cs = t.stride()
    if cs != 1:
        raise ValueError(f"{what}: channels are not contiguous")
    if T < 2:
        ts = 0
    if H < 2:
        hs = 0
    per16 = 16 // t.itemsize
    if ts % per16 or hs % per16 or t.data_ptr() % 16:
        raise ValueError(f"{what}: token and head rows are not 16-byte aligned (strides {t.stride()})")
    return T, ts, hs


def _kv4_stream(cache, stream) -> int:
    return cache._raw_stream(cache.index) if stream is None else stream.cuda_stream


def _kv4_new(cache, shape, dtype, stream):
    """A tensor that belongs to the stream that will fill it."""
    if stream is None:
        return cache.data.new_empty(shape, dtype=dtype)
    import torch
    with torch.cuda.stream(stream):
        return cache.data.new_empty(shape, dtype=dtype)


class Kv4Cache:
    """Device buffers of a 4-bit key/value cache (layout in include/vbq.h):
    n_pages pages of page_tokens tokens, n_kv_heads heads of head_dim
    channels. data: an existing uint8 buffer of nbytes, or None for a new one
    (zeroed)."""

    def __init__(self, n_pages: int, page_tokens: int, n_kv_heads: int, head_dim: int, device="cuda", data=None):
        import torch
        ints = max(page_tokens, n_kv_heads, head_dim) < 2 ** 31 and min(page_tokens, n_kv_heads, head_dim) > 0
        self.page_bytes = lib.kv4_page_bytes(page_tokens, n_kv_heads, head_dim) if ints else 0
        if self.page_bytes == 0 or not 1 <= n_pages < 2 ** 31:
            raise ValueError(f"Kv4Cache: {n_pages} pages of {page_tokens} tokens, {n_kv_heads} heads of {head_dim}: "
                             "pages take a power of two of tokens (32..65536), heads 64, 128, 192 or 256 channels")
        self.n_pages, self.page_tokens = int(n_pages), int(page_tokens)
        self.n_kv_heads, self.head_dim = int(n_kv_heads), int(head_dim)
        if data is None:
            if torch.device(device).type != "cuda":
                raise ValueError(f"Kv4Cache: on {device}, expected a GPU")
            data = torch.zeros(self.nbytes, dtype=torch.uint8, device=device)
        else:
            _need(data, "data", torch.uint8, (self.nbytes,))
        self.data = data
        self.flags = torch.zeros(1, dtype=torch.int32, device=data.device)
        self.desc = vbq_kv4(self.n_pages, self.page_tokens, self.n_kv_heads, self.head_dim, 0, data.data_ptr(),
                            self.flags.data_ptr())
        self._ref = C.byref(self.desc)
        self.index = data.get_device()
        self._i32 = torch.int32
        self._raw_stream = torch._C._cuda_getCurrentRawStream

    @property
    def device(self):
        return self.data.device

    @property
    def nbytes(self) -> int:
        return self.n_pages * self.page_bytes

    def check(self):
        """Waits for the device, all streams of it, and raises VbqError if a call
        so far met a page outside the cache, lengths that do not fit or too few free pages; returns
        True if a NaN was stored as 0, else False. The flags are cleared."""
        import torch
        torch.cuda.synchronize(self.device)
        f = int(self.flags.item())
        if f:
            self.flags.zero_()
            torch.cuda.current_stream(self.device).synchronize()   # or a later call's flag could be cleared with them
        if f & (KV4_FLAG_PAGE | KV4_FLAG_LENGTH | KV4_FLAG_FULL):
            raise VbqError(6, "Kv4Cache: " + " and ".join(
                n for b, n in ((KV4_FLAG_PAGE, "a block-table entry outside the cache"),
                               (KV4_FLAG_LENGTH, "lengths outside the table or the stated maxima"),
                               (KV4_FLAG_FULL, "fewer free pages than a fork needed")) if f & b))
        return bool(f & KV4_FLAG_NAN)


def _kv4_index(cache: Kv4Cache, block_table, vec, cu):
    """Batch and width of the block table, checked with the vectors beside it."""
    if getattr(block_table, "ndim", 0) != 2:
        raise ValueError("block_table: expected a 2-D torch tensor")
    B, W = block_table.shape
    i32, dev = cache._i32, cache.index
    try:
        fine = (block_table.dtype is i32 and vec.dtype is i32 and cu.dtype is i32 and block_table.get_device() == dev and
                vec.get_device() == dev and cu.get_device() == dev and block_table.is_contiguous() and
                vec.is_contiguous() and cu.is_contiguous() and vec.shape == (B,) and cu.shape == (B + 1,))
    except AttributeError:   # not a tensor
        fine = False
    if not fine:
        _need(block_table, "block_table", i32, (B, W), cache.device)
        _need(vec, "lengths", i32, (B,), cache.device)
        _need(cu, "cumulative lengths", i32, (B + 1,), cache.device)
    if B < 1 or W < 1:
        raise ValueError(f"block_table: shape {(B, W)}")
    return B, W


def kv4_append(cache: Kv4Cache, k, v, block_table, start, cu_tokens, max_tokens=None, stream=None):
    """Quantises k and v [tokens][n_kv_heads][head_dim] (fp16, bf16 or fp32;
    token and head rows may be strided) into the cache: sequence b's rows
    cu_tokens[b] .. cu_tokens[b+1] become its tokens start[b], start[b] + 1, ...
    block_table int32 [B][W], start int32 [B], cu_tokens int32 [B+1], all on
    the GPU. max_tokens: no sequence has more rows (default: all of them; the
    launch is sized for it, so a near bound saves time)."""
    B, W = _kv4_index(cache, block_table, start, cu_tokens)
    T, kts, khs = _kv4_rows(k, "k", cache.n_kv_heads, cache)
    Tv, vts, vhs = _kv4_rows(v, "v", cache.n_kv_heads, cache)
    dt = _kv4_dtype(k.dtype, "k")
    if v.dtype is not k.dtype or Tv != T:
        raise ValueError(f"v: {v.dtype} {tuple(v.shape)}, expected k's {k.dtype} {tuple(k.shape)}")
    try:
        r = _KV4_RANGE.pack(B, W, T, T if max_tokens is None else max_tokens, block_table.data_ptr(), start.data_ptr(),
                            cu_tokens.data_ptr())
    except struct.error as e:
        raise ValueError(f"kv4_append: max_tokens {max_tokens}, {T} tokens: {e}") from None
    st = lib.kv4_append(cache._ref, r, k.data_ptr(), v.data_ptr(), dt, kts, khs, vts, vhs, _kv4_stream(cache, stream))
    if st:
        _check(st, "kv4_append")


def kv4_read(cache: Kv4Cache, block_table, start, cu_tokens, total_tokens, dtype, max_tokens=None, out=None,
             stream=None):
    """Reads tokens back as k, v [total_tokens][n_kv_heads][head_dim] of
    `dtype` (fp16, bf16 or fp32), rows as in kv4_append. out: (k, v) tensors
    to fill. Rows of no sequence, and of one whose lengths do not fit (see
    Kv4Cache.check), are not written."""
    B, W = _kv4_index(cache, block_table, start, cu_tokens)
    dt = _kv4_dtype(dtype, "dtype")
    shape = (total_tokens, cache.n_kv_heads, cache.head_dim)
    if out is None:
        k = _kv4_new(cache, shape, dtype, stream)
        v = _kv4_new(cache, shape, dtype, stream)
    else:
        k, v = out
        _need(k, "out k", dtype, shape, cache.device)
        _need(v, "out v", dtype, shape, cache.device)
    try:
        r = _KV4_RANGE.pack(B, W, total_tokens, total_tokens if max_tokens is None else max_tokens,
                            block_table.data_ptr(), start.data_ptr(), cu_tokens.data_ptr())
    except struct.error as e:
        raise ValueError(f"kv4_read: max_tokens {max_tokens}, {total_tokens} tokens: {e}") from None
    st = lib.kv4_read(cache._ref, r, k.data_ptr(), v.data_ptr(), dt, _kv4_stream(cache, stream))
    if st:
        _check(st, "kv4_read")
    return k, v


def kv4_attention_workspace(cache: Kv4Cache, batch: int, total_q: int, n_heads: int, max_q: int, max_kv: int,
                            window: int = 0, sinks: int = 0, stream=None):
    """A workspace for kv4_attention calls of these sizes (or any that need no
    more, of kv4_attention_shared too) that do not overlap in time."""
    import torch
    try:
        a = _KV4_ATTN.pack(batch, 1, total_q, max_q, max_kv, n_heads, 0, 1, window, sinks, 1.0, 0, 0, 0, 0, 0, 0, 0, 0,
                           0, 0, 0)
        n = lib.kv4_attention_workspace(cache._ref, a)
    except struct.error:
        n = -1
    if n < 0:
        raise ValueError(f"kv4_attention: sizes refused (batch {batch}, {total_q} queries, {n_heads} heads over "
                         f"{cache.n_kv_heads}, max_q {max_q}, max_kv {max_kv}, window {window}, sinks {sinks})")
    w = _kv4_new(cache, (n,), cache.data.dtype, stream)
    if n:
        with torch.cuda.stream(stream):
            w[:8 * KV4_COUNTERS].zero_()
    return w


def kv4_attention(cache: Kv4Cache, q, block_table, kv_lens, cu_q, max_q: int, max_kv: int, scale=None,
                  causal: bool = True, window: int = 0, sinks: int = 0, out=None, lse=None, workspace=None,
                  stream=None):
    """Attention of q [queries][n_heads][head_dim] (fp16 or bf16, rows may be
    strided) over the cache. Sequence b holds kv_lens[b] tokens, and its
    queries, rows cu_q[b] .. cu_q[b+1] of q, are its last ones. A query sees the
    tokens up to its own (causal=False: all), with window > 0 only the last
    `window` of them and the first `sinks` of the sequence. n_heads is a
    multiple of the cache's heads. max_q, max_kv: no sequence has more queries
    or tokens. scale: 1/sqrt(head_dim) by default. Returns out, of q's type;
    lse: float32 [queries][n_heads] to fill, or None. Rows of no sequence, and of
    one whose lengths do not fit (see Kv4Cache.check), are not written. workspace:
    from kv4_attention_workspace, for calls that allocate nothing."""
    B, W = _kv4_index(cache, block_table, kv_lens, cu_q)
    H = q.shape[1] if getattr(q, "ndim", 0) == 3 else 0
    if H < 1 or H % cache.n_kv_heads:
        raise ValueError(f"q: shape {tuple(getattr(q, 'shape', ()))}, expected (queries, a multiple of "
                         f"{cache.n_kv_heads}, {cache.head_dim})")
    T, ts, hs = _kv4_rows(q, "q", H, cache)
    D, dtype = cache.head_dim, q.dtype
    dt = _kv4_dtype(dtype, "q", 1)
    if window and not causal:
        raise ValueError("window: needs causal=True")
    if out is None:
        out = _kv4_new(cache, (T, H, D), dtype, stream)
    else:
        _need(out, "out", dtype, (T, H, D), cache.device)
    if lse is not None:
        import torch
        _need(lse, "lse", torch.float32, (T, H), cache.device)
    if workspace is None:
        workspace = kv4_attention_workspace(cache, B, T, H, max_q, max_kv, window, sinks, stream)
    elif getattr(workspace, "dtype", None) is not cache.data.dtype or workspace.get_device() != cache.index or \
            not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor on the cache's device")
    try:
        a = _KV4_ATTN.pack(B, W, T, max_q, max_kv, H, dt, 1 if causal else 0, window, sinks,
                           D ** -0.5 if scale is None else scale, 0, block_table.data_ptr(), kv_lens.data_ptr(),
                           cu_q.data_ptr(), q.data_ptr(), ts, hs, out.data_ptr(), 0 if lse is None else lse.data_ptr(),
                           workspace.data_ptr(), workspace.numel())
    except struct.error as e:
        raise ValueError(f"kv4_attention: max_q {max_q}, max_kv {max_kv}, window {window}, sinks {sinks}: {e}") from None
    st = lib.kv4_attention(cache._ref, a, _kv4_stream(cache, stream))
    if st:
        _check(st, "kv4_attention")
    return out


# ---- several continuations of one prompt ---------------------------------------------
_HEAD_ROWS = struct.Struct("@2P4q4i")                   # vbq_head_rows
_KV4_FORK = struct.Struct("@4i9Pq")                     # vbq_kv4_fork
_KV4_GROUPS = struct.Struct("@4i2Pq")                   # vbq_kv4_groups
_LOGPROBS = struct.Struct("@4iq2P2i7Pq")                # vbq_logprobs
assert _HEAD_ROWS.size == C.sizeof(vbq_head_rows) and _KV4_FORK.size == C.sizeof(vbq_kv4_fork) and \
    _KV4_GROUPS.size == C.sizeof(vbq_kv4_groups) and _LOGPROBS.size == C.sizeof(vbq_logprobs)
LOGPROBS_MAX_TOP, LOGPROBS_COUNTERS = 32, 512
_NO_STREAM = contextlib.nullcontext()


class HeadRotary:
    """What head_norm_rotary needs beside its tensors: inv_freq float32
    [rotary_dim / 2] (radians a position), axis uint8 [rotary_dim / 2] (the row of
    the positions that a pair goes by; None: the only one), interleaved (pairs
    are neighbouring channels, else channel i and i + rotary_dim / 2), and the
    weights float32 [head_dim] of the norms of queries and keys (None: not
    normed). Tensors are kept, not copied; rotary_dim is a multiple of 16."""

    def __init__(self, head_dim: int, inv_freq=None, axis=None, axes: int = 1, interleaved: bool = False, q_weight=None,
                 k_weight=None, eps: float = 1e-6):
        import torch
        if head_dim not in (64, 128, 192, 256):
            raise ValueError(f"HeadRotary: head_dim {head_dim}, expected 64, 128, 192 or 256")
        given = [t for t in (inv_freq, q_weight, k_weight) if t is not None]
        if not given:
            raise ValueError("HeadRotary: neither inv_freq nor weights")
        half = 0 if inv_freq is None else inv_freq.numel()
        if half % 8 or 2 * half > head_dim:
            raise ValueError(f"inv_freq: {half} pairs, expected a multiple of 8, at most {head_dim // 2}")
        if not 1 <= axes <= 255 or (axis is None and axes > 1):
            raise ValueError(f"HeadRotary: {axes} axes{' and no axis of the pairs' if axis is None else ''}")
        if not 0.0 <= eps <= 3e38:
            raise ValueError(f"HeadRotary: eps {eps}")
        self.device = given[0].device
        if inv_freq is not None:
            _need(inv_freq, "inv_freq", torch.float32, (half,), self.device)
        for t, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if t is not None:
                _need(t, what, torch.float32, (head_dim,), self.device)
                if t.data_ptr() % 16:
                    raise ValueError(f"{what}: not 16-byte aligned")
        if axis is not None:
            _need(axis, "axis", torch.uint8, (half,), self.device)
            if half and int(axis.max()) >= axes:
                raise ValueError(f"axis: a row of the positions beyond the {axes}")
        if self.device.type != "cuda":
            raise ValueError(f"HeadRotary: on {self.device}, expected GPU tensors")
        self.head_dim, self.rotary_dim, self.axes = int(head_dim), 2 * half, int(axes)
        self.interleaved, self.eps = bool(interleaved), float(eps)
        self._keep = (inv_freq, axis, q_weight, k_weight)
        self.desc = vbq_head_rotary(self.head_dim, self.rotary_dim, self.axes, int(self.interleaved), self.eps, 0,
                                    *(None if t is None else t.data_ptr() for t in self._keep))
        self._ref = C.byref(self.desc)
        self.index = given[0].get_device()
        self._i32 = torch.int32
        self._raw_stream = torch._C._cuda_getCurrentRawStream


def _int32(*numbers) -> bool:
    """Whether all are numbers that an int32 holds (ctypes would cut off the rest)."""
    return all(-2 ** 31 <= n < 2 ** 31 for n in numbers)


def _current_device() -> int:
    global _current_device
    import torch
    _current_device = torch._C._cuda_getDevice    # (this function the first time only)
    return _current_device()


def _on_device(index: int, call, *args) -> int:
    """call(*args) with the tensors' device as the current one."""
    if _current_device() == index:
        return call(*args)
    import torch
    with torch.cuda.device(index):
        return call(*args)


def _new(t, shape, dtype, stream):
    """A tensor beside t that belongs to the stream that will fill it."""
    if stream is None:
        return t.new_empty(shape, dtype=dtype)
    import torch
    with torch.cuda.stream(stream):
        return t.new_empty(shape, dtype=dtype)


_NO_ROWS = _HEAD_ROWS.pack(0, 0, 0, 0, 0, 0, 0, 0, 0, 0)


def _head_rows(plan, x, what: str, out, dtype, stream):
    """The output for x, its tokens, its type and its vbq_head_rows."""
    dt = _kv4_dtype(getattr(x, "dtype", None), what)
    H = x.shape[1] if getattr(x, "ndim", 0) == 3 else 0
    T, ts, hs = _kv4_rows(x, what, H, plan)
    if out is None:
        D = plan.head_dim
        if dtype is None:
            dtype = x.dtype
        odt = _kv4_dtype(dtype, what + "_out")
        out = x.new_empty((T, H, D), dtype=dtype) if stream is None else _new(x, (T, H, D), dtype, stream)
        ots, ohs = H * D, D
    else:
        odt = _kv4_dtype(getattr(out, "dtype", None), what + "_out")
        if dtype is not None and out.dtype is not dtype:
            raise ValueError(f"{what}_out: {out.dtype}, expected {dtype}")
        To, ots, ohs = _kv4_rows(out, what + "_out", H, plan)
        if To != T:
            raise ValueError(f"{what}_out: {To} tokens, expected {T}")
    return out, T, dt, _HEAD_ROWS.pack(x.data_ptr(), out.data_ptr(), ts, hs, ots, ohs, H, dt, odt, 0)


def head_norm_rotary(plan: HeadRotary, q, k, positions, q_out=None, k_out=None, q_dtype=None, k_dtype=None,
                     stream=None):
    """Norms every head of q and k [tokens][heads][head_dim] (fp16, bf16 or fp32;
    token and head rows may be strided; either may be None) and rotates it by its
    token's positions, int32 [tokens] or [axes][tokens], in one pass. Returns the
    results, of q_dtype and k_dtype (the inputs' type by default). q_out and k_out:
    tensors to fill, the inputs themselves for example; what overlaps otherwise is
    not looked for, and must not."""
    rows_q = rows_k = _NO_ROWS
    T = types = None
    if q is not None:
        q_out, T, types, rows_q = _head_rows(plan, q, "q", q_out, q_dtype, stream)
    else:
        q_out = None
    if k is not None:
        k_out, Tk, dt, rows_k = _head_rows(plan, k, "k", k_out, k_dtype, stream)
        if T is not None and (Tk != T or dt != types):
            raise ValueError(f"k: {k.dtype} with {Tk} tokens, expected q's {q.dtype} with {T}")
        T = Tk
    else:
        k_out = None
        if T is None:
            raise ValueError("head_norm_rotary: neither q nor k")
    if T >= 2 ** 31:
        raise ValueError(f"head_norm_rotary: {T} tokens")
    at = None
    if plan.rotary_dim:
        shape = (T,) if plan.axes == 1 and getattr(positions, "ndim", 1) == 1 else (plan.axes, T)
        if getattr(positions, "dtype", None) is not plan._i32 or positions.shape != shape or \
                not positions.is_contiguous() or positions.get_device() != plan.index:
            _need(positions, "positions", plan._i32, shape, plan.device)
        at = positions.data_ptr()
    st = _on_device(plan.index, lib.head_norm_rotary, plan._ref, rows_q, rows_k, at, T, T, _kv4_stream(plan, stream))
    if st:
        _check(st, "head_norm_rotary")
    return q_out, k_out


def kv4_fork_workspace(cache: Kv4Cache, batch: int, table_width: int, batch_before=None, stream=None):
    """A workspace for kv4_fork calls to `batch` sequences from `batch_before` (default:
    as many) with tables of this width, or less of each, that do not overlap in time."""
    if batch_before is None:
        batch_before = batch
    n = lib.kv4_fork_workspace(cache._ref, batch_before, batch, table_width) if _int32(batch_before, batch, table_width) else -1
    if n < 0:
        raise ValueError(f"kv4_fork: sizes refused ({batch_before} to {batch} sequences, tables of {table_width} entries)")
    return _kv4_new(cache, (n,), cache.data.dtype, stream)


def kv4_fork(cache: Kv4Cache, refs, block_table, lens, parents, reserve=None, out=None, workspace=None, stream=None):
    """Makes sequences go on from others. block_table int32 [B][W] (-1: no page) and
    lens int32 [B] are the sequences before, refs int32 [n_pages] how many entries
    name each page (0: free); parents int32 [B'] says which of them each new
    sequence goes on from (-1: none, it is empty), reserve int32 [B'] (or None) for
    how many further tokens it gets pages. Whole pages are shared, part pages
    copied for all but the first continuation, pages of sequences that nothing
    goes on from are free afterwards. Returns the new block_table [B'][W], lens and
    refs; out: tensors to fill (not the inputs). Kv4Cache.check raises where pages ran
    out. Layers that share one table: a call for each layer's cache with the same
    inputs, out the first one's results. workspace: from kv4_fork_workspace, for calls that allocate nothing."""
    i32, dev = cache._i32, cache.index
    if getattr(block_table, "ndim", 0) != 2 or getattr(parents, "ndim", 0) != 1:
        raise ValueError("block_table, parents: expected a 2-D and a 1-D torch tensor")
    B, W = block_table.shape
    N = parents.shape[0]
    n = cache.n_pages
    try:
        fine = (block_table.dtype is i32 and lens.dtype is i32 and refs.dtype is i32 and parents.dtype is i32 and
                block_table.get_device() == dev and lens.get_device() == dev and refs.get_device() == dev and
                parents.get_device() == dev and block_table.is_contiguous() and lens.is_contiguous() and
                refs.is_contiguous() and parents.is_contiguous() and lens.shape == (B,) and refs.shape == (n,) and
                (reserve is None or (reserve.dtype is i32 and reserve.get_device() == dev and reserve.is_contiguous() and
                                     reserve.shape == (N,))))
    except AttributeError:   # not a tensor
        fine = False
    if not fine:
        for t, what, shape in ((block_table, "block_table", (B, W)), (lens, "lens", (B,)), (refs, "refs", (n,)),
                               (parents, "parents", (N,)), (reserve, "reserve", (N,))):
            if t is not None or what != "reserve":
                _need(t, what, i32, shape, cache.device)
    if min(B, W, N) < 1 or not _int32(B, W, N):
        raise ValueError(f"block_table: shape {(B, W)}, {N} parents")
    if out is None:
        if stream is None:
            out = (refs.new_empty((N, W)), refs.new_empty((N,)), refs.new_empty((n,)))
        else:
            out = tuple(_new(refs, shape, i32, stream) for shape in ((N, W), (N,), (n,)))
    else:
        for t, what, shape in zip(out, ("out block_table", "out lens", "out refs"), ((N, W), (N,), (cache.n_pages,))):
            _need(t, what, i32, shape, cache.device)
    table_out, lens_out, refs_out = out
    if workspace is None:
        workspace = kv4_fork_workspace(cache, N, W, B, stream)
    elif getattr(workspace, "dtype", None) is not cache.data.dtype or workspace.get_device() != dev or \
            not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor on the cache's device")
    f = _KV4_FORK.pack(B, N, W, 0, block_table.data_ptr(), lens.data_ptr(), refs.data_ptr(), parents.data_ptr(),
                       0 if reserve is None else reserve.data_ptr(), table_out.data_ptr(), lens_out.data_ptr(),
                       refs_out.data_ptr(), workspace.data_ptr(), workspace.numel())
    st = _on_device(dev, lib.kv4_fork, cache._ref, f, _kv4_stream(cache, stream))
    if st:
        _check(st, "kv4_fork")
    return table_out, lens_out, refs_out


def kv4_attention_shared_workspace(cache: Kv4Cache, batch: int, groups: int, total_q: int, n_heads: int, max_q: int,
                                   max_shared: int, max_own: int, max_group_q=None, stream=None):
    """A workspace for kv4_attention_shared calls of these sizes (or any that need no
    more, of kv4_attention too) that do not overlap in time."""
    import torch
    try:
        a = _KV4_ATTN.pack(batch, 1, total_q, max_q, 0, n_heads, 0, 1, 0, 0, 1.0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
        g = _KV4_GROUPS.pack(groups, max_shared, max_own, total_q if max_group_q is None else max_group_q, 0, 0, 0)
        n = lib.kv4_attention_shared_workspace(cache._ref, a, g)
    except struct.error:
        n = -1
    if n < 0:
        raise ValueError(f"kv4_attention_shared: sizes refused (batch {batch} in {groups} groups, {total_q} queries, "
                         f"{n_heads} heads over {cache.n_kv_heads}, max_q {max_q}, max_shared {max_shared}, max_own "
                         f"{max_own}, max_group_q {max_group_q})")
    w = _kv4_new(cache, (n,), cache.data.dtype, stream)
    with torch.cuda.stream(stream):
        w[:8 * KV4_COUNTERS].zero_()
    return w


def kv4_attention_shared(cache: Kv4Cache, q, block_table, kv_lens, cu_q, cu_groups, shared, max_q: int, max_shared: int,
                         max_own: int, max_group_q=None, scale=None, causal: bool = True, out=None, lse=None,
                         workspace=None, stream=None):
    """kv4_attention for sequences that have their first tokens in common: group g is
    sequences cu_groups[g] .. cu_groups[g+1] (int32 [groups + 1]), and its first shared[g]
    tokens (int32 [groups]) are read once for all of them, from the pages that the
    block table's row of its first sequence names. Queries stand behind the shared
    tokens. max_shared: no group shares more tokens; max_own: no sequence holds more
    beyond them; max_group_q: no group has more queries in all (default: any number).
    For steps of few queries: where a sequence has 128 rows (queries times query heads of a
    key/value head) or more, kv4_attention takes as long or less.
    The rest is as for kv4_attention, without windows; workspace: from
    kv4_attention_shared_workspace."""
    B, W = _kv4_index(cache, block_table, kv_lens, cu_q)
    if getattr(shared, "ndim", 0) != 1 or shared.shape[0] < 1:
        raise ValueError("shared: expected a 1-D torch tensor, a number for each group")
    n = shared.shape[0]
    i32, dev = cache._i32, cache.index
    try:
        fine = (shared.dtype is i32 and cu_groups.dtype is i32 and shared.get_device() == dev and
                cu_groups.get_device() == dev and shared.is_contiguous() and cu_groups.is_contiguous() and
                cu_groups.shape == (n + 1,))
    except AttributeError:   # not a tensor
        fine = False
    if not fine:
        _need(shared, "shared", i32, (n,), cache.device)
        _need(cu_groups, "cu_groups", i32, (n + 1,), cache.device)
    H = q.shape[1] if getattr(q, "ndim", 0) == 3 else 0
    if H < 1 or H % cache.n_kv_heads:
        raise ValueError(f"q: shape {tuple(getattr(q, 'shape', ()))}, expected (queries, a multiple of "
                         f"{cache.n_kv_heads}, {cache.head_dim})")
    D, dtype = cache.head_dim, getattr(q, "dtype", None)
    dt = _kv4_dtype(dtype, "q", 1)
    T, ts, hs = _kv4_rows(q, "q", H, cache)
    if out is None:
        out = _kv4_new(cache, (T, H, D), dtype, stream)
    else:
        _need(out, "out", dtype, (T, H, D), cache.device)
    if lse is not None:
        import torch
        _need(lse, "lse", torch.float32, (T, H), cache.device)
    if workspace is None:
        workspace = kv4_attention_shared_workspace(cache, B, n, T, H, max_q, max_shared, max_own, max_group_q, stream)
    elif getattr(workspace, "dtype", None) is not cache.data.dtype or workspace.get_device() != dev or \
            not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor on the cache's device")
    try:
        a = _KV4_ATTN.pack(B, W, T, max_q, 0, H, dt, 1 if causal else 0, 0, 0, D ** -0.5 if scale is None else scale, 0,
                           block_table.data_ptr(), kv_lens.data_ptr(), cu_q.data_ptr(), q.data_ptr(), ts, hs,
                           out.data_ptr(), 0 if lse is None else lse.data_ptr(), workspace.data_ptr(),
                           workspace.numel())
        g = _KV4_GROUPS.pack(n, max_shared, max_own, T if max_group_q is None else max_group_q, cu_groups.data_ptr(),
                             shared.data_ptr(), 0)
    except struct.error as e:
        raise ValueError(f"kv4_attention_shared: max_q {max_q}, max_shared {max_shared}, max_own {max_own}, "
                         f"max_group_q {max_group_q}: {e}") from None
    st = _on_device(dev, lib.kv4_attention_shared, cache._ref, a, g, _kv4_stream(cache, stream))
    if st:
        _check(st, "kv4_attention_shared")
    return out


_TOKEN_BYTES = {"torch.int32": 4, "torch.int64": 8}


def _on_stream(stream):
    """The stream as the current one, for what is allocated for it."""
    if stream is None:
        return _NO_STREAM
    import torch
    return torch.cuda.stream(stream)


class TokenLogprobs(typing.NamedTuple):
    """What token_logprobs returns; None for what was not asked for."""
    logprob: object        # float32 [rows], of the given tokens
    rank: object           # int32 [rows], their places in the order of the logits, from 0
    entropy: object        # float32 [rows]
    lse: object            # float32 [rows], log of the sum of exponentials
    top_logprob: object    # float32 [rows][top], of the most likely tokens
    top_index: object      # int32 [rows][top], their numbers


def token_logprobs_workspace(rows: int, vocab: int, top: int = 0, device="cuda", stream=None):
    """A workspace for token_logprobs calls of these sizes (or any that need no
    more) that do not overlap in time."""
    import torch
    n = lib.token_logprobs_workspace(rows, vocab, top) if _int32(rows, vocab, top) else -1
    if n < 0:
        raise ValueError(f"token_logprobs: sizes refused ({rows} rows of {vocab} logits, top {top})")
    with torch.cuda.stream(stream):
        w = torch.empty(n, dtype=torch.uint8, device=device)
        w[:4 * LOGPROBS_COUNTERS].zero_()
    return w


def token_logprobs(logits, tokens=None, top: int = 0, out=None, workspace=None, stream=None) -> TokenLogprobs:
    """Log probabilities of rows of logits [rows][vocab] (fp16, bf16 or fp32; rows may be
    strided): those of `tokens` (int32 or int64 [rows]) with their ranks, the rows'
    entropies and log-sum-exps, and the `top` most likely tokens (at most 32, ties go
    to the lower number). Logits may be -infinity; rows with a NaN or +infinity give
    NaN and -1. out: a TokenLogprobs of tensors to fill. workspace: from
    token_logprobs_workspace, for calls that allocate nothing."""
    if getattr(logits, "ndim", 0) != 2:
        raise ValueError("logits: expected a 2-D torch tensor")
    M, V = logits.shape
    dt = _kv4_dtype(logits.dtype, "logits")
    dev = logits.get_device()
    if dev < 0:
        raise ValueError(f"logits: on {logits.device}, expected a GPU tensor")
    row, step = logits.stride()
    if V > 1 and step != 1:
        raise ValueError("logits: a row is not contiguous")
    if not _int32(M, V):
        raise ValueError(f"logits: shape {(M, V)}")
    size = 0
    if tokens is not None:
        size = _TOKEN_BYTES.get(str(getattr(tokens, "dtype", None)), 0)
        if not size:
            raise ValueError(f"tokens: {getattr(tokens, 'dtype', type(tokens).__name__)}, expected int32 or int64")
        if tokens.shape != (M,) or not tokens.is_contiguous() or tokens.get_device() != dev:
            _need(tokens, "tokens", tokens.dtype, (M,), logits.device)
    if not 0 <= top <= min(LOGPROBS_MAX_TOP, V):
        raise ValueError(f"top: {top}, expected 0..{min(LOGPROBS_MAX_TOP, V)}")
    import torch
    f32, i32 = torch.float32, torch.int32
    if out is None:
        with _on_stream(stream):
            new = logits.new_empty
            # (one tensor for the three)
            entropy, lse, logprob = new((3, M), dtype=f32).unbind(0)
            rank = new((M,), dtype=i32) if size else None
            top_logprob, top_index = (new((M, top), dtype=f32), new((M, top), dtype=i32)) if top else (None, None)
        if not size:
            logprob = None
        out = TokenLogprobs(logprob, rank, entropy, lse, top_logprob, top_index)
    else:
        out = TokenLogprobs(*out)
        logprob, rank, entropy, lse, top_logprob, top_index = out
        for t, what, dtype, shape, want in ((logprob, "logprob", f32, (M,), size), (rank, "rank", i32, (M,), size),
                                            (entropy, "entropy", f32, (M,), entropy is not None),
                                            (lse, "lse", f32, (M,), lse is not None),
                                            (top_logprob, "top_logprob", f32, (M, top), top),
                                            (top_index, "top_index", i32, (M, top), top)):
            if want:
                _need(t, "out " + what, dtype, shape, logits.device)
    if workspace is None:
        workspace = token_logprobs_workspace(M, V, top, logits.device, stream)
    elif getattr(workspace, "dtype", None) is not torch.uint8 or workspace.get_device() != dev or \
            not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor on the logits' device")
    a = _LOGPROBS.pack(M, V, dt, top, row if M > 1 else V, logits.data_ptr(), tokens.data_ptr() if size else 0, size, 0,
                       logprob.data_ptr() if size else 0, rank.data_ptr() if size else 0,
                       0 if entropy is None else entropy.data_ptr(), 0 if lse is None else lse.data_ptr(),
                       top_logprob.data_ptr() if top else 0, top_index.data_ptr() if top else 0,
                       workspace.data_ptr(), workspace.numel())
    st = _on_device(dev, lib.token_logprobs, a,
                    torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check(st, "token_logprobs")
    return out
