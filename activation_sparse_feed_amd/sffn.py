"""Python binding of libsffn.so: argument marshalling only.

Every function takes torch tensors that live on the GPU, checks their dtype,
shape and contiguity, and passes raw device pointers plus the current HIP
stream to the C entry point of the same name.  All arithmetic happens in the
library's kernels; there is no fallback: if the library is missing, importing
this module raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsffn.so")

SFFN_OK, SFFN_ERR_ARG, SFFN_ERR_UNSUPPORTED, SFFN_ERR_WORKSPACE, SFFN_ERR_HIP = 0, -1, -2, -3, -4
SFFN_ERR_TOO_LARGE = -5
SFFN_F32, SFFN_BF16 = 0, 1
WS_HYBRID, WS_DENSE, WS_SPARSE, WS_PACK, WS_CONVERT, WS_PACK_L1, WS_BACKWARD = 0, 1, 2, 3, 4, 5, 6
TILE = 128

EXPORTED = ("twell_weight_norms", "twell_pack", "twell_pack_noalloc",
            "twell_pack_noalloc_max_bytes", "twell_pack_l1", "sparse_ffn_fwd", "sparse_ffn_fwd_union",
            "hybrid_route",
            "dense_ffn_ref", "sparse_ffn_bwd", "gate_preact", "twell_from_preact",
            "ell_from_preact", "sffn_probe_hbm", "sffn_probe_mfma", "sffn_probe_mfma_step",
            "sffn_probe_cached", "sffn_probe_gather", "sffn_probe_bf16_round",
            "sffn_workspace_bytes", "sparse_ffn_bwd_workspace_bytes", "sffn_strerror",
            "qk_norm_rope", "qk_norm_rope_bwd", "qk_norm_rope_bwd_workspace_bytes",
            "paged_kv_append", "paged_attn_fwd", "paged_attn_workspace_bytes",
            "paged_kv_append_mx4", "paged_kv_read_mx4", "paged_attn_mx4_fwd",
            "paged_attn_mx4_workspace_bytes")


class SffnError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: status {status} ({msg})")
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("tile", ctypes.c_int32), ("cap", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Heads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "n_q_heads", "n_kv_heads", "head_dim", "rot_dim", "rot_adjacent", "max_pos",
                 "norm")] + [("eps", ctypes.c_float), ("dtype", ctypes.c_int32)]


class PagedBatch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "n_seqs", "n_q_heads", "n_kv_heads", "head_dim", "page_size", "n_pages",
                 "max_pages", "max_q", "max_kv", "causal", "window")] + \
               [("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class Mx4Rows(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)] + \
               [(n, ctypes.c_int64) for n in ("page", "token", "head", "scale_page", "scale_token",
                                              "scale_head")]


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m activation_sparse_feed_amd.build` (hipcc, gfx950)")
    lib = ctypes.CDLL(path)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    sp = ctypes.POINTER(Shape)
    lib.twell_weight_norms.argtypes = [sp, vp, vp, vp]
    lib.twell_pack.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.twell_pack_noalloc.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.twell_pack_noalloc_max_bytes.argtypes = []
    lib.twell_pack_noalloc_max_bytes.restype = sz
    lib.twell_pack_l1.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, sz, vp]
    lib.sparse_ffn_fwd.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.sparse_ffn_fwd_union.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.hybrid_route.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.dense_ffn_ref.argtypes = [sp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.gate_preact.argtypes = [sp, vp, vp, vp, vp, vp]
    lib.sparse_ffn_bwd.argtypes = [sp] + [vp] * 11 + [i32, vp, ctypes.c_float] + [vp] * 5 + [vp, sz, vp]
    lib.sparse_ffn_bwd_workspace_bytes.argtypes = [sp, i32]
    lib.sparse_ffn_bwd_workspace_bytes.restype = sz
    lib.sffn_probe_hbm.argtypes = [vp, vp, sz, i32, vp]
    lib.sffn_probe_mfma.argtypes = [vp, i32, i32, vp]
    lib.sffn_probe_mfma_step.argtypes = [vp, vp, vp, vp, i32, vp]
    lib.sffn_probe_cached.argtypes = [vp, sz, i32, i32, vp]
    lib.sffn_probe_gather.argtypes = [vp, vp, vp, i32, i32, vp]
    lib.sffn_probe_bf16_round.argtypes = [vp, vp, sz, vp]
    lib.twell_from_preact.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.ell_from_preact.argtypes = [sp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    for fn in ("twell_weight_norms", "twell_pack", "twell_pack_noalloc", "twell_pack_l1",
               "sparse_ffn_fwd", "sparse_ffn_fwd_union", "hybrid_route", "dense_ffn_ref", "sparse_ffn_bwd", "gate_preact", "twell_from_preact",
               "ell_from_preact", "sffn_probe_hbm", "sffn_probe_mfma", "sffn_probe_mfma_step",
               "sffn_probe_cached", "sffn_probe_gather", "sffn_probe_bf16_round"):
        getattr(lib, fn).restype = i32
    hp, bp, i64 = ctypes.POINTER(Heads), ctypes.POINTER(PagedBatch), ctypes.c_int64
    rows, cache = [vp, i64, i64], [vp, i64, i64, i64]
    lib.qk_norm_rope.argtypes = [hp] + rows * 2 + [vp] * 4 + rows * 2 + [vp]
    lib.qk_norm_rope_bwd.argtypes = [hp] + rows * 2 + [vp] * 4 + rows * 4 + [vp] * 3 + [sz, vp]
    lib.paged_kv_append.argtypes = [hp] + rows * 3 + [vp] * 5 + rows + cache * 2 + [i32, i32, vp]
    lib.paged_attn_fwd.argtypes = [bp] + rows + cache * 2 + [vp] * 3 + rows + [vp, vp, sz, vp]
    mp = ctypes.POINTER(Mx4Rows)
    lib.paged_kv_append_mx4.argtypes = [hp] + rows * 3 + [vp] * 5 + rows + [mp, mp, i32, i32, vp]
    lib.paged_kv_read_mx4.argtypes = [i32] * 4 + [mp, mp, i32, i32, vp] + rows * 2 + [vp]
    lib.paged_attn_mx4_fwd.argtypes = [bp] + rows + [mp, mp] + [vp] * 3 + rows + [vp, vp, sz, vp]
    lib.paged_attn_mx4_workspace_bytes.argtypes = [bp]
    lib.paged_attn_mx4_workspace_bytes.restype = sz
    for fn in ("qk_norm_rope", "qk_norm_rope_bwd", "paged_kv_append", "paged_attn_fwd",
               "paged_kv_append_mx4", "paged_kv_read_mx4", "paged_attn_mx4_fwd"):
        getattr(lib, fn).restype = i32
    lib.qk_norm_rope_bwd_workspace_bytes.argtypes = [hp]
    lib.qk_norm_rope_bwd_workspace_bytes.restype = sz
    lib.paged_attn_workspace_bytes.argtypes = [bp]
    lib.paged_attn_workspace_bytes.restype = sz
    lib.sffn_workspace_bytes.argtypes = [sp, i32]
    lib.sffn_workspace_bytes.restype = sz
    lib.sffn_strerror.argtypes = [i32]
    lib.sffn_strerror.restype = ctypes.c_char_p
    return lib


_lib = load_library()


def strerror(status: int) -> str:
    return _lib.sffn_strerror(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != SFFN_OK:
        raise SffnError(fn, status, strerror(status))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SFFN_BF16
    if t.dtype == torch.float32:
        return SFFN_F32
    raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def make_shape(T: int, d_model: int, d_ff: int, cap: int, dtype: int, tile: int = TILE) -> Shape:
    return Shape(int(T), int(d_model), int(d_ff), int(tile), int(cap), int(dtype))


def shape_of(x: torch.Tensor, w: torch.Tensor, cap: int) -> Shape:
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be [T, d_model] and weights [d_ff, d_model]")
    if x.dtype != w.dtype:
        raise TypeError("x and the weights must share a dtype")
    return make_shape(x.shape[0], x.shape[1], w.shape[0], cap, _dtype_code(x))


def workspace_bytes(shape: Shape, which: int) -> int:
    return int(_lib.sffn_workspace_bytes(ctypes.byref(shape), int(which)))


def alloc_workspace(shape: Shape, which: int, device=None) -> torch.Tensor:
    """Device workspace for one call kind (no call needs initial contents; it
    is zero-filled only so that its bytes are defined)."""
    n = workspace_bytes(shape, which)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def alloc_twell(shape: Shape, device=None):
    """count [T, n_tiles] u16, idx [T, n_tiles, cap] u16, val [T, n_tiles, cap] dtype."""
    nt = shape.d_ff // shape.tile
    dt = torch.bfloat16 if shape.dtype == SFFN_BF16 else torch.float32
    dev = device or "cuda"
    count = torch.empty((shape.T, nt), dtype=torch.uint16, device=dev)
    idx = torch.empty((shape.T, nt, max(shape.cap, 1)), dtype=torch.uint16, device=dev)
    val = torch.empty((shape.T, nt, max(shape.cap, 1)), dtype=dt, device=dev)
    return count, idx, val


def twell_weight_norms(shape: Shape, wg_t, wg_norms, stream=None) -> None:
    _check("twell_weight_norms", _lib.twell_weight_norms(ctypes.byref(shape), _ptr(wg_t),
                                                         _ptr(wg_norms), _stream(stream)))


def twell_pack(shape: Shape, x, wg_t, b_g, count, idx, val, workspace, wg_norms=None,
               stream=None) -> None:
    ws_n = workspace.numel() * workspace.element_size()
    _check("twell_pack", _lib.twell_pack(ctypes.byref(shape), _ptr(x), _ptr(wg_t), _ptr(b_g),
                                         _ptr(wg_norms), _ptr(count), _ptr(idx), _ptr(val),
                                         _ptr(workspace), ws_n, _stream(stream)))


def twell_pack_noalloc(shape: Shape, x, wg_t, b_g, count, idx, val, wg_norms=None,
                       stream=None) -> None:
    _check("twell_pack_noalloc", _lib.twell_pack_noalloc(
        ctypes.byref(shape), _ptr(x), _ptr(wg_t), _ptr(b_g), _ptr(wg_norms), _ptr(count),
        _ptr(idx), _ptr(val), _stream(stream)))


def twell_pack_noalloc_max_bytes() -> int:
    return int(_lib.twell_pack_noalloc_max_bytes())


def twell_pack_l1(shape: Shape, x, wg_t, b_g, count, idx, val, lam: float, l1_value, workspace,
                  wg_norms=None, stream=None) -> None:
    if l1_value.dtype != torch.float32 or l1_value.numel() < 1:
        raise ValueError("l1_value must be a float32 device tensor with one element")
    ws_n = workspace.numel() * workspace.element_size()
    _check("twell_pack_l1", _lib.twell_pack_l1(
        ctypes.byref(shape), _ptr(x), _ptr(wg_t), _ptr(b_g), _ptr(wg_norms), _ptr(count),
        _ptr(idx), _ptr(val), float(lam), _ptr(l1_value), _ptr(workspace), ws_n, _stream(stream)))


def sparse_ffn_fwd(shape: Shape, x, wu_t, wd, count, idx, val, y, workspace=None,
                   stream=None) -> None:
    ws_n = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("sparse_ffn_fwd", _lib.sparse_ffn_fwd(
        ctypes.byref(shape), _ptr(x), _ptr(wu_t), _ptr(wd), _ptr(count), _ptr(idx), _ptr(val),
        _ptr(y), _ptr(workspace), ws_n, _stream(stream)))


def sparse_ffn_fwd_union(shape: Shape, x, wu_t, wd, count, idx, val, y, stream=None) -> None:
    _check("sparse_ffn_fwd_union", _lib.sparse_ffn_fwd_union(
        ctypes.byref(shape), _ptr(x), _ptr(wu_t), _ptr(wd), _ptr(count), _ptr(idx), _ptr(val),
        _ptr(y), _stream(stream)))


def hybrid_route(shape: Shape, x, wg_t, b_g, wu_t, wd, count, routed, n_routed, workspace, y,
                 stream=None) -> None:
    ws_n = workspace.numel() * workspace.element_size()
    _check("hybrid_route", _lib.hybrid_route(
        ctypes.byref(shape), _ptr(x), _ptr(wg_t), _ptr(b_g), _ptr(wu_t), _ptr(wd), _ptr(count),
        _ptr(routed), _ptr(n_routed), _ptr(workspace), ws_n, _ptr(y), _stream(stream)))


def probe_hbm(src, dst=None, workgroups: int = 4096, stream=None) -> None:
    """One streaming pass over src (copied to dst, or only read when dst is None)."""
    n = src.numel() * src.element_size()
    _check("sffn_probe_hbm", _lib.sffn_probe_hbm(_ptr(src), _ptr(dst), n, int(workgroups),
                                                 _stream(stream)))


def probe_mfma(out, iters: int, stream=None) -> None:
    """out: float32 with a multiple of 256 elements (one workgroup per 256)."""
    wgs = out.numel() // 256
    _check("sffn_probe_mfma", _lib.sffn_probe_mfma(_ptr(out), int(wgs), int(iters),
                                                   _stream(stream)))


def probe_cached(src, window_bytes: int, reps: int, workgroups: int, stream=None) -> None:
    """Every workgroup reads src[0:window_bytes] reps times (cached-load rate)."""
    if window_bytes > src.numel() * src.element_size():
        raise ValueError("window larger than the buffer")
    _check("sffn_probe_cached", _lib.sffn_probe_cached(_ptr(src), int(window_bytes), int(reps),
                                                       int(workgroups), _stream(stream)))


def probe_bf16_round(x, out, stream=None) -> None:
    """out = the library's float32 -> bfloat16 rounding of x (uint16 bits)."""
    if x.dtype != torch.float32 or out.dtype not in (torch.int16, torch.uint16):
        raise TypeError("x must be float32 and out 16-bit integer")
    if out.numel() < x.numel():
        raise ValueError("out too small")
    _check("sffn_probe_bf16_round", _lib.sffn_probe_bf16_round(_ptr(x), _ptr(out), int(x.numel()),
                                                               _stream(stream)))


def probe_gather(a, b, rows, row_bytes: int, max_row=None, stream=None) -> None:
    """Read rows[i] of a and of b (row_bytes per row) for every listed row.
    max_row: the largest entry of rows when the caller knows it (then rows is
    not read back from the device here, e.g. inside a timed region)."""
    if rows.dtype != torch.int32:
        raise TypeError("rows must be int32")
    n_a = a.numel() * a.element_size() // row_bytes
    n_b = b.numel() * b.element_size() // row_bytes
    top = (int(rows.max().item()) if rows.numel() else -1) if max_row is None else int(max_row)
    if top >= min(n_a, n_b):
        raise ValueError("row index beyond the matrices")
    _check("sffn_probe_gather", _lib.sffn_probe_gather(_ptr(a), _ptr(b), _ptr(rows),
                                                       int(rows.numel()), int(row_bytes),
                                                       _stream(stream)))


def probe_mfma_step(a, b, c, d, stream=None) -> None:
    """a, b: uint16/int16 [waves, 64, 8] operand registers; c, d: float32
    [waves, 64, 4] accumulators in and out (one MFMA per wave)."""
    waves = d.numel() // 256
    if a.numel() != waves * 512 or b.numel() != waves * 512 or c.numel() != waves * 256 \
            or d.numel() != waves * 256 or waves <= 0:
        raise ValueError("a, b: [waves, 64, 8]; c, d: [waves, 64, 4]")
    if c.dtype != torch.float32 or d.dtype != torch.float32:
        raise TypeError("c and d must be float32")
    _check("sffn_probe_mfma_step", _lib.sffn_probe_mfma_step(_ptr(a), _ptr(b), _ptr(c), _ptr(d),
                                                             int(waves), _stream(stream)))


def dense_ffn_ref(shape: Shape, x, wg_t, b_g, wu_t, wd, workspace, y, stream=None) -> None:
    ws_n = workspace.numel() * workspace.element_size()
    _check("dense_ffn_ref", _lib.dense_ffn_ref(
        ctypes.byref(shape), _ptr(x), _ptr(wg_t), _ptr(b_g), _ptr(wu_t), _ptr(wd),
        _ptr(workspace), ws_n, _ptr(y), _stream(stream)))


def backward_workspace_bytes(shape: Shape, max_routed: int) -> int:
    return int(_lib.sparse_ffn_bwd_workspace_bytes(ctypes.byref(shape), int(max_routed)))


def sparse_ffn_bwd(shape: Shape, x, wg_t, b_g, wu_t, wd, count, idx, val, routed, n_routed, gy,
                   gx, gwg_t, gwu_t, gwd, gb, workspace, wg_norms=None, l1_lambda: float = 0.0,
                   max_routed=None, stream=None) -> None:
    """max_routed: routed rows the workspace holds (default T, the workspace of
    alloc_workspace(shape, WS_BACKWARD)); see backward_workspace_bytes."""
    mr = shape.T if max_routed is None else int(max_routed)
    for name, t in (("gwg_t", gwg_t), ("gwu_t", gwu_t), ("gwd", gwd)):
        if t.dtype != torch.float32 or tuple(t.shape) != (shape.d_ff, shape.d_model):
            raise ValueError(f"{name} must be float32 [d_ff, d_model]")
    if gb is not None and (gb.dtype != torch.float32 or gb.numel() != shape.d_ff):
        raise ValueError("gb must be float32 [d_ff]")
    ws_n = workspace.numel() * workspace.element_size()
    _check("sparse_ffn_bwd", _lib.sparse_ffn_bwd(
        ctypes.byref(shape), _ptr(x), _ptr(wg_t), _ptr(b_g), _ptr(wu_t), _ptr(wd), _ptr(wg_norms),
        _ptr(count), _ptr(idx), _ptr(val), _ptr(routed), _ptr(n_routed), mr, _ptr(gy),
        float(l1_lambda), _ptr(gx), _ptr(gwg_t), _ptr(gwu_t), _ptr(gwd), _ptr(gb), _ptr(workspace),
        ws_n, _stream(stream)))


def gate_preact(shape: Shape, x, wg_t, b_g, z, stream=None) -> None:
    if z.dtype != torch.float32 or tuple(z.shape) != (shape.T, shape.d_ff):
        raise ValueError("z must be float32 [T, d_ff]")
    _check("gate_preact", _lib.gate_preact(ctypes.byref(shape), _ptr(x), _ptr(wg_t), _ptr(b_g),
                                           _ptr(z), _stream(stream)))


def twell_from_preact(shape: Shape, z, x, wg_t, b_g, count, idx, val, workspace, wg_norms=None,
                      stream=None) -> None:
    ws_n = workspace.numel() * workspace.element_size()
    _check("twell_from_preact", _lib.twell_from_preact(
        ctypes.byref(shape), _ptr(z), _ptr(x), _ptr(wg_t), _ptr(b_g), _ptr(wg_norms), _ptr(count),
        _ptr(idx), _ptr(val), _ptr(workspace), ws_n, _stream(stream)))


def alloc_ell(shape: Shape, width: int, device=None):
    """Row-wise ELLPACK buffers: count [T] u16, idx [T, width] u16, val [T, width] bf16."""
    dev = device or "cuda"
    count = torch.empty(shape.T, dtype=torch.uint16, device=dev)
    idx = torch.empty((shape.T, max(width, 1)), dtype=torch.uint16, device=dev)
    val = torch.empty((shape.T, max(width, 1)), dtype=torch.bfloat16, device=dev)
    return count, idx, val


def ell_from_preact(shape: Shape, width: int, z, x, wg_t, b_g, count, idx, val, workspace,
                    wg_norms=None, stream=None) -> None:
    ws_n = workspace.numel() * workspace.element_size()
    _check("ell_from_preact", _lib.ell_from_preact(
        ctypes.byref(shape), int(width), _ptr(z), _ptr(x), _ptr(wg_t), _ptr(b_g), _ptr(wg_norms),
        _ptr(count), _ptr(idx), _ptr(val), _ptr(workspace), ws_n, _stream(stream)))


# ------------------------------------------------ the attention side of the block
def _code(dtype) -> int:
    if dtype is torch.bfloat16 or dtype == SFFN_BF16:
        return SFFN_BF16
    if dtype is torch.float32 or dtype == SFFN_F32:
        return SFFN_F32
    raise TypeError(f"unsupported dtype {dtype}: float32 or bfloat16")


_TORCH_DTYPE = {SFFN_F32: torch.float32, SFFN_BF16: torch.bfloat16}


def make_heads(T: int, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype, rot_dim: int = 0,
               max_pos: int = 0, norm: bool = False, eps: float = 1e-6,
               adjacent: bool = False) -> Heads:
    """Heads of q and k with their norm and rotation.  dtype: torch.float32 or
    torch.bfloat16 (or the library's code); adjacent: pairs (2i, 2i+1) instead of
    (i, i + rot_dim/2)."""
    return Heads(int(T), int(n_q_heads), int(n_kv_heads), int(head_dim), int(rot_dim),
                 int(bool(adjacent)), int(max_pos), int(bool(norm)), float(eps), _code(dtype))


def make_paged_batch(T: int, n_seqs: int, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype,
                     page_size: int, n_pages: int, max_pages: int, max_q: int, max_kv: int,
                     causal: bool = True, window: int = 0, scale: float | None = None) -> PagedBatch:
    """A batch of sequences over a paged cache.  max_q, max_kv: upper bounds of
    one sequence's new tokens and length; scale: default 1 / sqrt(head_dim)."""
    return PagedBatch(int(T), int(n_seqs), int(n_q_heads), int(n_kv_heads), int(head_dim),
                      int(page_size), int(n_pages), int(max_pages), int(max_q), int(max_kv),
                      int(bool(causal)), int(window),
                      float(head_dim) ** -0.5 if scale is None else float(scale), _code(dtype))


def rotary_table(max_pos: int, rot_dim: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """cos and sin of p * theta^(-2i/rot_dim) for every position p, float32
    [max_pos, rot_dim]: the rot_dim / 2 cosines of a position, then the sines."""
    freq = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / max(rot_dim, 1))
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq[None, :]
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous().to(device)


def _rows(name: str, t, T: int, heads: int, dim: int, dtype):
    """Pointer, token stride and head stride of a [T, heads, dim] view."""
    if t is None or heads == 0:
        return None, 0, 0
    if t.shape != (T, heads, dim):
        raise ValueError(f"{name} must be [{T}, {heads}, {dim}], not {list(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError(f"{name}: head_dim must be contiguous")
    return t.data_ptr(), s0, s1


def _cache(name: str, t, n_pages: int, page_size: int, heads: int, dim: int, dtype):
    """Pointer and page, token and head strides of a paged cache."""
    if t.shape != (n_pages, page_size, heads, dim):
        raise ValueError(f"{name} must be [{n_pages}, {page_size}, {heads}, {dim}], "
                         f"not {list(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 and dim > 1:
        raise ValueError(f"{name}: head_dim must be contiguous")
    return t.data_ptr(), s0, s1, s2


def _array(name: str, t, n: int, dtype, exact: bool = False):
    """Pointer of a contiguous array of at least n elements (None: absent), exact: of n, as
    one row of norm weights for all heads."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    size = t.numel()
    if size < n or (exact and size > n):
        raise ValueError(f"{name} must have {n} elements, not {size}")
    return _pointer(t)


def _table(name: str, t, rows: int, cols: int, dtype):
    """The same of a table [rows or more, cols], or flat: the kernels step over rows of
    cols elements."""
    if t is None:
        return None
    if t.shape != (rows, cols):
        if t.dim() == 2 and t.shape[1] != cols:
            raise ValueError(f"{name} must have {cols} columns, not {t.shape[1]}")
        return _array(name, t, rows * cols, dtype)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    return _pointer(t)


def _pointer(t):
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _rotation(h: Heads, q_weight, k_weight, table, positions, dt):
    if h.rot_dim and table is not None and table.dim() == 2 and table.shape[1] != h.rot_dim:
        raise ValueError(f"the rotation table must be [max_pos, {h.rot_dim}]")
    return (_array("q_weight", q_weight, h.head_dim, dt, True),
            _array("k_weight", k_weight, h.head_dim, dt, True),
            _array("the rotation table", table, h.max_pos * h.rot_dim, torch.float32),
            _array("positions", positions, h.T, torch.int32))


def _stream_ptr(stream, t) -> int:
    """The stream given, or the current one of the current device, on which a call's
    tensors (t: one of them) must lie: its kernels would run beside their memory."""
    if stream is not None:
        return stream.cuda_stream
    # torch.cuda.current_stream().cuda_stream without building a Stream object,
    # which alone costs 2.5 us of the host's time for a small step
    device = torch._C._cuda_getDevice()
    if t is not None and t.get_device() != device:
        raise ValueError(f"tensors are on GPU {t.get_device()}, the current device is {device}")
    return torch._C._cuda_getCurrentRawStream(device)


def qk_norm_rope(heads: Heads, q, k, q_weight, k_weight, table, positions, q_out, k_out,
                 stream=None) -> None:
    """q_out, k_out = the heads of q and k, normalised and rotated by position."""
    T, D, dt = heads.T, heads.head_dim, _TORCH_DTYPE[heads.dtype]
    nq, nk = heads.n_q_heads, heads.n_kv_heads
    _check("qk_norm_rope", _lib.qk_norm_rope(
        heads, *_rows("q", q, T, nq, D, dt), *_rows("k", k, T, nk, D, dt),
        *_rotation(heads, q_weight, k_weight, table, positions, dt),
        *_rows("q_out", q_out, T, nq, D, dt), *_rows("k_out", k_out, T, nk, D, dt),
        _stream_ptr(stream, q if nq else k)))


def alloc_heads_workspace(heads: Heads, device=None) -> torch.Tensor:
    """Device workspace of qk_norm_rope_bwd."""
    n = int(_lib.qk_norm_rope_bwd_workspace_bytes(heads))
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def qk_norm_rope_bwd(heads: Heads, q, k, q_weight, k_weight, table, positions, gq_out, gk_out, gq,
                     gk, gq_weight, gk_weight, workspace, stream=None) -> None:
    """gq, gk (as q, k) and the float32 weight gradients [head_dim] (each may be
    None) from the gradients of qk_norm_rope's outputs."""
    T, D, dt = heads.T, heads.head_dim, _TORCH_DTYPE[heads.dtype]
    nq, nk = heads.n_q_heads, heads.n_kv_heads
    ws, ws_n = (None, 0) if workspace is None else \
        (_ptr(workspace), workspace.numel() * workspace.element_size())
    _check("qk_norm_rope_bwd", _lib.qk_norm_rope_bwd(
        heads, *_rows("q", q, T, nq, D, dt), *_rows("k", k, T, nk, D, dt),
        *_rotation(heads, q_weight, k_weight, table, positions, dt),
        *_rows("gq_out", gq_out, T, nq, D, dt), *_rows("gk_out", gk_out, T, nk, D, dt),
        *_rows("gq", gq, T, nq, D, dt), *_rows("gk", gk, T, nk, D, dt),
        _array("gq_weight", gq_weight, D, torch.float32, True),
        _array("gk_weight", gk_weight, D, torch.float32, True), ws, ws_n,
        _stream_ptr(stream, gq_out if nq else gk_out)))


def paged_kv_append(heads: Heads, q, k, v, q_weight, k_weight, table, positions, slots, q_out,
                    k_cache, v_cache, stream=None) -> None:
    """q normalised and rotated into q_out, k into its slots of k_cache, v copied
    into v_cache ([n_pages, page_size, n_kv_heads, head_dim], any strides).
    slots: int32 [T], page * page_size + offset, -1: not stored.  With
    heads.n_q_heads == 0, q and q_out may be None."""
    T, D, dt = heads.T, heads.head_dim, _TORCH_DTYPE[heads.dtype]
    nq, nk = heads.n_q_heads, heads.n_kv_heads
    n_pages, page_size = k_cache.shape[0], k_cache.shape[1]
    _check("paged_kv_append", _lib.paged_kv_append(
        heads, *_rows("q", q, T, nq, D, dt), *_rows("k", k, T, nk, D, dt),
        *_rows("v", v, T, nk, D, dt), *_rotation(heads, q_weight, k_weight, table, positions, dt),
        _array("slots", slots, T, torch.int32), *_rows("q_out", q_out, T, nq, D, dt),
        *_cache("k_cache", k_cache, n_pages, page_size, nk, D, dt),
        *_cache("v_cache", v_cache, n_pages, page_size, nk, D, dt), n_pages, page_size,
        _stream_ptr(stream, k_cache)))


def paged_attn_workspace_bytes(batch: PagedBatch) -> int:
    return int(_lib.paged_attn_workspace_bytes(batch))


def alloc_paged_workspace(batch: PagedBatch, device=None) -> torch.Tensor:
    """Device workspace of paged_attn_fwd (no initial contents needed)."""
    n = paged_attn_workspace_bytes(batch)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def paged_attn_fwd(batch: PagedBatch, q, k_cache, v_cache, q_start, kv_len, block_table, out,
                   workspace, lse=None, stream=None) -> None:
    """out [T, n_q_heads, head_dim] (and lse [T, n_q_heads] float32): attention of
    every sequence's new tokens, rows q_start[s] .. q_start[s+1] - 1 of q, over
    its kv_len[s] cached keys, found through block_table [n_seqs, max_pages]."""
    T, D, dt = batch.T, batch.head_dim, _TORCH_DTYPE[batch.dtype]
    nq, nk, ns = batch.n_q_heads, batch.n_kv_heads, batch.n_seqs
    ws, ws_n = (None, 0) if workspace is None else \
        (_ptr(workspace), workspace.numel() * workspace.element_size())
    _check("paged_attn_fwd", _lib.paged_attn_fwd(
        batch, *_rows("q", q, T, nq, D, dt),
        *_cache("k_cache", k_cache, batch.n_pages, batch.page_size, nk, D, dt),
        *_cache("v_cache", v_cache, batch.n_pages, batch.page_size, nk, D, dt),
        _array("q_start", q_start, ns + 1, torch.int32), _array("kv_len", kv_len, ns, torch.int32),
        _table("block_table", block_table, ns, batch.max_pages, torch.int32),
        *_rows("out", out, T, nq, D, dt), _table("lse", lse, T, nq, torch.float32), ws, ws_n,
        _stream_ptr(stream, out)))


class Mx4Cache:
    """A layer's keys and values in four bits (OCP MX FP4, blocks of 32 elements of a head):
    codes uint8 [n_pages, page_size, n_kv_heads, head_dim / 2] and scales uint8 [n_pages,
    page_size, n_kv_heads, ceil(head_dim / 32)] of each, any strides with the last dimension
    contiguous.  Allocated here, a page's tokens of one head lie side by side.  The tensors
    are the cache's own: they keep their places for its lifetime."""

    def __init__(self, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, device="cuda",
                 k_codes=None, k_scales=None, v_codes=None, v_scales=None):
        self.n_pages, self.page_size = int(n_pages), int(page_size)
        self.n_kv_heads, self.head_dim = int(n_kv_heads), int(head_dim)
        if self.head_dim <= 0 or self.head_dim % 8:
            raise ValueError(f"head_dim must be a positive multiple of 8, not {head_dim}")
        given = (k_codes, k_scales, v_codes, v_scales)
        if any(t is None for t in given):
            if any(t is not None for t in given):
                raise ValueError("codes and scales of k and v are given together or not at all")
            given = [torch.zeros((self.n_pages, self.n_kv_heads, self.page_size, n),
                                 dtype=torch.uint8, device=device).transpose(1, 2)
                     for n in (self.head_dim // 2, -(-self.head_dim // 32)) * 2]
        self._tensors = tuple(given)
        self._k = self._place("k", *given[:2])
        self._v = self._place("v", *given[2:])
        if len({t.device for t in given}) > 1:
            raise ValueError("the tensors of a cache must lie on one GPU")

    def _place(self, name, codes, scales) -> Mx4Rows:
        shape = self.n_pages, self.page_size, self.n_kv_heads
        c = _cache(name + "_codes", codes, *shape, self.head_dim // 2, torch.uint8)
        s = _cache(name + "_scales", scales, *shape, -(-self.head_dim // 32), torch.uint8)
        return Mx4Rows(c[0], s[0], *c[1:], *s[1:])

    k_codes = property(lambda self: self._tensors[0])
    k_scales = property(lambda self: self._tensors[1])
    v_codes = property(lambda self: self._tensors[2])
    v_scales = property(lambda self: self._tensors[3])

    def _check(self, fn: str, n_pages: int, page_size: int, heads: int, dim: int) -> None:
        if (n_pages, page_size, heads, dim) != (self.n_pages, self.page_size, self.n_kv_heads,
                                                self.head_dim):
            raise ValueError(f"{fn}: the cache has {self.n_pages} pages of {self.page_size}, "
                             f"{self.n_kv_heads} heads of {self.head_dim}, not {n_pages} of "
                             f"{page_size}, {heads} of {dim}")


def paged_kv_append_mx4(heads: Heads, q, k, v, q_weight, k_weight, table, positions, slots, q_out,
                        cache: Mx4Cache, stream=None) -> None:
    """paged_kv_append into a 4-bit cache: k, normalised and rotated, and v are quantised as
    they are written."""
    T, D, dt = heads.T, heads.head_dim, _TORCH_DTYPE[heads.dtype]
    nq, nk = heads.n_q_heads, heads.n_kv_heads
    cache._check("paged_kv_append_mx4", cache.n_pages, cache.page_size, nk, D)
    _check("paged_kv_append_mx4", _lib.paged_kv_append_mx4(
        heads, *_rows("q", q, T, nq, D, dt), *_rows("k", k, T, nk, D, dt),
        *_rows("v", v, T, nk, D, dt), *_rotation(heads, q_weight, k_weight, table, positions, dt),
        _array("slots", slots, T, torch.int32), *_rows("q_out", q_out, T, nq, D, dt), cache._k,
        cache._v, cache.n_pages, cache.page_size, _stream_ptr(stream, cache.k_codes)))


def paged_kv_read_mx4(cache: Mx4Cache, slots, k_out, v_out, stream=None) -> None:
    """k_out, v_out ([T, n_kv_heads, head_dim] float32 or bfloat16, each may be None): the
    values of the cache rows `slots` (int32 [T]); those of a slot outside the cache (-1)
    are left as they were."""
    out = k_out if k_out is not None else v_out
    if out is None:
        return
    T, nk, D, dt = out.shape[0], cache.n_kv_heads, cache.head_dim, out.dtype
    _check("paged_kv_read_mx4", _lib.paged_kv_read_mx4(
        T, nk, D, _code(dt), cache._k, cache._v, cache.n_pages, cache.page_size,
        _array("slots", slots, T, torch.int32), *_rows("k_out", k_out, T, nk, D, dt),
        *_rows("v_out", v_out, T, nk, D, dt), _stream_ptr(stream, cache.k_codes)))


def paged_attn_mx4_workspace_bytes(batch: PagedBatch) -> int:
    return int(_lib.paged_attn_mx4_workspace_bytes(batch))


def alloc_paged_mx4_workspace(batch: PagedBatch, device=None) -> torch.Tensor:
    """Device workspace of paged_attn_mx4_fwd (no initial contents needed)."""
    n = paged_attn_mx4_workspace_bytes(batch)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def paged_attn_mx4_fwd(batch: PagedBatch, q, cache: Mx4Cache, q_start, kv_len, block_table, out,
                       workspace, lse=None, stream=None) -> None:
    """paged_attn_fwd over a 4-bit cache."""
    T, D, dt = batch.T, batch.head_dim, _TORCH_DTYPE[batch.dtype]
    nq, nk, ns = batch.n_q_heads, batch.n_kv_heads, batch.n_seqs
    cache._check("paged_attn_mx4_fwd", batch.n_pages, batch.page_size, nk, D)
    ws, ws_n = (None, 0) if workspace is None else \
        (_ptr(workspace), workspace.numel() * workspace.element_size())
    _check("paged_attn_mx4_fwd", _lib.paged_attn_mx4_fwd(
        batch, *_rows("q", q, T, nq, D, dt), cache._k, cache._v,
        _array("q_start", q_start, ns + 1, torch.int32), _array("kv_len", kv_len, ns, torch.int32),
        _table("block_table", block_table, ns, batch.max_pages, torch.int32),
        *_rows("out", out, T, nq, D, dt), _table("lse", lse, T, nq, torch.float32), ws, ws_n,
        _stream_ptr(stream, cache.k_codes)))


def paged_slots(block_table, seq, positions, page_size: int) -> torch.Tensor:
    """Slots (int32) of tokens at `positions` of the sequences `seq`, through
    block_table; computed once a step, for all layers.  -1 (not stored) for positions
    outside the table, as -1 for padding tokens, and for pages that are not there (-1)."""
    pos = positions.long()
    inside = (pos >= 0) & (pos < block_table.shape[1] * page_size)
    pos = torch.where(inside, pos, 0)
    page = block_table[seq.long(), pos // page_size].long()
    return torch.where(inside & (page >= 0), page * page_size + pos % page_size, -1).to(torch.int32)


class PagedAttention:
    """Cache and buffers of one layer for repeated serving steps of one batch
    shape (T new tokens of n_seqs sequences).  ``forward`` issues paged_kv_append
    and paged_attn_fwd on one stream with no host synchronisation.  The caches
    may be given (``k_cache``, ``v_cache``), e.g. to use them with several batch
    shapes.  With ``mx4`` the cache is a 4-bit one, a new one (True) or the one given
    (an ``Mx4Cache``, kept as ``cache``), and the entry points are those of that form."""

    def __init__(self, T: int, n_seqs: int, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype,
                 page_size: int, n_pages: int, max_pages: int, max_q: int, max_kv: int,
                 rot_dim: int = 0, max_pos: int = 0, norm: bool = False, eps: float = 1e-6,
                 adjacent: bool = False, causal: bool = True, window: int = 0,
                 scale: float | None = None, k_cache=None, v_cache=None, device="cuda",
                 mx4: bool | Mx4Cache = False):
        self.heads = make_heads(T, n_q_heads, n_kv_heads, head_dim, dtype, rot_dim, max_pos, norm,
                                eps, adjacent)
        self.batch = make_paged_batch(T, n_seqs, n_q_heads, n_kv_heads, head_dim, dtype, page_size,
                                      n_pages, max_pages, max_q, max_kv, causal, window, scale)
        dt = _TORCH_DTYPE[self.heads.dtype]
        self.cache = self.k_cache = self.v_cache = None
        if mx4:
            if k_cache is not None or v_cache is not None:
                raise ValueError("a 4-bit cache is given as mx4, not as k_cache and v_cache")
            self.cache = mx4 if isinstance(mx4, Mx4Cache) else \
                Mx4Cache(n_pages, page_size, n_kv_heads, head_dim, device)
            self.cache._check("PagedAttention", n_pages, page_size, n_kv_heads, head_dim)
        else:
            shape = (n_pages, page_size, n_kv_heads, head_dim)
            self.k_cache = torch.empty(shape, dtype=dt, device=device) if k_cache is None else k_cache
            self.v_cache = torch.empty(shape, dtype=dt, device=device) if v_cache is None else v_cache
        self.q_out = torch.empty((T, n_q_heads, head_dim), dtype=dt, device=device)
        self.out = torch.empty((T, n_q_heads, head_dim), dtype=dt, device=device)
        self.lse = torch.empty((T, n_q_heads), dtype=torch.float32, device=device)
        self.workspace = alloc_paged_mx4_workspace(self.batch, device) if mx4 else \
            alloc_paged_workspace(self.batch, device)

    def forward(self, q, k, v, positions, slots, q_start, kv_len, block_table, table=None,
                q_weight=None, k_weight=None, stream=None) -> torch.Tensor:
        if self.cache is not None:
            paged_kv_append_mx4(self.heads, q, k, v, q_weight, k_weight, table, positions, slots,
                                self.q_out, self.cache, stream)
            paged_attn_mx4_fwd(self.batch, self.q_out, self.cache, q_start, kv_len, block_table,
                               self.out, self.workspace, self.lse, stream)
            return self.out
        paged_kv_append(self.heads, q, k, v, q_weight, k_weight, table, positions, slots,
                        self.q_out, self.k_cache, self.v_cache, stream)
        paged_attn_fwd(self.batch, self.q_out, self.k_cache, self.v_cache, q_start, kv_len,
                       block_table, self.out, self.workspace, self.lse, stream)
        return self.out


class SparseFFN:
    """Buffers for repeated sparse forwards of one shape: TwELL arrays, routed
    list, workspaces.  ``forward`` issues twell_pack, sparse_ffn_fwd and
    hybrid_route on one stream with no host synchronisation.  ``wg_norms``
    (from ``weight_norms``) may be passed to skip recomputing the gate-weight
    row norms on every call."""

    def __init__(self, T: int, d_model: int, d_ff: int, cap: int, dtype: torch.dtype,
                 device="cuda"):
        code = SFFN_BF16 if dtype == torch.bfloat16 else SFFN_F32
        self.shape = make_shape(T, d_model, d_ff, cap, code)
        self.dtype = dtype
        self.count, self.idx, self.val = alloc_twell(self.shape, device)
        self.routed = torch.empty(max(T, 1), dtype=torch.int32, device=device)
        self.n_routed = torch.zeros(1, dtype=torch.int32, device=device)
        self.ws_sparse = alloc_workspace(self.shape, WS_SPARSE, device)
        self.ws_pack = alloc_workspace(self.shape, WS_PACK, device)
        self.ws_hybrid = alloc_workspace(self.shape, WS_HYBRID, device)
        self.y = torch.empty((T, d_model), dtype=dtype, device=device)

    def weight_norms(self, wg_t, stream=None) -> torch.Tensor:
        n = torch.empty(self.shape.d_ff, dtype=torch.float32, device=wg_t.device)
        twell_weight_norms(self.shape, wg_t, n, stream)
        return n

    def forward(self, x, wg_t, b_g, wu_t, wd, wg_norms=None, stream=None) -> torch.Tensor:
        s = self.shape
        twell_pack(s, x, wg_t, b_g, self.count, self.idx, self.val, self.ws_pack, wg_norms, stream)
        sparse_ffn_fwd(s, x, wu_t, wd, self.count, self.idx, self.val, self.y, self.ws_sparse,
                       stream)
        hybrid_route(s, x, wg_t, b_g, wu_t, wd, self.count, self.routed, self.n_routed,
                     self.ws_hybrid, self.y, stream)
        return self.y


class DenseFFN:
    """Buffers for repeated dense reference forwards of one shape."""

    def __init__(self, T: int, d_model: int, d_ff: int, dtype: torch.dtype, device="cuda"):
        code = SFFN_BF16 if dtype == torch.bfloat16 else SFFN_F32
        self.shape = make_shape(T, d_model, d_ff, 0, code)
        self.ws = alloc_workspace(self.shape, WS_DENSE, device)
        self.y = torch.empty((T, d_model), dtype=dtype, device=device)

    def forward(self, x, wg_t, b_g, wu_t, wd, stream=None) -> torch.Tensor:
        dense_ffn_ref(self.shape, x, wg_t, b_g, wu_t, wd, self.ws, self.y, stream)
        return self.y
