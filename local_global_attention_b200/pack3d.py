"""Python binding of the PACK3D C ABI (include/pack3d.h) over ctypes.

Argument marshalling only: every step of the operator runs in the CUDA
library ``_build/libpack3d.so``.  Tensors are torch CUDA tensors; the functions
keep the C names and pass ``data_ptr()`` and the current (or given) stream.
If the library is missing or no CUDA device is present, the calls raise; there
is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

BF16, FP32 = 0, 1
ZERO_UNUSED_ROWS = 0x100  # or'ed into the dtype of a packed-sequence or rotary call's params
ROPE_AXIAL, ROPE_PACKED = 0, 1  # axial RoPE on grid coordinates / 1-D RoPE on the packed index
OK, ERR_ARG, ERR_COORDS, ERR_CUDA, ERR_TIMEOUT, ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5
ERR_LENGTHS = -6
ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}
ROTARY_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}

EXPORTS = ("pack3d_index_bytes", "pack3d_index_init", "pack3d_build_index", "pack3d_index_check",
           "pack3d_block_summaries", "pack3d_forward_workspace_bytes", "pack3d_forward",
           "pack3d_window_forward", "pack3d_stage_kv", "pack3d_forward_staged",
           "pack3d_backward_workspace_bytes", "pack3d_backward", "pack3d_backward_summary_grads",
           "pack3d_backward_from_summary_grads", "pack3d_backward_noalloc",
           "pack3d_kernel_launches", "pack3d_wait_selftest", "pack3d_strerror",
           "pack3d_seq_index_bytes", "pack3d_seq_index_init", "pack3d_seq_build_index",
           "pack3d_seq_index_check", "pack3d_seq_forward", "pack3d_seq_backward_workspace_bytes",
           "pack3d_seq_backward", "pack3d_rotary", "pack3d_rotary_backward")


class Params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "H", "head_dim", "Z", "Y", "X", "wz", "wy", "wx", "bz", "by", "bx")] + [
        ("rope_base", ctypes.c_float), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32),
        ("out_fp32", ctypes.c_int32), ("rope_mode", ctypes.c_int32), ("n_tokens", ctypes.c_int32),
        ("Z_total", ctypes.c_int32), ("z_origin", ctypes.c_int32), ("own_lo", ctypes.c_int32),
        ("own_hi", ctypes.c_int32)]


class Index(ctypes.Structure):
    _fields_ = [("vol", ctypes.c_void_p), ("perm", ctypes.c_void_p),
                ("tile_off", ctypes.c_void_p), ("nbr_off", ctypes.c_void_p),
                ("nbr", ctypes.c_void_p), ("rope", ctypes.c_void_p), ("err", ctypes.c_void_p),
                ("bcount", ctypes.c_void_p), ("bocc", ctypes.c_void_p),
                ("tile", ctypes.c_int32 * 3), ("n_tiles", ctypes.c_int32),
                ("n_halo", ctypes.c_int64)]


class SeqParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_seqs", "n_tokens", "Hq", "Hk", "head_dim",
                                              "causal")] + [
        ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class SeqStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("q", "k", "v", "out", "dout", "dq", "dk", "dv")]


class SeqIndexStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("pos", "seq", "pair", "query", "key", "err")] + [
        (n, ctypes.c_int32) for n in ("n_pair", "n_rows", "n_seqs", "n_tokens")]


class RotaryParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_tokens", "Hq", "Hk", "head_dim", "rot_dim",
                                              "layout", "dtype")] + [
        ("base", ctypes.c_float), ("scaling", ctypes.c_int32), ("factor", ctypes.c_float),
        ("original_length", ctypes.c_int32), ("low", ctypes.c_float), ("high", ctypes.c_float),
        ("amplitude", ctypes.c_float)] + [
        (n, ctypes.c_int64) for n in ("stride_q", "stride_k", "stride_q_out", "stride_k_out")]


class Pack3dError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {strerror(status)} ({status})")
        self.status = status


_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load libpack3d.so (building it in-tree first if it is missing)."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if not os.path.exists(path):
            if not build_if_missing:
                raise OSError(f"PACK3D CUDA library not built: {path}")
            _build.build()
        lib = ctypes.CDLL(path)
        P = ctypes.POINTER
        vp = ctypes.c_void_p
        lib.pack3d_index_bytes.argtypes = [P(Params)]
        lib.pack3d_index_bytes.restype = ctypes.c_size_t
        lib.pack3d_index_init.argtypes = [P(Params), vp, ctypes.c_size_t, P(Index)]
        lib.pack3d_build_index.argtypes = [P(Params), vp, P(Index), vp]
        lib.pack3d_index_check.argtypes = [P(Index), vp]
        lib.pack3d_block_summaries.argtypes = [P(Params), P(Index), vp, vp, vp, vp, vp]
        lib.pack3d_forward_workspace_bytes.argtypes = [P(Params)]
        lib.pack3d_forward_workspace_bytes.restype = ctypes.c_size_t
        lib.pack3d_forward.argtypes = [P(Params), P(Index), vp, vp, vp, vp, vp, vp,
                                       ctypes.c_size_t, vp, vp, vp]
        lib.pack3d_window_forward.argtypes = [P(Params), P(Index), vp, vp, vp, vp,
                                              ctypes.c_size_t, vp, vp, vp]
        lib.pack3d_stage_kv.argtypes = [P(Params), P(Index), vp, vp, vp, vp, vp, ctypes.c_size_t,
                                        vp]
        lib.pack3d_forward_staged.argtypes = [P(Params), P(Index), vp, vp, ctypes.c_size_t,
                                              ctypes.c_int, vp, vp, vp]
        lib.pack3d_backward_workspace_bytes.argtypes = [P(Params)]
        lib.pack3d_backward_workspace_bytes.restype = ctypes.c_size_t
        lib.pack3d_backward.argtypes = [P(Params), P(Index), vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                        vp, ctypes.c_size_t, vp]
        lib.pack3d_backward_summary_grads.argtypes = [P(Params), P(Index), vp, vp, vp, vp, vp,
                                                      vp, vp, vp, vp, vp, vp, ctypes.c_size_t,
                                                      vp]
        lib.pack3d_backward_from_summary_grads.argtypes = [P(Params), P(Index), vp, vp, vp,
                                                           ctypes.c_size_t, vp, vp, vp, vp]
        lib.pack3d_backward_noalloc.argtypes = [P(Params), P(Index), vp, vp, vp, vp, vp, vp, vp,
                                                vp, vp, vp]
        sp, si, ss = P(SeqParams), P(SeqIndexStruct), P(SeqStrides)
        lib.pack3d_seq_index_bytes.argtypes = [sp]
        lib.pack3d_seq_index_bytes.restype = ctypes.c_size_t
        lib.pack3d_seq_index_init.argtypes = [sp, vp, ctypes.c_size_t, si]
        lib.pack3d_seq_build_index.argtypes = [sp, vp, si, vp]
        lib.pack3d_seq_index_check.argtypes = [si, vp]
        lib.pack3d_seq_forward.argtypes = [sp, si, ss, vp, vp, vp, vp, vp, vp]
        lib.pack3d_seq_backward_workspace_bytes.argtypes = [sp]
        lib.pack3d_seq_backward_workspace_bytes.restype = ctypes.c_size_t
        lib.pack3d_seq_backward.argtypes = [sp, si, ss, *([vp] * 10), ctypes.c_size_t, vp]
        lib.pack3d_rotary.argtypes = [P(RotaryParams), *([vp] * 6)]
        lib.pack3d_rotary_backward.argtypes = [P(RotaryParams), *([vp] * 6)]
        lib.pack3d_wait_selftest.argtypes = [ctypes.c_uint32, vp]
        lib.pack3d_kernel_launches.argtypes = []
        lib.pack3d_kernel_launches.restype = ctypes.c_uint64
        lib.pack3d_strerror.argtypes = [ctypes.c_int]
        lib.pack3d_strerror.restype = ctypes.c_char_p
        for name in EXPORTS:
            getattr(lib, name).restype = getattr(lib, name).restype or ctypes.c_int
        _lib = lib
    return _lib


def pack3d_kernel_launches() -> int:
    """Kernels the library has launched in this process so far."""
    return int(load().pack3d_kernel_launches())


def pack3d_wait_selftest(polls: int = 1000, stream=None) -> int:
    """Status of a bounded device wait that runs out (ERR_TIMEOUT expected)."""
    return int(load().pack3d_wait_selftest(ctypes.c_uint32(polls), _stream(stream)))


def strerror(status: int) -> str:
    return load().pack3d_strerror(int(status)).decode()


def _check(status: int, what: str):
    if status != OK:
        raise Pack3dError(status, what)


def make_params(shape, dtype=None, scale: float = 0.0, out_fp32: bool = False) -> Params:
    """Params from any object with ``B, H, d, Z, Y, X, window, block, rope_base``
    (and ``dtype`` "bf16"/"fp32" unless given, ``rope_mode`` 0, ``n_tokens`` 0
    (a dense volume) and no z-slab (``Z_total``, ``z_origin``, ``own_lo``,
    ``own_hi``) unless set).  ``out_fp32`` makes the forward output fp32 for
    bf16 inputs."""
    dt = dtype if dtype is not None else getattr(shape, "dtype", "bf16")
    code = {"bf16": BF16, "fp32": FP32, torch.bfloat16: BF16, torch.float32: FP32}[dt]
    w, b = tuple(shape.window), tuple(shape.block)
    return Params(shape.B, shape.H, shape.d, shape.Z, shape.Y, shape.X, w[0], w[1], w[2],
                  b[0], b[1], b[2], float(shape.rope_base), float(scale), code, int(bool(out_fp32)),
                  int(getattr(shape, "rope_mode", 0) or 0), int(getattr(shape, "n_tokens", 0) or 0),
                  *(int(getattr(shape, f, 0) or 0) for f in ("Z_total", "z_origin", "own_lo",
                                                             "own_hi")))


def out_dtype(params: Params, like: torch.Tensor) -> torch.dtype:
    return torch.float32 if params.out_fp32 else like.dtype


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("PACK3D tensors must be CUDA tensors")
        if t is not None and not t.is_contiguous():
            raise ValueError("PACK3D tensors must be contiguous")


class IndexBuffers:
    """A built index: the caller-owned device buffer and the C struct over it."""

    def __init__(self, params: Params, device=None):
        lib = load()
        self.params = params
        nbytes = lib.pack3d_index_bytes(ctypes.byref(params))
        if nbytes == 0:
            raise Pack3dError(ERR_ARG, "pack3d_index_bytes")
        self.buffer = torch.empty(nbytes + 256, dtype=torch.uint8, device=device or "cuda")
        base = self.buffer.data_ptr()
        off = (-base) % 256
        self.struct = Index()
        _check(lib.pack3d_index_init(ctypes.byref(params), ctypes.c_void_p(base + off),
                                     ctypes.c_size_t(nbytes), ctypes.byref(self.struct)),
               "pack3d_index_init")
        self.nbytes = nbytes

    # Views of the index arrays (for tests and inspection).
    def _view(self, field, count, dtype):
        ptr = getattr(self.struct, field)
        off = ptr - self.buffer.data_ptr()
        esz = torch.tensor([], dtype=dtype).element_size()
        return self.buffer[off:off + count * esz].view(dtype)

    def arrays(self):
        p, s = self.params, self.struct
        V = p.Z * p.Y * p.X
        N = p.n_tokens or V
        T = s.n_tiles
        nb = (-(-(p.Z_total or p.Z) // p.bz)) * (-(-p.Y // p.by)) * (-(-p.X // p.bx))
        return {
            "vol": self._view("vol", p.B * V, torch.int32).view(p.B, V),
            "bcount": self._view("bcount", p.B * nb, torch.int32).view(p.B, nb),
            "perm": self._view("perm", p.B * N, torch.int32).view(p.B, N),
            "tile_off": self._view("tile_off", p.B * (T + 1), torch.int32).view(p.B, T + 1),
            "nbr_off": self._view("nbr_off", T + 1, torch.int32),
            "nbr": self._view("nbr", p.B * s.n_halo, torch.int32).view(p.B, s.n_halo),
            "rope": self._view("rope", 2 * (p.Z + p.Y + p.X) * (p.head_dim // 6), torch.float32),
            "err": self._view("err", 2, torch.int32),
        }


def pack3d_build_index(params: Params, coords: torch.Tensor, index: IndexBuffers = None,
                       stream=None) -> IndexBuffers:
    _need_cuda(coords)
    if coords.dtype != torch.int16:
        raise ValueError("coords must be int16 [B, N, 3]")
    if index is None:
        index = IndexBuffers(params, device=coords.device)
    _check(load().pack3d_build_index(ctypes.byref(params), _ptr(coords),
                                     ctypes.byref(index.struct), _stream(stream)),
           "pack3d_build_index")
    return index


def pack3d_index_check(index: IndexBuffers, stream=None) -> int:
    """Synchronise and return the index status code (0, ERR_COORDS, ERR_TIMEOUT)."""
    return int(load().pack3d_index_check(ctypes.byref(index.struct), _stream(stream)))


def _dims(params):
    return params.B, params.n_tokens or params.Z * params.Y * params.X, params.H, params.head_dim


def n_blocks(params: Params) -> int:
    """Blocks of the volume (a z-slab: of the whole volume); blocks that do not
    divide the volume are cut at its edge, so the counts round up."""
    Zg = params.Z_total or params.Z
    return (-(-Zg // params.bz)) * (-(-params.Y // params.by)) * (-(-params.X // params.bx))


def pack3d_block_summaries(params: Params, index: IndexBuffers, k, v, ksum=None, vsum=None,
                           stream=None):
    _need_cuda(k, v)
    B, N, H, d = _dims(params)
    nb = n_blocks(params)
    if ksum is None:
        ksum = torch.empty(B, H, nb, d, dtype=torch.float32, device=k.device)
    if vsum is None:
        vsum = torch.empty(B, H, nb, d, dtype=torch.float32, device=k.device)
    _need_cuda(ksum, vsum)
    _check(load().pack3d_block_summaries(ctypes.byref(params), ctypes.byref(index.struct),
                                         _ptr(k), _ptr(v), _ptr(ksum), _ptr(vsum),
                                         _stream(stream)), "pack3d_block_summaries")
    return ksum, vsum


def pack3d_forward_workspace_bytes(params: Params) -> int:
    return int(load().pack3d_forward_workspace_bytes(ctypes.byref(params)))


def _forward_workspace(params, workspace, device):
    nbytes = pack3d_forward_workspace_bytes(params)
    if workspace is None and nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if workspace is None:
        return None, 0
    _need_cuda(workspace)
    return workspace, workspace.numel() * workspace.element_size()


def pack3d_forward(params: Params, index: IndexBuffers, q, k, v, ksum, vsum, out=None, lse=None,
                   workspace=None, stream=None):
    _need_cuda(q, k, v, ksum, vsum)
    B, N, H, d = _dims(params)
    out = torch.empty_like(q, dtype=out_dtype(params, q)) if out is None else out
    lse = torch.empty(B, H, N, dtype=torch.float32, device=q.device) if lse is None else lse
    _need_cuda(out, lse)
    ws, nbytes = _forward_workspace(params, workspace, q.device)
    _check(load().pack3d_forward(ctypes.byref(params), ctypes.byref(index.struct), _ptr(q),
                                 _ptr(k), _ptr(v), _ptr(ksum), _ptr(vsum),
                                 None if ws is None else _ptr(ws), ctypes.c_size_t(nbytes),
                                 _ptr(out), _ptr(lse), _stream(stream)), "pack3d_forward")
    return out, lse


def pack3d_window_forward(params: Params, index: IndexBuffers, q, k, v, out=None, lse=None,
                          workspace=None, stream=None):
    _need_cuda(q, k, v)
    B, N, H, d = _dims(params)
    out = torch.empty_like(q, dtype=out_dtype(params, q)) if out is None else out
    lse = torch.empty(B, H, N, dtype=torch.float32, device=q.device) if lse is None else lse
    _need_cuda(out, lse)
    ws, nbytes = _forward_workspace(params, workspace, q.device)
    _check(load().pack3d_window_forward(ctypes.byref(params), ctypes.byref(index.struct),
                                        _ptr(q), _ptr(k), _ptr(v),
                                        None if ws is None else _ptr(ws),
                                        ctypes.c_size_t(nbytes), _ptr(out), _ptr(lse),
                                        _stream(stream)), "pack3d_window_forward")
    return out, lse


def pack3d_stage_kv(params: Params, index: IndexBuffers, k, v, ksum=None, vsum=None,
                    workspace=None, stream=None):
    """Stage rotated keys and values in grid order (and bf16 summaries) for
    pack3d_forward_staged; returns the workspace."""
    _need_cuda(k, v)
    ws, nbytes = _forward_workspace(params, workspace, k.device)
    _check(load().pack3d_stage_kv(ctypes.byref(params), ctypes.byref(index.struct), _ptr(k),
                                  _ptr(v), None if ksum is None else _ptr(ksum),
                                  None if vsum is None else _ptr(vsum),
                                  None if ws is None else _ptr(ws), ctypes.c_size_t(nbytes),
                                  _stream(stream)), "pack3d_stage_kv")
    return ws


def pack3d_forward_staged(params: Params, index: IndexBuffers, q, workspace, with_summaries=True,
                          out=None, lse=None, stream=None):
    _need_cuda(q, workspace)
    B, N, H, d = _dims(params)
    out = torch.empty_like(q, dtype=out_dtype(params, q)) if out is None else out
    lse = torch.empty(B, H, N, dtype=torch.float32, device=q.device) if lse is None else lse
    _need_cuda(out, lse)
    _check(load().pack3d_forward_staged(ctypes.byref(params), ctypes.byref(index.struct), _ptr(q),
                                        _ptr(workspace),
                                        ctypes.c_size_t(workspace.numel() *
                                                        workspace.element_size()),
                                        int(bool(with_summaries)), _ptr(out), _ptr(lse),
                                        _stream(stream)), "pack3d_forward_staged")
    return out, lse


def pack3d_backward_workspace_bytes(params: Params) -> int:
    return int(load().pack3d_backward_workspace_bytes(ctypes.byref(params)))


def pack3d_backward(params: Params, index: IndexBuffers, q, k, v, out, lse, dout, dq=None,
                    dk=None, dv=None, workspace=None, stream=None):
    _need_cuda(q, k, v, out, lse, dout)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    nbytes = pack3d_backward_workspace_bytes(params)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _need_cuda(dq, dk, dv, workspace)
    _check(load().pack3d_backward(ctypes.byref(params), ctypes.byref(index.struct), _ptr(q),
                                  _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
                                  _ptr(dk), _ptr(dv), _ptr(workspace),
                                  ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                                  _stream(stream)), "pack3d_backward")
    return dq, dk, dv


def pack3d_backward_summary_grads(params: Params, index: IndexBuffers, q, k, v, out, lse, dout,
                                  ksum=None, vsum=None, dks=None, dvs=None, workspace=None,
                                  stream=None):
    """First half of the two-call backward: stages the inputs into `workspace`
    (allocated when None) and returns (dks, dvs, workspace), the summary
    gradients [B, H, nb, d] fp32 over the call's owned queries."""
    _need_cuda(q, k, v, out, lse, dout)
    B, N, H, d = _dims(params)
    nb = n_blocks(params)
    dks = torch.empty(B, H, nb, d, dtype=torch.float32, device=q.device) if dks is None else dks
    dvs = torch.empty(B, H, nb, d, dtype=torch.float32, device=q.device) if dvs is None else dvs
    if workspace is None:
        workspace = torch.empty(pack3d_backward_workspace_bytes(params), dtype=torch.uint8,
                                device=q.device)
    _need_cuda(dks, dvs, workspace)
    if ksum is not None:
        _need_cuda(ksum, vsum)
    _check(load().pack3d_backward_summary_grads(
        ctypes.byref(params), ctypes.byref(index.struct), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
        _ptr(lse), _ptr(dout), _ptr(ksum), _ptr(vsum), _ptr(dks), _ptr(dvs), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream(stream)),
        "pack3d_backward_summary_grads")
    return dks, dvs, workspace


def pack3d_backward_from_summary_grads(params: Params, index: IndexBuffers, dks, dvs, workspace,
                                       dq, dk, dv, stream=None):
    """Second half: dq, dk, dv of the owned tokens from the staged workspace and
    the summary gradients of the whole volume."""
    _need_cuda(dks, dvs, workspace, dq, dk, dv)
    _check(load().pack3d_backward_from_summary_grads(
        ctypes.byref(params), ctypes.byref(index.struct), _ptr(dks), _ptr(dvs), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size()), _ptr(dq), _ptr(dk),
        _ptr(dv), _stream(stream)), "pack3d_backward_from_summary_grads")
    return dq, dk, dv


NOALLOC_SCRATCH_BYTES = 32 << 20


def pack3d_backward_noalloc(params: Params, index: IndexBuffers, q, k, v, out, lse, dout,
                            dq=None, dk=None, dv=None, stream=None):
    """pack3d_backward without a workspace argument: the library's static
    device scratch array (NOALLOC_SCRATCH_BYTES) stands in for it.  Calls that
    overlap on the GPU share that array and race; the first call on a device
    looks the array up and should precede any stream capture."""
    _need_cuda(q, k, v, out, lse, dout)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _need_cuda(dq, dk, dv)
    _check(load().pack3d_backward_noalloc(ctypes.byref(params), ctypes.byref(index.struct),
                                          _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                          _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                                          _stream(stream)), "pack3d_backward_noalloc")
    return dq, dk, dv


class Pack3D:
    """Convenience wrapper: one operator shape, its index, and the calls."""

    def __init__(self, shape, dtype=None, scale: float = 0.0, out_fp32: bool = False):
        self.params = make_params(shape, dtype, scale, out_fp32)
        self.index = None

    def build_index(self, coords, stream=None, check=True):
        self.index = pack3d_build_index(self.params, coords, self.index, stream)
        if check:
            st = pack3d_index_check(self.index, stream)
            _check(st, "pack3d_index_check")
        return self.index

    def forward(self, q, k, v, stream=None):
        ksum, vsum = pack3d_block_summaries(self.params, self.index, k, v, stream=stream)
        return pack3d_forward(self.params, self.index, q, k, v, ksum, vsum, stream=stream)

    def window_forward(self, q, k, v, stream=None):
        return pack3d_window_forward(self.params, self.index, q, k, v, stream=stream)

    def backward(self, q, k, v, out, lse, dout, stream=None):
        return pack3d_backward(self.params, self.index, q, k, v, out, lse, dout, stream=stream)


# ---- packed sequences: dense attention and rotary positions ------------------------------

_DTYPES = {"bf16": BF16, "fp32": FP32, torch.bfloat16: BF16, torch.float32: FP32}
_TORCH_DTYPE = {BF16: torch.bfloat16, FP32: torch.float32,
                BF16 | ZERO_UNUSED_ROWS: torch.bfloat16, FP32 | ZERO_UNUSED_ROWS: torch.float32}


def make_seq_params(n_seqs: int, n_tokens: int, heads: int, kv_heads: int = None,
                    head_dim: int = 96, causal: bool = True, dtype="bf16",
                    scale: float = 0.0) -> SeqParams:
    """Params of attention over ``n_seqs`` sequences in packed tensors of
    ``n_tokens`` rows; ``kv_heads`` (default: ``heads``) divides ``heads``,
    ``scale`` 0 selects 1 / sqrt(head_dim)."""
    return SeqParams(n_seqs, n_tokens, heads, heads if kv_heads is None else kv_heads, head_dim,
                     int(bool(causal)), float(scale), _DTYPES[dtype])


def make_rotary_params(head_dim: int, rot_dim: int = None, layout: str = "half",
                       base: float = 10000.0, dtype="bf16", scaling: str = "none",
                       factor: float = 1.0, original_length: int = 0, low: float = 0.0,
                       high: float = 0.0, amplitude: float = 0.0) -> RotaryParams:
    """Params of the rotary calls; ``rot_dim`` defaults to the whole head,
    ``amplitude`` 0 selects the scaling's own.  The rows, heads and strides are
    taken from the tensors of each call."""
    return RotaryParams(head_dim=head_dim, rot_dim=head_dim if rot_dim is None else rot_dim,
                        layout=ROTARY_LAYOUTS[layout], dtype=_DTYPES[dtype], base=float(base),
                        scaling=ROTARY_SCALINGS[scaling], factor=float(factor),
                        original_length=int(original_length), low=float(low), high=float(high),
                        amplitude=float(amplitude))


class _Launch:
    """The device and stream of one packed-sequence call: every tensor on one
    device, which is current while the call launches; the given stream (of that
    device) or the device's current one.  With a given stream, buffers are
    allocated on that stream (whose earlier work may still use the memory
    otherwise) and recorded on the caller's."""

    __slots__ = ("index", "given", "raw", "before", "caller")

    def __init__(self, like, stream):
        self.index = index = like.get_device()
        if index < 0:
            raise ValueError("PACK3D tensors must be CUDA tensors")
        if stream is None:
            self.given, self.raw = None, torch._C._cuda_getCurrentRawStream(index)
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=index)
            if stream.device.index != index:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {like.device}")
            self.caller = torch.cuda.current_stream(index)
            self.given, self.raw = torch.cuda.stream(stream), stream.cuda_stream

    def __enter__(self):
        if self.given is not None:
            self.given.__enter__()  # sets the device as well
            return self
        now = torch._C._cuda_getDevice()
        self.before = None if now == self.index else now
        if self.before is not None:
            torch.cuda.set_device(self.index)
        return self

    def __exit__(self, *exc):
        if self.given is not None:
            self.given.__exit__(*exc)
        elif self.before is not None:
            torch.cuda.set_device(self.before)

    def rows(self, t, shape, dtype, what):
        """The token stride of a [rows, heads, head_dim] tensor whose heads and
        channels lie without gaps (0: nor its tokens)."""
        if t.get_device() != self.index or t.dtype is not dtype or t.shape != shape:
            raise ValueError(f"{what} must be a {dtype} tensor {tuple(shape)} on cuda:{self.index}, "
                             f"not {t.dtype} {tuple(t.shape)} on {t.device}")
        if t.is_contiguous():
            return 0
        n, h, d = shape
        s = t.stride()
        if (d > 1 and s[2] != 1) or (h > 1 and s[1] != d):
            raise ValueError(f"{what}: the heads and channels of a token must be contiguous")
        if n <= 1:
            return 0
        if s[0] < h * d or s[0] % 8:
            raise ValueError(f"{what}: the token stride {s[0]} must be a multiple of 8 and at "
                             f"least {h * d}")
        return s[0]

    def flat(self, t, shape, dtype, what):
        if t.get_device() != self.index or t.dtype is not dtype or t.shape != shape or \
                not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous {dtype} tensor {tuple(shape)} on "
                             f"cuda:{self.index}")

    def like(self, t, shape, zero):
        """An empty tensor without gaps in the shape and type of t (the quickest way
        to one: the smallest calls spend most of their time on the host).  Its rows of
        no sequence must not stay what the memory held: the call zeroes them when all
        its outputs are new, and `zero` is for the others."""
        t = self.kept(torch.empty_like(t) if t.is_contiguous() else t.new_empty(shape))
        return t.zero_() if zero else t

    def kept(self, t):
        if self.given is not None:
            t.record_stream(self.caller)
        return t


class SeqIndex:
    """A built index of a pack: the device buffer and the C struct over it."""

    def __init__(self, params: SeqParams, device=None):
        lib = load()
        nbytes = lib.pack3d_seq_index_bytes(ctypes.byref(params))
        if nbytes == 0:
            raise Pack3dError(ERR_ARG, "pack3d_seq_index_bytes")
        self.params = params
        # zeros: calls with an index that was never built find no tile
        self.buffer = torch.zeros(nbytes + 256, dtype=torch.uint8, device=device or "cuda")
        self.device = self.buffer.get_device()
        self.struct = SeqIndexStruct()
        self.builds = 0  # calls that built it: what a forward's index held when it ran
        base = self.buffer.data_ptr()
        _check(lib.pack3d_seq_index_init(ctypes.byref(params), base + (-base) % 256, nbytes,
                                         ctypes.byref(self.struct)), "pack3d_seq_index_init")

    def _rows(self, field):
        off = getattr(self.struct, field) - self.buffer.data_ptr()
        return self.buffer[off:off + 4 * self.struct.n_tokens].view(torch.int32)

    @property
    def positions(self):
        """int32 [n_tokens]: each row's position in its sequence (-1 behind the last)."""
        return self._rows("pos")

    @property
    def sequences(self):
        """int32 [n_tokens]: the number of each row's sequence (-1 behind the last)."""
        return self._rows("seq")


def pack3d_seq_build_index(params: SeqParams, cu_seqlens: torch.Tensor, index: SeqIndex = None,
                           stream=None) -> SeqIndex:
    """Index of a pack from the prefix sums of its lengths (int32 [n_seqs + 1])."""
    with _Launch(cu_seqlens, stream) as at:
        at.flat(cu_seqlens, (params.n_seqs + 1,), torch.int32, "cu_seqlens")
        if index is None:
            index = SeqIndex(params, device=cu_seqlens.device)
            at.kept(index.buffer)
        elif index.device != at.index:
            raise ValueError(f"the index is on cuda:{index.device}, not on cuda:{at.index}")
        _check(load().pack3d_seq_build_index(params, cu_seqlens.data_ptr(), index.struct, at.raw),
               "pack3d_seq_build_index")
        index.builds += 1
    return index


def pack3d_seq_index_check(index: SeqIndex, stream=None) -> int:
    """Synchronise and return the index status code (0, ERR_LENGTHS, ERR_TIMEOUT)."""
    with _Launch(index.buffer, stream) as at:
        return int(load().pack3d_seq_index_check(index.struct, at.raw))


def _zeroing(params):
    """The params of a call that zeroes its outputs' rows of no sequence."""
    p = SeqParams.from_buffer_copy(params)
    p.dtype = params.dtype | ZERO_UNUSED_ROWS
    return p


def _seq_call(params, index, at):
    if index.device != at.index:
        raise ValueError(f"the index is on cuda:{index.device}, not on cuda:{at.index}")
    n, d, dt = params.n_tokens, params.head_dim, _TORCH_DTYPE[params.dtype]
    return (n, params.Hq, d), (n, params.Hk, d), (params.Hq, n), dt


def pack3d_seq_forward(params: SeqParams, index: SeqIndex, q, k, v, out=None, lse=None,
                       stream=None):
    """Attention over every sequence of the pack: (out, lse).  q, k, v may be
    slices of one tensor (any token stride that is a multiple of 8 elements).
    Rows behind the last sequence are left as they were in a given out or lse, and
    zero in a new one."""
    with _Launch(q, stream) as at:
        qs, ks, ls, dt = _seq_call(params, index, at)
        st = SeqStrides()
        if s := at.rows(q, qs, dt, "q"):  # (a structure's field costs host time)
            st.q = s
        if s := at.rows(k, ks, dt, "k"):
            st.k = s
        if s := at.rows(v, ks, dt, "v"):
            st.v = s
        new = out is None and lse is None
        if out is None:
            out = at.like(q, qs, not new)
        else:
            st.out = at.rows(out, qs, dt, "out")
        if lse is None:
            lse = at.kept(q.new_empty(ls, dtype=torch.float32))
            if not new:
                lse.zero_()
        else:
            at.flat(lse, ls, torch.float32, "lse")
        if new:
            params = _zeroing(params)
        _check(load().pack3d_seq_forward(params, index.struct, st, q.data_ptr(), k.data_ptr(),
                                         v.data_ptr(), out.data_ptr(), lse.data_ptr(), at.raw),
               "pack3d_seq_forward")
    return out, lse


def pack3d_seq_backward_workspace_bytes(params: SeqParams) -> int:
    return int(load().pack3d_seq_backward_workspace_bytes(ctypes.byref(params)))


def pack3d_seq_backward(params: SeqParams, index: SeqIndex, q, k, v, out, lse, dout, dq=None,
                        dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) from the forward's out and lse.  Rows behind the last
    sequence are left as they were in a given gradient, and zero in a new one."""
    with _Launch(q, stream) as at:
        qs, ks, ls, dt = _seq_call(params, index, at)
        st = SeqStrides()
        if s := at.rows(q, qs, dt, "q"):
            st.q = s
        if s := at.rows(k, ks, dt, "k"):
            st.k = s
        if s := at.rows(v, ks, dt, "v"):
            st.v = s
        if s := at.rows(out, qs, dt, "out"):
            st.out = s
        if s := at.rows(dout, qs, dt, "dout"):
            st.dout = s
        at.flat(lse, ls, torch.float32, "lse")
        new = dq is None and dk is None and dv is None
        if dq is None:
            dq = at.like(q, qs, not new)
        else:
            st.dq = at.rows(dq, qs, dt, "dq")
        if dk is None:
            dk = at.like(k, ks, not new)
        else:
            st.dk = at.rows(dk, ks, dt, "dk")
        if dv is None:
            dv = at.like(v, ks, not new)
        else:
            st.dv = at.rows(dv, ks, dt, "dv")
        if new:
            params = _zeroing(params)
        if workspace is None:
            workspace = at.kept(q.new_empty(pack3d_seq_backward_workspace_bytes(params),
                                            dtype=torch.uint8))
        elif workspace.get_device() != at.index or not workspace.is_contiguous():
            raise ValueError(f"the workspace must be a contiguous tensor on cuda:{at.index}")
        _check(load().pack3d_seq_backward(params, index.struct, st, q.data_ptr(), k.data_ptr(),
                                          v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                          dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                          dv.data_ptr(), workspace.data_ptr(),
                                          workspace.numel() * workspace.element_size(), at.raw),
               "pack3d_seq_backward")
    return dq, dk, dv


def _rotary(name, params, positions, q, k, q_out, k_out, stream):
    with _Launch(q, stream) as at:
        dt, d = _TORCH_DTYPE[params.dtype], params.head_dim
        if q.dim() != 3 or (k is not None and k.dim() != 3):
            raise ValueError("q and k must be [rows, heads, head_dim]")
        n, qs = q.shape[0], (q.shape[0], q.shape[1], d)
        at.flat(positions, (n,), torch.int32, "positions")
        p = RotaryParams.from_buffer_copy(params)
        p.n_tokens, p.Hq, p.Hk = n, q.shape[1], 0
        p.stride_q = at.rows(q, qs, dt, "q")
        new = q_out is None and (k is None or k_out is None)
        if new:
            p.dtype |= ZERO_UNUSED_ROWS
        if q_out is None:
            q_out = at.like(q, qs, not new)
        else:
            p.stride_q_out = at.rows(q_out, qs, dt, "q_out")
        if k is not None:
            ks = (n, k.shape[1], d)
            p.Hk, p.stride_k = k.shape[1], at.rows(k, ks, dt, "k")
            if k_out is None:
                k_out = at.like(k, ks, not new)
            else:
                p.stride_k_out = at.rows(k_out, ks, dt, "k_out")
        _check(getattr(load(), name)(p, positions.data_ptr(), q.data_ptr(),
                                     None if k is None else k.data_ptr(), q_out.data_ptr(),
                                     None if k is None else k_out.data_ptr(), at.raw), name)
    return q_out if k is None else (q_out, k_out)


def pack3d_rotary(params: RotaryParams, positions, q, k=None, q_out=None, k_out=None,
                  stream=None):
    """Turn q [rows, heads, head_dim] and k by their rows' positions (int32);
    returns q_out, or (q_out, k_out) with k.  ``q_out=q, k_out=k`` turns them in
    place.  Rows with a negative position are left as they were in a given output,
    and zero in a new one."""
    return _rotary("pack3d_rotary", params, positions, q, k, q_out, k_out, stream)


def pack3d_rotary_backward(params: RotaryParams, positions, dq_out, dk_out=None, dq=None, dk=None,
                           stream=None):
    """Gradients of pack3d_rotary's inputs from those of its outputs."""
    return _rotary("pack3d_rotary_backward", params, positions, dq_out, dk_out, dq, dk, stream)


class _Rotated(tuple):
    """A forward's (q, k) at their positions, with the index it ran with and that
    index's count of builds."""


class SeqAttention:
    """Convenience wrapper: one pack shape, its index, and the calls; ``rotary``
    (RotaryParams) turns q and k by their positions in their sequences first.  Rows
    behind the last sequence are zero in every tensor that it makes.

    ``build_index`` rebuilds the wrapper's index in place (a captured graph then
    follows the new lengths).  Packs in flight at once, such as micro-batches whose
    backwards run later, each need an index of their own: one of
    ``pack3d_seq_build_index(op.params, cu_seqlens)``, given to ``forward``."""

    def __init__(self, params: SeqParams, rotary: RotaryParams = None):
        self.params, self.rotary, self.index = params, rotary, None

    def build_index(self, cu_seqlens, stream=None, check=True):
        self.index = pack3d_seq_build_index(self.params, cu_seqlens, self.index, stream)
        if check:
            _check(pack3d_seq_index_check(self.index, stream), "pack3d_seq_index_check")
        return self.index

    def rotate(self, q, k, stream=None, index=None):
        """q and k at their positions (as they are without ``rotary``)."""
        if self.rotary is None:
            return q, k
        index = self.index if index is None else index
        return pack3d_rotary(self.rotary, index.positions, q, k, stream=stream)

    def forward(self, q, k, v, stream=None, index=None):
        """(out, lse, (q, k) at their positions, which the backward takes), with the
        wrapper's index or the given one."""
        index = self.index if index is None else index
        rotated = _Rotated(self.rotate(q, k, stream, index))
        rotated.index = index
        # (a captured forward runs with whatever the index holds at each replay)
        rotated.builds = None if torch.cuda.is_current_stream_capturing() else index.builds
        return (*pack3d_seq_forward(self.params, index, *rotated, v, stream=stream), rotated)

    def backward(self, rotated, v, out, lse, dout, stream=None, index=None):
        """(dq, dk, dv) with the index of the forward that gave ``rotated``; ValueError
        if a call has built that index anew since (not seen: replays of a captured build,
        and builds after a captured forward, whose replays follow them).  For a plain pair
        (q, k): with the given index, or the wrapper's."""
        if isinstance(rotated, _Rotated):
            if index is not None and index is not rotated.index:
                raise ValueError("the forward ran with another index")
            index = rotated.index
            if rotated.builds not in (None, index.builds):
                raise ValueError("the index was built anew after the forward: its sequences may "
                                 "not be the forward's (give each pack in flight its own index)")
        elif index is None:
            index = self.index
        qr, kr = rotated
        dq, dk, dv = pack3d_seq_backward(self.params, index, qr, kr, v, out, lse, dout,
                                         stream=stream)
        if self.rotary is not None:
            pack3d_rotary_backward(self.rotary, index.positions, dq, dk, dq, dk, stream)
        return dq, dk, dv
