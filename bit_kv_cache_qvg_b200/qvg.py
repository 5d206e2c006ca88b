"""Thin ctypes binding of libqvg.so (the C ABI in include/qvg.h).

Argument marshalling only: every step of the codec runs in the library's
CUDA kernels.  PyTorch supplies device memory and streams.  If the library is
missing, every call raises ``QvgError`` -- there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqvg.so")

BF16, FP32 = 0, 1
_DTYPES = {torch.bfloat16: BF16, torch.float32: FP32}
_TORCH = {BF16: torch.bfloat16, FP32: torch.float32}

STATUS = {
    0: "QVG_OK", 1: "QVG_ERR_INVALID_ARG", 2: "QVG_ERR_UNSUPPORTED", 3: "QVG_ERR_NO_MEMORY",
    4: "QVG_ERR_CUDA", 5: "QVG_ERR_DEVICE_TIMEOUT", 6: "QVG_ERR_WORKSPACE_TOO_SMALL",
    7: "QVG_ERR_CAPACITY",
}


class QvgError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}" if what else STATUS.get(status, str(status)))


ASYM, SYM = 0, 1     # qvg_scale_mode: scale and zero point per group, or one scale per group


class Config(C.Structure):
    _fields_ = [("K", C.c_int32), ("T", C.c_int32), ("group_size", C.c_int32),
                ("bits", C.c_int32), ("iters", C.c_int32), ("warm_iters", C.c_int32),
                ("scale_mode", C.c_int32)]

    def __repr__(self):
        return (f"Config(K={self.K}, T={self.T}, group_size={self.group_size}, bits={self.bits}, "
                f"iters={self.iters}, warm_iters={self.warm_iters}, scale_mode={self.scale_mode})")


class Policy(C.Structure):
    """qvg_adaptive_policy: a ladder of (T, group_size) settings chosen per
    chunk from the mean E4M3 code of the chunk's group ranges."""
    _fields_ = [("levels", C.c_int32), ("T", C.c_int32 * 4), ("group_size", C.c_int32 * 4),
                ("thresholds", C.c_int32 * 3), ("probe_group", C.c_int32), ("refresh_every", C.c_int32)]


def policy(T, group_size, thresholds=(), probe_group=16, refresh_every=0) -> Policy:
    """A policy of len(T) levels; thresholds in sixteenths of an E4M3 code."""
    p = Policy()
    p.levels = len(T)
    if not 1 <= p.levels <= 4 or len(group_size) != p.levels or len(thresholds) != p.levels - 1:
        raise QvgError(1, "policy: 1-4 levels, one group size per level, levels - 1 thresholds")
    for i in range(p.levels):
        p.T[i], p.group_size[i] = T[i], group_size[i]
    for i, t in enumerate(thresholds):
        p.thresholds[i] = t
    p.probe_group, p.refresh_every = probe_group, refresh_every
    return p


class _Packed(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scale", C.c_void_p), ("zero", C.c_void_p),
                ("assign", C.c_void_p), ("centroids", C.c_void_p)]


class _Batch(C.Structure):
    _fields_ = [("B", C.c_int32), ("group", C.c_int32), ("Nq", C.c_int64), ("Nt", C.c_int64), ("Q", C.c_void_p),
                ("q_pos", C.c_void_p), ("k_pos", C.c_void_p), ("tail_k", C.c_void_p), ("tail_v", C.c_void_p),
                ("tail_pos", C.c_void_p), ("tail_len", C.c_void_p), ("causal", C.c_int32)]


_lib = None

# Every exported symbol of include/qvg.h with its ctypes signature.
_SIGS = {
    "qvg_status_string": (C.c_char_p, [C.c_int]),
    "qvg_version": (C.c_char_p, []),
    "qvg_packed_bytes": (C.c_size_t, [C.POINTER(Config), C.c_int64, C.c_int32, C.c_int32, C.c_int]),
    "qvg_workspace_bytes": (C.c_size_t, [C.POINTER(Config), C.c_int64, C.c_int32, C.c_int32, C.c_int]),
    "qvg_quantize": (C.c_int, [C.POINTER(Config), C.c_void_p, C.c_int, C.c_int64, C.c_int32, C.c_int32,
                               C.c_void_p, C.POINTER(_Packed), C.c_void_p, C.c_size_t, C.c_void_p]),
    "qvg_quantize_static": (C.c_int, [C.POINTER(Config), C.c_void_p, C.c_int, C.c_int64, C.c_int32,
                                      C.c_int32, C.c_void_p, C.POINTER(_Packed), C.c_void_p]),
    "qvg_dequantize": (C.c_int, [C.POINTER(Config), C.POINTER(_Packed), C.c_int, C.c_int64, C.c_int32,
                                 C.c_int32, C.c_void_p, C.c_void_p]),
    "qvg_workspace_status": (C.c_int, [C.c_void_p, C.c_size_t, C.c_void_p]),
    "qvg_workspace_flagged": (C.c_int64, [C.c_void_p, C.c_size_t, C.c_void_p]),
    "qvg_cache_create": (C.c_int, [C.POINTER(Config), C.c_int, C.c_int32, C.c_int32, C.c_int64, C.c_int32,
                                   C.c_int64, C.POINTER(C.c_void_p)]),
    "qvg_cache_create_adaptive": (C.c_int, [C.POINTER(Config), C.POINTER(Policy), C.c_int, C.c_int32, C.c_int32,
                                            C.c_int64, C.c_int32, C.c_int64, C.POINTER(C.c_void_p)]),
    "qvg_cache_chunk_info": (C.c_int, [C.c_void_p, C.c_int32, C.POINTER(C.c_int32), C.POINTER(C.c_int32),
                                       C.POINTER(C.c_int32), C.POINTER(C.c_uint64)]),
    "qvg_cache_status": (C.c_int, [C.c_void_p, C.c_void_p]),
    "qvg_static_status": (C.c_int, [C.c_void_p]),
    "qvg_append_chunk": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p]),
    "qvg_cache_dequantize": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p]),
    "qvg_cache_tokens": (C.c_int64, [C.c_void_p]),
    "qvg_cache_chunks": (C.c_int32, [C.c_void_p]),
    "qvg_cache_chunk_view": (C.c_int, [C.c_void_p, C.c_int32, C.POINTER(_Packed), C.POINTER(C.c_int64),
                                       C.POINTER(C.c_int64)]),
    "qvg_cache_device_bytes": (C.c_size_t, [C.c_void_p]),
    "qvg_cache_destroy": (None, [C.c_void_p]),
    "qvg_rope_tables_bytes": (C.c_size_t, [C.c_int32, C.c_int64]),
    "qvg_rope_tables": (C.c_int, [C.c_double, C.c_int32, C.c_int64, C.c_void_p, C.c_size_t, C.c_void_p]),
    "qvg_attention": (C.c_int, [C.POINTER(Config), C.POINTER(_Packed), C.POINTER(_Packed), C.c_int64, C.c_int32,
                                C.c_int32, C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p, C.c_size_t, C.c_void_p,
                                C.c_void_p, C.c_size_t, C.c_void_p]),
    "qvg_attention_set_split": (C.c_int32, [C.c_int32]),
    "qvg_attention_split": (C.c_int32, [C.POINTER(Config), C.c_int64, C.c_int32, C.c_int64, C.c_size_t]),
    "qvg_attention_workspace_bytes": (C.c_size_t, [C.POINTER(Config), C.c_int64, C.c_int32, C.c_int64]),
    "qvg_attention_batch": (C.c_int, [C.POINTER(Config), C.POINTER(_Packed), C.POINTER(_Packed), C.c_int64, C.c_int32,
                                      C.c_int32, C.POINTER(_Batch), C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p,
                                      C.c_size_t, C.c_void_p]),
    "qvg_attention_weights": (C.c_int, [C.POINTER(Config), C.POINTER(_Packed), C.c_int64, C.c_int32, C.c_int32,
                                        C.POINTER(_Batch), C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p, C.c_void_p,
                                        C.c_size_t, C.c_void_p]),
    "qvg_attention_batch_workspace_bytes": (C.c_size_t, [C.POINTER(Config), C.c_int64, C.c_int32, C.POINTER(_Batch)]),
    "qvg_attention_weights_workspace_bytes": (C.c_size_t, [C.POINTER(Config), C.c_int64, C.c_int32,
                                                           C.POINTER(_Batch)]),
    "qvg_evict": (C.c_int, [C.POINTER(Config), C.POINTER(_Packed), C.POINTER(_Packed), C.c_int64, C.c_int32, C.c_int32,
                            C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.POINTER(_Packed),
                            C.POINTER(_Packed), C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "qvg_profile_enable": (None, [C.c_int]),
    "qvg_profile_reset": (None, []),
    "qvg_profile_launches": (C.c_int64, []),
    "qvg_profile_report": (C.c_int, [C.c_char_p, C.c_size_t]),
}


def lib():
    """Load libqvg.so (raises QvgError if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise QvgError(4, f"libqvg.so not found at {LIB_PATH}; run "
                              "python -m bit_kv_cache_qvg_b200.build")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return sorted(_SIGS)


def status_string(st: int) -> str:
    return lib().qvg_status_string(st).decode()


def _check(st: int, what: str):
    if st != 0:
        raise QvgError(st, what)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _torch_stream(stream, dev):
    """`stream` (a torch stream or a handle) as a torch stream of `dev`."""
    if isinstance(stream, torch.cuda.Stream):
        if dev.index is not None and stream.device != dev:
            raise QvgError(1, f"the stream must be one of {dev}")
        return stream
    handle = int(getattr(stream, "cuda_stream", stream))
    return torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)


def _memory(stream, dev, make, *args, **kw):
    """make(*args, **kw), memory for work on `stream` (None: the current one), from that
    stream's own blocks: a block that the current stream has let go of may still be in
    use by what is queued there, and nothing orders `stream` behind it."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(_torch_stream(stream, dev)):
        return make(*args, **kw)


def _returned(stream, dev, *tensors):
    """Tensors allocated for `stream` that the caller gets: not reused before what
    the caller's current stream has queued when they are freed."""
    if stream is not None:
        s = torch.cuda.current_stream(dev)
        for t in tensors:
            if t.numel():
                t.record_stream(s)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def config(K=256, T=2, group_size=64, iters=10, warm_iters=3, bits=2, scale_mode=ASYM) -> Config:
    return Config(K, T, group_size, bits, iters, warm_iters, scale_mode)


# Named operating points.  With one E4M3 scale per group the closed-form
# compression at K = 256 on a 38,000-token block is 6.97x for "qvg" and
# 5.03x for "qvg-pro" (the m.163.com article on Quant VideoGen, section 六,
# reports 6.94-7.05x and 4.97-5.20x; section 七 names G = 64 the best
# trade-off and G = 16 the high-quality setting).  The pages do not print the
# settings themselves: these are the ones the closed form admits.
PRESETS = {
    "qvg": dict(K=256, T=1, group_size=64, scale_mode=SYM),
    "qvg-pro": dict(K=256, T=4, group_size=16, scale_mode=SYM),
}


def preset(name: str, iters=10, warm_iters=3) -> Config:
    return config(iters=iters, warm_iters=warm_iters, **PRESETS[name])


@dataclass
class Packed:
    """Packed tensors of H blocks of N tokens (layouts of qvg_packed)."""
    codes: torch.Tensor       # [H][N][d/4] uint8
    scale: torch.Tensor       # [H][N][d/G] uint8 (E4M3)
    zero: torch.Tensor        # [H][N][d/G] uint8 (E4M3)
    assign: torch.Tensor      # [T][H][N] uint8
    centroids: torch.Tensor   # [T][H][K][d] storage dtype
    cfg: Config
    N: int
    H: int
    d: int
    dtype: int

    def struct(self) -> _Packed:
        """The tensors' addresses (0 for an empty one).  The library takes them as
        contiguous arrays of these sizes: a tensor that is not one is refused."""
        cfg, codes, scale, zero, assign, tables = self.cfg, self.codes, self.scale, self.zero, self.assign, self.centroids
        T, d, tokens, device = cfg.T, self.d, self.H * self.N, codes.get_device()
        groups = tokens * (d // (cfg.group_size or 1))
        row = cfg.K * d * (2 if self.dtype == BF16 else 4)
        if codes.nbytes * 4 != tokens * d or not codes.is_contiguous():
            self._refuse("codes")
        if scale.nbytes != groups or not scale.is_contiguous() or scale.get_device() != device:
            self._refuse("scale")
        if cfg.scale_mode == ASYM and (zero.nbytes != groups or not zero.is_contiguous() or zero.get_device() != device):
            self._refuse("zero")
        if T > 0 and (assign.nbytes != T * tokens or not assign.is_contiguous() or assign.get_device() != device):
            self._refuse("assign")
        if T > 0 and (tables.nbytes != T * self.H * row or not tables.is_contiguous() or tables.get_device() != device):
            self._refuse("centroids")
        return _Packed(codes.data_ptr(), scale.data_ptr(), zero.data_ptr(), assign.data_ptr(), tables.data_ptr())

    def _refuse(self, name: str):
        raise QvgError(1, f"{name} must be a contiguous tensor of the packed form's sizes, on the device of codes")

    def _addresses(self) -> _Packed:
        """struct of tensors that were allocated for these sizes just now."""
        return _Packed(self.codes.data_ptr(), self.scale.data_ptr(), self.zero.data_ptr(), self.assign.data_ptr(),
                       self.centroids.data_ptr())

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.codes, self.scale, self.zero, self.assign, self.centroids))


def packed_bytes(cfg: Config, N: int, H: int, d: int = 128, dtype: int = BF16) -> int:
    return int(lib().qvg_packed_bytes(C.byref(cfg), N, H, d, dtype))


def workspace_bytes(cfg: Config, N: int, H: int, d: int = 128, dtype: int = BF16) -> int:
    return int(lib().qvg_workspace_bytes(C.byref(cfg), N, H, d, dtype))


def alloc_packed(cfg: Config, N: int, H: int, d: int = 128, dtype: int = BF16, device="cuda") -> Packed:
    G, T, K = cfg.group_size, cfg.T, cfg.K
    u8 = dict(dtype=torch.uint8, device=device)
    return Packed(
        codes=torch.empty((H, N, d // 4), **u8),
        scale=torch.empty((H, N, d // G), **u8),
        zero=torch.empty((H, N, d // G) if cfg.scale_mode == ASYM else (0,), **u8),
        assign=torch.empty((T, H, N), **u8),
        centroids=torch.empty((T, H, K, d), dtype=_TORCH[dtype], device=device),
        cfg=cfg, N=N, H=H, d=d, dtype=dtype)


def alloc_workspace(cfg: Config, N: int, H: int, d: int = 128, dtype: int = BF16, device="cuda"):
    n = workspace_bytes(cfg, N, H, d, dtype)
    if n == 0:
        raise QvgError(1, "workspace size")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:16].zero_()     # status word and near-tie counter
    return ws


def _new_packed(cfg: Config, N: int, H: int, d: int, dtype: int, dev, stream) -> Packed:
    """alloc_packed for the result of work on `stream`."""
    p = _memory(stream, dev, alloc_packed, cfg, N, H, d, dtype, dev)
    _returned(stream, dev, p.codes, p.scale, p.zero, p.assign, p.centroids)
    return p


def quantize(X: torch.Tensor, cfg: Config, init: Optional[torch.Tensor] = None,
             out: Optional[Packed] = None, workspace: Optional[torch.Tensor] = None,
             stream=None) -> Packed:
    """qvg_quantize on X [H][N][d] (bf16 or fp32, CUDA, contiguous)."""
    if X.dim() != 3 or not X.is_contiguous():
        raise QvgError(1, "X must be a contiguous [H][N][d] tensor")
    H, N, d = X.shape
    dt = _DTYPES[X.dtype]
    if out is None:
        out = _new_packed(cfg, N, H, d, dt, X.device, stream)
    if workspace is None:
        workspace = _memory(stream, X.device, alloc_workspace, cfg, N, H, d, dt, X.device)
    ps = out.struct()
    st = lib().qvg_quantize(C.byref(cfg), _ptr(X), dt, N, H, d, _ptr(init), C.byref(ps),
                            _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "qvg_quantize")
    return out


def quantize_static(X: torch.Tensor, cfg: Config, init: Optional[torch.Tensor] = None,
                    out: Optional[Packed] = None, stream=None) -> Packed:
    """qvg_quantize_static on X [H][N][d]: no workspace argument; the library's
    per-device static reserve is the scratch (calls must not overlap)."""
    if X.dim() != 3 or not X.is_contiguous():
        raise QvgError(1, "X must be a contiguous [H][N][d] tensor")
    H, N, d = X.shape
    dt = _DTYPES[X.dtype]
    if out is None:
        out = _new_packed(cfg, N, H, d, dt, X.device, stream)
    ps = out.struct()
    st = lib().qvg_quantize_static(C.byref(cfg), _ptr(X), dt, N, H, d, _ptr(init), C.byref(ps), _stream(stream))
    _check(st, "qvg_quantize_static")
    return out


def dequantize(p: Packed, Y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    if Y is None:
        Y = _memory(stream, p.codes.device, torch.empty, (p.H, p.N, p.d), dtype=_TORCH[p.dtype], device=p.codes.device)
        _returned(stream, p.codes.device, Y)
    ps = p.struct()
    st = lib().qvg_dequantize(C.byref(p.cfg), C.byref(ps), p.dtype, p.N, p.H, p.d, _ptr(Y), _stream(stream))
    _check(st, "qvg_dequantize")
    return Y


def rope_tables(max_pos: int, base: float = 10000.0, d: int = 128, device="cuda", stream=None) -> torch.Tensor:
    """qvg_rope_tables: the rotary (cos, sin) tables for positions 0 .. max_pos
    (a uint8 device tensor; its first 4 bytes are the attention status word)."""
    n = int(lib().qvg_rope_tables_bytes(d, max_pos))
    if n == 0:
        raise QvgError(1, "qvg_rope_tables_bytes")
    device = torch.device(device)
    t = _memory(stream, device, torch.empty, n, dtype=torch.uint8, device=device)
    _returned(stream, device, t)
    _check(lib().qvg_rope_tables(float(base), d, max_pos, _ptr(t), n, _stream(stream)), "qvg_rope_tables")
    return t


def attention(kp: Packed, vp: Packed, Q: torch.Tensor, q_pos: torch.Tensor, tables: torch.Tensor,
              O: Optional[torch.Tensor] = None, stream=None, workspace=True) -> torch.Tensor:
    """qvg_attention: softmax(rope(Q) rope(K^)^T / sqrt(d)) V^ per head over the
    compressed caches kp (keys, before the rotary embedding) and vp (values);
    Q [H][Nq][d] bf16, q_pos [Nq] int64 (device); returns O [H][Nq][d] fp32.
    `workspace`: a uint8 device tensor, True (one of
    qvg_attention_workspace_bytes is allocated) or None (no workspace)."""
    if Q.dim() != 3 or not Q.is_contiguous() or Q.dtype != torch.bfloat16:
        raise QvgError(1, "Q must be a contiguous bf16 [H][Nq][d] tensor")
    H, Nq, d = Q.shape
    if O is None:
        O = _memory(stream, Q.device, torch.empty, (H, Nq, d), dtype=torch.float32, device=Q.device)
        _returned(stream, Q.device, O)
    if workspace is True:
        n = attention_workspace_bytes(kp.cfg, kp.N, H, Nq)
        workspace = _memory(stream, Q.device, torch.empty, n, dtype=torch.uint8, device=Q.device) if n > 0 else None
    ws_ptr, ws_n = (_ptr(workspace), workspace.numel()) if workspace is not None else (None, 0)
    ks, vs = kp.struct(), vp.struct()
    _check(lib().qvg_attention(C.byref(kp.cfg), C.byref(ks), C.byref(vs), kp.N, H, d, _ptr(Q),
                               _ptr(q_pos), Nq, _ptr(tables), tables.numel(), _ptr(O), ws_ptr, ws_n,
                               _stream(stream)),
           "qvg_attention")
    return O


def attention_set_split(split: int) -> int:
    """qvg_attention_set_split: fix the cluster split of qvg_attention for the
    process (1 .. 8; 0 = the library's choice); returns the previous setting."""
    prev = int(lib().qvg_attention_set_split(int(split)))
    if prev < 0:
        raise QvgError(1, "qvg_attention_set_split")
    return prev


def attention_split(cfg: Config, Nk: int, H: int, Nq: int, ws_bytes: int = 0) -> int:
    """qvg_attention_split: the ranges the cache of a query block is cut into
    by a qvg_attention call with these sizes and a workspace of ws_bytes."""
    n = int(lib().qvg_attention_split(C.byref(cfg), Nk, H, Nq, ws_bytes))
    if n < 0:
        raise QvgError(1, "qvg_attention_split")
    return n


def attention_workspace_bytes(cfg: Config, Nk: int, H: int, Nq: int) -> int:
    """qvg_attention_workspace_bytes: the workspace the preferred cut needs."""
    return int(lib().qvg_attention_workspace_bytes(C.byref(cfg), Nk, H, Nq))


@dataclass
class Tail:
    """Each sequence's own newest tokens, not compressed (the tail of a qvg_batch):
    k, v [B][H][Nt][d] bf16 (k before the rotary embedding; v is not read by
    attention_weights), pos [B][Nt] int64 (None: Nk + i) and length [B] int32
    (None: Nt), the tokens each tail holds."""
    k: torch.Tensor
    v: Optional[torch.Tensor] = None
    pos: Optional[torch.Tensor] = None
    length: Optional[torch.Tensor] = None


def _device_tensor(t: Optional[torch.Tensor], what: str, dtype, shape, device) -> int:
    """Check an argument's type, shape, layout and device; its address (None: 0)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise QvgError(1, f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _batch(p: Packed, Q: torch.Tensor, q_pos: torch.Tensor, k_pos, tail: Optional[Tail], causal: bool, values: bool,
           device) -> _Batch:
    if p.dtype != BF16:
        raise QvgError(2, "the cache must be a bf16 one")
    if Q.dim() != 4 or Q.shape[1] % p.H != 0 or Q.shape[3] != p.d:
        raise QvgError(1, "Q must be a [B][H * group][Nq][d] tensor")
    B, Hq, Nq, d = Q.shape
    H = p.H
    at_q, at_pos = _device_tensor(Q, "Q", torch.bfloat16, Q.shape, device), _device_tensor(q_pos, "q_pos", torch.int64, (B, Nq), device)
    at_k = _device_tensor(k_pos, "k_pos", torch.int64, (H, p.N), device)
    if tail is None:
        return _Batch(B, Hq // H, Nq, 0, at_q, at_pos, at_k, 0, 0, 0, 0, 1 if causal else 0)
    k = tail.k
    if k.dim() != 4:
        raise QvgError(1, "the tail's k must be a [B][H][Nt][d] tensor")
    Nt = k.shape[2]
    shape = (B, H, Nt, d)
    if values and tail.v is None:
        raise QvgError(1, "the tail has no values")
    return _Batch(B, Hq // H, Nq, Nt, at_q, at_pos, at_k, _device_tensor(k, "the tail's k", torch.bfloat16, shape, device),
                  _device_tensor(tail.v, "the tail's v", torch.bfloat16, shape, device),
                  _device_tensor(tail.pos, "the tail's pos", torch.int64, (B, Nt), device),
                  _device_tensor(tail.length, "the tail's length", torch.int32, (B,), device), 1 if causal else 0)


def _on_device(*tensors):
    """The device of the first tensor, a CUDA one, with the others on it."""
    dev = tensors[0].device
    if dev.type != "cuda" or any(t.device != dev for t in tensors):
        raise QvgError(1, "every tensor must be on the cache's CUDA device")
    return dev


def _same_kind(kp: Packed, vp: Packed):
    if vp.N != kp.N or vp.H != kp.H or vp.d != kp.d or vp.dtype != kp.dtype or \
            (vp.cfg is not kp.cfg and bytes(vp.cfg) != bytes(kp.cfg)):
        raise QvgError(1, "kp and vp must have the same sizes and configuration")


def _queue(dev, stream, call, *args) -> int:
    """call(*args, stream) with `dev` as the current device; stream None: its current one."""
    if torch.cuda.current_device() == dev.index:
        return call(*args, torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else _stream(stream))
    with torch.cuda.device(dev):
        return call(*args, _stream(stream))


def _workspace(workspace, size_call, p: Packed, b: _Batch, dev, stream) -> torch.Tensor:
    if workspace is None:
        if torch.cuda.current_device() == dev.index:
            need = size_call(C.byref(p.cfg), p.N, p.H, C.byref(b))
        else:
            with torch.cuda.device(dev):
                need = size_call(C.byref(p.cfg), p.N, p.H, C.byref(b))
        workspace = _memory(stream, dev, p.codes.new_empty, need)
    elif workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or workspace.device != dev:
        raise QvgError(1, f"the workspace must be a contiguous uint8 tensor on {dev}")
    return workspace


def _tables(tables: torch.Tensor) -> torch.Tensor:
    if tables.dtype is not torch.uint8 or tables.dim() != 1 or not tables.is_contiguous():
        raise QvgError(1, "tables must be a tensor of rope_tables")
    return tables


def attention_batch(kp: Packed, vp: Packed, Q: torch.Tensor, q_pos: torch.Tensor, tables: torch.Tensor,
                    tail: Optional[Tail] = None, k_pos: Optional[torch.Tensor] = None, causal: bool = False,
                    O: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """qvg_attention_batch: attention of B sequences over the compressed prefix
    they share (kp, vp: H blocks), joined with each one's own tail.
    Q [B][H * group][Nq][d] bf16 and q_pos [B][Nq] int64 (negative: a padding
    row); k_pos [H][N] int64, the cached tokens' positions (None: 0 .. N-1);
    returns O, like Q, zeros in rows that see no key.  `workspace`: a uint8
    tensor of attention_batch_workspace_bytes (None: allocated here), or a smaller
    one, down to what that gives for H = 1: fewer heads at a time."""
    dev = kp.codes.device
    b = _batch(kp, Q, q_pos, k_pos, tail, causal, True, dev)
    _same_kind(kp, vp)
    _device_tensor(O, "O", torch.bfloat16, Q.shape, dev)
    _on_device(kp.codes, vp.codes, _tables(tables))
    L = lib()
    ws = _workspace(workspace, L.qvg_attention_batch_workspace_bytes, kp, b, dev, stream)
    if O is None:
        O = _memory(stream, dev, torch.empty_like, Q)
        _returned(stream, dev, O)
    _check(_queue(dev, stream, L.qvg_attention_batch, C.byref(kp.cfg), C.byref(kp.struct()), C.byref(vp.struct()), kp.N, kp.H, kp.d,
                  C.byref(b), tables.data_ptr(), tables.numel(), O.data_ptr(), ws.data_ptr(), ws.numel()), "qvg_attention_batch")
    return O


def attention_weights(kp: Packed, Q: torch.Tensor, q_pos: torch.Tensor, tables: torch.Tensor,
                      received: Optional[torch.Tensor] = None, tail: Optional[Tail] = None,
                      k_pos: Optional[torch.Tensor] = None, causal: bool = False, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """qvg_attention_weights: received [H][N] fp32 (None: zeros) plus the softmax
    weight that each token of the prefix gets from the batch's rows (arguments
    as attention_batch).  `out` may be `received`, to add in place."""
    dev = kp.codes.device
    b = _batch(kp, Q, q_pos, k_pos, tail, causal, False, dev)
    shape = (kp.H, kp.N)
    _device_tensor(out, "out", torch.float32, shape, dev)
    before = _device_tensor(received, "received", torch.float32, shape, dev)
    _on_device(kp.codes, _tables(tables))
    L = lib()
    ws = _workspace(workspace, L.qvg_attention_weights_workspace_bytes, kp, b, dev, stream)
    if out is None:
        out = _memory(stream, dev, torch.empty, shape, dtype=torch.float32, device=dev)
        _returned(stream, dev, out)
    _check(_queue(dev, stream, L.qvg_attention_weights, C.byref(kp.cfg), C.byref(kp.struct()), kp.N, kp.H, kp.d, C.byref(b),
                  tables.data_ptr(), tables.numel(), before, out.data_ptr(), ws.data_ptr(), ws.numel()),
           "qvg_attention_weights")
    return out


def _batch_sizes(B: int, group: int, Nq: int, Nt: int) -> _Batch:
    return _Batch(B=B, group=group, Nq=Nq, Nt=Nt)


def attention_batch_workspace_bytes(cfg: Config, Nk: int, H: int, B: int, group: int, Nq: int, Nt: int = 0) -> int:
    """qvg_attention_batch_workspace_bytes for these sizes."""
    return int(lib().qvg_attention_batch_workspace_bytes(C.byref(cfg), Nk, H, C.byref(_batch_sizes(B, group, Nq, Nt))))


def attention_weights_workspace_bytes(cfg: Config, Nk: int, H: int, B: int, group: int, Nq: int, Nt: int = 0) -> int:
    """qvg_attention_weights_workspace_bytes for these sizes."""
    return int(lib().qvg_attention_weights_workspace_bytes(C.byref(cfg), Nk, H, C.byref(_batch_sizes(B, group, Nq, Nt))))


@dataclass
class Evicted:
    """What evict leaves: the closed-up caches, and of every kept token its
    index before, its position and its weight."""
    k: Packed
    v: Packed
    kept: torch.Tensor        # [H][keep] int32, ascending
    pos: torch.Tensor         # [H][keep] int64
    weights: torch.Tensor     # [H][keep] fp32


def _closed(kp: Packed, vp: Packed, keep: int):
    """Streams for `keep` tokens a head beside kp's and vp's own centroid tables,
    in one allocation, each stream from a 256-byte boundary."""
    H, d, T = kp.H, kp.d, kp.cfg.T
    w, ng = d // 4, d // kp.cfg.group_size
    n = H * keep
    codes, groups, assign = (n * w + 255) & -256, (n * ng + 255) & -256, (n * T + 255) & -256
    asym = kp.cfg.scale_mode == ASYM
    size = codes + groups * (2 if asym else 1) + assign
    cut = kp.codes.new_empty(2 * size).as_strided
    by_code, by_group, by_token = (keep * w, w, 1), (keep * ng, ng, 1), (n, keep, 1)
    out = []
    for p, at in ((kp, 0), (vp, size)):
        scale = at + codes
        out.append(Packed(cut((H, keep, w), by_code, at), cut((H, keep, ng), by_group, scale),
                          cut((H, keep, ng), by_group, scale + groups) if asym else p.zero,
                          cut((T, H, keep), by_token, at + size - assign), p.centroids, p.cfg, keep, H, d, p.dtype))
    return out


def _evicted(kp: Packed, vp: Packed, weights: torch.Tensor, keep: int) -> Evicted:
    shape, new = (kp.H, keep), weights.new_empty
    return Evicted(*_closed(kp, vp, keep), new(shape, dtype=torch.int32), new(shape, dtype=torch.int64), new(shape))


def evict(kp: Packed, vp: Packed, weights: torch.Tensor, keep: int, first: int = 0, recent: int = 0,
          k_pos: Optional[torch.Tensor] = None, stream=None) -> Evicted:
    """qvg_evict: keep the first `first` and the last `recent` tokens of every
    head and, up to `keep` in all, those with the largest weights [H][N] fp32.
    The caches returned share the centroid tables of kp and vp."""
    _same_kind(kp, vp)
    if not 1 <= keep <= kp.N or first < 0 or recent < 0 or first + recent > keep:
        raise QvgError(1, "keep must be 1 .. N, first + recent at most keep")
    dev, shape = kp.codes.device, (kp.H, kp.N)
    at_w = _device_tensor(weights, "weights", torch.float32, shape, dev)
    at_pos = _device_tensor(k_pos, "k_pos", torch.int64, shape, dev)
    _on_device(kp.codes, vp.codes)
    ks, vs = kp.struct(), vp.struct()
    e = _memory(stream, dev, _evicted, kp, vp, weights, keep)
    k, v = e.k, e.v
    _returned(stream, dev, e.kept, e.pos, e.weights, k.codes)       # both caches' streams are one allocation
    _check(_queue(dev, stream, lib().qvg_evict, C.byref(kp.cfg), C.byref(ks), C.byref(vs), kp.N, kp.H, kp.d, at_w,
                  at_pos, keep, first, recent, C.byref(k._addresses()), C.byref(v._addresses()), e.kept.data_ptr(),
                  e.pos.data_ptr(), e.weights.data_ptr()), "qvg_evict")
    return e


def profile_enable(on: bool = True):
    lib().qvg_profile_enable(1 if on else 0)


def profile_reset():
    lib().qvg_profile_reset()


def profile_launches() -> int:
    return int(lib().qvg_profile_launches())


def profile_report() -> dict:
    import json
    n = lib().qvg_profile_report(None, 0)
    buf = C.create_string_buffer(max(n, 2))
    st = lib().qvg_profile_report(buf, len(buf))
    if st != 0:
        raise QvgError(4, "qvg_profile_report")
    return json.loads(buf.value.decode())


def workspace_flagged(workspace: torch.Tensor, stream=None) -> int:
    return int(lib().qvg_workspace_flagged(_ptr(workspace), workspace.numel(), _stream(stream)))


def workspace_status(workspace: torch.Tensor, stream=None) -> int:
    return int(lib().qvg_workspace_status(_ptr(workspace), workspace.numel(), _stream(stream)))


def static_status(stream=None) -> int:
    """qvg_static_status: read and clear the static reserve's status word."""
    return int(lib().qvg_static_status(_stream(stream)))


class _DevView:
    """__cuda_array_interface__ wrapper of a raw device pointer (for views)."""

    def __init__(self, ptr: int, shape, typestr: str):
        self.__cuda_array_interface__ = dict(shape=tuple(shape), typestr=typestr, data=(ptr, False),
                                             version=3, strides=None)


def _view(ptr, shape, torch_dtype):
    if ptr is None or 0 in shape:
        return torch.empty(shape, dtype=torch_dtype, device="cuda")
    typestr = {torch.uint8: "|u1", torch.float32: "<f4", torch.bfloat16: "<u2"}[torch_dtype]
    t = torch.as_tensor(_DevView(ptr, shape, typestr), device="cuda")
    return t.view(torch.bfloat16) if torch_dtype == torch.bfloat16 else t


class Cache:
    """Streaming compressed KV cache (qvg_cache_*): append chunks, each
    warm-started from the previous chunk's centroids; dequantise all.  With a
    Policy (qvg_cache_create_adaptive) every chunk takes its own T and G."""

    def __init__(self, cfg: Config, H: int, max_tokens: int, max_chunks: int, d: int = 128,
                 dtype: int = BF16, max_chunk_tokens: int = 0, policy: Optional[Policy] = None):
        self.cfg, self.H, self.d, self.dtype, self.policy = cfg, H, d, dtype, policy
        self._h = C.c_void_p()
        h = C.c_void_p()
        if policy is None:
            _check(lib().qvg_cache_create(C.byref(cfg), dtype, H, d, max_tokens, max_chunks, max_chunk_tokens,
                                          C.byref(h)), "qvg_cache_create")
        else:
            _check(lib().qvg_cache_create_adaptive(C.byref(cfg), C.byref(policy), dtype, H, d, max_tokens,
                                                   max_chunks, max_chunk_tokens, C.byref(h)),
                   "qvg_cache_create_adaptive")
        self._h = h

    def chunk_info(self, c: int) -> dict:
        """qvg_cache_chunk_info: level, T, G and statistic of chunk c."""
        lvl, T, G, S = C.c_int32(), C.c_int32(), C.c_int32(), C.c_uint64()
        _check(lib().qvg_cache_chunk_info(self._h, c, C.byref(lvl), C.byref(T), C.byref(G), C.byref(S)),
               "qvg_cache_chunk_info")
        return dict(level=lvl.value, T=T.value, G=G.value, stat=S.value)

    def append(self, X: torch.Tensor, stream=None):
        if X.dim() != 3 or X.shape[0] != self.H or X.shape[2] != self.d or not X.is_contiguous():
            raise QvgError(1, "chunk must be a contiguous [H][N][d] tensor")
        _check(lib().qvg_append_chunk(self._h, _ptr(X), X.shape[1], _stream(stream)), "qvg_append_chunk")

    @property
    def tokens(self) -> int:
        return int(lib().qvg_cache_tokens(self._h))

    @property
    def chunks(self) -> int:
        return int(lib().qvg_cache_chunks(self._h))

    def device_bytes(self) -> int:
        return int(lib().qvg_cache_device_bytes(self._h))

    def status(self, stream=None) -> int:
        """qvg_cache_status: read and clear the cache's device status word."""
        return int(lib().qvg_cache_status(self._h, _stream(stream)))

    def dequantize(self, Y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        if Y is None:
            device = torch.device("cuda")
            Y = _memory(stream, device, torch.empty, (self.H, self.tokens, self.d), dtype=_TORCH[self.dtype], device=device)
            _returned(stream, device, Y)
        _check(lib().qvg_cache_dequantize(self._h, _ptr(Y), _stream(stream)), "qvg_cache_dequantize")
        return Y

    def chunk(self, c: int) -> Packed:
        """Device views of chunk c's packed arrays (valid while the cache lives)."""
        v = _Packed()
        first, n = C.c_int64(), C.c_int64()
        _check(lib().qvg_cache_chunk_view(self._h, c, C.byref(v), C.byref(first), C.byref(n)),
               "qvg_cache_chunk_view")
        H, d, N, cfg = self.H, self.d, n.value, self.cfg
        if self.policy is not None:             # the chunk's own settings
            info = self.chunk_info(c)
            cfg = config(K=cfg.K, T=info["T"], group_size=info["G"], bits=cfg.bits, iters=cfg.iters,
                         warm_iters=cfg.warm_iters, scale_mode=cfg.scale_mode)
        G, T, K = cfg.group_size, cfg.T, cfg.K
        return Packed(codes=_view(v.codes, (H, N, d // 4), torch.uint8),
                      scale=_view(v.scale, (H, N, d // G), torch.uint8),
                      zero=_view(v.zero, (H, N, d // G) if cfg.scale_mode == ASYM else (0,), torch.uint8),
                      assign=_view(v.assign, (T, H, N), torch.uint8),
                      centroids=_view(v.centroids, (T, H, K, d), _TORCH[self.dtype]),
                      cfg=cfg, N=N, H=H, d=d, dtype=self.dtype)

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().qvg_cache_destroy(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
