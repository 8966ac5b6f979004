"""Thin Python binding of the C ABI in include/llsa.h (ctypes).

Argument marshalling only: every step runs in the CUDA kernels of
libllsa.so.  PyTorch provides device memory and streams.  There is no CPU
fallback: if the library is missing or a call fails, an exception is raised.

The functions keep the C names without the ``llsa_`` prefix and take torch
CUDA tensors (or raw device addresses as ints):

    pool(problem, x, pyramid)            select(problem, pyrQ, pyrK, idx)
    reorder(problem, x_in, x_out, to_hier)
    select_level(problem, level, pyrQ, pyrK, idx)
    attn_fwd(problem, q, k, v, pyrK, pyrV, idx, o, lse)
    index_transpose(problem, idx, offs, qlist, scratch)
    attn_bwd(problem, q, k, v, o, dO, lse, pyrK, pyrV, idx, offs, qlist, dq, dk, dv, workspace)

``Pipeline`` allocates the buffers of one problem once and runs the whole
path (pool -> select -> attend -> transpose -> backward) through these calls.

Beside the self-attention, for conditional models, with the same manner of use:

    cross_attn_fwd(problem, q, k, v, o, lse, kv_len, key_mask, workspace)
    cross_attn_bwd(problem, q, k, v, o, dO, lse, dq, dk, dv, kv_len, key_mask, workspace)
    layer_norm_fwd(problem, x, weight, bias, y, mean, rstd)
    layer_norm_bwd(problem, x, dy, weight, mean, rstd, dx, dweight, dbias, workspace)

``CrossAttention`` and ``LayerNorm`` allocate one problem's buffers and run the
forward and the backward.  These calls take tensors with any batch, head and
token strides, check every tensor's shape, type and device, and run on the
tensors' device, on its current torch stream unless one is given.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from functools import lru_cache
from math import sqrt
from struct import Struct
from typing import Optional

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libllsa.so")

BF16, FP32 = 0, 1
MAX_LEVELS = 12

STATUS = {0: "ok", 1: "invalid argument", 2: "shape", 3: "alignment", 4: "workspace", 5: "cuda error",
          6: "device wait timed out", 7: "unsupported"}

EXPORTS = ("llsa_status_string", "llsa_validate", "llsa_level_sizes", "llsa_query_sizes", "llsa_reorder",
           "llsa_pool", "llsa_select", "llsa_select_level", "llsa_attn_fwd", "llsa_index_transpose",
           "llsa_attn_bwd", "llsa_device_error", "llsa_kernel_launches", "llsa_index_transpose_noalloc",
           "llsa_selftest_wait_timeout", "llsa_attn_paths", "llsa_cross_validate", "llsa_cross_query_sizes",
           "llsa_cross_attn_fwd", "llsa_cross_attn_bwd", "llsa_cross_attn_paths", "llsa_norm_validate",
           "llsa_norm_query_sizes", "llsa_layer_norm_fwd", "llsa_layer_norm_bwd")


class LLSAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class CProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("heads", ctypes.c_int), ("height", ctypes.c_int),
                ("width", ctypes.c_int), ("d", ctypes.c_int), ("B", ctypes.c_int), ("L", ctypes.c_int),
                ("K", ctypes.c_int), ("enrich_mask", ctypes.c_uint), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int)]


class CSizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("tokens_bytes", "lse_bytes", "pyramid_bytes", "idx_bytes",
                                                "offs_bytes", "qlist_bytes", "transpose_scratch_bytes",
                                                "bwd_workspace_bytes")]


class CStrides(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("head", ctypes.c_int64), ("token", ctypes.c_int64)]


class CCrossProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "heads", "kv_heads", "nq", "nk", "d")] + \
               [("scale", ctypes.c_float), ("dtype", ctypes.c_int)] + \
               [(n, CStrides) for n in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv")]


class CCrossBuffers(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("lse_bytes", "fwd_workspace_bytes", "bwd_workspace_bytes")]


class CNormProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "heads", "n", "c")] + [("eps", ctypes.c_float)] + \
               [(n, ctypes.c_int) for n in ("dtype", "param_dtype", "per_batch")] + \
               [(n, CStrides) for n in ("x", "y", "dy", "dx")] + \
               [(n, ctypes.c_int64) for n in ("weight_batch", "bias_batch")]


class CNormBuffers(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("stat_bytes", "bwd_workspace_bytes")]


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libllsa.so (built by __graft_entry__.build() or build.py)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python __graft_entry__.py build` "
                               "(nvcc, sm_100a); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(CProblem)
        X, M = ctypes.POINTER(CCrossProblem), ctypes.POINTER(CNormProblem)
        vp, i32 = ctypes.c_void_p, ctypes.c_int
        sig = {
            "llsa_status_string": ([i32], ctypes.c_char_p),
            "llsa_validate": ([P], i32),
            "llsa_level_sizes": ([P, vp, vp], i32),
            "llsa_query_sizes": ([P, ctypes.POINTER(CSizes)], i32),
            "llsa_reorder": ([P, vp, vp, i32, vp], i32),
            "llsa_pool": ([P, vp, vp, vp], i32),
            "llsa_select": ([P, vp, vp, vp, vp], i32),
            "llsa_select_level": ([P, i32, vp, vp, vp, vp], i32),
            "llsa_attn_fwd": ([P, vp, vp, vp, vp, vp, vp, vp, vp, vp], i32),
            "llsa_index_transpose": ([P, vp, vp, vp, vp, vp], i32),
            "llsa_index_transpose_noalloc": ([P, vp, vp, vp, vp], i32),
            "llsa_attn_bwd": ([P] + [vp] * 16, i32),
            "llsa_device_error": ([vp, ctypes.POINTER(i32)], i32),
            "llsa_kernel_launches": ([], ctypes.c_uint64),
            "llsa_selftest_wait_timeout": ([ctypes.c_uint, i32, i32, vp], i32),
            "llsa_attn_paths": ([P, ctypes.POINTER(i32), ctypes.POINTER(i32)], i32),
            "llsa_cross_validate": ([X], i32),
            "llsa_cross_query_sizes": ([X, ctypes.POINTER(CCrossBuffers)], i32),
            "llsa_cross_attn_fwd": ([vp] * 10, i32),
            "llsa_cross_attn_bwd": ([vp] * 14, i32),
            "llsa_cross_attn_paths": ([X, ctypes.POINTER(i32), ctypes.POINTER(i32)], i32),
            "llsa_norm_validate": ([M], i32),
            "llsa_norm_query_sizes": ([M, ctypes.POINTER(CNormBuffers)], i32),
            "llsa_layer_norm_fwd": ([vp] * 8, i32),
            "llsa_layer_norm_bwd": ([vp] * 11, i32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def status_string(s: int) -> str:
    try:
        return lib().llsa_status_string(s).decode()
    except Exception:
        return STATUS.get(s, "unknown")


@dataclass
class Problem:
    """Fields of llsa_problem.  enrich_mask defaults to every level; scale to 1/sqrt(d)."""
    batch: int
    heads: int
    height: int
    width: int
    d: int = 64
    B: int = 16
    L: int = 4
    K: int = 8
    enrich_mask: Optional[int] = None
    scale: Optional[float] = None
    dtype: int = BF16

    def __post_init__(self):
        if self.enrich_mask is None:
            self.enrich_mask = (1 << self.L) - 1
        if self.scale is None:
            self.scale = 1.0 / sqrt(self.d)

    @property
    def N(self) -> int:
        return self.height * self.width

    @property
    def BH(self) -> int:
        return self.batch * self.heads

    def c(self) -> CProblem:
        return CProblem(self.batch, self.heads, self.height, self.width, self.d, self.B, self.L, self.K,
                        self.enrich_mask, float(self.scale), self.dtype)


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st: int, what: str):
    if st != 0:
        raise LLSAError(st, what)


def validate(p: Problem) -> int:
    return lib().llsa_validate(ctypes.byref(p.c()))


def level_sizes(p: Problem):
    n = (ctypes.c_int64 * (p.L + 1))()
    k = (ctypes.c_int64 * (p.L + 1))()
    _check(lib().llsa_level_sizes(ctypes.byref(p.c()), ctypes.addressof(n), ctypes.addressof(k)), "level_sizes")
    return list(n), list(k)


def query_sizes(p: Problem) -> dict:
    s = CSizes()
    _check(lib().llsa_query_sizes(ctypes.byref(p.c()), ctypes.byref(s)), "query_sizes")
    return {name: getattr(s, name) for name, _ in CSizes._fields_}


def reorder(p: Problem, x_in, x_out, to_hier: bool, stream=None):
    _check(lib().llsa_reorder(ctypes.byref(p.c()), _ptr(x_in), _ptr(x_out), int(bool(to_hier)), _stream(stream)),
           "reorder")


def pool(p: Problem, x, pyramid, stream=None):
    _check(lib().llsa_pool(ctypes.byref(p.c()), _ptr(x), _ptr(pyramid), _stream(stream)), "pool")


def select(p: Problem, pyrQ, pyrK, idx, stream=None):
    _check(lib().llsa_select(ctypes.byref(p.c()), _ptr(pyrQ), _ptr(pyrK), _ptr(idx), _stream(stream)), "select")


def select_level(p: Problem, level: int, pyrQ, pyrK, idx, stream=None):
    _check(lib().llsa_select_level(ctypes.byref(p.c()), level, _ptr(pyrQ), _ptr(pyrK), _ptr(idx), _stream(stream)),
           "select_level")


def attn_fwd(p: Problem, q, k, v, pyrK, pyrV, idx, o, lse, stream=None):
    _check(lib().llsa_attn_fwd(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(pyrK), _ptr(pyrV), _ptr(idx),
                               _ptr(o), _ptr(lse), _stream(stream)), "attn_fwd")


def index_transpose(p: Problem, idx, offs, qlist, scratch, stream=None):
    _check(lib().llsa_index_transpose(ctypes.byref(p.c()), _ptr(idx), _ptr(offs), _ptr(qlist), _ptr(scratch),
                                      _stream(stream)), "index_transpose")


def index_transpose_noalloc(p: Problem, idx, offs, qlist, stream=None):
    """index_transpose with the library's own fixed scratch array: for callers
    that cannot allocate device memory.  Calls whose GPU work overlaps share
    that array and must be serialized."""
    _check(lib().llsa_index_transpose_noalloc(ctypes.byref(p.c()), _ptr(idx), _ptr(offs), _ptr(qlist),
                                              _stream(stream)), "index_transpose_noalloc")


def attn_bwd(p: Problem, q, k, v, o, dO, lse, pyrK, pyrV, idx, offs, qlist, dq, dk, dv, workspace, stream=None):
    _check(lib().llsa_attn_bwd(ctypes.byref(p.c()), *[_ptr(t) for t in (q, k, v, o, dO, lse, pyrK, pyrV, idx, offs,
                                                                          qlist, dq, dk, dv, workspace)],
                               _stream(stream)), "attn_bwd")


def attn_paths(p: Problem) -> dict:
    """Which kernels attn_fwd / attn_bwd run for p: "tensor" or "cuda-core"."""
    f, b = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().llsa_attn_paths(ctypes.byref(p.c()), ctypes.byref(f), ctypes.byref(b)), "attn_paths")
    name = {1: "tensor", 0: "cuda-core"}
    return {"fwd": name[f.value], "bwd": name[b.value]}


def kernel_launches() -> int:
    """Kernels launched by libllsa.so in this process so far."""
    return int(lib().llsa_kernel_launches())


def device_error(stream=None) -> int:
    code = ctypes.c_int(0)
    st = lib().llsa_device_error(_stream(stream), ctypes.byref(code))
    if st not in (0, 6):
        raise LLSAError(st, "device_error")
    return code.value


def selftest_wait_timeout(limit_us: int, code: int, arrive: bool = False, stream=None):
    """Launches the timeout-path self-test (llsa_selftest_wait_timeout)."""
    _check(lib().llsa_selftest_wait_timeout(int(limit_us), int(code), int(bool(arrive)), _stream(stream)),
           "selftest_wait_timeout")


# ------------------------------------------------------------------ layouts

def level_views(p: Problem, buf, per_token: int):
    """Per-level views [BH, n_l, per_token] of a level-packed buffer (per_token = d
    for pyramids, or -1 to use K_l for index lists)."""
    n, kl = level_sizes(p)
    out, o = [], 0
    for l in range(1, p.L + 1):
        w = kl[l] if per_token < 0 else per_token
        cnt = p.BH * n[l] * w
        out.append(buf[o:o + cnt].view(p.BH, n[l], w))
        o += cnt
    return out


def offs_views(p: Problem, buf):
    n, _ = level_sizes(p)
    out, o = [], 0
    for l in range(1, p.L + 1):
        cnt = p.BH * (n[l] + 1)
        out.append(buf[o:o + cnt].view(p.BH, n[l] + 1))
        o += cnt
    return out


class Pipeline:
    """Device buffers of one problem, allocated once, and the path run through the C ABI.

    With qk_norm, q and k go through a layer norm over each head's channels first (``norm_q`` and ``norm_k``, eps
    `norm_eps`), with the fp32 weights and biases [d] in ``q_weight``, ``q_bias``, ``k_weight``, ``k_bias`` (ones and
    zeros at first).  Then q and k may have any batch, head and token strides; dq and dk are gradients of what was
    passed in, and norm_q.dweight, norm_q.dbias, norm_k.dweight and norm_k.dbias those of the weights.  v and dO are
    contiguous in either case; next to q and k as a projection leaves them that is checked."""

    def __init__(self, p: Problem, device="cuda", backward: bool = True, qk_norm: bool = False,
                 norm_eps: float = 1e-6):
        import torch
        self.p = p
        _check(validate(p), "validate")
        self.sizes = query_sizes(p)
        self.n, self.Kl = level_sizes(p)
        dt = torch.bfloat16 if p.dtype == BF16 else torch.float32
        shape = (p.batch, p.heads, p.N, p.d)
        f32 = torch.float32
        nel_pyr = self.sizes["pyramid_bytes"] // 4
        self.pyrQ = torch.empty(nel_pyr, dtype=f32, device=device)
        self.pyrK = torch.empty(nel_pyr, dtype=f32, device=device)
        self.pyrV = torch.empty(nel_pyr, dtype=f32, device=device)
        self.idx = torch.empty(self.sizes["idx_bytes"] // 4, dtype=torch.int32, device=device)
        self.o = torch.empty(shape, dtype=dt, device=device)
        self.lse = torch.empty((p.batch, p.heads, p.N), dtype=f32, device=device)
        self.backward = backward
        if backward:
            self.offs = torch.empty(self.sizes["offs_bytes"] // 4, dtype=torch.int32, device=device)
            self.qlist = torch.empty(self.sizes["qlist_bytes"] // 4, dtype=torch.int32, device=device)
            self.tscratch = torch.empty(self.sizes["transpose_scratch_bytes"], dtype=torch.uint8, device=device)
            self.work = torch.empty(self.sizes["bwd_workspace_bytes"], dtype=torch.uint8, device=device)
            self.dq = torch.empty(shape, dtype=dt, device=device)
            self.dk = torch.empty(shape, dtype=dt, device=device)
            self.dv = torch.empty(shape, dtype=dt, device=device)
        self.qk_norm = qk_norm
        if qk_norm:
            n = NormProblem(p.batch, p.heads, p.N, p.d, eps=norm_eps, dtype=p.dtype, param_dtype=FP32)
            self.norm_q, self.norm_k = (LayerNorm(n, device, backward, own_dx=False) for _ in range(2))
            self.q_weight, self.k_weight = (torch.ones(p.d, dtype=f32, device=device) for _ in range(2))
            self.q_bias, self.k_bias = (torch.zeros(p.d, dtype=f32, device=device) for _ in range(2))

    def _contiguous(self, name: str, x):
        """Raises where x is not a tensor as the self-attention reads it, from its address alone."""
        if not isinstance(x, int) and (x.numel() != self.o.numel() or x.dtype != self.o.dtype or
                                       x.device != self.o.device or not x.is_contiguous()):
            raise ValueError(f"{name}: expected a contiguous {self.o.dtype} tensor of shape {tuple(self.o.shape)} on "
                             f"{self.o.device}, got {x.dtype} {tuple(x.shape)} with strides {x.stride()} on {x.device}")

    def forward(self, q, k, v, stream=None):
        p = self.p
        if self.qk_norm:
            self._contiguous("v", v)
            stream = _stream(stream)
            q = self.norm_q.forward(q, self.q_weight, self.q_bias, stream)
            k = self.norm_k.forward(k, self.k_weight, self.k_bias, stream)
        pool(p, q, self.pyrQ, stream)
        pool(p, k, self.pyrK, stream)
        pool(p, v, self.pyrV, stream)
        select(p, self.pyrQ, self.pyrK, self.idx, stream)
        attn_fwd(p, q, k, v, self.pyrK, self.pyrV, self.idx, self.o, self.lse, stream)
        return self.o, self.lse

    def backward_pass(self, q, k, v, dO, stream=None):
        p = self.p
        x, y = q, k
        if self.qk_norm:                                    # the attention saw the normed q and k of the forward call
            self._contiguous("v", v)
            self._contiguous("dO", dO)
            stream = _stream(stream)
            q, k = self.norm_q.y, self.norm_k.y
        index_transpose(p, self.idx, self.offs, self.qlist, self.tscratch, stream)
        attn_bwd(p, q, k, v, self.o, dO, self.lse, self.pyrK, self.pyrV, self.idx, self.offs, self.qlist,
                 self.dq, self.dk, self.dv, self.work, stream)
        if self.qk_norm:                                    # in place: from the normed to what was passed in
            self.norm_q.backward_pass(x, self.q_weight, self.dq, stream, dx=self.dq)
            self.norm_k.backward_pass(y, self.k_weight, self.dk, stream, dx=self.dk)
        return self.dq, self.dk, self.dv

    def step(self, q, k, v, dO=None, stream=None):
        """One pass of the whole path; backward too when dO is given."""
        self.forward(q, k, v, stream)
        if dO is not None:
            self.backward_pass(q, k, v, dO, stream)


# ------------------------------------------------------------------ cross attention and layer norm
#
# A call's time on the host is that of a small kernel: the C problem is packed from its fixed part, made once for
# each set of fields, and the tensors' strides.

_NO_STRIDES = (0, 0, 0)


def _checked(name: str, x, shape, dt, device):
    """The address of x, a tensor of this shape and type on this device."""
    if x.shape == shape and x.dtype is dt and x.device == device:
        return x.data_ptr()
    if x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {shape}")
    if x.dtype != dt:
        raise ValueError(f"{name}: {x.dtype}, expected {dt}")
    raise ValueError(f"{name}: on {x.device}, expected {device}")


def _strides(name: str, x):
    """Batch, head and token stride."""
    s = x.stride()
    if s[3] != 1 and x.shape[3] > 1:
        raise ValueError(f"{name}: the last dimension is not contiguous")
    if s[0] == s[1] == s[2] == 0 and x.shape[:3].numel() > 1:      # zeros stand for the contiguous layout
        raise ValueError(f"{name}: one token expanded over every dimension; materialise at least one of them")
    return s[:3]


def _flat(name: str, x, shape, dt, device):
    """The address of a contiguous tensor of this shape (or an int address, or None)."""
    if x is None or isinstance(x, int):
        return x
    if x.shape != shape or x.dtype != dt or x.device != device or not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dt} tensor of shape {shape} on {device}, "
                         f"got {x.dtype} {tuple(x.shape)} on {x.device}")
    return x.data_ptr()


def _work(x, nbytes: int, device):
    if x is None or isinstance(x, int):
        return x
    if x.device != device or x.nbytes < nbytes or not x.is_contiguous():
        raise ValueError(f"workspace: expected {nbytes} contiguous bytes on {device}")
    return x.data_ptr()


def _torch_dtype(dtype: int):
    import torch
    return torch.bfloat16 if dtype == BF16 else torch.float32


def _run(fn, what: str, device, stream, *args):
    """The call on the tensors' device, and on the given stream, else on the device's current one."""
    from torch._C import _cuda_getCurrentRawStream, _cuda_getDevice
    index = device.index
    if device.type != "cuda":
        raise ValueError(f"tensors on {device}: these calls take CUDA tensors")
    if stream is None:
        stream = _cuda_getCurrentRawStream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    before = _cuda_getDevice()
    if before == index:
        st = fn(*args, stream)
    else:
        from torch import cuda
        cuda.set_device(device)
        try:
            st = fn(*args, stream)
        finally:
            cuda.set_device(before)
    if st != 0:
        raise LLSAError(st, what)


@dataclass
class CrossProblem:
    """Fields of llsa_cross_problem; kv_heads defaults to heads, scale to 1/sqrt(d).  Strides come from the tensors."""
    batch: int
    heads: int
    nq: int
    nk: int
    d: int = 64
    kv_heads: Optional[int] = None
    scale: Optional[float] = None
    dtype: int = BF16

    def __post_init__(self):
        if self.kv_heads is None:
            self.kv_heads = self.heads
        if self.scale is None:
            self.scale = 1.0 / sqrt(self.d) if self.d > 0 else 0.0

    @property
    def q_shape(self):
        return (self.batch, self.heads, self.nq, self.d)

    @property
    def k_shape(self):
        return (self.batch, self.kv_heads, self.nk, self.d)

    def c(self) -> CCrossProblem:
        return CCrossProblem(self.batch, self.heads, self.kv_heads, self.nq, self.nk, self.d, float(self.scale),
                             self.dtype)


def cross_validate(p: CrossProblem) -> int:
    return lib().llsa_cross_validate(ctypes.byref(p.c()))


def cross_query_sizes(p: CrossProblem) -> dict:
    s = CCrossBuffers()
    _check(lib().llsa_cross_query_sizes(ctypes.byref(p.c()), ctypes.byref(s)), "cross_query_sizes")
    return {name: getattr(s, name) for name, _ in CCrossBuffers._fields_}


def cross_attn_paths(p: CrossProblem, q=None, k=None, v=None, dO=None) -> dict:
    """Which kernels cross_attn_fwd / cross_attn_bwd run for p and tensors with these strides (contiguous ones where none
    is given): "tensor", which the kernels for few queries are too, or "cuda-core"."""
    c = p.c()
    for name, field, x, shape in (("q", c.q, q, p.q_shape), ("k", c.k, k, p.k_shape), ("v", c.v, v, p.k_shape),
                                  ("dO", c.d_o, dO, p.q_shape)):
        if x is not None:
            _checked(name, x, shape, _torch_dtype(p.dtype), x.device)
            field.batch, field.head, field.token = _strides(name, x)
    f, b = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().llsa_cross_attn_paths(ctypes.byref(c), ctypes.byref(f), ctypes.byref(b)), "cross_attn_paths")
    name = {1: "tensor", 0: "cuda-core"}
    return {"fwd": name[f.value], "bwd": name[b.value]}


_PACK_CROSS = Struct("24q").pack          # q, k, v, o, d_o, dq, dk, dv
_PACK_NORM = Struct("14q").pack           # x, y, dy, dx, weight_batch, bias_batch
_CROSS_HEAD = CCrossProblem.q.offset
_NORM_HEAD = CNormProblem.x.offset


@lru_cache(maxsize=256)
def _cross_fixed(batch, heads, kv_heads, nq, nk, d, scale, dtype):
    """The C problem up to its strides, buffer sizes, shapes of q and k, element type."""
    p = CrossProblem(batch, heads, nq, nk, d, kv_heads, scale, dtype)
    sizes = cross_query_sizes(p)
    return bytes(p.c())[:_CROSS_HEAD], sizes, p.q_shape, p.k_shape, _torch_dtype(dtype)


def _cross_of(p: CrossProblem):
    return _cross_fixed(p.batch, p.heads, p.kv_heads, p.nq, p.nk, p.d, p.scale, p.dtype)


def _key_args(p: CrossProblem, kv_len, key_mask, device):
    import torch
    if kv_len is not None:
        kv_len = _flat("kv_len", kv_len, (p.batch,), torch.int32, device)
    if key_mask is not None and not isinstance(key_mask, int):
        if key_mask.dtype == torch.bool:
            key_mask = key_mask.view(torch.uint8)
        key_mask = _flat("key_mask", key_mask, (p.batch, p.nk), torch.uint8, device)
    return kv_len, key_mask


def cross_attn_fwd(p: CrossProblem, q, k, v, o, lse=None, kv_len=None, key_mask=None, workspace=None, stream=None):
    """q, o: [batch, heads, nq, d]; k, v: [batch, kv_heads, nk, d]; lse: fp32 [batch, heads, nq] or None; kv_len:
    int32 [batch] or None; key_mask: bool or uint8 [batch, nk], nonzero where the key is attended to, or None;
    workspace: fwd_workspace_bytes of device memory."""
    import torch
    fixed, sizes, qs, ks, dt = _cross_of(p)
    device = q.device
    a = (_checked("q", q, qs, dt, device), _checked("k", k, ks, dt, device), _checked("v", v, ks, dt, device))
    ao = _checked("o", o, qs, dt, device)
    c = fixed + _PACK_CROSS(*_strides("q", q), *_strides("k", k), *_strides("v", v), *_strides("o", o),
                            *_NO_STRIDES, *_NO_STRIDES, *_NO_STRIDES, *_NO_STRIDES)
    n, m = _key_args(p, kv_len, key_mask, device)
    ls = _flat("lse", lse, qs[:3], torch.float32, device)
    _run(lib().llsa_cross_attn_fwd, "cross_attn_fwd", device, stream, c, *a, n, m, ao, ls,
         _work(workspace, sizes["fwd_workspace_bytes"], device))


def cross_attn_bwd(p: CrossProblem, q, k, v, o, dO, lse, dq, dk, dv, kv_len=None, key_mask=None, workspace=None,
                   stream=None):
    """Gradients of cross_attn_fwd for the same kv_len and key_mask; workspace: bwd_workspace_bytes."""
    import torch
    fixed, sizes, qs, ks, dt = _cross_of(p)
    device = q.device
    a = (_checked("q", q, qs, dt, device), _checked("k", k, ks, dt, device), _checked("v", v, ks, dt, device))
    b = (_checked("o", o, qs, dt, device), _checked("dO", dO, qs, dt, device))
    g = (_checked("dq", dq, qs, dt, device), _checked("dk", dk, ks, dt, device), _checked("dv", dv, ks, dt, device))
    c = fixed + _PACK_CROSS(*_strides("q", q), *_strides("k", k), *_strides("v", v), *_strides("o", o),
                            *_strides("dO", dO), *_strides("dq", dq), *_strides("dk", dk), *_strides("dv", dv))
    n, m = _key_args(p, kv_len, key_mask, device)
    ls = _flat("lse", lse, qs[:3], torch.float32, device)
    _run(lib().llsa_cross_attn_bwd, "cross_attn_bwd", device, stream, c, *a, n, m, *b, ls, *g,
         _work(workspace, sizes["bwd_workspace_bytes"], device))


def _buffer(shape, dtype, device, token_major: bool):
    """A [batch, heads, tokens, d] tensor, in memory as such or (token_major) as [batch, tokens, heads, d]."""
    import torch
    if not token_major:
        return torch.empty(shape, dtype=dtype, device=device)
    b, h, n, d = shape
    return torch.empty((b, n, h, d), dtype=dtype, device=device).transpose(1, 2)


class CrossAttention:
    """Buffers of one cross-attention problem, allocated once, and its passes.  With token_major, o and the gradients
    lie in memory as [batch, tokens, heads, d], as the projections around the attention have them."""

    def __init__(self, p: CrossProblem, device="cuda", backward: bool = True, token_major: bool = False):
        import torch
        self.p = p
        _check(cross_validate(p), "cross_validate")
        self.sizes = cross_query_sizes(p)
        dt = _torch_dtype(p.dtype)
        self.o = _buffer(p.q_shape, dt, device, token_major)
        self.lse = torch.empty(p.q_shape[:3], dtype=torch.float32, device=device)
        need = max(self.sizes["fwd_workspace_bytes"], self.sizes["bwd_workspace_bytes"] if backward else 0)
        self.work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        self.backward = backward
        if backward:
            self.dq = _buffer(p.q_shape, dt, device, token_major)
            self.dk = _buffer(p.k_shape, dt, device, token_major)
            self.dv = _buffer(p.k_shape, dt, device, token_major)

    def forward(self, q, k, v, kv_len=None, key_mask=None, stream=None):
        cross_attn_fwd(self.p, q, k, v, self.o, self.lse, kv_len, key_mask, self.work, stream)
        return self.o, self.lse

    def backward_pass(self, q, k, v, dO, kv_len=None, key_mask=None, stream=None):
        """The gradients of the last forward call's problem (its o and lse are read)."""
        cross_attn_bwd(self.p, q, k, v, self.o, dO, self.lse, self.dq, self.dk, self.dv, kv_len, key_mask, self.work,
                       stream)
        return self.dq, self.dk, self.dv


@dataclass
class NormProblem:
    """Fields of llsa_norm_problem; param_dtype defaults to dtype.  Strides come from the tensors."""
    batch: int
    heads: int
    n: int
    c: int
    eps: float = 1e-6
    dtype: int = BF16
    param_dtype: Optional[int] = None
    per_batch: bool = False

    def __post_init__(self):
        if self.param_dtype is None:
            self.param_dtype = self.dtype

    @property
    def shape(self):
        return (self.batch, self.heads, self.n, self.c)

    @property
    def param_shape(self):
        return (self.batch, self.c) if self.per_batch else (self.c,)

    def cp(self) -> CNormProblem:
        return CNormProblem(self.batch, self.heads, self.n, self.c, float(self.eps), self.dtype, self.param_dtype,
                            int(self.per_batch))


def norm_validate(p: NormProblem) -> int:
    return lib().llsa_norm_validate(ctypes.byref(p.cp()))


def norm_query_sizes(p: NormProblem) -> dict:
    s = CNormBuffers()
    _check(lib().llsa_norm_query_sizes(ctypes.byref(p.cp()), ctypes.byref(s)), "norm_query_sizes")
    return {name: getattr(s, name) for name, _ in CNormBuffers._fields_}


@lru_cache(maxsize=256)
def _norm_fixed(batch, heads, n, c, eps, dtype, param_dtype, per_batch):
    """The C problem up to its strides, workspace bytes, shapes of rows and weights, their types."""
    p = NormProblem(batch, heads, n, c, eps, dtype, param_dtype, per_batch)
    need = norm_query_sizes(p)["bwd_workspace_bytes"]
    return bytes(p.cp())[:_NORM_HEAD], need, p.shape, p.param_shape, _torch_dtype(dtype), _torch_dtype(param_dtype)


def _norm_of(p: NormProblem):
    return _norm_fixed(p.batch, p.heads, p.n, p.c, p.eps, p.dtype, p.param_dtype, p.per_batch)


def _param(p: NormProblem, name: str, x, shape, dt, device):
    """Address and row stride of weight or bias: [c] contiguous, or [batch, c] with its rows apart by any stride."""
    if x is None or isinstance(x, int):
        return x, 0
    address = _checked(name, x, shape, dt, device)
    s = x.stride()
    if s[-1] != 1 and p.c > 1:
        raise ValueError(f"{name}: the last dimension is not contiguous")
    if not p.per_batch or p.batch == 1:
        return address, 0
    if s[0] == 0:                                           # zero stands for contiguous rows
        raise ValueError(f"{name}: one row expanded over the batch; per_batch=False takes it as [c]")
    return address, s[0]


def layer_norm_fwd(p: NormProblem, x, weight, bias, y, mean=None, rstd=None, stream=None):
    """x, y: [batch, heads, n, c]; weight, bias: [c] (per_batch: [batch, c], rows any stride apart) or None; mean,
    rstd: fp32 [batch, heads, n] or None."""
    import torch
    fixed, _, shape, pshape, dt, pt = _norm_of(p)
    device = x.device
    ax, ay = _checked("x", x, shape, dt, device), _checked("y", y, shape, dt, device)
    w, ws = _param(p, "weight", weight, pshape, pt, device)
    b, bs = _param(p, "bias", bias, pshape, pt, device)
    c = fixed + _PACK_NORM(*_strides("x", x), *_strides("y", y), *_NO_STRIDES, *_NO_STRIDES, ws, bs)
    f32 = torch.float32
    _run(lib().llsa_layer_norm_fwd, "layer_norm_fwd", device, stream, c, ax, w, b, ay,
         _flat("mean", mean, shape[:3], f32, device), _flat("rstd", rstd, shape[:3], f32, device))


def layer_norm_bwd(p: NormProblem, x, dy, weight, mean, rstd, dx=None, dweight=None, dbias=None, workspace=None,
                   stream=None):
    """Gradients of layer_norm_fwd; dx, dweight and dbias are written where given; workspace: bwd_workspace_bytes."""
    import torch
    fixed, need, shape, pshape, dt, pt = _norm_of(p)
    device = x.device
    ax, ag = _checked("x", x, shape, dt, device), _checked("dy", dy, shape, dt, device)
    ad, sd = None, _NO_STRIDES
    if dx is not None:
        ad, sd = _checked("dx", dx, shape, dt, device), _strides("dx", dx)
    w, ws = _param(p, "weight", weight, pshape, pt, device)
    c = fixed + _PACK_NORM(*_strides("x", x), *_NO_STRIDES, *_strides("dy", dy), *sd, ws, 0)
    f32 = torch.float32
    _run(lib().llsa_layer_norm_bwd, "layer_norm_bwd", device, stream, c, ax, ag, w,
         _flat("mean", mean, shape[:3], f32, device), _flat("rstd", rstd, shape[:3], f32, device), ad,
         _flat("dweight", dweight, pshape, pt, device), _flat("dbias", dbias, pshape, pt, device),
         _work(workspace, need, device))


class LayerNorm:
    """Buffers of one layer-norm problem, allocated once, and its passes (token_major as for CrossAttention).  Without
    own_dx the backward pass writes dx where it is told to (dx=)."""

    def __init__(self, p: NormProblem, device="cuda", backward: bool = True, token_major: bool = False,
                 own_dx: bool = True):
        import torch
        self.p = p
        _check(norm_validate(p), "norm_validate")
        dt, pt = _torch_dtype(p.dtype), _torch_dtype(p.param_dtype)
        self.y = _buffer(p.shape, dt, device, token_major)
        self.backward = backward
        self.mean = self.rstd = None
        if backward:
            self.mean = torch.empty(p.shape[:3], dtype=torch.float32, device=device)
            self.rstd = torch.empty(p.shape[:3], dtype=torch.float32, device=device)
            self.dx = _buffer(p.shape, dt, device, token_major) if own_dx else None
            self.dweight = torch.empty(p.param_shape, dtype=pt, device=device)
            self.dbias = torch.empty(p.param_shape, dtype=pt, device=device)
            self.work = torch.empty(norm_query_sizes(p)["bwd_workspace_bytes"], dtype=torch.uint8, device=device)

    def forward(self, x, weight=None, bias=None, stream=None):
        layer_norm_fwd(self.p, x, weight, bias, self.y, self.mean, self.rstd, stream)
        return self.y

    def backward_pass(self, x, weight, dy, stream=None, dx=None):
        """The gradients of the last forward call (its mean and rstd are read); dx: where to, if not to self.dx (dy
        itself will do)."""
        dx = self.dx if dx is None else dx
        layer_norm_bwd(self.p, x, dy, weight, self.mean, self.rstd, dx, self.dweight, self.dbias, self.work, stream)
        return dx, self.dweight, self.dbias
