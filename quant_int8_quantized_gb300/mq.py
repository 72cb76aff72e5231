"""Thin ctypes binding of libmq.so (include/mq.h), with the same entry-point names.

Argument marshalling only: torch tensors are checked for device, dtype and
contiguity, their data pointers and the current CUDA stream are passed to the
C ABI, and a non-zero status raises MQError. Every step of the computation
runs in the library's CUDA kernels; there is no other code path. If the
library has not been built, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libmq.so")

MQ_OK, MQ_ERR_NULL, MQ_ERR_SHAPE, MQ_ERR_ALIGN, MQ_ERR_ARCH, MQ_ERR_LAUNCH, MQ_ERR_DEVICE, MQ_ERR_SCRATCH, MQ_ERR_TYPE = range(9)
MQ_GEMV_MAX_ROWS = 8   # include/mq.h

EXPORTED = ["mq_plane_bytes", "mq_q4k_row_bytes", "mq_q6k_row_bytes", "mq_q6k_packed_row_bytes", "mq_prepack_q6k",
            "mq_quantize_q8", "mq_rms_quant",
            "mq_swiglu_quant", "mq_gemm_q4k", "mq_gemm_q6k", "mq_gemv_q4k", "mq_gemv_q6k",
            "mq_q5k_row_bytes", "mq_q4_0_row_bytes", "mq_q4_1_row_bytes", "mq_gemv_q5k", "mq_gemv_q4_0",
            "mq_gemv_q4_1", "mq_gemm_q4_0", "mq_gemm_q4_1", "mq_gemv_q6k_packed", "mq_gemm_q6k_static", "mq_gemm_q4k_pair",
            "mq_qk_norm_rope", "mq_attn_ws_bytes", "mq_attn_prefix", "mq_kv_evict",
            "mq_device_status", "mq_status_str"]


class MQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} (status {status})")


class CPlane(ctypes.Structure):
    _fields_ = [("qs", ctypes.c_void_p), ("d", ctypes.c_void_p), ("s", ctypes.c_void_p),
                ("ah", ctypes.c_void_p), ("ax", ctypes.c_void_p), ("af", ctypes.c_void_p),
                ("M", ctypes.c_int), ("K", ctypes.c_int)]


class CKV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("seq_stride", ctypes.c_longlong),
                ("row_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong), ("type", ctypes.c_int),
                ("n", ctypes.c_int), ("cap", ctypes.c_int), ("heads", ctypes.c_int), ("dim", ctypes.c_int)]


class CQKV(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v")] + \
               [(n, ctypes.c_longlong) for n in ("q_stride", "k_stride", "v_stride")] + \
               [(n, ctypes.c_void_p) for n in ("wq", "wk", "inv_freq", "axis", "pos")] + \
               [(n, ctypes.c_int) for n in ("M", "Hq", "n_pairs", "n_axes", "interleaved")] + [("eps", ctypes.c_float)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        _lib = _load(LIB_PATH)
    return _lib


def _load(path: str) -> ctypes.CDLL:
    """A build of the library with its entry points' signatures."""
    L = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    pp = ctypes.POINTER(CPlane)
    psz = ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "mq_plane_bytes": (sz, [i, i, psz, psz, psz, psz, psz, psz]),
        "mq_q4k_row_bytes": (sz, [i]),
        "mq_q6k_row_bytes": (sz, [i]),
        "mq_q6k_packed_row_bytes": (sz, [i]),
        "mq_prepack_q6k": (i, [vp, i, i, vp, vp]),
        "mq_quantize_q8": (i, [vp, i, i, pp, vp]),
        "mq_rms_quant": (i, [vp, vp, i, i, f, pp, vp]),
        "mq_swiglu_quant": (i, [vp, vp, i, i, pp, vp]),
        "mq_gemm_q4k": (i, [pp, vp, i, vp, vp]),
        "mq_gemm_q6k": (i, [pp, vp, i, vp, vp]),
        "mq_gemv_q4k": (i, [pp, vp, i, vp, vp]),
        "mq_gemv_q6k": (i, [pp, vp, i, vp, vp]),
        "mq_gemv_q6k_packed": (i, [pp, vp, i, vp, vp]),
        "mq_gemm_q6k_static": (i, [pp, vp, i, vp, vp]),
        "mq_gemm_q4k_pair": (i, [pp, vp, i, vp, vp, i, vp, vp]),
        "mq_q5k_row_bytes": (sz, [i]),
        "mq_q4_0_row_bytes": (sz, [i]),
        "mq_q4_1_row_bytes": (sz, [i]),
        "mq_gemv_q5k": (i, [pp, vp, i, vp, vp]),
        "mq_gemv_q4_0": (i, [pp, vp, i, vp, vp]),
        "mq_gemv_q4_1": (i, [pp, vp, i, vp, vp]),
        "mq_gemm_q4_0": (i, [pp, vp, i, vp, vp]),
        "mq_gemm_q4_1": (i, [pp, vp, i, vp, vp]),
        "mq_qk_norm_rope": (i, [ctypes.POINTER(CQKV), vp, ctypes.POINTER(CKV), vp, vp]),
        "mq_attn_ws_bytes": (sz, [i, i, i, i, i, i, i, i]),
        "mq_attn_prefix": (i, [vp, ctypes.c_longlong, i, i, i, ctypes.POINTER(CKV), ctypes.POINTER(CKV), vp, f, vp, i,
                               vp, vp, vp, vp, sz, vp]),
        "mq_kv_evict": (i, [ctypes.POINTER(CKV), vp, vp, i, i, ctypes.POINTER(CKV), vp, vp, vp, vp]),
        "mq_device_status": (i, [vp]),
        "mq_status_str": (ctypes.c_char_p, [i]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def status_str(status: int) -> str:
    return lib().mq_status_str(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return _current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _on(stream, device):
    """Allocations made inside belong to `stream` (None: the current one). The caching allocator hands what is freed
    to the same stream's next allocation, so memory that a call allocates for itself has to come from the stream that it
    runs on."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)
    return torch.cuda.stream(stream)


def _current_stream():
    """The current stream's handle, by the bindings under torch.cuda.current_stream() where they are
    there: building a Stream object takes 3 us on a Grace core, as long as the rest of a small call."""
    if _raw_stream is not None and torch.cuda.is_initialized():
        return ctypes.c_void_p(_raw_stream(_device()))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) if hasattr(torch._C, "_cuda_getDevice") else None
_device = getattr(torch._C, "_cuda_getDevice", None)


def _check(status: int, where: str):
    if status != MQ_OK:
        raise MQError(status, where)


def _dev_tensor(t, dtype, name):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous():
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


class Plane:
    """Device activation plane (include/mq.h): the q8 arrays qs int8 [M, K],
    d f32 [M, K/32], s int32 [M, K/32] (read by the GEMV), and/or the GEMM's
    operand arrays ah f16 [M, K], ax f16 [M, K/256, 16], af f32 [K/256, Mp]
    with Mp = M rounded up to a multiple of 4. Producers fill whichever groups
    are present."""

    def __init__(self, qs=None, d=None, s=None, ah=None, ax=None, af=None, M=None, K=None):
        self.qs, self.d, self.s, self.ah, self.ax, self.af = qs, d, s, ah, ax, af
        ref = qs if qs is not None else ah
        if ref is None:
            raise ValueError("a plane needs its q8 arrays, its operand arrays, or both")
        self.M, self.K = int(ref.shape[0]), int(ref.shape[1])
        if qs is not None:
            _dev_tensor(qs, torch.int8, "plane.qs")
            _dev_tensor(d, torch.float32, "plane.d")
            _dev_tensor(s, torch.int32, "plane.s")
        if ah is not None:
            _dev_tensor(ah, torch.float16, "plane.ah")
            _dev_tensor(ax, torch.float16, "plane.ax")
            _dev_tensor(af, torch.float32, "plane.af")

    @staticmethod
    def af_stride(M: int) -> int:
        return (M + 3) // 4 * 4

    @classmethod
    def empty(cls, M: int, K: int, device="cuda", q8: bool = True, op: bool = True) -> "Plane":
        """Allocate a plane with the q8 arrays (q8=True) and/or the operand arrays (op=True)."""
        kw = {}
        if q8:
            kw.update(qs=torch.empty((M, K), dtype=torch.int8, device=device),
                      d=torch.empty((M, K // 32), dtype=torch.float32, device=device),
                      s=torch.empty((M, K // 32), dtype=torch.int32, device=device))
        if op:
            kw.update(ah=torch.empty((M, K), dtype=torch.float16, device=device),
                      ax=torch.empty((M, K // 256, 16), dtype=torch.float16, device=device),
                      af=torch.empty((K // 256, cls.af_stride(M)), dtype=torch.float32, device=device))
        return cls(**kw)

    def c(self) -> CPlane:
        def p(t):
            return t.data_ptr() if t is not None else None
        return CPlane(p(self.qs), p(self.d), p(self.s), p(self.ah), p(self.ax), p(self.af), self.M, self.K)


def mq_plane_bytes(M: int, K: int):
    """(total, qs, d, s, ah, ax, af) bytes of an M x K plane."""
    v = [ctypes.c_size_t() for _ in range(6)]
    tot = lib().mq_plane_bytes(M, K, *[ctypes.byref(x) for x in v])
    return (int(tot),) + tuple(int(x.value) for x in v)


def mq_q4k_row_bytes(K: int) -> int:
    return int(lib().mq_q4k_row_bytes(K))


def mq_q6k_row_bytes(K: int) -> int:
    return int(lib().mq_q6k_row_bytes(K))


def mq_q6k_packed_row_bytes(K: int) -> int:
    return int(lib().mq_q6k_packed_row_bytes(K))


def mq_prepack_q6k(w: torch.Tensor, N: int, K: int, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Raw q6_K rows [N, K/256*210] (uint8) -> the prepacked layout [N, K/256*224] the GEMM reads. out:
    allocated on the call's stream if None."""
    _dev_tensor(w, torch.uint8, "w")
    if out is None:
        with _on(stream, w.device):
            out = torch.empty((N, mq_q6k_packed_row_bytes(K)), dtype=torch.uint8, device=w.device)
    _dev_tensor(out, torch.uint8, "out")
    _check(lib().mq_prepack_q6k(_ptr(w), int(N), int(K), _ptr(out), _stream(stream)), "mq_prepack_q6k")
    return out


def mq_quantize_q8(x: torch.Tensor, out: Plane, stream=None) -> Plane:
    _dev_tensor(x, torch.float32, "x")
    cp = out.c()
    _check(lib().mq_quantize_q8(_ptr(x), x.shape[0], x.shape[1], ctypes.byref(cp), _stream(stream)),
           "mq_quantize_q8")
    return out


def mq_rms_quant(x: torch.Tensor, w: torch.Tensor, eps: float, out: Plane, stream=None) -> Plane:
    _dev_tensor(x, torch.float32, "x")
    _dev_tensor(w, torch.float32, "w")
    cp = out.c()
    _check(lib().mq_rms_quant(_ptr(x), _ptr(w), x.shape[0], x.shape[1], float(eps), ctypes.byref(cp),
                              _stream(stream)), "mq_rms_quant")
    return out


def mq_swiglu_quant(g: torch.Tensor, u: torch.Tensor, out: Plane, stream=None) -> Plane:
    _dev_tensor(g, torch.float32, "g")
    _dev_tensor(u, torch.float32, "u")
    if g.shape != u.shape:
        raise ValueError("g and u must have the same shape")
    cp = out.c()
    _check(lib().mq_swiglu_quant(_ptr(g), _ptr(u), g.shape[0], g.shape[1], ctypes.byref(cp), _stream(stream)),
           "mq_swiglu_quant")
    return out


def _matmul(fn_name: str, a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream):
    _dev_tensor(w, torch.uint8, "w")
    _dev_tensor(out, torch.float32, "out")
    if out.numel() < a.M * N:
        raise ValueError(f"{fn_name}: out holds {out.numel()} floats, needs M * N = {a.M * N}")
    cp = a.c()
    _check(getattr(lib(), fn_name)(ctypes.byref(cp), _ptr(w), int(N), _ptr(out), _stream(stream)), fn_name)
    return out


def mq_gemm_q4k(a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    return _matmul("mq_gemm_q4k", a, w, N, out, stream)


def mq_gemm_q6k(a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    return _matmul("mq_gemm_q6k", a, w, N, out, stream)


def mq_gemv_q4k(a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    return _matmul("mq_gemv_q4k", a, w, N, out, stream)


def mq_gemv_q6k(a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    return _matmul("mq_gemv_q6k", a, w, N, out, stream)


def mq_gemv_q6k_packed(a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    """q6_K GEMV on prepacked rows (mq_prepack_q6k), the form the GEMM reads too."""
    return _matmul("mq_gemv_q6k_packed", a, w, N, out, stream)


def mq_gemm_q4k_pair(a: Plane, w0: torch.Tensor, N0: int, out0: torch.Tensor, w1: torch.Tensor, N1: int,
                     out1: torch.Tensor, stream=None):
    """Two q4_K GEMMs on one plane (include/mq.h): out0 = a x w0, out1 = a x w1, in one launch
    where that pays."""
    for t, n in ((w0, "w0"), (w1, "w1")):
        _dev_tensor(t, torch.uint8, n)
    for t, n, N in ((out0, "out0", N0), (out1, "out1", N1)):
        _dev_tensor(t, torch.float32, n)
        if t.numel() < a.M * N:
            raise ValueError(f"mq_gemm_q4k_pair: {n} holds {t.numel()} floats, needs M * N = {a.M * N}")
    cp = a.c()
    _check(lib().mq_gemm_q4k_pair(ctypes.byref(cp), _ptr(w0), int(N0), _ptr(out0), _ptr(w1), int(N1), _ptr(out1),
                                  _stream(stream)), "mq_gemm_q4k_pair")
    return out0, out1


def mq_gemm_q6k_static(a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    """mq_gemm_q6k for callers that cannot have device memory allocated for them: its scratch is
    a fixed array inside the library (see include/mq.h)."""
    return _matmul("mq_gemm_q6k_static", a, w, N, out, stream)


def mq_gemm_q4_0(a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    return _matmul("mq_gemm_q4_0", a, w, N, out, stream)


def mq_gemm_q4_1(a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    return _matmul("mq_gemm_q4_1", a, w, N, out, stream)


def mq_gemv_q5k(a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    return _matmul("mq_gemv_q5k", a, w, N, out, stream)


def mq_gemv_q4_0(a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    return _matmul("mq_gemv_q4_0", a, w, N, out, stream)


def mq_gemv_q4_1(a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    return _matmul("mq_gemv_q4_1", a, w, N, out, stream)


def mq_q5k_row_bytes(K: int) -> int:
    return int(lib().mq_q5k_row_bytes(K))


def mq_q4_0_row_bytes(K: int) -> int:
    return int(lib().mq_q4_0_row_bytes(K))


def mq_q4_1_row_bytes(K: int) -> int:
    return int(lib().mq_q4_1_row_bytes(K))


# ---------------------------------------------------------------- heads, caches, attention

_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}   # include/mq.h: MQ_F16, MQ_BF16, MQ_F32


class KV:
    """Keys and values of n sequences (include/mq.h, mq_kv): 16-bit CUDA tensors k and v of shape
    [n, cap, heads, dim], with the same strides and the last dim contiguous. A cache that is laid
    out [n, heads, cap, dim] is given as its transpose(1, 2)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        for t, name in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.device.type != "cuda":
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.dtype not in (torch.float16, torch.bfloat16):
                raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
            if t.dim() != 4 or (t.stride(3) != 1 and t.shape[3] > 1):
                raise ValueError(f"{name} must be [n, cap, heads, dim] with contiguous dims")
        if k.shape != v.shape or k.dtype != v.dtype or (k.stride() != v.stride() and k.numel()):
            raise ValueError("k and v must have the same shape, type and strides")
        self.k, self.v = k, v
        self.n, self.cap, self.heads, self.dim = (int(x) for x in k.shape)
        # an axis of one step has no stride that matters: torch may hold any number there
        st = [int(k.stride(i)) if k.shape[i] > 1 else 0 for i in range(3)]
        self._c = CKV(k.data_ptr(), v.data_ptr(), st[0], st[1], st[2], _TYPES[k.dtype], self.n, self.cap, self.heads,
                      self.dim)
        self._ref, self.dtype = ctypes.byref(self._c), k.dtype

    @classmethod
    def empty(cls, n: int, cap: int, heads: int, dim: int, dtype=torch.float16, device="cuda") -> "KV":
        return cls(torch.empty((n, cap, heads, dim), dtype=dtype, device=device),
                   torch.empty((n, cap, heads, dim), dtype=dtype, device=device))


def rope_freq(n_pairs: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """inv_freq for mq_qk_norm_rope: base^(-i / n_pairs), f32 [n_pairs]."""
    i = torch.arange(n_pairs, dtype=torch.float64)
    return (float(base) ** (-i / n_pairs)).to(torch.float32).to(device)


def rope_axes(sections, device="cuda") -> torch.Tensor:
    """axis for mq_qk_norm_rope: the first sections[0] pairs turn by axis 0, the next by axis 1, ..."""
    return torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], dtype=torch.uint8, device=device)


def _heads(t, name, M, D, heads=None):
    """f32 [M, heads, D] with each token's heads contiguous: (pointer, token stride, heads)."""
    if t is None:
        return None, 0, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.float32:
        raise TypeError(f"{name} must be torch.float32, got {t.dtype}")
    s, st = t.shape, t.stride()
    if len(s) != 3 or s[0] != M or s[2] != D or (heads is not None and s[1] != heads):
        raise ValueError(f"{name} must be [{M}, {'heads' if heads is None else heads}, {D}], got {tuple(s)}")
    if (st[2] != 1 and D > 1) or (st[1] != D and s[1] > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), (st[0] if M > 1 else s[1] * D), s[1]


def mq_qk_norm_rope(q, k, v, q_out, cache: KV, slot=None, pos=None, inv_freq=None, axis=None, wq=None, wk=None,
                    eps: float = 1e-6, interleaved: bool = False, stream=None):
    """Head norms of q and k, rotation by position, q to 16 bits and k, v into the cache rows slot
    (include/mq.h). q: f32 [M, Hq, D]; k, v: f32 [M, Hkv, D] (any may be None; a token's heads are
    contiguous, tokens at any stride); q_out: [M, Hq, D] of the cache's type; slot: int32 [M];
    pos: int32 [M] or [n_axes, M]; inv_freq: f32 [n_pairs]; axis: uint8 [n_pairs]."""
    if not isinstance(cache, KV):
        raise TypeError("cache must be a KV")
    first = q if q is not None else k if k is not None else v
    if first is None:
        raise ValueError("one of q, k and v is needed")
    if not isinstance(first, torch.Tensor):
        raise TypeError(f"{'q' if first is q else 'k' if first is k else 'v'} must be a torch.Tensor")
    M, D = first.shape[0], cache.dim
    q_ptr, q_stride, Hq = _heads(q, "q", M, D)
    k_ptr, k_stride, _ = _heads(k, "k", M, D, cache.heads)
    v_ptr, v_stride, _ = _heads(v, "v", M, D, cache.heads)
    out_ptr = slot_ptr = wq_ptr = wk_ptr = freq_ptr = axis_ptr = pos_ptr = None
    if q is not None:
        if _dev_tensor(q_out, cache.dtype, "q_out").numel() < M * Hq * D:
            raise ValueError(f"q_out holds {q_out.numel()} elements, needs {M * Hq * D}")
        out_ptr = q_out.data_ptr()
    if wq is not None:
        if _dev_tensor(wq, torch.float32, "wq").numel() != D:
            raise ValueError(f"wq must hold {D} weights")
        wq_ptr = wq.data_ptr()
    if wk is not None:
        if _dev_tensor(wk, torch.float32, "wk").numel() != D:
            raise ValueError(f"wk must hold {D} weights")
        wk_ptr = wk.data_ptr()
    n_pairs = n_axes = 0
    if inv_freq is not None:
        n_pairs = _dev_tensor(inv_freq, torch.float32, "inv_freq").numel()
    if n_pairs:
        n_axes = 1 if _dev_tensor(pos, torch.int32, "pos").dim() == 1 else pos.shape[0]
        if pos.numel() != n_axes * M:
            raise ValueError(f"pos must be [{M}] or [n_axes, {M}], got {tuple(pos.shape)}")
        if axis is not None:
            if _dev_tensor(axis, torch.uint8, "axis").numel() != n_pairs:
                raise ValueError(f"axis must hold {n_pairs} entries")
            axis_ptr = axis.data_ptr()
        freq_ptr, pos_ptr = inv_freq.data_ptr(), pos.data_ptr()
    if slot is not None:
        if _dev_tensor(slot, torch.int32, "slot").numel() != M:
            raise ValueError(f"slot must hold {M} entries")
        slot_ptr = slot.data_ptr()
    x = CQKV(q_ptr, k_ptr, v_ptr, q_stride, k_stride, v_stride, wq_ptr, wk_ptr, freq_ptr, axis_ptr, pos_ptr, M, Hq,
             n_pairs, n_axes, 1 if interleaved else 0, eps)
    _check((_lib or lib()).mq_qk_norm_rope(ctypes.byref(x), out_ptr, cache._ref, slot_ptr, _stream(stream)),
           "mq_qk_norm_rope")
    return q_out


def mq_attn_ws_bytes(B: int, T: int, Hq: int, Hkv: int, D: int, prefix_cap: int, own_cap: int,
                     scores: bool = False) -> int:
    return int(lib().mq_attn_ws_bytes(B, T, Hq, Hkv, D, prefix_cap, own_cap, int(bool(scores))))


def attn_workspace(B: int, T: int, Hq: int, Hkv: int, D: int, prefix_cap: int, own_cap: int, scores: bool = False,
                   device="cuda") -> torch.Tensor:
    """A workspace for mq_attn_prefix calls of these sizes on one stream. (Sizes choose the kernels, so a
    smaller call may need more; one that is too small is refused.)"""
    return torch.empty((max(16, mq_attn_ws_bytes(B, T, Hq, Hkv, D, prefix_cap, own_cap, scores)),), dtype=torch.uint8,
                       device=device)


def mq_attn_prefix(q: torch.Tensor, prefix, own, own_len, out: torch.Tensor, scale=None, lse=None, score=None,
                   score_out=None, ws=None, stream=None) -> torch.Tensor:
    """Attention of q [B, T, Hq, D] over a shared prefix (KV of one sequence, or None) and each
    sequence's own cache (KV of B sequences, or None) of own_len rows (include/mq.h). out: [B, T,
    Hq, D] in q's type or f32; lse: f32 [B, T, Hq]; score, score_out: f32 [B, Hkv, own.cap];
    scale: 1 / sqrt(D) if None; ws: attn_workspace(...), allocated on the call's stream for this call
    if None."""
    any_kv = own if own is not None else prefix
    if any_kv is None:
        raise ValueError("a prefix, an own cache or both are needed")
    if not isinstance(any_kv, KV) or (prefix is not None and not isinstance(prefix, KV)):
        raise TypeError("prefix and own must be KV")
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise TypeError("q must be a torch.Tensor [B, T, Hq, D]")
    B, T, Hq, D = q.shape
    dtype = q.dtype
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    if dtype is not any_kv.dtype:
        raise TypeError(f"q must be {any_kv.dtype}, got {dtype}")
    if D != any_kv.dim:
        raise ValueError(f"q's heads are {D} wide, the cache's {any_kv.dim}")
    rows = B * T * Hq
    st = q.stride()
    if rows and (st[3] != 1 or (Hq > 1 and st[2] != D) or (B > 1 and T > 1 and st[0] != T * st[1])):
        raise ValueError("q: a token's heads must be contiguous, and the tokens at one stride")
    row = st[1] if T > 1 else st[0] if B > 1 else Hq * D
    if not isinstance(out, torch.Tensor):
        raise TypeError("out must be a torch.Tensor")
    out_type = out.dtype
    if out_type is not dtype and out_type is not torch.float32:
        raise TypeError(f"out must be {dtype} or torch.float32, got {out_type}")
    if _dev_tensor(out, out_type, "out").numel() < rows * D:
        raise ValueError(f"out holds {out.numel()} elements, needs {rows * D}")
    own_ref = len_ptr = lse_ptr = score_ptr = score_out_ptr = None
    if own is not None:
        if _dev_tensor(own_len, torch.int32, "own_len").numel() != B:
            raise ValueError(f"own_len must hold {B} lengths")
        own_ref, len_ptr = own._ref, own_len.data_ptr()
    if lse is not None:
        if _dev_tensor(lse, torch.float32, "lse").numel() < rows:
            raise ValueError(f"lse needs {rows} elements")
        lse_ptr = lse.data_ptr()
    if score is not None:
        if own is None or _dev_tensor(score, torch.float32, "score").numel() < B * own.heads * own.cap:
            raise ValueError("score must be [B, Hkv, own.cap]")
        score_ptr = score.data_ptr()
    if score_out is not None:
        if own is None or _dev_tensor(score_out, torch.float32, "score_out").numel() < B * own.heads * own.cap:
            raise ValueError("score_out must be [B, Hkv, own.cap]")
        score_out_ptr = score_out.data_ptr()
    if ws is None:
        with _on(stream, q.device):
            ws = attn_workspace(B, T, Hq, any_kv.heads, D, prefix.cap if prefix is not None else 0,
                                own.cap if own is not None else 0, score is not None, q.device)
    _check((_lib or lib()).mq_attn_prefix(q.data_ptr(), row, B, T, Hq, prefix._ref if prefix is not None else None,
                                          own_ref, len_ptr, D ** -0.5 if scale is None else scale, out.data_ptr(),
                                          _TYPES[out_type], lse_ptr, score_ptr, score_out_ptr,
                                          _dev_tensor(ws, torch.uint8, "ws").data_ptr(), ws.numel(), _stream(stream)),
           "mq_attn_prefix")
    return out


def mq_kv_evict(src: KV, length: torch.Tensor, score: torch.Tensor, keep: int, recent: int, dst: KV,
                length_out: torch.Tensor, score_out, index: torch.Tensor, stream=None) -> KV:
    """Keep, per sequence and key head, the `recent` last rows of src and the best `keep - recent`
    others by score (include/mq.h). length, length_out: int32 [n]; score: f32 [n, heads, src.cap];
    score_out (or None): f32 [n, heads, dst.cap]; index: int32 [n, heads, dst.cap], the rows kept.
    dst may be src: the rows then move in place."""
    if not isinstance(src, KV) or not isinstance(dst, KV):
        raise TypeError("src and dst must be KV")
    if _dev_tensor(length, torch.int32, "length").numel() != src.n:
        raise ValueError(f"length must hold {src.n} lengths")
    if _dev_tensor(length_out, torch.int32, "length_out").numel() != src.n:
        raise ValueError(f"length_out must hold {src.n} lengths")
    if _dev_tensor(score, torch.float32, "score").numel() < src.n * src.heads * src.cap:
        raise ValueError("score must be [n, heads, src.cap]")
    need = dst.n * dst.heads * dst.cap
    score_out_ptr = None
    if score_out is not None:
        if _dev_tensor(score_out, torch.float32, "score_out").numel() < need:
            raise ValueError("score_out must be [n, heads, dst.cap]")
        score_out_ptr = score_out.data_ptr()
    if _dev_tensor(index, torch.int32, "index").numel() < need:
        raise ValueError("index must be [n, heads, dst.cap]")
    _check((_lib or lib()).mq_kv_evict(src._ref, length.data_ptr(), score.data_ptr(), keep, recent, dst._ref,
                                       length_out.data_ptr(), score_out_ptr, index.data_ptr(), _stream(stream)),
           "mq_kv_evict")
    return dst


def mq_device_status(stream=None) -> int:
    return int(lib().mq_device_status(_stream(stream)))


def gemm_weights(kind: str, w: torch.Tensor, N: int, K: int, stream=None) -> torch.Tensor:
    """The weight form the GEMM reads: q6_K rows prepacked, every other type as it is."""
    return mq_prepack_q6k(w, N, K, stream=stream) if kind == "q6k" else w


def gemm(kind: str, a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    return {"q4k": mq_gemm_q4k, "q6k": mq_gemm_q6k, "q4_0": mq_gemm_q4_0, "q4_1": mq_gemm_q4_1}[kind](a, w, N, out,
                                                                                                 stream)


def gemv(kind: str, a: Plane, w: torch.Tensor, N: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    return {"q4k": mq_gemv_q4k, "q6k": mq_gemv_q6k, "q5k": mq_gemv_q5k, "q4_0": mq_gemv_q4_0,
            "q4_1": mq_gemv_q4_1}[kind](a, w, N, out, stream)
