"""ctypes binding of liblbq.so (include/lbq.h).

Argument marshalling only: torch tensors give device pointers and the current
HIP stream; every step of the computation runs in the library's kernels (or,
for ``pack``, in its host packer). There is no fallback: if the library is not
built, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# LBQ_LIBRARY may name another build of the same library (the sanitizer build)
LIB_PATH = os.environ.get("LBQ_LIBRARY") or os.path.join(_HERE, "liblbq.so")

FMT_RTN_PLANES = 0
FMT_PVQ_4x8 = 1
PATH_AUTO, PATH_GEMV, PATH_GEMM, PATH_GEMM_MX = 0, 1, 2, 3
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
PATH_SPLIT_ROTATION = 0x100   # test flag: the GEMM's rotation in launches of <= 3 tokens

STATUS = {
    0: "LBQ_OK", -1: "LBQ_ERR_NULL", -2: "LBQ_ERR_SHAPE", -3: "LBQ_ERR_BITS", -4: "LBQ_ERR_ALIGN",
    -5: "LBQ_ERR_WORKSPACE", -6: "LBQ_ERR_RANGE", -7: "LBQ_ERR_HIP", -8: "LBQ_ERR_FORMAT",
}

# Every symbol include/lbq.h declares.
EXPORTS = [
    "lbq_status_string", "lbq_packed_bytes", "lbq_pack", "lbq_linear_workspace", "lbq_linear_forward",
    "lbq_linear_forward_path", "lbq_linear_forward_timed", "lbq_moe_workspace", "lbq_moe_forward", "lbq_moe_route", "lbq_unpack_codes",
    "lbq_rotate", "lbq_linear_forward_noalloc", "lbq_stream_read", "lbq_gptq_factor",
    "lbq_pack_gptq", "lbq_moe_forward_path", "lbq_split_nibbles", "lbq_readout_workspace", "lbq_readout_screened",
    "lbq_mx_bytes", "lbq_mx_quantize", "lbq_mx_quantize_t", "lbq_mx_dequantize", "lbq_mx_matmul_workspace",
    "lbq_mx_matmul", "lbq_mx_linear_workspace", "lbq_mx_linear_forward", "lbq_mx_grouped_workspace",
    "lbq_mx_grouped_forward", "lbq_moe_sort_workspace", "lbq_moe_sort", "lbq_moe_gather", "lbq_moe_gather_backward",
    "lbq_moe_combine", "lbq_moe_combine_backward", "lbq_moe_select", "lbq_moe_select_backward",
    "lbq_adapters_workspace", "lbq_adapters_backward_workspace", "lbq_adapters_forward", "lbq_adapters_backward",
]


class LbqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


class Weight(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("N", ctypes.c_int32), ("bits", ctypes.c_int32), ("format", ctypes.c_int32),
                ("planes", ctypes.c_void_p), ("meta", ctypes.c_void_p), ("codebook", ctypes.c_void_p),
                ("signs", ctypes.c_void_p)]


class Moe(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("hidden", ctypes.c_int32), ("ffn", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("bits", ctypes.c_void_p), ("gu_plane_off", ctypes.c_void_p), ("gu_meta_off", ctypes.c_void_p),
                ("dn_plane_off", ctypes.c_void_p), ("dn_meta_off", ctypes.c_void_p), ("planes", ctypes.c_void_p),
                ("meta", ctypes.c_void_p), ("signs_hidden", ctypes.c_void_p), ("signs_ffn", ctypes.c_void_p)]


class Readout(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("N", ctypes.c_int32), ("hi_planes", ctypes.c_void_p),
                ("lo_planes", ctypes.c_void_p), ("hi_meta", ctypes.c_void_p), ("meta", ctypes.c_void_p),
                ("signs", ctypes.c_void_p)]


class Mx(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


class Router(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("top_k", ctypes.c_int32), ("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_picks", ctypes.c_int32), ("renormalise", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class AdaptersView(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32), ("r", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load liblbq.so from this package directory; raises if it is not built."""
    global _lib
    if _lib is None:
        # torch ships its own HIP runtime under the same soname as /opt/rocm's;
        # loading torch first makes the library bind to that one copy, so
        # torch's streams and allocations are valid handles for our launches.
        import torch  # noqa: F401
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run bit_weight_only_amd.build.build() first")
        L = ctypes.CDLL(LIB_PATH)
        c_i32, c_vp, c_sz = ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
        p_sz = ctypes.POINTER(ctypes.c_size_t)
        L.lbq_status_string.argtypes = [c_i32]
        L.lbq_status_string.restype = ctypes.c_char_p
        L.lbq_packed_bytes.argtypes = [c_i32, c_i32, c_i32, c_i32, p_sz, p_sz]
        L.lbq_pack.argtypes = [c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp]
        L.lbq_linear_workspace.argtypes = [ctypes.POINTER(Weight), c_i32, p_sz]
        L.lbq_linear_forward.argtypes = [ctypes.POINTER(Weight), c_vp, c_i32, c_vp, c_vp, c_sz, c_vp]
        L.lbq_linear_forward_path.argtypes = [ctypes.POINTER(Weight), c_vp, c_i32, c_vp, c_vp, c_sz, c_i32, c_vp]
        L.lbq_linear_forward_timed.argtypes = [ctypes.POINTER(Weight), c_vp, c_i32, c_vp, c_vp, c_sz, c_vp, c_vp, c_vp]
        L.lbq_moe_workspace.argtypes = [ctypes.POINTER(Moe), c_i32, p_sz]
        L.lbq_moe_forward.argtypes = [ctypes.POINTER(Moe), c_vp, c_vp, c_i32, c_vp, c_vp, c_sz, c_vp]
        L.lbq_moe_forward_path.argtypes = [ctypes.POINTER(Moe), c_vp, c_vp, c_i32, c_vp, c_vp, c_sz, c_i32, c_vp]
        L.lbq_moe_route.argtypes = [c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]
        L.lbq_unpack_codes.argtypes = [ctypes.POINTER(Weight), c_vp, c_vp]
        L.lbq_rotate.argtypes = [c_vp, c_i32, c_i32, c_vp, c_vp, c_vp]
        L.lbq_linear_forward_noalloc.argtypes = [ctypes.POINTER(Weight), c_vp, c_i32, c_vp, c_vp]
        L.lbq_stream_read.argtypes = [c_vp, c_sz, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp]
        L.lbq_gptq_factor.argtypes = [c_vp, c_i32, c_vp, ctypes.c_double, c_vp]
        L.lbq_pack_gptq.argtypes = [c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp]
        L.lbq_split_nibbles.argtypes = [c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp]
        L.lbq_readout_workspace.argtypes = [ctypes.POINTER(Readout), c_i32, c_i32, p_sz]
        L.lbq_readout_screened.argtypes = [ctypes.POINTER(Readout), c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_sz,
                                           c_vp]
        p_mx = ctypes.POINTER(Mx)
        L.lbq_mx_bytes.argtypes = [c_i32, c_i32, p_sz, p_sz]
        L.lbq_mx_quantize.argtypes = [c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp]
        L.lbq_mx_quantize_t.argtypes = [c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp]
        L.lbq_mx_dequantize.argtypes = [p_mx, c_vp, c_i32, c_vp]
        L.lbq_mx_matmul_workspace.argtypes = [p_mx, p_mx, p_sz]
        L.lbq_mx_matmul.argtypes = [p_mx, p_mx, c_vp, c_i32, c_vp, c_sz, c_vp]
        L.lbq_mx_linear_workspace.argtypes = [p_mx, c_i32, p_sz]
        L.lbq_mx_linear_forward.argtypes = [p_mx, c_vp, c_i32, c_vp, c_i32, c_vp, c_sz, c_vp]
        L.lbq_mx_grouped_workspace.argtypes = [p_mx, c_i32, c_i32, c_i32, p_sz]
        L.lbq_mx_grouped_forward.argtypes = [p_mx, c_i32, c_vp, c_i32, c_vp, c_vp, c_i32, c_i32, c_vp, c_i32, c_vp, c_sz,
                                             c_vp]
        L.lbq_moe_sort_workspace.argtypes = [c_i32, c_i32, c_i32, p_sz]
        L.lbq_moe_sort.argtypes = [c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]
        L.lbq_moe_gather.argtypes = [c_vp, c_i32, c_i32, c_i32, c_vp, c_i32, c_i32, c_vp, c_vp]
        L.lbq_moe_gather_backward.argtypes = [c_vp, c_i32, c_i32, c_i32, c_vp, c_i32, c_i32, c_vp, c_vp]
        L.lbq_moe_combine.argtypes = [c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp]
        L.lbq_moe_combine_backward.argtypes = [c_vp, c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp,
                                               c_vp]
        p_ad, p_router = ctypes.POINTER(AdaptersView), ctypes.POINTER(Router)
        L.lbq_moe_select.argtypes = [p_router, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp]
        L.lbq_moe_select_backward.argtypes = [p_router, c_vp, c_vp, c_i32, c_vp, c_i32, c_vp, c_vp]
        L.lbq_adapters_workspace.argtypes = [p_ad, c_i32, c_i32, p_sz]
        L.lbq_adapters_backward_workspace.argtypes = [p_ad, c_i32, c_i32, p_sz]
        L.lbq_adapters_forward.argtypes = [p_ad, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]
        L.lbq_adapters_backward.argtypes = [p_ad, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                            c_sz, c_vp]
        for name in EXPORTS:
            if name != "lbq_status_string":
                getattr(L, name).restype = c_i32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().lbq_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise LbqError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# ------------------------------------------------------------------ host packing

def packed_bytes(K: int, N: int, bits: int, fmt: int = FMT_RTN_PLANES):
    pb, mb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().lbq_packed_bytes(K, N, bits, fmt, ctypes.byref(pb), ctypes.byref(mb)), "lbq_packed_bytes")
    return pb.value, mb.value


def pack(W: np.ndarray, bits: int, signs: np.ndarray, fmt: int = FMT_RTN_PLANES, codebook: np.ndarray | None = None):
    """Pack fp32 W [N][K] on the host. Returns (planes, meta) as uint8 numpy arrays."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    signs = np.ascontiguousarray(signs, dtype=np.int8)
    pb, mb = packed_bytes(K, N, bits, fmt)
    planes = np.empty(pb, dtype=np.uint8)
    meta = np.empty(mb, dtype=np.uint8)
    cb = None if codebook is None else np.ascontiguousarray(codebook, dtype=np.uint8)
    st = lib().lbq_pack(W.ctypes.data, K, N, bits, fmt, signs.ctypes.data,
                        None if cb is None else cb.ctypes.data, planes.ctypes.data, meta.ctypes.data)
    _check(st, "lbq_pack")
    return planes, meta


def gptq_factor(H: np.ndarray, signs: np.ndarray, damp: float = 0.01) -> np.ndarray:
    """lbq_gptq_factor: U [K][K] float64 from a host Hessian H [K][K] (original basis)."""
    H = np.ascontiguousarray(H, dtype=np.float64)
    K = H.shape[0]
    signs = np.ascontiguousarray(signs, dtype=np.int8)
    U = np.empty((K, K), dtype=np.float64)
    _check(lib().lbq_gptq_factor(H.ctypes.data, K, signs.ctypes.data, float(damp), U.ctypes.data), "lbq_gptq_factor")
    return U


def pack_gptq(W: np.ndarray, bits: int, signs: np.ndarray, U: np.ndarray):
    """lbq_pack_gptq: (planes, meta) uint8 arrays in the RTN bit-plane format."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    signs = np.ascontiguousarray(signs, dtype=np.int8)
    U = np.ascontiguousarray(U, dtype=np.float64)
    pb, mb = packed_bytes(K, N, bits, FMT_RTN_PLANES)
    planes = np.empty(pb, dtype=np.uint8)
    meta = np.empty(mb, dtype=np.uint8)
    _check(lib().lbq_pack_gptq(W.ctypes.data, K, N, bits, signs.ctypes.data, U.ctypes.data, planes.ctypes.data,
                               meta.ctypes.data), "lbq_pack_gptq")
    return planes, meta


# ------------------------------------------------------------------ device side

class PackedLinear:
    """Device-resident packed weight (caller-owned torch tensors) and its lbq_weight view."""

    def __init__(self, K, N, bits, fmt, planes, meta, signs, codebook=None):
        self.K, self.N, self.bits, self.fmt = int(K), int(N), int(bits), int(fmt)
        self.planes, self.meta, self.signs, self.codebook = planes, meta, signs, codebook
        self._w = Weight(self.K, self.N, self.bits, self.fmt, planes.data_ptr(), meta.data_ptr(),
                         0 if codebook is None else codebook.data_ptr(), signs.data_ptr())

    @classmethod
    def from_host(cls, planes: np.ndarray, meta: np.ndarray, signs: np.ndarray, K: int, N: int, bits: int,
                  fmt: int = FMT_RTN_PLANES, codebook: np.ndarray | None = None, device="cuda"):
        import torch

        def up(a):
            return torch.from_numpy(np.ascontiguousarray(a).view(np.uint8).reshape(-1)).to(device)

        return cls(K, N, bits, fmt, up(planes), up(meta), torch.from_numpy(np.ascontiguousarray(signs, np.int8)).to(device),
                   None if codebook is None else up(codebook))

    @property
    def struct(self) -> Weight:
        return self._w

    def workspace_bytes(self, M: int) -> int:
        b = ctypes.c_size_t()
        _check(lib().lbq_linear_workspace(ctypes.byref(self._w), int(M), ctypes.byref(b)), "lbq_linear_workspace")
        return b.value


def linear_forward(w: PackedLinear, x, y=None, ws=None, path: int = PATH_AUTO, stream=None):
    """y[M][N] = x[M][K] W_hat^T on the GPU (fp16 in, fp16 out)."""
    import torch

    M = int(x.shape[0])
    if y is None:
        y = torch.empty((M, w.N), dtype=torch.float16, device=x.device)
    if ws is None:
        ws = torch.empty(max(1, w.workspace_bytes(M)), dtype=torch.uint8, device=x.device)
    st = lib().lbq_linear_forward_path(ctypes.byref(w.struct), _ptr(x), M, _ptr(y), _ptr(ws), ws.numel(), int(path),
                                       _stream(stream))
    _check(st, "lbq_linear_forward")
    return y


def linear_forward_noalloc(w: PackedLinear, x, y=None, stream=None):
    """lbq_linear_forward_noalloc: y = x W_hat^T with the library's static device scratch (no workspace)."""
    import torch

    M = int(x.shape[0])
    if y is None:
        y = torch.empty((M, w.N), dtype=torch.float16, device=x.device)
    _check(lib().lbq_linear_forward_noalloc(ctypes.byref(w.struct), _ptr(x), M, _ptr(y), _stream(stream)),
           "lbq_linear_forward_noalloc")
    return y


def rotate(x, signs, out=None, stream=None):
    import torch

    M, K = int(x.shape[0]), int(x.shape[1])
    if out is None:
        out = torch.empty_like(x)
    _check(lib().lbq_rotate(_ptr(x), M, K, _ptr(signs), _ptr(out), _stream(stream)), "lbq_rotate")
    return out


def unpack_codes(w: PackedLinear, stream=None):
    import torch

    # RTN: codes [N][K]; product-VQ: indices [stages * N][K/4] (stage-major)
    n = w.N * w.K if w.fmt == FMT_RTN_PLANES else (w.bits // 2) * w.N * (w.K // 4)
    codes = torch.empty(n, dtype=torch.uint8, device=w.planes.device)
    _check(lib().lbq_unpack_codes(ctypes.byref(w.struct), _ptr(codes), _stream(stream)), "lbq_unpack_codes")
    return codes.view(w.N, -1) if w.fmt == FMT_RTN_PLANES else codes.view(-1, w.K // 4)


# ------------------------------------------------------------------ screened readout

def split_nibbles(planes8: np.ndarray, meta8: np.ndarray, K: int, N: int):
    """lbq_split_nibbles on the host: (hi_planes, lo_planes, hi_meta) as uint8 arrays."""
    planes8 = np.ascontiguousarray(planes8).view(np.uint8)
    meta8 = np.ascontiguousarray(meta8).view(np.uint8)
    G = K // 128
    hi = np.empty(N * G * 64, np.uint8)
    lo = np.empty(N * G * 64, np.uint8)
    hm = np.empty(N * G * 4, np.uint8)
    _check(lib().lbq_split_nibbles(planes8.ctypes.data, meta8.ctypes.data, K, N, hi.ctypes.data, lo.ctypes.data,
                                   hm.ctypes.data), "lbq_split_nibbles")
    return hi, lo, hm


class PackedReadout:
    """Device-resident nibble-split readout weight and its lbq_readout view."""

    def __init__(self, K, N, hi_planes, lo_planes, hi_meta, meta, signs):
        self.K, self.N = int(K), int(N)
        self.hi_planes, self.lo_planes, self.hi_meta, self.meta, self.signs = hi_planes, lo_planes, hi_meta, meta, signs
        self._r = Readout(self.K, self.N, hi_planes.data_ptr(), lo_planes.data_ptr(), hi_meta.data_ptr(),
                          meta.data_ptr(), signs.data_ptr())

    @classmethod
    def from_host(cls, planes8: np.ndarray, meta8: np.ndarray, signs: np.ndarray, K: int, N: int, device="cuda"):
        import torch

        hi, lo, hm = split_nibbles(planes8, meta8, K, N)

        def up(a):
            return torch.from_numpy(np.ascontiguousarray(a).view(np.uint8).reshape(-1)).to(device)

        return cls(K, N, up(hi), up(lo), up(hm), up(meta8), torch.from_numpy(np.ascontiguousarray(signs, np.int8)).to(device))

    @property
    def struct(self) -> Readout:
        return self._r

    def workspace_bytes(self, M: int, cand: int) -> int:
        b = ctypes.c_size_t()
        _check(lib().lbq_readout_workspace(ctypes.byref(self._r), int(M), int(cand), ctypes.byref(b)),
               "lbq_readout_workspace")
        return b.value


def readout_screened(r: PackedReadout, x, cand: int, ws=None, stream=None):
    """lbq_readout_screened: (coarse fp16 [M][N], ids int32 [M][cand], exact logits fp32 [M][cand])."""
    import torch

    M = int(x.shape[0])
    coarse = torch.empty((M, r.N), dtype=torch.float16, device=x.device)
    ids = torch.empty((M, cand), dtype=torch.int32, device=x.device)
    logits = torch.empty((M, cand), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = torch.empty(max(1, r.workspace_bytes(M, cand)), dtype=torch.uint8, device=x.device)
    _check(lib().lbq_readout_screened(ctypes.byref(r.struct), _ptr(x), M, int(cand), _ptr(coarse), _ptr(ids),
                                      _ptr(logits), _ptr(ws), ws.numel(), _stream(stream)), "lbq_readout_screened")
    return coarse, ids, logits


# ------------------------------------------------------------------ MoE

class PackedMoe:
    """Device-resident routed-expert block: all experts' planes and meta in two
    byte buffers with per-expert offsets (see lbq_moe in include/lbq.h)."""

    def __init__(self, E, hidden, ffn, top_k, bits, gu_plane_off, gu_meta_off, dn_plane_off, dn_meta_off, planes, meta,
                 signs_hidden, signs_ffn):
        self.E, self.hidden, self.ffn, self.top_k = int(E), int(hidden), int(ffn), int(top_k)
        self.tensors = (bits, gu_plane_off, gu_meta_off, dn_plane_off, dn_meta_off, planes, meta, signs_hidden,
                        signs_ffn)
        self._m = Moe(self.E, self.hidden, self.ffn, self.top_k, *[t.data_ptr() for t in self.tensors])

    @property
    def struct(self) -> Moe:
        return self._m

    def workspace_bytes(self, M: int) -> int:
        b = ctypes.c_size_t()
        _check(lib().lbq_moe_workspace(ctypes.byref(self._m), int(M), ctypes.byref(b)), "lbq_moe_workspace")
        return b.value


def moe_forward(m: PackedMoe, x, logits, y=None, ws=None, path: int = PATH_AUTO, stream=None):
    import torch

    M = int(x.shape[0])
    if y is None:
        y = torch.empty((M, m.hidden), dtype=torch.float16, device=x.device)
    if ws is None:
        ws = torch.empty(max(1, m.workspace_bytes(M)), dtype=torch.uint8, device=x.device)
    st = lib().lbq_moe_forward_path(ctypes.byref(m.struct), _ptr(x), _ptr(logits), M, _ptr(y), _ptr(ws), ws.numel(),
                                    int(path), _stream(stream))
    _check(st, "lbq_moe_forward")
    return y


def moe_route(logits, top_k: int, stream=None):
    """Returns (ids, weights, counts, offsets, perm) device tensors."""
    import torch

    M, E = int(logits.shape[0]), int(logits.shape[1])
    dev = logits.device
    ids = torch.empty((M, top_k), dtype=torch.int32, device=dev)
    wts = torch.empty((M, top_k), dtype=torch.float32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(max(1, M * top_k), dtype=torch.int32, device=dev)
    st = lib().lbq_moe_route(_ptr(logits), M, E, int(top_k), _ptr(ids), _ptr(wts), _ptr(counts), _ptr(offsets),
                             _ptr(perm), _stream(stream))
    _check(st, "lbq_moe_route")
    return ids, wts, counts, offsets, perm[:M * top_k]


def pack_moe_host(w_gu, w_dn, bits, signs_hidden, signs_ffn, align: int = 256):
    """Pack E experts on the host into the lbq_moe buffers.

    w_gu(e) -> fp32 [2*ffn][hidden] (gate rows first), w_dn(e) -> fp32 [hidden][ffn];
    bits: uint8 [E]. Returns a dict of numpy arrays: planes, meta (uint8),
    gu_plane_off, gu_meta_off, dn_plane_off, dn_meta_off (uint64 [E]).
    """
    E = len(bits)
    pieces_p, pieces_m = [], []
    offs = {k: np.zeros(E, dtype=np.uint64) for k in ("gu_plane_off", "gu_meta_off", "dn_plane_off", "dn_meta_off")}
    pos_p = pos_m = 0

    def put(lst, arr, pos):
        pad = (-pos) % align
        if pad:
            lst.append(np.zeros(pad, np.uint8))
        start = pos + pad
        lst.append(arr)
        return start, start + arr.size

    for e in range(E):
        b = int(bits[e])
        gp, gm = pack(w_gu(e), b, signs_hidden)
        dp, dm = pack(w_dn(e), b, signs_ffn)
        offs["gu_plane_off"][e], pos_p = put(pieces_p, gp, pos_p)
        offs["dn_plane_off"][e], pos_p = put(pieces_p, dp, pos_p)
        offs["gu_meta_off"][e], pos_m = put(pieces_m, gm, pos_m)
        offs["dn_meta_off"][e], pos_m = put(pieces_m, dm, pos_m)
    out = dict(planes=np.concatenate(pieces_p), meta=np.concatenate(pieces_m))
    out.update(offs)
    return out


def moe_from_host(packed: dict, bits, signs_hidden, signs_ffn, hidden: int, ffn: int, top_k: int, device="cuda"):
    import torch

    def up(a, dt=None):
        t = torch.from_numpy(np.ascontiguousarray(a))
        return t.to(device)

    return PackedMoe(len(bits), hidden, ffn, top_k, up(np.asarray(bits, np.uint8)),
                     up(packed["gu_plane_off"].view(np.int64)), up(packed["gu_meta_off"].view(np.int64)),
                     up(packed["dn_plane_off"].view(np.int64)), up(packed["dn_meta_off"].view(np.int64)),
                     up(packed["planes"]), up(packed["meta"]), up(np.asarray(signs_hidden, np.int8)),
                     up(np.asarray(signs_ffn, np.int8)))


# ------------------------------------------------------------------ MXFP4 tensors, expert dispatch
#
# These take torch tensors as they are used in a program, so they check them:
# one GPU, contiguous, the right type and shape (LbqError otherwise, nothing
# launched). They run on the tensors' GPU whatever the current one is, on the
# given stream or that GPU's current one; what they allocate belongs to that
# stream. On a given stream the caller orders the work before and after, but may
# let go of the tensors as soon as the call returns: their memory is not given
# out again before the stream is through with them. A call's own cost counts at
# one token (its kernels take 5 us), so the usual path keeps to a few attribute
# reads, one or two allocations and one foreign call. Results carry no
# gradient, whatever the inputs require: the gradients are calls of their own.

F16, BF16, F32 = 0, 1, 2
_MOST = 2 ** 31 - 1   # a size of the C ABI; ctypes would cut a larger one off without a word
_torch = None
_dtypes: dict = {}


def _ready():
    """The library and torch, loaded on first use."""
    global _torch
    L = lib()
    if _torch is None:
        import torch

        _dtypes.update({torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32})
        _torch = torch
    return L


def _dtype(t, where: str) -> int:
    code = _dtypes.get(t)
    if code is None:
        raise LbqError(-8, f"{where}: {t}")
    return code


def _need(where: str, gpu: int, dtype, shape, t):
    """t is contiguous, on that GPU, of this dtype and (where given) shape."""
    if gpu < 0 or t.get_device() != gpu:
        raise LbqError(-8, f"{where}: a tensor on {t.device}, another on {'no GPU' if gpu < 0 else gpu}")
    if t.dtype is not dtype:
        raise LbqError(-8, f"{where}: {t.dtype} instead of {dtype}")
    if not t.is_contiguous() or (shape is not None and t.shape != shape):
        raise LbqError(-2, f"{where}: shape {tuple(t.shape)}, strides {t.stride()}")


def _rows(where: str, t):
    """(GPU, rows, columns) of t, a contiguous matrix in a value type."""
    if t.dim() != 2:
        raise LbqError(-2, f"{where}: a matrix is needed, got {tuple(t.shape)}")
    rows, cols = t.shape
    if rows > _MOST or cols > _MOST:
        raise LbqError(-2, f"{where}: {rows} x {cols}")
    gpu = t.get_device()
    _need(where, gpu, t.dtype, None, t)
    return gpu, rows, cols


def _on(gpu: int, stream, go, *used):
    """go(raw stream) with that GPU current and its allocations on that stream; used: the caller's tensors."""
    cuda = _torch._C
    if stream is None:
        if cuda._cuda_getDevice() == gpu:
            return go(cuda._cuda_getCurrentRawStream(gpu))
        with _torch.cuda.device(gpu):
            return go(cuda._cuda_getCurrentRawStream(gpu))
    if stream.device.index != gpu:
        raise LbqError(-8, f"stream on {stream.device}, tensors on GPU {gpu}")
    with _torch.cuda.stream(stream):
        try:
            return go(stream.cuda_stream)
        finally:
            for t in used:
                if t is not None:
                    t.record_stream(stream)


@functools.lru_cache(maxsize=4096)
def _query(name: str, args: tuple) -> int:
    """A *_workspace query; sizes alone decide it. Tensors are given as (rows, cols)."""
    for a in args:
        for n in a if isinstance(a, tuple) else (a,):
            if not -_MOST <= n <= _MOST:
                raise LbqError(-2, f"{name}: {args}")
    need = ctypes.c_size_t()
    p = ctypes.c_void_p(16)   # aligned stand-in: queries look at sizes only
    views = [Mx(a[0], a[1], p, p) if isinstance(a, tuple) else a for a in args]
    f = getattr(lib(), name)
    _check(f(*[ctypes.byref(v) if isinstance(v, Mx) else v for v in views], ctypes.byref(need)), name)
    return need.value


def _workspace(ws, need: int, like, gpu: int, where: str):
    """(pointer, bytes, owner) of a workspace: the caller's, or one of need bytes."""
    if ws is None:
        if need == 0:
            return None, 0, None
        ws = like.new_empty(need, dtype=_torch.uint8)
        return ws.data_ptr(), need, ws
    if ws.get_device() != gpu or not ws.is_contiguous():
        raise LbqError(-5, where)
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


class MxTensor:
    """An MXFP4 tensor (see include/lbq.h): codes uint8 [rows][cols/2] and scales uint8 [cols/128][rows][4].

    It keeps both tensors and their addresses: what they hold may change, the tensors may not be replaced."""

    __slots__ = ("rows", "cols", "_codes", "_scales", "gpu", "struct", "ref")

    def __init__(self, codes, scales):
        _ready()
        if codes.dim() != 2 or codes.shape[1] % 64 or codes.shape[1] == 0:
            raise LbqError(-2, "MxTensor: codes are [rows][cols/2], cols a positive multiple of 128")
        rows, half = codes.shape
        if rows > _MOST or 2 * half > _MOST:
            raise LbqError(-2, f"MxTensor: {rows} x {2 * half}")
        gpu = codes.get_device()
        _need("MxTensor", gpu, _torch.uint8, None, codes)
        _need("MxTensor", gpu, _torch.uint8, (half // 64, rows, 4), scales)
        self._set(codes, scales, rows, 2 * half, gpu)

    def _set(self, codes, scales, rows, cols, gpu):
        self.rows, self.cols, self._codes, self._scales, self.gpu = rows, cols, codes, scales, gpu
        self.struct = Mx(rows, cols, codes.data_ptr(), scales.data_ptr())
        self.ref = ctypes.byref(self.struct)
        return self

    @property
    def codes(self):
        return self._codes

    @property
    def scales(self):
        return self._scales

    @property
    def device(self):
        return self._codes.device


def mx_quantize(x, transpose: bool = False, stream=None) -> MxTensor:
    """lbq_mx_quantize (transpose: lbq_mx_quantize_t, of one row at least) of x [rows][cols] in float16, bfloat16 or
    float32."""
    L = _ready()
    gpu, rows, cols = _rows("mx_quantize", x)
    dt = _dtype(x.dtype, "mx_quantize")
    tr, tc = (cols, -(-rows // 128) * 128) if transpose else (rows, cols)
    if tc % 128 or tc == 0:
        raise LbqError(-2, "mx_quantize: blocks run along a multiple of 128 values")

    def go(s):
        codes = x.new_empty((tr, tc // 2), dtype=_torch.uint8)
        scales = x.new_empty((tc // 128, tr, 4), dtype=_torch.uint8)
        f = L.lbq_mx_quantize_t if transpose else L.lbq_mx_quantize
        st = f(x.data_ptr(), dt, rows, cols, codes.data_ptr(), scales.data_ptr(), s)
        if st:
            raise LbqError(st, "lbq_mx_quantize_t" if transpose else "lbq_mx_quantize")
        return MxTensor.__new__(MxTensor)._set(codes, scales, tr, tc, gpu)
    return _on(gpu, stream, go, x)


def mx_dequantize(t: MxTensor, dtype, out=None, stream=None):
    """lbq_mx_dequantize: the values of t as a [rows][cols] tensor of dtype."""
    L = _ready()
    dt = _dtype(dtype, "mx_dequantize")
    if out is not None:
        _need("mx_dequantize", t.gpu, dtype, (t.rows, t.cols), out)

    def go(s):
        y = t._codes.new_empty((t.rows, t.cols), dtype=dtype) if out is None else out
        st = L.lbq_mx_dequantize(t.ref, y.data_ptr(), dt, s)
        if st:
            raise LbqError(st, "lbq_mx_dequantize")
        return y
    return _on(t.gpu, stream, go, t._codes, t._scales, out)


def mx_matmul(a: MxTensor, b: MxTensor, dtype=None, y=None, ws=None, stream=None):
    """lbq_mx_matmul: y [a.rows][b.rows] = A B^T in dtype (float32 if neither it nor y is given). Autograd does not
    see it: a layer's gradients are two more of these products."""
    L = _ready()
    if a.gpu != b.gpu:
        raise LbqError(-8, f"mx_matmul: tensors on {a.device} and {b.device}")
    if dtype is None:
        dtype = _torch.float32 if y is None else y.dtype
    dt = _dtype(dtype, "mx_matmul")
    if y is not None:
        _need("mx_matmul", a.gpu, dtype, (a.rows, b.rows), y)
    need = _query("lbq_mx_matmul_workspace", ((a.rows, a.cols), (b.rows, b.cols)))

    def go(s):
        out = a._codes.new_empty((a.rows, b.rows), dtype=dtype) if y is None else y
        p, size, keep = _workspace(ws, need, a._codes, a.gpu, "mx_matmul")
        st = L.lbq_mx_matmul(a.ref, b.ref, out.data_ptr(), dt, p, size, s)
        if st:
            raise LbqError(st, "lbq_mx_matmul")
        return out
    return _on(a.gpu, stream, go, a._codes, a._scales, b._codes, b._scales, y, ws)


def mx_linear_forward(w: MxTensor, x, y=None, ws=None, stream=None):
    """lbq_mx_linear_forward: y [M][w.rows] = Q(x) W^T, x [M][w.cols] in float16 or bfloat16, y in x's type; x is
    rounded to MXFP4 too. Autograd does not see it."""
    L = _ready()
    dtype = x.dtype
    dt = _dtype(dtype, "mx_linear_forward")
    _need("mx_linear_forward", w.gpu, dtype, None, x)
    if x.dim() != 2 or x.shape[1] != w.cols:
        raise LbqError(-2, "mx_linear_forward: x is [M][w.cols]")
    M = x.shape[0]
    if y is not None:
        _need("mx_linear_forward", w.gpu, dtype, (M, w.rows), y)
    need = _query("lbq_mx_linear_workspace", ((w.rows, w.cols), M))

    def go(s):
        out = x.new_empty((M, w.rows)) if y is None else y
        p, size, keep = _workspace(ws, need, x, w.gpu, "mx_linear_forward")
        st = L.lbq_mx_linear_forward(w.ref, x.data_ptr(), M, out.data_ptr(), dt, p, size, s)
        if st:
            raise LbqError(st, "lbq_mx_linear_forward")
        return out
    return _on(w.gpu, stream, go, w._codes, w._scales, x, y, ws)


def mx_grouped_forward(w: MxTensor, E: int, x, offsets, perm=None, top_k: int = 1, y=None, ws=None, stream=None):
    """lbq_mx_grouped_forward: w holds E experts of w.rows / E rows; y [T][w.rows / E], T the length of perm
    (of x without perm). Rows of y from offsets[E] on are left as they were (uninitialised if y is not given).
    Autograd does not see it."""
    L = _ready()
    where, gpu, dtype = "mx_grouped_forward", w.gpu, x.dtype
    dt = _dtype(dtype, where)
    _need(where, gpu, dtype, None, x)
    if x.dim() != 2 or x.shape[1] != w.cols:
        raise LbqError(-2, "mx_grouped_forward: x is [M][w.cols]")
    if E < 1 or w.rows % E or not 1 <= top_k <= _MOST:
        raise LbqError(-2, f"mx_grouped_forward: w holds E experts of equal rows; E {E}, top_k {top_k}")
    M, N = x.shape[0], w.rows // E
    _need(where, gpu, _torch.int32, (E + 1,), offsets)
    T = M
    if perm is not None:
        _need(where, gpu, _torch.int32, None, perm)
        T = perm.numel()
    if y is not None:
        _need(where, gpu, dtype, (T, N), y)
    need = _query("lbq_mx_grouped_workspace", ((w.rows, w.cols), E, M, T))

    def go(s):
        out = x.new_empty((T, N)) if y is None else y
        p, size, keep = _workspace(ws, need, x, gpu, where)
        st = L.lbq_mx_grouped_forward(w.ref, E, x.data_ptr(), M, offsets.data_ptr(),
                                      None if perm is None else perm.data_ptr(), top_k, T, out.data_ptr(), dt, p, size,
                                      s)
        if st:
            raise LbqError(st, "lbq_mx_grouped_forward")
        return out
    return _on(gpu, stream, go, w._codes, w._scales, x, offsets, perm, y, ws)


def moe_sort(ids, E: int, stream=None):
    """lbq_moe_sort of ids int32 [M][top_k]: (counts [E], offsets [E+1], perm [M*top_k], pos [M][top_k])."""
    L = _ready()
    gpu = ids.get_device()
    _need("moe_sort", gpu, _torch.int32, None, ids)
    if ids.dim() != 2:
        raise LbqError(-2, "moe_sort: ids are [M][top_k]")
    M, k = ids.shape
    need = _query("lbq_moe_sort_workspace", (M, E, k))
    n = M * k

    def go(s):
        pos = ids.new_empty((M, k))
        perm, counts, offsets, ws = ids.new_empty(n + 2 * E + 1 + need // 4).split((n, E, E + 1, need // 4))
        st = L.lbq_moe_sort(ids.data_ptr(), M, E, k, counts.data_ptr(), offsets.data_ptr(), perm.data_ptr(),
                            pos.data_ptr(), ws.data_ptr(), need, s)
        if st:
            raise LbqError(st, "lbq_moe_sort")
        return counts, offsets, perm, pos
    return _on(gpu, stream, go, ids)


def _places(where: str, gpu: int, pos):
    _need(where, gpu, _torch.int32, None, pos)
    if pos.dim() != 2:
        raise LbqError(-2, f"{where}: pos is [M][top_k]")
    M, k = pos.shape
    if M > _MOST or k > _MOST:
        raise LbqError(-2, f"{where}: {M} x {k} places")
    return M, k


def moe_gather(x, pos, out=None, stream=None):
    """lbq_moe_gather: out[pos[t][j]] = x[t]. out [T][H] is [M * top_k][H] if not given; rows that no place
    names are left as they were (uninitialised if out is not given). Autograd does not see it; its gradient is
    moe_gather_backward."""
    L = _ready()
    gpu, rows, H = _rows("moe_gather", x)
    dt = _dtype(x.dtype, "moe_gather")
    M, k = _places("moe_gather", gpu, pos)
    if rows != M:
        raise LbqError(-2, f"moe_gather: {rows} rows, places of {M}")
    T = M * k
    if out is not None:
        T = out.shape[0] if out.dim() == 2 else -1
        if not 0 <= T <= _MOST:
            raise LbqError(-2, f"moe_gather: out is [T][H], got {tuple(out.shape)}")
        _need("moe_gather", gpu, x.dtype, (T, H), out)

    def go(s):
        o = x.new_empty((T, H)) if out is None else out
        st = L.lbq_moe_gather(x.data_ptr(), dt, M, H, pos.data_ptr(), k, T, o.data_ptr(), s)
        if st:
            raise LbqError(st, "lbq_moe_gather")
        return o
    return _on(gpu, stream, go, x, pos, out)


def moe_gather_backward(d_out, pos, dx=None, stream=None):
    """lbq_moe_gather_backward: dx[t] = sum_j d_out[pos[t][j]]."""
    L = _ready()
    gpu, T, H = _rows("moe_gather_backward", d_out)
    dt = _dtype(d_out.dtype, "moe_gather_backward")
    M, k = _places("moe_gather_backward", gpu, pos)
    if dx is not None:
        _need("moe_gather_backward", gpu, d_out.dtype, (M, H), dx)

    def go(s):
        o = d_out.new_empty((M, H)) if dx is None else dx
        st = L.lbq_moe_gather_backward(d_out.data_ptr(), dt, T, H, pos.data_ptr(), M, k, o.data_ptr(), s)
        if st:
            raise LbqError(st, "lbq_moe_gather_backward")
        return o
    return _on(gpu, stream, go, d_out, pos, dx)


def moe_combine(o, pos, weights, y=None, stream=None):
    """lbq_moe_combine: y[t] = sum_j weights[t][j] o[pos[t][j]] (weights float32 [M][top_k]). Autograd does not see
    it; its gradients are moe_combine_backward."""
    L = _ready()
    gpu, T, H = _rows("moe_combine", o)
    dt = _dtype(o.dtype, "moe_combine")
    M, k = _places("moe_combine", gpu, pos)
    _need("moe_combine", gpu, _torch.float32, (M, k), weights)
    if y is not None:
        _need("moe_combine", gpu, o.dtype, (M, H), y)

    def go(s):
        out = o.new_empty((M, H)) if y is None else y
        st = L.lbq_moe_combine(o.data_ptr(), dt, T, H, pos.data_ptr(), weights.data_ptr(), M, k, out.data_ptr(), s)
        if st:
            raise LbqError(st, "lbq_moe_combine")
        return out
    return _on(gpu, stream, go, o, pos, weights, y)


def moe_combine_backward(dy, o, pos, weights, d_o=None, d_weights=None, stream=None):
    """lbq_moe_combine_backward: (d_o [T][H], d_weights float32 [M][top_k]). Rows of d_o that no place names are
    left as they were (uninitialised if d_o is not given)."""
    L = _ready()
    where = "moe_combine_backward"
    gpu, T, H = _rows(where, o)
    dt = _dtype(o.dtype, where)
    M, k = _places(where, gpu, pos)
    _need(where, gpu, _torch.float32, (M, k), weights)
    _need(where, gpu, o.dtype, (M, H), dy)
    if d_o is not None:
        _need(where, gpu, o.dtype, (T, H), d_o)
    if d_weights is not None:
        _need(where, gpu, _torch.float32, (M, k), d_weights)

    def go(s):
        go_, gw = o.new_empty((T, H)) if d_o is None else d_o, d_weights
        if gw is None:
            gw = weights.new_empty((M, k))
        st = L.lbq_moe_combine_backward(dy.data_ptr(), o.data_ptr(), dt, T, H, pos.data_ptr(), weights.data_ptr(), M,
                                        k, go_.data_ptr(), gw.data_ptr(), s)
        if st:
            raise LbqError(st, "lbq_moe_combine_backward")
        return go_, gw
    return _on(gpu, stream, go, dy, o, pos, weights, d_o, d_weights)


# ------------------------------------------------------------------ expert selection

def _router(E, top_k, score, groups, top_groups, group_picks, renormalise, scale):
    """The struct of these settings, kept by their values: what can change in place (a tensor as scale) is read now."""
    at = operator.index
    return _router_of(E, at(top_k), at(score), at(groups), at(top_groups), at(group_picks), bool(renormalise), float(scale))


@functools.lru_cache(maxsize=256)
def _router_of(E, top_k, score, groups, top_groups, group_picks, renormalise, scale):
    for n in (E, top_k, score, groups, top_groups, group_picks):
        if not -_MOST <= n <= _MOST:
            raise LbqError(-2, f"router: {n}")
    return ctypes.byref(Router(E, top_k, score, groups, top_groups, group_picks, renormalise, scale))


def moe_select(logits, top_k: int, bias=None, score: int = SCORE_SOFTMAX, groups: int = 1, top_groups: int = 1,
               group_picks: int = 1, renormalise: bool = True, scale: float = 1.0, ids=None, weights=None, stream=None):
    """lbq_moe_select of logits [M][E] (float16, bfloat16 or float32): (ids int32, weights float32), both [M][top_k].
    Autograd does not see it; its gradient is moe_select_backward."""
    L = _ready()
    gpu, M, E = _rows("moe_select", logits)
    dt = _dtype(logits.dtype, "moe_select")
    r = _router(E, top_k, score, groups, top_groups, group_picks, renormalise, scale)
    if bias is not None:
        _need("moe_select", gpu, _torch.float32, (E,), bias)
    if ids is not None:
        _need("moe_select", gpu, _torch.int32, (M, top_k), ids)
    if weights is not None:
        _need("moe_select", gpu, _torch.float32, (M, top_k), weights)

    def go(s):
        i = logits.new_empty((M, top_k), dtype=_torch.int32) if ids is None else ids
        w = logits.new_empty((M, top_k), dtype=_torch.float32) if weights is None else weights
        st = L.lbq_moe_select(r, logits.data_ptr(), dt, M, None if bias is None else bias.data_ptr(), i.data_ptr(),
                              w.data_ptr(), s)
        if st:
            raise LbqError(st, "lbq_moe_select")
        return i, w
    return _on(gpu, stream, go, logits, bias, ids, weights)


def moe_select_backward(d_weights, logits, ids, score: int = SCORE_SOFTMAX, renormalise: bool = True,
                        scale: float = 1.0, d_logits=None, stream=None):
    """lbq_moe_select_backward: d_logits [M][E] in logits' type, for moe_select's ids of these logits (the bias and the
    groups have no part in it)."""
    L = _ready()
    where = "moe_select_backward"
    gpu, M, E = _rows(where, logits)
    dt = _dtype(logits.dtype, where)
    if ids.dim() != 2:
        raise LbqError(-2, f"{where}: ids are [M][top_k]")
    k = ids.shape[1]
    _need(where, gpu, _torch.int32, (M, k), ids)
    _need(where, gpu, _torch.float32, (M, k), d_weights)
    if d_logits is not None:
        _need(where, gpu, logits.dtype, (M, E), d_logits)
    r = _router(E, k, score, 1, 1, 1, renormalise, scale)

    def go(s):
        d = logits.new_empty((M, E)) if d_logits is None else d_logits
        st = L.lbq_moe_select_backward(r, d_weights.data_ptr(), logits.data_ptr(), dt, ids.data_ptr(), M, d.data_ptr(), s)
        if st:
            raise LbqError(st, "lbq_moe_select_backward")
        return d
    return _on(gpu, stream, go, d_weights, logits, ids, d_logits)


# ------------------------------------------------------------------ low-rank adapters

class Adapters:
    """L low-rank adapters (see lbq_adapters in include/lbq.h): a [L][r][K] and b [L][N][r], both float16 or both
    bfloat16, scales float32 [L].

    It keeps the tensors and their addresses: what they hold may change, the tensors may not be replaced."""

    __slots__ = ("L", "K", "N", "r", "dtype", "gpu", "_tensors", "struct", "ref")

    def __init__(self, a, b, scales):
        _ready()
        where = "Adapters"
        if a.dim() != 3 or b.dim() != 3:
            raise LbqError(-2, f"{where}: a is [L][r][K] and b is [L][N][r]")
        dt = _dtype(a.dtype, where)
        L, r, K = a.shape
        N = b.shape[1]
        gpu = a.get_device()
        if max(L, r, K, N) > _MOST:
            raise LbqError(-2, f"{where}: {tuple(a.shape)}, {tuple(b.shape)}")
        _need(where, gpu, a.dtype, None, a)
        _need(where, gpu, a.dtype, (L, N, r), b)
        _need(where, gpu, _torch.float32, (L,), scales)
        self.L, self.K, self.N, self.r, self.dtype, self.gpu = L, K, N, r, a.dtype, gpu
        self._tensors = (a, b, scales)
        self.struct = AdaptersView(L, K, N, r, dt, a.data_ptr(), b.data_ptr(), scales.data_ptr())
        self.ref = ctypes.byref(self.struct)

    @property
    def a(self):
        return self._tensors[0]

    @property
    def b(self):
        return self._tensors[1]

    @property
    def scales(self):
        return self._tensors[2]

    def workspace_bytes(self, M: int, sorted: bool = False, backward: bool = False) -> int:
        name = "lbq_adapters_backward_workspace" if backward else "lbq_adapters_workspace"
        return _adapters_query(name, self.L, self.K, self.N, self.r, self.struct.dtype, int(M), bool(sorted))


@functools.lru_cache(maxsize=4096)
def _adapters_query(name, L, K, N, r, dtype, M, ordered) -> int:
    if not -_MOST <= M <= _MOST:
        raise LbqError(-2, f"{name}: {M}")
    need = ctypes.c_size_t()
    p = ctypes.c_void_p(16)   # aligned stand-in: queries look at sizes only
    _check(getattr(lib(), name)(ctypes.byref(AdaptersView(L, K, N, r, dtype, p, p, p)), M, ordered, ctypes.byref(need)), name)
    return need.value


def _tokens(where: str, ad: Adapters, rows, cols: int, ids, order):
    """(M, pointers of the order) after the checks that both directions share."""
    if rows.dim() != 2 or rows.shape[1] != cols:
        raise LbqError(-2, f"{where}: rows of {cols} are needed, got {tuple(rows.shape)}")
    _need(where, ad.gpu, ad.dtype, None, rows)
    M = rows.shape[0]
    _need(where, ad.gpu, _torch.int32, (M,), ids)
    if order is None:
        return M, None, None
    offsets, perm = order
    _need(where, ad.gpu, _torch.int32, (ad.L + 1,), offsets)
    _need(where, ad.gpu, _torch.int32, (M,), perm)
    return M, offsets.data_ptr(), perm.data_ptr()


def adapters_forward(ad: Adapters, x, ids, base=None, y=None, h=None, order=None, ws=None, stream=None):
    """lbq_adapters_forward: y [M][N] = base + scales[ids] (x A^T) B^T, a token with an id outside [0, L) without the
    second part. y may be base. h: float32 [M][r], written for adapters_backward. order: (offsets, perm) of
    moe_sort(ids[:, None], L), where the program keeps it. Autograd does not see it."""
    L = _ready()
    where = "adapters_forward"
    M, po, pp = _tokens(where, ad, x, ad.K, ids, order)
    if base is not None:
        _need(where, ad.gpu, ad.dtype, (M, ad.N), base)
    if y is not None:
        _need(where, ad.gpu, ad.dtype, (M, ad.N), y)
    if h is not None:
        _need(where, ad.gpu, _torch.float32, (M, ad.r), h)
    need = _adapters_query("lbq_adapters_workspace", ad.L, ad.K, ad.N, ad.r, ad.struct.dtype, M, order is not None)

    def go(s):
        out = x.new_empty((M, ad.N)) if y is None else y
        p, size, keep = _workspace(ws, need, x, ad.gpu, where)
        st = L.lbq_adapters_forward(ad.ref, x.data_ptr(), M, ids.data_ptr(), po, pp,
                                    None if base is None else base.data_ptr(), out.data_ptr(),
                                    None if h is None else h.data_ptr(), p, size, s)
        if st:
            raise LbqError(st, "lbq_adapters_forward")
        return out
    return _on(ad.gpu, stream, go, *ad._tensors, x, ids, base, y, h, ws, *(order or ()))


def adapters_backward(ad: Adapters, dy, x, h, ids, base=None, dx=None, d_a=None, d_b=None, order=None, ws=None,
                      stream=None):
    """lbq_adapters_backward: (dx [M][K], d_a float32 [L][r][K], d_b float32 [L][N][r]) from dy, x and the h that
    adapters_forward wrote. base: the shared projection's own dx, added to dx; dx may be base."""
    L = _ready()
    where = "adapters_backward"
    M, po, pp = _tokens(where, ad, x, ad.K, ids, order)
    _need(where, ad.gpu, ad.dtype, (M, ad.N), dy)
    _need(where, ad.gpu, _torch.float32, (M, ad.r), h)
    for t in (base, dx):
        if t is not None:
            _need(where, ad.gpu, ad.dtype, (M, ad.K), t)
    if d_a is not None:
        _need(where, ad.gpu, _torch.float32, (ad.L, ad.r, ad.K), d_a)
    if d_b is not None:
        _need(where, ad.gpu, _torch.float32, (ad.L, ad.N, ad.r), d_b)
    need = _adapters_query("lbq_adapters_backward_workspace", ad.L, ad.K, ad.N, ad.r, ad.struct.dtype, M,
                           order is not None)

    def go(s):
        ox = x.new_empty((M, ad.K)) if dx is None else dx
        oa = h.new_empty((ad.L, ad.r, ad.K)) if d_a is None else d_a
        ob = h.new_empty((ad.L, ad.N, ad.r)) if d_b is None else d_b
        p, size, keep = _workspace(ws, need, x, ad.gpu, where)
        st = L.lbq_adapters_backward(ad.ref, dy.data_ptr(), x.data_ptr(), h.data_ptr(), M, ids.data_ptr(), po, pp,
                                     None if base is None else base.data_ptr(), ox.data_ptr(), oa.data_ptr(),
                                     ob.data_ptr(), p, size, s)
        if st:
            raise LbqError(st, "lbq_adapters_backward")
        return ox, oa, ob
    return _on(ad.gpu, stream, go, *ad._tensors, dy, x, h, ids, base, dx, d_a, d_b, ws, *(order or ()))
