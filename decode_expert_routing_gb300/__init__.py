"""GB300-native MoE decode routing: router GEMV, top-k gate, sort, MXFP8 quant,
the experts' products, and the norm, rows and FP8 products around them.

Thin Python binding over the C ABI of libmoe_route.so (include/moe_route.h):
the functions below have the ABI's names without the ``mr_`` prefix, check
dtypes/devices/contiguity, allocate outputs with torch when none are given,
and pass raw pointers plus torch's current CUDA stream.  Every step of the
path runs in the library's CUDA kernels; there is no other implementation
behind these calls.  If the library is missing or fails to load, every call
raises.

bf16 tensors are torch.bfloat16; MXFP8 codes and E8M0 scales are uint8.
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "MoeRouteError", "MoeRouteUnsupported", "Scratch", "library_path", "load_library",
    "set_launch_flags", "get_launch_flags", "LAUNCH_PDL", "LAUNCH_TEST_STALL", "LAUNCH_LEGACY_MMA",
    "LAUNCH_TEST_SLOW_SIGMOID", "LAUNCH_CHECK_SCRATCH", "set_wait_limit_ns",
    "device_error", "router_gemv_supported", "scratch_bytes", "sort_capacity", "router_gemv", "route_topk",
    "moe_sort", "mxfp8_quant", "moe_route_sort_quant", "router_gemv_noalloc", "shared_gate_up", "moe_route",
    "PreparedRoute", "moe_sort_quant", "mxfp4_quant", "norm_apply", "moe_route_sort_quant_norm",
    "MxWeight", "ExpertScratch", "mx_gemm", "moe_gate_up", "moe_down", "PreparedMxGemm", "PreparedGateUp",
    "PreparedDown",
    "add_rms_norm", "PreparedAddNorm", "fp8_quant", "fp8_gemm", "PreparedFp8Gemm", "moe_permute", "PreparedPermute",
    "moe_permute_grad", "PreparedPermuteGrad", "moe_combine", "PreparedCombine", "moe_combine_grad",
    "PreparedCombineGrad",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libmoe_route.so")
_lib = None

(MR_OK, MR_ERR_UNSUPPORTED, MR_ERR_INVALID_ARG, MR_ERR_SCRATCH_TOO_SMALL, MR_ERR_CUDA, MR_ERR_TIMEOUT,
 MR_ERR_SCRATCH_DIRTY) = range(7)
SCORING = {"softmax": 0, "sigmoid": 1}
NORM_KIND = {"rms": 0, "gemma": 1}
QUANT_FORMAT = {None: 0, "mxfp8": 1, "mxfp4": 2}
SCRATCH_COUNTER_BYTES = 32768
PSORT_MAX_ASSIGN = 65536   # mr_moe_sort: one launch, no scratch, up to this many assignments
QUANT_SORTED_ROWS = 0x100  # mr_moe_sort_quant: quantised rows in sorted order


class MoeRouteError(RuntimeError):
    """The library rejected the call or CUDA reported an error."""

    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {_load().mr_status_string(status).decode()}"
        if status == MR_ERR_CUDA:
            msg += f" (cudaError_t {_load().mr_last_cuda_error()})"
        super().__init__(msg)


class MoeRouteUnsupported(MoeRouteError):
    """The shape is outside what the kernels cover (MR_ERR_UNSUPPORTED)."""


def library_path() -> str:
    return _LIB_PATH


# (name, restype, argtypes) of every exported symbol; the ABI test checks this
# list against include/moe_route.h.
_P, _I, _I64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "mr_status_string": (ctypes.c_char_p, [_I]),
    "mr_abi_version": (_I, []),
    "mr_set_launch_flags": (_I, [_I]),
    "mr_get_launch_flags": (_I, []),
    "mr_router_gemv_supported": (_I, [_I, _I, _I, _I64]),
    "mr_scratch_bytes": (_SZ, [_I, _I, _I, _I]),
    "mr_scratch_reset": (_I, [_P, _SZ, _P]),
    "mr_router_gemv": (_I, [_P, _I64, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "mr_route_topk": (_I, [_P, _I, _I, _I, _I, _P, _I, _P, _P, _P]),
    "mr_sort_capacity": (_I64, [_I, _I, _I, _I]),
    "mr_moe_sort": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _I64, _P, _SZ, _P]),
    "mr_mxfp8_quant": (_I, [_P, _I64, _I, _I, _P, _P, _P]),
    "mr_moe_route_sort_quant": (_I, [_P, _I64, _P, _I, _I, _I, _I, _I, _P, _I, _I, _P, _P, _P,
                                     _P, _P, _P, _I64, _P, _P, _P, _SZ, _P]),
    "mr_router_gemv_noalloc": (_I, [_P, _I64, _P, _P, _I, _I, _I, _P]),
    "mr_moe_route_sort_quant_norm": (_I, [_P, _I64, _P, _P, _I, _P, _I, _I, _I, _I, _I, _P, _I, _I, _P, _P, _P,
                                          _P, _P, _P, _I64, _P, _P, _P, _SZ, _P]),
    "mr_norm_apply": (_I, [_P, _I64, _P, _P, _I, _I, _I, _P, _P]),
    "mr_mxfp4_quant": (_I, [_P, _I64, _I, _I, _P, _P, _P]),
    "mr_moe_route": (_I, [_P, _P]),
    "mr_moe_sort_quant": (_I, [_P, _I, _I, _I, _I, _P, _I64, _I, _I, _P, _P, _P, _I64, _P, _P, _P]),
    "mr_set_wait_limit_ns": (_I, [ctypes.c_uint64]),
    "mr_device_error": (_I, [_I]),
    "mr_shared_gate_up": (_I, [_P, _I64, _P, _P, _I, _I, _I, _P, _P]),
    "mr_last_cuda_error": (_I, []),
    "mr_mx_packed_scale_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "mr_mx_pack_scales": (_I, [_P, _I, _I, _I, _I, _I, _P, _P]),
    "mr_expert_scratch_bytes": (_SZ, [_I, _I, _I]),
    "mr_mx_gemm": (_I, [_P, _P]),
    "mr_moe_gate_up": (_I, [_P, _P]),
    "mr_moe_down": (_I, [_P, _P]),
    "mr_add_rms_norm": (_I, [_P, _P]),
    "mr_fp8_quant": (_I, [_P, _I64, _I, _I, _P, _P, _P]),
    "mr_fp8_gemm": (_I, [_P, _P]),
    "mr_moe_permute": (_I, [_P, _P]),
    "mr_moe_combine": (_I, [_P, _P]),
    "mr_moe_combine_grad": (_I, [_P, _P]),
}


def load_library(path: str | None = None):
    """Load libmoe_route.so (built by decode_expert_routing_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"libmoe_route.so not found at {p}: build it with "
            "`python -m decode_expert_routing_gb300.build` (nvcc, sm_103a)")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


_load = load_library


def _check(status: int, what: str):
    if status == MR_OK:
        return
    if status == MR_ERR_UNSUPPORTED:
        raise MoeRouteUnsupported(status, what)
    raise MoeRouteError(status, what)


# ---------------------------------------------------------------- helpers

def _torch():
    import torch
    return torch


def _stream_ptr(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev_ptr(t, name, dtype=None, allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _row_major_2d(x, name):
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with a contiguous last dimension")
    return x.stride(0)


def _one_device(**tensors):
    """The one CUDA device of every given tensor (None entries skipped)."""
    devs = {}
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        devs.setdefault(t.device, name)
    if len(devs) != 1:
        raise ValueError("tensors on different devices: " + ", ".join(f"{n} on {d}" for d, n in devs.items()))
    return next(iter(devs))


def _check_out(t, name, shape, dtype, device, min_numel=False):
    """A caller-passed output: contiguous, of this dtype and shape (or at
    least this many elements when min_numel), on this device."""
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if min_numel:
        if t.numel() < shape:
            raise ValueError(f"{name} needs at least {shape} elements, has {t.numel()}")
    elif tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_scratch(scratch, device):
    if scratch is not None and scratch.tensor.device != device:
        raise ValueError(f"scratch must be on {device}")


def _launch_ctx(device):
    """The calling thread's current device set to device for the C call (the
    library launches on the current device, on the given stream)."""
    return _torch().cuda.device(device)


def _stream_on(device, stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


LAUNCH_PDL = 1
LAUNCH_TEST_STALL = 2  # test hook: the cluster kernels' bounded waits run out
LAUNCH_LEGACY_MMA = 4  # router GEMV of more than 64 rows: split-K mma.sync kernel instead of tcgen05
LAUNCH_TEST_SLOW_SIGMOID = 8  # test hook: every exact sigmoid score through its double-double path
LAUNCH_CHECK_SCRATCH = 16  # debug: calls that use scratch counters verify they are zero first (synchronous)


def set_launch_flags(flags: int) -> None:
    """Process-wide launch options (LAUNCH_PDL: programmatic dependent launch)."""
    _check(_load().mr_set_launch_flags(int(flags)), "mr_set_launch_flags")


def get_launch_flags() -> int:
    return int(_load().mr_get_launch_flags())


def set_wait_limit_ns(ns: int) -> None:
    """Limit of every bounded wait inside the cluster kernels (default 1 s)."""
    _check(_load().mr_set_wait_limit_ns(int(ns)), "mr_set_wait_limit_ns")


def device_error(clear: bool = False) -> int:
    """MR_OK, or MR_ERR_TIMEOUT once a bounded wait ran out on the current
    device (synchronous; call after the streams have finished)."""
    st = int(_load().mr_device_error(int(clear)))
    if st not in (MR_OK, MR_ERR_TIMEOUT):
        _check(st, "mr_device_error")
    return st


def router_gemv_supported(M: int, N: int, K: int, ldx: int | None = None) -> bool:
    return bool(_load().mr_router_gemv_supported(M, N, K, K if ldx is None else ldx))


def scratch_bytes(M_max: int, N: int, K: int, topk: int) -> int:
    return int(_load().mr_scratch_bytes(M_max, N, K, topk))


def sort_capacity(M: int, topk: int, N: int, block: int) -> int:
    return int(_load().mr_sort_capacity(M, topk, N, block))


class Scratch:
    """A caller-owned scratch buffer (torch uint8 on a CUDA device), zeroed
    once at creation; every call of the library leaves it reusable."""

    def __init__(self, M_max: int, N: int, K: int, topk: int, device=None):
        torch = _torch()
        self.nbytes = scratch_bytes(M_max, N, K, topk)
        if self.nbytes == 0:
            raise ValueError("scratch size query rejected the arguments")
        self.tensor = torch.empty(self.nbytes, dtype=torch.uint8,
                                  device=device if device is not None else "cuda")
        self.reset()

    def reset(self, stream=None):
        _check(_load().mr_scratch_reset(ctypes.c_void_p(self.tensor.data_ptr()), self.nbytes,
                                        _stream_ptr(stream)), "mr_scratch_reset")

    @property
    def ptr(self):
        return ctypes.c_void_p(self.tensor.data_ptr())

    def counters(self):
        """The counter prefix as int32 (all zero between calls)."""
        return self.tensor[:SCRATCH_COUNTER_BYTES].view(_torch().int32)


# ---------------------------------------------------------------- the path

def router_gemv(x, w, out=None, scratch: Scratch | None = None, stream=None):
    """fp32 logits [M, N] = x [M, K] (bf16) @ w [N, K]^T (bf16)."""
    torch = _torch()
    dev = _one_device(x=x, w=w, out=out)
    ldx = _row_major_2d(x, "x")
    M, K = x.shape
    N = w.shape[0]
    if w.dim() != 2 or not w.is_contiguous() or w.shape[1] != K:
        raise ValueError("w must be contiguous [N, K]")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    _check_out(out, "out", (M, N), torch.float32, dev)
    if scratch is None:
        scratch = Scratch(M, N, K, 1, device=dev)
    _check_scratch(scratch, dev)
    with _launch_ctx(dev):
        _check(_load().mr_router_gemv(_dev_ptr(x, "x", torch.bfloat16), ldx, _dev_ptr(w, "w", torch.bfloat16),
                                      _dev_ptr(out, "out", torch.float32), M, N, K, scratch.ptr,
                                      scratch.nbytes, _stream_on(dev, stream)), "mr_router_gemv")
    return out


def router_gemv_noalloc(x, w, out=None, stream=None):
    """Router GEMV using the library's own fixed-size device scratch (no
    scratch argument, nothing allocated by the library).  For callers that
    cannot allocate; calls on one device share that scratch, so overlapping
    calls race.  The first call per device does a one-time set-up."""
    torch = _torch()
    dev = _one_device(x=x, w=w, out=out)
    ldx = _row_major_2d(x, "x")
    M, K = x.shape
    N = w.shape[0]
    if w.dim() != 2 or not w.is_contiguous() or w.shape[1] != K:
        raise ValueError("w must be contiguous [N, K]")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    _check_out(out, "out", (M, N), torch.float32, dev)
    with _launch_ctx(dev):
        _check(_load().mr_router_gemv_noalloc(_dev_ptr(x, "x", torch.bfloat16), ldx,
                                              _dev_ptr(w, "w", torch.bfloat16),
                                              _dev_ptr(out, "out", torch.float32), M, N, K,
                                              _stream_on(dev, stream)), "mr_router_gemv_noalloc")
    return out


def route_topk(logits, topk: int, scoring: str = "softmax", bias=None, renormalize: bool = True,
               ids=None, weights=None, stream=None):
    """(topk_ids int32 [M, k], topk_weights fp32 [M, k])."""
    torch = _torch()
    dev = _one_device(logits=logits, bias=bias, ids=ids, weights=weights)
    if logits.dim() != 2 or not logits.is_contiguous():
        raise ValueError("logits must be contiguous [M, N]")
    M, N = logits.shape
    if bias is not None:
        _check_out(bias, "bias", (N,), torch.float32, dev)
    if ids is None:
        ids = torch.empty((M, topk), dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty((M, topk), dtype=torch.float32, device=dev)
    _check_out(ids, "ids", (M, topk), torch.int32, dev)
    _check_out(weights, "weights", (M, topk), torch.float32, dev)
    with _launch_ctx(dev):
        _check(_load().mr_route_topk(_dev_ptr(logits, "logits", torch.float32), M, N, topk, SCORING[scoring],
                                     _dev_ptr(bias, "bias", torch.float32, allow_none=True), int(renormalize),
                                     _dev_ptr(ids, "ids", torch.int32), _dev_ptr(weights, "weights", torch.float32),
                                     _stream_on(dev, stream)), "mr_route_topk")
    return ids, weights


def moe_sort(topk_ids, num_experts: int, block: int, out=None, scratch: Scratch | None = None,
             stream=None):
    """(sorted_token_ids [cap], expert_ids [cap/block], num_tokens_post_padded [1]) int32."""
    torch = _torch()
    st0, ex0, nt0 = out if out is not None else (None, None, None)
    dev = _one_device(topk_ids=topk_ids, sorted_token_ids=st0, expert_ids=ex0, num_tokens_post_padded=nt0)
    if topk_ids.dim() != 2 or not topk_ids.is_contiguous():
        raise ValueError("topk_ids must be contiguous [M, k]")
    M, k = topk_ids.shape
    cap = sort_capacity(M, k, num_experts, block)
    if cap < 0:
        raise MoeRouteUnsupported(MR_ERR_UNSUPPORTED, "mr_sort_capacity")
    if out is None:
        out = (torch.empty(cap, dtype=torch.int32, device=dev),
               torch.empty(cap // block, dtype=torch.int32, device=dev),
               torch.empty(1, dtype=torch.int32, device=dev))
    st, ex, nt = out
    _check_sort_out(st, ex, nt, cap, block, dev)
    _check_scratch(scratch, dev)
    sp, sb = (scratch.ptr, scratch.nbytes) if scratch is not None else (None, 0)
    if scratch is None and M * k > PSORT_MAX_ASSIGN:
        scratch = Scratch(M, num_experts, 512, k, device=dev)
        sp, sb = scratch.ptr, scratch.nbytes
    with _launch_ctx(dev):
        _check(_load().mr_moe_sort(_dev_ptr(topk_ids, "topk_ids", torch.int32), M, k, num_experts, block,
                                   _dev_ptr(st, "sorted_token_ids", torch.int32),
                                   _dev_ptr(ex, "expert_ids", torch.int32),
                                   _dev_ptr(nt, "num_tokens_post_padded", torch.int32), st.numel(), sp, sb,
                                   _stream_on(dev, stream)), "mr_moe_sort")
    return st, ex, nt


def _check_sort_out(st, ex, nt, cap, block, dev):
    """The sort's outputs: st holds at least the capacity (its length is the
    capacity passed on), ex one entry per block of it, nt one entry."""
    torch = _torch()
    _check_out(st, "sorted_token_ids", cap, torch.int32, dev, min_numel=True)
    _check_out(ex, "expert_ids", st.numel() // block, torch.int32, dev, min_numel=True)
    _check_out(nt, "num_tokens_post_padded", 1, torch.int32, dev, min_numel=True)


def mxfp8_quant(x, out=None, stream=None):
    """(q uint8 [M, K] e4m3 codes, scale uint8 [M, K/32] e8m0)."""
    return _mx_quant(x, out, stream, fp4=False)


def _mx_quant(x, out, stream, fp4):
    torch = _torch()
    dev = _one_device(x=x, **({} if out is None else dict(q=out[0], scale=out[1])))
    ldx = _row_major_2d(x, "x")
    M, K = x.shape
    qk = K // 2 if fp4 else K
    if out is None:
        out = (torch.empty((M, qk), dtype=torch.uint8, device=dev),
               torch.empty((M, K // 32), dtype=torch.uint8, device=dev))
    q, s = out
    _check_out(q, "q", (M, qk), torch.uint8, dev)
    _check_out(s, "scale", (M, K // 32), torch.uint8, dev)
    fn, name = (_load().mr_mxfp4_quant, "mr_mxfp4_quant") if fp4 else (_load().mr_mxfp8_quant, "mr_mxfp8_quant")
    with _launch_ctx(dev):
        _check(fn(_dev_ptr(x, "x", torch.bfloat16), ldx, M, K, _dev_ptr(q, "q", torch.uint8),
                  _dev_ptr(s, "scale", torch.uint8), _stream_on(dev, stream)), name)
    return q, s


def route_output_layout(M: int, N: int, K: int, topk: int, block: int, quant=True):
    """[(name, dtype, shape, byte offset)] of the one-launch route's outputs
    packed into one buffer (each 16-byte aligned), and the buffer's bytes."""
    torch = _torch()
    cap = sort_capacity(M, topk, N, block)
    items = [("logits", torch.float32, (M, N)), ("topk_ids", torch.int32, (M, topk)),
             ("topk_weights", torch.float32, (M, topk)), ("sorted_token_ids", torch.int32, (cap,)),
             ("expert_ids", torch.int32, (cap // block,)), ("num_tokens_post_padded", torch.int32, (1,))]
    if quant:
        items += [("q", torch.uint8, (M, K // 2 if quant == "mxfp4" else K)), ("scale", torch.uint8, (M, K // 32))]
    layout, off = [], 0
    for name, dt, shape in items:
        n = 1
        for d in shape:
            n *= d
        layout.append((name, dt, shape, off))
        off += (n * torch.tensor([], dtype=dt).element_size() + 15) // 16 * 16
    return layout, off


def route_outputs_in(buf, M: int, N: int, K: int, topk: int, block: int, quant=True, offset: int = 0):
    """Views of the route's outputs inside the uint8 buffer buf, from byte
    offset (16-byte aligned) on: one copy of buf moves every output."""
    layout, nbytes = route_output_layout(M, N, K, topk, block, quant)
    if offset % 16 or buf.dtype != _torch().uint8 or buf.numel() < offset + nbytes:
        raise ValueError("buf must be uint8 with room for the outputs at a 16-byte aligned offset")
    out = {}
    for name, dt, shape, off in layout:
        n = 1
        for d in shape:
            n *= d
        esz = _torch().tensor([], dtype=dt).element_size()
        out[name] = buf[offset + off: offset + off + n * esz].view(dt).view(shape)
    return out


def mxfp4_quant(x, out=None, stream=None):
    """(q uint8 [M, K/2] packed e2m1 codes, element 2j in the low nibble;
    scale uint8 [M, K/32] e8m0)."""
    return _mx_quant(x, out, stream, fp4=True)


def alloc_route_outputs(M: int, N: int, K: int, topk: int, block: int, device, quant=True):
    """Output tensors of the one-launch route (a dict).  quant: True or
    "mxfp8" (q [M, K]), "mxfp4" (q [M, K/2]), False or None (no q / scale)."""
    torch = _torch()
    cap = sort_capacity(M, topk, N, block)
    out = dict(
        logits=torch.empty((M, N), dtype=torch.float32, device=device),
        topk_ids=torch.empty((M, topk), dtype=torch.int32, device=device),
        topk_weights=torch.empty((M, topk), dtype=torch.float32, device=device),
        sorted_token_ids=torch.empty(cap, dtype=torch.int32, device=device),
        expert_ids=torch.empty(cap // block, dtype=torch.int32, device=device),
        num_tokens_post_padded=torch.empty(1, dtype=torch.int32, device=device),
    )
    if quant:
        out["q"] = torch.empty((M, K // 2 if quant == "mxfp4" else K), dtype=torch.uint8, device=device)
        out["scale"] = torch.empty((M, K // 32), dtype=torch.uint8, device=device)
    return out


def _check_route_out(out, M, N, K, topk, block, quant, dev):
    """Every output of the one-launch route: dtype, shape (the sort's at
    least the capacity), contiguity and device."""
    torch = _torch()
    cap = sort_capacity(M, topk, N, block)
    if cap < 0:
        raise MoeRouteUnsupported(MR_ERR_UNSUPPORTED, "mr_sort_capacity")
    _check_out(out["logits"], "logits", (M, N), torch.float32, dev)
    _check_out(out["topk_ids"], "topk_ids", (M, topk), torch.int32, dev)
    _check_out(out["topk_weights"], "topk_weights", (M, topk), torch.float32, dev)
    _check_sort_out(out["sorted_token_ids"], out["expert_ids"], out["num_tokens_post_padded"], cap, block, dev)
    if quant:
        _check_out(out["q"], "q", (M, K // 2 if quant == "mxfp4" else K), torch.uint8, dev)
        _check_out(out["scale"], "scale", (M, K // 32), torch.uint8, dev)


def _check_w(w, K):
    if w.dim() != 2 or not w.is_contiguous() or w.shape[1] != K:
        raise ValueError("w must be contiguous [N, K]")


def _check_bias(bias, N, dev):
    if bias is not None:
        _check_out(bias, "bias", (N,), _torch().float32, dev)


def moe_route_sort_quant(x, w, topk: int, block: int, scoring: str = "softmax", bias=None,
                         renormalize: bool = True, quant: bool = True, out=None,
                         scratch: Scratch | None = None, stream=None):
    """The whole path for M <= 64 tokens in one launch; returns a dict of outputs."""
    torch = _torch()
    dev = _one_device(x=x, w=w, bias=bias)
    ldx = _row_major_2d(x, "x")
    M, K = x.shape
    N = w.shape[0]
    _check_w(w, K)
    _check_bias(bias, N, dev)
    if out is None:
        out = alloc_route_outputs(M, N, K, topk, block, dev, quant)
    _check_route_out(out, M, N, K, topk, block, quant, dev)
    if scratch is None:
        scratch = Scratch(M, N, K, topk, device=dev)
    _check_scratch(scratch, dev)
    q = out.get("q") if quant else None
    s = out.get("scale") if quant else None
    with _launch_ctx(dev):
        st = _load().mr_moe_route_sort_quant(
        _dev_ptr(x, "x", torch.bfloat16), ldx, _dev_ptr(w, "w", torch.bfloat16), M, N, K, topk,
        SCORING[scoring], _dev_ptr(bias, "bias", torch.float32, allow_none=True), int(renormalize), block,
        _dev_ptr(out["logits"], "logits", torch.float32), _dev_ptr(out["topk_ids"], "topk_ids", torch.int32),
        _dev_ptr(out["topk_weights"], "topk_weights", torch.float32),
        _dev_ptr(out["sorted_token_ids"], "sorted_token_ids", torch.int32),
        _dev_ptr(out["expert_ids"], "expert_ids", torch.int32),
        _dev_ptr(out["num_tokens_post_padded"], "num_tokens_post_padded", torch.int32),
        out["sorted_token_ids"].numel(), _dev_ptr(q, "q", torch.uint8, allow_none=True),
        _dev_ptr(s, "scale", torch.uint8, allow_none=True), scratch.ptr, scratch.nbytes,
        _stream_on(dev, stream))
    _check(st, "mr_moe_route_sort_quant")
    return out


def norm_apply(sres, rstd, norm_weight, norm: str = "gemma", out=None, stream=None):
    """The router input on the norm's scale, written out: bf16 [M, K] with
    xn[m, k] = bf16((sres[m, k] * rstd[m]) * s[k]), s = g or 1 + g."""
    torch = _torch()
    dev = _one_device(sres=sres, rstd=rstd, norm_weight=norm_weight, out=out)
    ldx = _row_major_2d(sres, "sres")
    M, K = sres.shape
    _check_norm_args(rstd, norm_weight, M, K)
    if out is None:
        out = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    _check_out(out, "out", (M, K), torch.bfloat16, dev)
    with _launch_ctx(dev):
        _check(_load().mr_norm_apply(_dev_ptr(sres, "sres", torch.bfloat16), ldx,
                                     _dev_ptr(rstd, "rstd", torch.float32),
                                     _dev_ptr(norm_weight, "norm_weight", torch.bfloat16), NORM_KIND[norm], M, K,
                                     _dev_ptr(out, "out", torch.bfloat16), _stream_on(dev, stream)),
               "mr_norm_apply")
    return out


def _check_norm_args(rstd, norm_weight, M, K):
    if rstd.dim() != 1 or rstd.shape[0] != M or not rstd.is_contiguous():
        raise ValueError("rstd must be contiguous [M]")
    if norm_weight.dim() != 1 or norm_weight.shape[0] != K or not norm_weight.is_contiguous():
        raise ValueError("norm_weight must be contiguous [K]")


def moe_route_sort_quant_norm(sres, rstd, norm_weight, w, topk: int, block: int, norm: str = "gemma",
                              scoring: str = "softmax", bias=None, renormalize: bool = True, quant: bool = True,
                              out=None, scratch: Scratch | None = None, stream=None):
    """The one-launch route with its input on the norm's scale (residual rows,
    per-token rstd, norm weight); returns a dict of outputs."""
    torch = _torch()
    dev = _one_device(sres=sres, rstd=rstd, norm_weight=norm_weight, w=w, bias=bias)
    ldx = _row_major_2d(sres, "sres")
    M, K = sres.shape
    N = w.shape[0]
    _check_w(w, K)
    _check_bias(bias, N, dev)
    _check_norm_args(rstd, norm_weight, M, K)
    if out is None:
        out = alloc_route_outputs(M, N, K, topk, block, dev, quant)
    _check_route_out(out, M, N, K, topk, block, quant, dev)
    if scratch is None:
        scratch = Scratch(M, N, K, topk, device=dev)
    _check_scratch(scratch, dev)
    q = out.get("q") if quant else None
    s = out.get("scale") if quant else None
    with _launch_ctx(dev):
        st = _load().mr_moe_route_sort_quant_norm(
        _dev_ptr(sres, "sres", torch.bfloat16), ldx, _dev_ptr(rstd, "rstd", torch.float32),
        _dev_ptr(norm_weight, "norm_weight", torch.bfloat16), NORM_KIND[norm],
        _dev_ptr(w, "w", torch.bfloat16), M, N, K, topk,
        SCORING[scoring], _dev_ptr(bias, "bias", torch.float32, allow_none=True), int(renormalize), block,
        _dev_ptr(out["logits"], "logits", torch.float32), _dev_ptr(out["topk_ids"], "topk_ids", torch.int32),
        _dev_ptr(out["topk_weights"], "topk_weights", torch.float32),
        _dev_ptr(out["sorted_token_ids"], "sorted_token_ids", torch.int32),
        _dev_ptr(out["expert_ids"], "expert_ids", torch.int32),
        _dev_ptr(out["num_tokens_post_padded"], "num_tokens_post_padded", torch.int32),
        out["sorted_token_ids"].numel(), _dev_ptr(q, "q", torch.uint8, allow_none=True),
        _dev_ptr(s, "scale", torch.uint8, allow_none=True), scratch.ptr, scratch.nbytes,
        _stream_on(dev, stream))
    _check(st, "mr_moe_route_sort_quant_norm")
    return out


class RouteParams(ctypes.Structure):
    """mr_route_params of moe_route.h, field for field."""
    _fields_ = [
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("rstd", ctypes.c_void_p),
        ("norm_weight", ctypes.c_void_p), ("norm_kind", ctypes.c_int), ("w", ctypes.c_void_p),
        ("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int), ("topk", ctypes.c_int),
        ("scoring", ctypes.c_int), ("sel_bias", ctypes.c_void_p), ("renormalize", ctypes.c_int),
        ("block", ctypes.c_int), ("quant_format", ctypes.c_int), ("logits", ctypes.c_void_p),
        ("topk_ids", ctypes.c_void_p), ("topk_weights", ctypes.c_void_p), ("sorted_token_ids", ctypes.c_void_p),
        ("expert_ids", ctypes.c_void_p), ("num_tokens_post_padded", ctypes.c_void_p), ("capacity", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("scratch", ctypes.c_void_p),
        ("scratch_bytes", ctypes.c_size_t), ("shared_w13", ctypes.c_void_p), ("shared_w13_scale", ctypes.c_void_p),
        ("shared_inter", ctypes.c_int), ("shared_act", ctypes.c_void_p),
    ]


def moe_route(x, w, topk: int, block: int, scoring: str = "softmax", bias=None, renormalize: bool = True,
              quant="mxfp8", rstd=None, norm_weight=None, norm: str = "gemma", out=None,
              scratch: Scratch | None = None, stream=None, shared=None):
    """The one-launch route with every option (mr_moe_route): quant "mxfp8",
    "mxfp4" or None; with rstd (and norm_weight) x holds the residual rows
    and the route runs on the norm's scale; shared = (w13 E4M3 codes [2I, K],
    scale bytes [2I, K/32]) adds the shared expert's gate/up + SwiGLU to the
    launch (out["shared_act"], bf16 [M, I]).  Returns a dict of outputs."""
    call = PreparedRoute(x, w, topk, block, scoring, bias, renormalize, quant, rstd, norm_weight, norm, out, scratch,
                         shared)
    call(stream)
    return call.out


def _check_shared(shared, M, K, dev):
    """(w13, w13_scale) of the shared expert: uint8 [2I, K] and [2I, K/32]; returns I."""
    torch = _torch()
    w13, sc = shared
    if w13.dim() != 2 or w13.shape[1] != K or w13.shape[0] % 2:
        raise ValueError("w13 must be [2I, K]")
    R = w13.shape[0]
    _check_out(w13, "w13", (R, K), torch.uint8, dev)
    _check_out(sc, "w13_scale", (R, K // 32), torch.uint8, dev)
    return R // 2


def shared_gate_up(x, w13, w13_scale, out=None, stream=None):
    """The shared expert's gate/up projection and SwiGLU (mr_shared_gate_up):
    bf16 [M, I] = silu(x . gate^T) * (x . up^T) with MXFP8 w13 (E4M3 codes
    [2I, K], gate rows first, E8M0 scales [2I, K/32]); M <= 16."""
    torch = _torch()
    dev = _one_device(x=x, w13=w13, w13_scale=w13_scale, out=out)
    ldx = _row_major_2d(x, "x")
    M, K = x.shape
    I = _check_shared((w13, w13_scale), M, K, dev)
    if out is None:
        out = torch.empty((M, I), dtype=torch.bfloat16, device=dev)
    _check_out(out, "out", (M, I), torch.bfloat16, dev)
    with _launch_ctx(dev):
        _check(_load().mr_shared_gate_up(_dev_ptr(x, "x", torch.bfloat16), ldx, _dev_ptr(w13, "w13", torch.uint8),
                                         _dev_ptr(w13_scale, "w13_scale", torch.uint8), M, K, I,
                                         _dev_ptr(out, "out", torch.bfloat16), _stream_on(dev, stream)),
               "mr_shared_gate_up")
    return out


def _torch_stream(device, raw: int):
    """The torch stream of a raw cudaStream_t (0 and 1: the default stream,
    which ExternalStream does not take)."""
    torch = _torch()
    return torch.cuda.default_stream(device) if raw in (0, 1) else torch.cuda.ExternalStream(raw, device=device)


def _given_stream(device, stream):
    """A torch stream of a call's stream argument (a torch stream or a raw
    cudaStream_t of that device), or None."""
    if stream is None:
        return None
    if isinstance(stream, int):
        return _torch_stream(device, stream)
    if stream.device != device:
        raise ValueError(f"stream must be on {device}")
    return stream


_CUDA = None  # torch's raw CUDA calls, once a prepared call has been made


def _cuda_calls():
    global _CUDA
    _torch().cuda.init()
    _CUDA = _torch()._C
    return _CUDA


class _Prepared:
    """A call over fixed buffers: its parameter block is built and checked
    once, and each call is one ABI call on the given (or torch's current)
    stream.  The tensors are referenced for the object's life.  Outputs and
    scratch that an expert product's object makes itself are memory of the
    stream that is current then, and may be used on any."""

    _home, _made, _weights, _ready, _streams = None, (), (), None, None

    def _own(self, made, weights, once):
        """made: the buffers that the object made itself, on the stream that
        is current now.  Their memory may have been given back there a moment
        ago, with work on it still to run, and goes back there when the object
        goes: the first call on another stream waits for what is queued now,
        and is waited for then.  weights: the call's MxWeights, whose packed
        scales are kept for each stream likewise.  once: the object is called
        at once and on the current stream only."""
        torch = _torch()
        self._home = torch._C._cuda_getCurrentRawStream(self.device.index)
        self._made, self._weights, self._streams = [t for t in made if t is not None], weights, set()
        if self._made and not once:
            with _launch_ctx(self.device):
                if torch.cuda.is_current_stream_capturing():
                    self._ready = torch.cuda.current_stream()  # (an event of this capture is of no use to others)
                else:
                    self._ready = torch.cuda.Event()
                    self._ready.record()

    def _first_on(self, sp):
        """The object's first call on the stream sp."""
        torch = _torch()
        if sp != self._home and self._made:
            own = _torch_stream(self.device, sp)

            def capturing(stream):
                with torch.cuda.stream(stream):
                    return torch.cuda.is_current_stream_capturing()

            # (a capture takes no event from outside; what was queued before it has run when the graph does)
            if isinstance(self._ready, torch.cuda.Event):
                if not capturing(own):
                    own.wait_event(self._ready)
            elif self._ready is not None and capturing(self._ready) and capturing(own):
                own.wait_stream(self._ready)
            for t in self._made:
                t.record_stream(own)
        for w in self._weights:
            w._used_on(sp)
        self._streams.add(sp)

    def __call__(self, stream=None):
        """Launch on the buffers' device; stream: a torch stream of that
        device, a raw cudaStream_t (int) of that device, or None (torch's
        current stream there)."""
        c, index = _CUDA or _cuda_calls(), self.device.index
        if stream is None:
            sp = c._cuda_getCurrentRawStream(index)  # (current_stream().cuda_stream costs 2 us)
        elif isinstance(stream, int):
            sp = stream
        else:
            if stream.device != self.device:
                raise ValueError(f"stream must be on {self.device}")
            sp = stream.cuda_stream
        if self._streams is not None and sp not in self._streams:
            self._first_on(sp)
        if c._cuda_getDevice() == index:
            status = self._fn(self._ref, sp)
        else:
            with _launch_ctx(self.device):
                status = self._fn(self._ref, sp)
        if status != MR_OK:
            _check(status, self._name)
        return self.out


class PreparedRoute(_Prepared):
    """The one-launch route over fixed buffers: the arguments are checked and
    the mr_route_params block is built once; each call is one launch of
    mr_moe_route on the given (or torch's current) stream.  The tensors are
    referenced for the object's life; refill x (and rstd) in place between
    calls.  Arguments as moe_route."""

    def __init__(self, x, w, topk: int, block: int, scoring: str = "softmax", bias=None, renormalize: bool = True,
                 quant="mxfp8", rstd=None, norm_weight=None, norm: str = "gemma", out=None,
                 scratch: Scratch | None = None, shared=None):
        self.p, self.out, self._keep = _route_params(x, w, topk, block, scoring, bias, renormalize, quant, rstd,
                                                     norm_weight, norm, out, scratch, shared)
        self.device = x.device
        self._ref = ctypes.byref(self.p)
        self._fn, self._name = _load().mr_moe_route, "mr_moe_route"


def _route_params(x, w, topk, block, scoring, bias, renormalize, quant, rstd, norm_weight, norm, out, scratch,
                  shared=None):
    torch = _torch()
    ldx = _row_major_2d(x, "x")
    M, K = x.shape
    N = w.shape[0]
    _check_w(w, K)
    if quant not in QUANT_FORMAT:
        raise ValueError(f"quant must be one of {list(QUANT_FORMAT)}")
    if rstd is not None:
        if norm_weight is None:
            raise ValueError("rstd needs norm_weight")
        _check_norm_args(rstd, norm_weight, M, K)
    dev = _one_device(x=x, w=w, bias=bias, rstd=rstd, norm_weight=norm_weight)
    _check_bias(bias, N, dev)
    if out is None:
        out = alloc_route_outputs(M, N, K, topk, block, dev, quant)
    _check_route_out(out, M, N, K, topk, block, quant, dev)
    if scratch is None:
        scratch = Scratch(M, N, K, topk, device=dev)
    _check_scratch(scratch, dev)
    p = RouteParams()
    p.x = _dev_ptr(x, "x", torch.bfloat16)
    p.ldx = ldx
    p.rstd = _dev_ptr(rstd, "rstd", torch.float32, allow_none=True)
    p.norm_weight = _dev_ptr(norm_weight, "norm_weight", torch.bfloat16, allow_none=True)
    p.norm_kind = NORM_KIND[norm]
    p.w = _dev_ptr(w, "w", torch.bfloat16)
    p.M, p.N, p.K, p.topk = M, N, K, topk
    p.scoring = SCORING[scoring]
    p.sel_bias = _dev_ptr(bias, "bias", torch.float32, allow_none=True)
    p.renormalize = int(renormalize)
    p.block = block
    p.quant_format = QUANT_FORMAT[quant]
    p.logits = _dev_ptr(out["logits"], "logits", torch.float32)
    p.topk_ids = _dev_ptr(out["topk_ids"], "topk_ids", torch.int32)
    p.topk_weights = _dev_ptr(out["topk_weights"], "topk_weights", torch.float32)
    p.sorted_token_ids = _dev_ptr(out["sorted_token_ids"], "sorted_token_ids", torch.int32)
    p.expert_ids = _dev_ptr(out["expert_ids"], "expert_ids", torch.int32)
    p.num_tokens_post_padded = _dev_ptr(out["num_tokens_post_padded"], "num_tokens_post_padded", torch.int32)
    p.capacity = out["sorted_token_ids"].numel()
    if quant is not None:
        qt, st = out["q"], out["scale"]
        p.q = _dev_ptr(qt, "q", torch.uint8)
        p.scale = _dev_ptr(st, "scale", torch.uint8)
    p.scratch = scratch.ptr
    p.scratch_bytes = scratch.nbytes
    if shared is not None:
        I = _check_shared(shared, M, K, dev)
        if "shared_act" not in out:
            out["shared_act"] = torch.empty((M, I), dtype=torch.bfloat16, device=dev)
        _check_out(out["shared_act"], "shared_act", (M, I), torch.bfloat16, dev)
        p.shared_w13 = _dev_ptr(shared[0], "w13", torch.uint8)
        p.shared_w13_scale = _dev_ptr(shared[1], "w13_scale", torch.uint8)
        p.shared_inter = I
        p.shared_act = _dev_ptr(out["shared_act"], "shared_act", torch.bfloat16)
    return p, out, (x, w, bias, rstd, norm_weight, scratch, shared)


def moe_sort_quant(topk_ids, x, num_experts: int, block: int, quant: str = "mxfp8", out=None, stream=None,
                   sorted_rows: bool = False):
    """Sort and stage-1 quant in one launch (decode batches, M * topk <= 65536):
    (sorted_token_ids, expert_ids, num_tokens_post_padded, q, scale).  q and
    scale are in token order ([M, K or K/2], [M, K/32]), or with sorted_rows
    in sorted order ([capacity, ...] rows: row p quantises the token of the
    assignment at sorted position p, padding rows are zero, rows past
    num_tokens_post_padded are left as they were)."""
    torch = _torch()
    if topk_ids.dim() != 2 or not topk_ids.is_contiguous():
        raise ValueError("topk_ids must be contiguous [M, k]")
    M, k = topk_ids.shape
    ldx = _row_major_2d(x, "x")
    if x.shape[0] != M:
        raise ValueError("x must have the rows of topk_ids")
    K = x.shape[1]
    if quant not in ("mxfp8", "mxfp4"):
        raise ValueError("quant must be mxfp8 or mxfp4")
    dev = _one_device(topk_ids=topk_ids, x=x)
    cap = sort_capacity(M, k, num_experts, block)
    if cap < 0:
        raise MoeRouteUnsupported(MR_ERR_UNSUPPORTED, "mr_sort_capacity")
    rows = cap if sorted_rows else M
    qk = K // 2 if quant == "mxfp4" else K
    if out is None:
        out = (torch.empty(cap, dtype=torch.int32, device=dev), torch.empty(cap // block, dtype=torch.int32, device=dev),
               torch.empty(1, dtype=torch.int32, device=dev), torch.empty((rows, qk), dtype=torch.uint8, device=dev),
               torch.empty((rows, K // 32), dtype=torch.uint8, device=dev))
    st, ex, nt, q, s = out
    _check_sort_out(st, ex, nt, cap, block, dev)
    if sorted_rows and st.numel() != cap:
        raise ValueError("sorted rows: sorted_token_ids must hold exactly the capacity (its rows index q)")
    _check_out(q, "q", (rows, qk), torch.uint8, dev)
    _check_out(s, "scale", (rows, K // 32), torch.uint8, dev)
    fmt = QUANT_FORMAT[quant] | (QUANT_SORTED_ROWS if sorted_rows else 0)
    with _launch_ctx(dev):
        status = _load().mr_moe_sort_quant(_dev_ptr(topk_ids, "topk_ids", torch.int32), M, k, num_experts, block,
                                           _dev_ptr(x, "x", torch.bfloat16), ldx, K, fmt,
                                           _dev_ptr(st, "sorted_token_ids", torch.int32),
                                           _dev_ptr(ex, "expert_ids", torch.int32),
                                           _dev_ptr(nt, "num_tokens_post_padded", torch.int32), st.numel(),
                                           _dev_ptr(q, "q", torch.uint8), _dev_ptr(s, "scale", torch.uint8),
                                           _stream_on(dev, stream))
    _check(status, "mr_moe_sort_quant")
    return st, ex, nt, q, s


# ---------------------------------------------------------------- expert products

def _call_once(device, stream, make):
    """One call of make(), a prepared form, on the given (or torch's current)
    stream.  Buffers that it makes itself come from that stream's memory, as
    if it were the current one; the result is kept for the current one too."""
    own = _given_stream(device, stream)
    if own is None:
        return make()()
    torch = _torch()
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(own):
        call = make()
        call()
    if here != own:
        outs = call.out
        for t in outs.values() if isinstance(outs, dict) else outs if isinstance(outs, tuple) else (outs,):
            if any(t is m for m in call._made):
                t.record_stream(here)
    return call.out


class MxWeight:
    """An MX weight of mx_gemm ([R, K]) or of the experts ([E, R, K]): codes
    uint8 (E4M3 [..., K], or E2M1 [..., K/2] as mxfp4_quant packs them) and
    E8M0 scale bytes [..., K/32], both contiguous.  The codes are used where
    they are; the scales are laid out once for the tensor core, here, on the
    given (or torch's current) stream (refresh() after changing them), in
    memory of that stream; calls on other streams have to come after it.
    gate_up: the weight of moe_gate_up, R = 2I with the gate rows first."""

    def __init__(self, codes, scale, format: str = "mxfp8", gate_up: bool = False, stream=None):
        torch = _torch()
        if format not in ("mxfp8", "mxfp4"):
            raise ValueError("format must be mxfp8 or mxfp4")
        if codes.dim() not in (2, 3):
            raise ValueError("codes must be [R, K] or [E, R, K]")
        dev = _one_device(codes=codes, scale=scale)
        self.format, self.gate_up, self.codes, self.scale, self.device = format, bool(gate_up), codes, scale, dev
        self.E = codes.shape[0] if codes.dim() == 3 else 1
        self.R = codes.shape[-2]
        self.K = codes.shape[-1] * (2 if format == "mxfp4" else 1)
        if self.K % 32:
            raise ValueError("K must be a multiple of 32")
        _check_out(codes, "codes", codes.shape, torch.uint8, dev)
        _check_out(scale, "scale", (*codes.shape[:-1], self.K // 32), torch.uint8, dev)
        n = int(_load().mr_mx_packed_scale_bytes(self.E, self.R, self.K, QUANT_FORMAT[format], int(self.gate_up)))
        if n == 0:
            raise MoeRouteUnsupported(MR_ERR_UNSUPPORTED, "mr_mx_packed_scale_bytes")
        with torch.cuda.stream(_given_stream(dev, stream)):
            self.packed = torch.empty(n, dtype=torch.uint8, device=dev)
            self._streams = {torch._C._cuda_getCurrentRawStream(dev.index)}
        self.refresh(stream)

    def refresh(self, stream=None):
        """Lay the scales out again (after they were changed in place)."""
        torch = _torch()
        own = _given_stream(self.device, stream) or torch.cuda.current_stream(self.device)
        self._used_on(own.cuda_stream)
        with _launch_ctx(self.device):
            _check(_load().mr_mx_pack_scales(ctypes.c_void_p(self.scale.data_ptr()), self.E, self.R, self.K,
                                             QUANT_FORMAT[self.format], int(self.gate_up),
                                             ctypes.c_void_p(self.packed.data_ptr()),
                                             ctypes.c_void_p(own.cuda_stream)), "mr_mx_pack_scales")

    def _used_on(self, sp):
        """The packed scales are used on the stream sp: their memory is not
        given to others before that stream is done with them."""
        if sp not in self._streams:
            self.packed.record_stream(_torch_stream(self.device, sp))
            self._streams.add(sp)


# moe_down keeps up to this many numbers on their way to the sum (M * topk * R) in fp32 unless it is told otherwise,
# 64 MB, half of L2; more are rounded to bf16.  128 experts x 6144 x 768, E4M3, top-8: of 64 tokens 83.7 us instead of
# 82.1, of 256 (12.6 million) 105 instead of 101; of 512 they would take 125 instead of 108, of 4096 417 instead of 260.
SLOTS_FP32_MAX = 1 << 24


class ExpertScratch:
    """A caller-owned scratch buffer of moe_down for up to M_max tokens of
    topk slots and R output columns: torch uint8 tensors whose contents do not
    matter between calls, tensor for the slots' rows (bf16, or the upper halves
    of fp32) and low for the lower halves.  slots_fp32: True for calls of any
    size with slots_fp32; False for none (no low); None for those whose size
    has them so."""

    def __init__(self, M_max: int, topk: int, R: int, device=None, slots_fp32: bool | None = None):
        torch = _torch()
        self.nbytes = int(_load().mr_expert_scratch_bytes(M_max, topk, R))
        if self.nbytes == 0:
            raise ValueError("scratch size query rejected the arguments")
        dev = device if device is not None else "cuda"
        self.tensor = torch.empty(self.nbytes, dtype=torch.uint8, device=dev)
        self.low_nbytes = (self.nbytes if slots_fp32 else 0 if slots_fp32 is not None
                           else min(self.nbytes, 2 * SLOTS_FP32_MAX))
        self.low = torch.empty(self.low_nbytes, dtype=torch.uint8, device=dev) if self.low_nbytes else None

    @property
    def ptr(self):
        return ctypes.c_void_p(self.tensor.data_ptr())

    @property
    def low_ptr(self):
        return None if self.low is None else ctypes.c_void_p(self.low.data_ptr())


class MxGemmParams(ctypes.Structure):
    """mr_mx_gemm_params of moe_route.h, field for field."""
    _fields_ = [("q", _P), ("ldq", _I64), ("scale", _P), ("lds", _I64), ("w", _P), ("w_scale", _P), ("M", _I),
                ("R", _I), ("K", _I), ("format", _I), ("out", _P), ("ldo", _I64), ("out_fp32", _I)]


class GateUpParams(ctypes.Structure):
    """mr_moe_gate_up_params of moe_route.h, field for field."""
    _fields_ = [("q", _P), ("ldq", _I64), ("scale", _P), ("lds", _I64), ("sorted_rows", _I), ("w13", _P),
                ("w13_scale", _P), ("E", _I), ("I", _I), ("K", _I), ("format", _I), ("sorted_token_ids", _P),
                ("expert_ids", _P), ("n_blocks", _I), ("block", _I), ("M", _I), ("topk", _I), ("out_format", _I),
                ("act", _P), ("act_scale", _P)]


class DownParams(ctypes.Structure):
    """mr_moe_down_params of moe_route.h, field for field."""
    _fields_ = [("q", _P), ("ldq", _I64), ("scale", _P), ("lds", _I64), ("w2", _P), ("w2_scale", _P), ("E", _I),
                ("R", _I), ("I", _I), ("format", _I), ("sorted_token_ids", _P), ("expert_ids", _P), ("n_blocks", _I),
                ("block", _I), ("M", _I), ("topk", _I), ("topk_ids", _P), ("topk_weights", _P), ("add", _P),
                ("out", _P), ("scratch", _P), ("scratch_bytes", _SZ), ("scratch_low", _P), ("scratch_low_bytes", _SZ)]


def _mx_rows(p, q, scale, K, fmt, what="q"):
    """Codes and scales of an MX activation, rows of K elements, into p; returns the rows."""
    torch = _torch()
    if q.dim() != 2 or q.shape[1] != (K // 2 if fmt == "mxfp4" else K) or (q.shape[1] > 1 and q.stride(1) != 1):
        raise ValueError(f"{what} must be [rows, {K // 2 if fmt == 'mxfp4' else K}] with a contiguous last dimension")
    if scale.dim() != 2 or tuple(scale.shape) != (q.shape[0], K // 32) or (K > 32 and scale.stride(1) != 1):
        raise ValueError(f"{what}'s scale must be [{q.shape[0]}, {K // 32}] with a contiguous last dimension")
    p.q = _dev_ptr(q, what, torch.uint8)
    p.scale = _dev_ptr(scale, "scale", torch.uint8)
    # one row: any stride will do
    p.ldq = q.stride(0) if q.shape[0] > 1 else q.shape[1]
    p.lds = scale.stride(0) if q.shape[0] > 1 else scale.shape[1]
    return q.shape[0]


def _check_sorted(st, ex, block, dev):
    """The sort's outputs as the expert products read them; returns the blocks."""
    torch = _torch()
    if block < 1:
        raise ValueError("block must be at least 1")
    for t, name in ((st, "sorted_token_ids"), (ex, "expert_ids")):
        if t.dim() != 1 or t.dtype != torch.int32 or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"{name} must be a contiguous int32 vector on {dev}")
    n = min(ex.numel(), st.numel() // block)
    if n < 1:
        raise ValueError("sorted_token_ids and expert_ids hold no block")
    return n


class PreparedMxGemm(_Prepared):
    """mx_gemm over fixed buffers; arguments as mx_gemm."""

    def __init__(self, q, scale, w: MxWeight, out=None, out_dtype=None, _once=False):
        torch = _torch()
        if w.codes.dim() != 2 or w.gate_up:
            raise ValueError("mx_gemm takes a weight [R, K] laid out without gate_up")
        dev = _one_device(q=q, scale=scale, w=w.codes, out=out)
        p = self.p = MxGemmParams()
        M = _mx_rows(p, q, scale, w.K, w.format)
        made = out is None
        if made:
            out = torch.empty((M, w.R), dtype=out_dtype or torch.bfloat16, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out must be {out_dtype}, got {out.dtype}")
        if out.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out must be bfloat16 or float32")
        if tuple(out.shape) != (M, w.R) or (w.R > 1 and out.stride(1) != 1) or (M > 1 and out.stride(0) < w.R):
            raise ValueError(f"out must have shape {(M, w.R)} with a contiguous last dimension")
        p.w, p.w_scale = w.codes.data_ptr(), w.packed.data_ptr()
        p.M, p.R, p.K, p.format = M, w.R, w.K, QUANT_FORMAT[w.format]
        p.out, p.ldo, p.out_fp32 = out.data_ptr(), out.stride(0) if M > 1 else w.R, int(out.dtype == torch.float32)
        self.out, self.device, self._keep = out, dev, (q, scale, w)
        self._ref = ctypes.byref(p)
        self._fn, self._name = _load().mr_mx_gemm, "mr_mx_gemm"
        self._own((out,) if made else (), (w,), _once)


def mx_gemm(q, scale, w: MxWeight, out=None, out_dtype=None, stream=None):
    """Product of microscaled operands: [M, R] (bf16, or out_dtype fp32) =
    x [M, K] @ w [R, K]^T with x given as the codes q and scales of
    mxfp8_quant / mxfp4_quant, in the weight's format."""
    return _call_once(_one_device(q=q), stream, lambda: PreparedMxGemm(q, scale, w, out, out_dtype, _once=True))


class PreparedGateUp(_Prepared):
    """moe_gate_up over fixed buffers; arguments as moe_gate_up."""

    def __init__(self, q, scale, w13: MxWeight, sorted_token_ids, expert_ids, topk: int, block: int,
                 num_tokens: int | None = None, sorted_rows: bool = False, quant=None, out=None, _once=False):
        torch = _torch()
        if w13.codes.dim() != 3 or not w13.gate_up:
            raise ValueError("moe_gate_up takes a weight [E, 2I, K] laid out with gate_up=True")
        if quant not in QUANT_FORMAT:
            raise ValueError(f"quant must be one of {list(QUANT_FORMAT)}")
        o0, o1 = (out, None) if quant is None or out is None else out
        dev = _one_device(q=q, scale=scale, w13=w13.codes, sorted_token_ids=sorted_token_ids, expert_ids=expert_ids,
                          out=o0, out_scale=o1)
        p = self.p = GateUpParams()
        rows = _mx_rows(p, q, scale, w13.K, w13.format)
        n = _check_sorted(sorted_token_ids, expert_ids, block, dev)
        if sorted_rows:
            if num_tokens is None:
                raise ValueError("sorted rows need num_tokens")
            if rows < n * block:
                raise ValueError(f"sorted rows: q needs {n * block} rows, has {rows}")
        elif num_tokens is not None and num_tokens != rows:
            raise ValueError("num_tokens differs from the rows of q")
        M = num_tokens if sorted_rows else rows
        I = w13.R // 2
        cap = sorted_token_ids.numel()
        made = out is None
        if quant is None:
            if o0 is None:
                o0 = torch.empty((cap, I), dtype=torch.bfloat16, device=dev)
            _check_out(o0, "out", (cap, I), torch.bfloat16, dev)
            out = o0
        else:
            iq = I // 2 if quant == "mxfp4" else I
            if o0 is None:
                o0 = torch.empty((cap, iq), dtype=torch.uint8, device=dev)
                o1 = torch.empty((cap, I // 32), dtype=torch.uint8, device=dev)
            _check_out(o0, "out codes", (cap, iq), torch.uint8, dev)
            _check_out(o1, "out scale", (cap, I // 32), torch.uint8, dev)
            out = (o0, o1)
        p.sorted_rows = int(sorted_rows)
        p.w13, p.w13_scale = w13.codes.data_ptr(), w13.packed.data_ptr()
        p.E, p.I, p.K, p.format = w13.E, I, w13.K, QUANT_FORMAT[w13.format]
        p.sorted_token_ids, p.expert_ids = sorted_token_ids.data_ptr(), expert_ids.data_ptr()
        p.n_blocks, p.block, p.M, p.topk = n, block, M, topk
        p.out_format, p.act = QUANT_FORMAT[quant], o0.data_ptr()
        p.act_scale = None if quant is None else o1.data_ptr()
        self.out, self.device, self._keep = out, dev, (q, scale, w13, sorted_token_ids, expert_ids)
        self._ref = ctypes.byref(p)
        self._fn, self._name = _load().mr_moe_gate_up, "mr_moe_gate_up"
        self._own((o0, o1) if made else (), (w13,), _once)


def moe_gate_up(q, scale, w13: MxWeight, sorted_token_ids, expert_ids, topk: int, block: int,
                num_tokens: int | None = None, sorted_rows: bool = False, quant=None, out=None, stream=None):
    """Stage 1 of the routed experts (mr_moe_gate_up): silu(x . gate^T) *
    (x . up^T) of every assignment, at its sorted position.  q, scale: the
    quantised tokens [M, ...], or with sorted_rows the rows at the sorted
    positions (moe_sort_quant(..., sorted_rows=True); num_tokens is then the
    number of tokens).  quant None: bf16 [capacity, I]; "mxfp8" / "mxfp4":
    (codes, scales), as mxfp8_quant / mxfp4_quant of those rows.  Rows that
    hold no assignment are left as they were."""
    return _call_once(_one_device(q=q), stream,
                      lambda: PreparedGateUp(q, scale, w13, sorted_token_ids, expert_ids, topk, block, num_tokens,
                                             sorted_rows, quant, out, _once=True))


class PreparedDown(_Prepared):
    """moe_down over fixed buffers; arguments as moe_down."""

    def __init__(self, q, scale, w2: MxWeight, topk_ids, topk_weights, sorted_token_ids, expert_ids, block: int,
                 add=None, out=None, scratch: ExpertScratch | None = None, slots_fp32: bool | None = None, _once=False):
        torch = _torch()
        if w2.codes.dim() != 3 or w2.gate_up:
            raise ValueError("moe_down takes a weight [E, R, I] laid out without gate_up")
        dev = _one_device(q=q, scale=scale, w2=w2.codes, topk_ids=topk_ids, topk_weights=topk_weights,
                          sorted_token_ids=sorted_token_ids, expert_ids=expert_ids, add=add, out=out)
        p = self.p = DownParams()
        rows = _mx_rows(p, q, scale, w2.K, w2.format)
        n = _check_sorted(sorted_token_ids, expert_ids, block, dev)
        if rows < n * block:
            raise ValueError(f"q needs {n * block} rows, has {rows}")
        if topk_ids.dim() != 2:
            raise ValueError("topk_ids must be contiguous [M, k]")
        M, topk = topk_ids.shape
        _check_out(topk_ids, "topk_ids", (M, topk), torch.int32, dev)
        _check_out(topk_weights, "topk_weights", (M, topk), torch.float32, dev)
        if add is not None:
            _check_out(add, "add", (M, w2.R), torch.bfloat16, dev)
        made = []
        if out is None:
            out = torch.empty((M, w2.R), dtype=torch.bfloat16, device=dev)
            made.append(out)
        _check_out(out, "out", (M, w2.R), torch.bfloat16, dev)
        if slots_fp32 is None:
            slots_fp32 = M * topk * w2.R <= SLOTS_FP32_MAX and (scratch is None or scratch.low is not None)
        if scratch is None:
            scratch = ExpertScratch(M, topk, w2.R, device=dev, slots_fp32=slots_fp32)
            made += [scratch.tensor, scratch.low]
        _check_scratch(scratch, dev)
        if slots_fp32 and scratch.low is None:
            raise ValueError("slots_fp32 needs a scratch that is made for it")
        p.w2, p.w2_scale = w2.codes.data_ptr(), w2.packed.data_ptr()
        p.E, p.R, p.I, p.format = w2.E, w2.R, w2.K, QUANT_FORMAT[w2.format]
        p.sorted_token_ids, p.expert_ids = sorted_token_ids.data_ptr(), expert_ids.data_ptr()
        p.n_blocks, p.block, p.M, p.topk = n, block, M, topk
        p.topk_ids, p.topk_weights = topk_ids.data_ptr(), topk_weights.data_ptr()
        p.add = None if add is None else add.data_ptr()
        p.out = out.data_ptr()
        p.scratch, p.scratch_bytes = scratch.ptr, scratch.nbytes
        if slots_fp32:
            p.scratch_low, p.scratch_low_bytes = scratch.low_ptr, scratch.low_nbytes
        self.out, self.device = out, dev
        self._keep = (q, scale, w2, topk_ids, topk_weights, sorted_token_ids, expert_ids, add)
        self.scratch = scratch
        self._ref = ctypes.byref(p)
        self._fn, self._name = _load().mr_moe_down, "mr_moe_down"
        self._own(made, (w2,), _once)


def moe_down(q, scale, w2: MxWeight, topk_ids, topk_weights, sorted_token_ids, expert_ids, block: int, add=None,
             out=None, scratch: ExpertScratch | None = None, stream=None, slots_fp32: bool | None = None):
    """Stage 2 of the routed experts and the combination (mr_moe_down): bf16
    [M, R] = add + sum over a token's slots of topk_weights times its row of
    act @ w2^T.  q, scale: act's codes and scales at the sorted positions, as
    moe_gate_up(..., quant=...) returns them.  Slots whose id is outside
    [0, E) add nothing.  slots_fp32: True keeps the slots' rows in fp32 on
    their way to the sum; False rounds them to bf16, which adds up to 2^-8 of
    every weighted row to a result's error; None: in fp32 while M * topk * R is
    at most SLOTS_FP32_MAX and a given scratch has room for it."""
    return _call_once(_one_device(q=q), stream,
                      lambda: PreparedDown(q, scale, w2, topk_ids, topk_weights, sorted_token_ids, expert_ids, block, add,
                                           out, scratch, slots_fp32, _once=True))


# ---------------------------------------------------------------- residual norm, FP8 with scales per 128

NORM_QUANT = {**QUANT_FORMAT, "fp8": 3}  # of add_rms_norm


class AddNormParams(ctypes.Structure):
    """mr_add_rms_norm_params of moe_route.h, field for field."""
    _fields_ = [("x", _P), ("ldx", _I64), ("residual", _P), ("ldr", _I64), ("norm_weight", _P), ("norm_kind", _I),
                ("eps", ctypes.c_float), ("M", _I), ("K", _I), ("quant_format", _I), ("sres", _P), ("lds", _I64),
                ("rstd", _P), ("xn", _P), ("q", _P), ("scale", _P)]


class Fp8GemmParams(ctypes.Structure):
    """mr_fp8_gemm_params of moe_route.h, field for field."""
    _fields_ = [("q", _P), ("ldq", _I64), ("x_scale", _P), ("ldxs", _I64), ("w", _P), ("ldw", _I64), ("w_scale", _P),
                ("ldws", _I64), ("M", _I), ("R", _I), ("K", _I), ("out", _P), ("ldo", _I64), ("out_fp32", _I)]


def _ld(t, multiple: int = 1):
    """Row stride of a 2-D tensor; of a single row any will do."""
    return t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // multiple) * multiple


class PreparedAddNorm(_Prepared):
    """add_rms_norm over fixed buffers; arguments as add_rms_norm."""

    def __init__(self, x, residual, norm_weight, eps: float = 1e-6, norm: str = "gemma", quant=None, outputs=None,
                 out=None, _once=False):
        torch = _torch()
        if quant not in NORM_QUANT:
            raise ValueError(f"quant must be one of {list(NORM_QUANT)}")
        if norm not in NORM_KIND:
            raise ValueError(f"norm must be one of {list(NORM_KIND)}")
        out = dict(out or {})
        codes = {"q", "scale"} if quant is not None else set()
        if outputs is None:
            outputs = {"sres", "rstd"} | (codes or {"xn"})
        wanted = set(outputs) | set(out) | codes
        known = {"sres", "rstd", "xn"} | codes
        if wanted - known or not wanted:
            raise ValueError(f"outputs must be some of {sorted(known)}")
        dev = _one_device(x=x, residual=residual, norm_weight=norm_weight, **out)
        _row_major_2d(x, "x")
        M, K = x.shape
        if residual is not None:
            _row_major_2d(residual, "residual")
            if residual.shape != x.shape:
                raise ValueError("residual must have the shape of x")
        if norm_weight.dim() != 1 or norm_weight.shape[0] != K or not norm_weight.is_contiguous():
            raise ValueError("norm_weight must be contiguous [K]")
        if quant in ("mxfp8", "mxfp4") and K % 32:
            raise ValueError("K must be a multiple of 32")
        bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
        spec = {"sres": ((M, K), bf16), "rstd": ((M,), f32), "xn": ((M, K), bf16),
                "q": ((M, K // 2 if quant == "mxfp4" else K), u8),
                "scale": ((M, -(-K // 128)), f32) if quant == "fp8" else ((M, K // 32), u8)}
        made = []
        for name in ("sres", "rstd", "xn", "q", "scale"):
            if name not in wanted:
                continue
            shape, dt = spec[name]
            if name not in out:
                out[name] = torch.empty(shape, dtype=dt, device=dev)
                made.append(out[name])
            elif name == "sres":  # (as x: any row stride)
                if out[name].shape != x.shape or out[name].dtype != bf16:
                    raise ValueError(f"sres must be bfloat16 {tuple(x.shape)}")
                _row_major_2d(out[name], "sres")
            else:
                _check_out(out[name], name, shape, dt, dev)
        p = self.p = AddNormParams()
        p.x, p.ldx = _dev_ptr(x, "x", bf16), _ld(x, 8)
        p.residual = _dev_ptr(residual, "residual", bf16, allow_none=True)
        p.ldr = 0 if residual is None else _ld(residual, 8)
        p.norm_weight, p.norm_kind = _dev_ptr(norm_weight, "norm_weight", bf16), NORM_KIND[norm]
        p.eps, p.M, p.K, p.quant_format = float(eps), M, K, NORM_QUANT[quant]
        for name in wanted:
            setattr(p, name, out[name].data_ptr())
        p.lds = _ld(out["sres"], 8) if "sres" in wanted else 0
        self.out, self.device, self._keep = out, dev, (x, residual, norm_weight)
        self._ref = ctypes.byref(p)
        self._fn, self._name = _load().mr_add_rms_norm, "mr_add_rms_norm"
        self._own(made, (), _once)


def add_rms_norm(x, residual, norm_weight, eps: float = 1e-6, norm: str = "gemma", quant=None, outputs=None, out=None,
                 stream=None):
    """The residual's addition and the RMSNorm behind it (mr_add_rms_norm): a
    dict of sres = bf16(x + residual) (residual None: x), rstd [M] fp32, xn
    = bf16((sres * rstd) * s) with s = g ("rms") or 1 + g ("gemma"), and with
    quant its codes q and scales: "mxfp8" / "mxfp4" (uint8 [M, K/32]) or "fp8"
    (fp32 [M, ceil(K/128)], as fp8_quant).  outputs: which ones (default sres,
    rstd and the codes, or xn without quant); out: a dict of given tensors
    (sres may be x or residual itself)."""
    return _call_once(_one_device(x=x), stream,
                      lambda: PreparedAddNorm(x, residual, norm_weight, eps, norm, quant, outputs, out, _once=True))


def fp8_quant(x, out=None, stream=None):
    """(q uint8 [M, K] e4m3 codes, scale fp32 [M, ceil(K/128)]) of bf16 rows."""
    torch = _torch()
    dev = _one_device(x=x, **({} if out is None else dict(q=out[0], scale=out[1])))
    _row_major_2d(x, "x")
    M, K = x.shape
    with torch.cuda.stream(_given_stream(dev, stream)):
        if out is None:
            out = (torch.empty((M, K), dtype=torch.uint8, device=dev),
                   torch.empty((M, -(-K // 128)), dtype=torch.float32, device=dev))
    q, s = out
    _check_out(q, "q", (M, K), torch.uint8, dev)
    _check_out(s, "scale", (M, -(-K // 128)), torch.float32, dev)
    own = _given_stream(dev, stream) or torch.cuda.current_stream(dev)
    with _launch_ctx(dev):
        _check(_load().mr_fp8_quant(_dev_ptr(x, "x", torch.bfloat16), _ld(x, 8), M, K, _dev_ptr(q, "q", torch.uint8),
                                    _dev_ptr(s, "scale", torch.float32), ctypes.c_void_p(own.cuda_stream)),
               "mr_fp8_quant")
        here = torch.cuda.current_stream(dev)
        if own != here:  # (kept for the current stream too, whose results they are)
            for t in out:
                t.record_stream(here)
    return q, s


class PreparedFp8Gemm(_Prepared):
    """fp8_gemm over fixed buffers; arguments as fp8_gemm."""

    def __init__(self, q, scale, w, w_scale, out=None, out_dtype=None, _once=False):
        torch = _torch()
        dev = _one_device(q=q, scale=scale, w=w, w_scale=w_scale, out=out)
        for t, name in ((q, "q"), (scale, "scale"), (w, "w"), (w_scale, "w_scale")):
            if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
                raise ValueError(f"{name} must be 2-D with a contiguous last dimension")
        M, K = q.shape
        R, kb = w.shape[0], -(-K // 128)
        if w.shape[1] != K:
            raise ValueError(f"w must be [R, {K}]")
        if tuple(scale.shape) != (M, kb):
            raise ValueError(f"scale must be {(M, kb)}")
        if tuple(w_scale.shape) != (-(-R // 128), kb):
            raise ValueError(f"w_scale must be {(-(-R // 128), kb)}")
        made = out is None
        if made:
            out = torch.empty((M, R), dtype=out_dtype or torch.bfloat16, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out must be {out_dtype}, got {out.dtype}")
        if out.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out must be bfloat16 or float32")
        if tuple(out.shape) != (M, R) or (R > 1 and out.stride(1) != 1) or (M > 1 and out.stride(0) < R):
            raise ValueError(f"out must have shape {(M, R)} with a contiguous last dimension")
        p = self.p = Fp8GemmParams()
        p.q, p.ldq = _dev_ptr(q, "q", torch.uint8), _ld(q, 16)
        p.x_scale, p.ldxs = _dev_ptr(scale, "scale", torch.float32), _ld(scale)
        p.w, p.ldw = _dev_ptr(w, "w", torch.uint8), _ld(w, 16)
        p.w_scale, p.ldws = _dev_ptr(w_scale, "w_scale", torch.float32), _ld(w_scale)
        p.M, p.R, p.K = M, R, K
        p.out, p.ldo, p.out_fp32 = out.data_ptr(), _ld(out), int(out.dtype == torch.float32)
        self.out, self.device, self._keep = out, dev, (q, scale, w, w_scale)
        self._ref = ctypes.byref(p)
        self._fn, self._name = _load().mr_fp8_gemm, "mr_fp8_gemm"
        self._own((out,) if made else (), (), _once)


def fp8_gemm(q, scale, w, w_scale, out=None, out_dtype=None, stream=None):
    """Product of E4M3 operands with fp32 scales per 128 (mr_fp8_gemm): [M, R]
    (bf16, or out_dtype fp32) = x [M, K] @ w [R, K]^T with x given as the codes
    q (uint8) and scales [M, ceil(K/128)] of fp8_quant, w as codes (uint8) and
    scales [ceil(R/128), ceil(K/128)].  Rows start on 16 bytes."""
    return _call_once(_one_device(q=q), stream,
                      lambda: PreparedFp8Gemm(q, scale, w, w_scale, out, out_dtype, _once=True))


# ---------------------------------------------------------------- rows to the experts and back

class PermuteParams(ctypes.Structure):
    """mr_moe_permute_params of moe_route.h, field for field."""
    _fields_ = [("x", _P), ("ldx", _I64), ("row_type", _I), ("M", _I), ("K", _I), ("topk", _I), ("E", _I),
                ("topk_ids", _P), ("sorted_token_ids", _P), ("num_tokens_post_padded", _P), ("capacity", _I64),
                ("rows", _P), ("positions", _P)]


class CombineParams(ctypes.Structure):
    """mr_moe_combine_params of moe_route.h, field for field."""
    _fields_ = [("y", _P), ("ldy", _I64), ("row_type", _I), ("capacity", _I64), ("M", _I), ("K", _I), ("topk", _I),
                ("positions", _P), ("topk_weights", _P), ("add", _P), ("ldadd", _I64), ("out", _P)]


class CombineGradParams(ctypes.Structure):
    """mr_moe_combine_grad_params of moe_route.h, field for field."""
    _fields_ = [("grad_out", _P), ("ldg", _I64), ("y", _P), ("ldy", _I64), ("row_type", _I), ("capacity", _I64),
                ("M", _I), ("K", _I), ("topk", _I), ("positions", _P), ("topk_weights", _P), ("sorted_token_ids", _P),
                ("num_tokens_post_padded", _P), ("grad_y", _P), ("grad_weights", _P)]


def _row_type(t, name, codes=False):
    torch = _torch()
    types = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, **({torch.uint8: 3} if codes else {})}
    if t.dtype not in types:
        raise ValueError(f"{name} must be one of {[str(d) for d in types]}, got {t.dtype}")
    return types[t.dtype]


def _rows_like(t, name, shape, dtype):
    """An operand of rows: any row stride."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} with a contiguous last dimension")


def _check_sorted_ids(st, nt, dev):
    torch = _torch()
    if st.dim() != 1 or st.numel() < 1:
        raise ValueError("sorted_token_ids must be a vector")
    _check_out(st, "sorted_token_ids", st.numel(), torch.int32, dev, min_numel=True)
    _check_out(nt, "num_tokens_post_padded", 1, torch.int32, dev, min_numel=True)


class PreparedPermute(_Prepared):
    """moe_permute over fixed buffers; arguments as moe_permute."""

    def __init__(self, x, topk_ids, num_experts: int, sorted_token_ids, num_tokens_post_padded, out=None,
                 positions=None, _once=False):
        torch = _torch()
        dev = _one_device(x=x, topk_ids=topk_ids, sorted_token_ids=sorted_token_ids,
                          num_tokens_post_padded=num_tokens_post_padded, out=out, positions=positions)
        if x.dim() != 2 or topk_ids.dim() != 2:
            raise ValueError("x must be [M, K] and topk_ids [M, k]")
        (M, K), topk = x.shape, topk_ids.shape[1]
        _rows_like(x, "x", (M, K), x.dtype)
        _check_out(topk_ids, "topk_ids", (M, topk), torch.int32, dev)
        _check_sorted_ids(sorted_token_ids, num_tokens_post_padded, dev)
        cap, made = sorted_token_ids.numel(), []
        if out is None:
            out = torch.empty((cap, K), dtype=x.dtype, device=dev)
            made.append(out)
        _check_out(out, "out", (cap, K), x.dtype, dev)
        if positions is None:
            positions = torch.empty((M, topk), dtype=torch.int32, device=dev)
            made.append(positions)
        _check_out(positions, "positions", (M, topk), torch.int32, dev)
        p = self.p = PermuteParams()
        p.x, p.ldx, p.row_type = x.data_ptr(), _ld(x), _row_type(x, "x", codes=True)
        p.M, p.K, p.topk, p.E = M, K, topk, num_experts
        p.topk_ids, p.sorted_token_ids = topk_ids.data_ptr(), sorted_token_ids.data_ptr()
        p.num_tokens_post_padded, p.capacity = num_tokens_post_padded.data_ptr(), cap
        p.rows, p.positions = out.data_ptr(), positions.data_ptr()
        self.out, self.device = (out, positions), dev
        self._keep = (x, topk_ids, sorted_token_ids, num_tokens_post_padded)
        self._ref = ctypes.byref(p)
        self._fn, self._name = _load().mr_moe_permute, "mr_moe_permute"
        self._own(made, (), _once)


def moe_permute(x, topk_ids, num_experts: int, sorted_token_ids, num_tokens_post_padded, out=None, positions=None,
                stream=None):
    """Rows of tokens to the sorted positions of their assignments
    (mr_moe_permute): (rows [capacity, K] in x's type, positions int32 [M, k]).
    x: [M, K], bf16, fp16, fp32 or uint8 (codes, scale bytes).  Padding rows
    are zero, rows behind num_tokens_post_padded are left as they were, and an
    assignment that the sort left out has position -1."""
    return _call_once(_one_device(x=x), stream,
                      lambda: PreparedPermute(x, topk_ids, num_experts, sorted_token_ids, num_tokens_post_padded, out,
                                              positions, _once=True))


class PreparedCombine(_Prepared):
    """moe_combine over fixed buffers; arguments as moe_combine."""

    def __init__(self, y, positions, topk_weights=None, add=None, out=None, _once=False):
        torch = _torch()
        dev = _one_device(y=y, positions=positions, topk_weights=topk_weights, add=add, out=out)
        if y.dim() != 2 or positions.dim() != 2:
            raise ValueError("y must be [capacity, K] and positions [M, k]")
        (cap, K), (M, topk) = y.shape, positions.shape
        _rows_like(y, "y", (cap, K), y.dtype)
        _check_out(positions, "positions", (M, topk), torch.int32, dev)
        if topk_weights is not None:
            _check_out(topk_weights, "topk_weights", (M, topk), torch.float32, dev)
        if add is not None:
            _rows_like(add, "add", (M, K), y.dtype)
        made = out is None
        if made:
            out = torch.empty((M, K), dtype=y.dtype, device=dev)
        _check_out(out, "out", (M, K), y.dtype, dev)
        p = self.p = CombineParams()
        p.y, p.ldy, p.row_type, p.capacity = y.data_ptr(), _ld(y), _row_type(y, "y"), cap
        p.M, p.K, p.topk, p.positions = M, K, topk, positions.data_ptr()
        p.topk_weights = None if topk_weights is None else topk_weights.data_ptr()
        if add is not None:
            p.add, p.ldadd = add.data_ptr(), _ld(add)
        p.out = out.data_ptr()
        self.out, self.device, self._keep = out, dev, (y, positions, topk_weights, add)
        self._ref = ctypes.byref(p)
        self._fn, self._name = _load().mr_moe_combine, "mr_moe_combine"
        self._own((out,) if made else (), (), _once)


def moe_combine(y, positions, topk_weights=None, add=None, out=None, stream=None):
    """Rows at the sorted positions back to their tokens (mr_moe_combine):
    [M, K] = add + sum over a token's slots of topk_weights (None: one) times
    the row of y [capacity, K] at positions [M, k]; positions outside y add
    nothing.  out may be add itself."""
    return _call_once(_one_device(y=y), stream,
                      lambda: PreparedCombine(y, positions, topk_weights, add, out, _once=True))


class PreparedPermuteGrad(PreparedCombine):
    """moe_permute_grad over fixed buffers; arguments as moe_permute_grad."""

    def __init__(self, grad_rows, positions, out=None, _once=False):
        super().__init__(grad_rows, positions, out=out, _once=_once)


def moe_permute_grad(grad_rows, positions, out=None, stream=None):
    """Gradient of moe_permute for x: [M, K] = the sum over a token's slots of
    the rows of grad_rows [capacity, K] at positions [M, k] (those of padding
    positions count for nothing)."""
    return _call_once(_one_device(grad_rows=grad_rows), stream,
                      lambda: PreparedPermuteGrad(grad_rows, positions, out, _once=True))


class PreparedCombineGrad(_Prepared):
    """moe_combine_grad over fixed buffers; arguments as moe_combine_grad."""

    def __init__(self, grad_out, y, positions, topk_weights, sorted_token_ids, num_tokens_post_padded, out=None,
                 grad_weights=None, _once=False):
        torch = _torch()
        dev = _one_device(grad_out=grad_out, y=y, positions=positions, topk_weights=topk_weights,
                          sorted_token_ids=sorted_token_ids, num_tokens_post_padded=num_tokens_post_padded, out=out,
                          grad_weights=grad_weights)
        if grad_out.dim() != 2 or positions.dim() != 2:
            raise ValueError("grad_out must be [M, K] and positions [M, k]")
        (M, K), topk = grad_out.shape, positions.shape[1]
        _rows_like(grad_out, "grad_out", (M, K), grad_out.dtype)
        _check_out(positions, "positions", (M, topk), torch.int32, dev)
        if topk_weights is not None:
            _check_out(topk_weights, "topk_weights", (M, topk), torch.float32, dev)
        _check_sorted_ids(sorted_token_ids, num_tokens_post_padded, dev)
        cap, made = sorted_token_ids.numel(), []
        _rows_like(y, "y", (cap, K), grad_out.dtype)
        if out is None:
            out = torch.empty((cap, K), dtype=y.dtype, device=dev)
            made.append(out)
        _check_out(out, "out", (cap, K), y.dtype, dev)
        if grad_weights is None:
            grad_weights = torch.empty((M, topk), dtype=torch.float32, device=dev)
            made.append(grad_weights)
        _check_out(grad_weights, "grad_weights", (M, topk), torch.float32, dev)
        p = self.p = CombineGradParams()
        p.grad_out, p.ldg, p.y, p.ldy = grad_out.data_ptr(), _ld(grad_out), y.data_ptr(), _ld(y)
        p.row_type, p.capacity = _row_type(y, "y"), cap
        p.M, p.K, p.topk, p.positions = M, K, topk, positions.data_ptr()
        p.topk_weights = None if topk_weights is None else topk_weights.data_ptr()
        p.sorted_token_ids = sorted_token_ids.data_ptr()
        p.num_tokens_post_padded = num_tokens_post_padded.data_ptr()
        p.grad_y, p.grad_weights = out.data_ptr(), grad_weights.data_ptr()
        self.out, self.device = (out, grad_weights), dev
        self._keep = (grad_out, y, positions, topk_weights, sorted_token_ids, num_tokens_post_padded)
        self._ref = ctypes.byref(p)
        self._fn, self._name = _load().mr_moe_combine_grad, "mr_moe_combine_grad"
        self._own(made, (), _once)


def moe_combine_grad(grad_out, y, positions, topk_weights, sorted_token_ids, num_tokens_post_padded, out=None,
                     grad_weights=None, stream=None):
    """Gradients of moe_combine for its y and topk_weights (mr_moe_combine_grad):
    (grad_y [capacity, K], grad_weights fp32 [M, k]).  grad_y has zeros at
    padding positions and is left as it was behind num_tokens_post_padded;
    out may be y itself.  (The gradient of add is grad_out.)"""
    return _call_once(_one_device(grad_out=grad_out), stream,
                      lambda: PreparedCombineGrad(grad_out, y, positions, topk_weights, sorted_token_ids,
                                                  num_tokens_post_padded, out, grad_weights, _once=True))
