"""ctypes binding of libbitopt.so (include/bitopt.h), argument marshalling only.

Every function takes torch tensors (device tensors for device entry points),
checks shapes/dtypes/devices, passes raw pointers and the current HIP stream to
the C ABI, and raises BitoptError on a non-zero status.  All arithmetic of the
step runs in the library's HIP kernels; if the library is not built, loading
fails with an error instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbitopt.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_DEVICE = 0, -1, -2, -3
DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
OPTIMIZERS = {"adam": 0, "adamw": 0, "ademamix": 1, "momentum": 2, "lion": 3, "rmsprop": 4, "adagrad": 5}
TWO_STATE = ("adam", "adamw", "ademamix")
SCALAR_NAMES = ["lr", "b1", "b2", "eps", "wd", "omb1", "omb2", "ic1", "rs2", "decay",
                "b3t", "omb3", "alpha_t", "max_unorm"]


class BitoptError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class HParams(ctypes.Structure):
    """Mirror of bitopt_hparams."""
    _fields_ = [
        ("optimizer", ctypes.c_int32),
        ("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
        ("beta3", ctypes.c_float), ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
        ("alpha", ctypes.c_float),
        ("t_alpha", ctypes.c_int32), ("t_beta3", ctypes.c_int32),
        ("max_unorm", ctypes.c_float),
        ("skip_zeros", ctypes.c_int32),
        ("blocksize", ctypes.c_int32),
    ]


def make_hparams(hp: dict) -> HParams:
    """bitopt_hparams from a dict; missing keys take the Optimizer2State defaults."""
    if isinstance(hp, HParams):
        return hp
    h = HParams()
    h.optimizer = OPTIMIZERS[hp["optimizer"]]
    h.lr = hp.get("lr", 1e-3)
    h.beta1 = hp.get("beta1", 0.9)
    h.beta2 = hp.get("beta2", 0.999)
    h.beta3 = hp.get("beta3", 0.9999)
    h.eps = hp.get("eps", 1e-8)
    h.weight_decay = hp.get("weight_decay", 0.0)
    h.alpha = hp.get("alpha", 0.0)
    h.t_alpha = hp.get("t_alpha") or 0
    h.t_beta3 = hp.get("t_beta3") or 0
    h.max_unorm = hp.get("max_unorm", 0.0)
    h.skip_zeros = 1 if hp.get("skip_zeros", False) else 0
    h.blocksize = hp.get("blocksize", 256)
    return h


class Tensor(ctypes.Structure):
    """Mirror of bitopt_tensor."""
    _fields_ = [
        ("p", ctypes.c_void_p), ("g", ctypes.c_void_p),
        ("state1", ctypes.c_void_p), ("state2", ctypes.c_void_p),
        ("absmax1", ctypes.c_void_p), ("absmax2", ctypes.c_void_p),
        ("n", ctypes.c_int64), ("dtype", ctypes.c_int32), ("is_8bit", ctypes.c_int32),
    ]


class MultiLaunch(ctypes.Structure):
    """Mirror of bitopt_multi_launch."""
    _fields_ = [("kind8", ctypes.c_int32), ("dtype", ctypes.c_int32), ("first", ctypes.c_int32),
                ("count", ctypes.c_int32), ("tiles", ctypes.c_int64)]


MULTI_MAX_LAUNCHES = 64


class MultiPlanC(ctypes.Structure):
    """Mirror of bitopt_multi_plan."""
    _fields_ = [("optimizer", ctypes.c_int32), ("blocksize", ctypes.c_int32), ("count", ctypes.c_int32),
                ("nlaunch", ctypes.c_int32), ("workspace", ctypes.c_void_p),
                ("launch", MultiLaunch * MULTI_MAX_LAUNCHES)]


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                              "or python bit_optimizers_block_amd/build.py")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        HP = ctypes.POINTER(HParams)
        sigs = {
            "bitopt_last_error": ([], ctypes.c_char_p),
            "bitopt_abi_version": ([], i32),
            "bitopt_create_dynamic_map": ([ctypes.c_int, P], ctypes.c_int),
            "bitopt_step_scalars": ([HP, i32, P], ctypes.c_int),
            "bitopt_quantize_blockwise": ([P, i32, i64, P, i32, P, P, P], ctypes.c_int),
            "bitopt_dequantize_blockwise": ([P, P, P, i64, i32, P, i32, P], ctypes.c_int),
            "bitopt_step_8bit_blockwise_2state": ([HP, i32, P, P, i32, i64, P, P, P, P, P, P, P], ctypes.c_int),
            "bitopt_step_8bit_blockwise_1state": ([HP, i32, P, P, i32, i64, P, P, P, P], ctypes.c_int),
            "bitopt_step_32bit_2state": ([HP, i32, P, P, i32, i64, P, P, P], ctypes.c_int),
            "bitopt_step_32bit_1state": ([HP, i32, P, P, i32, i64, P, P], ctypes.c_int),
            "bitopt_multi_workspace_bytes": ([i32], i64),
            "bitopt_tensorwise_workspace_bytes": ([], i64),
            "bitopt_host_state_alloc": ([i64, ctypes.POINTER(ctypes.c_void_p)], ctypes.c_int),
            "bitopt_host_state_free": ([P], ctypes.c_int),
            "bitopt_step_8bit_tensorwise": ([HP, i32, P, P, i32, i64, P, P, P, P, P, P, P, P], ctypes.c_int),
            "bitopt_step_8bit_tensorwise_noalloc": ([HP, i32, P, P, i32, i64, P, P, P, P, P, P, P], ctypes.c_int),
            "bitopt_tensorwise_scratch_bytes": ([], i64),
            "bitopt_paged_staging_bytes": ([HP, i64], i64),
            "bitopt_step_8bit_paged": ([HP, i32, P, P, i32, i64, P, P, P, P, P, P, P, i64, P, P, P], ctypes.c_int),
            "bitopt_page_pool_frame_bytes": ([HP, i64], i64),
            "bitopt_page_pool_create": ([HP, i64, P, i64, ctypes.POINTER(P)], ctypes.c_int),
            "bitopt_page_pool_destroy": ([P], ctypes.c_int),
            "bitopt_step_8bit_pooled": ([P, HP, i32, P, P, i32, i64, P, P, P, P, P, P, P], ctypes.c_int),
            "bitopt_page_pool_flush": ([P, i32, P], ctypes.c_int),
            "bitopt_page_pool_stats": ([P, ctypes.POINTER(i64)], ctypes.c_int),
            "bitopt_step_multi": ([HP, i32, ctypes.POINTER(Tensor), i32, P, P, P, i64, P], ctypes.c_int),
            "bitopt_multi_plan_build": ([HP, ctypes.POINTER(Tensor), i32, P, i64, ctypes.POINTER(MultiPlanC), P],
                                        ctypes.c_int),
            "bitopt_step_multi_planned": ([ctypes.POINTER(MultiPlanC), HP, i32, P, P, P], ctypes.c_int),
            "bitopt_device_scalars_bytes": ([], i64),
            "bitopt_device_scalars_write": ([HP, i32, P, i64], ctypes.c_int),
            "bitopt_mx_code_bytes": ([i64, i32], i64),
            "bitopt_mx_scale_bytes": ([i64], i64),
            "bitopt_mx_quantize": ([P, i32, i64, i64, i64, i32, P, P, P], ctypes.c_int),
            "bitopt_mx_dequantize": ([P, P, i32, i64, i64, P, i32, i64, P], ctypes.c_int),
            "bitopt_mx_matmul": ([P, P, i32, P, P, i32, i64, i64, i64, P, i32, i64, P], ctypes.c_int),
            "bitopt_mx_linear": ([P, i32, i64, P, P, i32, i64, i64, i64, P, i32, i64, P], ctypes.c_int),
            "bitopt_mx_linear_grad_input": ([P, i32, i64, P, P, i32, i64, i64, i64, P, i32, i64, P], ctypes.c_int),
            "bitopt_mx_linear_grad_weight": ([P, i32, i64, P, P, i32, i64, i64, i64, P, i32, i64, i32, P],
                                             ctypes.c_int),
            "bitopt_swiglu_forward_mx8": ([P, P, i32, i64, i64, i64, i64, P, i64, P, P, P, P, P], ctypes.c_int),
            "bitopt_swiglu_backward_mx8": ([P, i32, i64, i64, i64, P, P, P, P, P, i64, P, i64, P], ctypes.c_int),
            "bitopt_step_multi_planned_dscalars": ([ctypes.POINTER(MultiPlanC), HP, P, P, P, P], ctypes.c_int),
        }
        for name, (args, res) in sigs.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def last_error() -> str:
    return lib().bitopt_last_error().decode()


def _check(rc: int):
    if rc != OK:
        raise BitoptError(rc, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# --------------------------------------------------------------- state outside HBM

_host_states = {}     # address -> bytes of live bitopt_host_state_alloc buffers


def _free_host_state(ptr):
    _host_states.pop(ptr, None)
    lib().bitopt_host_state_free(ctypes.c_void_p(ptr))


def host_state(numel: int, dtype=torch.uint8) -> torch.Tensor:
    """A CPU tensor over pinned host memory mapped into the GPU address space
    (bitopt_host_state_alloc): optimizer state kept outside HBM, which every step
    accepts in place of device state.  The memory is freed when the tensor is
    garbage-collected; synchronize the streams that use it before dropping it."""
    import weakref
    import numpy as np
    nbytes = int(numel) * torch.empty(0, dtype=dtype).element_size()
    ptr = ctypes.c_void_p()
    _check(lib().bitopt_host_state_alloc(max(nbytes, 1), ctypes.byref(ptr)))
    buf = (ctypes.c_uint8 * max(nbytes, 1)).from_address(ptr.value)
    arr = np.frombuffer(buf, dtype=np.uint8)[:nbytes]
    _host_states[ptr.value] = max(nbytes, 1)
    weakref.finalize(buf, _free_host_state, ptr.value)
    return torch.from_numpy(arr).view(dtype)


def _is_host_state(t) -> bool:
    a = t.data_ptr()
    return any(p <= a and a + t.numel() * t.element_size() <= p + n for p, n in _host_states.items())


def _need(t, name, dtype=None, numel=None, device=True):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device == "state":
        if not (t.is_cuda or _is_host_state(t)):
            raise ValueError(f"{name} must be a device tensor or a host_state() tensor")
    elif device and not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")


def _dt(t):
    if t.dtype not in DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return DTYPES[t.dtype]


def abi_version() -> int:
    return lib().bitopt_abi_version()


def create_dynamic_map(signed: bool = True) -> torch.Tensor:
    """The 256-entry dynamic-exponent codebook (host fp32 tensor)."""
    out = torch.empty(256, dtype=torch.float32)
    _check(lib().bitopt_create_dynamic_map(1 if signed else 0, _ptr(out)))
    return out


def step_scalars(hp, step: int) -> dict:
    h = make_hparams(hp)
    out = torch.empty(14, dtype=torch.float32)
    _check(lib().bitopt_step_scalars(ctypes.byref(h), int(step), _ptr(out)))
    return dict(zip(SCALAR_NAMES, out.tolist()))


def nblocks(n: int, blocksize: int) -> int:
    return (n + blocksize - 1) // blocksize


def quantize_blockwise(x, qmap, blocksize: int = 256, codes=None, absmax=None, stream=None):
    n = x.numel()
    _need(x, "x"); _need(qmap, "qmap", torch.float32, 256)
    if codes is None:
        codes = torch.empty(n, dtype=torch.uint8, device=x.device)
    if absmax is None:
        absmax = torch.empty(nblocks(n, blocksize), dtype=torch.float32, device=x.device)
    _need(codes, "codes", torch.uint8, n); _need(absmax, "absmax", torch.float32, nblocks(n, blocksize))
    _check(lib().bitopt_quantize_blockwise(_ptr(x), _dt(x), n, _ptr(qmap), blocksize, _ptr(codes),
                                           _ptr(absmax), _stream(stream)))
    return codes, absmax


def dequantize_blockwise(codes, absmax, qmap, blocksize: int = 256, out=None, dtype=torch.float32, stream=None):
    n = codes.numel()
    _need(codes, "codes", torch.uint8); _need(qmap, "qmap", torch.float32, 256)
    _need(absmax, "absmax", torch.float32, nblocks(n, blocksize))
    if out is None:
        out = torch.empty(n, dtype=dtype, device=codes.device)
    _need(out, "out", numel=n)
    _check(lib().bitopt_dequantize_blockwise(_ptr(codes), _ptr(absmax), _ptr(qmap), n, blocksize,
                                             _ptr(out), _dt(out), _stream(stream)))
    return out


def step_8bit_blockwise_2state(hp, step, p, g, state1, state2, absmax1, absmax2, qmap1, qmap2, stream=None):
    h = make_hparams(hp)
    n = p.numel()
    k = 2 if h.optimizer == OPTIMIZERS["ademamix"] else 1
    nb = nblocks(n, h.blocksize)
    _need(p, "p"); _need(g, "g", p.dtype, n)
    _need(state1, "state1", torch.uint8, k * n, device="state"); _need(state2, "state2", torch.uint8, n, device="state")
    _need(absmax1, "absmax1", torch.float32, k * nb, device="state"); _need(absmax2, "absmax2", torch.float32, nb, device="state")
    _need(qmap1, "qmap1", torch.float32, 256); _need(qmap2, "qmap2", torch.float32, 256)
    _check(lib().bitopt_step_8bit_blockwise_2state(ctypes.byref(h), int(step), _ptr(p), _ptr(g), _dt(p), n,
                                                   _ptr(state1), _ptr(state2), _ptr(absmax1), _ptr(absmax2),
                                                   _ptr(qmap1), _ptr(qmap2), _stream(stream)))


def step_8bit_blockwise_1state(hp, step, p, g, state1, absmax1, qmap1, stream=None):
    h = make_hparams(hp)
    n = p.numel()
    _need(p, "p"); _need(g, "g", p.dtype, n)
    _need(state1, "state1", torch.uint8, n, device="state"); _need(absmax1, "absmax1", torch.float32, nblocks(n, h.blocksize), device="state")
    _need(qmap1, "qmap1", torch.float32, 256)
    _check(lib().bitopt_step_8bit_blockwise_1state(ctypes.byref(h), int(step), _ptr(p), _ptr(g), _dt(p), n,
                                                   _ptr(state1), _ptr(absmax1), _ptr(qmap1), _stream(stream)))


def step_32bit_2state(hp, step, p, g, state1, state2, stream=None):
    h = make_hparams(hp)
    n = p.numel()
    k = 2 if h.optimizer == OPTIMIZERS["ademamix"] else 1
    _need(p, "p"); _need(g, "g", p.dtype, n)
    _need(state1, "state1", torch.float32, k * n, device="state"); _need(state2, "state2", torch.float32, n, device="state")
    _check(lib().bitopt_step_32bit_2state(ctypes.byref(h), int(step), _ptr(p), _ptr(g), _dt(p), n,
                                          _ptr(state1), _ptr(state2), _stream(stream)))


def step_32bit_1state(hp, step, p, g, state1, stream=None):
    h = make_hparams(hp)
    n = p.numel()
    _need(p, "p"); _need(g, "g", p.dtype, n); _need(state1, "state1", torch.float32, n, device="state")
    _check(lib().bitopt_step_32bit_1state(ctypes.byref(h), int(step), _ptr(p), _ptr(g), _dt(p), n,
                                          _ptr(state1), _stream(stream)))


def tensorwise_workspace_bytes() -> int:
    return lib().bitopt_tensorwise_workspace_bytes()


def step_8bit_tensorwise(hp, step, p, g, state1, absmax1, qmap1, state2=None, absmax2=None, qmap2=None,
                         workspace=None, stream=None):
    """Non-block-wise 8-bit step (hp blocksize 0): one absmax per state for the whole
    tensor.  Returns the workspace tensor used (pass it back to reuse it)."""
    h = make_hparams(hp)
    n = p.numel()
    k = 2 if h.optimizer == OPTIMIZERS["ademamix"] else 1
    two = h.optimizer in (OPTIMIZERS["adam"], OPTIMIZERS["ademamix"])
    _need(p, "p"); _need(g, "g", p.dtype, n)
    _need(state1, "state1", torch.uint8, k * n, device="state"); _need(absmax1, "absmax1", torch.float32, k, device="state")
    _need(qmap1, "qmap1", torch.float32, 256)
    if two:
        _need(state2, "state2", torch.uint8, n, device="state"); _need(absmax2, "absmax2", torch.float32, 1, device="state")
        _need(qmap2, "qmap2", torch.float32, 256)
    if workspace is None:
        workspace = torch.empty(tensorwise_workspace_bytes(), dtype=torch.uint8, device=p.device)
    _check(lib().bitopt_step_8bit_tensorwise(ctypes.byref(h), int(step), _ptr(p), _ptr(g), _dt(p), n,
                                             _ptr(state1), _ptr(state2), _ptr(absmax1), _ptr(absmax2),
                                             _ptr(qmap1), _ptr(qmap2), _ptr(workspace), _stream(stream)))
    return workspace


def step_8bit_tensorwise_noalloc(hp, step, p, g, state1, absmax1, qmap1, state2=None, absmax2=None, qmap2=None,
                                 stream=None):
    """The tensor-wide step with the library's own scratch array as its workspace
    (no device allocation by the call; calls that overlap on one GPU race)."""
    h = make_hparams(hp)
    n = p.numel()
    k = 2 if h.optimizer == OPTIMIZERS["ademamix"] else 1
    two = h.optimizer in (OPTIMIZERS["adam"], OPTIMIZERS["ademamix"])
    _need(p, "p"); _need(g, "g", p.dtype, n)
    _need(state1, "state1", torch.uint8, k * n, device="state"); _need(absmax1, "absmax1", torch.float32, k, device="state")
    _need(qmap1, "qmap1", torch.float32, 256)
    if two:
        _need(state2, "state2", torch.uint8, n, device="state"); _need(absmax2, "absmax2", torch.float32, 1, device="state")
        _need(qmap2, "qmap2", torch.float32, 256)
    _check(lib().bitopt_step_8bit_tensorwise_noalloc(ctypes.byref(h), int(step), _ptr(p), _ptr(g), _dt(p), n,
                                                     _ptr(state1), _ptr(state2), _ptr(absmax1), _ptr(absmax2),
                                                     _ptr(qmap1), _ptr(qmap2), _stream(stream)))


def paged_staging_bytes(hp, chunk_elems: int) -> int:
    return lib().bitopt_paged_staging_bytes(ctypes.byref(make_hparams(hp)), int(chunk_elems))


def step_8bit_paged(hp, step, p, g, state1, absmax1, qmap1, state2=None, absmax2=None, qmap2=None,
                    staging=None, h2d_stream=None, d2h_stream=None, stream=None):
    """8-bit step with the state in host memory (host_state() tensors), paged through
    a device staging buffer chunk by chunk (bitopt_step_8bit_paged).  h2d_stream and
    d2h_stream: torch streams distinct from the step stream.  Returns the staging
    tensor used (pass it back to reuse it)."""
    h = make_hparams(hp)
    n = p.numel()
    k = 2 if h.optimizer == OPTIMIZERS["ademamix"] else 1
    two = h.optimizer in (OPTIMIZERS["adam"], OPTIMIZERS["ademamix"])
    nb = nblocks(n, h.blocksize)
    _need(p, "p"); _need(g, "g", p.dtype, n)
    for t, name, dt, cnt in ((state1, "state1", torch.uint8, k * n), (absmax1, "absmax1", torch.float32, k * nb)) + (
            ((state2, "state2", torch.uint8, n), (absmax2, "absmax2", torch.float32, nb)) if two else ()):
        _need(t, name, dt, cnt, device=False)
        if t.is_cuda:
            raise ValueError(f"{name} must be host memory (host_state())")
    if staging is None:
        staging = torch.empty(paged_staging_bytes(hp, min(n, 1 << 22)), dtype=torch.uint8, device=p.device)
    if h2d_stream is None or d2h_stream is None:
        raise ValueError("step_8bit_paged needs two copy streams")
    _check(lib().bitopt_step_8bit_paged(ctypes.byref(h), int(step), _ptr(p), _ptr(g), _dt(p), n, _ptr(state1),
                                        _ptr(state2), _ptr(absmax1), _ptr(absmax2), _ptr(qmap1), _ptr(qmap2),
                                        _ptr(staging), staging.numel(), _stream(h2d_stream), _stream(d2h_stream),
                                        _stream(stream)))
    return staging


def page_pool_frame_bytes(hp, page_elems: int) -> int:
    return lib().bitopt_page_pool_frame_bytes(ctypes.byref(make_hparams(hp)), int(page_elems))


class PagePool:
    """An HBM page pool in front of host-resident 8-bit state (bitopt_page_pool_*):
    pages stay in its frames while they fit and are written back and replaced, least
    recently used first, when they do not.  `frames` is a device uint8 tensor (made
    for `nframes` frames when not given); the pool keeps it alive."""

    def __init__(self, hp, page_elems: int, nframes: int = None, frames=None, device="cuda"):
        self.hp = dict(hp)
        fb = page_pool_frame_bytes(hp, page_elems)
        if fb < 0:
            raise ValueError(f"invalid page pool arguments (page_elems={page_elems})")
        if frames is None:
            frames = torch.empty(fb * int(nframes), dtype=torch.uint8, device=device)
        self.frames = frames
        self.page_elems = int(page_elems)
        self.frame_bytes = fb
        h = ctypes.c_void_p()
        _check(lib().bitopt_page_pool_create(ctypes.byref(make_hparams(hp)), self.page_elems, _ptr(frames),
                                             frames.numel() * frames.element_size(), ctypes.byref(h)))
        self._h = h

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("the page pool is closed")
        return self._h

    def step(self, hp, step, p, g, state1, absmax1, qmap1, state2=None, absmax2=None, qmap2=None, stream=None):
        """One 8-bit step on host_state() buffers through the pool."""
        h = make_hparams(hp)
        n = p.numel()
        k = 2 if h.optimizer == OPTIMIZERS["ademamix"] else 1
        two = h.optimizer in (OPTIMIZERS["adam"], OPTIMIZERS["ademamix"])
        nb = nblocks(n, h.blocksize)
        _need(p, "p"); _need(g, "g", p.dtype, n)
        for t, name, dt, cnt in ((state1, "state1", torch.uint8, k * n),
                                 (absmax1, "absmax1", torch.float32, k * nb)) + (
                ((state2, "state2", torch.uint8, n), (absmax2, "absmax2", torch.float32, nb)) if two else ()):
            _need(t, name, dt, cnt, device=False)
            if t.is_cuda:
                raise ValueError(f"{name} must be host memory (host_state())")
        _check(lib().bitopt_step_8bit_pooled(self.handle, ctypes.byref(h), int(step), _ptr(p), _ptr(g), _dt(p), n,
                                             _ptr(state1), _ptr(state2), _ptr(absmax1), _ptr(absmax2), _ptr(qmap1),
                                             _ptr(qmap2), _stream(stream)))

    def flush(self, evict: bool = False, stream=None):
        _check(lib().bitopt_page_pool_flush(self.handle, 1 if evict else 0, _stream(stream)))

    def stats(self) -> dict:
        out = (ctypes.c_int64 * 4)()
        _check(lib().bitopt_page_pool_stats(self.handle, out))
        return dict(resident=out[0], page_ins=out[1], write_backs=out[2], hits=out[3])

    def close(self):
        if self._h is not None:
            h, self._h = self._h, None
            _check(lib().bitopt_page_pool_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def multi_workspace_bytes(count: int) -> int:
    return lib().bitopt_multi_workspace_bytes(int(count))


def _tensor_array(h, tensors):
    """bitopt_tensor descriptors of a list of dicts (keys p, g, state1, state2,
    absmax1, absmax2, is_8bit), with their shapes and dtypes checked."""
    two = h.optimizer in (OPTIMIZERS["adam"], OPTIMIZERS["ademamix"])
    k = 2 if h.optimizer == OPTIMIZERS["ademamix"] else 1
    arr = (Tensor * max(1, len(tensors)))()
    dev = None
    for i, t in enumerate(tensors):
        p, g = t["p"], t["g"]
        n = p.numel()
        nb = nblocks(n, h.blocksize)
        eight = bool(t.get("is_8bit", True))
        _need(p, "p"); _need(g, "g", p.dtype, n)
        sdt = torch.uint8 if eight else torch.float32
        _need(t["state1"], "state1", sdt, k * n, device="state")
        if two:
            _need(t["state2"], "state2", sdt, n, device="state")
        if eight:
            _need(t["absmax1"], "absmax1", torch.float32, k * nb, device="state")
            if two:
                _need(t["absmax2"], "absmax2", torch.float32, nb, device="state")
        arr[i] = Tensor(p.data_ptr(), g.data_ptr(), t["state1"].data_ptr(),
                        t["state2"].data_ptr() if two else None,
                        t["absmax1"].data_ptr() if eight else None,
                        t["absmax2"].data_ptr() if (eight and two) else None,
                        n, _dt(p), 1 if eight else 0)
        dev = p.device
    return arr, dev


class MultiPlan:
    """A built multi-tensor plan (bitopt_multi_plan_build): the host struct, its device
    workspace, and references to the tensors it names (kept alive with it)."""

    def __init__(self, hp, tensors, workspace=None, stream=None):
        h = make_hparams(hp)
        arr, dev = _tensor_array(h, tensors)
        need = multi_workspace_bytes(len(tensors))
        if workspace is None or workspace.numel() < need:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        self.c = MultiPlanC()
        self.workspace = workspace
        self.tensors = list(tensors)
        _check(lib().bitopt_multi_plan_build(ctypes.byref(h), arr, len(tensors), _ptr(workspace),
                                             workspace.numel(), ctypes.byref(self.c), _stream(stream)))

    def step(self, hp, step, qmap1=None, qmap2=None, stream=None):
        h = make_hparams(hp)
        _check(lib().bitopt_step_multi_planned(ctypes.byref(self.c), ctypes.byref(h), int(step), _ptr(qmap1),
                                               _ptr(qmap2), _stream(stream)))

    def step_dscalars(self, hp, scalars, qmap1=None, qmap2=None, stream=None):
        """The planned step with its per-step scalars read from `scalars` (a device
        uint8 tensor of device_scalars_bytes() bytes, see device_scalars) when the
        kernels run: a captured graph of this call steps with the buffer's contents
        at each replay."""
        h = make_hparams(hp)
        _need(scalars, "scalars", torch.uint8)
        if scalars.numel() < device_scalars_bytes():
            raise ValueError("scalars is too small")
        _check(lib().bitopt_step_multi_planned_dscalars(ctypes.byref(self.c), ctypes.byref(h), _ptr(scalars),
                                                        _ptr(qmap1), _ptr(qmap2), _stream(stream)))


def device_scalars_bytes() -> int:
    return int(lib().bitopt_device_scalars_bytes())


def device_scalars(hp, step) -> torch.Tensor:
    """The per-step scalars of (hp, step) in the kernels' device layout, as a CPU uint8
    tensor (copy it into the device buffer that step_dscalars reads)."""
    out = torch.empty(device_scalars_bytes(), dtype=torch.uint8)
    _check(lib().bitopt_device_scalars_write(ctypes.byref(make_hparams(hp)), int(step), _ptr(out), out.numel()))
    return out


def step_multi(hp, step, tensors, qmap1=None, qmap2=None, workspace=None, stream=None):
    """One step over many tensors (plan and step in one call; it waits for the
    descriptor copy -- a training loop builds a MultiPlan once instead).  `tensors`:
    list of dicts with keys p, g, state1, state2, absmax1, absmax2 (torch tensors or
    None) and is_8bit (bool).  Returns the workspace tensor used (pass it back to
    reuse it)."""
    h = make_hparams(hp)
    arr, dev = _tensor_array(h, tensors)
    need = multi_workspace_bytes(len(tensors))
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    _check(lib().bitopt_step_multi(ctypes.byref(h), int(step), arr, len(tensors), _ptr(qmap1), _ptr(qmap2),
                                   _ptr(workspace), workspace.numel(), _stream(stream)))
    return workspace


# ------------------------------------------------------------------- MX matrices
#
# These calls run once per layer and token, so a call on the current device and stream
# takes the short way: each argument is looked at once, and the stream's handle is read
# without building a stream object.
#
# They record nothing for automatic differentiation, whether or not an argument requires a
# gradient: results are new tensors without a history (or the caller's own).  Gradients come
# from the calls for them, mx_linear_grad_input, mx_linear_grad_weight and swiglu_backward8,
# which a torch.autograd.Function of the caller's may wrap; quantization has none.

MX_FORMATS = {"e2m1": 0, "e4m3": 1}


def mx_code_bytes(cols: int, fmt: str = "e2m1") -> int:
    """Bytes of codes in one row of an MX matrix: rows are padded to 128 elements."""
    return (cols + 127) // 128 * (128 if _mx_format(fmt) else 64)


def mx_scale_bytes(cols: int) -> int:
    """Scale bytes in one row of an MX matrix."""
    return (cols + 127) // 128 * 4


def _mx_format(fmt):
    f = MX_FORMATS.get(fmt)
    if f is None:
        raise ValueError(f"unknown MX format {fmt!r} (one of {sorted(MX_FORMATS)})")
    return f


def _rows(t, name, device=None):
    """A device matrix with contiguous rows: (rows, columns, distance of rows in elements)."""
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, other arguments on {device}")
    rows, cols = t.shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous (strides {(ld, one)})")
    if rows > 1:
        if ld < cols:
            raise ValueError(f"{name}: its rows overlap (strides {(ld, one)})")
        return rows, cols, ld
    return rows, cols, cols


def _mx_bytes(t, rows, width, name, cols, fmt, device):
    if t.dtype is not torch.uint8:
        raise TypeError(f"{name}: expected torch.uint8, got {t.dtype}")
    if t.shape != (rows, width) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous matrix of {width} bytes a row for {cols} {fmt} columns and as "
                         f"many rows of codes as of scales, got shape {tuple(t.shape)}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be on {device}" if device.type == "cuda" else f"{name} must be a device tensor")


def _mx_operand(codes, scales, cols, fmt, name, device):
    """Checks an MX matrix of `cols` columns; returns its format and rows."""
    f = MX_FORMATS.get(fmt)
    if f is None:
        _mx_format(fmt)
    pads = (cols + 127) // 128
    rows = codes.size(0) if codes.dim() == 2 else -1
    _mx_bytes(codes, rows, pads * (128 if f else 64), name + " codes", cols, fmt, device)
    _mx_bytes(scales, rows, pads * 4, name + " scales", cols, fmt, device)
    return f, rows


def _elsewhere(device, stream):
    """None when work on `device` belongs on its current stream and it is the current device.
    Otherwise a context that makes `device` (and `stream`, if given) current: results allocated
    inside then belong to the stream that writes them."""
    if stream is None:
        return None if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):       # any object with a stream's handle
        handle = int(stream.cuda_stream or 0)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the arguments on {device}")
    return torch.cuda.stream(stream)


def _current(device):
    """Handle of the current stream of `device`."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _mx_result(out, rows, cols, dtype, device, name):
    if out is None:
        if dtype not in DTYPES:
            raise TypeError(f"unsupported dtype {dtype}")
        return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device), cols
    if out.shape != (rows, cols):
        raise ValueError(f"{name}: expected shape {(rows, cols)}, got {tuple(out.shape)}")
    return out, _rows(out, name, device)[2]


def _mx_new(codes, scales, rows, cols, fmt, device, name):
    """Result codes and scales: allocated, or the caller's, checked."""
    f, pads = _mx_format(fmt), (cols + 127) // 128
    if codes is None:
        width = pads * (128 if f else 64)
        codes = torch.empty_strided((rows, width), (width, 1), dtype=torch.uint8, device=device)
        if scales is None:
            return codes, torch.empty_strided((rows, pads * 4), (pads * 4, 1), dtype=torch.uint8, device=device), f
    if scales is None:
        scales = torch.empty((rows, pads * 4), dtype=torch.uint8, device=device)
    if _mx_operand(codes, scales, cols, fmt, name, device)[1] != rows:
        raise ValueError(f"{name}: expected {rows} rows of codes, got {codes.size(0)}")
    return codes, scales, f


def mx_quantize(x, fmt: str = "e2m1", codes=None, scales=None, stream=None):
    """The MX form of a matrix: (codes, scales), blocks of 32 along its rows."""
    rows, cols, ldx = _rows(x, "x")
    dt, device = _dt(x), x.device
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return mx_quantize(x, fmt, codes, scales)
    codes, scales, f = _mx_new(codes, scales, rows, cols, fmt, device, "the result")
    _check(lib().bitopt_mx_quantize(x.data_ptr(), dt, rows, cols, ldx, f, codes.data_ptr(), scales.data_ptr(),
                                    _current(device)))
    return codes, scales


def mx_dequantize(codes, scales, cols: int, fmt: str = "e2m1", out=None, dtype=torch.float32, stream=None):
    """The values of an MX matrix of `cols` columns."""
    device = codes.device
    f, rows = _mx_operand(codes, scales, cols, fmt, "the input", device)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return mx_dequantize(codes, scales, cols, fmt, out, dtype)
    out, ldo = _mx_result(out, rows, cols, dtype, device, "out")
    _check(lib().bitopt_mx_dequantize(codes.data_ptr(), scales.data_ptr(), f, rows, cols, out.data_ptr(), _dt(out), ldo,
                                      _current(device)))
    return out


def mx_matmul(a_codes, a_scales, b_codes, b_scales, k: int, a_fmt: str = "e2m1", b_fmt: str = "e2m1", out=None,
              dtype=torch.bfloat16, stream=None):
    """a b^T for MX matrices a (m x k) and b (n x k)."""
    device = a_codes.device
    fa, m = _mx_operand(a_codes, a_scales, k, a_fmt, "a", device)
    fb, n = _mx_operand(b_codes, b_scales, k, b_fmt, "b", device)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return mx_matmul(a_codes, a_scales, b_codes, b_scales, k, a_fmt, b_fmt, out, dtype)
    out, ldo = _mx_result(out, m, n, dtype, device, "out")
    _check(lib().bitopt_mx_matmul(a_codes.data_ptr(), a_scales.data_ptr(), fa, b_codes.data_ptr(), b_scales.data_ptr(),
                                  fb, m, n, k, out.data_ptr(), _dt(out), ldo, _current(device)))
    return out


def mx_linear(x, w_codes, w_scales, fmt: str = "e2m1", out=None, dtype=None, stream=None):
    """x W^T for a 16-bit x (tokens x k) and MX weights W (n x k); dtype defaults to x's."""
    tokens, k, ldx = _rows(x, "x")
    dt, device = _dt(x), x.device
    f, n = _mx_operand(w_codes, w_scales, k, fmt, "w", device)
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return mx_linear(x, w_codes, w_scales, fmt, out, dtype)
    out, ldo = _mx_result(out, tokens, n, dtype or x.dtype, device, "out")
    _check(lib().bitopt_mx_linear(x.data_ptr(), dt, ldx, w_codes.data_ptr(), w_scales.data_ptr(), f, tokens, n, k,
                                  out.data_ptr(), _dt(out), ldo, _current(device)))
    return out


def mx_linear_grad_input(dy, w_codes, w_scales, k: int, fmt: str = "e2m1", out=None, dtype=None, stream=None):
    """dy W: the gradient of mx_linear's x from dy (tokens x n); dtype defaults to dy's."""
    tokens, n, lddy = _rows(dy, "dy")
    dt, device = _dt(dy), dy.device
    f, rows = _mx_operand(w_codes, w_scales, k, fmt, "w", device)
    if rows != n:
        raise ValueError(f"dy has {n} columns, w {rows} rows")
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return mx_linear_grad_input(dy, w_codes, w_scales, k, fmt, out, dtype)
    out, ldo = _mx_result(out, tokens, k, dtype or dy.dtype, device, "out")
    _check(lib().bitopt_mx_linear_grad_input(dy.data_ptr(), dt, lddy, w_codes.data_ptr(), w_scales.data_ptr(), f,
                                             tokens, n, k, out.data_ptr(), _dt(out), ldo, _current(device)))
    return out


def mx_linear_grad_weight(dy, x_codes, x_scales, k: int, fmt: str = "e4m3", out=None, dtype=torch.float32,
                          accumulate: bool = False, stream=None):
    """dy^T x: the gradient of mx_linear's weights (n x k) from dy (tokens x n) and the
    input kept as an MX matrix (tokens x k); `accumulate` adds it to `out`."""
    tokens, n, lddy = _rows(dy, "dy")
    dt, device = _dt(dy), dy.device
    f, rows = _mx_operand(x_codes, x_scales, k, fmt, "x", device)
    if rows != tokens:
        raise ValueError(f"dy has {tokens} rows, x {rows}")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return mx_linear_grad_weight(dy, x_codes, x_scales, k, fmt, out, dtype, accumulate)
    out, ldo = _mx_result(out, n, k, dtype, device, "out")
    _check(lib().bitopt_mx_linear_grad_weight(dy.data_ptr(), dt, lddy, x_codes.data_ptr(), x_scales.data_ptr(), f,
                                              tokens, n, k, out.data_ptr(), _dt(out), ldo, 1 if accumulate else 0,
                                              _current(device)))
    return out


def swiglu_save8(gate, up, y=None, saved=None, stream=None):
    """gate * sigmoid(gate) * up, and its inputs in 8 bits for swiglu_backward8: (y, saved),
    saved = (gate_codes, gate_scales, up_codes, up_scales) in MX E4M3.  y may be gate or up."""
    rows, cols, ldg = _rows(gate, "gate")
    dt, device, dtype = _dt(gate), gate.device, gate.dtype
    urows, ucols, ldu = _rows(up, "up", device)
    if (urows, ucols) != (rows, cols) or up.dtype != dtype:
        raise ValueError("gate and up must have one shape and type")
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return swiglu_save8(gate, up, y, saved)
    y, ldy = _mx_result(y, rows, cols, dtype, device, "y")
    if y.dtype != dtype:
        raise TypeError(f"y: expected {dtype}, got {y.dtype}")
    gc, gs, uc, us = saved if saved is not None else (None, None, None, None)
    gc, gs, _ = _mx_new(gc, gs, rows, cols, "e4m3", device, "saved gate")
    uc, us, _ = _mx_new(uc, us, rows, cols, "e4m3", device, "saved up")
    _check(lib().bitopt_swiglu_forward_mx8(gate.data_ptr(), up.data_ptr(), dt, rows, cols, ldg, ldu, y.data_ptr(), ldy,
                                           gc.data_ptr(), gs.data_ptr(), uc.data_ptr(), us.data_ptr(), _current(device)))
    return y, (gc, gs, uc, us)


def swiglu_backward8(dy, saved, dgate=None, dup=None, stream=None):
    """(dgate, dup) of swiglu_save8 from dy and what it saved.  dgate or dup may be dy."""
    rows, cols, lddy = _rows(dy, "dy")
    dt, device, dtype = _dt(dy), dy.device, dy.dtype
    gc, gs, uc, us = saved
    if _mx_operand(gc, gs, cols, "e4m3", "saved gate", device)[1] != rows or \
            _mx_operand(uc, us, cols, "e4m3", "saved up", device)[1] != rows:
        raise ValueError(f"what was saved does not have dy's {rows} rows")
    other = _elsewhere(device, stream)
    if other is not None:
        with other:
            return swiglu_backward8(dy, saved, dgate, dup)
    dgate, lddg = _mx_result(dgate, rows, cols, dtype, device, "dgate")
    dup, lddu = _mx_result(dup, rows, cols, dtype, device, "dup")
    if dgate.dtype != dtype or dup.dtype != dtype:
        raise TypeError(f"dgate and dup must be {dtype}")
    _check(lib().bitopt_swiglu_backward_mx8(dy.data_ptr(), dt, rows, cols, lddy, gc.data_ptr(), gs.data_ptr(),
                                            uc.data_ptr(), us.data_ptr(), dgate.data_ptr(), lddg, dup.data_ptr(), lddu,
                                            _current(device)))
    return dgate, dup
