"""Python binding of libflashbob (argument marshalling only).

The functions carry the C names of ``include/flashbob.h``.  Tensors are
PyTorch CUDA tensors used only as device memory; every step of the
computation runs in the library's kernels.  Loading fails loudly when the
library has not been built: there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

torch = None  # bound by _ready(): building and loading the library need no torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libflashbob.so")

FLASHBOB_OK = 0
FLASHBOB_ERR_INVALID_ARG = 1
FLASHBOB_ERR_UNSUPPORTED = 2
FLASHBOB_ERR_MISALIGNED = 3
FLASHBOB_ERR_CUDA = 4
FLASHBOB_ERR_TIMEOUT = 5
FLASHBOB_F32 = 0
FLASHBOB_BF16 = 1

# Every entry point the header declares, with its ctypes signature.
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SIGNATURES = {
    "flashbob_prep": ([_P] * 7 + [_I] * 6 + [_F, _I, _I, _P], _I),
    "flashbob_bob": ([_P] * 10 + [_F] + [_P] * 6 + [_I] * 8 + [_P], _I),
    "flashbob_bob_pass1": ([_P] * 10 + [_F] + [_P] * 4 + [_I] * 8 + [_P], _I),
    "flashbob_bob_pass2": ([_P] * 11 + [_F] + [_P] * 2 + [_I] * 8 + [_P], _I),
    "flashbob_attention_jvp": ([_P] * 8 + [_F] + [_P] * 2 + [_I] * 8 + [_P], _I),
    "flashbob_attention_workspace": ([_I] * 7 + [ctypes.POINTER(ctypes.c_size_t)] * 2, _I),
    "flashbob_attention": ([_P] * 6 + [_F, _F] + [_P] * 3 + [ctypes.c_size_t] + [_I] * 8 + [_P],
                           _I),
    "flashbob_attention_grad": ([_P] * 9 + [_F, _F] + [_P] * 4 + [ctypes.c_size_t] + [_I] * 8
                                + [_P], _I),
    "flashbob_attention_ranges": ([_P] * 5 + [_I] * 5 + [_P], _I),
    "flashbob_qk_norm_rope": ([_P] * 6 + [_F] + [_P] * 3 + [_I] * 10 + [_P], _I),
    "flashbob_qk_norm_rope_workspace": ([_I] * 6 + [ctypes.POINTER(ctypes.c_size_t)], _I),
    "flashbob_qk_norm_rope_grad": ([_P] * 5 + [_F] + [_P] * 7 + [ctypes.c_size_t] + [_I] * 10
                                   + [_P], _I),
    "flashbob_bob_launches": ([_I] * 7 + [ctypes.POINTER(_I)], _I),
    "flashbob_bob_tile_sizes": ([_I, _I] + [ctypes.POINTER(_I)] * 4
                                + [ctypes.POINTER(ctypes.c_size_t)] * 2, _I),
    "flashbob_last_device_error": ([], _I),
    "flashbob_check_wait_timeout": ([_P], _I),
    "flashbob_mma_cycles": ([_I, _I, _P, ctypes.POINTER(ctypes.c_double)], _I),
    "flashbob_status_string": ([_I], ctypes.c_char_p),
}

_lib = None


class FlashbobError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {flashbob_status_string(status)}")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libflashbob.so (once) and declare the signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with exact_second_order_gb300.build.build()")
    lib = ctypes.CDLL(path)
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


_bound = None  # the library, once torch is bound too


def _ready() -> ctypes.CDLL:
    """load_library() for the calls that work on tensors at once."""
    global torch, _bound
    import torch as module
    torch = module
    _bound = load_library()
    return _bound


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return FLASHBOB_F32
    if t.dtype == torch.bfloat16:
        return FLASHBOB_BF16
    raise TypeError(f"unsupported input dtype {t.dtype}")


def _stream_handle(stream) -> int | None:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _check(where: str, Q, K, spec) -> None:
    """The C ABI sees only pointers and sizes, so the binding checks what the
    header fixes for each tensor before handing its pointer on: a CUDA tensor
    on Q's device, contiguous (row-major), with the shape and dtype of its
    role.  ``spec`` lists (name, tensor, role, dtype) with role "q"
    ([B, H, N_q, d]), "k" ([B, H_kv, N_k, d]) or "row" ([B, H, N_q]) and
    dtype "in" (the inputs' common dtype, Q's) or "f32"; None tensors are
    skipped (the ABI decides which may be NULL)."""
    import torch
    for name, t in (("Q", Q), ("K", K)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{where}: {name} must be a 4-d tensor [B, heads, rows, d]")
    B, H, Nq, d = Q.shape
    Hkv, Nk = K.shape[1], K.shape[2]
    shapes = {"q": (B, H, Nq, d), "k": (B, Hkv, Nk, d), "row": (B, H, Nq)}
    for name, t, role, dt in spec:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != Q.device:
            raise ValueError(f"{where}: {name} must be a CUDA tensor on {Q.device}")
        if tuple(t.shape) != shapes[role]:
            raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, "
                             f"expected {shapes[role]}")
        want = Q.dtype if dt == "in" else torch.float32
        if t.dtype != want:
            raise TypeError(f"{where}: {name} is {t.dtype}, expected {want}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous")


def _input_specs(Q, K, V, dO, UQ, UK, UV):
    """Check list of the seven inputs of the BoB calls (one common dtype)."""
    return [("Q", Q, "q", "in"), ("K", K, "k", "in"), ("V", V, "k", "in"),
            ("dO", dO, "q", "in"), ("UQ", UQ, "q", "in"), ("UK", UK, "k", "in"),
            ("UV", UV, "k", "in")]


def _device(t):
    """The CUDA device context of tensor ``t``: the library works on the
    current device, so every call runs with its tensors' device current."""
    import torch
    return torch.cuda.device(t.device)


def flashbob_status_string(status: int) -> str:
    return load_library().flashbob_status_string(status).decode()


def flashbob_prep(Q, K, V, dO, O, L, D, tau: float, causal: bool = False, stream=None) -> None:
    """O, L, D of [B, H, Nq, d] queries and [B, Hkv, Nk, d] keys/values
    (see flashbob_prep in the header); dO = D = None computes O and L only."""
    _check("flashbob_prep", Q, K, [("Q", Q, "q", "in"), ("K", K, "k", "in"),
                                    ("V", V, "k", "in"), ("dO", dO, "q", "in"),
                                    ("O", O, "q", "f32"), ("L", L, "row", "f32"),
                                    ("D", D, "row", "f32")])
    B, H, Nq, d = Q.shape
    Hkv, Nk = K.shape[1], K.shape[2]
    with _device(Q):
        st = load_library().flashbob_prep(
            _ptr(Q), _ptr(K), _ptr(V), _ptr(dO), _ptr(O), _ptr(L), _ptr(D), B, H, Hkv, Nq, Nk,
            d, float(tau), int(causal), _dtype_code(Q), _stream_handle(stream))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_prep")


def flashbob_bob(Q, K, V, O, dO, L, D, UQ, UK, UV, tau: float, dQt, dKt, dVt, ddOt, alpha, E,
                 causal: bool = False, stream=None) -> None:
    """d~Q, d~K, d~V, d~dO, alpha, E (see flashbob_bob in the header)."""
    _check("flashbob_bob", Q, K, _input_specs(Q, K, V, dO, UQ, UK, UV) + [
        ("O", O, "q", "f32"), ("L", L, "row", "f32"), ("D", D, "row", "f32"),
        ("dQt", dQt, "q", "f32"), ("dKt", dKt, "k", "f32"), ("dVt", dVt, "k", "f32"),
        ("ddOt", ddOt, "q", "f32"), ("alpha", alpha, "row", "f32"), ("E", E, "row", "f32")])
    B, H, Nq, d = Q.shape
    Hkv, Nk = K.shape[1], K.shape[2]
    with _device(Q):
        st = load_library().flashbob_bob(
            _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(L), _ptr(D), _ptr(UQ),
            _ptr(UK), _ptr(UV), float(tau), _ptr(dQt), _ptr(dKt), _ptr(dVt), _ptr(ddOt),
            _ptr(alpha), _ptr(E), B, H, Hkv, Nq, Nk, d, int(causal), _dtype_code(Q),
            _stream_handle(stream))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_bob")


def flashbob_bob_pass1(Q, K, V, O, dO, L, D, UQ, UK, UV, tau: float, dQt, ddOt, alpha, E,
                       causal: bool = False, stream=None) -> None:
    """Pass 1 only: d~Q, d~dO, alpha, E (see flashbob_bob_pass1 in the header)."""
    _check("flashbob_bob_pass1", Q, K, _input_specs(Q, K, V, dO, UQ, UK, UV) + [
        ("O", O, "q", "f32"), ("L", L, "row", "f32"), ("D", D, "row", "f32"),
        ("dQt", dQt, "q", "f32"), ("ddOt", ddOt, "q", "f32"), ("alpha", alpha, "row", "f32"),
        ("E", E, "row", "f32")])
    B, H, Nq, d = Q.shape
    Hkv, Nk = K.shape[1], K.shape[2]
    with _device(Q):
        st = load_library().flashbob_bob_pass1(
            _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(L), _ptr(D), _ptr(UQ),
            _ptr(UK), _ptr(UV), float(tau), _ptr(dQt), _ptr(ddOt), _ptr(alpha), _ptr(E), B, H,
            Hkv, Nq, Nk, d, int(causal), _dtype_code(Q), _stream_handle(stream))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_bob_pass1")


def flashbob_bob_pass2(Q, K, V, dO, L, D, alpha, E, UQ, UK, UV, tau: float, dKt, dVt,
                       causal: bool = False, stream=None) -> None:
    """Pass 2 only: d~K, d~V from pass 1's alpha, E (see flashbob_bob_pass2)."""
    _check("flashbob_bob_pass2", Q, K, _input_specs(Q, K, V, dO, UQ, UK, UV) + [
        ("L", L, "row", "f32"), ("D", D, "row", "f32"), ("alpha", alpha, "row", "f32"),
        ("E", E, "row", "f32"), ("dKt", dKt, "k", "f32"), ("dVt", dVt, "k", "f32")])
    B, H, Nq, d = Q.shape
    Hkv, Nk = K.shape[1], K.shape[2]
    with _device(Q):
        st = load_library().flashbob_bob_pass2(
            _ptr(Q), _ptr(K), _ptr(V), _ptr(dO), _ptr(L), _ptr(D), _ptr(alpha), _ptr(E),
            _ptr(UQ), _ptr(UK), _ptr(UV), float(tau), _ptr(dKt), _ptr(dVt), B, H, Hkv, Nq, Nk,
            d, int(causal), _dtype_code(Q), _stream_handle(stream))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_bob_pass2")


def flashbob_attention_jvp(Q, K, V, O, L, UQ, UK, UV, tau: float, Od, Ld,
                           causal: bool = False, stream=None) -> None:
    """O' and L' along the tangents (U_Q, U_K, U_V) (see flashbob_attention_jvp)."""
    _check("flashbob_attention_jvp", Q, K, [
        ("Q", Q, "q", "in"), ("K", K, "k", "in"), ("V", V, "k", "in"), ("UQ", UQ, "q", "in"),
        ("UK", UK, "k", "in"), ("UV", UV, "k", "in"), ("O", O, "q", "f32"),
        ("L", L, "row", "f32"), ("Od", Od, "q", "f32"), ("Ld", Ld, "row", "f32")])
    B, H, Nq, d = Q.shape
    Hkv, Nk = K.shape[1], K.shape[2]
    with _device(Q):
        st = load_library().flashbob_attention_jvp(
            _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(L), _ptr(UQ), _ptr(UK), _ptr(UV),
            float(tau), _ptr(Od), _ptr(Ld), B, H, Hkv, Nq, Nk, d, int(causal), _dtype_code(Q),
            _stream_handle(stream))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_attention_jvp")


# ---------------------------------------------------------------------------
# The operators around an attention layer.  Their calls are short (a token of
# one request is ten microseconds of GPU time), so the checks ask a tensor each
# thing once and the contexts are entered only where they change something.
# ---------------------------------------------------------------------------

def _cuda_index(where: str, name: str, t, shape_text: str, dims: int) -> int:
    """The CUDA device of the tensor that fixes a call's sizes."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != dims:
        raise ValueError(f"{where}: {name} must be a {dims}-d CUDA tensor {shape_text}")
    return t.get_device()


def _check_tensor(where: str, name: str, t, shape, dtype, index: int) -> None:
    """One tensor of a call: contiguous, on CUDA device ``index``, with the
    shape and dtype of its role."""
    try:
        if (t.get_device() == index and t.shape == shape and t.dtype is dtype
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{where}: {name} must be a CUDA tensor on cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{where}: {name} is {t.dtype}, expected {dtype}")
    raise ValueError(f"{where}: {name} must be contiguous")


def _check_sizes(where: str, *sizes: int) -> None:
    """The C ABI takes sizes as int, and ctypes keeps the low 32 bits of a
    larger one without a word."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"{where}: sizes must be below 2^31, got {max(sizes)}")


def _check_workspace(where: str, t, index: int) -> None:
    if t is not None and not (isinstance(t, torch.Tensor) and t.is_cuda
                              and t.get_device() == index and t.is_contiguous()):
        raise ValueError(f"{where}: workspace must be a contiguous CUDA tensor on cuda:{index}")


def _torch_stream(index: int, stream):
    """The torch stream of a stream argument: a torch stream or a handle, 0 for
    the default stream (torch's ExternalStream would take a stream of its pool
    for 0)."""
    device = getattr(stream, "device", None)
    if device is not None and device.index != index:
        raise ValueError(f"the stream is on {device}, the tensors are on cuda:{index}")
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(getattr(stream, "cuda_stream", stream))
    if handle == 0:
        return torch.cuda.default_stream(index)
    return torch.cuda.ExternalStream(handle, device=index)


@contextlib.contextmanager
def _entered(index: int, stream):
    with torch.cuda.device(index):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(_torch_stream(index, stream)):
                yield


def _elsewhere(index: int, stream):
    """None when CUDA device ``index`` and its current stream are what a call
    works on; else the context that makes them so.  What a wrapper allocates
    and frees inside (a workspace) is then reused in that stream's order."""
    if stream is None and torch._C._cuda_getDevice() == index:
        return None
    return _entered(index, stream)


def _raw_stream(index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index)


def _bytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _check_attention(where: str, Q, K, V, slopes, ranges, q_pos):
    """Checks of the inputs that the attention calls with key ranges share;
    returns the device, the sizes and the dtype code."""
    index = _cuda_index(where, "Q", Q, "[B, H, Nq, d]", 4)
    _cuda_index(where, "K", K, "[B, Hkv, Nk, d]", 4)
    dt = Q.dtype
    B, H, Nq, d = Q.shape
    _, Hkv, Nk, _ = key = K.shape
    if key[0] != B or key[3] != d:
        raise ValueError(f"{where}: K has shape {tuple(key)}, expected {(B, Hkv, Nk, d)}")
    _check_sizes(where, B, H, Hkv, Nq, Nk)
    _check_tensor(where, "Q", Q, Q.shape, dt, index)
    _check_tensor(where, "K", K, key, dt, index)
    _check_tensor(where, "V", V, key, dt, index)
    if slopes is not None:
        _check_tensor(where, "slopes", slopes, (H,), torch.float32, index)
    if ranges is not None:
        _check_tensor(where, "ranges", ranges, (B, Nq, 2), torch.int32, index)
    if q_pos is not None:
        _check_tensor(where, "q_pos", q_pos, (B, Nq), torch.int32, index)
    return index, (B, H, Hkv, Nq, Nk, d), _dtype_code(Q)


@functools.lru_cache(maxsize=256)
def flashbob_attention_workspace(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int,
                                 in_dtype: int) -> tuple[int, int]:
    """Workspace bytes of flashbob_attention and of flashbob_attention_grad."""
    _check_sizes("flashbob_attention_workspace", B, H, Hkv, Nq, Nk, d)
    n = [ctypes.c_size_t() for _ in range(2)]
    st = load_library().flashbob_attention_workspace(B, H, Hkv, Nq, Nk, d, in_dtype,
                                                     *(ctypes.byref(x) for x in n))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_attention_workspace")
    return n[0].value, n[1].value


def _run_attention(lib, index, sizes, code, Q, K, V, ranges, q_pos, slopes, tau, cap, O, L,
                   workspace, causal) -> None:
    st = lib.flashbob_attention(
        Q.data_ptr(), K.data_ptr(), V.data_ptr(), _ptr(ranges), _ptr(q_pos), _ptr(slopes),
        float(tau), float(cap), O.data_ptr(), L.data_ptr(), _ptr(workspace), _bytes(workspace),
        *sizes, int(causal), code, _raw_stream(index))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_attention")


def flashbob_attention(Q, K, V, ranges, q_pos, slopes, tau: float, cap: float, O, L, workspace,
                       causal: bool = False, stream=None) -> None:
    """O, L of attention with key ranges (see flashbob_attention in the header);
    ``workspace`` is any contiguous CUDA tensor of enough bytes, or None."""
    lib, where = _bound or _ready(), "flashbob_attention"
    index, sizes, code = _check_attention(where, Q, K, V, slopes, ranges, q_pos)
    _check_tensor(where, "O", O, Q.shape, Q.dtype, index)
    _check_tensor(where, "L", L, Q.shape[:3], torch.float32, index)
    _check_workspace(where, workspace, index)
    with _elsewhere(index, stream) or contextlib.nullcontext():
        _run_attention(lib, index, sizes, code, Q, K, V, ranges, q_pos, slopes, tau, cap, O, L,
                       workspace, causal)


def attention(Q, K, V, tau: float, cap: float = 0.0, slopes=None, ranges=None, q_pos=None,
              causal: bool = False, stream=None):
    """O (of Q's dtype) and L of attention with capped scores, a distance bias
    and key ranges; allocates them, and the workspace, on Q's device."""
    lib = _bound or _ready()
    index, sizes, code = _check_attention("attention", Q, K, V, slopes, ranges, q_pos)
    need = flashbob_attention_workspace(*sizes, code)[0]

    def run():
        O = torch.empty_like(Q)
        L = torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device)
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device) if need else None
        _run_attention(lib, index, sizes, code, Q, K, V, ranges, q_pos, slopes, tau, cap, O, L,
                       workspace, causal)
        return O, L

    context = _elsewhere(index, stream)
    if context is None:
        return run()
    with context:
        return run()


def _check_attention_grad(where: str, Q, K, V, O, L, dO, slopes, ranges, q_pos):
    checked = _check_attention(where, Q, K, V, slopes, ranges, q_pos)
    _check_tensor(where, "O", O, Q.shape, Q.dtype, checked[0])
    _check_tensor(where, "L", L, Q.shape[:3], torch.float32, checked[0])
    _check_tensor(where, "dO", dO, Q.shape, Q.dtype, checked[0])
    return checked


def _run_attention_grad(lib, index, sizes, code, Q, K, V, O, L, dO, ranges, q_pos, slopes, tau,
                        cap, dQ, dK, dV, workspace, causal) -> None:
    st = lib.flashbob_attention_grad(
        Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), L.data_ptr(), dO.data_ptr(),
        _ptr(ranges), _ptr(q_pos), _ptr(slopes), float(tau), float(cap), dQ.data_ptr(),
        dK.data_ptr(), dV.data_ptr(), _ptr(workspace), _bytes(workspace), *sizes, int(causal), code,
        _raw_stream(index))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_attention_grad")


def flashbob_attention_grad(Q, K, V, O, L, dO, ranges, q_pos, slopes, tau: float, cap: float,
                            dQ, dK, dV, workspace, causal: bool = False, stream=None) -> None:
    """dQ, dK, dV of attention with key ranges (see flashbob_attention_grad)."""
    lib, where = _bound or _ready(), "flashbob_attention_grad"
    index, sizes, code = _check_attention_grad(where, Q, K, V, O, L, dO, slopes, ranges, q_pos)
    _check_tensor(where, "dQ", dQ, Q.shape, Q.dtype, index)
    _check_tensor(where, "dK", dK, K.shape, Q.dtype, index)
    _check_tensor(where, "dV", dV, K.shape, Q.dtype, index)
    _check_workspace(where, workspace, index)
    with _elsewhere(index, stream) or contextlib.nullcontext():
        _run_attention_grad(lib, index, sizes, code, Q, K, V, O, L, dO, ranges, q_pos, slopes, tau,
                            cap, dQ, dK, dV, workspace, causal)


def attention_grad(Q, K, V, O, L, dO, tau: float, cap: float = 0.0, slopes=None, ranges=None,
                   q_pos=None, causal: bool = False, stream=None):
    """dQ, dK, dV (of Q's dtype) of ``attention`` from its O and L and the
    gradient dO; allocates them, and the workspace, on Q's device."""
    lib = _bound or _ready()
    index, sizes, code = _check_attention_grad("attention_grad", Q, K, V, O, L, dO, slopes, ranges,
                                               q_pos)
    need = flashbob_attention_workspace(*sizes, code)[1]

    def run():
        dQ, dK, dV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(K)
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
        _run_attention_grad(lib, index, sizes, code, Q, K, V, O, L, dO, ranges, q_pos, slopes, tau,
                            cap, dQ, dK, dV, workspace, causal)
        return dQ, dK, dV

    context = _elsewhere(index, stream)
    if context is None:
        return run()
    with context:
        return run()


def _check_ranges(where: str, index: int, doc_offsets, prefix, q_start, B: int, Nq: int,
                  Nk: int) -> int:
    """Checks of the arrays that ranges are built from; returns the documents."""
    _check_sizes(where, B, Nq, Nk)
    M = 0
    if doc_offsets is not None:
        _cuda_index(where, "doc_offsets", doc_offsets, "[B, M + 1]", 2)
        M = doc_offsets.shape[1] - 1
        _check_sizes(where, M)
        _check_tensor(where, "doc_offsets", doc_offsets, (B, M + 1), torch.int32, index)
    if prefix is not None:
        _check_tensor(where, "prefix", prefix, (B, M), torch.int32, index)
    if q_start is not None:
        _check_tensor(where, "q_start", q_start, (B,), torch.int32, index)
    return M


def _run_ranges(lib, index, doc_offsets, prefix, q_start, ranges, q_pos, B, M, Nq, Nk,
                causal) -> None:
    st = lib.flashbob_attention_ranges(
        _ptr(doc_offsets), _ptr(prefix), _ptr(q_start), ranges.data_ptr(), _ptr(q_pos), B, M, Nq,
        int(Nk), int(causal), _raw_stream(index))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_attention_ranges")


def flashbob_attention_ranges(doc_offsets, prefix, q_start, ranges, q_pos, Nk: int,
                              causal: bool = False, stream=None) -> None:
    """Key ranges of queries by document (see flashbob_attention_ranges)."""
    lib, where = _bound or _ready(), "flashbob_attention_ranges"
    index = _cuda_index(where, "ranges", ranges, "[B, Nq, 2]", 3)
    B, Nq, _ = ranges.shape
    _check_tensor(where, "ranges", ranges, (B, Nq, 2), torch.int32, index)
    if q_pos is not None:
        _check_tensor(where, "q_pos", q_pos, (B, Nq), torch.int32, index)
    M = _check_ranges(where, index, doc_offsets, prefix, q_start, B, Nq, Nk)
    with _elsewhere(index, stream) or contextlib.nullcontext():
        _run_ranges(lib, index, doc_offsets, prefix, q_start, ranges, q_pos, B, M, Nq, Nk, causal)


def attention_ranges(B: int, Nq: int, Nk: int, doc_offsets=None, prefix=None, q_start=None,
                     causal: bool = False, device=None, stream=None):
    """ranges [B, Nq, 2] and q_pos [B, Nq] of queries by document, on the
    device of the first array given (``device``, or the current one, if none)."""
    lib, where = _bound or _ready(), "attention_ranges"
    given = doc_offsets if doc_offsets is not None else q_start
    if given is not None:
        device = given.device
    else:
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else \
            torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"{where}: the arrays must be on a CUDA device, not {device}")
    index = torch.cuda.current_device() if device.index is None else device.index
    M = _check_ranges(where, index, doc_offsets, prefix, q_start, B, Nq, Nk)

    def run():
        ranges = torch.empty((B, Nq, 2), dtype=torch.int32, device=device)
        q_pos = torch.empty((B, Nq), dtype=torch.int32, device=device)
        _run_ranges(lib, index, doc_offsets, prefix, q_start, ranges, q_pos, B, M, Nq, Nk, causal)
        return ranges, q_pos

    context = _elsewhere(index, stream)
    if context is None:
        return run()
    with context:
        return run()


def _check_norm(where: str, QKV, wq, wk, freqs, positions):
    """Checks of the norm-and-rotation calls; returns the device and B, N, the
    heads, d, R, axes."""
    index = _cuda_index(where, "QKV", QKV, "[B, N, H + 2 Hkv, d]", 4)
    _check_tensor(where, "QKV", QKV, QKV.shape, QKV.dtype, index)
    B, N, heads, d = QKV.shape
    _check_sizes(where, B, N, heads, d)
    R, axes = 0, 1
    if freqs is not None:
        _cuda_index(where, "freqs", freqs, "[axes, R / 2]", 2)
        axes, R = freqs.shape
        _check_sizes(where, axes, 2 * R)
        _check_tensor(where, "freqs", freqs, freqs.shape, torch.float32, index)
        R *= 2
    if positions is not None:
        _check_tensor(where, "positions", positions, (axes, B, N), torch.int32, index)
    if wq is not None:
        _check_tensor(where, "wq", wq, (d,), torch.float32, index)
    if wk is not None:
        _check_tensor(where, "wk", wk, (d,), torch.float32, index)
    return index, (B, N, heads, d, R, axes)


def _check_cache(where: str, QKV, H: int, K, V, kv_start, index: int, sizes):
    """K, V (and the rows they get) beside a checked projection; returns Hkv, Nk."""
    B, _, heads, d, _, _ = sizes
    _cuda_index(where, "K", K, "[B, Hkv, Nk, d]", 4)
    Hkv, Nk = K.shape[1], K.shape[2]
    _check_sizes(where, Nk)
    if H + 2 * Hkv != heads:
        raise ValueError(f"{where}: QKV has {heads} heads, expected {H} + 2 * {Hkv}")
    _check_tensor(where, "K", K, (B, Hkv, Nk, d), QKV.dtype, index)
    _check_tensor(where, "V", V, (B, Hkv, Nk, d), QKV.dtype, index)
    if kv_start is not None:
        _check_tensor(where, "kv_start", kv_start, (B,), torch.int32, index)
    return Hkv, Nk


def _run_norm(lib, index, sizes, QKV, wq, wk, freqs, positions, kv_start, eps, Q, K, V, H, Hkv,
              Nk, interleaved) -> None:
    B, N, _, d, R, axes = sizes
    st = lib.flashbob_qk_norm_rope(
        QKV.data_ptr(), _ptr(wq), _ptr(wk), _ptr(freqs), _ptr(positions), _ptr(kv_start),
        float(eps), Q.data_ptr(), K.data_ptr(), V.data_ptr(), B, N, H, Hkv, Nk, d, R, axes, int(interleaved),
        _dtype_code(QKV), _raw_stream(index))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_qk_norm_rope")


def flashbob_qk_norm_rope(QKV, wq, wk, freqs, positions, kv_start, eps: float, Q, K, V,
                          interleaved: bool = False, stream=None) -> None:
    """Head-major Q, K, V of the packed projection, normed and rotated (see
    flashbob_qk_norm_rope in the header)."""
    lib, where = _bound or _ready(), "flashbob_qk_norm_rope"
    index, sizes = _check_norm(where, QKV, wq, wk, freqs, positions)
    _cuda_index(where, "Q", Q, "[B, H, N, d]", 4)
    H = Q.shape[1]
    _check_tensor(where, "Q", Q, (sizes[0], H, sizes[1], sizes[3]), QKV.dtype, index)
    Hkv, Nk = _check_cache(where, QKV, H, K, V, kv_start, index, sizes)
    with _elsewhere(index, stream) or contextlib.nullcontext():
        _run_norm(lib, index, sizes, QKV, wq, wk, freqs, positions, kv_start, eps, Q, K, V, H, Hkv,
                  Nk, interleaved)


def qk_norm_rope(QKV, H: int, wq=None, wk=None, freqs=None, positions=None, eps: float = 1e-6,
                 interleaved: bool = False, K=None, V=None, kv_start=None, stream=None):
    """Q, K, V (head-major) of the packed projection QKV with H query heads:
    the norm of queries and keys for each head and the rotation by position.
    Allocates them on QKV's device; K and V may be given (a cache, whose rows
    kv_start[b] + n are written)."""
    lib, where = _bound or _ready(), "qk_norm_rope"
    index, sizes = _check_norm(where, QKV, wq, wk, freqs, positions)
    B, N, heads, d, _, _ = sizes
    if not 0 < H < heads or (heads - H) % 2:
        raise ValueError(f"{where}: {heads} heads are not {H} query heads and two equal groups of "
                         "key and value heads")
    if (K is None) != (V is None):
        raise ValueError(f"{where}: K and V are given together or not at all")
    if K is not None:
        Hkv, Nk = _check_cache(where, QKV, H, K, V, kv_start, index, sizes)
    elif kv_start is not None:
        raise ValueError(f"{where}: kv_start needs K and V")
    else:
        Hkv, Nk = (heads - H) // 2, N

    def run():
        Q = torch.empty((B, H, N, d), dtype=QKV.dtype, device=QKV.device)
        k, v = K, V
        if k is None:
            k = torch.empty((B, Hkv, N, d), dtype=QKV.dtype, device=QKV.device)
            v = torch.empty_like(k)
        _run_norm(lib, index, sizes, QKV, wq, wk, freqs, positions, kv_start, eps, Q, k, v, H, Hkv,
                  Nk, interleaved)
        return Q, k, v

    context = _elsewhere(index, stream)
    if context is None:
        return run()
    with context:
        return run()


@functools.lru_cache(maxsize=256)
def flashbob_qk_norm_rope_workspace(B: int, N: int, H: int, Hkv: int, d: int,
                                    in_dtype: int) -> int:
    """Workspace bytes of flashbob_qk_norm_rope_grad with gains."""
    _check_sizes("flashbob_qk_norm_rope_workspace", B, N, H, Hkv, d)
    n = ctypes.c_size_t()
    st = load_library().flashbob_qk_norm_rope_workspace(B, N, H, Hkv, d, in_dtype,
                                                        ctypes.byref(n))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_qk_norm_rope_workspace")
    return n.value


def _check_norm_grad(where: str, QKV, dQ, dK, dV, wq, wk, freqs, positions):
    index, sizes = _check_norm(where, QKV, wq, wk, freqs, positions)
    B, N, heads, d, _, _ = sizes
    _cuda_index(where, "dQ", dQ, "[B, H, N, d]", 4)
    _cuda_index(where, "dK", dK, "[B, Hkv, N, d]", 4)
    H, Hkv = dQ.shape[1], dK.shape[1]
    if H + 2 * Hkv != heads:
        raise ValueError(f"{where}: QKV has {heads} heads, expected {H} + 2 * {Hkv}")
    _check_tensor(where, "dQ", dQ, (B, H, N, d), dQ.dtype, index)
    _check_tensor(where, "dK", dK, (B, Hkv, N, d), dQ.dtype, index)
    _check_tensor(where, "dV", dV, (B, Hkv, N, d), dQ.dtype, index)
    return index, sizes, H, Hkv


def _run_norm_grad(lib, index, sizes, H, Hkv, QKV, wq, wk, freqs, positions, eps, dQ, dK, dV, dQKV,
                   dwq, dwk, workspace, interleaved) -> None:
    B, N, _, d, R, axes = sizes
    st = lib.flashbob_qk_norm_rope_grad(
        QKV.data_ptr(), _ptr(wq), _ptr(wk), _ptr(freqs), _ptr(positions), float(eps), dQ.data_ptr(),
        dK.data_ptr(), dV.data_ptr(), dQKV.data_ptr(), _ptr(dwq), _ptr(dwk), _ptr(workspace),
        _bytes(workspace), B, N, H, Hkv, d, R, axes, int(interleaved), _dtype_code(QKV),
        _dtype_code(dQ), _raw_stream(index))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_qk_norm_rope_grad")


def flashbob_qk_norm_rope_grad(QKV, wq, wk, freqs, positions, eps: float, dQ, dK, dV, dQKV, dwq,
                               dwk, workspace, interleaved: bool = False, stream=None) -> None:
    """dQKV, dwq, dwk of flashbob_qk_norm_rope (see the header)."""
    lib, where = _bound or _ready(), "flashbob_qk_norm_rope_grad"
    index, sizes, H, Hkv = _check_norm_grad(where, QKV, dQ, dK, dV, wq, wk, freqs, positions)
    _check_tensor(where, "dQKV", dQKV, QKV.shape, QKV.dtype, index)
    if dwq is not None:
        _check_tensor(where, "dwq", dwq, (sizes[3],), torch.float32, index)
    if dwk is not None:
        _check_tensor(where, "dwk", dwk, (sizes[3],), torch.float32, index)
    _check_workspace(where, workspace, index)
    with _elsewhere(index, stream) or contextlib.nullcontext():
        _run_norm_grad(lib, index, sizes, H, Hkv, QKV, wq, wk, freqs, positions, eps, dQ, dK, dV,
                       dQKV, dwq, dwk, workspace, interleaved)


def qk_norm_rope_grad(QKV, dQ, dK, dV, wq=None, wk=None, freqs=None, positions=None,
                      eps: float = 1e-6, interleaved: bool = False, stream=None):
    """dQKV, dwq, dwk of ``qk_norm_rope`` from the gradients of Q, K and V
    (fp32 or bf16); dwq and dwk are None without gains."""
    lib = _bound or _ready()
    index, sizes, H, Hkv = _check_norm_grad("qk_norm_rope_grad", QKV, dQ, dK, dV, wq, wk, freqs,
                                            positions)
    need = 0 if wq is None else flashbob_qk_norm_rope_workspace(
        sizes[0], sizes[1], H, Hkv, sizes[3], _dtype_code(QKV))

    def run():
        dQKV = torch.empty_like(QKV)
        dwq = None if wq is None else torch.empty_like(wq)
        dwk = None if wk is None else torch.empty_like(wk)
        workspace = torch.empty(need, dtype=torch.uint8, device=QKV.device) if need else None
        _run_norm_grad(lib, index, sizes, H, Hkv, QKV, wq, wk, freqs, positions, eps, dQ, dK, dV,
                       dQKV, dwq, dwk, workspace, interleaved)
        return dQKV, dwq, dwk

    context = _elsewhere(index, stream)
    if context is None:
        return run()
    with context:
        return run()


def flashbob_bob_launches(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int,
                          in_dtype: int) -> int:
    """Kernel launches of one flashbob_bob call with these sizes."""
    n = ctypes.c_int()
    st = load_library().flashbob_bob_launches(B, H, Hkv, Nq, Nk, d, in_dtype, ctypes.byref(n))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_bob_launches")
    return n.value


def flashbob_bob_tile_sizes(d: int, in_dtype: int) -> dict:
    """Tiles and dynamic shared memory of flashbob_bob for (d, in_dtype)."""
    v = [ctypes.c_int() for _ in range(4)]
    s = [ctypes.c_size_t() for _ in range(2)]
    st = load_library().flashbob_bob_tile_sizes(d, in_dtype, *(ctypes.byref(x) for x in v),
                                                *(ctypes.byref(x) for x in s))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_bob_tile_sizes")
    return {"Br1": v[0].value, "Bc1": v[1].value, "Br2": v[2].value, "Bc2": v[3].value,
            "smem_bytes_pass1": s[0].value, "smem_bytes_pass2": s[1].value}


def flashbob_check_wait_timeout(stream=None) -> None:
    """Launch the diagnostic whose bounded wait runs out (see the header)."""
    st = load_library().flashbob_check_wait_timeout(_stream_handle(stream))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_check_wait_timeout")


def flashbob_mma_cycles(n: int, a_in_tmem: bool, stream=None) -> float:
    """SM cycles per tcgen05.mma of M = 128, N = n, K = 16 (see the header)."""
    c = ctypes.c_double()
    st = load_library().flashbob_mma_cycles(n, int(a_in_tmem), _stream_handle(stream),
                                             ctypes.byref(c))
    if st != FLASHBOB_OK:
        raise FlashbobError(st, "flashbob_mma_cycles")
    return c.value


def flashbob_last_device_error() -> int:
    """Status of the device error word (synchronises the device, then clears)."""
    return load_library().flashbob_last_device_error()


# ---------------------------------------------------------------------------
# Convenience wrappers: allocate the outputs with torch, then call the ABI.
# ---------------------------------------------------------------------------

def prep(Q, K, V, dO, tau: float, causal: bool = False, stream=None):
    """Allocate O, L, D on Q's device and run flashbob_prep (dO = None: the
    forward only, D is returned as None)."""
    import torch
    B, H, Nq, d = Q.shape
    O = torch.empty((B, H, Nq, d), dtype=torch.float32, device=Q.device)
    L = torch.empty((B, H, Nq), dtype=torch.float32, device=Q.device)
    D = None if dO is None else torch.empty((B, H, Nq), dtype=torch.float32, device=Q.device)
    flashbob_prep(Q, K, V, dO, O, L, D, tau, causal, stream)
    return O, L, D


def attention_jvp(Q, K, V, UQ, UK, UV, tau: float, causal: bool = False, O=None, L=None,
                  stream=None):
    """O, L (from flashbob_prep when not given) and the tangents O', L'."""
    import torch
    if O is None or L is None:
        O, L, _ = prep(Q, K, V, None, tau, causal, stream)
    Od = torch.empty_like(O)
    Ld = torch.empty_like(L)
    flashbob_attention_jvp(Q, K, V, O, L, UQ, UK, UV, tau, Od, Ld, causal, stream)
    return O, L, Od, Ld


def alloc_bob_outputs(Q, fill: float | None = None, K=None) -> dict:
    """fp32 output buffers of flashbob_bob (optionally filled, e.g. with NaN);
    d~K and d~V take K's head count and length (grouped-query, rectangular
    attention) when K is given."""
    import torch
    B, H, Nq, d = Q.shape
    Hkv, Nk = (K.shape[1], K.shape[2]) if K is not None else (H, Nq)
    out = {k: torch.empty((B, H, Nq, d), dtype=torch.float32, device=Q.device)
           for k in ("dQt", "ddOt")}
    out.update({k: torch.empty((B, Hkv, Nk, d), dtype=torch.float32, device=Q.device)
                for k in ("dKt", "dVt")})
    out.update({k: torch.empty((B, H, Nq), dtype=torch.float32, device=Q.device)
                for k in ("alpha", "E")})
    if fill is not None:
        for t in out.values():
            t.fill_(fill)
    return out


def bob(Q, K, V, O, dO, L, D, UQ, UK, UV, tau: float, out: dict | None = None,
        causal: bool = False, stream=None):
    """Run flashbob_bob into ``out`` (allocated when None); returns the dict."""
    if out is None:
        out = alloc_bob_outputs(Q, K=K)
    flashbob_bob(Q, K, V, O, dO, L, D, UQ, UK, UV, tau, out["dQt"], out["dKt"], out["dVt"],
                 out["ddOt"], out["alpha"], out["E"], causal, stream)
    return out
