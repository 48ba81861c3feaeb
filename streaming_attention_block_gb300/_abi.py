"""ctypes marshalling for libsab.so.  Same names as the C ABI, without the
``sab_`` prefix.  Tensors are passed as device pointers taken from torch
tensors (which must be CUDA, contiguous and of the documented dtype); streams
default to torch's current stream."""

from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
KV_BF16 = 0
KV_FP8_E4M3 = 1
KV_INT8K_FP8V = 2

_STATUS = {
    0: "SAB_OK", 1: "SAB_ERR_INVALID_ARG", 2: "SAB_ERR_UNSUPPORTED", 3: "SAB_ERR_OUT_OF_RANGE",
    4: "SAB_ERR_WORKSPACE", 5: "SAB_ERR_CUDA", 6: "SAB_ERR_TIMEOUT", 7: "SAB_ERR_BOUNDS",
}
ERR_TIMEOUT = 6
ERR_BOUNDS = 7
# sab_debug_inject_bounds_error kinds
DEBUG_INJECT_APPEND_SLOT = 1
DEBUG_INJECT_KEY_ROW = 2
DEBUG_INJECT_WS_TILE = 3


class SabError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = int(status)
        super().__init__(f"{what}: {_STATUS.get(self.status, self.status)}")


class RingDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_layers", "batch", "heads", "head_dim", "chunk_tokens", "ring_slots", "has_sink", "kv_dtype")]


_lib = None


def library_path() -> str:
    return os.environ.get("SAB_LIBRARY", os.path.join(_HERE, "libsab.so"))


def library() -> ctypes.CDLL:
    """Load libsab.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"libsab.so not found at {path}: build it with "
                          "`python -m streaming_attention_block_gb300.build` (there is no fallback)")
    lib = ctypes.CDLL(path)
    P, I, LL, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t, ctypes.c_float
    DP = ctypes.POINTER(RingDesc)
    sigs = {
        "sab_kv_ring_bytes": (SZ, [DP]),
        "sab_kv_ring_create": (I, [DP, P, SZ, P, ctypes.POINTER(P)]),
        "sab_kv_ring_destroy": (I, [P]),
        "sab_kv_ring_get_desc": (I, [P, DP]),
        "sab_kv_ring_layer_ptrs": (I, [P, I, ctypes.POINTER(P), ctypes.POINTER(P), ctypes.POINTER(P),
                                       ctypes.POINTER(P)]),
        "sab_kv_ring_set_sink": (I, [P, I, P, P, P]),
        "sab_kv_ring_append": (I, [P, I, LL, P, P, P]),
        "sab_kv_ring_slot_of": (I, [P, I, LL, ctypes.POINTER(I)]),
        "sab_kv_ring_get_state": (I, [P, ctypes.POINTER(LL), ctypes.POINTER(I), ctypes.POINTER(I)]),
        "sab_kv_ring_set_state": (I, [P, ctypes.POINTER(LL), ctypes.POINTER(I), ctypes.POINTER(I)]),
        "sab_chunk_attention_workspace": (SZ, [P, I]),
        "sab_chunk_attention": (I, [P, I, LL, P, P, P, I, I, I, F, P, P, P, SZ, P]),
        "sab_chunk_attention_noalloc": (I, [P, I, LL, P, P, P, I, I, I, F, P, P, P]),
        "sab_chunk_attention_dev": (I, [P, I, P, P, P, P, I, I, I, F, P, P, P, SZ, P]),
        "sab_kv_ring_append_dev": (I, [P, I, P, P, P, P]),
        "sab_chunk_counter_add": (I, [P, LL, P]),
        "sab_block_causal_attention_workspace": (SZ, [I, I, I, I, I]),
        "sab_block_causal_attention": (I, [P, P, P, I, I, I, I, I, I, I, F, P, P, P, SZ, P]),
        "sab_get_last_device_error": (I, [P]),
        "sab_debug_bounds_enabled": (I, []),
        "sab_debug_inject_bounds_error": (I, [I]),
        "sab_selftest_bounded_wait": (I, [ctypes.c_ulonglong, P]),
        "sab_selftest_split_abort": (I, [P, I, LL, P, P, P, I, I, I, F, P, P, P, SZ, I, P]),
        "sab_qk_norm_rope": (I, [P, I, LL, P, P, P, P, P, P, P, P, P, I, P]),
        "sab_block_causal_attention_backward_workspace": (SZ, [I, I, I]),
        "sab_block_causal_attention_backward": (I, [P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, SZ, P]),
        "sab_memory_prefix_attention": (I, [P, P, P, I, I, I, I, I, P, I, I, F, P, P, P]),
        "sab_chunk_attention_fp8mma": (I, [P, I, LL, P, I, I, I, F, P, P, P, SZ, P]),
        "sab_memory_prefix_attention_backward": (I, [P, P, P, P, P, P, I, I, I, I, I, P, I, I, F, P, P, P, P, SZ,
                                                     P]),
        "sab_rotary_plan_init": (I, [P, P]),
        "sab_rotary": (I, [P, P, P, P, LL, I, I, I, I, P]),
        "sab_rotary_backward": (I, [P, P, P, P, LL, I, I, I, I, P]),
        "sab_decay_attention_workspace": (SZ, [I, I, I, I]),
        "sab_decay_attention": (I, [P, P, P, P, P, P, I, I, I, I, F, P, P, P, SZ, P]),
        "sab_decay_attention_step": (I, [P, P, P, P, P, P, I, I, I, F, P, P, P]),
        "sab_decay_attention_backward_workspace": (SZ, [I, I, I, I]),
        "sab_decay_attention_backward": (I, [P] * 8 + [I, I, I, I, F] + [P] * 5 + [SZ, P]),
        "sab_status_string": (ctypes.c_char_p, [I]),
        "sab_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        raise SabError(status, what)


def _stream(stream, dev=None):
    if stream is None:  # the raw handle of torch.cuda.current_stream(), without building the object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev is None else dev)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor or a device pointer")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def status_string(status: int) -> str:
    return library().sab_status_string(int(status)).decode()


def version() -> str:
    return library().sab_version().decode()


def _desc(desc) -> RingDesc:
    if isinstance(desc, RingDesc):
        return desc
    return RingDesc(**desc)


def kv_ring_bytes(desc) -> int:
    return int(library().sab_kv_ring_bytes(ctypes.byref(_desc(desc))))


def kv_ring_create(desc, mem: torch.Tensor, stream=None) -> ctypes.c_void_p:
    d = _desc(desc)
    h = ctypes.c_void_p()
    _check(library().sab_kv_ring_create(ctypes.byref(d), _ptr(mem, torch.uint8, "mem"),
                                        mem.numel(), _stream(stream), ctypes.byref(h)), "kv_ring_create")
    return h


def kv_ring_destroy(handle):
    _check(library().sab_kv_ring_destroy(handle), "kv_ring_destroy")


def kv_ring_get_desc(handle) -> RingDesc:
    d = RingDesc()
    _check(library().sab_kv_ring_get_desc(handle, ctypes.byref(d)), "kv_ring_get_desc")
    return d


def kv_ring_layer_ptrs(handle, layer: int):
    k, v, ks, vs = (ctypes.c_void_p() for _ in range(4))
    _check(library().sab_kv_ring_layer_ptrs(handle, int(layer), ctypes.byref(k), ctypes.byref(v),
                                            ctypes.byref(ks), ctypes.byref(vs)), "kv_ring_layer_ptrs")
    return k.value, v.value, ks.value, vs.value


def kv_ring_set_sink(handle, layer: int, K, V, stream=None):
    _check(library().sab_kv_ring_set_sink(handle, int(layer), _ptr(K, torch.bfloat16, "K"),
                                          _ptr(V, torch.bfloat16, "V"), _stream(stream)), "kv_ring_set_sink")


def kv_ring_append(handle, layer: int, chunk: int, K, V, stream=None):
    _check(library().sab_kv_ring_append(handle, int(layer), int(chunk), _ptr(K, torch.bfloat16, "K"),
                                        _ptr(V, torch.bfloat16, "V"), _stream(stream)), "kv_ring_append")


def kv_ring_slot_of(handle, layer: int, chunk: int) -> int:
    s = ctypes.c_int()
    _check(library().sab_kv_ring_slot_of(handle, int(layer), int(chunk), ctypes.byref(s)), "kv_ring_slot_of")
    return s.value


def kv_ring_get_state(handle, num_layers: int):
    n = (ctypes.c_longlong * num_layers)()
    h = (ctypes.c_int * num_layers)()
    s = (ctypes.c_int * num_layers)()
    _check(library().sab_kv_ring_get_state(handle, n, h, s), "kv_ring_get_state")
    return list(n), list(h), list(s)


def kv_ring_set_state(handle, newest, held, sink_set):
    L = len(newest)
    _check(library().sab_kv_ring_set_state(handle, (ctypes.c_longlong * L)(*newest), (ctypes.c_int * L)(*held),
                                           (ctypes.c_int * L)(*sink_set)), "kv_ring_set_state")


def chunk_attention_workspace(handle, num_splits: int) -> int:
    return int(library().sab_chunk_attention_workspace(handle, int(num_splits)))


def chunk_attention(handle, layer: int, chunk: int, Q, K_cur, V_cur, window: int, use_sink: bool,
                    num_splits: int, softmax_scale: float, O, LSE=None, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(library().sab_chunk_attention(
        handle, int(layer), int(chunk), _ptr(Q, torch.bfloat16, "Q"), _ptr(K_cur, torch.bfloat16, "K_cur"),
        _ptr(V_cur, torch.bfloat16, "V_cur"), int(window), int(bool(use_sink)), int(num_splits),
        float(softmax_scale), _ptr(O, torch.bfloat16, "O"), _ptr(LSE, torch.float32, "LSE"),
        _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream)), "chunk_attention")


def chunk_attention_noalloc(handle, layer: int, chunk: int, Q, K_cur, V_cur, window: int, use_sink: bool,
                            num_splits: int, softmax_scale: float, O, LSE=None, stream=None):
    """sab_chunk_attention_noalloc: the split merge uses the library's own
    device scratch instead of a caller workspace (see include/sab.h)."""
    _check(library().sab_chunk_attention_noalloc(
        handle, int(layer), int(chunk), _ptr(Q, torch.bfloat16, "Q"), _ptr(K_cur, torch.bfloat16, "K_cur"),
        _ptr(V_cur, torch.bfloat16, "V_cur"), int(window), int(bool(use_sink)), int(num_splits),
        float(softmax_scale), _ptr(O, torch.bfloat16, "O"), _ptr(LSE, torch.float32, "LSE"), _stream(stream)),
        "chunk_attention_noalloc")


def chunk_attention_dev(handle, layer: int, d_chunk, Q, K_cur, V_cur, window: int, use_sink: bool,
                        num_splits: int, softmax_scale: float, O, LSE=None, workspace=None, stream=None):
    """sab_chunk_attention_dev: the chunk index is read from ``d_chunk`` (a
    device int64 tensor) when the kernel runs, so the call can be captured
    once in a CUDA graph and replayed for every chunk (see include/sab.h)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(library().sab_chunk_attention_dev(
        handle, int(layer), _ptr(d_chunk, torch.int64, "d_chunk"), _ptr(Q, torch.bfloat16, "Q"),
        _ptr(K_cur, torch.bfloat16, "K_cur"), _ptr(V_cur, torch.bfloat16, "V_cur"), int(window),
        int(bool(use_sink)), int(num_splits), float(softmax_scale), _ptr(O, torch.bfloat16, "O"),
        _ptr(LSE, torch.float32, "LSE"), _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream)),
        "chunk_attention_dev")


def kv_ring_append_dev(handle, layer: int, d_chunk, K, V, stream=None):
    """sab_kv_ring_append_dev: append into slot (*d_chunk mod R), chunk read on the device."""
    _check(library().sab_kv_ring_append_dev(handle, int(layer), _ptr(d_chunk, torch.int64, "d_chunk"),
                                            _ptr(K, torch.bfloat16, "K"), _ptr(V, torch.bfloat16, "V"),
                                            _stream(stream)), "kv_ring_append_dev")


def chunk_counter_add(d_chunk, delta: int = 1, stream=None):
    """sab_chunk_counter_add: *d_chunk += delta on the stream."""
    _check(library().sab_chunk_counter_add(_ptr(d_chunk, torch.int64, "d_chunk"), int(delta), _stream(stream)),
           "chunk_counter_add")


def block_causal_attention_backward_workspace(B: int, L: int, H: int) -> int:
    return int(library().sab_block_causal_attention_backward_workspace(B, L, H))


def block_causal_attention_backward(Q, K, V, O, dO, LSE, chunk_tokens: int, window: int, softmax_scale: float,
                                    dQ, dK, dV, workspace=None, stream=None):
    """sab_block_causal_attention_backward: (dQ, dK, dV) of block-causal
    attention from the forward's O and LSE (see include/sab.h)."""
    B, L, H, D = Q.shape
    if workspace is None:
        n = int(library().sab_block_causal_attention_backward_workspace(B, L, H))
        workspace = torch.empty(n, dtype=torch.uint8, device=Q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(library().sab_block_causal_attention_backward(
        _ptr(Q, torch.bfloat16, "Q"), _ptr(K, torch.bfloat16, "K"), _ptr(V, torch.bfloat16, "V"),
        _ptr(O, torch.bfloat16, "O"), _ptr(dO, torch.bfloat16, "dO"), _ptr(LSE, torch.float32, "LSE"),
        B, L, H, D, int(chunk_tokens), int(window), float(softmax_scale), _ptr(dQ, torch.bfloat16, "dQ"),
        _ptr(dK, torch.bfloat16, "dK"), _ptr(dV, torch.bfloat16, "dV"), _ptr(workspace, None, "workspace"),
        ws_bytes, _stream(stream)), "block_causal_attention_backward")


def chunk_attention_fp8mma(handle, layer: int, chunk: int, Q, window: int, use_sink: bool, softmax_scale: float,
                           O, LSE=None, stream=None, num_splits: int = 1, workspace=None):
    """sab_chunk_attention_fp8mma: chunk attention over an E4M3 ring with Q and
    P rounded to E4M3 for the tensor-core products (see include/sab.h);
    ``num_splits`` and ``workspace`` as in ``chunk_attention``."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(library().sab_chunk_attention_fp8mma(
        handle, int(layer), int(chunk), _ptr(Q, torch.bfloat16, "Q"), int(window), 1 if use_sink else 0,
        int(num_splits), float(softmax_scale), _ptr(O, torch.bfloat16, "O"), _ptr(LSE, torch.float32, "LSE"),
        _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream)), "chunk_attention_fp8mma")


def memory_prefix_attention(Q, K, V, mem_pad: int, mem_len, chunk_tokens: int, window: int, softmax_scale: float,
                            O, LSE=None, stream=None):
    """sab_memory_prefix_attention: block-causal target chunks behind a
    per-sample memory prefix of mem_pad positions, mem_len (device int32 [B])
    of them real (see include/sab.h)."""
    B, L, H, D = Q.shape
    _check(library().sab_memory_prefix_attention(
        _ptr(Q, torch.bfloat16, "Q"), _ptr(K, torch.bfloat16, "K"), _ptr(V, torch.bfloat16, "V"),
        B, L, H, D, int(mem_pad), _ptr(mem_len, torch.int32, "mem_len"), int(chunk_tokens), int(window),
        float(softmax_scale), _ptr(O, torch.bfloat16, "O"), _ptr(LSE, torch.float32, "LSE"), _stream(stream)),
        "memory_prefix_attention")


def memory_prefix_attention_backward(Q, K, V, O, dO, LSE, mem_pad: int, mem_len, chunk_tokens: int, window: int,
                                     softmax_scale: float, dQ, dK, dV, workspace=None, stream=None):
    """sab_memory_prefix_attention_backward: (dQ, dK, dV) of
    memory_prefix_attention from its O and LSE (see include/sab.h)."""
    B, L, H, D = Q.shape
    if workspace is None:
        n = int(library().sab_block_causal_attention_backward_workspace(B, L, H))
        workspace = torch.empty(n, dtype=torch.uint8, device=Q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(library().sab_memory_prefix_attention_backward(
        _ptr(Q, torch.bfloat16, "Q"), _ptr(K, torch.bfloat16, "K"), _ptr(V, torch.bfloat16, "V"),
        _ptr(O, torch.bfloat16, "O"), _ptr(dO, torch.bfloat16, "dO"), _ptr(LSE, torch.float32, "LSE"),
        B, L, H, D, int(mem_pad), _ptr(mem_len, torch.int32, "mem_len"), int(chunk_tokens), int(window),
        float(softmax_scale), _ptr(dQ, torch.bfloat16, "dQ"), _ptr(dK, torch.bfloat16, "dK"),
        _ptr(dV, torch.bfloat16, "dV"), _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream)),
        "memory_prefix_attention_backward")


def block_causal_attention_workspace(B: int, L: int, H: int, D: int, num_splits: int) -> int:
    return int(library().sab_block_causal_attention_workspace(B, L, H, D, num_splits))


def block_causal_attention(Q, K, V, chunk_tokens: int, window: int, num_splits: int, softmax_scale: float,
                           O, LSE=None, workspace=None, stream=None):
    B, L, H, D = Q.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(library().sab_block_causal_attention(
        _ptr(Q, torch.bfloat16, "Q"), _ptr(K, torch.bfloat16, "K"), _ptr(V, torch.bfloat16, "V"),
        B, L, H, D, int(chunk_tokens), int(window), int(num_splits), float(softmax_scale),
        _ptr(O, torch.bfloat16, "O"), _ptr(LSE, torch.float32, "LSE"), _ptr(workspace, None, "workspace"),
        ws_bytes, _stream(stream)), "block_causal_attention")


def get_last_device_error(stream=None) -> int:
    return int(library().sab_get_last_device_error(_stream(stream)))


def debug_bounds_enabled() -> bool:
    """True when the loaded library is the debug build (device index checks)."""
    return bool(library().sab_debug_bounds_enabled())


def debug_inject_bounds_error(what: int):
    """sab_debug_inject_bounds_error (debug builds only)."""
    _check(library().sab_debug_inject_bounds_error(int(what)), "debug_inject_bounds_error")


# Canary bands: a device buffer can be allocated between two bands of
# GUARD_BYTE that no call may write.  While a watch is open every guarded
# allocation is recorded, and closing the watch counts the band bytes that
# changed (buffer overruns or underruns by any kernel that wrote near it).
GUARD_BYTE = 0xA5
_guard_watch = None


def _guarded(nbytes: int, guard: int, device, zero: bool = False):
    """(storage, view): ``view`` is ``nbytes`` of 256-byte-aligned device
    memory, with ``guard`` bytes (rounded up to 256) of canaries on each side."""
    g = (int(guard) + 255) // 256 * 256
    mem = torch.empty(nbytes + 2 * g + 256, dtype=torch.uint8, device=device)
    off = (-mem.data_ptr()) % 256 + g
    buf = mem[off:off + nbytes]
    if zero:
        buf.zero_()
    if g:
        mem[:off].fill_(GUARD_BYTE)
        mem[off + nbytes:].fill_(GUARD_BYTE)
        if _guard_watch is not None:
            _guard_watch.append((mem, ((0, off), (off + nbytes, mem.numel()))))
    return mem, buf


def guard_watch_begin():
    """Start recording guarded allocations."""
    global _guard_watch
    _guard_watch = []


def guard_watch_end() -> int:
    """Stop recording; return how many canary bytes of the recorded
    allocations no longer hold GUARD_BYTE (0: no call wrote outside them)."""
    global _guard_watch
    watched, _guard_watch = _guard_watch or [], None
    bad = 0
    for mem, bands in watched:
        for lo, hi in bands:
            bad += int((mem[lo:hi] != GUARD_BYTE).sum().item())
    return bad


def selftest_bounded_wait(timeout_ns: int, stream=None):
    """sab_selftest_bounded_wait: a device wait that nothing completes gives up
    after timeout_ns; read the result with get_last_device_error."""
    _check(library().sab_selftest_bounded_wait(int(timeout_ns), _stream(stream)), "selftest_bounded_wait")


def selftest_split_abort(handle, layer: int, chunk: int, Q, K_cur, V_cur, window: int, use_sink: bool,
                         num_splits: int, softmax_scale: float, O, LSE, workspace, abort_split: int, stream=None):
    """sab_selftest_split_abort: a split call (num_splits > 8, workspace merge)
    whose split ``abort_split`` reports itself as having given up a wait."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(library().sab_selftest_split_abort(
        handle, int(layer), int(chunk), _ptr(Q, torch.bfloat16, "Q"), _ptr(K_cur, torch.bfloat16, "K_cur"),
        _ptr(V_cur, torch.bfloat16, "V_cur"), int(window), int(bool(use_sink)), int(num_splits),
        float(softmax_scale), _ptr(O, torch.bfloat16, "O"), _ptr(LSE, torch.float32, "LSE"),
        _ptr(workspace, None, "workspace"), ws_bytes, int(abort_split), _stream(stream)), "selftest_split_abort")


class RopeDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("frames", "height", "width", "band_t", "band_h", "band_w")] + [
        ("base", ctypes.c_float), ("eps", ctypes.c_float)]


def qk_norm_rope(handle, layer: int, chunk: int, Q, K, V, rope: RopeDesc, Q_out, K_out=None, V_out=None,
                 gamma_q=None, gamma_k=None, append: bool = False, stream=None):
    """sab_qk_norm_rope: q' = RoPE(RMSNorm(q)), k' = RoPE(RMSNorm(k)) of one
    chunk, optionally appending k', v into the ring slot (see include/sab.h)."""
    _check(library().sab_qk_norm_rope(
        handle, int(layer), int(chunk), _ptr(Q, torch.bfloat16, "Q"), _ptr(K, torch.bfloat16, "K"),
        _ptr(V, torch.bfloat16, "V"), _ptr(gamma_q, torch.float32, "gamma_q"), _ptr(gamma_k, torch.float32, "gamma_k"),
        ctypes.byref(rope), _ptr(Q_out, torch.bfloat16, "Q_out"), _ptr(K_out, torch.bfloat16, "K_out"),
        _ptr(V_out, torch.bfloat16, "V_out"), int(bool(append)), _stream(stream)), "qk_norm_rope")


# ---------------------------------------------------------------- rotary

ROTARY_INTERLEAVED = 0
ROTARY_HALF = 1
ROTARY_SCALE_NONE = 0
ROTARY_SCALE_LINEAR = 1
ROTARY_SCALE_BASE = 2
ROTARY_SCALE_RAMP = 3
DTYPE_BF16 = 0
DTYPE_FP32 = 1
_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}


class RotaryDesc(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int), ("axes", ctypes.c_int), ("band", ctypes.c_int * 3),
                ("scaling", ctypes.c_int)] + [(n, ctypes.c_double) for n in (
                    "base", "factor", "original_context", "ramp_fast", "ramp_slow", "magnitude")]


class RotaryPlan(ctypes.Structure):
    """Frequencies of one rotary embedding (plain host data, see ``rotary_plan``)."""

    _fields_ = [("magic", ctypes.c_uint), ("layout", ctypes.c_int), ("axes", ctypes.c_int), ("dims", ctypes.c_int),
                ("magnitude", ctypes.c_float), ("axis", ctypes.c_ubyte * 128), ("step", ctypes.c_ulonglong * 128)]


class RotaryRows(ctypes.Structure):
    _fields_ = [("inp", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int)] + [
        (n, ctypes.c_longlong) for n in ("in_batch", "in_token", "out_batch", "out_token")]


def rotary_plan(bands, layout: int = ROTARY_INTERLEAVED, base: float = 10000.0, scaling: int = ROTARY_SCALE_NONE,
                factor: float = 1.0, original_context: float = 0.0, ramp_fast: float = 32.0, ramp_slow: float = 1.0,
                magnitude: float = 1.0) -> RotaryPlan:
    """sab_rotary_plan_init: the frequencies of one rotary embedding.
    ``bands``: rotated dimensions per position axis (one to three even
    numbers; their sum may be less than the head dimension).  Keep the plan
    and pass it to every call (see include/sab.h)."""
    bands = tuple(int(n) for n in bands)
    if not 1 <= len(bands) <= 3:
        raise SabError(1, "rotary_plan: one to three bands")
    d = RotaryDesc(int(layout), len(bands), (ctypes.c_int * 3)(*bands), int(scaling), float(base), float(factor),
                   float(original_context), float(ramp_fast), float(ramp_slow), float(magnitude))
    plan = RotaryPlan()
    _check(library().sab_rotary_plan_init(ctypes.byref(d), ctypes.byref(plan)), "rotary_plan")
    return plan


def _refuse(t, name, dev, dtypes, shape=None):
    """Raise what is wrong with a tensor argument that failed its check."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: must be contiguous")


def _device():
    """Index of the current device (-2: there is none, so no tensor is on it)."""
    try:
        return torch._C._cuda_getDevice()  # torch.cuda.current_device() without its start-up check
    except (RuntimeError, AttributeError):
        return -2


def _arg(t, shape, dtype, name, dev):
    """Device pointer of a contiguous tensor of this shape and type on the
    current device ``dev`` (None and raw pointers pass through)."""
    if t is None:
        return None
    try:
        if t.get_device() == dev and t.dtype == dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        if isinstance(t, int):
            return t
    _refuse(t, name, dev, (dtype,), shape)


_ROWS = struct.Struct("@PPiqqqq")  # the layout of RotaryRows, packed faster than the structure is built


def _rotary_rows(x, out, name, dev):
    """Token rows of ``x`` and ``out``, [B, L, H, D] with contiguous heads, and
    what the call's other tensors have to agree with."""
    if not isinstance(x, torch.Tensor) or not isinstance(out, torch.Tensor) or x.dim() != 4 or out.dim() != 4:
        raise TypeError(f"{name}, {name}_out: expected [B, L, H, D] torch tensors")
    dtype = x.dtype
    if x.get_device() != dev or dtype not in _DTYPES:
        _refuse(x, name, dev, tuple(_DTYPES))
    B, L, H, D = shape = x.shape
    ib, il, ih, id_ = x.stride()
    if out is x:
        ob, ol, oh, od = ib, il, ih, id_
    else:
        if out.get_device() != dev:
            _refuse(out, name + "_out", dev, (dtype,))
        if out.dtype != dtype or out.shape != shape:
            raise ValueError(f"{name}_out: expected the shape and type of {name}")
        ob, ol, oh, od = out.stride()
    if ((id_ != 1 or od != 1) and D > 1) or ((ih != D or oh != D) and H > 1):
        raise ValueError(f"{name}, {name}_out: a token's heads must be contiguous")
    if B == 1:  # strides of axes of one entry say nothing
        ib = ob = H * D
    if L == 1:
        il = ol = H * D
    return _ROWS.pack(x.data_ptr(), out.data_ptr(), H, ib, il, ob, ol), B, L, D, dtype


def _rotary(fn, what, plan, Q, K, Q_out, K_out, positions, first_position, stream):
    dev = _device()
    q, B, L, D, dtype = _rotary_rows(Q, Q_out, "Q", dev)
    if B * L > 1 << 31:  # would be cut to 32 bits on the way to the library
        raise SabError(1, what)
    k = None
    if K is not None:
        k, *same = _rotary_rows(K, K_out, "K", dev)
        if same != [B, L, D, dtype]:
            raise ValueError("K: expected Q's batch, length, head dimension and type")
    if positions is not None and positions.__class__ is not int:
        want = (plan.axes, B, L)
        if not isinstance(positions, torch.Tensor) or positions.get_device() != dev or \
                positions.dtype != torch.int64 or not positions.is_contiguous():
            _refuse(positions, "positions", dev, (torch.int64,))
        # the order of the numbers is what counts: axes of one entry may be left out or added
        if positions.shape != want and [n for n in positions.shape if n != 1] != [n for n in want if n != 1]:
            raise ValueError(f"positions: expected shape {want}, got {tuple(positions.shape)}")
        positions = positions.data_ptr()
    status = fn(ctypes.byref(plan), q, k, positions, int(first_position), B, L, D, _DTYPES[dtype],
                _stream(stream, dev))
    if status != 0:
        raise SabError(status, what)


def rotary(plan: RotaryPlan, Q, K, Q_out, K_out=None, positions=None, first_position: int = 0, stream=None):
    """sab_rotary: rotate queries ``Q`` [B, L, Hq, D] and keys ``K``
    [B, L, Hk, D] (or None) into ``Q_out``, ``K_out``; an output may be its
    input.  Batch and token strides are free, a token's heads contiguous.
    ``positions``: int64 [axes, B, L] ([B, L] for one axis), or None for
    first_position + t (see include/sab.h)."""
    _rotary(library().sab_rotary, "rotary", plan, Q, K, Q_out, K_out, positions, first_position, stream)


def rotary_backward(plan: RotaryPlan, dQ_out, dK_out, dQ, dK=None, positions=None, first_position: int = 0,
                    stream=None):
    """sab_rotary_backward: gradients of ``rotary``'s inputs (``dQ``, ``dK``)
    from those of its outputs; shapes, strides and positions as there."""
    _rotary(library().sab_rotary_backward, "rotary_backward", plan, dQ_out, dK_out, dQ, dK, positions,
            first_position, stream)


# -------------------------------------------------------- decay attention

def decay_attention_workspace(B: int, L: int, H: int, D: int) -> int:
    return int(library().sab_decay_attention_workspace(int(B), int(L), int(H), int(D)))


def decay_attention_backward_workspace(B: int, L: int, H: int, D: int) -> int:
    return int(library().sab_decay_attention_backward_workspace(int(B), int(L), int(H), int(D)))


def _workspace(t, dev):
    """(pointer, bytes) of a workspace tensor on device ``dev``."""
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        _refuse(t, "workspace", dev, (t.dtype,))
    return t.data_ptr(), t.numel() * t.element_size()


def _empty_on(shape, dtype, device, stream):
    """Uninitialised memory for a call on ``stream`` (None: the current one),
    from that stream's own pool: what the current stream has freed may still be
    in use there, and is safe only for work queued behind it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)  # 0 names the default stream, but would make ExternalStream take a new one
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _scratch(nbytes, like, stream):
    """``nbytes`` of device scratch for one call on ``stream`` (None: 0 bytes)."""
    return None if nbytes == 0 else _empty_on(nbytes, torch.uint8, like.device, stream)


def _output(like, stream):
    """An output for a call on ``stream`` that the current stream will use."""
    out = _empty_on(like.shape, like.dtype, like.device, stream)
    if stream is not None:
        out.record_stream(torch.cuda.current_stream(like.device))
    return out


def decay_attention(Q, K, V, log_decay, scale: float, O, state_in=None, state_out=None, seq_len=None,
                    workspace=None, stream=None):
    """sab_decay_attention: linear attention of [B, L, H, D] bf16 sequences with
    a decay per head, from the state [B, H, D, D] fp32 ``state_in`` to
    ``state_out`` (see include/sab.h)."""
    B, L, H, D = Q.shape
    dev = _device()
    x, st, bf, f4 = (B, L, H, D), (B, H, D, D), torch.bfloat16, torch.float32
    q = _arg(Q, x, bf, "Q", dev)  # before scratch is made on its device
    if workspace is None:
        workspace = _scratch(decay_attention_workspace(B, L, H, D), Q, stream)
    ws, ws_bytes = _workspace(workspace, dev)
    _check(library().sab_decay_attention(
        q, _arg(K, x, bf, "K", dev), _arg(V, x, bf, "V", dev),
        _arg(log_decay, (H,), f4, "log_decay", dev), _arg(seq_len, (B,), torch.int32, "seq_len", dev),
        _arg(state_in, st, f4, "state_in", dev), B, L, H, D, float(scale), _arg(O, x, bf, "O", dev),
        _arg(state_out, st, f4, "state_out", dev), ws, ws_bytes, _stream(stream, dev)), "decay_attention")


def decay_attention_step(Q, K, V, log_decay, scale: float, state_in, state_out, O, active=None, stream=None):
    """sab_decay_attention_step: one token [B, H, D] of every sequence;
    ``state_out`` may be ``state_in`` (see include/sab.h)."""
    B, H, D = Q.shape
    dev = _device()
    x, st, bf, f4 = (B, H, D), (B, H, D, D), torch.bfloat16, torch.float32
    _check(library().sab_decay_attention_step(
        _arg(Q, x, bf, "Q", dev), _arg(K, x, bf, "K", dev), _arg(V, x, bf, "V", dev),
        _arg(log_decay, (H,), f4, "log_decay", dev), _arg(active, (B,), torch.int32, "active", dev),
        _arg(state_in, st, f4, "state_in", dev), B, H, D, float(scale), _arg(O, x, bf, "O", dev),
        _arg(state_out, st, f4, "state_out", dev), _stream(stream, dev)), "decay_attention_step")


def decay_attention_backward(Q, K, V, dO, log_decay, scale: float, dQ, dK, dV, state_in=None, d_state_out=None,
                             d_state_in=None, seq_len=None, workspace=None, stream=None):
    """sab_decay_attention_backward: (dQ, dK, dV) and d_state_in of
    decay_attention (see include/sab.h)."""
    B, L, H, D = Q.shape
    dev = _device()
    x, st, bf, f4 = (B, L, H, D), (B, H, D, D), torch.bfloat16, torch.float32
    q = _arg(Q, x, bf, "Q", dev)  # before scratch is made on its device
    if workspace is None:
        workspace = _scratch(decay_attention_backward_workspace(B, L, H, D), Q, stream)
    ws, ws_bytes = _workspace(workspace, dev)
    _check(library().sab_decay_attention_backward(
        q, _arg(K, x, bf, "K", dev), _arg(V, x, bf, "V", dev), _arg(dO, x, bf, "dO", dev),
        _arg(log_decay, (H,), f4, "log_decay", dev), _arg(seq_len, (B,), torch.int32, "seq_len", dev),
        _arg(state_in, st, f4, "state_in", dev), _arg(d_state_out, st, f4, "d_state_out", dev), B, L, H, D,
        float(scale), _arg(dQ, x, bf, "dQ", dev), _arg(dK, x, bf, "dK", dev), _arg(dV, x, bf, "dV", dev),
        _arg(d_state_in, st, f4, "d_state_in", dev), ws, ws_bytes, _stream(stream, dev)),
        "decay_attention_backward")


class DecayState:
    """The carried state of one decay-attention layer for ``batch`` streams,
    the constant-size companion of a ``KVRing``: ``attention`` feeds a chunk,
    ``step`` a token, both in place."""

    def __init__(self, log_decay, batch, head_dim):
        if log_decay.dim() != 1:
            raise ValueError("log_decay: expected [heads]")
        self.log_decay = log_decay
        self.state = torch.zeros((batch, log_decay.numel(), head_dim, head_dim), dtype=torch.float32,
                                 device=log_decay.device)

    def reset(self):
        self.state.zero_()

    def attention(self, Q, K, V, scale=None, O=None, seq_len=None, workspace=None, stream=None):
        O = _output(Q, stream) if O is None else O
        decay_attention(Q, K, V, self.log_decay, Q.shape[-1] ** -0.5 if scale is None else scale, O, self.state,
                        self.state, seq_len, workspace, stream)
        return O

    def step(self, Q, K, V, scale=None, O=None, active=None, stream=None):
        O = _output(Q, stream) if O is None else O
        decay_attention_step(Q, K, V, self.log_decay, Q.shape[-1] ** -0.5 if scale is None else scale, self.state,
                             self.state, O, active, stream)
        return O


class KVRing:
    """A ring KV cache on torch-owned device memory (memory + handle).

    ``guard_bytes`` (default ``KVRing.default_guard_bytes``, 0) puts canary
    bands of that many bytes around the ring memory and around every
    workspace ``workspace()`` allocates (see ``guard_watch_begin``)."""

    default_guard_bytes = 0

    def __init__(self, num_layers, batch, heads, head_dim, chunk_tokens, ring_slots, has_sink=False,
                 kv_dtype=KV_BF16, device="cuda", stream=None, guard_bytes=None):
        self.desc = RingDesc(num_layers, batch, heads, head_dim, chunk_tokens, ring_slots, int(bool(has_sink)),
                             int(kv_dtype))
        nbytes = kv_ring_bytes(self.desc)
        if nbytes == 0:
            raise SabError(1, "invalid ring shape")
        self.guard_bytes = self.default_guard_bytes if guard_bytes is None else int(guard_bytes)
        self.mem, self.buf = _guarded(nbytes, self.guard_bytes, device)
        self.handle = kv_ring_create(self.desc, self.buf, stream)
        self.rows = (self.desc.has_sink + ring_slots) * chunk_tokens

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.sab_kv_ring_destroy(h)
            self.handle = None

    def _view(self, ptr, nbytes, dtype, shape):
        off = ptr - self.buf.data_ptr()
        return self.buf[off:off + nbytes].view(dtype).view(shape)

    def layer_views(self, layer):
        """(K, V, K_scale, V_scale) torch views of one layer's ring memory."""
        d = self.desc
        k, v, ks, vs = kv_ring_layer_ptrs(self.handle, layer)
        fp8 = d.kv_dtype != KV_BF16  # one byte per element (E4M3, or INT8 keys)
        dt, es = (torch.uint8, 1) if fp8 else (torch.bfloat16, 2)
        shape = (d.batch, d.heads, self.rows, d.head_dim)
        n = d.batch * d.heads * self.rows * d.head_dim * es
        K = self._view(k, n, dt, shape)
        V = self._view(v, n, dt, shape)
        if not fp8:
            return K, V, None, None
        sshape = (d.batch, d.heads, d.has_sink + d.ring_slots)
        sn = d.batch * d.heads * (d.has_sink + d.ring_slots) * 4
        return K, V, self._view(ks, sn, torch.float32, sshape), self._view(vs, sn, torch.float32, sshape)

    def set_sink(self, layer, K, V, stream=None):
        kv_ring_set_sink(self.handle, layer, K, V, stream)

    def append(self, layer, chunk, K, V, stream=None):
        kv_ring_append(self.handle, layer, chunk, K, V, stream)

    def slot_of(self, layer, chunk):
        return kv_ring_slot_of(self.handle, layer, chunk)

    def workspace(self, num_splits):
        n = chunk_attention_workspace(self.handle, num_splits)
        if n == 0:
            return None
        return _guarded(n, self.guard_bytes, self.buf.device, zero=True)[1]

    def attention(self, layer, chunk, Q, K_cur=None, V_cur=None, window=2, use_sink=False, num_splits=1,
                  softmax_scale=None, O=None, LSE=None, workspace=None, stream=None):
        d = self.desc
        if softmax_scale is None:
            softmax_scale = d.head_dim ** -0.5
        if O is None:
            O = torch.empty_like(Q)
        if LSE is None:
            LSE = torch.empty((d.batch, d.heads, d.chunk_tokens), dtype=torch.float32, device=Q.device)
        if num_splits > 1 and workspace is None:
            workspace = self.workspace(num_splits)
        chunk_attention(self.handle, layer, chunk, Q, K_cur, V_cur, window, use_sink, num_splits, softmax_scale,
                        O, LSE, workspace, stream)
        return O, LSE
