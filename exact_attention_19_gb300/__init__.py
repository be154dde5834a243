"""GB300-native fused exact attention (sm_103a): forward, split-KV, sliding
window and backward; rotary positions; a paged K/V cache with its append,
attention over it, and attention of a batch that shares a prefix.

Thin ctypes binding over ``libfa_gb300.so`` (C ABI in ``include/fa.h``):
argument marshalling only, every step of the computation runs in the CUDA
kernels.  PyTorch supplies device memory and streams.

    o, lse = fwd(q, k, v, causal=False)          # torch bf16 [B, H, N, d]
    dq, dk, dv = bwd(q, k, v, o, lse, do, causal=False)
    q, k = rope(q, k, inv_freq)                  # rope_bwd turns the gradients back
    q = kv_append(q, k, v, k_cache, v_cache, block_table, seq_lens, inv_freq)
    o, lse = fwd_paged(q, k_cache, v_cache, block_table, seq_lens)
    o, lse = fwd_prefix(q, k_cache, v_cache, prefix_pages, prefix_len, block_table, seq_lens)
    fa_fwd(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Nq, Nk, d, scale, causal, stream)

There is no fallback: if the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

__all__ = [
    "FaError", "STATUS", "NOALLOC_SCRATCH_BYTES", "library_path", "load",
    "fwd", "bwd", "rope_freqs", "rope", "rope_bwd", "kv_append", "fwd_paged", "fwd_prefix",
    "fa_fwd", "fa_fwd_window", "fa_fwd_splitkv", "fa_fwd_splitkv_noalloc", "fa_splitkv_workspace_bytes",
    "fa_splitkv_heuristic", "fa_bwd", "fa_bwd_window", "fa_bwd_workspace_bytes", "fa_probe_exp2", "fa_selftest_wait",
    "fa_rope", "fa_kv_append", "fa_fwd_paged", "fa_fwd_prefix", "fa_paged_workspace_bytes",
    "fa_fwd_status",
    "fa_strerror", "fa_version",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "_lib", "libfa_gb300.so")

STATUS = {
    0: "FA_OK", 1: "FA_ERR_NULL", 2: "FA_ERR_ALIGN", 3: "FA_ERR_SHAPE", 4: "FA_ERR_HEADDIM",
    5: "FA_ERR_CAUSAL_SHAPE", 6: "FA_ERR_LAUNCH", 7: "FA_ERR_DEVICE", 8: "FA_ERR_TIMEOUT",
    9: "FA_ERR_SCALE", 10: "FA_ERR_POINTER", 11: "FA_ERR_WORKSPACE",
    12: "FA_ERR_PAGE", 13: "FA_ERR_STRIDE",
}

NOALLOC_SCRATCH_BYTES = 16 << 20  # FA_NOALLOC_SCRATCH_BYTES in include/fa.h

_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, where: str = "fa_fwd"):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({fa_strerror(status)})")


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libfa_gb300.so (built by ``build.py`` / ``__graft_entry__.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is missing: build it with "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i32 = ctypes.c_void_p, ctypes.c_int
        lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_float, i32, vp]
        lib.fa_fwd.restype = i32
        lib.fa_strerror.argtypes = [i32]
        lib.fa_strerror.restype = ctypes.c_char_p
        lib.fa_version.argtypes = []
        lib.fa_version.restype = i32
        lib.fa_fwd_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint), i32]
        lib.fa_fwd_status.restype = i32
        lib.fa_probe_exp2.argtypes = [i32, ctypes.POINTER(ctypes.c_double), vp]
        lib.fa_probe_exp2.restype = i32
        lib.fa_selftest_wait.argtypes = [i32, ctypes.POINTER(ctypes.c_uint), ctypes.POINTER(ctypes.c_ulonglong), vp]
        lib.fa_selftest_wait.restype = i32
        lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_float, i32, i32, vp,
                                       ctypes.c_size_t, vp]
        lib.fa_fwd_splitkv.restype = i32
        lib.fa_splitkv_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.fa_splitkv_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_splitkv_heuristic.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.fa_splitkv_heuristic.restype = i32
        lib.fa_fwd_splitkv_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_float, i32,
                                               i32, vp]
        lib.fa_fwd_splitkv_noalloc.restype = i32
        lib.fa_fwd_window.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_float, i32, i32, vp]
        lib.fa_fwd_window.restype = i32
        lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_float, i32, vp,
                               ctypes.c_size_t, vp]
        lib.fa_bwd.restype = i32
        lib.fa_bwd_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_float, i32,
                                      i32, vp, ctypes.c_size_t, vp]
        lib.fa_bwd_window.restype = i32
        lib.fa_bwd_workspace_bytes.argtypes = [i32, i32, i32]
        lib.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
        i64 = ctypes.c_longlong
        lib.fa_rope.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, vp, i32, i32, i32, i32, i32, i32, ctypes.c_float,
                                i32, i32, vp]
        lib.fa_rope.restype = i32
        lib.fa_kv_append.argtypes = [vp] * 11 + [i32] * 9 + [i64, ctypes.c_float, i32, vp]
        lib.fa_kv_append.restype = i32
        lib.fa_fwd_paged.argtypes = [vp] * 9 + [i32] * 8 + [ctypes.c_float, i32, i32, vp, ctypes.c_size_t, vp]
        lib.fa_fwd_paged.restype = i32
        lib.fa_fwd_prefix.argtypes = [vp] * 6 + [i32] + [vp] * 4 + [i32] * 8 + [ctypes.c_float, vp, ctypes.c_size_t,
                                                                               vp]
        lib.fa_fwd_prefix.restype = i32
        lib.fa_paged_workspace_bytes.argtypes = [i32] * 6
        lib.fa_paged_workspace_bytes.restype = ctypes.c_size_t
        _lib = lib
    return _lib


def fa_strerror(status: int) -> str:
    return load().fa_strerror(int(status)).decode()


def fa_version() -> int:
    return int(load().fa_version())


def fa_fwd(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, stream) -> int:
    """Raw C-ABI call with integer device pointers and a raw stream handle.

    Returns the status code (0 = FA_OK); does not raise.
    """
    return int(load().fa_fwd(q, k, v, o, lse, int(B), int(H), int(Nq), int(Nk), int(d), float(scale),
                             int(causal), stream))


def fa_fwd_window(q, k, v, o, lse, B, H, Nq, Nk, d, scale, window_left, window_right, stream) -> int:
    """Raw C-ABI sliding-window call (bottom-right aligned, -1 = unbounded); returns the status code."""
    return int(load().fa_fwd_window(q, k, v, o, lse, int(B), int(H), int(Nq), int(Nk), int(d), float(scale),
                                    int(window_left), int(window_right), stream))


def fa_fwd_splitkv(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, n_splits, workspace, workspace_bytes,
                   stream) -> int:
    """Raw C-ABI split-KV call; returns the status code (does not raise)."""
    return int(load().fa_fwd_splitkv(q, k, v, o, lse, int(B), int(H), int(Nq), int(Nk), int(d), float(scale),
                                     int(causal), int(n_splits), workspace, int(workspace_bytes), stream))


def fa_fwd_splitkv_noalloc(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, n_splits, stream) -> int:
    """Raw C-ABI split-KV call that allocates nothing (the library's fixed
    device array holds the slice buffers); returns the status code.

    For callers that cannot allocate device memory themselves.  Calls that
    overlap on the GPU share that array and must be serialised by the caller.
    """
    return int(load().fa_fwd_splitkv_noalloc(q, k, v, o, lse, int(B), int(H), int(Nq), int(Nk), int(d),
                                             float(scale), int(causal), int(n_splits), stream))


def fa_splitkv_workspace_bytes(B, H, Nq, Nk, d, n_splits) -> int:
    return int(load().fa_splitkv_workspace_bytes(int(B), int(H), int(Nq), int(Nk), int(d), int(n_splits)))


def fa_splitkv_heuristic(B, H, Nq, Nk, d, causal) -> int:
    return int(load().fa_splitkv_heuristic(int(B), int(H), int(Nq), int(Nk), int(d), int(causal)))


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H, Nq, Nk, d, scale, causal, workspace, workspace_bytes,
           stream) -> int:
    """Raw C-ABI backward call; returns the status code (does not raise)."""
    return int(load().fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, int(B), int(H), int(Nq), int(Nk), int(d),
                             float(scale), int(causal), workspace, int(workspace_bytes), stream))


def fa_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, B, H, Nq, Nk, d, scale, window_left, window_right, workspace,
                  workspace_bytes, stream) -> int:
    """Raw C-ABI sliding-window backward call (bottom-right aligned, -1 = unbounded); returns the status code."""
    return int(load().fa_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, int(B), int(H), int(Nq), int(Nk), int(d),
                                    float(scale), int(window_left), int(window_right), workspace,
                                    int(workspace_bytes), stream))


def fa_bwd_workspace_bytes(B, H, Nq) -> int:
    return int(load().fa_bwd_workspace_bytes(int(B), int(H), int(Nq)))


def _longs(values):
    """A host array of long long for a strides argument (None stays None)."""
    return None if values is None else (ctypes.c_longlong * len(values))(*values)


def fa_rope(q, k, q_out, k_out, inv_freq, positions, position_stride, offset, strides, B, H, Hk, N, d, rot, mag,
            interleaved, backward, stream) -> int:
    """Raw C-ABI rotary call (``strides``: 12 integers or None); returns the status code."""
    return load().fa_rope(q, k, q_out, k_out, inv_freq, positions, position_stride, offset, _longs(strides), B, H, Hk,
                          N, d, rot, mag, interleaved, backward, stream)


def fa_kv_append(q, k, v, q_out, k_cache, v_cache, inv_freq, block_table, seq_lens, new_lens, strides, B, H, Hk, T, d,
                 rot, n_pages, page_size, max_pages, offset, mag, interleaved, stream) -> int:
    """Raw C-ABI append to the paged cache (``strides``: 18 integers); returns the status code."""
    return load().fa_kv_append(q, k, v, q_out, k_cache, v_cache, inv_freq, block_table, seq_lens, new_lens,
                               _longs(strides), B, H, Hk, T, d, rot, n_pages, page_size, max_pages, offset, mag,
                               interleaved, stream)


def fa_fwd_paged(q, k_cache, v_cache, o, lse, block_table, seq_lens, new_lens, strides, B, H, Hk, T, d, n_pages,
                 page_size, max_pages, scale, window_left, window_right, workspace, workspace_bytes, stream) -> int:
    """Raw C-ABI attention over the paged cache (``strides``: 6 integers); returns the status code."""
    return load().fa_fwd_paged(q, k_cache, v_cache, o, lse, block_table, seq_lens, new_lens, _longs(strides), B, H,
                               Hk, T, d, n_pages, page_size, max_pages, scale, window_left, window_right, workspace,
                               workspace_bytes, stream)


def fa_fwd_prefix(q, k_cache, v_cache, o, lse, prefix_pages, prefix_len, block_table, seq_lens, new_lens, strides, B,
                  H, Hk, T, d, n_pages, page_size, max_pages, scale, workspace, workspace_bytes, stream) -> int:
    """Raw C-ABI shared-prefix attention (``strides``: 6 integers); returns the status code."""
    return load().fa_fwd_prefix(q, k_cache, v_cache, o, lse, prefix_pages, prefix_len, block_table, seq_lens, new_lens,
                                _longs(strides), B, H, Hk, T, d, n_pages, page_size, max_pages, scale, workspace,
                                workspace_bytes, stream)


def fa_paged_workspace_bytes(B, H, Hk, T, d, prefix_len) -> int:
    return int(load().fa_paged_workspace_bytes(int(B), int(H), int(Hk), int(T), int(d), int(prefix_len)))


def fa_fwd_status(stream=None, clear: bool = False):
    """(status, raw device status word) after synchronising ``stream``."""
    word = ctypes.c_uint(0)
    st = int(load().fa_fwd_status(stream, ctypes.byref(word), int(bool(clear))))
    return st, int(word.value)


def fa_probe_exp2(method: int = 0, stream=None) -> float:
    """2^x results per SM clock: method 0 ex2.approx (special-function unit), 1 cubic polynomial on the
    FMA pipes.  Synchronises ``stream``."""
    rate = ctypes.c_double(0.0)
    st = int(load().fa_probe_exp2(int(method), ctypes.byref(rate), stream))
    if st != 0:
        raise FaError(st, "fa_probe_exp2")
    return float(rate.value)


def fa_selftest_wait(mode: int, stream=None):
    """Run the bounded-wait self-test (0: time limit, 1: abort flag); returns (status word, wait ns)."""
    word, ns = ctypes.c_uint(0), ctypes.c_ulonglong(0)
    st = int(load().fa_selftest_wait(int(mode), ctypes.byref(word), ctypes.byref(ns), stream))
    if st != 0:
        raise FaError(st, "fa_selftest_wait")
    return int(word.value), int(ns.value)


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None, stream=None,
        n_splits: int | None = None, workspace=None, window: tuple | None = None):
    """O = softmax(q k^T * scale) v and the per-row LSE, on the GPU.

    q: [B, H, Nq, d], k, v: [B, H, Nk, d] torch.bfloat16 CUDA tensors,
    contiguous.  ``scale`` defaults to 1/sqrt(d).  ``out`` (bf16 [B,H,Nq,d])
    and ``lse`` (fp32 [B,H,Nq]) may be given to avoid allocation.  Runs on
    ``stream`` (default: the current torch stream), asynchronously.

    ``n_splits``: K/V slices per query tile (split-KV, for shapes with too few
    query tiles to fill the GPU); None asks the library's heuristic, 1 forces
    the single-pass kernel.  ``workspace`` (a CUDA tensor of at least
    ``fa_splitkv_workspace_bytes`` bytes) may be given to avoid allocating it.

    ``window=(left, right)``: sliding-window mask aligned bottom-right (key j
    visible to row i iff i+Nk-Nq-left <= j <= i+Nk-Nq+right, -1 = unbounded);
    replaces ``causal`` and runs the single-pass kernel.
    """
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA torch.bfloat16 tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, H, N, d] tensor")
    B, H, Nq, d = q.shape
    if k.shape[:2] != (B, H) or k.shape[3] != d or v.shape != k.shape:
        raise ValueError(f"shape mismatch: q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    Nk = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor shaped like q")
    if lse.shape != (B, H, Nq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, Nq] tensor")
    if window is not None:
        st = fa_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Nq, Nk,
                           d, scale, int(window[0]), int(window[1]), _stream_handle(stream))
        if st != 0:
            raise FaError(st, "fa_fwd_window")
        return out, lse
    if n_splits is None:
        n_splits = fa_splitkv_heuristic(B, H, Nq, Nk, d, int(bool(causal))) if Nq > 0 else 1
    if n_splits > 1:
        need = fa_splitkv_workspace_bytes(B, H, Nq, Nk, d, n_splits)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        if not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"workspace must be a CUDA tensor of at least {need} bytes")
        st = fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Nq,
                            Nk, d, scale, int(bool(causal)), n_splits, workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), _stream_handle(stream))
        if st != 0:
            raise FaError(st, "fa_fwd_splitkv")
        return out, lse
    st = fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Nq, Nk, d,
                scale, int(bool(causal)), _stream_handle(stream))
    if st != 0:
        raise FaError(st)
    return out, lse


def bwd(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None, dq=None, dk=None, dv=None,
        workspace=None, stream=None, window: tuple | None = None):
    """(dq, dk, dv) of attention by recomputation from the forward's ``lse``.

    q, o, dout: [B, H, Nq, d]; k, v: [B, H, Nk, d], CUDA bf16, contiguous;
    lse: fp32 [B, H, Nq] from ``fwd``.  ``workspace`` (CUDA tensor of at least
    ``fa_bwd_workspace_bytes`` bytes) may be given to avoid allocating it.
    ``window=(left, right)``: the sliding-window mask of ``fwd(window=...)``
    (pass the same window to both; ``causal`` is then ignored).
    """
    import torch

    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous CUDA torch.bfloat16 tensor")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if o.shape != q.shape or dout.shape != q.shape or v.shape != k.shape or k.shape[:2] != (B, H) or k.shape[3] != d:
        raise ValueError("shape mismatch")
    if lse.shape != (B, H, Nq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, Nq] tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if (not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda or
                not t.is_contiguous() or t.shape != like.shape):
            raise ValueError(f"{name} must be a contiguous CUDA bf16 tensor shaped like {tuple(like.shape)}")
    need = fa_bwd_workspace_bytes(B, H, Nq)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if window is not None:
        st = fa_bwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                           dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Nq, Nk, d, scale, int(window[0]),
                           int(window[1]), workspace.data_ptr(), ws_bytes, _stream_handle(stream))
        if st != 0:
            raise FaError(st, "fa_bwd_window")
        return dq, dk, dv
    st = fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Nq, Nk, d, scale, int(bool(causal)),
                workspace.data_ptr(), ws_bytes, _stream_handle(stream))
    if st != 0:
        raise FaError(st, "fa_bwd")
    return dq, dk, dv


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rope_freqs(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               original_len: int = 4096, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(inv_freq, mag) for ``rope`` and ``kv_append``: fp64 [rot / 2] radians per position, and the factor on
    the rotated part.

    ``scaling`` for contexts ``factor`` times longer than trained on:
    ``"linear"``: every frequency divided by ``factor``;
    ``"base"``: the base stretched by factor^(rot / (rot - 2)), which divides the slowest frequency by
    ``factor`` and keeps the fastest;
    ``"by_parts"``: pairs that turn at least ``fast`` times within ``original_len`` positions keep their
    frequency, pairs below ``slow`` turns are divided by ``factor``, with a linear ramp in the number of turns
    between, and mag = 0.1 ln(factor) + 1.
    """
    import torch

    if rot < 2 or rot % 2:
        raise ValueError("rot must be a positive even number")
    if not (math.isfinite(base) and base > 0 and math.isfinite(factor) and factor >= 1):
        raise ValueError("base must be finite and > 0, factor finite and >= 1")
    expo = -torch.arange(0, rot, 2, dtype=torch.float64) / rot
    if scaling == "base":
        if rot < 4:
            raise ValueError("a stretched base needs rot >= 4")
        base = base * factor ** (rot / (rot - 2))
    w = torch.full_like(expo, base).pow(expo)
    mag = 1.0
    if scaling == "linear":
        w = w / factor
    elif scaling == "by_parts":
        if not (original_len > 0 and fast > slow >= 0):
            raise ValueError("by_parts needs original_len > 0 and fast > slow >= 0")
        turns = original_len * w / (2.0 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        w = w * keep + (w / factor) * (1.0 - keep)
        mag = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return w.to(device), mag


def _empty(shape, dtype, like, stream):
    """Memory that ``stream`` may write at once: from its own allocator pool when it is not the current stream."""
    import torch

    if stream is None or stream == torch.cuda.current_stream(like.device):
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _handle(stream, like):
    import torch

    return (torch.cuda.current_stream(like.device) if stream is None else stream).cuda_stream


def _need(name, t, dtype, dim=None):
    import torch

    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA {dtype} tensor")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, has {t.dim()}")


def _strides3(name, t):
    """Strides of a 4-D view's first three dimensions; a dimension of size 1 gets a stride that is valid anywhere."""
    n0, n1, n2, d = t.shape
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 and t.numel():
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return (s0 if n0 > 1 else d, s1 if n1 > 1 else d, s2 if n2 > 1 else d)


def _rope_like(name, t, out, stream):
    """``out`` or a new contiguous tensor shaped like the bf16 [B, heads, N, d] view ``t``."""
    import torch

    if out is None:
        return _empty(t.shape, torch.bfloat16, t, stream)
    _need(name, out, torch.bfloat16, 4)
    if out.shape != t.shape:
        raise ValueError(f"{name} must be shaped like its input, {tuple(t.shape)}")
    return out


def _rope(where, backward, q, k, inv_freq, positions, offset, interleaved, mag, q_out, k_out, stream):
    import torch

    _need("q", q, torch.bfloat16, 4)
    B, H, N, d = q.shape
    _need("inv_freq", inv_freq, torch.float64, 1)
    if not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be contiguous")
    Hk = 0
    if k is not None:
        _need("k", k, torch.bfloat16, 4)
        Hk = k.shape[1]
        if k.shape[0] != B or k.shape[2] != N or k.shape[3] != d or Hk == 0:
            raise ValueError(f"shape mismatch: q{tuple(q.shape)} k{tuple(k.shape)}")
    elif k_out is not None:
        raise ValueError("k_out without k")
    p_stride = 0
    if positions is not None:
        _need("positions", positions, torch.int32)
        if positions.shape == (B, N):
            p_stride = positions.stride(0) if B > 1 else 0
        elif positions.shape != (N,):
            raise ValueError(f"positions must be [{B}, {N}] or [{N}], is {tuple(positions.shape)}")
        if N > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous along the last dimension")
    q_out = _rope_like("q_out", q, q_out, stream)
    k_out = _rope_like("k_out", k, k_out, stream) if Hk else None
    strides = None
    if not (q.is_contiguous() and q_out.is_contiguous() and (not Hk or (k.is_contiguous() and k_out.is_contiguous()))):
        none = (d, d, d)
        strides = (_strides3("q", q) + (_strides3("k", k) if Hk else none) + _strides3("q_out", q_out) +
                   (_strides3("k_out", k_out) if Hk else none))
    st = fa_rope(q.data_ptr(), k.data_ptr() if Hk else None, q_out.data_ptr(), k_out.data_ptr() if Hk else None,
                 inv_freq.data_ptr(), None if positions is None else positions.data_ptr(), p_stride, offset, strides,
                 B, H, Hk, N, d, 2 * inv_freq.shape[0], mag, int(interleaved), backward, _handle(stream, q))
    if st != 0:
        raise FaError(st, where)
    return q_out, k_out


def rope(q, k, inv_freq, positions=None, offset: int = 0, interleaved: bool = False, mag: float = 1.0, q_out=None,
         k_out=None, stream=None):
    """(q, k) turned by their positions, ready for ``fwd``; ``k`` may be None and may have fewer heads.

    q: [B, H, N, d], k: [B, Hk, N, d] CUDA bf16, d contiguous and the other strides free (multiples of 8
    elements), so views of a packed projection need no copy; the outputs default to contiguous tensors and may
    be the inputs themselves.  ``inv_freq``: fp64 [rot / 2] on the GPU (``rope_freqs``); the first rot elements
    of a head turn, the others are copied.  ``positions``: int32 [B, N] or [N]; None: 0, 1, 2, ...;
    ``offset`` is added.  ``interleaved``: pairs (2i, 2i + 1) instead of (i, i + rot / 2).  ``mag`` multiplies
    the turned part.
    """
    return _rope("fa_rope", 0, q, k, inv_freq, positions, offset, interleaved, mag, q_out, k_out, stream)


def rope_bwd(dq, dk, inv_freq, positions=None, offset: int = 0, interleaved: bool = False, mag: float = 1.0,
             q_out=None, k_out=None, stream=None):
    """Gradients of ``rope``'s inputs from those of its outputs (from ``bwd``): the transposed rotation, same
    arguments; ``q_out`` and ``k_out`` may be views of a packed gradient."""
    return _rope("fa_rope", 1, dq, dk, inv_freq, positions, offset, interleaved, mag, q_out, k_out, stream)


# ---------------------------------------------------------------------------
# the paged K/V cache
# ---------------------------------------------------------------------------
def _cache_args(k_cache, v_cache, block_table, seq_lens, new_lens, B, d):
    """Checks shared by the cache's calls; the strides of both caches."""
    import torch

    _need("k_cache", k_cache, torch.bfloat16, 4)
    _need("v_cache", v_cache, torch.bfloat16, 4)
    if v_cache.shape != k_cache.shape or k_cache.shape[3] != d:
        raise ValueError(f"shape mismatch: k_cache{tuple(k_cache.shape)} v_cache{tuple(v_cache.shape)}, d = {d}")
    _need("block_table", block_table, torch.int32, 2)
    _need("seq_lens", seq_lens, torch.int32, 1)
    if block_table.shape[0] != B or not block_table.is_contiguous():
        raise ValueError(f"block_table must be a contiguous [{B}, max_pages] tensor")
    if seq_lens.shape[0] != B or not seq_lens.is_contiguous():
        raise ValueError(f"seq_lens must be a contiguous [{B}] tensor")
    if new_lens is not None:
        _need("new_lens", new_lens, torch.int32, 1)
        if new_lens.shape[0] != B or not new_lens.is_contiguous():
            raise ValueError(f"new_lens must be a contiguous [{B}] tensor")
    return _strides3("k_cache", k_cache) + _strides3("v_cache", v_cache)


def kv_append(q, k, v, k_cache, v_cache, block_table, seq_lens, inv_freq=None, new_lens=None, offset: int = 0,
              interleaved: bool = False, mag: float = 1.0, q_out=None, stream=None):
    """Put the new tokens' k (turned by position) and v into the paged cache and return their q, turned.

    q: [B, H, T, d] or None; k, v: [B, Hk, T, d] CUDA bf16, d contiguous, other strides free.
    k_cache, v_cache: [n_pages, Hk, page_size, d] views, page_size 16..256 (a power of two), d contiguous;
    token-major pages are ``pages.transpose(1, 2)``.  block_table: int32 [B, max_pages].  seq_lens: int32 [B],
    each sequence's cached tokens WITH the new ones; new_lens: int32 [B], how many of the T rows are tokens
    (None: all).  Row t is the token at own position seq_lens - new_lens + t; its rotation uses ``offset`` + that
    (``inv_freq`` None: no rotation).  Padding rows are not written (q_out included).  Asynchronous; a page index
    outside the cache is skipped and reported by ``fa_fwd_status``.
    """
    import torch

    _need("k", k, torch.bfloat16, 4)
    _need("v", v, torch.bfloat16, 4)
    B, Hk, T, d = k.shape
    if v.shape != k.shape:
        raise ValueError(f"shape mismatch: k{tuple(k.shape)} v{tuple(v.shape)}")
    caches = _cache_args(k_cache, v_cache, block_table, seq_lens, new_lens, B, d)
    if k_cache.shape[1] != Hk:
        raise ValueError(f"the cache has {k_cache.shape[1]} heads, k has {Hk}")
    H = 0
    qs = os_ = (d, d, d)
    if q is not None:
        _need("q", q, torch.bfloat16, 4)
        H = q.shape[1]
        if q.shape[0] != B or q.shape[2] != T or q.shape[3] != d or H == 0:
            raise ValueError(f"shape mismatch: q{tuple(q.shape)} k{tuple(k.shape)}")
        q_out = _rope_like("q_out", q, q_out, stream)
        qs, os_ = _strides3("q", q), _strides3("q_out", q_out)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot = 0
    if inv_freq is not None:
        _need("inv_freq", inv_freq, torch.float64, 1)
        if not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be contiguous")
        rot = 2 * inv_freq.shape[0]
    st = fa_kv_append(q.data_ptr() if H else None, k.data_ptr(), v.data_ptr(), q_out.data_ptr() if H else None,
                      k_cache.data_ptr(), v_cache.data_ptr(), inv_freq.data_ptr() if rot else None,
                      block_table.data_ptr(), seq_lens.data_ptr(), None if new_lens is None else new_lens.data_ptr(),
                      qs + _strides3("k", k) + _strides3("v", v) + os_ + caches, B, H, Hk, T, d, rot,
                      k_cache.shape[0], k_cache.shape[2], block_table.shape[1], offset, mag, int(interleaved),
                      _handle(stream, k))
    if st != 0:
        raise FaError(st, "fa_kv_append")
    return q_out


def _paged_args(q, k_cache, v_cache, block_table, seq_lens, new_lens, scale, out, lse, workspace, stream, prefix_len):
    import torch

    _need("q", q, torch.bfloat16, 4)
    if not q.is_contiguous():
        raise ValueError("q must be a contiguous [B, H, T, d] tensor")
    B, H, T, d = q.shape
    strides = _cache_args(k_cache, v_cache, block_table, seq_lens, new_lens, B, d)
    if out is None:
        out = _empty(q.shape, torch.bfloat16, q, stream)
    elif out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_cuda or not out.is_contiguous():
        raise ValueError("out must be a contiguous CUDA bf16 tensor shaped like q")
    if lse is None:
        lse = _empty((B, H, T), torch.float32, q, stream)
    elif lse.shape != (B, H, T) or lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous CUDA fp32 [B, H, T] tensor")
    if workspace is None:
        need = load().fa_paged_workspace_bytes(B, H, k_cache.shape[1], T, d, prefix_len)
        workspace = _empty((need,), torch.uint8, q, stream)
        ws_bytes = need
    else:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_bytes = workspace.numel() * workspace.element_size()
    dims = (B, H, k_cache.shape[1], T, d, k_cache.shape[0], k_cache.shape[2], block_table.shape[1])
    return out, lse, workspace, ws_bytes, strides, dims, 1.0 / math.sqrt(d) if scale is None else scale


def fwd_paged(q, k_cache, v_cache, block_table, seq_lens, scale: float | None = None, new_lens=None,
              window: tuple = (-1, 0), out=None, lse=None, workspace=None, stream=None):
    """(O, LSE) of the new tokens' queries over their sequences' cached keys.

    q: [B, H, T, d] contiguous CUDA bf16 (as ``kv_append`` returns it), T from 1 (decoding) to a prompt's chunk;
    H a multiple of the cache's heads (query head h reads K/V head h // (H / Hk)).  The cache, block_table,
    seq_lens (with the new tokens) and new_lens as in ``kv_append``.  ``window=(left, right)`` as in ``fwd``,
    around the token's own position: (-1, 0) is causal, (-1, -1) every cached key.  Padding rows and rows
    that see no key get O = 0 and LSE = -inf.  The lengths are read on the GPU, so a captured call stays
    right as they grow.  ``workspace`` (``fa_paged_workspace_bytes(B, H, Hk, T, d, 0)`` bytes) may be given; calls
    that may overlap need one each.
    """
    out, lse, workspace, ws_bytes, strides, dims, scale = _paged_args(
        q, k_cache, v_cache, block_table, seq_lens, new_lens, scale, out, lse, workspace, stream, 0)
    st = fa_fwd_paged(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), lse.data_ptr(),
                      block_table.data_ptr(), seq_lens.data_ptr(), None if new_lens is None else new_lens.data_ptr(),
                      strides, *dims, scale, window[0], window[1], workspace.data_ptr(), ws_bytes, _handle(stream, q))
    if st != 0:
        raise FaError(st, "fa_fwd_paged")
    return out, lse


def fwd_prefix(q, k_cache, v_cache, prefix_pages, prefix_len: int, block_table, seq_lens, scale: float | None = None,
               new_lens=None, out=None, lse=None, workspace=None, stream=None):
    """(O, LSE) of ``fwd_paged`` (causal) for sequences that all begin with the same ``prefix_len`` tokens, whose
    K and V (``prefix_pages``: int32 page indices, in the same cache) are read once for the whole batch.

    block_table and seq_lens describe the sequences' own tokens after the prefix (``kv_append`` with
    ``offset=prefix_len`` puts them there).  An entry with seq_lens <= 0 is empty: O = 0, LSE = -inf.
    ``workspace``: ``fa_paged_workspace_bytes(B, H, Hk, T, d, prefix_len)`` bytes.
    """
    import torch

    _need("prefix_pages", prefix_pages, torch.int32, 1)
    if prefix_len <= 0:
        raise ValueError("prefix_len must be > 0 (without a prefix: fwd_paged)")
    out, lse, workspace, ws_bytes, strides, dims, scale = _paged_args(
        q, k_cache, v_cache, block_table, seq_lens, new_lens, scale, out, lse, workspace, stream, prefix_len)
    if not prefix_pages.is_contiguous() or prefix_pages.shape[0] * dims[6] < prefix_len:
        raise ValueError(f"prefix_pages must be contiguous and hold {prefix_len} tokens of {dims[6]} to a page")
    st = fa_fwd_prefix(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), lse.data_ptr(),
                       prefix_pages.data_ptr(), prefix_len, block_table.data_ptr(), seq_lens.data_ptr(),
                       None if new_lens is None else new_lens.data_ptr(), strides, *dims, scale, workspace.data_ptr(),
                       ws_bytes, _handle(stream, q))
    if st != 0:
        raise FaError(st, "fa_fwd_prefix")
    return out, lse
