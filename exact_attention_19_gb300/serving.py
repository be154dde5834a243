"""Rotary positions and the paged K/V cache on torch tensors: ``rope_freqs``,
``rope``, ``rope_bwd``, ``kv_append``, ``fwd_paged``, ``fwd_prefix`` (re-exported by
the package).

Argument checks and marshalling only; the kernels do the work.  A decoding step
makes these calls for a few microseconds of GPU work each, so the usual case
(everything in order, the current stream) goes through ``fa_torch`` (C++, the same
checks); what that does not take comes to the code here, which also raises the
errors.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import math
import os
import struct

import torch

from . import FaError, load
from .build import torch_lib_path

_BF16, _F32, _F64, _I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
_Tensor = torch.Tensor
_pack6, _pack12, _pack18 = (struct.Struct(f"{n}q").pack for n in (6, 12, 18))
_raw_stream = torch._C._cuda_getCurrentRawStream


def _load_native():
    """The fa_torch module, bound to the loaded library's functions."""
    path = torch_lib_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    loader = importlib.machinery.ExtensionFileLoader("fa_torch", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("fa_torch", path, loader=loader))
    loader.exec_module(module)
    lib = load()
    module.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                  for f in ("fa_rope", "fa_kv_append", "fa_fwd_paged", "fa_fwd_prefix", "fa_paged_workspace_bytes")))
    return module


_native = _load_native()
_native_rope, _native_append, _native_paged = _native.rope, _native.kv_append, _native.paged


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
    if rot < 2 or rot % 2:
        raise ValueError("rot must be a positive even number")
    if not (math.isfinite(base) and base > 0 and math.isfinite(factor) and factor >= 1):
        raise ValueError("base must be finite and > 0, factor finite and >= 1")
    expo = -torch.arange(0, rot, 2, dtype=_F64) / rot
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


def _c_int(name, value, bits):
    """``value`` for a C integer of ``bits`` bits, which ctypes would cut to them without a word."""
    if not -(1 << (bits - 1)) <= value < 1 << (bits - 1):
        raise ValueError(f"{name} = {value} does not fit {bits} bits")
    return value


def _reach(name, value):
    """One side of a window: past 2^31 - 1 it is open whatever its size, as no cache holds so many keys."""
    return _c_int(name, min(value, (1 << 31) - 1), 32)


def _need(name, t, dtype, dim):
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA {dtype} tensor")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, has {t.dim()}")


def _empty(shape, dtype, like, stream):
    """Memory that ``stream`` may write at once: from its own allocator pool when it is not the current stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _handle(stream, like):
    return _raw_stream(like.get_device()) if stream is None else stream.cuda_stream


def _strides3(name, t, shape):
    """Strides of a 4-D view's first three dimensions; a dimension of size 1 gets a stride that is valid anywhere."""
    s0, s1, s2, s3 = t.stride()
    n0, n1, n2, d = shape
    if s3 != 1 and n0 * n1 * n2:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return (s0 if n0 > 1 else d, s1 if n1 > 1 else d, s2 if n2 > 1 else d)


def _rope_like(name, t, shape, out, stream):
    """``out`` or a new contiguous tensor shaped like the bf16 [B, heads, N, d] view ``t``."""
    if out is None:
        return _empty(shape, _BF16, t, stream)
    _need(name, out, _BF16, 4)
    if out.shape != shape:
        raise ValueError(f"{name} must be shaped like its input, {tuple(shape)}")
    return out


def _rot(inv_freq):
    _need("inv_freq", inv_freq, _F64, 1)
    if not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be contiguous")
    return 2 * inv_freq.shape[0]


def _rope(backward, q, k, inv_freq, positions, offset, interleaved, mag, q_out, k_out, stream):
    if stream is None:
        done = _native_rope(backward, q, k, inv_freq, positions, offset, interleaved, mag, q_out, k_out)
        if done is not None:
            return done
    offset = _c_int("offset", offset, 64)
    _need("q", q, _BF16, 4)
    q_shape = q.shape
    B, H, N, d = q_shape
    rot = _rot(inv_freq)
    Hk = 0
    if k is not None:
        _need("k", k, _BF16, 4)
        k_shape = k.shape
        Hk = k_shape[1]
        if Hk == 0 or k_shape != (B, Hk, N, d):
            raise ValueError(f"shape mismatch: q{tuple(q_shape)} k{tuple(k_shape)}")
    elif k_out is not None:
        raise ValueError("k_out without k")
    p_ptr, p_stride = None, 0
    if positions is not None:
        if not (isinstance(positions, _Tensor) and positions.dtype is _I32 and positions.is_cuda):
            raise TypeError("positions must be a CUDA torch.int32 tensor")
        if positions.shape == (B, N):
            p_stride = positions.stride(0) if B > 1 else 0
        elif positions.shape != (N,):
            raise ValueError(f"positions must be [{B}, {N}] or [{N}], is {tuple(positions.shape)}")
        if N > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous along the last dimension")
        p_ptr = positions.data_ptr()
    q_out = _rope_like("q_out", q, q_shape, q_out, stream)
    none = (d, d, d)
    if Hk:
        k_out = _rope_like("k_out", k, k_shape, k_out, stream)
        k_ptr, ko_ptr = k.data_ptr(), k_out.data_ptr()
        ks, ko = _strides3("k", k, k_shape), _strides3("k_out", k_out, k_shape)
    else:
        k_ptr = ko_ptr = None
        ks = ko = none
    strides = _pack12(*_strides3("q", q, q_shape), *ks, *_strides3("q_out", q_out, q_shape), *ko)
    st = load().fa_rope(q.data_ptr(), k_ptr, q_out.data_ptr(), ko_ptr, inv_freq.data_ptr(), p_ptr, p_stride, offset,
                        strides, B, H, Hk, N, d, rot, mag, bool(interleaved), backward, _handle(stream, q))
    if st != 0:
        raise FaError(st, "fa_rope")
    return q_out, k_out


def rope(q, k, inv_freq, positions=None, offset: int = 0, interleaved: bool = False, mag: float = 1.0, q_out=None,
         k_out=None, stream=None):
    """(q, k) turned by their positions, ready for ``fwd``; ``k`` may be None and may have fewer heads.

    q: [B, H, N, d], k: [B, Hk, N, d] CUDA bf16, d contiguous and the other strides free (multiples of 8
    elements), so views of a packed projection need no copy; the outputs default to contiguous tensors and may
    be the inputs themselves.  ``inv_freq``: fp64 [rot / 2] on the GPU (``rope_freqs``); the first rot elements
    of a head turn, the others are copied.  ``positions``: int32 [B, N] or [N]; None: 0, 1, 2, ...;
    ``offset`` is added.  ``interleaved``: pairs (2i, 2i + 1) instead of (i, i + rot / 2).  ``mag`` multiplies
    the turned part.  Runs on ``stream`` (default: the current torch stream), asynchronously.  Records no
    autograd graph: ``rope_bwd`` turns the gradients back.
    """
    return _rope(False, q, k, inv_freq, positions, offset, interleaved, mag, q_out, k_out, stream)


def rope_bwd(dq, dk, inv_freq, positions=None, offset: int = 0, interleaved: bool = False, mag: float = 1.0,
             q_out=None, k_out=None, stream=None):
    """Gradients of ``rope``'s inputs from those of its outputs (from ``bwd``): the transposed rotation, same
    arguments; ``q_out`` and ``k_out`` may be views of a packed gradient."""
    return _rope(True, dq, dk, inv_freq, positions, offset, interleaved, mag, q_out, k_out, stream)


# ---------------------------------------------------------------------------
# the paged K/V cache
# ---------------------------------------------------------------------------
def _cache(k_cache, v_cache, block_table, seq_lens, new_lens, B, d):
    """Checks shared by the cache's calls: (shape, strides of both caches, max_pages, pointer of new_lens)."""
    _need("k_cache", k_cache, _BF16, 4)
    _need("v_cache", v_cache, _BF16, 4)
    shape = k_cache.shape
    if v_cache.shape != shape or shape[3] != d:
        raise ValueError(f"shape mismatch: k_cache{tuple(shape)} v_cache{tuple(v_cache.shape)}, d = {d}")
    _need("block_table", block_table, _I32, 2)
    _need("seq_lens", seq_lens, _I32, 1)
    rows, max_pages = block_table.shape
    if rows != B or not block_table.is_contiguous():
        raise ValueError(f"block_table must be a contiguous [{B}, max_pages] tensor")
    if seq_lens.shape[0] != B or not seq_lens.is_contiguous():
        raise ValueError(f"seq_lens must be a contiguous [{B}] tensor")
    new = None
    if new_lens is not None:
        _need("new_lens", new_lens, _I32, 1)
        if new_lens.shape[0] != B or not new_lens.is_contiguous():
            raise ValueError(f"new_lens must be a contiguous [{B}] tensor")
        new = new_lens.data_ptr()
    return shape, _strides3("k_cache", k_cache, shape) + _strides3("v_cache", v_cache, shape), max_pages, new


def kv_append(q, k, v, k_cache, v_cache, block_table, seq_lens, inv_freq=None, new_lens=None, offset: int = 0,
              interleaved: bool = False, mag: float = 1.0, q_out=None, stream=None):
    """Put the new tokens' k (turned by position) and v into the paged cache and return their q, turned.

    q: [B, H, T, d] or None; k, v: [B, Hk, T, d] CUDA bf16, d contiguous, other strides free.
    k_cache, v_cache: [n_pages, Hk, page_size, d] views, page_size 16..256 (a power of two), d contiguous;
    token-major pages are ``pages.transpose(1, 2)``.  block_table: int32 [B, max_pages].  seq_lens: int32 [B],
    each sequence's cached tokens WITH the new ones; new_lens: int32 [B], how many of the T rows are tokens
    (None: all).  Row t is the token at own position seq_lens - new_lens + t; its rotation uses ``offset`` + that
    (``inv_freq`` None: no rotation).  Padding rows are not written (q_out included).  Two tokens must not share
    a slot.  Asynchronous; a page index outside the cache is skipped and reported by ``fa_fwd_status``.
    """
    if stream is None:
        done = _native_append(q, k, v, k_cache, v_cache, block_table, seq_lens, inv_freq, new_lens, offset,
                              interleaved, mag, q_out)
        if done is not None:
            return done
    offset = _c_int("offset", offset, 64)
    _need("k", k, _BF16, 4)
    _need("v", v, _BF16, 4)
    k_shape = k.shape
    B, Hk, T, d = k_shape
    if v.shape != k_shape:
        raise ValueError(f"shape mismatch: k{tuple(k_shape)} v{tuple(v.shape)}")
    shape, caches, max_pages, new = _cache(k_cache, v_cache, block_table, seq_lens, new_lens, B, d)
    if shape[1] != Hk:
        raise ValueError(f"the cache has {shape[1]} heads, k has {Hk}")
    H = 0
    q_ptr = qo_ptr = None
    qs = qo = (d, d, d)
    if q is not None:
        _need("q", q, _BF16, 4)
        q_shape = q.shape
        H = q_shape[1]
        if H == 0 or q_shape != (B, H, T, d):
            raise ValueError(f"shape mismatch: q{tuple(q_shape)} k{tuple(k_shape)}")
        q_out = _rope_like("q_out", q, q_shape, q_out, stream)
        q_ptr, qo_ptr = q.data_ptr(), q_out.data_ptr()
        qs, qo = _strides3("q", q, q_shape), _strides3("q_out", q_out, q_shape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot, w_ptr = 0, None
    if inv_freq is not None:
        rot, w_ptr = _rot(inv_freq), inv_freq.data_ptr()
    strides = _pack18(*qs, *_strides3("k", k, k_shape), *_strides3("v", v, k_shape), *qo, *caches)
    st = load().fa_kv_append(q_ptr, k.data_ptr(), v.data_ptr(), qo_ptr, k_cache.data_ptr(), v_cache.data_ptr(), w_ptr,
                             block_table.data_ptr(), seq_lens.data_ptr(), new, strides, B, H, Hk, T, d, rot, shape[0],
                             shape[2], max_pages, offset, mag, bool(interleaved), _handle(stream, k))
    if st != 0:
        raise FaError(st, "fa_kv_append")
    return q_out


@functools.lru_cache(maxsize=256)
def _workspace_bytes(device, B, H, Hk, T, d, prefix_len):
    """fa_paged_workspace_bytes, a function of the sizes and the device alone."""
    with torch.cuda.device(device):
        return load().fa_paged_workspace_bytes(B, H, Hk, T, d, prefix_len)


def _paged_args(q, k_cache, v_cache, block_table, seq_lens, new_lens, scale, out, lse, workspace, stream, prefix_len):
    _need("q", q, _BF16, 4)
    if not q.is_contiguous():
        raise ValueError("q must be a contiguous [B, H, T, d] tensor")
    q_shape = q.shape
    B, H, T, d = q_shape
    shape, caches, max_pages, new = _cache(k_cache, v_cache, block_table, seq_lens, new_lens, B, d)
    if out is None:
        out = _empty(q_shape, _BF16, q, stream)
    elif out.shape != q_shape or out.dtype is not _BF16 or not out.is_cuda or not out.is_contiguous():
        raise ValueError("out must be a contiguous CUDA bf16 tensor shaped like q")
    if lse is None:
        lse = _empty((B, H, T), _F32, q, stream)
    elif lse.shape != (B, H, T) or lse.dtype is not _F32 or not lse.is_cuda or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous CUDA fp32 [B, H, T] tensor")
    Hk = shape[1]
    if Hk == 0 or H % Hk:
        raise ValueError(f"{H} query heads do not share {Hk} K/V heads evenly")
    if workspace is None:
        ws_bytes = _workspace_bytes(q.get_device(), B, H, Hk, T, d, prefix_len)
        workspace = _empty((ws_bytes,), torch.uint8, q, stream)
    else:
        if not isinstance(workspace, _Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_bytes = workspace.numel() * workspace.element_size()
    rest = (_pack6(*caches), B, H, Hk, T, d, shape[0], shape[2], max_pages,
            1.0 / math.sqrt(d) if scale is None else scale)
    return out, lse, workspace, ws_bytes, new, rest


def fwd_paged(q, k_cache, v_cache, block_table, seq_lens, scale: float | None = None, new_lens=None,
              window: tuple = (-1, 0), out=None, lse=None, workspace=None, stream=None):
    """(O, LSE) of the new tokens' queries over their sequences' cached keys.

    q: [B, H, T, d] contiguous CUDA bf16 (as ``kv_append`` returns it), T from 1 (decoding) to a prompt's chunk;
    H a multiple of the cache's heads (query head h reads K/V head h // (H / Hk)).  The cache, block_table,
    seq_lens (with the new tokens) and new_lens as in ``kv_append``.  ``window=(left, right)`` as in ``fwd``,
    around the token's own position: (-1, 0) is causal, (-1, -1) every cached key (an encoder's states: from
    rows at negative positions too).  Rows past new_lens and rows that see no key get O = 0 and LSE = -inf.  The lengths are read on the GPU, so a captured call stays
    right as they grow.  ``workspace`` (``fa_paged_workspace_bytes(B, H, Hk, T, d, 0)`` bytes) may be given; calls
    that may overlap need one each.  Runs on ``stream`` (default: the current torch stream), asynchronously.
    """
    if stream is None:
        done = _native_paged(q, k_cache, v_cache, None, 0, block_table, seq_lens, scale, new_lens, window[0], window[1],
                             out, lse, workspace)
        if done is not None:
            return done
    left, right = _reach("window[0]", window[0]), _reach("window[1]", window[1])
    out, lse, workspace, ws_bytes, new, rest = _paged_args(
        q, k_cache, v_cache, block_table, seq_lens, new_lens, scale, out, lse, workspace, stream, 0)
    st = load().fa_fwd_paged(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), lse.data_ptr(),
                             block_table.data_ptr(), seq_lens.data_ptr(), new, *rest, left, right,
                             workspace.data_ptr(), ws_bytes, _handle(stream, q))
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
    if stream is None and prefix_pages is not None:
        done = _native_paged(q, k_cache, v_cache, prefix_pages, prefix_len, block_table, seq_lens, scale, new_lens, -1,
                             0, out, lse, workspace)
        if done is not None:
            return done
    _need("prefix_pages", prefix_pages, _I32, 1)
    if _c_int("prefix_len", prefix_len, 32) <= 0:
        raise ValueError("prefix_len must be > 0 (without a prefix: fwd_paged)")
    out, lse, workspace, ws_bytes, new, rest = _paged_args(
        q, k_cache, v_cache, block_table, seq_lens, new_lens, scale, out, lse, workspace, stream, prefix_len)
    page = k_cache.shape[2]
    if not prefix_pages.is_contiguous() or prefix_pages.shape[0] * page < prefix_len:
        raise ValueError(f"prefix_pages must be contiguous and hold {prefix_len} tokens of {page} to a page")
    st = load().fa_fwd_prefix(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), lse.data_ptr(),
                              prefix_pages.data_ptr(), prefix_len, block_table.data_ptr(), seq_lens.data_ptr(), new,
                              *rest, workspace.data_ptr(), ws_bytes, _handle(stream, q))
    if st != 0:
        raise FaError(st, "fa_fwd_prefix")
    return out, lse
