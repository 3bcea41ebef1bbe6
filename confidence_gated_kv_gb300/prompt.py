"""Operators of a prompt's path: head norms with rotary positions, and packed
prompt attention (include/confkv.h: confkv_qk_rotary, confkv_prompt_attention).

Argument marshalling only, as in binding.py; layer-wise prefill and read-back
of a cache are methods of Cache.
"""
from __future__ import annotations

import ctypes
import math
import struct

from .binding import _check, _stream, dtype_code, lib, on_device

SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

_ROTARY = struct.Struct("=10i2f4Q8q4Q")
_PROMPT = struct.Struct("=8if4x7Q8q")


class Rotary:
    """Frequencies of a rotary embedding of the first `rot_dim` channels, kept
    on `device` (default: the current one).  scaling: "none", "linear", "ntk"
    or "yarn", for positions beyond the trained `original_length`; the formulas
    are with confkv_rotary_frequencies."""

    def __init__(self, rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original_length: float = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 interleaved: bool = False, device=None):
        import torch
        if scaling not in SCALINGS:
            raise ValueError("scaling is one of %s" % ", ".join(SCALINGS))
        self.rot_dim, self.interleaved = int(rot_dim), bool(interleaved)
        host = (ctypes.c_uint64 * max(1, self.rot_dim // 2))()
        mscale = ctypes.c_float()
        _check(lib().confkv_rotary_frequencies(self.rot_dim, float(base), SCALINGS[scaling], float(factor),
                                               float(original_length), float(beta_fast), float(beta_slow), host,
                                               ctypes.byref(mscale)), "confkv_rotary_frequencies")
        self.mscale = float(mscale.value)
        self.turns_host = [int(x) for x in host][:self.rot_dim // 2]
        signed = [x - (1 << 64) if x >= 1 << 63 else x for x in self.turns_host]
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.turns = torch.tensor(signed, dtype=torch.int64, device=dev)


def _rows(t, name, heads=None):
    """Checks a [rows, heads, d] tensor; (rows, heads, d)."""
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError("%s: a [rows, heads, channels] tensor with contiguous channels is wanted" % name)
    if not t.is_cuda:
        raise ValueError("%s: a CUDA tensor is wanted" % name)
    return t.shape


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError("%s is on %s, not on %s" % (name, t.device, dev))


def _vector(t, name, n, dtype=None):
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1) or (dtype is not None and t.dtype != dtype):
        raise ValueError("%s: a contiguous vector of %d%s is wanted"
                         % (name, n, "" if dtype is None else " " + str(dtype)))


def qk_rotary(q, k, positions, rotary, q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None, k_out=None,
              stream=None):
    """Per-head RMS norm (where a weight is given) and rotary rotation of
    q [n, Hq, d] and k [n, Hkv, d] at int32 `positions` [n].  `rotary` may be
    None (norms only), k None (queries only).  Returns (q_out, k_out): new
    tensors of the inputs' type, or the given ones, which may be of another
    type, strided, or the inputs themselves."""
    import torch
    n, Hq, d = _rows(q, "q")
    Hkv = 0
    if k is not None:
        nk, Hkv, dk = _rows(k, "k")
        if nk != n or dk != d or k.dtype != q.dtype:
            raise ValueError("k: rows, channels and type of q are wanted")
    dev = q.device
    if q_out is None:
        q_out = torch.empty((n, Hq, d), dtype=q.dtype, device=dev)
    elif tuple(_rows(q_out, "q_out")) != (n, Hq, d):
        raise ValueError("q_out: the shape of q is wanted")
    if k is not None:
        if k_out is None:
            k_out = torch.empty((n, Hkv, d), dtype=k.dtype, device=dev)
        elif tuple(_rows(k_out, "k_out")) != (n, Hkv, d):
            raise ValueError("k_out: the shape of k is wanted")
    w = q_weight if q_weight is not None else k_weight
    if q_weight is not None:
        _vector(q_weight, "q_weight", d)
    if k_weight is not None:
        _vector(k_weight, "k_weight", d, w.dtype)
    rot, interleaved, mscale, turns = 0, 0, 1.0, None
    if rotary is not None:
        rot, interleaved, mscale, turns = rotary.rot_dim, int(rotary.interleaved), rotary.mscale, rotary.turns
        if positions is None:
            raise ValueError("positions are wanted with a rotary table")
        _vector(positions, "positions", n, torch.int32)
    _same_device(dev, k=k, positions=positions, turns=turns, q_weight=q_weight, k_weight=k_weight, q_out=q_out,
                 k_out=k_out if k is not None else None)

    def at(t):
        return 0 if t is None else t.data_ptr()

    def strides(t):
        return (0, 0) if t is None else t.stride()[:2]

    ko = k_out if k is not None else None
    args = _ROTARY.pack(n, Hq, Hkv, d, rot, interleaved, dtype_code(q.dtype),
                        dtype_code(w.dtype) if w is not None else 0, dtype_code(q_out.dtype),
                        dtype_code(ko.dtype) if ko is not None else 0, eps, mscale, q.data_ptr(), at(k),
                        q_out.data_ptr(), at(ko), *q.stride()[:2], *strides(k), *q_out.stride()[:2], *strides(ko),
                        at(q_weight), at(k_weight), at(positions) if rot else 0, at(turns))
    with on_device(dev):
        _check(lib().confkv_qk_rotary(args, _stream(stream, dev.index)), "confkv_qk_rotary")
    return q_out, k_out


def prompt_attention(q, k, v, cu_seqlens, cu_seqlens_k=None, causal: bool = True, scale=None, out=None, lse=None,
                     return_lse: bool = False, stream=None):
    """Attention of packed sequences: q [rows, Hq, d], k and v [rows_k, Hkv, d],
    all fp16 or all bf16, d 64 or 128.  cu_seqlens (int32 [B + 1], on the
    device): first query row of each sequence and the end; cu_seqlens_k the
    same for keys (default: cu_seqlens).  With `causal` the queries are the
    last of their sequence's keys.  scale defaults to 1 / sqrt(d).  Returns
    out, or (out, lse) with return_lse; lse is fp32 [rows, Hq]."""
    import torch
    nq, Hq, d = _rows(q, "q")
    nk, Hkv, dk = _rows(k, "k")
    if tuple(_rows(v, "v")) != (nk, Hkv, dk) or dk != d:
        raise ValueError("k and v: one shape, and the channels of q, are wanted")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v: one type is wanted")
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens
    B = cu_seqlens.shape[0] - 1
    _vector(cu_seqlens, "cu_seqlens", B + 1, torch.int32)
    _vector(cu_seqlens_k, "cu_seqlens_k", B + 1, torch.int32)
    dev = q.device
    if out is None:
        out = torch.empty((nq, Hq, d), dtype=q.dtype, device=dev)
    elif tuple(_rows(out, "out")) != (nq, Hq, d) or out.dtype != q.dtype:
        raise ValueError("out: the shape and type of q are wanted")
    if lse is None:
        if return_lse:
            lse = torch.empty((nq, Hq), dtype=torch.float32, device=dev)
    elif tuple(lse.shape) != (nq, Hq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse: a contiguous fp32 [rows, heads] tensor is wanted")
    _same_device(dev, k=k, v=v, cu_seqlens=cu_seqlens, cu_seqlens_k=cu_seqlens_k, out=out, lse=lse)
    args = _PROMPT.pack(B, Hq, Hkv, d, dtype_code(q.dtype), int(causal), nq, nk,
                        1.0 / math.sqrt(d) if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                        out.data_ptr(), 0 if lse is None else lse.data_ptr(), cu_seqlens.data_ptr(),
                        cu_seqlens_k.data_ptr(), *q.stride()[:2], *k.stride()[:2], *v.stride()[:2],
                        *out.stride()[:2])
    with on_device(dev):
        _check(lib().confkv_prompt_attention(args, _stream(stream, dev.index)), "confkv_prompt_attention")
    return (out, lse) if return_lse else out


def prompt_status(stream=None) -> int:
    """Status bits of the prompt attention kernels on the current device since
    the last call (0: every wait was met); synchronises and clears them."""
    bits = ctypes.c_int32()
    r = lib().confkv_prompt_status(ctypes.byref(bits), _stream(stream))
    if r not in (0, -6):
        _check(r, "confkv_prompt_status")
    return int(bits.value)
