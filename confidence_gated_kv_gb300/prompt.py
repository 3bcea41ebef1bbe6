"""Operators of a prompt's path: head norms with rotary positions, and packed
prompt attention (include/confkv.h: confkv_qk_rotary, confkv_prompt_attention).

Argument marshalling only, as in binding.py; layer-wise prefill and read-back
of a cache are methods of Cache.

Calls run on `stream`, or on the current stream when it is None.  With a
torch.cuda.Stream, tensors may be freed as soon as the call returns; with a
raw handle or an ExternalStream the caller keeps them until the stream has
done the work.  New outputs belong to `stream`: another stream waits for it
before it uses them.
"""
from __future__ import annotations

import ctypes
import struct

from .binding import FP32, _check, _stream, allocating_on, call_on, dtype_code, lib, no_gradients, used_on

SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

_ROTARY = struct.Struct("=10i2f4Q8q4Q")
_PROMPT = struct.Struct("=8if4x7Q8q")


torch = None      # bound by the first call: importing the package does not load torch


def _bind():
    global torch
    import torch as t
    torch = t


class Rotary:
    """Frequencies of a rotary embedding of the first `rot_dim` channels, kept
    on `device` (default: the current one).  scaling: "none", "linear", "ntk"
    or "yarn", for positions beyond the trained `original_length`; the formulas
    are with confkv_rotary_frequencies.  "yarn" ramps linearly in the turns of
    a pair within the trained length, as the paper does; checkpoints tuned with
    a ramp over the pair index need another table."""

    def __init__(self, rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original_length: float = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 interleaved: bool = False, device=None):
        if torch is None:
            _bind()
        if scaling not in SCALINGS:
            raise ValueError("scaling is one of %s" % ", ".join(SCALINGS))
        self.rot_dim, self.interleaved = int(rot_dim), int(bool(interleaved))
        host = (ctypes.c_uint64 * max(1, self.rot_dim // 2))()
        mscale = ctypes.c_float()
        _check(lib().confkv_rotary_frequencies(self.rot_dim, float(base), SCALINGS[scaling], float(factor),
                                               float(original_length), float(beta_fast), float(beta_slow), host,
                                               ctypes.byref(mscale)), "confkv_rotary_frequencies")
        self.mscale, self._host = mscale.value, host
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.turns = torch.frombuffer(host, dtype=torch.int64).to(dev)
        self.turns_at, self.device_index = self.turns.data_ptr(), self.turns.get_device()


    @property
    def turns_host(self):
        """Turns of each pair per position, in units of 2^-64."""
        return list(self._host)[:self.rot_dim // 2]


def _unfit(what):
    raise ValueError(what)


def _dims(t, name, dev=None):
    """(rows, heads, d) and strides of a [rows, heads, d] CUDA tensor with
    contiguous channels, on device `dev` if one is given."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (stride[2] != 1 and shape[2] > 1):
        _unfit("%s: a [rows, heads, channels] tensor with contiguous channels is wanted" % name)
    if not t.is_cuda or (dev is not None and t.get_device() != dev):
        _unfit("%s: a CUDA tensor%s is wanted, not one on %s"
               % (name, "" if dev is None else " on the device of q", t.device))
    return shape, stride


def _vector(t, name, n, dtype, dev):
    """Address of a contiguous vector of n elements on device `dev`."""
    if t.shape != (n,) or (n > 1 and not t.is_contiguous()) or (dtype is not None and t.dtype != dtype):
        _unfit("%s: a contiguous vector of %d%s is wanted" % (name, n, "" if dtype is None else " " + str(dtype)))
    if t.get_device() != dev:
        _unfit("%s is on %s, not on the device of q" % (name, t.device))
    return t.data_ptr()


def _like(t, stream):
    """New contiguous tensor of the shape, type and device of t, to be written
    on `stream`."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)
    with allocating_on(stream, t.get_device()):
        return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def qk_rotary(q, k, positions, rotary, q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None, k_out=None,
              stream=None):
    """Per-head RMS norm (where a weight is given) and rotary rotation of
    q [n, Hq, d] and k [n, Hkv, d] at int32 `positions` [n].  `rotary` may be
    None (norms only), k None (queries only).  Returns (q_out, k_out): new
    tensors of the inputs' type, or the given ones, which may be of another
    type, strided, or the inputs themselves.  No derivatives: inputs that
    require gradients are refused while gradients are enabled, and inputs with
    forward-mode tangents always."""
    if torch is None:
        _bind()
    (n, Hq, d), qs = _dims(q, "q")
    no_gradients(q, k, q_weight, k_weight)
    dev, code = q.get_device(), dtype_code(q.dtype)
    if q_out is None:
        q_out, qo_code, qos = _like(q, stream), code, (Hq * d, d)
    else:
        shape, qos = _dims(q_out, "q_out", dev)
        qo_code = dtype_code(q_out.dtype)
        if shape != q.shape:
            _unfit("q_out: the shape of q is wanted")
    Hkv, ks, kos, k_at, ko_at, ko_code = 0, (0, 0), (0, 0), 0, 0, 0
    if k is None:
        k_out = None
    else:
        (nk, Hkv, dk), ks = _dims(k, "k", dev)
        if nk != n or dk != d or k.dtype != q.dtype:
            _unfit("k: rows, channels and type of q are wanted")
        if k_out is None:
            k_out, ko_code, kos = _like(k, stream), code, (Hkv * d, d)
        else:
            shape, kos = _dims(k_out, "k_out", dev)
            ko_code = dtype_code(k_out.dtype)
            if shape != k.shape:
                _unfit("k_out: the shape of k is wanted")
        k_at, ko_at = k.data_ptr(), k_out.data_ptr()
    qw_at = kw_at = w_code = pos_at = turns_at = rot = interleaved = 0
    mscale = 1.0
    if q_weight is not None:
        w_code, qw_at = dtype_code(q_weight.dtype), _vector(q_weight, "q_weight", d, None, dev)
    if k_weight is not None:
        kw_at = _vector(k_weight, "k_weight", d, None if q_weight is None else q_weight.dtype, dev)
        w_code = dtype_code(k_weight.dtype)
    if rotary is not None:
        rot, interleaved, mscale, turns_at = rotary.rot_dim, rotary.interleaved, rotary.mscale, rotary.turns_at
        if positions is None or rotary.device_index != dev:
            _unfit("positions, and a rotary table on the device of q, are wanted")
        pos_at = _vector(positions, "positions", n, torch.int32, dev)
    args = _ROTARY.pack(n, Hq, Hkv, d, rot, interleaved, code, w_code, qo_code, ko_code, eps, mscale, q.data_ptr(),
                        k_at, q_out.data_ptr(), ko_at, qs[0], qs[1], ks[0], ks[1], qos[0], qos[1], kos[0], kos[1],
                        qw_at, kw_at, pos_at, turns_at)
    call_on(dev, lib().confkv_qk_rotary, "confkv_qk_rotary", (args,), stream)
    if stream is not None:
        used_on(stream, q, k, q_out, k_out, q_weight, k_weight, positions if rot else None,
                rotary.turns if rot else None)
    return q_out, k_out


def prompt_attention(q, k, v, cu_seqlens, cu_seqlens_k=None, causal: bool = True, scale=None, out=None, lse=None,
                     return_lse: bool = False, stream=None):
    """Attention of packed sequences: q [rows, Hq, d], k and v [rows_k, Hkv, d],
    all fp16 or all bf16, d 64 or 128.  cu_seqlens (int32 [B + 1], on the
    device): first query row of each sequence and the end; cu_seqlens_k the
    same for keys (default: cu_seqlens).  With `causal` the queries are the
    last of their sequence's keys.  scale defaults to 1 / sqrt(d).  Returns
    out, or (out, lse) with return_lse; lse is fp32 [rows, Hq].  No
    derivatives: inputs that require gradients are refused while gradients are
    enabled, and inputs with forward-mode tangents always.  A
    sequence's last bits may depend on the sizes of the whole call: the keys of
    few rows are split over more of the GPU and joined."""
    if torch is None:
        _bind()
    (nq, Hq, d), qs = _dims(q, "q")
    no_gradients(q, k, v)
    dev, dtype = q.get_device(), q.dtype
    (nk, Hkv, dk), ks = _dims(k, "k", dev)
    shape, vs = _dims(v, "v", dev)
    if shape != k.shape or dk != d or k.dtype != dtype or v.dtype != dtype:
        _unfit("k and v: one shape, and the channels and type of q, are wanted")
    B = len(cu_seqlens) - 1
    cu_at = cuk_at = _vector(cu_seqlens, "cu_seqlens", B + 1, torch.int32, dev)
    if cu_seqlens_k is not None:
        cuk_at = _vector(cu_seqlens_k, "cu_seqlens_k", B + 1, torch.int32, dev)
    if out is None:
        out, os = _like(q, stream), (Hq * d, d)
    else:
        shape, os = _dims(out, "out", dev)
        if shape != q.shape or out.dtype != dtype:
            _unfit("out: the shape and type of q are wanted")
    lse_at = 0
    if lse is not None:
        if lse.shape != (nq, Hq) or dtype_code(lse.dtype) != FP32 or not lse.is_contiguous() or lse.get_device() != dev:
            _unfit("lse: a contiguous fp32 [rows, heads] tensor on the device of q is wanted")
        lse_at = lse.data_ptr()
    elif return_lse:
        with allocating_on(stream, dev):
            lse = torch.empty((nq, Hq), dtype=torch.float32, device=q.device)
        lse_at = lse.data_ptr()
    args = _PROMPT.pack(B, Hq, Hkv, d, dtype_code(dtype), 1 if causal else 0, nq, nk,
                        d ** -0.5 if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                        out.data_ptr(), lse_at, cu_at, cuk_at, qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], os[0], os[1])
    call_on(dev, lib().confkv_prompt_attention, "confkv_prompt_attention", (args,), stream)
    used_on(stream, q, k, v, cu_seqlens, cu_seqlens_k, out, lse)
    return (out, lse) if return_lse else out


def prompt_status(stream=None) -> int:
    """Status bits of the prompt attention kernels on the current device since
    the last call (0: every wait was met); synchronises and clears them."""
    bits = ctypes.c_int32()
    r = lib().confkv_prompt_status(ctypes.byref(bits), _stream(stream))
    if r not in (0, -6):
        _check(r, "confkv_prompt_status")
    return int(bits.value)
