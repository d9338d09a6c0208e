"""Operators around the attention-KL call, through the same C ABI.

``streamkl_qk_norm_rope_fwd`` / ``_bwd`` take the queries and keys of a
projection to the layout that ``streamkl_fwd`` reads (norm and rotation of
every head in one pass, grouped key heads repeated on request) and the KL's
gradients back. ``streamkl_paged_append`` puts a trained student's new keys
and values into a paged cache, ``streamkl_paged_attn`` is the attention of new
tokens (one, or a chunk) over it. As in ``binding``: argument marshalling only,
PyTorch provides device memory and the current stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

import torch

from .binding import _check, _ptr, load, new_status

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_NO_GUARD = contextlib.nullcontext()


def _guard(device):
    """Make ``device`` the current one for a call (launches and tensor maps go
    to the current device)."""
    if device.index == torch.cuda.current_device():
        return _NO_GUARD
    return torch.cuda.device(device)


def _stream(stream, device):
    s = torch.cuda.current_stream(device) if stream is None else stream
    if s.device != device:
        raise ValueError(f"stream of {s.device} for tensors on {device}")
    return s.cuda_stream


def _strides(*values):
    return (ctypes.c_longlong * len(values))(*values)


def _rows(name, t, dim, dtype=None, device=None):
    """A CUDA tensor of ``dim`` dimensions whose last one is contiguous."""
    if not isinstance(t, torch.Tensor) or t.dim() != dim:
        raise ValueError(f"{name} must be a {dim}-D tensor")
    if not t.is_cuda or t.stride(-1) != 1:
        raise ValueError(f"{name} must be a CUDA tensor with a contiguous last dimension")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _vector(name, t, n, dtype, device):
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device or t.dim() != 1
            or t.shape[0] != n or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} vector [{n}] on {device}")
    return t


def _status(dev_status, device):
    if dev_status is None:
        return new_status(device)
    if dev_status.dtype != torch.int32 or dev_status.device != device or dev_status.numel() < 1:
        raise ValueError(f"dev_status must be an int32 tensor on {device}")
    return dev_status


def _workspace(need, device, workspace):
    if need == 0:
        return None
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace too small: need {need} bytes")
    return workspace


def _tables(cos, sin, device):
    _rows("cos", cos, 2, torch.float32, device)
    _rows("sin", sin, 2, torch.float32, device)
    if cos.shape != sin.shape or not cos.is_contiguous() or not sin.is_contiguous():
        raise ValueError("cos and sin must be contiguous and of one shape [positions, rot / 2]")
    return cos.shape[0], 2 * cos.shape[1]


class _RopeSide:
    """One of q, k of a call: its tensor, sizes and the shape of its outer rows."""

    def __init__(self, name, x, positions, weight, repeat):
        packed = x.dim() == 3
        self.name, self.x, self.packed, self.repeat = name, x, packed, repeat
        if packed:
            self.B, (self.N, self.H, self.d) = 1, x.shape
            self.outer = (self.N, self.H * repeat, self.d)
        else:
            self.B, self.N, self.H, self.d = x.shape
            self.outer = (self.B, self.H * repeat, self.N, self.d)
        self.weight = _vector(f"{name}_weight", weight, self.d, torch.float32, x.device)
        self.pos, self.pos_stride = positions, 0
        if positions is not None:
            p = positions
            if not isinstance(p, torch.Tensor) or p.dtype != torch.int32 or p.device != x.device:
                raise ValueError(f"positions of {name} must be an int32 tensor on {x.device}")
            if p.shape == (self.N,) and (self.N == 1 or p.stride(0) == 1):
                return
            if packed or p.shape != (self.B, self.N) or (self.N > 1 and p.stride(1) != 1) or p.stride(0) < 0:
                raise ValueError(f"positions of {name} must be [{self.N}]"
                                 + ("" if packed else f" or [{self.B}, {self.N}]") + ", tokens contiguous")
            self.pos_stride = p.stride(0)

    def inner_strides(self, t):
        s = t.stride()
        return (0, s[0], s[1]) if self.packed else (s[0], s[1], s[2])

    def outer_strides(self, t):
        s = t.stride()
        return (0, s[0], s[1]) if self.packed else (s[0], s[2], s[1])

    def check_outer(self, name, t):
        _rows(name, t, len(self.outer), self.x.dtype, self.x.device)
        if t.shape != self.outer:
            raise ValueError(f"{name} must be {list(self.outer)}, got {list(t.shape)}")
        return t

    def check_inner(self, name, t):
        _rows(name, t, self.x.dim(), self.x.dtype, self.x.device)
        if t.shape != self.x.shape:
            raise ValueError(f"{name} must be {list(self.x.shape)}, got {list(t.shape)}")
        return t


def _rope_sides(q, k, positions, k_positions, q_weight, k_weight, k_repeat):
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    if not isinstance(x, torch.Tensor) or x.dim() not in (3, 4):
        raise ValueError("q and k must be [B, N, H, d] or packed [total, H, d]")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported type {x.dtype} (bf16, fp16, fp32)")
    if int(k_repeat) < 1:
        raise ValueError("k_repeat must be >= 1")
    if k_positions is None and (q is None or k is None or q.shape[-3] == k.shape[-3]):
        k_positions = positions
    elif k is not None and positions is not None and k_positions is None:
        raise ValueError("q and k of different lengths need k_positions beside positions")
    sides = []
    for name, t, p, w, r in (("q", q, positions, q_weight, 1), ("k", k, k_positions, k_weight, int(k_repeat))):
        if t is None:
            sides.append(None)
            continue
        _rows(name, t, x.dim(), x.dtype, x.device)
        sides.append(_RopeSide(name, t, p, w, r))
    sq, sk = sides
    if sq and sk and (sq.B != sk.B or sq.d != sk.d):
        raise ValueError("q and k differ in batch size or head dim")
    if x.dim() == 3 and ((sq and positions is None) or (sk and k_positions is None)):
        raise ValueError("a packed batch needs the positions of its tokens")
    return x, sq, sk


def _rope_args(x, sq, sk, strides, cos, sin, eps, interleaved, k_repeat):
    length, rot = _tables(cos, sin, x.device)
    a = sq or sk
    return (_DTYPES[x.dtype], a.B, sq.N if sq else 0, sk.N if sk else 0, sq.H if sq else 0, sk.H if sk else 0,
            a.d, rot, _strides(*strides), cos.data_ptr(), sin.data_ptr(), length,
            _ptr(sq.pos) if sq else None, sq.pos_stride if sq else 0,
            _ptr(sk.pos) if sk else None, sk.pos_stride if sk else 0,
            _ptr(sq.weight) if sq else None, _ptr(sk.weight) if sk else None, float(eps),
            int(bool(interleaved)), int(k_repeat))


def streamkl_qk_norm_rope_fwd(q, k, cos, sin, positions=None, k_positions=None, q_weight=None,
                              k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                              k_repeat: int = 1, out=None, dev_status=None, stream=None):
    """Norm and rotation of queries and keys per head, in one pass.

    q [B, N, H, d], k [B, NK, HK, d] (or packed [total, H, d]; either may be
    None), bf16, fp16 or fp32, any strides with d contiguous, e.g. slices of
    one projection. Returns (q_out, k_out): [B, H, N, d] as ``streamkl_fwd``
    takes them (packed: [total, H, d], as ``streamkl_fwd_varlen``), each head
    of k standing ``k_repeat`` times. cos, sin: fp32 [positions, rot / 2];
    positions: int32 [N] or [B, N] (packed: [total]; for k too unless
    k_positions is given); without them key n stands at position n and the
    queries at the last N positions of the keys. Weights: fp32 [d], None for
    rotation without norm."""
    x, sq, sk = _rope_sides(q, k, positions, k_positions, q_weight, k_weight, k_repeat)
    outs, inner, outer = [], [], []
    for i, s in enumerate((sq, sk)):
        if s is None:
            outs.append(None)
            inner += (0, 0, 0)
            outer += (0, 0, 0)
            continue
        y = out[i] if out is not None else None
        y = s.check_outer(f"out[{i}]", y) if y is not None else torch.empty(s.outer, dtype=x.dtype, device=x.device)
        outs.append(y)
        inner += s.inner_strides(s.x)
        outer += s.outer_strides(y)
    if all(s is None or s.x.numel() == 0 for s in (sq, sk)):
        return tuple(outs)
    status = _status(dev_status, x.device)
    args = _rope_args(x, sq, sk, inner + outer, cos, sin, eps, interleaved, k_repeat)
    with _guard(x.device):
        st = load().streamkl_qk_norm_rope_fwd(_ptr(q), _ptr(k), *args, _ptr(outs[0]), _ptr(outs[1]),
                                              status.data_ptr(), _stream(stream, x.device))
    if st:
        _check(st, "streamkl_qk_norm_rope_fwd")
    return tuple(outs)


def streamkl_qk_norm_rope_bwd_workspace_size(B, NQ, NK, HQ, HK, d) -> int:
    return int(load().streamkl_qk_norm_rope_bwd_workspace_size(B, NQ, NK, HQ, HK, d))


def streamkl_qk_norm_rope_bwd(q, k, dq_out, dk_out, cos, sin, positions=None, k_positions=None,
                              q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                              k_repeat: int = 1, out=None, workspace=None, dev_status=None, stream=None):
    """Gradients of ``streamkl_qk_norm_rope_fwd`` from those of its outputs
    (``streamkl_bwd``'s dq, dk): (dq, dk, dq_weight, dk_weight). dq, dk have
    the shapes of q, k (``out`` = (dq, dk) may be slices of one buffer); the
    gradients of a key head's repeats are summed; weight gradients are fp32
    [d], None where there is no weight."""
    x, sq, sk = _rope_sides(q, k, positions, k_positions, q_weight, k_weight, k_repeat)
    dev = x.device
    grads, dws, ins, inner, outer, back = [], [], [], [], [], []
    for i, (s, g) in enumerate(((sq, dq_out), (sk, dk_out))):
        if s is None:
            for to in (inner, outer, back):
                to += (0, 0, 0)
            for to in (grads, dws, ins):
                to.append(None)
            continue
        ins.append(s.check_outer(f"d{s.name}_out", g))
        t = out[i] if out is not None else None
        t = s.check_inner(f"out[{i}]", t) if t is not None else torch.empty(s.x.shape, dtype=x.dtype, device=dev)
        grads.append(t)
        dws.append(None if s.weight is None else torch.empty(s.d, dtype=torch.float32, device=dev))
        inner += s.inner_strides(s.x)
        outer += s.outer_strides(g)
        back += s.inner_strides(t)
    if all(s is None or s.x.numel() == 0 for s in (sq, sk)):
        return (*grads, *(w if w is None else w.zero_() for w in dws))
    status = _status(dev_status, dev)
    args = _rope_args(x, sq, sk, inner + outer + back, cos, sin, eps, interleaved, k_repeat)
    with _guard(dev):
        need = 0
        if dws[0] is not None or dws[1] is not None:
            need = streamkl_qk_norm_rope_bwd_workspace_size(*args[1:7])
        ws = _workspace(need, dev, workspace)
        st = load().streamkl_qk_norm_rope_bwd(_ptr(q), _ptr(k), _ptr(ins[0]), _ptr(ins[1]), *args,
                                              _ptr(grads[0]), _ptr(grads[1]), _ptr(dws[0]), _ptr(dws[1]),
                                              _ptr(ws), need, status.data_ptr(), _stream(stream, dev))
    if st:
        _check(st, "streamkl_qk_norm_rope_bwd")
    return (*grads, *dws)


def _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, total):
    """Checks of the paged cache; (B, total, HK, d, page_size, num_pages, max_pages)."""
    dev = k_cache.device
    _rows("k_cache", k_cache, 4)
    if k_cache.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"unsupported cache type {k_cache.dtype} (bf16, fp16)")
    _rows("v_cache", v_cache, 4, k_cache.dtype, dev)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must both be [pages, heads, page size, d]")
    if (block_table.dtype != torch.int32 or block_table.device != dev or block_table.dim() != 2
            or (block_table.shape[1] > 1 and block_table.stride(1) != 1)):
        raise ValueError(f"block_table must be int32 [B, pages of a sequence] on {dev}, rows contiguous")
    B = block_table.shape[0]
    _vector("kv_lens", kv_lens, B, torch.int32, dev)
    if kv_lens is None:
        raise ValueError("kv_lens must be given")
    _vector("cu_seqlens", cu_seqlens, B + 1, torch.int32, dev)
    if cu_seqlens is None and total != B:
        raise ValueError(f"without cu_seqlens each of the {B} sequences has one token, got {total}")
    pages, heads, page, d = k_cache.shape
    return B, total, heads, d, page, pages, block_table.shape[1]


def streamkl_paged_append(k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None, cos=None, sin=None,
                          k_weight=None, eps: float = 1e-6, interleaved: bool = False, dev_status=None,
                          stream=None):
    """Append new tokens to a paged cache, keys normed and rotated on the way.

    k, v [total, HK, d]: the new tokens of B sequences one after the other
    (cu_seqlens int32 [B + 1]; None: one token a sequence; tokens behind the
    last sequence are ignored). kv_lens int32 [B]: lengths with the new
    tokens. block_table int32 [B, pages]; caches [pages, HK, page size, d],
    bf16 or fp16, any strides with d contiguous. cos, sin, k_weight as in
    ``streamkl_qk_norm_rope_fwd``, None to leave out the rotation or the norm.
    Writes the caches in place and returns them."""
    _rows("k", k, 3, k_cache.dtype, k_cache.device)
    _rows("v", v, 3, k_cache.dtype, k_cache.device)
    sizes = _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, k.shape[0])
    if k.shape != v.shape or k.shape[1:] != (sizes[2], sizes[3]):
        raise ValueError(f"k and v must both be [total, {sizes[2]}, {sizes[3]}]")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin must be given together")
    dev = k.device
    length, rot = _tables(cos, sin, dev) if cos is not None else (0, 0)
    _vector("k_weight", k_weight, sizes[3], torch.float32, dev)
    status = _status(dev_status, dev)
    if k.numel() == 0:
        return k_cache, v_cache
    strides = _strides(*k_cache.stride()[:3], *v_cache.stride()[:3], *k.stride()[:2], *v.stride()[:2])
    with _guard(dev):
        st = load().streamkl_paged_append(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                          block_table.data_ptr(), block_table.stride(0), kv_lens.data_ptr(),
                                          _ptr(cu_seqlens), _DTYPES[k.dtype], *sizes, strides, rot, _ptr(cos),
                                          _ptr(sin), length, _ptr(k_weight), float(eps), int(bool(interleaved)),
                                          status.data_ptr(), _stream(stream, dev))
    if st:
        _check(st, "streamkl_paged_append")
    return k_cache, v_cache


def streamkl_paged_attn_splits(B, T, HQ, HK, d, max_seqlen_q, max_kv_len) -> int:
    """Key splits of ``streamkl_paged_attn`` for these sizes."""
    return int(load().streamkl_paged_attn_splits(B, T, HQ, HK, d, max_seqlen_q, max_kv_len))


def streamkl_paged_attn_workspace_size(B, T, HQ, HK, d, max_seqlen_q, max_kv_len, num_splits=0) -> int:
    return int(load().streamkl_paged_attn_workspace_size(B, T, HQ, HK, d, max_seqlen_q, max_kv_len, num_splits))


def streamkl_paged_attn(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None,
                        max_seqlen_q: Optional[int] = None, max_kv_len: Optional[int] = None,
                        scale: Optional[float] = None, causal: bool = True, num_splits: int = 0, out=None,
                        workspace=None, dev_status=None, stream=None):
    """Attention of new tokens over a paged cache: (out [total, H, d], lse
    fp32 [total, H]).

    q [total, H, d]: the new tokens of B sequences (cu_seqlens int32 [B + 1];
    None: one token a sequence), the last ones of kv_lens int32 [B] keys, which
    lie in the caches as ``streamkl_paged_append`` puts them (append first).
    H is a multiple of the caches' heads. max_seqlen_q, max_kv_len: bounds of
    the sequences' new tokens and lengths (default: every token, every page of
    block_table); close ones give a better grid. Rows that see no key get
    zeros and -inf; rows behind the last sequence stay as they were."""
    _rows("q", q, 3, k_cache.dtype, k_cache.device)
    dev = q.device
    total, HQ, d = q.shape
    B, _, HK, dk, page, pages, width = sizes = _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, total)
    if dk != d or HK < 1 or HQ % HK:
        raise ValueError(f"q [total, H, d] needs d = {dk} and H a multiple of {HK}, got {list(q.shape)}")
    max_q = int(max_seqlen_q) if max_seqlen_q is not None else (1 if cu_seqlens is None else total)
    max_kv = int(max_kv_len) if max_kv_len is not None else page * width
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        o, lse = torch.empty((total, HQ, d), dtype=q.dtype, device=dev), None
    else:
        o, lse = out
        if _rows("out[0]", o, 3, q.dtype, dev).shape != q.shape:
            raise ValueError(f"out[0] must be {list(q.shape)}, got {list(o.shape)}")
    if lse is None:
        lse = torch.empty((total, HQ), dtype=torch.float32, device=dev)
    elif lse.shape != (total, HQ) or lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous():
        raise ValueError(f"out[1] must be contiguous fp32 [{total}, {HQ}] on {dev}")
    status = _status(dev_status, dev)
    if q.numel() == 0:
        return o, lse
    lib = load()
    strides = _strides(*k_cache.stride()[:3], *v_cache.stride()[:3], *q.stride()[:2], *o.stride()[:2])
    with _guard(dev):
        need = lib.streamkl_paged_attn_workspace_size(B, total, HQ, HK, d, max_q, max_kv, int(num_splits))
        ws = _workspace(need, dev, workspace)
        st = lib.streamkl_paged_attn(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                                     block_table.stride(0), kv_lens.data_ptr(), _ptr(cu_seqlens), _DTYPES[q.dtype],
                                     B, total, HQ, *sizes[2:], strides, max_q, max_kv, scale, int(bool(causal)),
                                     int(num_splits), o.data_ptr(), lse.data_ptr(), _ptr(ws), need,
                                     status.data_ptr(), _stream(stream, dev))
    if st:
        _check(st, "streamkl_paged_attn")
    return o, lse
