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

import math
import struct
from typing import Optional

import torch

from .binding import _check, load, new_status

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
# the current stream's handle without making a Stream object (2 us of a call
# whose kernel takes 3)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_NONE = (0, 0, 0, 0)

# The argument structs of the C ABI, field by field (native alignment)
_ROWS = "Pqqq"
_ROPE = struct.Struct("N" + 6 * _ROWS + "PPPqPqPPPPPNP11if")
_APPEND = struct.Struct("N" + 4 * _ROWS + "PqPPPPPP11if")
_ATTN = struct.Struct("N" + 4 * _ROWS + "PqPPPPNP13if")


def _on_device(call, device, kwargs):
    """Run ``call`` with ``device`` current: launches and tensor maps go to
    the current device."""
    with torch.cuda.device(device):
        return call(**kwargs)


def _stream(stream, device):
    if stream is None:
        return _raw_stream(device.index)
    if stream.device != device:
        raise ValueError(f"stream of {stream.device} for tensors on {device}")
    return stream.cuda_stream


def _rows(name, t, dim, dtype, device):
    """A CUDA tensor of ``dim`` dimensions whose last one is contiguous; its
    strides."""
    if not isinstance(t, torch.Tensor) or t.dim() != dim:
        raise ValueError(f"{name} must be a {dim}-D tensor")
    strides = t.stride()
    if strides[-1] != 1 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor with a contiguous last dimension")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return strides


def _vector(name, t, n, dtype, device):
    """The address of a contiguous vector, 0 for None."""
    if t is None:
        return 0
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device or t.shape != (n,)
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} vector [{n}] on {device}")
    return t.data_ptr()


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
    n, half = cos.shape
    return n, 2 * half


def _rope_sizes(q, k, positions, k_positions, k_repeat):
    """(a given tensor, packed, positions of q and of k)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    if not isinstance(x, torch.Tensor) or x.dim() not in (3, 4):
        raise ValueError("q and k must be [B, N, H, d] or packed [total, H, d]")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported type {x.dtype} (bf16, fp16, fp32)")
    if k_repeat < 1:
        raise ValueError("k_repeat must be >= 1")
    packed = x.dim() == 3
    if k_positions is None and positions is not None and k is not None:
        if q is not None and q.shape[-3] != k.shape[-3]:
            raise ValueError("q and k of different lengths need k_positions beside positions")
        k_positions = positions
    if packed and ((q is not None and positions is None) or (k is not None and k_positions is None)):
        raise ValueError("a packed batch needs the positions of its tokens")
    return x, packed, positions, k_positions


def _rope_side(name, t, x, packed, pos, weight, repeat):
    """Checks of q or k: (B, N, H, d, its rows, shape of the outer rows,
    positions and their batch stride, weight)."""
    s = _rows(name, t, 3 if packed else 4, x.dtype, x.device)
    if packed:
        N, H, d = t.shape
        B, inner, outer = 1, (t.data_ptr(), 0, s[0], s[1]), (N, H * repeat, d)
    else:
        B, N, H, d = t.shape
        inner, outer = (t.data_ptr(), s[0], s[1], s[2]), (B, H * repeat, N, d)
    w = _vector("q_weight" if name == "q" else "k_weight", weight, d, torch.float32, x.device)
    at, stride = 0, 0
    if pos is not None:
        if not isinstance(pos, torch.Tensor) or pos.dtype != torch.int32 or pos.device != x.device:
            raise ValueError(f"positions of {name} must be an int32 tensor on {x.device}")
        ps, pst = pos.shape, pos.stride()
        if ps == (B, N) and not packed and pst[0] >= 0 and (N <= 1 or pst[1] == 1):
            stride = pst[0]
        elif ps != (N,) or (N > 1 and pst[0] != 1):
            raise ValueError(f"positions of {name} must be [{N}]" + ("" if packed else f" or [{B}, {N}]")
                             + ", tokens contiguous")
        at = pos.data_ptr()
    return B, N, H, d, inner, outer, at, stride, w


def _rope_rows(name, t, shape, x, packed):
    """Address and strides (batch, token, head) of an outer tensor."""
    s = _rows(name, t, len(shape), x.dtype, x.device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return (t.data_ptr(), 0, s[0], s[1]) if packed else (t.data_ptr(), s[0], s[2], s[1])


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
    k_repeat = int(k_repeat)
    x, packed, q_pos, k_pos = _rope_sizes(q, k, positions, k_positions, k_repeat)
    dev, dtype = x.device, x.dtype
    if x.is_cuda and dev.index != torch.cuda.current_device():
        return _on_device(streamkl_qk_norm_rope_fwd, dev, dict(
            q=q, k=k, cos=cos, sin=sin, positions=positions, k_positions=k_positions, q_weight=q_weight,
            k_weight=k_weight, eps=eps, interleaved=interleaved, k_repeat=k_repeat, out=out, dev_status=dev_status,
            stream=stream))
    yq = yk = None
    B = NQ = NK = HQ = HK = pq = pk = sq = sk = wq = wk = 0
    iq = ik = oq = ok = _NONE
    if q is not None:
        B, NQ, HQ, d, iq, shape, pq, sq, wq = _rope_side("q", q, x, packed, q_pos, q_weight, 1)
        yq = out[0] if out is not None else None
        if yq is None:
            yq = torch.empty(shape, dtype=dtype, device=dev)
        oq = _rope_rows("out[0]", yq, shape, x, packed)
    if k is not None:
        Bk, NK, HK, dk, ik, shape, pk, sk, wk = _rope_side("k", k, x, packed, k_pos, k_weight, k_repeat)
        if q is not None and (Bk != B or dk != d):
            raise ValueError("q and k differ in batch size or head dim")
        B, d = Bk, dk
        yk = out[1] if out is not None else None
        if yk is None:
            yk = torch.empty(shape, dtype=dtype, device=dev)
        ok = _rope_rows("out[1]", yk, shape, x, packed)
    length, rot = _tables(cos, sin, dev)
    status = _status(dev_status, dev)
    if B * (NQ * HQ + NK * HK) == 0:
        return yq, yk
    args = _ROPE.pack(_ROPE.size, *iq, *ik, *oq, *ok, *_NONE, *_NONE, cos.data_ptr(), sin.data_ptr(), pq, sq, pk, sk,
                      wq, wk, 0, 0, 0, 0, status.data_ptr(), _DTYPES[dtype], B, NQ, NK, HQ, HK, d, rot, length,
                      bool(interleaved), k_repeat, eps)
    st = load().streamkl_qk_norm_rope_fwd(args, _stream(stream, dev))
    if st:
        _check(st, "streamkl_qk_norm_rope_fwd")
    return yq, yk


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
    k_repeat = int(k_repeat)
    x, packed, q_pos, k_pos = _rope_sizes(q, k, positions, k_positions, k_repeat)
    dev, dtype = x.device, x.dtype
    if x.is_cuda and dev.index != torch.cuda.current_device():
        return _on_device(streamkl_qk_norm_rope_bwd, dev, dict(
            q=q, k=k, dq_out=dq_out, dk_out=dk_out, cos=cos, sin=sin, positions=positions, k_positions=k_positions,
            q_weight=q_weight, k_weight=k_weight, eps=eps, interleaved=interleaved, k_repeat=k_repeat, out=out,
            workspace=workspace, dev_status=dev_status, stream=stream))
    dq = dk = dwq = dwk = None
    B = NQ = NK = HQ = HK = pq = pk = sq = sk = wq = wk = dwq_at = dwk_at = 0
    iq = ik = oq = ok = gq = gk = _NONE
    if q is not None:
        B, NQ, HQ, d, iq, shape, pq, sq, wq = _rope_side("q", q, x, packed, q_pos, q_weight, 1)
        oq = _rope_rows("dq_out", dq_out, shape, x, packed)
        dq = out[0] if out is not None else None
        if dq is None:
            dq = torch.empty(q.shape, dtype=dtype, device=dev)
        gq = _rope_grad("out[0]", dq, q, packed)
        if wq:
            dwq = torch.empty(d, dtype=torch.float32, device=dev)
            dwq_at = dwq.data_ptr()
    if k is not None:
        Bk, NK, HK, dim, ik, shape, pk, sk, wk = _rope_side("k", k, x, packed, k_pos, k_weight, k_repeat)
        if q is not None and (Bk != B or dim != d):
            raise ValueError("q and k differ in batch size or head dim")
        B, d = Bk, dim
        ok = _rope_rows("dk_out", dk_out, shape, x, packed)
        dk = out[1] if out is not None else None
        if dk is None:
            dk = torch.empty(k.shape, dtype=dtype, device=dev)
        gk = _rope_grad("out[1]", dk, k, packed)
        if wk:
            dwk = torch.empty(d, dtype=torch.float32, device=dev)
            dwk_at = dwk.data_ptr()
    length, rot = _tables(cos, sin, dev)
    status = _status(dev_status, dev)
    if B * (NQ * HQ + NK * HK) == 0:
        for w in (dwq, dwk):
            if w is not None:
                w.zero_()
        return dq, dk, dwq, dwk
    lib = load()
    need = lib.streamkl_qk_norm_rope_bwd_workspace_size(B, NQ, NK, HQ, HK, d) if wq or wk else 0
    ws = _workspace(need, dev, workspace)
    args = _ROPE.pack(_ROPE.size, *iq, *ik, *oq, *ok, *gq, *gk, cos.data_ptr(), sin.data_ptr(), pq, sq, pk, sk, wq, wk,
                      dwq_at, dwk_at, ws.data_ptr() if need else 0, need, status.data_ptr(), _DTYPES[dtype], B, NQ, NK,
                      HQ, HK, d, rot, length, bool(interleaved), k_repeat, eps)
    st = lib.streamkl_qk_norm_rope_bwd(args, _stream(stream, dev))
    if st:
        _check(st, "streamkl_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


def _rope_grad(name, t, x, packed):
    """Address and strides (batch, token, head) of an output in the place of x."""
    s = _rows(name, t, 3 if packed else 4, x.dtype, x.device)
    if t.shape != x.shape:
        raise ValueError(f"{name} must be {list(x.shape)}, got {list(t.shape)}")
    return (t.data_ptr(), 0, s[0], s[1]) if packed else (t.data_ptr(), s[0], s[1], s[2])


def _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, total):
    """Checks of the paged cache: (HK, d, (page size, pages, pages of a
    sequence), B, cu_seqlens given, the caches' and the tables' fields)."""
    dev, dtype = k_cache.device, k_cache.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError(f"unsupported cache type {dtype} (bf16, fp16)")
    ks = _rows("k_cache", k_cache, 4, dtype, dev)
    vs = _rows("v_cache", v_cache, 4, dtype, dev)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must both be [pages, heads, page size, d]")
    if block_table.dtype != torch.int32 or block_table.device != dev or block_table.dim() != 2:
        raise ValueError(f"block_table must be int32 [B, pages of a sequence] on {dev}")
    B, width = block_table.shape
    bs = block_table.stride()
    if width > 1 and bs[1] != 1:
        raise ValueError("block_table rows must be contiguous")
    if kv_lens is None:
        raise ValueError("kv_lens must be given")
    lens = _vector("kv_lens", kv_lens, B, torch.int32, dev)
    cu = _vector("cu_seqlens", cu_seqlens, B + 1, torch.int32, dev)
    if cu_seqlens is None and total != B:
        raise ValueError(f"without cu_seqlens each of the {B} sequences has one token, got {total}")
    pages, heads, page, d = shape
    return heads, d, (page, pages, width), B, cu != 0, (
        k_cache.data_ptr(), ks[0], ks[1], ks[2], v_cache.data_ptr(), vs[0], vs[1], vs[2], block_table.data_ptr(), bs[0],
        lens, cu)


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
    dev, dtype = k_cache.device, k_cache.dtype
    if k_cache.is_cuda and dev.index != torch.cuda.current_device():
        return _on_device(streamkl_paged_append, dev, dict(
            k=k, v=v, k_cache=k_cache, v_cache=v_cache, block_table=block_table, kv_lens=kv_lens,
            cu_seqlens=cu_seqlens, cos=cos, sin=sin, k_weight=k_weight, eps=eps, interleaved=interleaved,
            dev_status=dev_status, stream=stream))
    ks = _rows("k", k, 3, dtype, dev)
    vs = _rows("v", v, 3, dtype, dev)
    total, HK, d = k.shape
    heads, dim, pages, B, _, cache = _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, total)
    if k.shape != v.shape or HK != heads or d != dim:
        raise ValueError(f"k and v must both be [total, {heads}, {dim}]")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin must be given together")
    length, rot = _tables(cos, sin, dev) if cos is not None else (0, 0)
    w = _vector("k_weight", k_weight, d, torch.float32, dev)
    status = _status(dev_status, dev)
    if total == 0 or HK == 0:
        return k_cache, v_cache
    args = _APPEND.pack(_APPEND.size, k.data_ptr(), 0, ks[0], ks[1], v.data_ptr(), 0, vs[0], vs[1], *cache,
                        cos.data_ptr() if rot else 0, sin.data_ptr() if rot else 0, w, status.data_ptr(),
                        _DTYPES[dtype], B, total, HK, d, *pages, rot, length, bool(interleaved), eps)
    st = load().streamkl_paged_append(args, _stream(stream, dev))
    if st:
        _check(st, "streamkl_paged_append")
    return k_cache, v_cache


def streamkl_paged_attn_splits(B, T, HQ, HK, d, max_seqlen_q, max_kv_len) -> int:
    """Key splits that ``streamkl_paged_attn`` takes for these sizes (0: its
    kernel for few rows, which shares the keys evenly over the GPU)."""
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
    dev, dtype = k_cache.device, k_cache.dtype
    if k_cache.is_cuda and dev.index != torch.cuda.current_device():
        return _on_device(streamkl_paged_attn, dev, dict(
            q=q, k_cache=k_cache, v_cache=v_cache, block_table=block_table, kv_lens=kv_lens, cu_seqlens=cu_seqlens,
            max_seqlen_q=max_seqlen_q, max_kv_len=max_kv_len, scale=scale, causal=causal, num_splits=num_splits,
            out=out, workspace=workspace, dev_status=dev_status, stream=stream))
    qs = _rows("q", q, 3, dtype, dev)
    shape = q.shape
    total, HQ, d = shape
    HK, dim, pages, B, offsets, cache = _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, total)
    if dim != d or HK < 1 or HQ % HK:
        raise ValueError(f"q [total, H, d] needs d = {dim} and H a multiple of {HK}, got {list(shape)}")
    max_q = (total if offsets else 1) if max_seqlen_q is None else max_seqlen_q
    max_kv = pages[0] * pages[2] if max_kv_len is None else max_kv_len
    o, lse = (None, None) if out is None else out
    if o is None:
        o = torch.empty(shape, dtype=dtype, device=dev)
    os = _rows("out[0]", o, 3, dtype, dev)
    if o.shape != shape:
        raise ValueError(f"out[0] must be {list(shape)}, got {list(o.shape)}")
    if lse is None:
        lse = torch.empty((total, HQ), dtype=torch.float32, device=dev)
    elif lse.shape != (total, HQ) or lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous():
        raise ValueError(f"out[1] must be contiguous fp32 [{total}, {HQ}] on {dev}")
    status = _status(dev_status, dev)
    if total == 0 or HQ == 0:
        return o, lse
    lib = load()
    need = lib.streamkl_paged_attn_workspace_size(B, total, HQ, HK, d, max_q, max_kv, num_splits)
    ws = _workspace(need, dev, workspace)
    args = _ATTN.pack(_ATTN.size, q.data_ptr(), 0, qs[0], qs[1], o.data_ptr(), 0, os[0], os[1], *cache, lse.data_ptr(),
                      ws.data_ptr() if need else 0, need, status.data_ptr(), _DTYPES[dtype], B, total, HQ, HK, d,
                      *pages, max_q, max_kv, bool(causal), num_splits,
                      1.0 / math.sqrt(d) if scale is None else scale)
    st = lib.streamkl_paged_attn(args, _stream(stream, dev))
    if st:
        _check(st, "streamkl_paged_attn")
    return o, lse
