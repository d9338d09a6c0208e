"""Operators around the attention-KL call, through the same C ABI.

``streamkl_qk_norm_rope_fwd`` / ``_bwd`` take the queries and keys of a
projection to the layout that ``streamkl_fwd`` reads (norm and rotation of
every head in one pass, grouped key heads repeated on request) and the KL's
gradients back. ``streamkl_paged_append`` puts a trained student's new keys
and values into a paged cache, ``streamkl_paged_attn`` is the attention of new
tokens (one, or a chunk) over it. As in ``binding``: argument marshalling only,
PyTorch provides device memory and the current stream.

Each call tries ``csrc/marshal.cpp`` first, which takes ordinary arguments in a
third of the time and returns None for any others; these, and all refusals, are
dealt with here.
"""
from __future__ import annotations

import math
import struct
from typing import Optional

import torch

from .binding import StreamKLError, _check, load, new_status

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


def _pack(fields, *values):
    try:
        return fields.pack(fields.size, *values)
    except struct.error as error:
        raise ValueError(f"an argument is no number or out of range: {error}") from error


def _elsewhere(call, device, stream, kwargs):
    """Run ``call`` with ``device`` current (launches and tensor maps go to the
    current device) and ``stream``, if given, the current stream: what the call
    allocates then belongs to the stream that its kernels run on."""
    if stream is None:
        with torch.cuda.device(device):
            return call(**kwargs)
    if stream.device != device:
        raise ValueError(f"stream of {stream.device} for tensors on {device}")
    with torch.cuda.stream(stream):  # (and its device)
        return call(**kwargs)


# The checks below are on the way of every call, some of which take 3 us on the
# GPU: each reads a tensor's properties once and words its refusal only then.
def _rows(name, t, dim, dtype, index):
    """Strides of a CUDA tensor of ``dim`` dimensions, the last contiguous."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a {dim}-D tensor")
    strides = t.stride()
    if len(strides) != dim or strides[-1] != 1 or t.dtype is not dtype or t.get_device() != index or index < 0:
        _refuse_rows(name, t, dim, dtype, index)
    return strides


def _refuse_rows(name, t, dim, dtype, index):
    if t.dim() != dim:
        raise ValueError(f"{name} must be a {dim}-D tensor")
    if not t.is_cuda or t.stride(-1) != 1:
        raise ValueError(f"{name} must be a CUDA tensor with a contiguous last dimension")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _vector(name, t, n, dtype, index):
    """The address of a contiguous vector, 0 for None."""
    if t is None:
        return 0
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index or t.shape != (n,)
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} vector [{n}] on cuda:{index}")
    return t.data_ptr()


def _status(dev_status, index):
    """The address of the status word (and the tensor, to keep it alive)."""
    if dev_status is None:
        dev_status = new_status(torch.device("cuda", index))
    elif dev_status.dtype is not torch.int32 or dev_status.get_device() != index or dev_status.numel() < 1:
        raise ValueError(f"dev_status must be an int32 tensor on cuda:{index}")
    return dev_status.data_ptr(), dev_status


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


def _tables(cos, sin, index):
    """(positions, rot, address of cos, of sin)."""
    f32 = torch.float32
    shape = cos.shape
    if (cos.dtype is not f32 or sin.dtype is not f32 or cos.get_device() != index or sin.get_device() != index
            or sin.shape != shape or len(shape) != 2 or not cos.is_contiguous() or not sin.is_contiguous()):
        raise ValueError("cos and sin must be contiguous fp32 and of one shape [positions, rot / 2] "
                         f"on cuda:{index}")
    n, half = shape
    return n, 2 * half, cos.data_ptr(), sin.data_ptr()


def _rope_sizes(q, k, positions, k_positions, k_repeat):
    """(a given tensor, packed, positions of k)."""
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
    return x, packed, k_positions


def _rope_side(name, t, x, packed, index, pos, weight, repeat):
    """Checks of q or k: (B, N, H, d, its rows, shape of the outer rows,
    positions and their batch stride, weight)."""
    if packed:
        s0, s1, _ = _rows(name, t, 3, x.dtype, index)
        N, H, d = t.shape
        B, inner, outer = 1, (t.data_ptr(), 0, s0, s1), (N, H * repeat, d)
    else:
        s0, s1, s2, _ = _rows(name, t, 4, x.dtype, index)
        B, N, H, d = t.shape
        inner, outer = (t.data_ptr(), s0, s1, s2), (B, H * repeat, N, d)
    at, stride = 0, 0
    if pos is not None:
        if not isinstance(pos, torch.Tensor) or pos.dtype is not torch.int32 or pos.get_device() != index:
            raise ValueError(f"positions of {name} must be an int32 tensor on cuda:{index}")
        ps, pst = pos.shape, pos.stride()
        if ps == (N,) and (N <= 1 or pst[0] == 1):
            pass
        elif ps == (B, N) and not packed and pst[0] >= 0 and (N <= 1 or pst[1] == 1):
            stride = pst[0]
        else:
            raise ValueError(f"positions of {name} must be [{N}]" + ("" if packed else f" or [{B}, {N}]")
                             + ", tokens contiguous")
        at = pos.data_ptr()
    return (B, N, H, d, inner, outer, at, stride,
            _vector("q_weight" if name == "q" else "k_weight", weight, d, torch.float32, index))


def _rope_rows(name, t, shape, x, packed, index):
    """Address and strides (batch, token, head) of an outer tensor."""
    s = _rows(name, t, len(shape), x.dtype, index)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return (t.data_ptr(), 0, s[0], s[1]) if packed else (t.data_ptr(), s[0], s[2], s[1])


def _rope_outer(name, t, shape, x, packed, index):
    """An outer output, made here unless given, with its address and strides
    (batch, token, head)."""
    if t is not None:
        return t, _rope_rows(name, t, shape, x, packed, index)
    t = torch.empty(shape, dtype=x.dtype, device=x.device)
    if packed:
        _, H, d = shape
        return t, (t.data_ptr(), 0, H * d, d)
    _, H, N, d = shape
    return t, (t.data_ptr(), H * N * d, d, N * d)


def _rope_grad(name, t, like, packed, index):
    """An output in the place of ``like``, made here unless given, with its
    address and strides (batch, token, head)."""
    if t is None:
        t = torch.empty(like.shape, dtype=like.dtype, device=like.device)
    s = _rows(name, t, 3 if packed else 4, like.dtype, index)
    if t.shape != like.shape:
        raise ValueError(f"{name} must be {list(like.shape)}, got {list(t.shape)}")
    return t, ((t.data_ptr(), 0, s[0], s[1]) if packed else (t.data_ptr(), s[0], s[1], s[2]))


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
    if out is None and stream is None and (native := load().native) is not None:
        done = native.rope_fwd(q, k, cos, sin, positions, k_positions, q_weight, k_weight, eps, interleaved, k_repeat,
                               dev_status)
        if done is not None:
            return done
    k_repeat = int(k_repeat)
    x, packed, k_pos = _rope_sizes(q, k, positions, k_positions, k_repeat)
    index = x.get_device()
    if index >= 0 and (stream is not None or index != torch.cuda.current_device()):
        return _elsewhere(streamkl_qk_norm_rope_fwd, x.device, stream, dict(
            q=q, k=k, cos=cos, sin=sin, positions=positions, k_positions=k_positions, q_weight=q_weight,
            k_weight=k_weight, eps=eps, interleaved=interleaved, k_repeat=k_repeat, out=out, dev_status=dev_status))
    yq = yk = None
    B = NQ = NK = HQ = HK = pq = pk = sq = sk = wq = wk = 0
    iq = ik = oq = ok = _NONE
    if q is not None:
        B, NQ, HQ, d, iq, shape, pq, sq, wq = _rope_side("q", q, x, packed, index, positions, q_weight, 1)
        yq, oq = _rope_outer("out[0]", out[0] if out is not None else None, shape, x, packed, index)
    if k is not None:
        Bk, NK, HK, dk, ik, shape, pk, sk, wk = _rope_side("k", k, x, packed, index, k_pos, k_weight, k_repeat)
        if q is not None and (Bk != B or dk != d):
            raise ValueError("q and k differ in batch size or head dim")
        B, d = Bk, dk
        yk, ok = _rope_outer("out[1]", out[1] if out is not None else None, shape, x, packed, index)
    length, rot, cos_at, sin_at = _tables(cos, sin, index)
    status, _keep = _status(dev_status, index)
    if B * (NQ * HQ + NK * HK) == 0:
        return yq, yk
    args = _pack(_ROPE, *iq, *ik, *oq, *ok, *_NONE, *_NONE, cos_at, sin_at, pq, sq, pk, sk, wq, wk, 0, 0, 0, 0,
                      status, _DTYPES[x.dtype], B, NQ, NK, HQ, HK, d, rot, length, bool(interleaved), k_repeat, eps)
    st = load().streamkl_qk_norm_rope_fwd(args, _raw_stream(index))
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
    [d], made by the call, None where there is no weight."""
    if out is None and stream is None and (native := load().native) is not None:
        done = native.rope_bwd(q, k, dq_out, dk_out, cos, sin, positions, k_positions, q_weight, k_weight, eps, interleaved,
                               k_repeat, workspace, dev_status)
        if done is not None:
            return done
    k_repeat = int(k_repeat)
    x, packed, k_pos = _rope_sizes(q, k, positions, k_positions, k_repeat)
    index = x.get_device()
    if index >= 0 and (stream is not None or index != torch.cuda.current_device()):
        return _elsewhere(streamkl_qk_norm_rope_bwd, x.device, stream, dict(
            q=q, k=k, dq_out=dq_out, dk_out=dk_out, cos=cos, sin=sin, positions=positions, k_positions=k_positions,
            q_weight=q_weight, k_weight=k_weight, eps=eps, interleaved=interleaved, k_repeat=k_repeat, out=out,
            workspace=workspace, dev_status=dev_status))
    dev = x.device
    dq = dk = dwq = dwk = None
    B = NQ = NK = HQ = HK = pq = pk = sq = sk = wq = wk = dwq_at = dwk_at = 0
    iq = ik = oq = ok = gq = gk = _NONE
    if q is not None:
        B, NQ, HQ, d, iq, shape, pq, sq, wq = _rope_side("q", q, x, packed, index, positions, q_weight, 1)
        oq = _rope_rows("dq_out", dq_out, shape, x, packed, index)
        dq, gq = _rope_grad("out[0]", out[0] if out is not None else None, q, packed, index)
    if k is not None:
        Bk, NK, HK, dim, ik, shape, pk, sk, wk = _rope_side("k", k, x, packed, index, k_pos, k_weight, k_repeat)
        if q is not None and (Bk != B or dim != d):
            raise ValueError("q and k differ in batch size or head dim")
        B, d = Bk, dim
        ok = _rope_rows("dk_out", dk_out, shape, x, packed, index)
        dk, gk = _rope_grad("out[1]", out[1] if out is not None else None, k, packed, index)
    if wq:
        dwq = torch.empty(d, dtype=torch.float32, device=dev)
        dwq_at = dwq.data_ptr()
    if wk:
        dwk = torch.empty(d, dtype=torch.float32, device=dev)
        dwk_at = dwk.data_ptr()
    length, rot, cos_at, sin_at = _tables(cos, sin, index)
    status, _keep = _status(dev_status, index)
    # a side without rows is absent in the C call, which leaves its weight gradient
    if B * NQ * HQ == 0:
        NQ = HQ = wq = dwq_at = 0
        if dwq is not None:
            dwq.zero_()
    if B * NK * HK == 0:
        NK = HK = wk = dwk_at = 0
        if dwk is not None:
            dwk.zero_()
    if NQ + NK == 0:
        return dq, dk, dwq, dwk
    lib = load()
    need = lib.streamkl_qk_norm_rope_bwd_workspace_size(B, NQ, NK, HQ, HK, d) if wq or wk else 0
    ws = _workspace(need, dev, workspace)
    args = _pack(_ROPE, *iq, *ik, *oq, *ok, *gq, *gk, cos_at, sin_at, pq, sq, pk, sk, wq, wk, dwq_at, dwk_at,
                      ws.data_ptr() if need else 0, need, status, _DTYPES[x.dtype], B, NQ, NK, HQ, HK, d, rot, length,
                      bool(interleaved), k_repeat, eps)
    st = lib.streamkl_qk_norm_rope_bwd(args, _raw_stream(index))
    if st:
        _check(st, "streamkl_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


def _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, total, dtype, index):
    """Checks of the paged cache: (HK, d, (page size, pages, pages of a
    sequence), B, cu_seqlens given, the caches' and the tables' fields)."""
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError(f"unsupported cache type {dtype} (bf16, fp16)")
    k0, k1, k2, _ = _rows("k_cache", k_cache, 4, dtype, index)
    v0, v1, v2, _ = _rows("v_cache", v_cache, 4, dtype, index)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must both be [pages, heads, page size, d]")
    if block_table.dtype is not torch.int32 or block_table.get_device() != index or block_table.dim() != 2:
        raise ValueError(f"block_table must be int32 [B, pages of a sequence] on cuda:{index}")
    B, width = block_table.shape
    b0, b1 = block_table.stride()
    if width > 1 and b1 != 1:
        raise ValueError("block_table rows must be contiguous")
    if kv_lens is None:
        raise ValueError("kv_lens must be given")
    lens = _vector("kv_lens", kv_lens, B, torch.int32, index)
    cu = _vector("cu_seqlens", cu_seqlens, B + 1, torch.int32, index)
    if cu_seqlens is None and total != B:
        raise ValueError(f"without cu_seqlens each of the {B} sequences has one token, got {total}")
    pages, heads, page, d = shape
    return heads, d, (page, pages, width), B, cu != 0, (
        k_cache.data_ptr(), k0, k1, k2, v_cache.data_ptr(), v0, v1, v2, block_table.data_ptr(), b0, lens, cu)


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
    if stream is None and (native := load().native) is not None:
        if native.append(k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens, cos, sin, k_weight, eps, interleaved,
                         dev_status):
            return k_cache, v_cache
    index, dtype = k_cache.get_device(), k_cache.dtype
    if index >= 0 and (stream is not None or index != torch.cuda.current_device()):
        return _elsewhere(streamkl_paged_append, k_cache.device, stream, dict(
            k=k, v=v, k_cache=k_cache, v_cache=v_cache, block_table=block_table, kv_lens=kv_lens,
            cu_seqlens=cu_seqlens, cos=cos, sin=sin, k_weight=k_weight, eps=eps, interleaved=interleaved,
            dev_status=dev_status))
    k0, k1, _ = _rows("k", k, 3, dtype, index)
    v0, v1, _ = _rows("v", v, 3, dtype, index)
    total, HK, d = shape = k.shape
    heads, dim, pages, B, _, cache = _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, total, dtype, index)
    if v.shape != shape or HK != heads or d != dim:
        raise ValueError(f"k and v must both be [total, {heads}, {dim}]")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin must be given together")
    length, rot, cos_at, sin_at = _tables(cos, sin, index) if cos is not None else _NONE
    w = _vector("k_weight", k_weight, d, torch.float32, index)
    status, _keep = _status(dev_status, index)
    if total == 0 or HK == 0:
        return k_cache, v_cache
    args = _pack(_APPEND, k.data_ptr(), 0, k0, k1, v.data_ptr(), 0, v0, v1, *cache, cos_at, sin_at, w, status,
                        _DTYPES[dtype], B, total, HK, d, *pages, rot, length, bool(interleaved), eps)
    st = load().streamkl_paged_append(args, _raw_stream(index))
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
    if out is None and stream is None and (native := load().native) is not None:
        done = native.attn(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, max_seqlen_q, max_kv_len, scale, causal,
                           num_splits, workspace, dev_status)
        if done is not None:
            return done
    index, dtype = k_cache.get_device(), k_cache.dtype
    if index >= 0 and (stream is not None or index != torch.cuda.current_device()):
        return _elsewhere(streamkl_paged_attn, k_cache.device, stream, dict(
            q=q, k_cache=k_cache, v_cache=v_cache, block_table=block_table, kv_lens=kv_lens, cu_seqlens=cu_seqlens,
            max_seqlen_q=max_seqlen_q, max_kv_len=max_kv_len, scale=scale, causal=causal, num_splits=num_splits,
            out=out, workspace=workspace, dev_status=dev_status))
    q0, q1, _ = _rows("q", q, 3, dtype, index)
    total, HQ, d = shape = q.shape
    HK, dim, pages, B, offsets, cache = _cache(k_cache, v_cache, block_table, kv_lens, cu_seqlens, total, dtype, index)
    if dim != d or HK < 1 or HQ % HK:
        raise ValueError(f"q [total, H, d] needs d = {dim} and H a multiple of {HK}, got {list(shape)}")
    max_q = (total if offsets else 1) if max_seqlen_q is None else max_seqlen_q
    max_kv = pages[0] * pages[2] if max_kv_len is None else max_kv_len
    dev = q.device
    o, lse = (None, None) if out is None else out
    if o is None:
        o = torch.empty(shape, dtype=dtype, device=dev)
        o0, o1 = HQ * d, d
    else:
        o0, o1, _ = _rows("out[0]", o, 3, dtype, index)
        if o.shape != shape:
            raise ValueError(f"out[0] must be {list(shape)}, got {list(o.shape)}")
    if lse is None:
        lse = torch.empty((total, HQ), dtype=torch.float32, device=dev)
    elif (lse.shape != (total, HQ) or lse.dtype is not torch.float32 or lse.get_device() != index
          or not lse.is_contiguous()):
        raise ValueError(f"out[1] must be contiguous fp32 [{total}, {HQ}] on cuda:{index}")
    status, _keep = _status(dev_status, index)
    if total == 0 or HQ == 0:
        return o, lse
    lib = load()
    if workspace is None:
        need = lib.streamkl_paged_attn_workspace_size(B, total, HQ, HK, d, max_q, max_kv, num_splits)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    args = _pack(_ATTN, q.data_ptr(), 0, q0, q1, o.data_ptr(), 0, o0, o1, *cache, lse.data_ptr(),
                      workspace.data_ptr(), workspace.nbytes, status, _DTYPES[dtype], B, total, HQ, HK, d, *pages, max_q,
                      max_kv, bool(causal), num_splits, 1.0 / math.sqrt(d) if scale is None else scale)
    st = lib.streamkl_paged_attn(args, _raw_stream(index))
    if st:
        try:
            _check(st, "streamkl_paged_attn")
        except StreamKLError as error:
            need = lib.streamkl_paged_attn_workspace_size(B, total, HQ, HK, d, max_q, max_kv, num_splits)
            if workspace.nbytes < need:
                raise ValueError(f"workspace too small: need {need} bytes") from error
            raise
    return o, lse
