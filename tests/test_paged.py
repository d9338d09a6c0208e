"""The paged cache: append of new keys and values, and the attention of new
tokens over it, against fp64 (bounds beside each test; u = 2^-24)."""
import ctypes

import numpy as np
import pytest
import torch

import attention_kl_loss_gb300 as skl
from attention_kl_loss_gb300 import binding
from oracle import model_ops as orc

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _np(t):
    return t.double().cpu().numpy()


def _tables(n, rot, dev):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return tuple(torch.from_numpy(f(ang)).float().to(dev) for f in (np.cos, np.sin))


def _round_tol(ref, dt):
    return torch.finfo(dt).eps / 2 * np.abs(ref) + 2.0 ** -25 * (dt == torch.float16)


class Cache:
    """A paged cache with scattered pages; what no sequence owns is NaN."""

    def __init__(self, lens, HK, d, page, dt, seed=0, spare=2, fill=True, layout="heads"):
        g = torch.Generator().manual_seed(seed)
        dev = torch.device("cuda")
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        shape = (pages, HK, page, d)
        if layout == "heads":  # [pages, HK, page, d]
            self.k, self.v = (torch.full(shape, float("nan"), dtype=dt, device=dev) for _ in range(2))
        else:  # slots before heads, keys and values in one tensor
            both = torch.full((pages, 2, page, HK, d), float("nan"), dtype=dt, device=dev)
            self.k, self.v = (both[:, i].transpose(1, 2) for i in range(2))
        order = torch.randperm(pages, generator=g).tolist()
        width = max(max(need), 1) + 1
        # entries that no position uses are no page numbers at all
        self.table = torch.full((len(lens), width), 1 << 30, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.rows = []
        for b, n in enumerate(lens):
            k, v = (torch.randn(n, HK, d, generator=g).to(dt) for _ in range(2))
            self.rows.append((k, v))
            if fill and n:
                p = self.table[b, torch.arange(n) // page].long().to(dev)
                s = (torch.arange(n) % page).to(dev)
                self.k[p, :, s] = k.to(dev)
                self.v[p, :, s] = v.to(dev)
        self.table = self.table.to(dev)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=dev)


def _cu(new):
    return torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- append
@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,HK,d,page,dtype,rot,norm,inter,layout", [
    ([1], [1], 1, 64, 16, "bf16", 64, True, False, "heads"),
    ([1, 1, 1, 1, 1], [1, 17, 16, 40, 33], 3, 128, 16, "bf16", 128, True, False, "heads"),
    ([5, 0, 130, 1, 31], [5, 9, 131, 64, 31], 2, 128, 32, "fp16", 64, False, True, "slots"),
    ([257, 3], [300, 1000], 9, 64, 64, "bf16", 16, True, True, "heads"),
    ([40, 24], [40, 1030], 8, 64, 1024, "fp16", 0, False, False, "slots"),
    ([7, 70], [100, 71], 5, 128, 256, "bf16", 0, True, False, "heads"),
])
def test_append_writes_the_new_slots_and_nothing_else(new, lens, HK, d, page, dtype, rot, norm, inter, layout):
    """Keys within 16 u of |a cos| + |b sin| and half a step (test_norm_rope.py
    derives it), values and every other slot bit for bit."""
    dt = TYPES[dtype]
    c = Cache(lens, HK, d, page, dt, layout=layout)
    dev = c.k.device
    g = torch.Generator().manual_seed(9)
    total, pad = sum(new), 3
    kv = torch.randn(total + pad, 2 * HK, d, generator=g).to(dt).to(dev)
    k, v = kv[:, :HK], kv[:, HK:]
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(dev) if norm else None
    cos, sin = _tables(max(lens), rot, dev) if rot else (None, None)
    before = [t.clone() for t in (c.k, c.v)]
    st = binding.new_status(dev)
    out = skl.streamkl_paged_append(k, v, c.k, c.v, c.table, c.lens, cu_seqlens=_cu(new), cos=cos, sin=sin, k_weight=w,
                                    interleaved=inter, dev_status=st)
    binding.raise_on_device_status(st)
    assert out[0] is c.k and out[1] is c.v
    at = 0
    for b, n in enumerate(new):
        for i in range(n):
            pos = lens[b] - n + i
            p, s = int(c.table[b, pos // page]), pos % page
            assert torch.equal(c.v[p, :, s], v[at + i])
            x = _np(k[at + i])
            cc, ss = (_np(t[pos]) if rot else np.zeros(0) for t in (cos, sin)) if rot else (np.zeros(0), np.zeros(0))
            ref, mag = orc.norm_rope(x, None if w is None else _np(w), cc, ss, 1e-6, inter)
            assert np.all(np.abs(_np(c.k[p, :, s]) - ref) <= _round_tol(ref, dt) + 16 * U * mag)
            for now, old in zip((c.k, c.v), before):
                old[p, :, s] = now[p, :, s]
        at += n
    for now, old in zip((c.k, c.v), before):
        assert torch.equal(now.contiguous().view(torch.int16), old.contiguous().view(torch.int16))


@pytest.mark.gpu
def test_append_of_single_tokens_without_offsets_and_copies_exactly():
    lens = [1, 16, 17, 33, 128, 5, 6]
    a, b = (Cache(lens, 4, 128, 16, torch.bfloat16) for _ in range(2))
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(7, 4, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    cos, sin = _tables(128, 128, k.device)
    skl.streamkl_paged_append(k, v, a.k, a.v, a.table, a.lens, cos=cos, sin=sin)
    skl.streamkl_paged_append(k, v, b.k, b.v, b.table, b.lens, cu_seqlens=_cu([1] * 7), cos=cos, sin=sin)
    for x, y in ((a.k, b.k), (a.v, b.v)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    skl.streamkl_paged_append(k, v, a.k, a.v, a.table, a.lens)  # neither norm nor rotation: a copy
    for i, n in enumerate(lens):
        p, s = int(a.table[i, (n - 1) // 16]), (n - 1) % 16
        assert torch.equal(a.k[p, :, s], k[i]) and torch.equal(a.v[p, :, s], v[i])


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["page", "negative page", "length", "short length", "table", "offsets"])
def test_append_reports_what_does_not_fit_and_writes_the_rest(what):
    lens = [20, 40, 30]
    c = Cache(lens, 2, 64, 16, torch.bfloat16)
    new = [2, 2, 2]
    k, v = (torch.ones(6, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cos, sin = _tables(64, 64, k.device)
    cu = _cu(new)
    bad = [2, 3]
    if what == "page":
        c.table[1, 2] = c.k.shape[0]
    elif what == "negative page":
        c.table[1, 2] = -1
    elif what == "length":
        c.lens[1] = 16 * c.table.shape[1] + 1
        bad = [3]  # the first of its tokens fits: its page number is none
        c.table[1, -1] = 1 << 30
        bad = [2, 3]
    elif what == "short length":
        c.lens[1] = 1
    elif what == "table":
        cos, sin = cos[:39].contiguous(), sin[:39].contiguous()
        bad = [3]
    else:
        cu[3] = 7  # past the tokens that are there
        bad = [4, 5]
    before = [c.k.clone(), c.v.clone()]
    st = binding.new_status(k.device)
    skl.streamkl_paged_append(k, v, c.k, c.v, c.table, c.lens, cu_seqlens=cu, cos=cos, sin=sin, dev_status=st)
    with pytest.raises(binding.StreamKLError):
        binding.raise_on_device_status(st)
    for b in range(3):
        for i in range(2):
            t = 2 * b + i
            if t in bad:
                continue
            pos = lens[b] - 2 + i
            p, s = int(c.table[b, pos // 16]), pos % 16
            assert torch.all(c.v[p, :, s] == 1)
            for now, old in zip((c.k, c.v), before):
                old[p, :, s] = now[p, :, s]
    for now, old in zip((c.k, c.v), before):
        assert torch.equal(now.view(torch.int16), old.view(torch.int16))


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    from attention_kl_loss_gb300 import build
    build.build()
    return binding.load()


APPEND = dict(k=4096, v=4096, kc=4096, vc=4096, table=4096, ts=4, lens=4096, cu=4096, dtype=0, B=2, T=5, HK=2, d=64,
              page=16, pages=9, most=4, strides=[2048, 1024, 64] * 2 + [128, 64] * 2, rot=64, cos=4096, sin=4096, len=64,
              w=None, eps=1e-6, inter=0, st=4096)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), 2), (dict(d=80), 2), (dict(B=0), 1), (dict(T=0), 1), (dict(HK=0), 1), (dict(pages=0), 1),
    (dict(page=8), 2), (dict(page=48), 2), (dict(page=2048), 2), (dict(most=1 << 27), 2), (dict(ts=3), 1),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(cu=None), 1), (dict(k=4104), 1), (dict(v=None), 1),
    (dict(kc=None), 1), (dict(vc=4100), 1), (dict(strides=[2048, 1024, 60] + [2048, 1024, 64] + [128, 64] * 2), 1),
    (dict(strides=[2048, 1024, 0] + [2048, 1024, 64] + [128, 64] * 2), 1),
    (dict(strides=[2048, 1024, 64] * 2 + [-128, 64] * 2), 1), (dict(cos=None), 1), (dict(rot=8), 2), (dict(rot=72), 2),
    (dict(len=0), 1), (dict(eps=-1.0), 1), (dict(eps=-1.0, cos=None, sin=None), 1), (dict(inter=2), 1), (dict(st=None), 1),
    (dict(T=1 << 30, HK=4), 2), (dict(strides=None), 1),
])
def test_append_c_call_refuses(lib, over, status):
    a = {**APPEND, **over}
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_longlong * 10)(*a["strides"])
    got = lib.streamkl_paged_append(*[a[n] for n in ("k", "v", "kc", "vc", "table", "ts", "lens", "cu", "dtype", "B", "T",
                                                     "HK", "d", "page", "pages", "most", "strides", "rot", "cos", "sin",
                                                     "len", "w", "eps", "inter", "st")], None)
    assert got == status and lib.streamkl_last_error()


@pytest.mark.gpu
def test_append_python_call_refuses():
    c = Cache([20, 40], 2, 64, 16, torch.bfloat16)
    k = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    call = skl.streamkl_paged_append
    ok = (k, k, c.k, c.v, c.table, c.lens)

    def swap(**at):
        return [at.get(f"_{i}", t) for i, t in enumerate(ok)]

    for match, args, kw in [
        ("k must be", swap(_0=k.half()), {}), ("k and v", swap(_1=k[:1]), {}), ("k and v", swap(_0=k[..., :32], _1=k[..., :32]), {}),
        ("v_cache", swap(_3=c.v.half()), {}), ("both be", swap(_3=c.v[1:]), {}), ("unsupported cache", swap(
            _0=k.float(), _1=k.float(), _2=c.k.float(), _3=c.v.float()), {}),
        ("block_table", swap(_4=c.table.long()), {}), ("block_table", swap(_4=c.table[0]), {}),
        ("kv_lens", swap(_5=c.lens[:1]), {}), ("kv_lens", swap(_5=None), {}), ("cu_seqlens", ok, dict(cu_seqlens=_cu([2]))),
        ("one token", swap(_0=k[:1], _1=k[:1]), {}), ("together", ok, dict(cos=torch.ones(4, 32, device="cuda"))),
        ("k_weight", ok, dict(k_weight=torch.ones(32, device="cuda"))),
    ]:
        with pytest.raises(ValueError, match=match):
            call(*args, **kw)
