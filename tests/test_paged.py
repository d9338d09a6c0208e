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


# ---------------------------------------------------------------- attention
def _check_attn(o, lse, q, c, new, lens, scale, causal, dt):
    """Per element: a score of d fp32-accumulated products is within
    (d + 4) 2^-23 of S = scale sum |q k|, its exponent's product and difference
    add 8 x 2^-23 of it and ex2 2^-22, so a term of the softmax and its sum are
    each within D = (d + 12) 2^-23 S + 2^-21, the sums over L keys within
    L 2^-23 more; P is rounded to the type, half a step, and so is o: eps / 2
    of sum p |v| and of |o|. fp16 terms below 2^-14 of a row's reference lose
    up to 2^-25 each instead, of at most the largest |v|."""
    at = 0
    half = torch.finfo(dt).eps / 2
    for b, n in enumerate(new):
        k, v = (_np(torch.stack(list(t)).transpose(0, 1)) if len(t) else np.zeros((q.shape[1], 0, q.shape[2]))
                for t in (c.rows[b][0][:lens[b]], c.rows[b][1][:lens[b]]))
        x = _np(q[at:at + n])
        ref, ref_lse, mag = orc.paged_attn(x, k, v, scale, causal)
        got, got_lse = _np(o[at:at + n]), _np(lse[at:at + n])
        at += n
        if n == 0 or lens[b] == 0:
            assert np.all(got == 0) and np.all(np.isneginf(got_lse))
            continue
        G = x.shape[1] // k.shape[0]
        S = scale * max(np.max(np.abs(x[:, h]) @ np.abs(k[h // G]).T) for h in range(x.shape[1]))
        D = (x.shape[2] + 12) * 2.0 ** -23 * S + 2.0 ** -21
        E = 2 * D + lens[b] * 2.0 ** -23
        tol = half * np.abs(ref) + (half + E) * mag
        if dt == torch.float16:
            tol = tol + lens[b] * 2.0 ** -25 * np.abs(v).max() + 2.0 ** -25
        empty = np.isneginf(ref_lse)
        assert np.array_equal(empty, np.isneginf(got_lse))
        assert np.all(got[empty] == 0)
        err = np.abs(got - ref)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        fin = ~empty
        assert np.all(np.abs(got_lse[fin] - ref_lse[fin]) <= E + 2.0 ** -22 * np.abs(ref_lse[fin]))


ATTN = [
    # new, lens, HQ, HK, d, page, type, causal, splits, layout
    ([1], [1], 1, 1, 64, 16, "bf16", True, 0, "heads"),
    ([1], [200], 4, 1, 128, 16, "bf16", True, 0, "heads"),
    ([1, 1, 1, 1], [1, 128, 129, 700], 8, 2, 128, 32, "bf16", True, 0, "heads"),
    ([1, 1, 1], [700, 2, 300], 6, 2, 64, 64, "fp16", False, 3, "slots"),
    ([3, 0, 5, 1], [3, 40, 600, 257], 3, 3, 128, 16, "bf16", True, 1, "slots"),
    ([40, 1, 17], [300, 1000, 17], 10, 2, 128, 128, "fp16", True, 2, "heads"),
    ([128], [128], 1, 1, 64, 256, "bf16", True, 0, "heads"),
    ([129, 2], [129, 513], 2, 1, 128, 64, "bf16", True, 0, "heads"),
    ([300, 77], [300, 1111], 3, 1, 64, 16, "bf16", True, 1, "heads"),
    ([257, 130], [700, 130], 4, 4, 128, 1024, "bf16", True, 3, "slots"),
    ([65], [900], 21, 3, 128, 32, "fp16", False, 0, "heads"),
    ([2, 9], [0, 5], 4, 2, 64, 16, "bf16", True, 0, "heads"),       # rows without a key
    ([300], [140], 1, 1, 128, 16, "bf16", True, 2, "heads"),
    ([4, 4], [0, 0], 2, 2, 128, 16, "fp16", False, 0, "heads"),
    ([6], [33], 160, 1, 64, 32, "bf16", True, 0, "heads"),          # one token's group wider than a tile
]


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,HQ,HK,d,page,dtype,causal,splits,layout", ATTN)
def test_attention_matches_fp64(new, lens, HQ, HK, d, page, dtype, causal, splits, layout):
    dt = TYPES[dtype]
    c = Cache(lens, HK, d, page, dt, layout=layout, seed=sum(lens))
    g = torch.Generator().manual_seed(HQ + d)
    total, pad = sum(new), 2
    # strided queries: the first heads of a wider projection
    q = torch.randn(total + pad, HQ + 2, d, generator=g).to(dt).cuda()[:, :HQ]
    o = torch.full((total + pad, HQ, d), 3.0, dtype=dt, device="cuda")
    lse = torch.full((total + pad, HQ), 3.0, device="cuda")
    st = binding.new_status()
    scale = d ** -0.5
    cu = _cu(new)
    ret = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=cu, max_seqlen_q=max(new),
                                  max_kv_len=max(lens), causal=causal, num_splits=splits, out=(o, lse), dev_status=st)
    binding.raise_on_device_status(st)
    assert ret[0] is o and ret[1] is lse
    assert torch.all(o[total:] == 3) and torch.all(lse[total:] == 3)  # rows behind the last sequence
    _check_attn(o, lse, q, c, new, lens, scale, causal, dt)
    # bounds left at their defaults, outputs made by the call: the same rows
    o2, lse2 = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=cu, causal=causal, dev_status=st)
    binding.raise_on_device_status(st)
    _check_attn(o2, lse2, q, c, new, lens, scale, causal, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_logits_move_the_reference(dtype):
    """Keys that grow along the sequence raise the running maximum far past the
    2^8 that leaves the reference alone, and a last key decides some rows."""
    dt = TYPES[dtype]
    lens, HQ, HK, d = [700], 4, 2, 64
    c = Cache(lens, HK, d, 16, dt, seed=4)
    ramp = torch.linspace(0.1, 6.0, 700)
    k = (c.rows[0][0].float() * ramp[:, None, None]).to(dt)
    k[-1] *= 2
    c.rows[0] = (k, c.rows[0][1])
    pos = torch.arange(700)
    c.k[c.table[0, pos // 16].long(), :, (pos % 16).cuda()] = k.cuda()
    for n in (1, 60, 140):
        q = 3 * torch.randn(n, HQ, d, generator=torch.Generator().manual_seed(n))
        q = q.to(dt).cuda()
        for splits in (1, 3):
            o, lse = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=_cu([n]), num_splits=splits)
            _check_attn(o, lse, q, c, [n], lens, d ** -0.5, True, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,n,rise,run", [(128, 100, 1, 64), (128, 100, -1, 64), (128, 60, 1, 64), (64, 100, 1, 64),
                                          (128, 100, 1, 32), (128, 100, -1, 32), (128, 300, 1, 96)])
def test_logits_that_rise_within_a_tile(d, n, rise, run, dtype):
    """Scores of even rows rise (odd ones fall) by about 10 from one run of keys to the next, so that the reference
    moves in the middle of a tile, for some rows of a warp; the last rows also at the sequence's ragged end."""
    dt = TYPES[dtype]
    c = Cache([700], 1, d, 16, dt, fill=False)
    g = torch.Generator().manual_seed(d + n)
    u = torch.randn(d, generator=g)
    u *= d ** 0.5 / u.norm()
    steps = torch.arange(700) // run * rise * 10 / d ** 0.5
    k = (steps[:, None, None] * u + 0.1 * torch.randn(700, 1, d, generator=g)).to(dt)
    v = torch.randn(700, 1, d, generator=g).to(dt)
    c.rows = [(k, v)]
    at = torch.arange(700)
    p, s = c.table[0, at.cuda() // 16].long(), (at % 16).cuda()
    c.k[p, :, s], c.v[p, :, s] = k.cuda(), v.cuda()
    sign = torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)[:, None, None]
    q = (sign * u + 0.1 * torch.randn(n, 2, d, generator=g)).to(dt).cuda()
    for splits, causal in ((1, True), (2, False)):
        st = binding.new_status()
        o, lse = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=_cu([n]), max_kv_len=700, causal=causal,
                                         num_splits=splits, dev_status=st)
        binding.raise_on_device_status(st)
        _check_attn(o, lse, q, c, [n], [700], d ** -0.5, causal, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("B,n,L,HQ,HK,page,splits", [(32, 1, 9000, 8, 8, 16, 1), (16, 1, 20000, 16, 4, 32, 0),
                                                     (4, 300, 5000, 8, 4, 128, 0), (2, 40, 30000, 8, 4, 64, 3)])
def test_long_sequences_that_wait_for_memory(B, n, L, HQ, HK, page, splits):
    """More keys than the caches hold on chip, so that loads arrive late: every
    wait of the kernel is needed. Against torch in fp64 on the device, bounds
    as in _check_attn with the relative 2-norm: the term (eps / 2) sum p |v| is
    there a sum of L independent roundings, at most eps / 2 of the norm of p v,
    and o's own rounding eps / 2 of o; E adds under 2e-3: 2^-8 + 2^-8 + 2e-3."""
    d, dt = 128, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(L)
    per = -(-L // page)
    k, v = (torch.randn(B * per, HK, page, d, generator=g, device="cuda").to(dt) for _ in range(2))
    table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    lens = torch.randint(L // 2, L + 1, (B,), generator=g, device="cuda").to(torch.int32)
    q = torch.randn(B * n, HQ, d, generator=g, device="cuda").to(dt)
    st = binding.new_status()
    o, lse = skl.streamkl_paged_attn(q, k, v, table, lens, cu_seqlens=_cu([n] * B), max_seqlen_q=n, max_kv_len=L,
                                     num_splits=splits, dev_status=st)
    binding.raise_on_device_status(st)
    for b in range(B):
        length = int(lens[b])
        ks, vs = (t[table[b].long()].transpose(0, 1).reshape(HK, -1, d)[:, :length].double() for t in (k, v))
        x = q[b * n:(b + 1) * n].double().transpose(0, 1).reshape(HK, -1, d)  # [HK, G n, d]
        s = x @ ks.transpose(1, 2) * d ** -0.5
        keys = torch.arange(length, device="cuda")
        row = torch.arange(n, device="cuda").repeat(HQ // HK)
        s = s.masked_fill(keys > (length - n + row)[:, None], -float("inf"))
        z = torch.logsumexp(s, -1, keepdim=True)
        ref = ((s - z).exp() @ vs).view(HQ, n, d).transpose(0, 1)
        got = o[b * n:(b + 1) * n].double()
        rel = ((got - ref).norm(dim=-1) / ref.norm(dim=-1)).max()
        assert float(rel) <= 2.0 ** -7 + 2e-3, (b, float(rel))
        dl = (lse[b * n:(b + 1) * n].double() - z.view(HQ, n).T).abs().max()
        assert float(dl) <= 1e-3


@pytest.mark.gpu
@pytest.mark.parametrize("B,HQ,HK,d,page,most,n", [(300, 6, 3, 64, 16, 300, 1), (700, 2, 2, 64, 32, 40, 1),
                                                   (129, 8, 1, 128, 16, 700, 3), (5, 32, 8, 64, 64, 3000, 8)])
def test_many_ragged_sequences_of_few_rows(B, HQ, HK, d, page, most, n):
    """Items of zero, one and many key tiles side by side, more sequences than
    a block has threads, stretches of the persistent CTAs that begin and end
    anywhere in them."""
    dt = torch.bfloat16
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, most + 1, (B,), generator=g)
    lens[torch.rand(B, generator=g) < 0.1] = 0
    lens[torch.rand(B, generator=g) < 0.1] = 128
    new = torch.randint(0, n + 1, (B,), generator=g).tolist()
    new[0] = n
    lens = lens.tolist()
    c = Cache(lens, HK, d, page, dt)
    q = torch.randn(sum(new), HQ, d, generator=g).to(dt).cuda()
    st = binding.new_status()
    assert skl.streamkl_paged_attn_splits(B, sum(new), HQ, HK, d, n, most) == 0
    o, lse = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=_cu(new), max_seqlen_q=n,
                                     max_kv_len=max(lens), dev_status=st)
    binding.raise_on_device_status(st)
    _check_attn(o, lse, q, c, new, lens, d ** -0.5, True, dt)


@pytest.mark.gpu
def test_single_tokens_without_offsets():
    lens = [5, 300, 64]
    c = Cache(lens, 2, 128, 16, torch.bfloat16)
    q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    a = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens)
    b = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=_cu([1, 1, 1]), max_seqlen_q=1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    _check_attn(*a, q, c, [1, 1, 1], lens, 128 ** -0.5, True, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 40])
def test_sequences_may_share_one_row_of_pages(n):
    """Several continuations of one prefix: a broadcast row of the block table."""
    c = Cache([333], 2, 64, 16, torch.bfloat16)
    q = torch.randn(3 * n, 4, 64, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    lens = torch.full((3,), 333, dtype=torch.int32, device="cuda")
    a = skl.streamkl_paged_attn(q, c.k, c.v, c.table.expand(3, -1), lens, cu_seqlens=_cu([n] * 3), max_seqlen_q=n)
    b = skl.streamkl_paged_attn(q, c.k, c.v, c.table.repeat(3, 1), lens, cu_seqlens=_cu([n] * 3), max_seqlen_q=n)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("n,splits", [(1, 0), (40, 1), (40, 3)])
def test_rows_in_front_of_the_first_sequence_stay(n, splits):
    c = Cache([500, 300], 2, 64, 16, torch.bfloat16, seed=n)
    q = torch.randn(2 * n + 5, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    o, lse = torch.full_like(q, 3.0), torch.full((2 * n + 5, 4), 3.0, device="cuda")
    st = binding.new_status()
    cu = torch.tensor([3, 3 + n, 3 + 2 * n], dtype=torch.int32, device="cuda")
    skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=cu, max_seqlen_q=n, max_kv_len=500,
                            num_splits=splits, out=(o, lse), dev_status=st)
    binding.raise_on_device_status(st)
    for rows in (slice(0, 3), slice(3 + 2 * n, None)):
        assert torch.all(o[rows] == 3) and torch.all(lse[rows] == 3)
    at = slice(3, 3 + 2 * n)
    _check_attn(o[at], lse[at], q[at], c, [n, n], [500, 300], 64 ** -0.5, True, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("B,HQ,HK,d,n,most", [(1, 8, 8, 64, 1, 130), (5, 12, 3, 128, 2, 300), (38, 32, 8, 64, 1, 512),
                                              (40, 8, 8, 64, 1, 512), (9, 2, 2, 128, 16, 512),
                                              (64, 8, 8, 64, 1, 250), (100, 16, 8, 128, 1, 200), (700, 2, 1, 64, 3, 100)])
def test_short_sequences_of_few_rows(B, HQ, HK, d, n, most):
    """Up to and past 2 x 152 (sequence, key head) pairs; sequences without keys or new tokens among them."""
    r = np.random.default_rng(B + d)
    lens = [most] + [int(x) for x in r.integers(0, most + 1, B - 1)]
    new = [n] + [int(x) for x in r.integers(0, n + 1, B - 1)]
    if B > 3:
        lens[1], new[1], new[2] = 0, n, 0
    c = Cache(lens, HK, d, 16, torch.bfloat16, seed=B)
    q = torch.randn(sum(new) + 1, HQ, d, generator=torch.Generator().manual_seed(B)).bfloat16().cuda()
    for causal in (True, False):
        o, lse = torch.full_like(q, 3.0), torch.full((sum(new) + 1, HQ), 3.0, device="cuda")
        st = binding.new_status()
        skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=_cu(new), max_seqlen_q=n, max_kv_len=most,
                                causal=causal, out=(o, lse), dev_status=st)
        binding.raise_on_device_status(st)
        assert torch.all(o[-1] == 3) and torch.all(lse[-1] == 3)
        _check_attn(o[:-1], lse[:-1], q[:-1], c, new, lens, d ** -0.5, causal, torch.bfloat16)


@pytest.mark.gpu
def test_single_tokens_whose_items_are_whole_follow_one_another():
    """Two tiles a sequence, none cut: each call's output is the next one's queries."""
    B, d = 152, 64
    c = Cache([256] * B, 1, d, 16, torch.bfloat16)
    table = torch.nn.functional.pad(c.table, (0, 60))  # (room for 1,024 keys, so that the joining kernel is launched)
    q0 = torch.randn(B, 1, d, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()

    def chain(wait):
        q = q0
        for _ in range(20):
            o, _ = skl.streamkl_paged_attn(q, c.k, c.v, table, c.lens, max_kv_len=1024)
            q = o * 16
            if wait:
                torch.cuda.synchronize()
        return q

    assert torch.equal(chain(True), chain(False))


@pytest.mark.gpu
@pytest.mark.parametrize("n,bound,splits", [(1, 300, 0), (1, 1024, 0), (40, 300, 1), (40, 1024, 3)])
def test_each_kernel_reports_and_leaves_the_other_sequences_right(n, bound, splits):
    """Whole sequences, equal shares of the tiles, chunks, chunks with split keys."""
    lens, HK, d = [300, 190], 2, 64
    q = torch.randn(2 * n, 4, d, generator=torch.Generator().manual_seed(n)).bfloat16().cuda()
    for what in ("nothing", "page", "negative page", "length", "negative length", "offsets", "NaN"):
        c = Cache(lens, HK, d, 16, torch.bfloat16)
        table = torch.nn.functional.pad(c.table, (0, 60), value=-7)
        cu = _cu([n, n])
        if what == "page":
            table[0, 5] = c.k.shape[0]
        elif what == "negative page":
            table[0, 18] = -1
        elif what == "length":
            c.lens[0] = bound + 1
        elif what == "negative length":
            c.lens[0] = -3
        elif what == "offsets":
            cu[0] = -1
        elif what == "NaN":
            c.k[c.table[0, 3].long(), 0, 5] = float("nan")
        st = binding.new_status()
        o, lse = skl.streamkl_paged_attn(q, c.k, c.v, table, c.lens, cu_seqlens=cu, max_seqlen_q=n, max_kv_len=bound,
                                         num_splits=splits, dev_status=st)
        if what in ("nothing", "NaN"):
            binding.raise_on_device_status(st)
        else:
            with pytest.raises(binding.StreamKLError):
                binding.raise_on_device_status(st)
        _check_attn(o[n:], lse[n:], q[n:], type("", (), {"rows": c.rows[1:]}), [n], lens[1:], d ** -0.5, True,
                    torch.bfloat16)
        if what == "NaN":
            assert torch.all(torch.isnan(o[:n, :2])) and torch.all(torch.isnan(lse[:n, :2]))
            assert torch.all(torch.isfinite(o[:n, 2:]))


@pytest.mark.gpu
def test_nan_in_one_sequence_stays_there():
    lens = [200, 200]
    c = Cache(lens, 1, 64, 16, torch.bfloat16)
    c.k[c.table[0, 3].long(), 0, 5] = float("nan")
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    q[1, 2, 9] = float("inf")
    o, lse = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens)
    assert torch.all(torch.isnan(o[0])) and torch.all(torch.isnan(lse[0]))
    assert torch.all(torch.isnan(o[1, 2])) and torch.all(torch.isfinite(o[1, [0, 1, 3]]))


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 1], [70, 40]])
def test_pages_past_32_bits(new):
    """Caches of more than 2^31 elements each, the sequences in the last pages."""
    HK, d, page, dt = 8, 128, 128, torch.bfloat16
    pages = (1 << 31) // (HK * page * d) + 40
    small = Cache([300, 1000], HK, d, page, dt, spare=0)
    big = []
    for t in (small.k, small.v):
        x = torch.empty(pages, HK, page, d, dtype=dt, device="cuda")
        x[pages - t.shape[0]:] = t
        big.append(x)
    table = torch.where(small.table < small.k.shape[0], small.table + (pages - small.k.shape[0]), small.table)
    q = torch.randn(sum(new), 16, d, generator=torch.Generator().manual_seed(0)).to(dt).cuda()
    kw = dict(cu_seqlens=_cu(new), max_seqlen_q=max(new), max_kv_len=1000)
    a = skl.streamkl_paged_attn(q, *big, table, small.lens, **kw)
    b = skl.streamkl_paged_attn(q, small.k, small.v, small.table, small.lens, **kw)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    k, v = (torch.randn(sum(new), HK, d, generator=torch.Generator().manual_seed(i)).to(dt).cuda() for i in (1, 2))
    skl.streamkl_paged_append(k, v, *big, table, small.lens, cu_seqlens=kw["cu_seqlens"])
    skl.streamkl_paged_append(k, v, small.k, small.v, small.table, small.lens, cu_seqlens=kw["cu_seqlens"])
    for x, y in zip(big, (small.k, small.v)):
        assert torch.equal(x[pages - y.shape[0]:].view(torch.int16), y.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["page", "length", "new tokens", "offsets"])
def test_attention_reports_what_does_not_fit(what):
    lens, new = [40, 300], [3, 3]
    c = Cache(lens, 2, 64, 16, torch.bfloat16)
    q = torch.randn(6, 4, 64, device="cuda").to(torch.bfloat16)
    cu = _cu(new)
    kw = dict(max_seqlen_q=3, max_kv_len=300)
    if what == "page":
        c.table[1, 5] = c.k.shape[0]
    elif what == "length":
        kw["max_kv_len"] = 299
    elif what == "new tokens":
        kw["max_seqlen_q"] = 2
    else:
        cu[2] = 7
    st = binding.new_status()
    skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=cu, dev_status=st, **kw)
    with pytest.raises(binding.StreamKLError) as e:
        binding.raise_on_device_status(st)
    assert e.value.status == binding.STREAMKL_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [0, 2])
def test_cache_lives_through_prefill_and_captured_decode_steps(splits):
    """A chunk of new tokens, then single tokens: norm + rotation of the
    queries, append, attention. The decode step is captured once and replayed,
    lengths advancing on the device; each step equals the eager calls bit for
    bit, and the whole the definition in fp64: rounding q and k to bf16 moves a
    logit by at most 2^-8 S each (S = scale sum |q k|, about 8 for these
    normal rows), so terms by 2 x 2^-8 S and the sums of terms and values by
    twice that; o differs by at most that share of sum p |v|."""
    dt, HQ, HK, d, page, eps = torch.bfloat16, 4, 2, 64, 16, 1e-6
    g = torch.Generator().manual_seed(0)
    start, steps = [37, 5, 300], 6
    B, width = len(start), 32
    dev = torch.device("cuda")
    cos, sin = _tables(width * page, d, dev)
    wq, wk = (1 + 0.2 * torch.randn(2, d, generator=g)).to(dev)
    table = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width).to(dev)

    def fresh():
        return [torch.full((B * width, HK, page, d), float("nan"), dtype=dt, device=dev) for _ in range(2)]

    pre = torch.randn(sum(start), HQ + 2 * HK, d, generator=g).to(dt).to(dev)
    dec = torch.randn(steps, B, HQ + 2 * HK, d, generator=g).to(dt).to(dev)
    cu = _cu(start)
    st = binding.new_status(dev)

    def forward(x, positions, caches, lens, cu_seqlens, n, ws, out=None):
        q, k, v = x[:, :HQ], x[:, HQ:HQ + HK], x[:, HQ + HK:]
        q, _ = skl.streamkl_qk_norm_rope_fwd(q, None, cos, sin, positions=positions, q_weight=wq, eps=eps, dev_status=st)
        skl.streamkl_paged_append(k, v, *caches, table, lens, cu_seqlens=cu_seqlens, cos=cos, sin=sin, k_weight=wk,
                                  eps=eps, dev_status=st)
        return skl.streamkl_paged_attn(q, *caches, table, lens, cu_seqlens=cu_seqlens, max_seqlen_q=n,
                                       num_splits=splits, out=out, workspace=ws, dev_status=st)

    pos = torch.cat([torch.arange(n) for n in start]).to(torch.int32).to(dev)
    ws = torch.empty(8 << 20, dtype=torch.uint8, device=dev)

    def prefill(caches):
        lens = torch.tensor(start, dtype=torch.int32, device=dev)
        return lens, forward(pre, pos, caches, lens, cu, max(start), ws)

    eager, eager_out = fresh(), []
    lens, first = prefill(eager)
    for i in range(steps):
        lens += 1
        eager_out.append([t.clone() for t in forward(dec[i], lens - 1, eager, lens, None, 1, ws)])

    caches = fresh()
    lens, again = prefill(caches)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    x = torch.empty_like(dec[0])
    out = (torch.empty(B, HQ, d, dtype=dt, device=dev), torch.empty(B, HQ, device=dev))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens.add_(1)
        forward(x, lens - 1, caches, lens, None, 1, ws, out)
    for i in range(steps):
        x.copy_(dec[i])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, eager_out[i]))
    for a, b in zip(eager, caches):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    binding.raise_on_device_status(st)

    tables = [_np(t) for t in (cos, sin)]
    for b in range(B):
        rows = torch.cat([pre[cu[b]:cu[b + 1]]] + [dec[i, b:b + 1] for i in range(steps)])
        n = rows.shape[0]
        c, s = (t[:n, None] for t in tables)
        q, _ = orc.norm_rope(_np(rows[:, :HQ]), _np(wq), c, s, eps, False)
        k, _ = orc.norm_rope(_np(rows[:, HQ:HQ + HK]), _np(wk), c, s, eps, False)
        k, v = (np.swapaxes(t, 0, 1) for t in (k, _np(rows[:, HQ + HK:])))
        ref, ref_lse, mag = orc.paged_attn(q, k, v, d ** -0.5, True)
        got = torch.cat([first[0][cu[b]:cu[b + 1]]] + [o[0][b:b + 1] for o in eager_out])
        got_lse = torch.cat([first[1][cu[b]:cu[b + 1]]] + [o[1][b:b + 1] for o in eager_out])
        S = d ** -0.5 * max(np.max(np.abs(q[:, h]) @ np.abs(k[h // 2]).T) for h in range(HQ))
        move = 2 * 2.0 ** -8 * S
        assert np.all(np.abs(_np(got) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * move) * mag)
        assert np.all(np.abs(_np(got_lse) - ref_lse) <= 1.1 * move)


@pytest.mark.gpu
def test_on_another_stream_and_the_same_in_every_run():
    lens, new = [900, 300], [40, 20]
    c = Cache(lens, 2, 128, 32, torch.bfloat16)
    q = torch.randn(60, 8, 128, device="cuda").to(torch.bfloat16)
    kw = dict(cu_seqlens=_cu(new), max_seqlen_q=40, max_kv_len=900, num_splits=3)
    a = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, stream=side,
                                workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # status, workspace and outputs made by the call, while the current stream
    # is held up: they belong to the stream given
    torch.cuda._sleep(20_000_000)
    b = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, stream=side, **kw)
    del kw["num_splits"]
    one = skl.streamkl_paged_attn(q[:2], c.k, c.v, c.table, c.lens, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    torch.cuda.synchronize()
    two = skl.streamkl_paged_attn(q[:2], c.k, c.v, c.table, c.lens)
    assert all(torch.equal(x, y) for x, y in zip(one, two))
    kw["num_splits"] = 3
    for _ in range(3):
        b = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, **kw)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 40])
def test_two_captured_calls_at_once(n):
    """Two graphs with a workspace each, replayed on two streams side by side."""
    lens = [900, 3000]
    c = Cache(lens, 2, 128, 32, torch.bfloat16)
    st = binding.new_status()
    graphs = []
    for seed in (0, 1):
        q = torch.randn(2 * n, 8, 128, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
        kw = dict(cu_seqlens=_cu([n, n]), max_seqlen_q=n, max_kv_len=3000, dev_status=st)
        ref = [t.clone() for t in skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, **kw)]
        kw["out"] = (torch.empty_like(ref[0]), torch.empty_like(ref[1]))
        kw["workspace"] = torch.empty(skl.streamkl_paged_attn_workspace_size(2, 2 * n, 8, 2, 128, n, 3000),
                                      dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, **kw)
        graphs.append((graph, torch.cuda.Stream(), kw, ref, q))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream, *_ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    binding.raise_on_device_status(st)
    for _, _, kw, ref, _ in graphs:
        assert all(torch.equal(x, y) for x, y in zip(kw["out"], ref))


@pytest.mark.gpu
@pytest.mark.parametrize("n,layout", [(1, "heads"), (40, "slots")])
def test_the_native_way_and_the_one_in_python_do_the_same(n, layout, monkeypatch):
    lens = [500, 300]
    g = torch.Generator().manual_seed(n)
    kv = torch.randn(2 * n, 2, 3, 64, generator=g).bfloat16().cuda()[:, :, :2]
    q = torch.randn(2 * n, 4, 64, generator=g).bfloat16().cuda()
    cos, sin = _tables(600, 32, "cuda")
    w = torch.randn(64, generator=g).cuda()
    native, st = binding.load().native, binding.new_status()
    cu = _cu([n, n])
    got = []
    for way in (native, None):
        monkeypatch.setattr(binding.load(), "native", way)
        c = Cache(lens, 2, 64, 16, torch.bfloat16, layout=layout)
        for offsets in [cu] + ([None] if n == 1 else []):
            for extra in (dict(), dict(cos=cos, sin=sin, k_weight=w, dev_status=st, interleaved=True)):
                skl.streamkl_paged_append(kv[:, 0], kv[:, 1], c.k, c.v, c.table, c.lens, cu_seqlens=offsets, **extra)
                got += [c.k.clone(), c.v.clone()]
            space = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
            for extra in (dict(), dict(max_seqlen_q=n, max_kv_len=500, scale=0.2, causal=False, workspace=space,
                                       dev_status=st), dict(scale=np.float64(0.2), num_splits=2)):
                got += skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=offsets, **extra)
    binding.raise_on_device_status(st)
    half = len(got) // 2
    assert all(torch.equal(torch.nan_to_num(a.float(), 7.0), torch.nan_to_num(b.float(), 7.0))
               for a, b in zip(got[:half], got[half:]))
    # it is the native way that takes ordinary calls, and it leaves the others alone
    assert native.attn(q, c.k, c.v, c.table, c.lens, cu, n, 500, 0.2, True, 0, None, st) is not None
    assert native.append(kv[:, 0], kv[:, 1], c.k, c.v, c.table, c.lens, cu, None, None, None, 1e-6, False, st) is True
    for bad in (dict(q=q.float()), dict(lens=c.lens.long()), dict(lens=c.lens[:1]), dict(q=q[:, :3]), dict(q=q.cpu()),
                dict(q=None), dict(table=c.table[0]), dict(cu=cu[:2]), dict(max_q=3 * n), dict(max_kv=1 << 20),
                dict(max_kv=1 << 40), dict(scale=0.0), dict(scale=1e300), dict(splits=-1), dict(space=space[:16])):
        a = dict(dict(q=q, lens=c.lens, table=c.table, cu=cu, max_q=n, max_kv=500, scale=0.2, splits=2, space=None), **bad)
        assert native.attn(a["q"], c.k, c.v, a["table"], a["lens"], a["cu"], a["max_q"], a["max_kv"], a["scale"], True,
                           a["splits"], a["space"], st) is None, bad


@pytest.mark.gpu
def test_debug_build_finds_nothing_and_gives_the_same():
    """Every TMA copy, TMEM access and barrier range-checked: no check fails
    and the results are the release build's."""
    for new, lens, HQ, HK, d, page, dtype, causal, splits, layout in ATTN:
        dt = TYPES[dtype]
        c = Cache(lens, HK, d, page, dt, layout=layout)
        q = torch.randn(sum(new), HQ, d, device="cuda").to(dt)
        kw = dict(cu_seqlens=_cu(new), max_seqlen_q=max(new), max_kv_len=max(lens), causal=causal, num_splits=splits)
        st = binding.new_status()
        a = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, dev_status=st, **kw)
        with binding.use_debug_library():
            b = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, dev_status=st, **kw)
        binding.raise_on_device_status(st)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------- the softmax's reference
def _put(c, b, k, v):
    """Sequence b of the cache holds keys k and values v [length, HK, d]."""
    n = k.shape[0]
    page = c.k.shape[2]
    at = torch.arange(n)
    p, s = c.table[b, at.cuda() // page].long(), (at % page).cuda()
    c.k[p, :, s], c.v[p, :, s] = k.cuda(), v.cuda()
    c.rows[b] = (k, v)


def _two_directions(d, g):
    """Orthogonal vectors of d elements 1 and -1 that begin alike: a score is scale q k, so k = x / d^0.5 of the query's
    own vector gives x."""
    a = torch.where(torch.rand(d, generator=g) < 0.5, 1.0, -1.0)
    return a, torch.cat((a[:d // 2], -a[d // 2:]))


def _rising_keys(L, d, first, second, keys, rise, dt, g):
    """Keys of small random scores, but for those at first[1] (second[1]) of every 128 from the 128th on, where the
    score of queries along first[0] (second[0]) is `rise` times the tile's number."""
    k = 0.05 * torch.randn(L, 1, d, generator=g)
    for vec, place in (first, second):
        for at in range(128 + place, L, 128):
            if at < keys:
                k[at, 0] += at // 128 * rise / d ** 0.5 * vec
    return k.to(dt)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rise", [("fp16", 20.0), ("bf16", 100.0)])
@pytest.mark.parametrize("d,n,splits", [(128, 150, 1), (128, 150, 2), (128, 40, 1), (64, 150, 1), (128, 16, 0), (64, 3, 0)])
@pytest.mark.parametrize("places", [(40, 110), (100, 127), (95, 96)])
def test_rows_of_a_warp_rise_at_different_keys_of_a_tile(d, n, splits, places, dtype, rise):
    """Even rows (head 0) meet a score far above all before it at one key of a tile, odd rows (head 1) at another:
    fp16 terms of 20 nats over the old reference (2^28) and bf16 terms of 100 (2^144) are infinite unless every row's
    reference moves. Bounds as in _check_attn."""
    dt = TYPES[dtype]
    g = torch.Generator().manual_seed(d + n)
    u, w = _two_directions(d, g)
    c = Cache([700], 1, d, 16, dt, fill=False)
    k = _rising_keys(700, d, (u, places[0]), (w, places[1]), 500, rise, dt, g)
    _put(c, 0, k, torch.randn(700, 1, d, generator=g).to(dt))
    q = torch.stack((u, w)).expand(n, 2, d).to(dt).cuda()
    for causal in (True, False):
        st = binding.new_status()
        o, lse = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=_cu([n]), max_kv_len=700, causal=causal,
                                         num_splits=splits, dev_status=st)
        binding.raise_on_device_status(st)
        _check_attn(o, lse, q, c, [n], [700], d ** -0.5, causal, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rise", [("fp16", 20.0), ("bf16", 100.0)])
@pytest.mark.parametrize("d,n,L,splits", [(128, 1, 500, 0), (64, 1, 700, 0), (128, 2, 3000, 0), (64, 8, 400, 0),
                                          (128, 150, 700, 1), (128, 40, 700, 2), (128, 20, 700, 1), (64, 150, 700, 1)])
def test_a_nan_query_leaves_the_other_rows_right(d, n, L, splits, dtype, rise):
    """One row of NaN (the last token's head 2) beside rows whose scores rise in every tile."""
    dt = TYPES[dtype]
    g = torch.Generator().manual_seed(d + n)
    u, w = _two_directions(d, g)
    c = Cache([L], 1, d, 16, dt, fill=False)
    k = _rising_keys(L, d, (u, 40), (w, 110), 600, rise, dt, g)
    _put(c, 0, k, torch.randn(L, 1, d, generator=g).to(dt))
    q = torch.stack((u, w, u, w)).repeat(n, 1, 1).to(dt).cuda()
    q[-1, 2, 7] = float("nan")
    st = binding.new_status()
    o, lse = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=_cu([n]), max_kv_len=L, num_splits=splits,
                                     dev_status=st)
    binding.raise_on_device_status(st)
    assert torch.all(torch.isnan(o[-1, 2])) and bool(torch.isnan(lse[-1, 2]))
    rest = [0, 1, 3]
    _check_attn(o[:, rest], lse[:, rest], q[:, rest], c, [n], [L], d ** -0.5, True, dt)
    if n > 1:
        _check_attn(o[:-1, 2:3], lse[:-1, 2:3], q[:-1, 2:3], type("", (), {"rows": [(k[:L - 1], c.rows[0][1][:L - 1])]}),
                    [n - 1], [L - 1], d ** -0.5, True, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("d,n,L,splits,where", [(128, 1, 100_001, 0, 5), (64, 2, 100_001, 0, 99_000), (128, 20, 60_013, 1, 70_000),
                                                (128, 40, 60_013, 3, 5), (128, 130, 20_011, 1, 5), (64, 130, 20_011, 1, 19_000)])
def test_fp16_keeps_many_small_terms_beside_a_large_one(d, n, L, splits, where):
    """One key (its value 0) 17.7 nats above all others: what the others add, terms of 2^-25.5 of the largest, is the
    output. A term is at least 2^6 times that against the row's reference, where fp16 steps are 2^-24: off by 2^-25 at
    most, 2^-31 of the largest term, which the sum of terms exceeds: L 2^-31 max |v| in all. The rest as in _check_attn,
    relative to sum p |v|. (With the largest term at 2^0 all others are below 2^-25 and lost.)"""
    dt = torch.float16
    g = torch.Generator().manual_seed(n)
    u, _ = _two_directions(d, g)
    where = min(where, L - n)
    c = Cache([L], 1, d, 64, dt, fill=False)
    k = (-(1.5625 if d == 128 else 2.2109375) * u).expand(L, 1, d).clone()
    v = 0.5 + torch.rand(L, 1, d, generator=g)
    k[where], v[where] = 0, 0
    _put(c, 0, k.to(dt), v.to(dt))
    q = u.expand(n, 1, d).to(dt).cuda()
    st = binding.new_status()
    o, lse = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=_cu([n]), max_kv_len=L, causal=False,
                                     num_splits=splits, dev_status=st)
    binding.raise_on_device_status(st)
    x, kk, vv = _np(q[:1]), _np(c.rows[0][0].transpose(0, 1)), _np(c.rows[0][1].transpose(0, 1))
    ref, ref_lse, mag = orc.paged_attn(x, kk, vv, d ** -0.5, False)  # (all rows alike)
    half = torch.finfo(dt).eps / 2
    S = d ** -0.5 * float(np.max(np.abs(x[0, 0]) @ np.abs(kk[0]).T))
    E = 2 * ((d + 12) * 2.0 ** -23 * S + 2.0 ** -21) + L * 2.0 ** -23
    tol = half * np.abs(ref) + (half + E) * mag + L * 2.0 ** -31 * np.abs(vv).max() + 2.0 ** -25
    err = np.abs(_np(o) - ref)
    assert np.all(err <= tol), float((err / tol).max())
    assert np.all(np.abs(_np(lse) - ref_lse) <= E + 2.0 ** -22 * np.abs(ref_lse))


@pytest.mark.gpu
@pytest.mark.parametrize("base", [4096, 8192, 16384, 20480])
@pytest.mark.parametrize("d,n,splits", [(128, 1, 0), (64, 4, 0), (128, 20, 1), (128, 150, 1), (64, 150, 1)])
def test_fp16_logits_whose_own_rounding_exceeds_a_term(d, n, splits, base):
    """Scores of 2^25 to 2^28 (log2), of which fp32 keeps steps of 2 to 16, and a maximum that rises by a few of them from
    tile to tile: fp16 ends 2^2 above the largest term that may stand against an old reference. All values are 1, so each
    output is a sum of rounded terms over their sum: 2^-11 off, the half step of a term, and 2^-11 of its own, beside
    fp32 sums of 23 tiles, 2^-17. lse is the largest score, within (d + 12) 2^-23 of it (_check_attn), and the log of up to
    L terms."""
    dt, L = torch.float16, 23 * 128
    g = torch.Generator().manual_seed(n)
    u, _ = _two_directions(d, g)
    u[0] = 1
    c = Cache([L], 1, d, 16, dt, fill=False)
    k = 0.5 * base * u.expand(L, 1, d).clone()
    for j in range(23):
        at = 128 * j + int(torch.randint(0, 128, (1,), generator=g))
        k[at, 0] = base * u
        k[at, 0, 0] = base * (1 + j / 512)
    _put(c, 0, k.to(dt), torch.ones(L, 1, d).to(dt))
    q = (480 * u * (128 / d) ** 0.5).repeat(n, 2, 1)
    q[:, 0, 0] = torch.randint(1, 9, (n,), generator=g).float() * 8
    q[:, 1, 0] = torch.randint(1, 400, (n,), generator=g).float()
    q = q.to(dt).cuda()
    st = binding.new_status()
    o, lse = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, cu_seqlens=_cu([n]), max_kv_len=L, causal=False,
                                     num_splits=splits, dev_status=st)
    binding.raise_on_device_status(st)
    assert torch.all((o.float() - 1).abs() <= 2.0 ** -10 + 2.0 ** -17)
    top = ((q.double() @ c.rows[0][0][:, 0].double().T.cuda()).amax(-1) * d ** -0.5)
    assert torch.all((lse.double() - top).abs() <= (d + 12) * 2.0 ** -23 * top + np.log(L))


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    from attention_kl_loss_gb300 import build
    build.build()
    return binding.load()


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_longlong * 3)]


_TABLES = [("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_longlong), ("kv_lens", ctypes.c_void_p),
           ("cu_seqlens", ctypes.c_void_p)]


class AppendArgs(ctypes.Structure):
    """streamkl_append_args of the header."""
    _fields_ = ([("struct_size", ctypes.c_size_t)] + [(n, Rows) for n in ("k", "v", "k_cache", "v_cache")] + _TABLES
                + [(n, ctypes.c_void_p) for n in ("cos", "sin", "k_weight", "dev_status")]
                + [(n, ctypes.c_int) for n in ("dtype", "B", "T", "HK", "d", "page_size", "num_pages", "max_pages", "rot",
                                               "table_len", "interleaved")] + [("eps", ctypes.c_float)])


class AttnArgs(ctypes.Structure):
    """streamkl_paged_attn_args of the header."""
    _fields_ = ([("struct_size", ctypes.c_size_t)] + [(n, Rows) for n in ("q", "out", "k_cache", "v_cache")] + _TABLES
                + [(n, ctypes.c_void_p) for n in ("lse", "workspace")] + [("ws_bytes", ctypes.c_size_t),
                                                                          ("dev_status", ctypes.c_void_p)]
                + [(n, ctypes.c_int) for n in ("dtype", "B", "T", "HQ", "HK", "d", "page_size", "num_pages", "max_pages",
                                               "max_seqlen_q", "max_kv_len", "causal", "num_splits")]
                + [("scale", ctypes.c_float)])


def _raw(cls, over, **base):
    """Arguments that only the host looks at: a refused call never uses its addresses."""
    a = cls(ctypes.sizeof(cls), block_table=4096, table_stride=4, kv_lens=4096, cu_seqlens=4096, dev_status=4096, B=2,
            T=5, HK=2, d=64, page_size=16, num_pages=9, max_pages=4, **base)
    for n, s in (("k_cache", (2048, 1024, 64)), ("v_cache", (2048, 1024, 64)), ("k", (0, 128, 64)), ("v", (0, 128, 64)),
                 ("q", (0, 256, 64)), ("out", (0, 256, 64))):
        if hasattr(a, n):
            setattr(a, n, Rows(4096, s))
    for n, v in over.items():
        rows, _, field = n.partition("__")
        if not field:
            setattr(a, n, v)
        elif field == "data":
            getattr(a, rows).data = v
        else:
            getattr(a, rows).stride[:] = v
    return ctypes.byref(a)


CACHE_REFUSED = [
    (dict(struct_size=8), 1), (dict(dtype=2), 2), (dict(d=80), 2), (dict(B=0), 1), (dict(T=0), 1), (dict(HK=0), 1),
    (dict(num_pages=0), 1), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=2048), 2),
    (dict(max_pages=1 << 27), 2), (dict(table_stride=-1), 1), (dict(block_table=None), 1), (dict(kv_lens=None), 1),
    (dict(cu_seqlens=None), 1), (dict(k_cache__data=None), 1), (dict(v_cache__data=4100), 1),
    (dict(k_cache__stride=(2048, 1024, 60)), 1), (dict(k_cache__stride=(2048, 1024, 0)), 1),
    (dict(v_cache__stride=(0, 1024, 64)), 1), (dict(dev_status=None), 1),
    (dict(k_cache__stride=(1024, 1024, 64)), 1), (dict(v_cache__stride=(2048, 1016, 64)), 1),  # pages, heads overlap
]


@pytest.mark.parametrize("over,status", CACHE_REFUSED + [
    (dict(table_stride=3), 1), (dict(k__data=4104), 1), (dict(v__data=None), 1), (dict(k__stride=(0, -128, 64)), 1),
    (dict(cos=None), 1),
    (dict(rot=8), 2), (dict(rot=72), 2), (dict(table_len=0), 1), (dict(eps=-1.0), 1),
    (dict(eps=-1.0, cos=None, sin=None), 1), (dict(interleaved=2), 1), (dict(T=1 << 30, HK=4), 2),
    (dict(k_weight=4104), 1),
])
def test_append_c_call_refuses(lib, over, status):
    a = _raw(AppendArgs, over, cos=4096, sin=4096, rot=64, table_len=64, eps=1e-6)
    assert lib.streamkl_paged_append(a, None) == status and lib.streamkl_last_error()


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
    with pytest.raises(ValueError, match="out of range"):
        call(*ok, eps="1")
    with pytest.raises(binding.StreamKLError):  # (infinite as a float)
        call(*ok, eps=1e300)


@pytest.mark.parametrize("over,status", CACHE_REFUSED + [
    (dict(HQ=0), 1), (dict(HQ=3), 1), (dict(max_seqlen_q=0), 1), (dict(max_seqlen_q=6), 1), (dict(max_kv_len=-1), 1),
    (dict(max_kv_len=65), 1), (dict(q__data=4104), 1), (dict(out__data=None), 1), (dict(out__data=4104), 1),
    (dict(lse=None), 1), (dict(causal=2), 1), (dict(num_splits=-1), 1), (dict(scale=0.0), 1),
    (dict(scale=float("inf")), 1), (dict(q__stride=(0, 256, 60)), 1), (dict(out__stride=(0, 256, 0)), 1),
    (dict(out__stride=(0, 128, 64)), 1), (dict(out__stride=(0, 64, 312)), 1),
    (dict(B=40000, T=40000, cu_seqlens=None, max_seqlen_q=1), 2),
    (dict(num_splits=2, max_pages=40, table_stride=40, max_kv_len=640), 1),
    (dict(num_splits=2, max_pages=40, table_stride=40, max_kv_len=640, workspace=4100, ws_bytes=1 << 20), 1),
])
def test_attention_c_call_refuses(lib, over, status):
    a = _raw(AttnArgs, over, HQ=4, max_seqlen_q=4, max_kv_len=64, scale=0.1, causal=1, num_splits=1, lse=4096)
    assert lib.streamkl_paged_attn(a, None) == status and lib.streamkl_last_error()


def test_native_calls_leave_what_they_do_not_know(lib):
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    for call in (lib.native.rope_fwd, lib.native.rope_bwd, lib.native.append, lib.native.attn):
        assert call() is None and call(None) is None and call(*[x] * 12) is None
        assert all(call(*[a] * n) is None for n in (12, 13, 15) for a in (x, None, 1, "text"))


def test_attention_splits_on_the_host(lib):
    splits, size = skl.streamkl_paged_attn_splits, skl.streamkl_paged_attn_workspace_size
    assert splits(1, 1, 32, 8, 128, 1, 4096) == 0                 # few rows: the persistent kernel
    assert splits(1, 8, 32, 8, 128, 8, 4096) == 0 and splits(1, 9, 32, 8, 128, 9, 4096) > 1
    assert splits(64, 64 * 512, 32, 8, 128, 512, 4096) == 1
    assert splits(1, 64, 32, 8, 128, 64, 100) == 1
    assert splits(1, 1, 32, 5, 128, 1, 100) == -1
    for args in ((1, 40, 32, 8, 128, 40, 4096), (3, 700, 8, 8, 64, 512, 131072)):
        s = splits(*args)
        need = s * args[1] * args[2] * (args[4] + 1) * 4 if s > 1 else 0
        assert need <= size(*args) < need + 256
    assert size(1, 1, 32, 8, 128, 1, 4096, 1) == 0
    # two parts of 32 rows a CTA; no more CTAs than key tiles
    assert size(1, 1, 4, 1, 64, 1, 1024) == 2 * 8 * 32 * 65 * 4
    assert size(1, 1, 4, 1, 64, 1, 512) == 0 and size(64, 64, 8, 8, 64, 1, 250) == 0  # CTAs take whole ones
    assert size(39, 39, 8, 8, 64, 1, 512) == 2 * 304 * 32 * 65 * 4                    # (more than 2 x 152 of them)
    assert size(64, 64, 32, 8, 128, 1, 16384) == size(1, 1, 1, 1, 128, 1, 1 << 20)


@pytest.mark.gpu
def test_attention_python_call_refuses():
    c = Cache([20, 40], 2, 64, 16, torch.bfloat16)
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    call = skl.streamkl_paged_attn
    for match, args, kw in [
        ("q must be", (q.half(), c.k, c.v, c.table, c.lens), {}),
        ("multiple of 2", (q[:, :3], c.k, c.v, c.table, c.lens), {}),
        ("d = 64", (q[..., :32], c.k, c.v, c.table, c.lens), {}),
        ("one token", (q[:1], c.k, c.v, c.table, c.lens), {}),
        (r"out\[0\]", (q, c.k, c.v, c.table, c.lens), dict(out=(q[:1], None))),
        (r"out\[1\]", (q, c.k, c.v, c.table, c.lens), dict(out=(q, torch.zeros(2, 3, device="cuda")))),
        ("workspace", (q, c.k, c.v, c.table, c.lens),
         dict(num_splits=2, max_kv_len=48, workspace=torch.empty(9, device="cuda"))),
    ]:
        if match == "workspace":
            kw["num_splits"], kw["max_kv_len"] = 2, None
            args = (q, c.k, c.v, c.table.repeat(1, 8), c.lens)
        with pytest.raises(ValueError, match=match):
            call(*args, **kw)
    o, lse = call(q[:0], c.k, c.v, c.table[:0], c.lens[:0], cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
