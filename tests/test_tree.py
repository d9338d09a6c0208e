"""Attention of drafted tokens over a paged cache against fp64, and a serving loop
of all that speculative decoding does with the cache (bounds as in test_paged.py)."""
import ctypes

import numpy as np
import pytest
import torch

import attention_kl_loss_gb300 as skl
from attention_kl_loss_gb300 import binding
from oracle import model_ops
from oracle import page_ops as orc
from test_paged import AttnArgs, CACHE_REFUSED, Cache, TYPES, _cu, _np, _put, _raw, _tables, _two_directions


def _masks(new, kind, seed=0):
    """Bits of each sequence's drafted tokens [n, n]."""
    rng = np.random.default_rng(seed)
    out = []
    for n in new:
        if kind == "tree":
            out.append(orc.ancestors([-1 if i == 0 or rng.random() < 0.1 else int(rng.integers(max(0, i - 6), i))
                                      for i in range(n)]))
        elif kind == "causal":
            out.append(np.tril(np.ones((n, n), dtype=bool)))
        elif kind == "any":  # later tokens, not oneself, whatever
            out.append(rng.random((n, n)) < 0.4)
        elif kind == "none":
            out.append(np.zeros((n, n), dtype=bool))
        else:  # every third row sees nothing of the drafted ones
            b = rng.random((n, n)) < 0.5
            b[::3] = False
            out.append(b)
    return out


def _words(bits, words, pad=0, spare=1):
    """The masks as the call takes them, rows `spare` words further apart than they are long; bits past a sequence's own
    tokens are set, which says nothing."""
    rows = []
    for b in bits:
        full = np.ones((b.shape[0], 32 * words), dtype=bool)
        full[:, :b.shape[1]] = b
        rows.append(orc.words_of(full, words + spare))
    rows.append(np.zeros((pad, words + spare), dtype=np.int32))
    return torch.from_numpy(np.concatenate(rows)).cuda()[:, :words]


def _check(o, lse, q, c, bits, new, lens, scale, dt):
    """Per element as test_paged._check_attn: a term of the softmax and its sum are each within D = (d + 12) 2^-23 S +
    2^-21 (S = scale sum |q k|), sums over L keys within L 2^-23 more; P and o are rounded to the type, eps / 2 of
    sum p |v| and of |o|; fp16 terms lose up to 2^-25 each of at most the largest |v|."""
    half = torch.finfo(dt).eps / 2
    at = 0
    for b, n in enumerate(new):
        k, v = (_np(t[:lens[b]].transpose(0, 1)) for t in c.rows[b])
        x = _np(q[at:at + n])
        seen = orc.seen_keys(bits[b], lens[b])
        ref, ref_lse, mag = orc.tree_attn(x, k, v, scale, seen)
        got, got_lse = _np(o[at:at + n]), _np(lse[at:at + n])
        at += n
        empty = np.isneginf(ref_lse)
        assert np.array_equal(empty, np.isneginf(got_lse)) and np.all(got[empty] == 0)
        if n == 0 or not seen.any():
            continue
        G = x.shape[1] // k.shape[0]
        there = seen.any(0)
        S = scale * max(np.max(np.abs(x[:, h]) @ np.abs(k[h // G][there]).T) for h in range(x.shape[1]))
        E = 2 * ((x.shape[2] + 12) * 2.0 ** -23 * S + 2.0 ** -21) + lens[b] * 2.0 ** -23
        tol = half * np.abs(ref) + (half + E) * mag
        if dt == torch.float16:
            tol = tol + lens[b] * 2.0 ** -25 * np.abs(v).max() + 2.0 ** -25
        err = np.abs(got - ref)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        fin = ~empty
        assert np.all(np.abs(got_lse[fin] - ref_lse[fin]) <= E + 2.0 ** -22 * np.abs(ref_lse[fin]))


TREE = [
    # new, lens, HQ, HK, d, page, type, masks, layout
    ([1], [1], 1, 1, 64, 16, "bf16", "tree", "heads"),
    ([1], [300], 4, 1, 128, 16, "bf16", "none", "heads"),
    ([8], [2048], 8, 2, 128, 16, "bf16", "tree", "heads"),
    ([5, 0, 8, 1], [5, 17, 700, 129], 6, 2, 64, 32, "fp16", "any", "slots"),
    ([7, 3, 8], [7, 3, 8], 4, 1, 128, 64, "bf16", "holes", "slots"),      # no key before the drafted: empty rows
    ([16, 9], [1000, 128], 8, 2, 128, 16, "fp16", "tree", "heads"),
    ([33, 20], [700, 20], 3, 1, 128, 16, "bf16", "any", "slots"),
    ([31, 32, 33], [159, 160, 161], 2, 1, 64, 16, "bf16", "tree", "heads"),  # a tile's border in every place
    ([64, 1, 40], [300, 2000, 64], 8, 8, 64, 128, "fp16", "tree", "heads"),
    ([64, 63], [128, 127], 4, 2, 128, 16, "bf16", "holes", "heads"),
    ([130], [900], 1, 1, 128, 256, "bf16", "tree", "heads"),
    ([100, 257], [2000, 300], 4, 4, 128, 16, "fp16", "any", "slots"),
    ([300, 4], [300, 513], 6, 2, 64, 32, "bf16", "tree", "heads"),
    ([290], [3000], 2, 1, 128, 1024, "bf16", "holes", "slots"),
    ([12, 30], [5, 0], 4, 2, 128, 16, "bf16", "causal", "heads"),          # fewer keys than drafted tokens
    ([150], [40], 2, 1, 64, 16, "fp16", "any", "heads"),
    ([6], [77], 160, 1, 64, 32, "bf16", "tree", "heads"),                  # one token's group wider than a tile
]


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,HQ,HK,d,page,dtype,kind,layout", TREE)
def test_tree_attention_matches_fp64(new, lens, HQ, HK, d, page, dtype, kind, layout):
    dt = TYPES[dtype]
    c = Cache(lens, HK, d, page, dt, layout=layout, seed=sum(lens))
    g = torch.Generator().manual_seed(HQ + d)
    total, pad = sum(new), 2
    q = torch.randn(total + pad, HQ + 2, d, generator=g).to(dt).cuda()[:, :HQ]
    bits = _masks(new, kind, seed=total)
    words = -(-max(new) // 32)
    mask = _words(bits, words, pad)
    o = torch.full((total + pad, HQ, d), 3.0, dtype=dt, device="cuda")
    lse = torch.full((total + pad, HQ), 3.0, device="cuda")
    st = binding.new_status()
    scale = d ** -0.5
    kw = dict(cu_seqlens=_cu(new), dev_status=st)
    ret = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, mask, max_seqlen_q=max(new), max_kv_len=max(lens),
                                       out=(o, lse), **kw)
    binding.raise_on_device_status(st)
    assert ret[0] is o and ret[1] is lse
    assert torch.all(o[total:] == 3) and torch.all(lse[total:] == 3)  # rows behind the last sequence
    _check(o, lse, q, c, bits, new, lens, scale, dt)
    # bounds left at their defaults, outputs made by the call
    o2, lse2 = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, mask, **kw)
    binding.raise_on_device_status(st)
    _check(o2, lse2, q, c, bits, new, lens, scale, dt)
    if kind == "causal" or len(new) == 1:  # a chain is a chunk
        chain = _words(_masks(new, "causal"), words, pad)
        a = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, chain, **kw)
        b = skl.streamkl_paged_attn(q, c.k, c.v, c.table, c.lens, **kw)
        binding.raise_on_device_status(st)
        assert torch.allclose(a[0][:total].float(), b[0][:total].float(), rtol=2 ** -6, atol=2 ** -6)


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,most,HQ,HK,d,page,dtype,kind,layout", [
    ([8], [8100], 8192, 16, 4, 128, 16, "bf16", "tree", "heads"),            # sixteen CTAs, four tiles each
    ([32], [4096], 5000, 2, 2, 64, 1024, "fp16", "any", "slots"),
    ([5, 0, 8, 1, 7], [5, 17, 1300, 129, 0], 4096, 8, 2, 128, 16, "bf16", "any", "heads"),  # fewer tiles than CTAs, or none
    ([8, 3], [3, 0], 4000, 4, 1, 128, 64, "fp16", "holes", "slots"),
    ([16, 11, 16, 9], [2000, 1025, 897, 896], 2000, 8, 4, 64, 32, "bf16", "holes", "heads"),
    ([8, 7, 6], [400, 385, 384], 400, 32, 8, 128, 16, "fp16", "tree", "slots"),
    ([4] * 20, list(range(250, 1250, 50)), 1200, 8, 4, 128, 128, "bf16", "tree", "heads"),
    ([1] * 9, [1, 2, 127, 128, 129, 255, 256, 257, 1000], 1000, 8, 4, 128, 16, "bf16", "tree", "heads"),
    # more than 32 rows: one and two row tiles, clusters of 8, 4 and 2
    ([16], [1000], 1024, 16, 4, 128, 16, "bf16", "tree", "heads"),
    ([30, 2, 0, 5], [1100, 1, 60, 0], 1200, 8, 2, 128, 32, "fp16", "any", "slots"),
    ([20] * 6, [1000, 129, 128, 640, 20, 7], 1024, 16, 8, 128, 64, "bf16", "holes", "heads"),
    ([64, 33, 1], [2000, 1500, 130], 2048, 8, 8, 64, 16, "bf16", "tree", "slots"),
    ([40] * 8, [1900, 1, 50, 128, 129, 700, 1024, 1999], 2048, 8, 8, 64, 128, "fp16", "any", "heads"),
    ([60, 17, 40], [1000, 300, 40], 1024, 32, 8, 128, 16, "bf16", "tree", "heads"),
    ([100, 90], [1024, 700], 1024, 24, 4, 128, 256, "fp16", "holes", "heads"),  # blocks of rows; the last of few
    ([200, 130, 3], [900, 513, 600], 1024, 4, 4, 64, 64, "bf16", "any", "slots"),
    ([100, 90, 70, 100], [900, 90, 512, 1023], 1024, 16, 4, 128, 32, "bf16", "any", "slots"),
])
def test_rows_over_a_cluster(new, lens, most, HQ, HK, d, page, dtype, kind, layout):
    dt = TYPES[dtype]
    c = Cache(lens, HK, d, page, dt, layout=layout, seed=sum(lens))
    table = _wide(c.table, page, most)
    q = torch.randn(sum(new), HQ, d, generator=torch.Generator().manual_seed(d)).to(dt).cuda()
    bits = _masks(new, kind, seed=len(lens))
    st = binding.new_status()
    ret = [skl.streamkl_paged_tree_attn(q, c.k, c.v, table, c.lens, _words(bits, -(-max(new) // 32)), cu_seqlens=_cu(new),
                                        max_seqlen_q=max(new), max_kv_len=most, dev_status=st) for _ in range(2)]
    binding.raise_on_device_status(st)
    assert skl.streamkl_paged_tree_attn_workspace_size(len(new), sum(new), HQ, HK, d, max(new), most) == 0
    _check(*ret[0], q, c, bits, new, lens, d ** -0.5, dt)
    assert torch.equal(ret[0][0], ret[1][0]) and torch.equal(ret[0][1], ret[1][1])


def _wide(table, page, most):
    """A table for sequences of up to `most` keys: behind the pages that are there, anything."""
    out = torch.full((table.shape[0], -(-most // page)), 2 ** 30, dtype=torch.int32, device="cuda")
    out[:, :table.shape[1]] = torch.where(table < 0, 2 ** 30, table)[:, :out.shape[1]]
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("most", [4096, 16384, 1 << 17, 1 << 20])
@pytest.mark.parametrize("new,lens,HQ,HK,d,page,dtype,kind,layout", [t for t in TREE if max(t[1]) > 100])
def test_any_bound_of_the_lengths(new, lens, HQ, HK, d, page, dtype, kind, layout, most):
    """max_kv_len decides how the work is dealt out (clusters, whole items, an even share; one or two row tiles), not what
    comes out."""
    dt = TYPES[dtype]
    c = Cache(lens, HK, d, page, dt, layout=layout, seed=sum(lens))
    q = torch.randn(sum(new), HQ, d, generator=torch.Generator().manual_seed(HQ + d)).to(dt).cuda()
    bits = _masks(new, kind, seed=sum(new))
    st = binding.new_status()
    o, lse = skl.streamkl_paged_tree_attn(q, c.k, c.v, _wide(c.table, page, most), c.lens, _words(bits, -(-max(new) // 32)),
                                          cu_seqlens=_cu(new), max_seqlen_q=max(new), max_kv_len=most, dev_status=st)
    binding.raise_on_device_status(st)
    _check(o, lse, q, c, bits, new, lens, d ** -0.5, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("most", [4096, 1 << 17])
@pytest.mark.parametrize("dtype,rise", [("fp16", 20.0), ("bf16", 100.0)])
@pytest.mark.parametrize("d,n", [(128, 16), (64, 16), (128, 50), (64, 50), (128, 150), (64, 150)])
def test_scores_that_rise_for_any_bound(d, n, dtype, rise, most):
    """Keys far above all before them, within the drafted ones and before; key 3 is not seen by any row, its key is NaN."""
    dt, L = TYPES[dtype], 900
    g = torch.Generator().manual_seed(d + n)
    u, w = _two_directions(d, g)
    c = Cache([L], 1, d, 16, dt, fill=False)
    k = 0.05 * torch.randn(L, 1, d, generator=g)
    for i, at in enumerate(range(40, L, 37)):
        k[at, 0] += (i % 7 + 1) * rise / d ** 0.5 * (u if i % 2 else w)
    _put(c, 0, k.to(dt), torch.randn(L, 1, d, generator=g).to(dt))
    q = torch.stack((u, w)).expand(n, 2, d).to(dt).cuda()
    bits = _masks([n], "any", seed=n)
    hidden = L - n + 3
    bits[0][:, 3] = False
    c.k[c.table[0, hidden // 16], 0, hidden % 16] = float("nan")
    st = binding.new_status()
    o, lse = skl.streamkl_paged_tree_attn(q, c.k, c.v, _wide(c.table, 16, most), c.lens, _words(bits, -(-n // 32)),
                                          cu_seqlens=_cu([n]), max_seqlen_q=n, max_kv_len=most, dev_status=st)
    binding.raise_on_device_status(st)
    _check(o, lse, q, c, bits, [n], [L], d ** -0.5, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("B,n,HQ,HK,d,most", [(B, n, HQ, HK, d, most) for n, HQ, HK, d in ((3, 8, 2, 128), (9, 6, 3, 64), (40, 4, 2, 128),
                                                                                       (70, 8, 8, 64), (33, 16, 2, 128))
                                              for B, most in ((2, 500), (2, 30000), (37, 130), (37, 4000), (330, 200), (330, 3000))])
def test_sequences_without_keys(B, n, HQ, HK, d, most):
    """Some sequences of length 0, among them the first and the last, however the work is dealt out: their rows are zeros
    and -inf, the others' right, rows of none as they were."""
    dt = torch.bfloat16
    rng = np.random.default_rng(B + n)
    lens = [0 if b in (0, B - 1) and B > 2 or rng.random() < 0.3 else int(rng.integers(1, min(most, 200))) for b in range(B)]
    new = [n] + [int(x) for x in rng.integers(0, n + 1, B - 1)]
    if B == 2:
        lens[0] = 0
    c = Cache(lens, HK, d, 16, dt, seed=n)
    total = sum(new)
    q = torch.randn(total + 3, HQ, d, generator=torch.Generator().manual_seed(B)).to(dt).cuda()
    bits = _masks(new, "holes", seed=B)
    o, lse = torch.full((total + 3, HQ, d), 3.0, dtype=dt, device="cuda"), torch.full((total + 3, HQ), 3.0, device="cuda")
    st = binding.new_status()
    skl.streamkl_paged_tree_attn(q, c.k, c.v, _wide(c.table, 16, most), c.lens, _words(bits, -(-n // 32), 3), cu_seqlens=_cu(new),
                                 max_seqlen_q=n, max_kv_len=most, dev_status=st, out=(o, lse))
    binding.raise_on_device_status(st)
    assert torch.all(o[total:] == 3) and torch.all(lse[total:] == 3)
    half, at, scale = torch.finfo(dt).eps / 2, 0, d ** -0.5
    for b, (m, length) in enumerate(zip(new, lens)):  # (bounds as in _check)
        r = slice(at, at + m)
        at += m
        if m == 0 or length == 0:
            assert not o[r].any() and torch.all(lse[r].isneginf())
            continue
        seen = torch.from_numpy(orc.seen_keys(bits[b], length)).cuda()
        ref, ref_lse, mag, S = _plain_parts(q[r], *(t.transpose(0, 1).cuda() for t in c.rows[b]), scale, seen, HQ // HK)
        E = 2 * ((d + 12) * 2.0 ** -23 * S + 2.0 ** -21) + length * 2.0 ** -23
        assert torch.all((o[r].double() - ref).abs() <= half * ref.abs() + (half + E) * mag), b
        none = ref_lse.isneginf()
        assert torch.equal(none, lse[r].isneginf()) and not o[r][none].any()
        assert torch.all((lse[r].double() - ref_lse)[~none].abs() <= E + 2.0 ** -22 * ref_lse[~none].abs()), b


@pytest.mark.gpu
@pytest.mark.parametrize("n,HQ,d", [(3, 4, 128), (40, 4, 64), (200, 2, 128)])
def test_no_keys_at_all(n, HQ, d):
    """max_kv_len 0, and sequences without tokens only."""
    c = Cache([0, 0, 0], 1, d, 16, torch.bfloat16)
    new = [n, 0, 2]
    q = torch.ones(sum(new), HQ, d, dtype=torch.bfloat16, device="cuda")
    mask = _words(_masks(new, "causal"), -(-n // 32))
    st = binding.new_status()
    kw = dict(max_seqlen_q=n, dev_status=st)
    for most in (0, 16):
        o, lse = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, mask, cu_seqlens=_cu(new), max_kv_len=most, **kw)
        assert not o.any() and torch.all(lse.isneginf())
        o, lse = torch.full_like(q, 3.0), torch.full((sum(new), HQ), 3.0, device="cuda")
        skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, mask, cu_seqlens=_cu([0, 0, 0]), max_kv_len=most, out=(o, lse), **kw)
        assert torch.all(o == 3) and torch.all(lse == 3)
    binding.raise_on_device_status(st)


@pytest.mark.gpu
def test_single_tokens_without_offsets():
    """One drafted token a sequence: its bit says whether it sees itself."""
    lens = [1, 16, 17, 129, 400]
    c = Cache(lens, 2, 128, 16, torch.bfloat16, seed=5)
    q = torch.randn(5, 8, 128, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    bits = [np.array([[b]]) for b in (False, True, False, True, False)]
    st = binding.new_status()
    o, lse = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, _words(bits, 1), dev_status=st)
    binding.raise_on_device_status(st)
    assert torch.all(torch.isneginf(lse[0])) and not o[0].any()  # the only key is not seen
    _check(o, lse, q, c, bits, [1] * 5, lens, 128 ** -0.5, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("d,n,HQ", [(128, 7, 4), (128, 40, 2), (64, 60, 1), (128, 150, 2), (64, 150, 2)])
def test_hidden_keys_may_hold_anything(d, n, HQ):
    """Drafted tokens 2 and 5 have keys of NaN and infinity (their values are numbers): rows that do not see them are
    right, and the tokens that see them are NaN or whatever these give."""
    dt, L = torch.bfloat16, 333
    c = Cache([L], 1, d, 16, dt, seed=n)
    k, v = c.rows[0]
    base = L - n
    for t, value in ((2, float("nan")), (5, float("inf"))):
        pos = base + t
        c.k[c.table[0, pos // 16], 0, pos % 16] = value
        k[pos] = value
    bits = _masks([n], "any", seed=n)[0]
    clean = ~(bits[:, 2] | bits[:, 5])
    assert 0 < clean.sum() < n
    q = torch.randn(n, HQ, d, generator=torch.Generator().manual_seed(n)).to(dt).cuda()
    st = binding.new_status()
    o, lse = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, _words([bits], -(-n // 32)), cu_seqlens=_cu([n]),
                                          max_kv_len=L, dev_status=st)
    binding.raise_on_device_status(st)
    rows = np.flatnonzero(clean)
    c.rows[0] = (torch.nan_to_num(k, nan=0.0, posinf=0.0), v)
    # (the rows as a sequence of their own: what they see of the drafted tokens)
    seen = orc.seen_keys(bits, L)[rows]
    kk, vv = (_np(t.transpose(0, 1)) for t in c.rows[0])
    ref, ref_lse, mag = orc.tree_attn(_np(q)[rows], kk, vv, d ** -0.5, seen)
    half = torch.finfo(dt).eps / 2
    S = d ** -0.5 * max(np.max(np.abs(_np(q)[rows][:, h]) @ np.abs(kk[0]).T) for h in range(HQ))
    E = 2 * ((d + 12) * 2.0 ** -23 * S + 2.0 ** -21) + L * 2.0 ** -23
    assert np.all(np.abs(_np(o)[rows] - ref) <= half * np.abs(ref) + (half + E) * mag)
    assert np.all(np.abs(_np(lse)[rows] - ref_lse) <= E + 2.0 ** -22 * np.abs(ref_lse))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rise", [("fp16", 20.0), ("bf16", 100.0)])
@pytest.mark.parametrize("d,n", [(128, 16), (64, 16), (128, 50), (64, 50), (128, 150), (64, 150)])
def test_scores_that_rise_within_the_drafted_keys(d, n, dtype, rise):
    """Even rows (head 0) meet a drafted key far above all before it, odd rows (head 1) another; whether they see it is
    the mask's."""
    dt, L = TYPES[dtype], 700
    g = torch.Generator().manual_seed(d + n)
    u, w = _two_directions(d, g)
    c = Cache([L], 1, d, 16, dt, fill=False)
    k = 0.05 * torch.randn(L, 1, d, generator=g)
    base = L - n
    for i, at in enumerate(range(base, L, 5)):
        k[at, 0] += (i % 7 + 1) * rise / d ** 0.5 * (u if i % 2 else w)
    _put(c, 0, k.to(dt), torch.randn(L, 1, d, generator=g).to(dt))
    q = torch.stack((u, w)).expand(n, 2, d).to(dt).cuda()
    for kind in ("tree", "any", "none"):
        bits = _masks([n], kind, seed=n)
        st = binding.new_status()
        o, lse = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, _words(bits, -(-n // 32)), cu_seqlens=_cu([n]),
                                              max_kv_len=L, dev_status=st)
        binding.raise_on_device_status(st)
        _check(o, lse, q, c, bits, [n], [L], d ** -0.5, dt)


def _plain(q, k, v, table, lens, cu, bits, scale):
    """fp64 on the device, a sequence at a time."""
    o, lse = [], []
    for b, n in enumerate(lens.tolist()):
        a, e = int(cu[b]), int(cu[b + 1])
        page = k.shape[2]
        p = table[b, :-(-n // page)].long()
        ks, vs = (t[p].transpose(0, 1).flatten(1, 2)[:, :n].double() for t in (k, v))
        seen = torch.from_numpy(orc.seen_keys(bits[b], n)).cuda()
        G = q.shape[1] // ks.shape[0]
        x = torch.einsum("ihd,hjd->ihj", q[a:e].double(), ks.repeat_interleave(G, 0)) * scale
        x = x.masked_fill(~seen[:, None], float("-inf"))
        z = torch.logsumexp(x, -1, keepdim=True)
        o.append(torch.einsum("ihj,hjd->ihd", (x - z).exp(), vs.repeat_interleave(G, 0)))
        lse.append(z[..., 0])
    return torch.cat(o), torch.cat(lse)


def _random(B, n, L, HQ, HK, d, page, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = -(-L // page)
    k, v = (torch.randn(B * per, HK, page, d, generator=g, device="cuda").to(dt) for _ in range(2))
    table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    rng = np.random.default_rng(seed)
    new = [n] + [int(x) for x in rng.integers(1, n + 1, B - 1)]
    lens = [L] + [int(max(a, x)) for a, x in zip(new[1:], rng.integers(1, L + 1, B - 1))]
    q = torch.randn(sum(new), HQ, d, generator=g, device="cuda").to(dt)
    return k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), new, q


@pytest.mark.gpu
@pytest.mark.parametrize("B,n,L,HQ,HK,d,page,dtype", [
    (32, 8, 9000, 16, 4, 128, 16, "bf16"), (20, 16, 12000, 16, 4, 128, 32, "bf16"), (9, 61, 7000, 16, 8, 64, 16, "fp16"),
    (40, 32, 3000, 8, 2, 128, 128, "fp16"), (3, 200, 15000, 8, 4, 128, 64, "bf16"), (100, 30, 800, 4, 4, 64, 64, "bf16"),
    (150, 33, 400, 2, 1, 128, 16, "bf16"), (1, 128, 40000, 1, 1, 128, 16, "bf16"), (2, 100, 30000, 8, 8, 64, 16, "bf16"),
    # three or four items to a CTA, cut where an equal share ends; and whole ones in turn
    (230, 40, 1500, 2, 2, 128, 16, "bf16"), (230, 150, 1500, 2, 2, 128, 32, "fp16"), (460, 40, 1500, 2, 2, 64, 16, "bf16"),
    (230, 140, 1500, 2, 2, 64, 64, "bf16"), (150, 50, 300, 4, 2, 128, 16, "bf16"), (300, 70, 300, 4, 2, 64, 16, "fp16"),
    (100, 90, 400, 8, 2, 128, 64, "bf16")])
def test_long_and_many_sequences(B, n, L, HQ, HK, d, page, dtype):
    """Loads that arrive late and items of every length. The relative 2-norm of o: rounding P gives at most eps / 2 of
    sum p |v| a term, in the norm at most eps / 2 of the norm of p v's parts (test_paged.py), o's own rounding eps / 2,
    E under 2e-3: eps + 2e-3; each element within half |o| + (half + E) sum p |v| is left to the tests above."""
    dt = TYPES[dtype]
    k, v, table, lens, new, q = _random(B, n, L, HQ, HK, d, page, dt, B + n)
    bits = _masks(new, "tree", seed=B)
    cu = _cu(new)
    st = binding.new_status()
    o, lse = skl.streamkl_paged_tree_attn(q, k, v, table, lens, _words(bits, -(-n // 32)), cu_seqlens=cu, max_seqlen_q=n,
                                          max_kv_len=L, dev_status=st)
    binding.raise_on_device_status(st)
    ref, ref_lse = _plain(q, k, v, table, lens, cu, bits, d ** -0.5)
    assert float((o.double() - ref).norm() / ref.norm()) <= torch.finfo(dt).eps + 2e-3
    # every row by itself: none is lost among the many
    worst = ((o.double() - ref).norm(dim=-1) / ref.norm(dim=-1)).max()
    assert float(worst) <= 2 * torch.finfo(dt).eps + 4e-3
    assert float((lse.double() - ref_lse).abs().max()) <= 2e-4
    again = skl.streamkl_paged_tree_attn(q, k, v, table, lens, _words(bits, -(-n // 32)), cu_seqlens=cu, max_seqlen_q=n,
                                         max_kv_len=L, dev_status=st)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])  # the same in every run


def _plain_parts(q, k, v, scale, seen, G):
    """fp64 on the device, one sequence: o, lse, sum_j p_j |v_j|, and scale sum |q k| at most."""
    ks, vs = k.double().repeat_interleave(G, 0), v.double().repeat_interleave(G, 0)
    x = torch.einsum("ihd,hjd->ihj", q.double(), ks) * scale
    most = float(torch.einsum("ihd,hjd->ihj", q.double().abs(), ks.abs()).max()) * scale
    x = x.masked_fill(~seen[:, None], float("-inf"))
    lse = torch.logsumexp(x, -1)
    p = (x - lse.masked_fill(lse.isneginf(), 0)[..., None]).exp()  # (0 in a row that sees nothing)
    return torch.einsum("ihj,hjd->ihd", p, vs), lse, torch.einsum("ihj,hjd->ihd", p, vs.abs()), most


@pytest.mark.gpu
@pytest.mark.parametrize("B,n,L,HQ,HK,d,page,dtype", [
    (32, 8, 9000, 16, 4, 128, 16, "bf16"), (20, 16, 12000, 16, 4, 128, 32, "fp16"), (9, 61, 7000, 16, 8, 64, 16, "fp16"),
    (3, 200, 15000, 8, 4, 128, 64, "bf16"), (1, 128, 40000, 1, 1, 128, 16, "bf16"), (2, 100, 30000, 8, 8, 64, 128, "bf16"),
    (230, 40, 1500, 2, 2, 128, 16, "bf16"), (230, 150, 1500, 2, 2, 128, 32, "fp16"), (460, 40, 1500, 2, 2, 64, 16, "bf16"),
    (230, 140, 1500, 2, 2, 64, 64, "bf16"), (6, 300, 9000, 4, 4, 64, 32, "fp16"), (2, 13, 50000, 8, 4, 64, 16, "bf16")])
def test_every_row_has_a_key_of_its_own(B, n, L, HQ, HK, d, page, dtype):
    """Long contexts and cut stretches, key by key: each row's query is one of the keys (of entries +-a, so that its own
    score stands some ten nats above all others together), at a border of a tile or page, an end of the sequence, or among
    the drafted tokens, hidden ones too. A key that is lost or leaks then is the whole row. Bounds per element as in
    _check."""
    dt = TYPES[dtype]
    k, v, table, lens, new, q = _random(B, n, L, HQ, HK, d, page, dt, B + n)
    g = torch.Generator(device="cuda").manual_seed(n)
    a = 1.5 if d == 128 else 2.0
    k.copy_((torch.randint(0, 2, k.shape, generator=g, device="cuda") * 2 - 1) * a)
    bits = _masks(new, "tree", seed=B)
    rng = np.random.default_rng(B + L)
    G, scale, ends = HQ // HK, d ** -0.5, np.cumsum([0] + new)
    flat = [c.transpose(1, 2).reshape(-1, HK, d) for c in (k, v)]  # [page slots, heads, d]
    rows = []  # of each sequence
    for b, length in enumerate(lens.tolist()):
        at = torch.arange(length, device="cuda")
        rows.append(table[b].long()[at // page] * page + at % page)
        m = new[b]
        edges = [x for t in range(0, length + 1, min(128, page)) for x in (t - 1, t) if 0 <= x < length]
        edges = edges + 8 * [x for x in (0, length - m - 1, length - m, length - 1) if x >= 0]
        wanted = np.where(rng.random((m, HQ)) < 0.4, rng.integers(length - m, length, (m, HQ)), rng.choice(edges, (m, HQ)))
        slots = rows[b][torch.from_numpy(wanted).cuda()]
        q[ends[b]:ends[b + 1]] = flat[0][slots, torch.arange(HQ, device="cuda") // G]
    st = binding.new_status()
    o, lse = skl.streamkl_paged_tree_attn(q, k, v, table, lens, _words(bits, -(-n // 32)), cu_seqlens=_cu(new), max_seqlen_q=n,
                                          max_kv_len=L, dev_status=st)
    binding.raise_on_device_status(st)
    half = torch.finfo(dt).eps / 2
    own = total = 0
    for b, length in enumerate(lens.tolist()):
        r = slice(int(ends[b]), int(ends[b + 1]))
        seen = torch.from_numpy(orc.seen_keys(bits[b], length)).cuda()
        kk, vv = (c[rows[b]].transpose(0, 1) for c in flat)
        ref, ref_lse, mag, S = _plain_parts(q[r], kk, vv, scale, seen, G)
        E = 2 * ((d + 12) * 2.0 ** -23 * S + 2.0 ** -21) + length * 2.0 ** -23
        tol = half * ref.abs() + (half + E) * mag
        if dt == torch.float16:
            tol = tol + length * 2.0 ** -25 * float(vv.abs().max()) + 2.0 ** -25
        assert torch.all((o[r].double() - ref).abs() <= tol), b
        assert torch.all((lse[r].double() - ref_lse).abs() <= E + 2.0 ** -22 * ref_lse.abs()), b
        own += int((ref_lse > S - 1).sum())
        total += ref_lse.numel()
    # (of the inputs, by the fp64 sums: 0.6 of the rows are given a key at a border; short sequences hide many of those)
    assert 0.3 * total < own < total


@pytest.mark.gpu
@pytest.mark.parametrize("n,HQ", [(6, 4), (25, 4), (90, 4)])
def test_one_bad_sequence_leaves_the_others_right(n, HQ):
    """Lengths, pages and offsets that do not fit are reported; the other sequences' rows are computed."""
    lens, new = [200, 300, 250], [n, n - 2, n]
    bits = _masks(new, "tree")
    for what in ("page", "length", "negative"):
        c = Cache(lens, 1, 128, 16, torch.bfloat16, seed=3)
        q = torch.randn(sum(new), HQ, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
        if what == "page":
            c.table[1, 3] = -4
        else:
            c.lens[1] = 16 * c.table.shape[1] + 1 if what == "length" else -1
        st = binding.new_status()
        o, lse = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, _words(bits, -(-n // 32)), cu_seqlens=_cu(new),
                                              max_kv_len=300, dev_status=st)
        assert int(st.item()) == binding.STREAMKL_ERR_INVALID_ARG
        for b, at in ((0, 0), (2, sum(new[:2]))):
            rows = slice(at, at + new[b])
            one = type("", (), {"rows": [c.rows[b]]})
            _check(o[rows], lse[rows], q[rows], one, [bits[b]], [new[b]], [lens[b]], 128 ** -0.5, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("n,HQ", [(6, 4), (25, 4), (90, 4)])
def test_captured_on_another_stream_and_both_ways(n, HQ, monkeypatch):
    """A captured call with its own workspace replays with new lengths and masks; a given stream is used; ctypes does what
    the native way does."""
    L = 500
    c = Cache([L, 300], 2, 64, 16, torch.bfloat16, seed=n)
    q = torch.randn(2 * n, HQ, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    words = -(-n // 32)
    bits = _masks([n, n], "tree", seed=1)
    mask = _words(bits, words).contiguous()
    st = binding.new_status()
    kw = dict(cu_seqlens=_cu([n, n]), max_seqlen_q=n, max_kv_len=L, dev_status=st)
    a = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, mask, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, mask, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    lib = binding.load()
    with monkeypatch.context() as m:
        m.setattr(lib, "native", None)
        w = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, mask, **kw)
    for x in (b, w):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, mask, **kw)
    bits = _masks([n, n], "any", seed=7)
    mask.copy_(_words(bits, words))
    c.lens.copy_(torch.tensor([440, 299], dtype=torch.int32))
    graph.replay()
    binding.raise_on_device_status(st)
    _check(out[0], out[1], q, c, bits, [n, n], [440, 299], 64 ** -0.5, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("n,HQ,L", [(6, 4, 300), (25, 4, 300), (25, 4, 20000), (90, 4, 300), (90, 4, 9000)])
def test_rows_in_front_of_the_first_sequence_stay(n, HQ, L):
    c = Cache([L, 100], 1, 64, 16, torch.bfloat16, seed=n)
    new = [n, 3]
    total = sum(new) + 7
    q = torch.randn(total, HQ, 64, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    bits = _masks(new, "tree", seed=2)
    mask = torch.zeros(total, -(-n // 32), dtype=torch.int32, device="cuda")
    mask[4:4 + sum(new)] = _words(bits, -(-n // 32))
    o = torch.full((total, HQ, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total, HQ), 3.0, device="cuda")
    st = binding.new_status()
    skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, mask, cu_seqlens=_cu(new) + 4, max_seqlen_q=n, max_kv_len=L,
                                 out=(o, lse), dev_status=st)
    binding.raise_on_device_status(st)
    for rows in (slice(0, 4), slice(4 + sum(new), None)):
        assert torch.all(o[rows] == 3) and torch.all(lse[rows] == 3)
    own = slice(4, 4 + sum(new))
    _check(o[own], lse[own], q[own], c, bits, new, [L, 100], 64 ** -0.5, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("d,n", [(128, 2), (64, 8), (128, 12), (64, 20), (128, 40), (64, 40)])
def test_a_nan_query_leaves_the_other_rows_right(d, n):
    """Scores rise by 100 (log: of bf16's terms to infinity) along the keys; one row, the last token's head 2, is NaN."""
    dt, L, HQ = torch.bfloat16, 600, 4
    g = torch.Generator().manual_seed(d + n)
    u, w = _two_directions(d, g)
    c = Cache([L], 1, d, 16, dt, fill=False)
    k = 0.05 * torch.randn(L, 1, d, generator=g)
    for at in range(40, L, 90):
        k[at, 0] += at / 6 / d ** 0.5 * (u if at % 4 else w)
    _put(c, 0, k.to(dt), torch.randn(L, 1, d, generator=g).to(dt))
    q = torch.stack((u, w, u, w)).repeat(n, 1, 1).to(dt).cuda()
    q[-1, 2, 7] = float("nan")
    bits = _masks([n], "causal")
    st = binding.new_status()
    o, lse = skl.streamkl_paged_tree_attn(q, c.k, c.v, c.table, c.lens, _words(bits, -(-n // 32)), cu_seqlens=_cu([n]),
                                          max_kv_len=L, dev_status=st)
    binding.raise_on_device_status(st)
    assert torch.all(torch.isnan(o[-1, 2])) and bool(torch.isnan(lse[-1, 2]))
    rest = [0, 1, 3]
    _check(o[:, rest], lse[:, rest], q[:, rest], c, bits, [n], [L], d ** -0.5, dt)
    if n > 1:
        one = type("", (), {"rows": [(c.rows[0][0][:L - 1], c.rows[0][1][:L - 1])]})
        _check(o[:-1, 2:3], lse[:-1, 2:3], q[:-1, 2:3], one, [bits[0][:-1, :-1]], [n - 1], [L - 1], d ** -0.5, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("n,HQ,L", [(6, 4, 4000), (25, 4, 9000), (90, 4, 3000)])
def test_two_captured_calls_at_once(n, HQ, L):
    """Two graphs, each with the workspace that its capture made, replayed on two streams at the same time."""
    parts = []
    for seed in (0, 1):
        k, v, table, lens, new, q = _random(5, n, L, HQ, 1, 128, 16, torch.bfloat16, seed)
        args = (q, k, v, table, lens, _words(_masks(new, "tree", seed), -(-n // 32)))
        kw = dict(cu_seqlens=_cu(new), max_seqlen_q=n, max_kv_len=L, dev_status=binding.new_status())
        want = skl.streamkl_paged_tree_attn(*args, **kw)
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            out = skl.streamkl_paged_tree_attn(*args, **kw)
        parts.append((graph, stream, want, out, kw["dev_status"], args, kw))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream, *_ in parts:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, want, out, st, *_ in parts:
        binding.raise_on_device_status(st)
        assert torch.equal(want[0], out[0]) and torch.equal(want[1], out[1])


def test_workspace_sizes_on_the_host(lib):
    size = skl.streamkl_paged_tree_attn_workspace_size
    assert size(1, 8, 32, 8, 128, 8, 512) == 0                           # few rows of few tiles: whole ones
    assert size(1, 8, 32, 8, 128, 8, 65536) == 2 * 304 * 32 * 129 * 4     # few rows, cut: two parts of 32 rows a CTA
    assert size(1, 8, 32, 8, 128, 8, 2048) == 0                            # a cluster for each item
    assert size(1, 9, 32, 8, 128, 9, 512) == 0 and size(64, 64 * 16, 32, 8, 128, 16, 128) == 0

    def parts(ctas, rows, d):
        return (2 * ctas * rows * (d + 1) * 4 + ctas * 24 + 255) // 256 * 256

    assert size(64, 64 * 16, 32, 8, 128, 16, 16384) == parts(152, 128, 128)
    assert size(4, 4 * 256, 32, 8, 128, 256, 16384) == parts(152, 256, 128)
    assert size(24, 24 * 61, 8, 8, 64, 61, 5000) == parts(304, 128, 64)    # two CTAs an SM
    assert size(1, 40, 1, 1, 128, 40, 16384) == parts(128, 128, 128)       # no more CTAs than key tiles
    assert size(1, 40, 1, 1, 128, 40, 1000) == 0                           # a cluster of them
    assert size(1, 40, 3, 2, 128, 40, 1000) == 0 and size(1, 40, 1, 1, 80, 40, 1000) == 0  # no sizes of a call


@pytest.mark.gpu
def test_debug_build_finds_nothing_and_gives_the_same():
    from attention_kl_loss_gb300 import build
    build.build(debug=True)
    for n, HQ, d in ((8, 4, 128), (30, 4, 128), (90, 2, 64), (200, 2, 128)):
        k, v, table, lens, new, q = _random(4, n, 2000, HQ, 1, d, 16, torch.bfloat16, n)
        args = (q, k, v, table, lens, _words(_masks(new, "tree"), -(-n // 32)))
        kw = dict(cu_seqlens=_cu(new), max_seqlen_q=n, max_kv_len=2000)
        st = binding.new_status()
        a = skl.streamkl_paged_tree_attn(*args, dev_status=st, **kw)
        with binding.use_debug_library():
            b = skl.streamkl_paged_tree_attn(*args, dev_status=st, **kw)
        binding.raise_on_device_status(st)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------- all together
@pytest.mark.gpu
@pytest.mark.parametrize("seed,HQ,HK,d,page,dtype", [(0, 4, 2, 64, 16, "bf16"), (1, 8, 2, 128, 32, "fp16")])
def test_a_serving_loop(seed, HQ, HK, d, page, dtype):
    """Prompts, beams on them, drafted trees, accepted paths, ends: two layers over one set of tables. Keys are normed and
    rotated by their depth on the way in. What each sequence's cache holds is what a list of its own tokens holds, and the
    attention of every drafted token is that of fp64 over that list and its branch (bounds as in _check)."""
    dt = TYPES[dtype]
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    B, width, pages, layers = 6, 12, 50, 2
    dev = torch.device("cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    caches = [[torch.full((pages, HK, page, d), float("nan"), dtype=dt, device=dev) for _ in range(2)] for _ in range(layers)]
    held = [[[] for _ in range(B)] for _ in range(layers)]  # (key, value) rows of each sequence
    weight = (1 + 0.1 * torch.randn(d, generator=g)).to(dev)
    cos, sin = _tables(width * page, d, dev)
    st = binding.new_status()

    def i32(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)

    def resize(to):
        copies = skl.streamkl_paged_resize(refs, table, lens, i32(to), page, dev_status=st)
        for k, v in caches:
            skl.streamkl_paged_copy(k, v, copies, dev_status=st)
        assert lens.tolist() == list(to)
        orc.check_held(refs.cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy(), page)

    def put(new, depths):
        """New tokens of every sequence, whose pages are there: keys normed and rotated by position, then appended."""
        total = sum(new)
        if total == 0:
            return
        for layer, (k, v) in enumerate(caches):
            kv = torch.randn(total, 2 * HK, d, generator=g).to(dt).to(dev)
            _, rows = skl.streamkl_qk_norm_rope_fwd(None, kv[:, :HK], cos, sin, k_positions=i32(depths), k_weight=weight,
                                                    dev_status=st)
            skl.streamkl_paged_append(rows, kv[:, HK:], k, v, table, lens, cu_seqlens=_cu(new), dev_status=st)
            at = 0
            for b, n in enumerate(new):
                held[layer][b] += [(rows[at + i].cpu(), kv[at + i, HK:].cpu()) for i in range(n)]
                at += n

    def check_caches():
        t, n = table.cpu().numpy(), lens.tolist()
        for layer, pair in enumerate(caches):
            for b in range(B):
                for which in range(2):
                    cache = pair[which].cpu()
                    for pos in range(n[b]):
                        assert torch.equal(cache[t[b, pos // page], :, pos % page], held[layer][b][pos][which]), (layer, b, pos)

    prompts = [37, 0, 0, 20, 0, page]
    resize(prompts)
    put(prompts, [i for n in prompts for i in range(n)])
    source = [0, 0, 0, 3, 3, 5]  # beams of the two prompts
    skl.streamkl_paged_fork(refs, table, lens, i32(source), dev_status=st)
    for layer in range(layers):
        held[layer] = [list(held[layer][s]) for s in source]
    check_caches()
    for step in range(6):
        base = lens.tolist()
        new = [int(x) for x in rng.integers(1, 14, B)]
        if step == 3:  # some end, others go on from their neighbours
            source = [1, 1, 2, 4, 4, 2]
            skl.streamkl_paged_fork(refs, table, lens, i32(source), dev_status=st)
            base = lens.tolist()
            for layer in range(layers):
                held[layer] = [list(held[layer][s]) for s in source]
        if step == 4:
            resize([0 if b == 2 else n for b, n in enumerate(base)])
            base = lens.tolist()
            for layer in range(layers):
                held[layer][2] = []
        resize([a + n for a, n in zip(base, new)])
        parents = [[-1 if i == 0 else int(rng.integers(max(0, i - 4), i)) for i in range(n)] for n in new]
        bits = [orc.ancestors(p) for p in parents]
        put(new, [base[b] + int(x.sum()) - 1 for b, rows in enumerate(bits) for x in rows])
        check_caches()
        total, mask = sum(new), _words(bits, 1)
        for layer, (k, v) in enumerate(caches):
            q = torch.randn(total, HQ, d, generator=g).to(dt).to(dev)
            o, lse = skl.streamkl_paged_tree_attn(q, k, v, table, lens, mask, cu_seqlens=_cu(new), max_seqlen_q=max(new),
                                                  dev_status=st)
            binding.raise_on_device_status(st)
            rows = [tuple(torch.stack([x[i] for x in held[layer][b]]) for i in range(2)) for b in range(B)]
            _check(o, lse, q, type("", (), {"rows": rows}), bits, new, lens.tolist(), d ** -0.5, dt)
        # a branch of each tree is accepted
        paths = [np.flatnonzero(bits[b][int(rng.integers(0, new[b]))]).tolist() for b in range(B)]
        kept = np.zeros((B, 14), np.int32)
        for b, p in enumerate(paths):
            kept[b, :len(p)] = p
        for k, v in caches:
            skl.streamkl_paged_compact(k, v, table, lens, _cu(new), i32(kept), i32([len(p) for p in paths]), dev_status=st)
        for layer in range(layers):
            for b, p in enumerate(paths):
                tail = held[layer][b][base[b]:]
                held[layer][b] = held[layer][b][:base[b]] + [tail[i] for i in p]
        resize([a + len(p) for a, p in zip(base, paths)])
        check_caches()
    resize([0] * B)
    assert not refs.any() and torch.all(table == -1)
    binding.raise_on_device_status(st)


@pytest.mark.gpu
@pytest.mark.parametrize("HQ,HK,d,dtype", [(4, 2, 64, "bf16"), (40, 2, 128, "fp16")])
def test_a_captured_step_without_enough_pages_leaves_the_others_keys(HQ, HK, d, dtype):
    """Sequences 0 and 1 hold the same partly filled last page and no page is free: neither gets places, nothing of theirs
    changes, and 2, which needs no page, goes on. Once 3 has ended the same graph serves all."""
    dt, page, pages, n = TYPES[dtype], 16, 5, 4
    g = torch.Generator().manual_seed(d)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.full((4, 3), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(pages, HK, page, d, dtype=dt, device="cuda") for _ in range(2))

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def rows(count, heads):
        return torch.randn(count, heads, d, generator=g).to(dt).cuda()

    first = [20, 0, 22, 9]
    skl.streamkl_paged_resize(refs, table, lens, i32(first), page)
    x = rows(sum(first), HK), rows(sum(first), HK)
    skl.streamkl_paged_append(*x, k, v, table, lens, cu_seqlens=_cu(first))
    skl.streamkl_paged_fork(refs, table, lens, i32([0, 0, 2, 3]))
    held = [[t[a:e] for t in x] for a, e in ((0, 20), (0, 20), (20, 42), (42, 51))]
    assert lens.tolist() == [20, 20, 22, 9] and refs.tolist() == [2, 2, 1, 1, 1]
    new, bits = [n, n, n, 0], _masks([n, n, n, 0], "causal")
    mask, cu, q, x = _words(bits, 1).contiguous(), _cu(new), rows(3 * n, HQ), (rows(3 * n, HK), rows(3 * n, HK))
    kept, wanted, step = i32([[0, 2]] * 4), i32([24, 24, 26, 9]), torch.full((4,), -9, dtype=torch.int32, device="cuda")
    room, st = binding.new_status(), binding.new_status()

    def one_step():
        before = lens.clone()
        copies = skl.streamkl_paged_resize(refs, table, lens, wanted, page, dev_status=room, step_lens=step)
        skl.streamkl_paged_copy(k, v, copies, dev_status=st)
        skl.streamkl_paged_append(*x, k, v, table, step, cu_seqlens=cu, dev_status=st)
        out = skl.streamkl_paged_tree_attn(q, k, v, table, step, mask, cu_seqlens=cu, max_seqlen_q=n, max_kv_len=48, dev_status=st)
        num = ((step > 0) * i32_two).to(torch.int32)
        skl.streamkl_paged_compact(k, v, table, step, cu, kept, num, dev_status=st)
        skl.streamkl_paged_resize(refs, table, lens, before + num, page, dev_status=st)
        return out

    def check_held():
        t, ln = table.cpu().numpy(), lens.tolist()
        for b in range(4):
            assert ln[b] == len(held[b][0]), b
            for cache, want in zip((k, v), held[b]):
                got = [cache[t[b, p // page], :, p % page] for p in range(ln[b])]
                assert ln[b] == 0 or torch.equal(torch.stack(got), want), b
        orc.check_held(refs.cpu().numpy(), t, np.array(ln, dtype=np.int32), page)

    i32_two = i32([2, 2, 2, 0])
    side = [t.clone() for t in (refs, table, lens, k, v)]  # (the calls' first run, undone)
    one_step()
    for t, old in zip((refs, table, lens, k, v), side):
        t.copy_(old)
    for word in (room, st):
        word.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = one_step()
    check_held()

    graph.replay()
    assert int(room.item()) == binding.STREAMKL_ERR_NO_PAGES and step.tolist() == [0, 0, 26, 9]
    assert int(st.item()) == binding.STREAMKL_ERR_INVALID_ARG  # tokens without places
    o, lse = out
    assert not o[:2 * n].any() and torch.all(torch.isneginf(lse[:2 * n]))
    one = type("", (), {"rows": [[torch.cat((a, y[2 * n:])) for a, y in zip(held[2], x)]]})
    _check(o[2 * n:], lse[2 * n:], q[2 * n:], one, [bits[2]], [n], [26], d ** -0.5, dt)
    held[2] = [torch.cat((a, y[[2 * n, 2 * n + 2]])) for a, y in zip(held[2], x)]
    check_held()

    for word in (room, st):
        word.zero_()
    skl.streamkl_paged_resize(refs, table, lens, i32([20, 20, 24, 0]), page)
    held[3] = [t[:0] for t in held[3]]
    wanted.copy_(i32([24, 24, 28, 0]))
    graph.replay()
    for word in (room, st):
        binding.raise_on_device_status(word)
    assert step.tolist() == [24, 24, 28, 0]
    all_rows = type("", (), {"rows": [[torch.cat((a, y[b * n:(b + 1) * n])) for a, y in zip(held[b], x)] for b in range(3)]})
    _check(o, lse, q, all_rows, bits, [n] * 3, [24, 24, 28], d ** -0.5, dt)
    held[:3] = [[torch.cat((a, y[[b * n, b * n + 2]])) for a, y in zip(held[b], x)] for b in range(3)]
    check_held()


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    from attention_kl_loss_gb300 import build
    build.build()
    return binding.load()


class TreeArgs(ctypes.Structure):
    """streamkl_paged_tree_attn_args of the header."""
    _fields_ = [("struct_size", ctypes.c_size_t), ("attn", AttnArgs), ("mask", ctypes.c_void_p),
                ("mask_stride", ctypes.c_longlong), ("mask_words", ctypes.c_int)]


@pytest.mark.parametrize("over,status", CACHE_REFUSED + [
    (dict(HQ=3), 1), (dict(max_seqlen_q=0), 1), (dict(max_seqlen_q=6), 1), (dict(max_kv_len=65), 1), (dict(q__data=4104), 1),
    (dict(out__data=None), 1), (dict(lse=None), 1), (dict(causal=1), 1), (dict(num_splits=2), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(out__stride=(0, 128, 64)), 1)])
def test_tree_c_call_refuses_what_the_attention_does(lib, over, status):
    base = dict(HQ=4, max_seqlen_q=4, max_kv_len=64, scale=0.1, causal=0, num_splits=0, lse=4096)
    attn = _raw(AttnArgs, over, **base)._obj
    t = TreeArgs(ctypes.sizeof(TreeArgs), attn, 4096, 1, 1)
    assert lib.streamkl_paged_tree_attn(ctypes.byref(t), None) == status and lib.streamkl_last_error()


@pytest.mark.parametrize("over", [dict(struct_size=8), dict(mask=None), dict(mask=4098), dict(mask_words=0),
                                  dict(mask_stride=-1), dict(T=40)])
def test_tree_c_call_refuses_masks(lib, over):
    over = dict(over)
    T = over.pop("T", 5)
    attn = _raw(AttnArgs, dict(T=T), HQ=4, max_seqlen_q=T - 1, max_kv_len=64, scale=0.1, causal=0, num_splits=0, lse=4096)._obj
    t = TreeArgs(ctypes.sizeof(TreeArgs), attn, 4096, 1, 1)
    for n, v in over.items():
        setattr(t, n, v)
    assert lib.streamkl_paged_tree_attn(ctypes.byref(t), None) == 1 and lib.streamkl_last_error()


@pytest.mark.gpu
def test_tree_python_call_refuses():
    c = Cache([20, 40], 2, 64, 16, torch.bfloat16)
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    mask = torch.ones(2, 1, dtype=torch.int32, device="cuda")
    call = skl.streamkl_paged_tree_attn
    for match, args, kw in [
        ("tree_mask", (q, c.k, c.v, c.table, c.lens, None), {}),
        ("tree_mask", (q, c.k, c.v, c.table, c.lens, mask[:1]), {}),
        ("tree_mask", (q, c.k, c.v, c.table, c.lens, mask.long()), {}),
        ("tree_mask", (q, c.k, c.v, c.table, c.lens, mask[:, :0]), {}),
        ("tree_mask", (q, c.k, c.v, c.table, c.lens, mask[:, 0]), {}),
        ("q must be", (q.half(), c.k, c.v, c.table, c.lens, mask), {}),
        (r"out\[0\]", (q, c.k, c.v, c.table, c.lens, mask), dict(out=(q[:1], None))),
    ]:
        with pytest.raises(ValueError, match=match):
            call(*args, **kw)
    many = torch.ones(40, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.StreamKLError, match="mask of 1 words"):
        call(many, c.k, c.v, c.table, c.lens, mask[:1].expand(40, 1), cu_seqlens=_cu([33, 7]), max_seqlen_q=33)
    o, lse = call(q[:0], c.k, c.v, c.table[:0], c.lens[:0], mask[:0], cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_masks_of_the_oracle():
    """The oracle's words and trees, on the CPU: bit t % 32 of word t / 32; a token sees its ancestors."""
    bits = orc.ancestors([-1, 0, 0, 1, 2, -1])
    assert [np.flatnonzero(r).tolist() for r in bits] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4], [5]]
    wide = np.zeros((1, 70), dtype=bool)
    wide[0, [0, 31, 32, 69]] = True
    assert orc.words_of(wide, 3).view(np.uint32).tolist() == [[0x80000001, 1, 32]]
    # a chain is the causal mask of a chunk
    q, k, v = (np.random.default_rng(0).standard_normal(s) for s in ((3, 2, 8), (1, 9, 8), (1, 9, 8)))
    a = orc.tree_attn(q, k, v, 0.3, orc.seen_keys(np.tril(np.ones((3, 3), dtype=bool)), 9))
    b = model_ops.paged_attn(q, k, v, 0.3, True)
    assert all(np.allclose(x, y, rtol=1e-12) for x, y in zip(a, b))
