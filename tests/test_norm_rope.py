"""Norm and rotation of queries and keys, forward and backward, against fp64.

Bounds, per element, from the arithmetic (u = 2^-24, one fp32 operation):
forward: the mean of squares is within 13 u (8 fma, 1 + log2(d / 16) adds, eps),
rsqrtf (2 ulp) of it within 10 u, times w and x 12 u, the turn's two products
and one sum 2 u on |a cos| + |b sin|: 16 u of that covers it. Backward: the
sum over R repeats (R - 1) u and the turn 2 u of the absolute form of g; the
mean of u x 16 u, r^2 22 u, the last products and difference 4 u: (64 + R) u of
the absolute form. Weight gradients: at most one fma for each row and 64 u
more. Then one rounding to the type, half a step: eps / 2 of the value, and
for fp16 half of the smallest subnormal, 2^-25."""
import ctypes

import numpy as np
import pytest
import torch

import attention_kl_loss_gb300 as skl
from attention_kl_loss_gb300 import binding
from oracle import model_ops as orc

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _np(t):
    return t.double().cpu().numpy()


def _tables(n, rot, dev):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return tuple(torch.from_numpy(f(ang)).float().to(dev) for f in (np.cos, np.sin))


def _round_tol(ref, dt):
    return torch.finfo(dt).eps / 2 * np.abs(ref) + 2.0 ** -25 * (dt == torch.float16)


def _inputs(B, NQ, NK, HQ, HK, d, dt, packed, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    lead_q, lead_k = ((NQ,), (NK,)) if packed else ((B, NQ), (B, NK))
    dev = torch.device("cuda")
    if NQ == NK:  # slices of one projection
        qkv = (std * torch.randn(*lead_q, HQ + 2 * HK, d, generator=g)).to(dt).to(dev)
        q, k = qkv[..., :HQ, :], qkv[..., HQ:HQ + HK, :]
    else:
        q = (std * torch.randn(*lead_q, HQ, d, generator=g)).to(dt).to(dev)
        k = (std * torch.randn(*lead_k, HK, d, generator=g)).to(dt).to(dev)
    wq, wk = (1 + 0.2 * torch.randn(2, d, generator=g)).to(dev)
    return q, k, wq, wk, g


def _check_fwd(y, x, w, pos, cos, sin, eps, inter, repeat, packed):
    c, s = (_np(t)[_np(pos).astype(np.int64)][..., None, :] for t in (cos, sin))
    ref, mag = orc.norm_rope(_np(x), None if w is None else _np(w), c, s, eps, inter)
    ref, mag = (np.repeat(t, repeat, -2) for t in (ref, mag))
    got = _np(y if packed else y.transpose(1, 2))
    assert got.shape == ref.shape
    assert np.all(np.abs(got - ref) <= _round_tol(ref, y.dtype) + 16 * U * mag)


def _check_bwd(dx, dw, x, w, dy, pos, cos, sin, eps, inter, repeat, packed):
    c, s = (_np(t)[_np(pos).astype(np.int64)][..., None, :] for t in (cos, sin))
    g = _np(dy if packed else dy.transpose(1, 2))
    g = g.reshape(*g.shape[:-2], -1, repeat, g.shape[-1])
    ref, mag, rw, rwa = orc.norm_rope_bwd(_np(x), None if w is None else _np(w), g.sum(-2), np.abs(g).sum(-2), c, s,
                                          eps, inter)
    assert np.all(np.abs(_np(dx) - ref) <= _round_tol(ref, dx.dtype) + (64 + repeat) * U * mag)
    if w is None:
        assert dw is None
        return
    rows = int(np.prod(ref.shape[:-1]))
    axes = tuple(range(rw.ndim - 1))
    assert np.all(np.abs(_np(dw) - rw.sum(axes)) <= (64 + repeat + rows) * U * rwa.sum(axes))


SHAPES = [
    # B, NQ, NK, HQ, HK, d, rot, type, norm, interleaved, repeat, packed
    (1, 1, 1, 1, 1, 64, 64, "bf16", True, False, 1, False),
    (2, 5, 5, 3, 1, 128, 128, "bf16", True, False, 3, False),
    (1, 129, 129, 8, 2, 128, 64, "fp16", True, True, 4, False),
    (3, 7, 33, 6, 6, 64, 16, "bf16", True, False, 1, False),
    (1, 1, 300, 32, 8, 128, 128, "bf16", True, False, 1, False),
    (2, 65, 65, 9, 9, 64, 48, "fp32", True, False, 1, False),
    (2, 65, 65, 4, 2, 128, 96, "fp32", False, True, 2, False),
    (1, 203, 203, 5, 5, 128, 128, "fp16", False, False, 1, True),
    (1, 1031, 1031, 17, 1, 64, 32, "bf16", True, True, 17, True),
    (1, 77, 77, 40, 8, 128, 128, "fp32", True, False, 5, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,NQ,NK,HQ,HK,d,rot,dtype,norm,inter,repeat,packed", SHAPES)
def test_forward_and_backward_match_fp64(B, NQ, NK, HQ, HK, d, rot, dtype, norm, inter, repeat, packed):
    dt, eps = TYPES[dtype], 1e-6
    q, k, wq, wk, g = _inputs(B, NQ, NK, HQ, HK, d, dt, packed, seed=NQ + d)
    wq, wk = (wq, wk) if norm else (None, None)
    dev = q.device
    cos, sin = _tables(2 * NK + 3, rot, dev)
    st = binding.new_status(dev)
    kw = dict(q_weight=wq, k_weight=wk, eps=eps, interleaved=inter, k_repeat=repeat, dev_status=st)
    if packed:  # any positions
        pq = torch.randint(0, 2 * NK + 3, (NQ,), generator=g).to(torch.int32).to(dev)
        pk = pq
        kw["positions"] = pq
    else:  # the framework's bottom-right alignment
        pq, pk = torch.arange(NQ) + NK - NQ, torch.arange(NK)
    yq, yk = skl.streamkl_qk_norm_rope_fwd(q, k, cos, sin, **kw)
    dq_out, dk_out = (torch.randn(y.shape, generator=g).to(dt).to(dev) for y in (yq, yk))
    dq, dk, dwq, dwk = skl.streamkl_qk_norm_rope_bwd(q, k, dq_out, dk_out, cos, sin, **kw)
    binding.raise_on_device_status(st)
    assert yq.is_contiguous() and yk.is_contiguous()
    _check_fwd(yq, q, wq, pq, cos, sin, eps, inter, 1, packed)
    _check_fwd(yk, k, wk, pk, cos, sin, eps, inter, repeat, packed)
    _check_bwd(dq, dwq, q, wq, dq_out, pq, cos, sin, eps, inter, 1, packed)
    _check_bwd(dk, dwk, k, wk, dk_out, pk, cos, sin, eps, inter, repeat, packed)


@pytest.mark.gpu
def test_one_side_alone_equals_both_and_is_the_same_in_every_run():
    q, k, wq, wk, g = _inputs(2, 50, 50, 8, 4, 128, torch.bfloat16, False)
    cos, sin = _tables(50, 128, q.device)
    pos = torch.stack([torch.randperm(50, generator=g) for _ in range(2)]).to(torch.int32).cuda()
    kw = dict(positions=pos)
    yq, yk = skl.streamkl_qk_norm_rope_fwd(q, k, cos, sin, q_weight=wq, k_weight=wk, **kw)
    one, none = skl.streamkl_qk_norm_rope_fwd(q, None, cos, sin, q_weight=wq, **kw)
    assert none is None and torch.equal(one, yq)
    none, one = skl.streamkl_qk_norm_rope_fwd(None, k, cos, sin, k_weight=wk, **kw)
    assert none is None and torch.equal(one, yk)
    _check_fwd(yq, q, wq, pos, cos, sin, 1e-6, False, 1, False)
    a = skl.streamkl_qk_norm_rope_bwd(q, k, yq, yk, cos, sin, q_weight=wq, k_weight=wk, **kw)
    for _ in range(2):
        b = skl.streamkl_qk_norm_rope_bwd(q, k, yq, yk, cos, sin, q_weight=wq, k_weight=wk, **kw)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    dq, none, dw, none_w = skl.streamkl_qk_norm_rope_bwd(q, None, yq, None, cos, sin, q_weight=wq, **kw)
    assert none is None and none_w is None and torch.equal(dq, a[0])
    _check_bwd(dq, dw, q, wq, yq, pos, cos, sin, 1e-6, False, 1, False)


@pytest.mark.gpu
def test_outputs_into_slices_of_one_buffer_leave_the_rest():
    q, k, wq, wk, g = _inputs(1, 37, 37, 4, 2, 64, torch.bfloat16, True)
    cos, sin = _tables(37, 64, q.device)
    pos = torch.arange(37, dtype=torch.int32, device=q.device)
    kw = dict(positions=pos, q_weight=wq, k_weight=wk)
    buf = torch.full((37, 9, 64), 7.0, dtype=q.dtype, device=q.device)
    ref = skl.streamkl_qk_norm_rope_fwd(q, k, cos, sin, **kw)
    out = skl.streamkl_qk_norm_rope_fwd(q, k, cos, sin, out=(buf[:, 1:5], buf[:, 6:8]), **kw)
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    assert torch.all(buf[:, [0, 5, 8]] == 7)
    grads = skl.streamkl_qk_norm_rope_bwd(q, k, *ref, cos, sin, **kw)
    buf.fill_(7.0)
    skl.streamkl_qk_norm_rope_bwd(q, k, *ref, cos, sin, out=(buf[:, :4], buf[:, 4:6]), **kw)
    assert torch.equal(buf[:, :4], grads[0]) and torch.equal(buf[:, 4:6], grads[1]) and torch.all(buf[:, 6:] == 7)


@pytest.mark.gpu
def test_position_outside_the_tables_is_reported_and_its_rows_left():
    q, k, wq, wk, _ = _inputs(1, 9, 9, 2, 2, 64, torch.bfloat16, True)
    cos, sin = _tables(9, 64, q.device)
    for bad in (-1, 9, 2 ** 31 - 1):
        pos = torch.arange(9, dtype=torch.int32, device=q.device)
        pos[4] = bad
        st = binding.new_status(q.device)
        out = tuple(torch.full((9, 2, 64), 5.0, dtype=q.dtype, device=q.device) for _ in range(2))
        kw = dict(positions=pos, q_weight=wq, k_weight=wk, dev_status=st)
        skl.streamkl_qk_norm_rope_fwd(q, k, cos, sin, out=out, **kw)
        with pytest.raises(binding.StreamKLError):
            binding.raise_on_device_status(st)
        keep = [i for i in range(9) if i != 4]
        for y, x, w in ((out[0], q, wq), (out[1], k, wk)):
            assert torch.all(y[4] == 5)
            _check_fwd(y[keep], x[keep], w, pos[keep], cos, sin, 1e-6, False, 1, True)
        dys = tuple(torch.ones_like(t) for t in out)
        grads = tuple(torch.full((9, 2, 64), 5.0, dtype=q.dtype, device=q.device) for _ in range(2))
        *_, dwq, _ = skl.streamkl_qk_norm_rope_bwd(q, k, *dys, cos, sin, out=grads, **kw)
        assert torch.all(grads[0][4] == 5) and torch.all(grads[1][4] == 5)
        _check_bwd(grads[0][keep], dwq, q[keep], wq, dys[0][keep], pos[keep], cos, sin, 1e-6, False, 1, True)


@pytest.mark.gpu
def test_zero_rows_infinities_and_nan_stay_in_their_rows():
    q, k, wq, wk, _ = _inputs(1, 12, 12, 2, 2, 128, torch.bfloat16, True)
    cos, sin = _tables(12, 64, q.device)
    pos = torch.arange(12, dtype=torch.int32, device=q.device)
    q[3] = 0
    q[5, 0, 7] = float("nan")
    q[6, 1, 100] = float("inf")  # beyond the rotated part
    (yq, _) = skl.streamkl_qk_norm_rope_fwd(q, k, cos, sin, positions=pos, q_weight=wq, k_weight=wk)
    assert torch.all(yq[3] == 0) and torch.all(torch.isnan(yq[5, 0])) and torch.isnan(yq[6, 1, 100])
    keep = [i for i in range(12) if i not in (5, 6)]
    _check_fwd(yq[keep], q[keep], wq, pos[keep], cos, sin, 1e-6, False, 1, True)
    (yq, _) = skl.streamkl_qk_norm_rope_fwd(q, k, cos, sin, positions=pos)  # no norm: element by element
    assert torch.isinf(yq[6, 1, 100]) and int(torch.isfinite(yq[6, 1]).sum()) == 127
    assert int(torch.isnan(yq[5, 0]).sum()) == 2


@pytest.mark.gpu
def test_gradient_equals_differences():
    """Central differences of sum(dy * y) in fp64 (step 1e-5: truncation about
    1e-10 of the third derivative, rounding about 1e-11) against the kernel's
    fp32 gradients, which are within (64 + 2) u of their absolute form."""
    q, k, wq, wk, g = _inputs(1, 2, 2, 2, 1, 64, torch.float32, False, seed=3)
    cos, sin = _tables(2, 32, q.device)
    dy = tuple(torch.randn(1, 2, 2, 64, generator=g).cuda() for _ in range(2))
    dq, dk, dwq, dwk = skl.streamkl_qk_norm_rope_bwd(q, k, *dy, cos, sin, q_weight=wq, k_weight=wk, k_repeat=2)
    c, s = (_np(t)[:, None] for t in (cos, sin))

    def loss(x, w, d, repeat):
        y, _ = orc.norm_rope(x, w, c, s, 1e-6, False)
        return (np.repeat(y, repeat, -2) * np.swapaxes(_np(d), 1, 2)).sum()

    for x, w, dx, dw, d, repeat in ((q, wq, dq, dwq, dy[0], 1), (k, wk, dk, dwk, dy[1], 2)):
        args = [_np(x), _np(w)]
        for which, grad in ((0, _np(dx)), (1, _np(dw))):
            flat = args[which].reshape(-1)
            for i in range(0, flat.size, 5):
                keep, h = flat[i], 1e-5
                flat[i] = keep + h
                hi = loss(*args, d, repeat)
                flat[i] = keep - h
                lo = loss(*args, d, repeat)
                flat[i] = keep
                assert abs((hi - lo) / (2 * h) - grad.reshape(-1)[i]) <= 5e-5


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    q, k, wq, wk, g = _inputs(1, 200, 200, 4, 2, 128, torch.bfloat16, False)
    cos, sin = _tables(200, 128, q.device)
    st = binding.new_status(q.device)
    kw = dict(q_weight=wq, k_weight=wk, k_repeat=2, dev_status=st)
    out = tuple(torch.empty(1, 4, 200, 128, dtype=q.dtype, device=q.device) for _ in range(2))
    back = (torch.empty(1, 200, 4, 128, dtype=q.dtype, device=q.device),
            torch.empty(1, 200, 2, 128, dtype=q.dtype, device=q.device))
    dws = []

    def step():
        skl.streamkl_qk_norm_rope_fwd(q, k, cos, sin, out=out, **kw)
        dws[:] = skl.streamkl_qk_norm_rope_bwd(q, k, *out, cos, sin, out=back, **kw)[2:]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    captured = list(dws)
    for seed in (1, 2):
        torch.manual_seed(seed)
        q.copy_(torch.randn_like(q))
        k.copy_(torch.randn_like(k))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, *back, *captured)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (*out, *back, *dws)))
    binding.raise_on_device_status(st)
    # everything made by the calls, while the current stream is held up
    del kw["dev_status"]
    torch.cuda._sleep(20_000_000)
    ys = skl.streamkl_qk_norm_rope_fwd(q, k, cos, sin, stream=side, **kw)
    grads = skl.streamkl_qk_norm_rope_bwd(q, k, *ys, cos, sin, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*ys, *grads), (*out, *back, *dws)))


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_the_native_way_and_the_one_in_python_do_the_same(packed, monkeypatch):
    g = torch.Generator().manual_seed(9)
    lead = (37,) if packed else (2, 37)
    qkv = torch.randn(*lead, 10, 64, generator=g).half().cuda()
    q, k = qkv[..., :6, :], qkv[..., 6:8, :]
    cos, sin = _tables(64, 32, "cuda")
    w = [torch.randn(64, generator=g).cuda() for _ in range(2)]
    pos = torch.randint(0, 64, (37,), generator=g, dtype=torch.int32).cuda()
    both = pos if packed else torch.stack([pos, pos.flip(0)])
    native, st = binding.load().native, binding.new_status()
    space = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    got = []
    for way in (native, None):
        monkeypatch.setattr(binding.load(), "native", way)
        for kw in (dict(positions=pos, dev_status=st), dict(positions=both, q_weight=w[0], k_weight=w[1], k_repeat=3),
                   dict(positions=pos, k_positions=both, interleaved=True, q_weight=w[0]),
                   dict(positions=pos, k_repeat=np.int64(2), eps=0)):
            for a, b in ((q, k), (q, None), (None, k)):
                ya, yb = skl.streamkl_qk_norm_rope_fwd(a, b, cos, sin, **kw)
                back = dict(kw, workspace=space) if kw.get("interleaved") else kw
                got += [ya, yb, *skl.streamkl_qk_norm_rope_bwd(a, b, ya, yb, cos, sin, **back)]
    binding.raise_on_device_status(st)
    half = len(got) // 2
    for a, b in zip(got[:half], got[half:]):
        assert (a is None) == (b is None)
        if a is not None:
            assert a.dtype == b.dtype and a.stride() == b.stride() and torch.equal(a, b)

    def fwd(**at):
        a = dict(dict(q=q, k=k, cos=cos, pos=pos, w=w[0], eps=1e-6, inter=False, repeat=1), **at)
        return native.rope_fwd(a["q"], a["k"], a["cos"], sin, a["pos"], None, a["w"], w[1], a["eps"], a["inter"], a["repeat"],
                               st)

    assert fwd() is not None
    for bad in (dict(q=q.cpu()), dict(q=q.float()), dict(q=q[..., :32]), dict(q=q[..., :30, :, :]), dict(q=q[None]),
                dict(k=k[..., 1:, :, :]), dict(cos=cos[1:]), dict(cos=cos.double()), dict(pos=pos.long()), dict(pos=pos[1:]),
                dict(w=w[0][1:]), dict(w=w[0].half()), dict(eps=-1.0), dict(eps=1e300), dict(inter=1), dict(repeat=0),
                dict(repeat=1 << 40), dict(q=torch.nn.Parameter(q[..., 1:]))):
        assert fwd(**bad) is None, bad


@pytest.mark.gpu
def test_training_step_from_projection_to_its_gradients():
    """Projection -> norm + rotation -> KL -> its gradients -> back: as a
    training step uses them together, grouped heads repeated for the KL,
    against fp64 autograd of the whole. Bounds: the KL's gradients are held to
    a relative norm of 1e-2 of their own (the framework's tolerance); the norm
    and rotation add two roundings to bf16 (2^-8 each) on the way in, which move
    the logits and so the gradients by about as much again, and one on the way
    back: 3e-2 in all."""
    dev = torch.device("cuda")
    B, N, HQ, HK, d = 1, 200, 4, 2, 64
    g = torch.Generator().manual_seed(0)
    teacher, student = ((torch.randn(B, N, HQ + HK, d, generator=g)).to(torch.bfloat16).to(dev) for _ in range(2))
    wq, wk = (1 + 0.1 * torch.randn(2, d, generator=g)).to(dev)
    cos, sin = _tables(N, d, dev)
    kw = dict(q_weight=wq, k_weight=wk, k_repeat=2)
    st = binding.new_status(dev)

    def heads(x):
        return skl.streamkl_qk_norm_rope_fwd(x[:, :, :HQ], x[:, :, HQ:], cos, sin, dev_status=st, **kw)

    (q1, k1), (q2, k2) = heads(teacher), heads(student)
    kl, l1, l2 = skl.streamkl_fwd(q1, k1, q2, k2, causal=True, dev_status=st)
    up = torch.full_like(kl, 1.0 / kl.numel())
    dq2, dk2, _, _ = skl.streamkl_bwd(q1, k1, q2, k2, kl, l1, l2, up, causal=True, dev_status=st)
    grad = torch.empty_like(student)
    _, _, dwq, dwk = skl.streamkl_qk_norm_rope_bwd(student[:, :, :HQ], student[:, :, HQ:], dq2, dk2, cos, sin,
                                                   out=(grad[:, :, :HQ], grad[:, :, HQ:]), dev_status=st, **kw)
    binding.raise_on_device_status(st)

    x = student.double().cpu().requires_grad_()
    ws = [w.double().cpu().requires_grad_() for w in (wq, wk)]
    c, s = (t.double().cpu()[:, None] for t in (cos, sin))

    def ref_heads(x, wq, wk):
        y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        y = torch.cat((y[:, :, :HQ] * wq, y[:, :, HQ:] * wk), 2)
        a, b = y[..., :d // 2], y[..., d // 2:]
        y = torch.cat((a * c - b * s, b * c + a * s), -1).transpose(1, 2)
        return y[:, :HQ], y[:, HQ:].repeat_interleave(2, 1)

    mask = torch.full((N, N), -float("inf"), dtype=torch.float64).triu(1)

    def logp(q, k):
        return torch.log_softmax(q @ k.transpose(2, 3) / d ** 0.5 + mask, -1)

    with torch.no_grad():
        p1 = logp(*ref_heads(teacher.double().cpu(), *(w.double().cpu() for w in (wq, wk))))
    p2 = logp(*ref_heads(x, *ws))
    live = torch.isfinite(p1)
    ref = (p1.exp() * torch.where(live, p1 - p2, 0.0)).nan_to_num(0.0).sum(-1)
    ref.mean().backward()

    def rel(a, b):
        return float((a.double().cpu() - b).norm() / b.norm())

    assert rel(kl, ref.detach()) <= 3e-2
    assert rel(grad, x.grad) <= 3e-2
    assert rel(dwq, ws[0].grad) <= 3e-2 and rel(dwk, ws[1].grad) <= 3e-2


@pytest.mark.gpu
@pytest.mark.parametrize("empty", ["tokens", "heads"])
@pytest.mark.parametrize("side", ["q", "k"])
@pytest.mark.parametrize("packed", [False, True])
def test_weight_gradient_of_an_empty_side_is_zero(side, empty, packed):
    """Queries without a token or a head beside keys that have some, and the reverse: nothing to sum on that side, the
    other side as alone. Memory that the outputs may get holds NaN."""
    q, k, wq, wk, g = _inputs(2, 40, 40, 4, 2, 64, torch.bfloat16, packed)
    x = {"q": q, "k": k}
    x[side] = x[side][..., :0, :, :] if empty == "tokens" else x[side][..., :0, :]
    cos, sin = _tables(40, 64, q.device)
    pos = {n: torch.arange(t.shape[-3], dtype=torch.int32, device=t.device) for n, t in x.items()}
    kw = dict(positions=pos["q"], k_positions=pos["k"], q_weight=wq, k_weight=wk)
    y = skl.streamkl_qk_norm_rope_fwd(x["q"], x["k"], cos, sin, **kw)
    dy = [torch.randn(t.shape, generator=g).bfloat16().cuda() for t in y]
    for given in (False, True):
        out = tuple(torch.empty_like(x[n], memory_format=torch.contiguous_format) for n in "qk") if given else None
        junk = [torch.full((64,), float("nan"), device=q.device) for _ in range(64)]
        del junk
        st = binding.new_status(q.device)
        dq, dk, dwq, dwk = skl.streamkl_qk_norm_rope_bwd(x["q"], x["k"], *dy, cos, sin, out=out, dev_status=st, **kw)
        binding.raise_on_device_status(st)
        assert dq.shape == x["q"].shape and dk.shape == x["k"].shape
        if side == "q":
            _, one, _, dw = skl.streamkl_qk_norm_rope_bwd(None, x["k"], None, dy[1], cos, sin, k_positions=pos["k"], k_weight=wk)
            assert torch.all(dwq == 0) and torch.equal(dk, one) and torch.equal(dwk, dw)
        else:
            one, _, dw, _ = skl.streamkl_qk_norm_rope_bwd(x["q"], None, dy[0], None, cos, sin, positions=pos["q"], q_weight=wq)
            assert torch.all(dwk == 0) and torch.equal(dq, one) and torch.equal(dwq, dw)


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    from attention_kl_loss_gb300 import build
    build.build()
    return binding.load()


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_longlong * 3)]


class RopeArgs(ctypes.Structure):
    """streamkl_rope_args of the header."""
    _fields_ = ([("struct_size", ctypes.c_size_t)] + [(n, Rows) for n in ("q", "k", "q_out", "k_out", "dq", "dk")]
                + [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("q_positions", ctypes.c_void_p),
                   ("q_pos_stride", ctypes.c_longlong), ("k_positions", ctypes.c_void_p),
                   ("k_pos_stride", ctypes.c_longlong)]
                + [(n, ctypes.c_void_p) for n in ("q_weight", "k_weight", "dq_weight", "dk_weight", "workspace")]
                + [("ws_bytes", ctypes.c_size_t), ("dev_status", ctypes.c_void_p)]
                + [(n, ctypes.c_int) for n in ("dtype", "B", "NQ", "NK", "HQ", "HK", "d", "rot", "table_len",
                                               "interleaved", "k_repeat")] + [("eps", ctypes.c_float)])


def _raw_args(**over):
    """Arguments that only the host looks at: a refused call never uses its addresses."""
    a = RopeArgs(ctypes.sizeof(RopeArgs), cos=4096, sin=4096, dev_status=4096, B=2, NQ=4, NK=4, HQ=2, HK=2, d=64, rot=64,
                 table_len=4, k_repeat=1, eps=1e-6)
    for n in ("q", "k", "q_out", "k_out", "dq", "dk"):
        setattr(a, n, Rows(4096, (512, 128, 64)))
    for n, v in over.items():
        rows, _, field = n.partition("__")
        if not field:
            setattr(a, n, v)
        elif field == "data":
            getattr(a, rows).data = v
        else:
            getattr(a, rows).stride[:] = v
    return a


REFUSED = [
    (dict(struct_size=8), 1), (dict(q__data=None, k__data=None), 1), (dict(dtype=3), 2), (dict(d=96), 2),
    (dict(rot=0), 2), (dict(rot=80), 2), (dict(rot=24), 2), (dict(cos=None), 1), (dict(sin=4100), 1),
    (dict(table_len=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(interleaved=2), 1), (dict(B=0), 1), (dict(NQ=0), 1), (dict(HK=0), 1), (dict(k_repeat=0), 1),
    (dict(NQ=1 << 30, NK=1 << 30, HQ=4), 2), (dict(NQ=5), 1), (dict(dev_status=None), 1), (dict(q__data=4104), 1),
    (dict(k__data=8193), 1), (dict(q_out__data=None), 1), (dict(k_out__data=4100), 1),
    (dict(q__stride=(512, 128, 60)), 1), (dict(k_out__stride=(512, -128, 64)), 1), (dict(q_weight=4100), 1),
    (dict(q_out__stride=(512, 128, 0)), 1), (dict(k_out__stride=(0, 128, 64)), 1),
    (dict(q_out__stride=(512, 64, 64)), 1), (dict(q_out__stride=(64, 256, 64)), 1),  # rows overlap
]


@pytest.mark.parametrize("over,status", REFUSED)
def test_c_call_refuses(lib, over, status):
    if "k_out__stride" in over and over["k_out__stride"][0] == 0 or over.get("q_out__stride"):
        backward = []  # there these are inputs, which may repeat rows
    else:
        backward = [lib.streamkl_qk_norm_rope_bwd]
    for call in [lib.streamkl_qk_norm_rope_fwd] + backward:
        assert call(ctypes.byref(_raw_args(**over)), None) == status
        assert lib.streamkl_last_error()


@pytest.mark.parametrize("over,status", [
    (dict(dq__data=None), 1), (dict(dk__stride=(512, 0, 64)), 1), (dict(dq__stride=(384, 128, 64)), 1), (dict(q_weight=4096), 1),
    (dict(q_weight=4096, dq_weight=4096), 1), (dict(k_weight=4096, dk_weight=4096, workspace=4100, ws_bytes=1 << 20), 1),
    (dict(k_weight=4096, dk_weight=4096, workspace=4096, ws_bytes=16), 1),
])
def test_c_backward_refuses(lib, over, status):
    assert lib.streamkl_qk_norm_rope_bwd(ctypes.byref(_raw_args(**over)), None) == status
    assert lib.streamkl_last_error()


def test_no_arguments_are_refused(lib):
    for call in (lib.streamkl_qk_norm_rope_fwd, lib.streamkl_qk_norm_rope_bwd, lib.streamkl_paged_append,
                 lib.streamkl_paged_attn):
        assert call(None, None) == 1


def test_workspace_size_on_the_host(lib):
    assert skl.streamkl_qk_norm_rope_bwd_workspace_size(1, 1, 1, 1, 1, 64) == 2 * 64 * 4
    big = skl.streamkl_qk_norm_rope_bwd_workspace_size(1, 65536, 65536, 32, 32, 128)
    assert 0 < big <= 2 * 152 * 8 * 128 * 4
    assert skl.streamkl_qk_norm_rope_bwd_workspace_size(1, 4, 4, 1, 1, 96) == 0


def test_python_call_refuses():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    cs = torch.zeros(4, 32)
    with pytest.raises(ValueError, match="both None"):
        skl.streamkl_qk_norm_rope_fwd(None, None, cs, cs)
    with pytest.raises(ValueError, match="CUDA"):
        skl.streamkl_qk_norm_rope_fwd(x, x, cs, cs)
    with pytest.raises(ValueError, match="unsupported type"):
        skl.streamkl_qk_norm_rope_fwd(x.double(), None, cs, cs)
    with pytest.raises(ValueError, match="k_repeat"):
        skl.streamkl_qk_norm_rope_fwd(x, x, cs, cs, k_repeat=0)
    with pytest.raises(ValueError, match=r"\[B, N, H, d\]"):
        skl.streamkl_qk_norm_rope_fwd(x[0, 0], None, cs, cs)


@pytest.mark.gpu
def test_python_call_refuses_on_the_device():
    q, k, wq, wk, _ = _inputs(2, 8, 8, 2, 2, 64, torch.bfloat16, False)
    cos, sin = _tables(8, 64, q.device)
    fwd = skl.streamkl_qk_norm_rope_fwd
    pos = torch.arange(8, dtype=torch.int32, device=q.device)
    for match, args, kw in [
        ("positions of q", (q, k, cos, sin), dict(positions=pos.long())),
        ("positions of q", (q, k, cos, sin), dict(positions=pos[:7])),
        ("positions of q", (q, k, cos, sin), dict(positions=pos.cpu())),
        ("q_weight", (q, k, cos, sin), dict(q_weight=wq.half())),
        ("q_weight", (q, k, cos, sin), dict(q_weight=wq[:32])),
        ("one shape", (q, k, cos, sin[:4]), {}),
        ("cos", (q, k, cos.half(), sin), {}),
        ("k must be", (q, k.half(), cos, sin), {}),
        ("batch size or head dim", (q, k[:1], cos, sin), {}),
        ("contiguous last", (q, k.transpose(2, 3), cos, sin), {}),
        ("packed batch needs", (q[0], k[0], cos, sin), {}),
        ("k_positions", (q[:, :4], k, cos, sin), dict(positions=pos[:4])),
        ("out", (q, k, cos, sin), dict(out=(q, None))),
        ("dev_status", (q, k, cos, sin), dict(dev_status=torch.zeros(1, device=q.device))),
    ]:
        with pytest.raises(ValueError, match=match):
            fwd(*args, **kw)
    with pytest.raises(binding.StreamKLError):  # more queries than keys without positions
        fwd(q, k[:, :4], cos, sin)
    with pytest.raises(ValueError, match="workspace"):
        skl.streamkl_qk_norm_rope_bwd(q, k, q.transpose(1, 2), k.transpose(1, 2), cos, sin, q_weight=wq, k_weight=wk,
                                      workspace=torch.empty(8, dtype=torch.uint8, device=q.device))
    empty = fwd(q[:, :0], k[:, :0], cos, sin)
    assert empty[0].shape == (2, 2, 0, 64)
