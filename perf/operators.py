"""Cases, inputs and plain forms of the operators around the attention-KL call.

A training step takes queries and keys from one fused projection, normalises
and rotates them per head (`norm_rope_fwd`), hands them to the KL, and takes
the KL's gradients back to the projection (`norm_rope_bwd`). The trained
student is then run over long contexts: new keys and values go into a paged
cache (`append`) and the new tokens attend to it (`attn`).

With ``own`` False `run` computes an operator from elementary torch operations
in 32 bits; with ``own`` True it makes the calls of this package. `exact`
states the same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the smallest training step (256 tokens, two heads of 64): latency of one small call
        dict(name="rope fwd tiny", op="norm_rope_fwd", packed=False, B=1, N=256, Hq=2, Hk=2, d=64, rot=64,
             dtype="bf16", norm=True, interleaved=False, repeat=1, mix=1),
        # an ordinary step with four query heads to a key head, keys repeated for the KL call
        dict(name="rope fwd mid grouped", op="norm_rope_fwd", packed=False, B=2, N=4096, Hq=16, Hk=4, d=128,
             rot=128, dtype="bf16", norm=True, interleaved=False, repeat=4, mix=2),
        # a packed long-context batch of odd length, grouped heads
        dict(name="rope fwd packed 64K", op="norm_rope_fwd", packed=True, B=5, N=65521, Hq=32, Hk=8, d=128,
             rot=128, dtype="bf16", norm=True, interleaved=False, repeat=1, mix=3),
        # the ordinary training step's way back
        dict(name="rope bwd mid", op="norm_rope_bwd", packed=False, B=2, N=4096, Hq=16, Hk=16, d=128, rot=128,
             dtype="bf16", norm=True, interleaved=False, repeat=1, mix=4),
        # the 64K-context, 32-head step's way back
        dict(name="rope bwd 64K", op="norm_rope_bwd", packed=False, B=1, N=65536, Hq=32, Hk=32, d=128, rot=128,
             dtype="bf16", norm=True, interleaved=False, repeat=1, mix=5),
        # a ragged batch with partly rotated heads of 64, interleaved pairs and repeated keys, fp16
        dict(name="rope bwd packed d64", op="norm_rope_bwd", packed=True, B=7, N=4099, Hq=8, Hk=2, d=64, rot=32,
             dtype="fp16", norm=True, interleaved=True, repeat=4, mix=6),
        # one decode step of 64 sequences: one new token each
        dict(name="append decode", op="append", B=64, n=1, L=1024, Hk=8, d=128, rot=128, page=16, dtype="bf16",
             norm=True, interleaved=False, mix=7),
        # a prefill step: ragged chunks of up to 2048 new tokens
        dict(name="append chunks", op="append", B=8, n=2048, L=4096, Hk=8, d=128, rot=64, page=64, dtype="fp16",
             norm=False, interleaved=True, mix=8),
        # one sequence, one token: latency of a single decode step
        dict(name="attn decode one", op="attn", B=1, n=1, L=4096, Hq=32, Hk=8, d=128, page=16, dtype="bf16",
             mix=9),
        # a decode batch of ragged contexts up to 16K
        dict(name="attn decode batch", op="attn", B=64, n=1, L=16384, Hq=32, Hk=8, d=128, page=16, dtype="bf16",
             mix=10),
        # a chunk of 512 new rows against a 128K context
        dict(name="attn chunk 128K", op="attn", B=1, n=512, L=131072, Hq=32, Hk=8, d=128, page=128, dtype="bf16",
             mix=11),
        # ragged chunks of up to 2048 rows, heads of 64, one key head to a query head
        dict(name="attn chunks d64", op="attn", B=4, n=2048, L=16384, Hq=8, Hk=8, d=64, page=32, dtype="fp16",
             mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}  # by operator
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        op = rng.choice(["norm_rope_fwd", "norm_rope_bwd", "append", "attn", "attn"])
        d = rng.choice([64, 128])
        mix = rng.randrange(1 << 20)
        if op in ("norm_rope_fwd", "norm_rope_bwd"):
            Hk = _log(rng, 1, 32)
            group = rng.choice([1, 2, 3, 4, 8])
            c = dict(op=op, packed=rng.random() < 0.5, B=rng.randint(1, 8), N=_log(rng, 16, 65536), Hq=Hk * group,
                     Hk=Hk, d=d, rot=rng.choice([d, d // 2]), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                     norm=rng.random() < 0.75, interleaved=rng.random() < 0.3, repeat=rng.choice([1, group]), mix=mix)
            if c["Hq"] > 64:
                continue
        else:
            Hk = _log(rng, 1, 16)
            c = dict(op=op, B=_log(rng, 1, 128), n=rng.choice([1, _log(rng, 1, 2048)]), L=_log(rng, 16, 131072), d=d,
                     Hk=Hk, page=rng.choice([16, 32, 64, 128, 256]), dtype=rng.choice(["bf16", "bf16", "fp16"]), mix=mix)
            c["n"] = min(c["n"], c["L"])
            if op == "append":
                c.update(rot=rng.choice([d, d // 2]), norm=rng.random() < 0.5, interleaved=rng.random() < 0.3)
                if c["B"] * c["L"] * Hk * d > 2 ** 30:
                    continue
            else:
                c["Hq"] = Hk * rng.choice([1, 2, 3, 4, 8])
                # the padded scores of the plain form, and the pages
                if c["B"] * c["n"] * c["L"] * c["Hq"] > 2 ** 31 or c["B"] * c["L"] * Hk * d > 2 ** 30 or c["Hq"] > 64:
                    continue
        if _cost(c) <= most[op]:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _lengths(c):
    """(new tokens, length afterwards) of each sequence: the longest ones as the case says, the others ragged."""
    r = random.Random(c["mix"])
    new, total = [], []
    for b in range(c["B"]):
        n = c["n"] if b == 0 else r.randint(max(1, c["n"] // 4), c["n"])
        t = c["L"] if b == 0 else r.randint(max(n, c["L"] // 4), max(n, c["L"]))
        new.append(n)
        total.append(t)
    return new, total


def _packed_positions(c):
    """Positions of a packed batch: B sequences of ragged lengths, N tokens in all, each counting from 0."""
    r = random.Random(c["mix"])
    cuts = sorted(r.randint(0, c["N"]) for _ in range(c["B"] - 1))
    ends = [0] + cuts + [c["N"]]
    return torch.cat([torch.arange(b - a) for a, b in zip(ends, ends[1:])])


def work(c):
    size = 4 if c["dtype"] == "fp32" else 2
    if c["op"] in ("norm_rope_fwd", "norm_rope_bwd"):
        tokens = c["N"] * (1 if c["packed"] else c["B"])
        q, k = tokens * c["Hq"] * c["d"], tokens * c["Hk"] * c["d"]
        outer = q + k * c["repeat"]  # what the KL call takes and gives back
        elems = (q + k) + outer if c["op"] == "norm_rope_fwd" else 2 * (q + k) + outer
        return {"bytes": elems * size + c["N"] * c["rot"] * 4, "flops": 10 * (q + k)}
    new, total = _lengths(c)
    if c["op"] == "append":
        return {"bytes": sum(new) * (4 * c["Hk"] * c["d"] * size + c["rot"] * 4), "flops": 8 * sum(new) * c["Hk"] * c["d"]}
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, total))
    rows = sum(new) * c["Hq"]
    return {"bytes": 2 * sum(total) * c["Hk"] * c["d"] * size + 2 * rows * c["d"] * size + 4 * rows,
            "flops": 4 * c["d"] * c["Hq"] * pairs}


# ---------------------------------------------------------------- inputs
def _tables(length, rot, device):
    """cos, sin of position x frequency (base 10000), angles in 64 bits, kept in 32."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(length, dtype=torch.float64, device=device)[:, None] * freq
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    s = {"case": c}
    if c["op"] in ("norm_rope_fwd", "norm_rope_bwd"):
        lead = (c["N"],) if c["packed"] else (c["B"], c["N"])
        H = c["Hq"] + 2 * c["Hk"]  # one projection: queries, keys, values
        qkv = randn(*lead, H * c["d"]).view(*lead, H, c["d"])
        s["q"], s["k"] = qkv[..., :c["Hq"], :], qkv[..., c["Hq"]:c["Hq"] + c["Hk"], :]
        s["positions"] = (_packed_positions(c) if c["packed"] else torch.arange(c["N"])).to(torch.int32).to(dev)
        s["cos"], s["sin"] = _tables(c["N"], c["rot"], dev)
        for w in ("q_weight", "k_weight"):
            s[w] = 1 + 0.1 * torch.randn(c["d"], generator=gen, device=dev) if c["norm"] else None
        if c["op"] == "norm_rope_bwd":
            Hk = c["Hk"] * c["repeat"]
            if c["packed"]:
                s["dq"], s["dk"] = randn(c["N"], c["Hq"], c["d"]), randn(c["N"], Hk, c["d"])
            else:
                s["dq"], s["dk"] = randn(c["B"], c["Hq"], c["N"], c["d"]), randn(c["B"], Hk, c["N"], c["d"])
    else:
        new, total = _lengths(c)
        width = -(-max(total) // c["page"])
        pages = sum(-(-t // c["page"]) for t in total) + 3
        shape = (pages, c["Hk"], c["page"], c["d"])
        s["k_cache"], s["v_cache"] = randn(*shape), randn(*shape)
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        table = torch.zeros(c["B"], width, dtype=torch.int32, device=dev)
        at = 0
        for b, t in enumerate(total):
            p = -(-t // c["page"])
            table[b, :p] = order[at:at + p]
            at += p
        s["block_table"] = table
        s["kv_lens"] = torch.tensor(total, dtype=torch.int32, device=dev)
        s["cu_seqlens"] = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
        s["max_new"], s["max_len"], s["tokens"] = max(new), max(total), sum(new)
        if c["op"] == "append":
            kv = randn(sum(new), 2 * c["Hk"], c["d"])
            s["k"], s["v"] = kv[:, :c["Hk"]], kv[:, c["Hk"]:]
            s["cos"], s["sin"] = _tables(max(total), c["rot"], dev)
            s["k_weight"] = 1 + 0.1 * torch.randn(c["d"], generator=gen, device=dev) if c["norm"] else None
        else:
            s["q"] = randn(sum(new), c["Hq"], c["d"])
            s["scale"] = 1 / math.sqrt(c["d"])
    return s


# ---------------------------------------------------------------- run
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_rope(s):
    from attention_kl_loss_gb300 import new_status, streamkl_qk_norm_rope_fwd

    if "status" not in s:  # kept by the caller from step to step
        s["status"] = new_status()
    c = s["case"]
    return streamkl_qk_norm_rope_fwd(s["q"], s["k"], s["cos"], s["sin"], positions=s["positions"],
                                     q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                     interleaved=c["interleaved"], k_repeat=c["repeat"], dev_status=s["status"])


def _own_rope_bwd(s):
    from attention_kl_loss_gb300 import new_status, streamkl_qk_norm_rope_bwd

    if "status" not in s:
        s["status"] = new_status()
    c = s["case"]
    return streamkl_qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["cos"], s["sin"], positions=s["positions"],
                                     q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                     interleaved=c["interleaved"], k_repeat=c["repeat"], dev_status=s["status"])


def _own_append(s):
    from attention_kl_loss_gb300 import new_status, streamkl_paged_append

    if "status" not in s:
        s["status"] = new_status()
    c = s["case"]
    return streamkl_paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                                 cu_seqlens=s["cu_seqlens"], cos=s["cos"], sin=s["sin"], k_weight=s["k_weight"],
                                 eps=EPS, interleaved=c["interleaved"], dev_status=s["status"])


def _own_attn(s):
    from attention_kl_loss_gb300 import new_status, streamkl_paged_attn, streamkl_paged_attn_workspace_size

    c = s["case"]
    if "status" not in s:
        s["status"] = new_status()
        need = streamkl_paged_attn_workspace_size(c["B"], s["tokens"], c["Hq"], c["Hk"], c["d"], s["max_new"],
                                                  s["max_len"])
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return streamkl_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                               cu_seqlens=s["cu_seqlens"], max_seqlen_q=s["max_new"], max_kv_len=s["max_len"],
                               scale=s["scale"], workspace=s["workspace"], dev_status=s["status"])


_own = {"norm_rope_fwd": _own_rope, "norm_rope_bwd": _own_rope_bwd, "append": _own_append, "attn": _own_attn}


# ---------------------------------------------------------------- plain forms
def _turn(x, cos, sin, rot, interleaved, back=False):
    """Rotate the first `rot` components; cos, sin broadcast against x[..., :rot / 2]."""
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    sin = -sin if back else sin
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((r, rest), -1)


def _plain_side(x, w, s, heads):
    """Norm and rotation of x [..., N, H, d], in 32 bits; heads repeated, moved before the tokens unless packed."""
    c = s["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    cos, sin = (s[t][s["positions"].long()][:, None] for t in ("cos", "sin"))
    y = _turn(x, cos, sin, c["rot"], c["interleaved"]).repeat_interleave(heads, -2)
    return (y if c["packed"] else y.transpose(1, 2)).to(DTYPES[c["dtype"]]).contiguous()


def _plain_rope(s):
    return (_plain_side(s["q"], s["q_weight"], s, 1), _plain_side(s["k"], s["k_weight"], s, s["case"]["repeat"]))


def _plain_side_bwd(x, w, dy, s, heads):
    c = s["case"]
    x, g = x.float(), dy.float()
    if not c["packed"]:
        g = g.transpose(1, 2)
    g = g.unflatten(-2, (-1, heads)).sum(-2)
    cos, sin = (s[t][s["positions"].long()][:, None] for t in ("cos", "sin"))
    g = _turn(g, cos, sin, c["rot"], c["interleaved"], back=True)
    if w is None:
        return g.to(dy.dtype).contiguous(), None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    dw = (g * x * r).flatten(0, -2).sum(0)
    u = g * w
    dx = r * (u - x * r.square() * (u * x).mean(-1, keepdim=True))
    return dx.to(dy.dtype), dw


def _plain_rope_bwd(s):
    dq, dwq = _plain_side_bwd(s["q"], s["q_weight"], s["dq"], s, 1)
    dk, dwk = _plain_side_bwd(s["k"], s["k_weight"], s["dk"], s, s["case"]["repeat"])
    return dq, dk, dwq, dwk


def _places(s):
    """Sequence and position of every new token."""
    cu = s["cu_seqlens"].long()
    token = torch.arange(s["tokens"], device=cu.device)
    seq = torch.searchsorted(cu, token, right=True) - 1
    return seq, s["kv_lens"].long()[seq] - cu[seq + 1] + token


def _plain_append(s):
    c = s["case"]
    seq, pos = _places(s)
    k = s["k"].float()
    if s["k_weight"] is not None:
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["k_weight"]
    k = _turn(k, s["cos"][pos][:, None], s["sin"][pos][:, None], c["rot"], c["interleaved"])
    page, slot = s["block_table"].long()[seq, pos // c["page"]], pos % c["page"]
    s["k_cache"][page, :, slot] = k.to(s["k_cache"].dtype)
    s["v_cache"][page, :, slot] = s["v"]
    return s["k_cache"], s["v_cache"]


def _plain_attn(s):
    c = s["case"]
    dev = s["q"].device
    B, n, group = c["B"], s["max_new"], c["Hq"] // c["Hk"]
    table, lens = s["block_table"].long(), s["kv_lens"].long()
    k, v = (t[table].permute(0, 2, 1, 3, 4).flatten(2, 3).float() for t in (s["k_cache"], s["v_cache"]))
    seq, pos = _places(s)
    cu = s["cu_seqlens"].long()
    row = torch.arange(s["tokens"], device=dev) - cu[seq]
    q = torch.zeros(B, n, c["Hk"], group, c["d"], device=dev)
    q[seq, row] = s["q"].float().unflatten(1, (c["Hk"], group))
    first = lens - (cu[1:] - cu[:-1])  # tokens before the new ones
    keys = torch.arange(k.shape[2], device=dev)
    seen = keys < torch.minimum(first[:, None] + 1 + torch.arange(n, device=dev), lens[:, None])[..., None]
    v = torch.where((keys < lens[:, None])[:, None, :, None], v, 0)  # what lies past the end of a sequence
    # rows (head of the group, token) of one key head; scores [B, Hk, group, n, keys]
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).flatten(2, 3), k.transpose(2, 3)).unflatten(2, (group, n)).mul_(s["scale"])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), v).unflatten(2, (group, n)) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log())[..., 0]
    o, lse = o.permute(0, 3, 1, 2, 4)[seq, row], lse.permute(0, 3, 1, 2)[seq, row]
    return o.flatten(1, 2).to(s["q"].dtype), lse.flatten(1, 2)


_plain = {"norm_rope_fwd": _plain_rope, "norm_rope_bwd": _plain_rope_bwd, "append": _plain_append,
          "attn": _plain_attn}


# ---------------------------------------------------------------- 64 bits
def _spin(x, cos, sin, rot, interleaved):
    """The rotation as a product of complex numbers, in 64 bits."""
    z = torch.complex(cos.double(), sin.double())
    out = x.double().clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y = torch.complex(out[..., first], out[..., second]) * z
    out[..., first], out[..., second] = y.real, y.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope_fwd": _exact_rope, "norm_rope_bwd": _exact_rope_bwd, "append": _exact_append,
            "attn": _exact_attn}[case["op"]](s)


def _unit(x, w):
    x = x.double()
    return x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()


def _exact_rope(s):
    c = s["case"]
    cos, sin = s["cos"][s["positions"].long()].unsqueeze(1), s["sin"][s["positions"].long()].unsqueeze(1)
    outs = []
    for x, w, heads in ((s["q"], s["q_weight"], 1), (s["k"], s["k_weight"], c["repeat"])):
        y = _spin(_unit(x, w), cos, sin, c["rot"], c["interleaved"])
        y = torch.stack([y] * heads, -2).flatten(-3, -2)
        outs.append(y if c["packed"] else y.movedim(-2, 1).contiguous())
    return tuple(outs)


def _exact_rope_bwd(s):
    """The derivative of sum(dy * y) as the vector-Jacobian product of the norm, row by row."""
    c = s["case"]
    cos, sin = s["cos"][s["positions"].long()].unsqueeze(1), s["sin"][s["positions"].long()].unsqueeze(1)
    grads, weights = [], []
    for x, w, dy, heads in ((s["q"], s["q_weight"], s["dq"], 1), (s["k"], s["k_weight"], s["dk"], c["repeat"])):
        g = dy.double() if c["packed"] else dy.double().movedim(1, -2)
        g = sum(g[..., j::heads, :] for j in range(heads))
        g = _spin(g, cos, -sin, c["rot"], c["interleaved"])  # the inverse rotation
        if w is None:
            grads.append(g)
            weights.append(None)
            continue
        x = x.double()
        size = (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
        e = x / size
        weights.append((g * e).sum(tuple(range(g.dim() - 1))))
        g = g * w.double()
        grads.append((g - e * (g * e).sum(-1, keepdim=True) / c["d"]) / size)
        del g, e, size, x
    return (*grads, *weights)


def _exact_append(s):
    c = s["case"]
    cu, lens, table = s["cu_seqlens"].tolist(), s["kv_lens"].tolist(), s["block_table"].tolist()
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    for b in range(c["B"]):
        a, e = cu[b], cu[b + 1]
        pos = torch.arange(lens[b] - (e - a), lens[b], device=s["k"].device)
        k = _spin(_unit(s["k"][a:e], s["k_weight"]), s["cos"][pos].unsqueeze(1), s["sin"][pos].unsqueeze(1), c["rot"],
                  c["interleaved"])
        pages = torch.tensor(table[b], device=pos.device)[pos // c["page"]]
        for cache, new in zip(caches, (k, s["v"][a:e].double())):
            cache[pages, :, pos % c["page"]] = new
    return tuple(caches)


def _exact_attn(s):
    c = s["case"]
    if work(c)["flops"] > 1.5e13:  # at about 1 TFLOP/s in 64 bits
        return None
    cu, lens, group = s["cu_seqlens"].tolist(), s["kv_lens"].tolist(), c["Hq"] // c["Hk"]
    o = torch.zeros(s["tokens"], c["Hq"], c["d"], dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["tokens"], c["Hq"], dtype=torch.float64, device=s["q"].device)
    for b in range(c["B"]):
        a, e, length = cu[b], cu[b + 1], lens[b]
        pages = s["block_table"][b, :-(-length // c["page"])].long()
        ks, vs = (t[pages].movedim(1, 0).flatten(1, 2)[:, :length].double() for t in (s["k_cache"], s["v_cache"]))
        bias = torch.full((e - a, length), -math.inf, dtype=torch.float64, device=o.device).triu(length - (e - a) + 1)
        for h in range(c["Hq"]):
            x = s["q"][a:e, h].double() @ ks[h // group].T * s["scale"] + bias
            z = torch.logsumexp(x, -1, keepdim=True)
            o[a:e, h] = (x - z).exp() @ vs[h // group]
            lse[a:e, h] = z[:, 0]
    return o, lse
