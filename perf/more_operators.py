"""Cases, inputs and plain forms of speculative decoding over the paged cache.

A serving step that verifies a tree of drafted tokens gives every sequence the
pages that they take (`resize`), copies the last pages that other sequences
hold too (`copy`), lets the drafted tokens attend to the cache and to their own
branch (`tree`), moves the accepted ones to the front (`compact`) and gives the
other pages back (`resize` again). Beams and shared prompts are sequences that
hold the same pages (`fork`).

With `own` False `run` computes an operator from elementary torch operations
(in 32 bits, whole numbers in 64); with `own` True it makes the calls of this
package. `exact` states the same from the definitions, sequence by sequence.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one sequence, a small tree: latency of a single user's step
        dict(name="tree one", op="tree", B=1, n=8, L=2048, Hq=32, Hk=8, d=128, page=16, dtype="bf16", mix=1),
        # a serving batch of ragged contexts up to 16K, trees of up to 16 tokens
        dict(name="tree batch", op="tree", B=64, n=16, L=16384, Hq=32, Hk=8, d=128, page=16, dtype="bf16", mix=2),
        # ragged trees of up to 61 tokens, heads of 64, one key head to a query head
        dict(name="tree d64", op="tree", B=24, n=61, L=5000, Hq=8, Hk=8, d=64, page=32, dtype="fp16", mix=3),
        # few sequences, wide trees
        dict(name="tree wide", op="tree", B=4, n=256, L=16384, Hq=32, Hk=8, d=128, page=128, dtype="bf16", mix=4),
        # the accepted tokens of a serving batch
        dict(name="compact step", op="compact", B=64, n=32, kept=6, L=1024, Hk=8, d=128, page=16, dtype="bf16", mix=5),
        # whole sequences of which about half of the tokens stay in the cache
        dict(name="compact prune", op="compact", B=8, n=8192, kept=4100, L=8192, Hk=8, d=128, page=64, dtype="fp16",
             mix=6),
        # last pages of a few beams
        dict(name="copy step", op="copy", pairs=64, share=0.25, Hk=8, d=128, page=16, dtype="bf16", mix=7),
        # prompts copied whole, large pages
        dict(name="copy many", op="copy", pairs=1000, share=1.0, Hk=8, d=128, page=128, dtype="bf16", mix=8),
        # four beams each of 16 requests
        dict(name="fork beams", op="fork", B=64, beams=4, L=4096, page=16, mix=9),
        # many sequences of long contexts
        dict(name="fork long", op="fork", B=512, beams=8, L=65536, page=16, mix=10),
        # a serving step: a few tokens more, a few less
        dict(name="resize step", op="resize", B=64, L=2048, step=48, page=16, spare=300, full=False, mix=11),
        # a scheduler's turn: long sequences end, others come, over two million pages
        dict(name="resize long", op="resize", B=500, L=131072, step=131072, page=16, spare=5000, full=False,
             mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}  # by operator
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        op = rng.choice(["tree", "tree", "tree", "compact", "copy", "fork", "resize"])
        c = dict(op=op, page=rng.choice([16, 32, 64, 128, 256]), mix=rng.randrange(1 << 20))
        if op in ("tree", "compact", "copy"):
            c.update(Hk=_log(rng, 1, 16), d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "fp16"]))
        if op == "tree":
            c.update(B=_log(rng, 1, 100), n=_log(rng, 1, 400), L=_log(rng, 16, 100000))
            c.update(n=min(c["n"], c["L"]), Hq=c["Hk"] * rng.choice([1, 2, 3, 4, 8]))
            # the padded scores of the plain form, and the pages
            if c["B"] * c["n"] * c["L"] * c["Hq"] > 2 ** 30 or c["B"] * c["L"] * c["Hk"] * c["d"] > 2 ** 30:
                continue
            if c["Hq"] > 64:
                continue
        elif op == "compact":
            c.update(B=_log(rng, 1, 256), n=_log(rng, 2, 8192))
            c.update(kept=_log(rng, 1, c["n"]), L=c["n"] + _log(rng, 1, 2000))
            if c["B"] * c["L"] * c["Hk"] * c["d"] > 2 ** 28:
                continue
        elif op == "copy":
            c.update(pairs=_log(rng, 1, 4000), share=rng.choice([0.2, 0.6, 1.0]))
        elif op == "fork":
            c.update(B=_log(rng, 2, 512), beams=rng.choice([2, 3, 4, 8, 16]), L=_log(rng, 16, 65536))
        else:
            c.update(B=_log(rng, 1, 500), L=_log(rng, 64, 131072), spare=_log(rng, 2, 5000))
            c.update(step=_log(rng, 1, c["L"]), full=rng.random() < 0.25)  # full: too few pages for some
        if _cost(c) <= most[op]:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _lengths(c):
    """(drafted tokens, length with them) of each sequence: the longest ones as the case says, the others ragged."""
    r = random.Random(c["mix"])
    new, total = [], []
    for b in range(c["B"]):
        n = c["n"] if b == 0 else r.randint(max(1, c["n"] // 4), c["n"])
        t = c["L"] if b == 0 else r.randint(max(n, c["L"] // 4), max(n, c["L"]))
        new.append(n)
        total.append(t)
    return new, total


def _parents(c):
    """A tree a sequence: token i's parent among the eight before it, or none."""
    r = random.Random(c["mix"] + 1)
    return [[-1 if i == 0 or r.random() < 0.05 else r.randint(max(0, i - 8), i - 1) for i in range(n)]
            for n in _lengths(c)[0]]


def _kept(c):
    """The drafted tokens that stay, rising, of each sequence; at most c["kept"]."""
    r = random.Random(c["mix"] + 2)
    lists = []
    for b, n in enumerate(_lengths(c)[0]):
        k = min(n, c["kept"]) if b == 0 else r.randint(0, min(n, c["kept"]))
        lists.append(sorted(r.sample(range(n), k)))
    return lists


def _seated(c):
    """Lengths before and after a step of `resize`; sequences that share a prompt (fork of the one before)."""
    r = random.Random(c["mix"])
    before, after, shared = [], [], []
    for b in range(c["B"]):
        shared.append(b > 0 and r.random() < 0.3)  # as long as the one before, its pages
        before.append(before[-1] if shared[-1] else r.randint(0, c["L"]))
        after.append(max(0, min(c["L"], before[-1] + r.randint(-c["step"], c["step"]))))
    return before, after, shared


def _sources(c):
    """Each beam goes on from one of its request's."""
    r = random.Random(c["mix"] + 3)
    return [min(c["B"] - 1, b - b % c["beams"] + r.randrange(c["beams"])) for b in range(c["B"])]


def _held(c):
    r = random.Random(c["mix"])
    return [r.randint(c["L"] // 2, c["L"]) for _ in range(c["B"])]


def work(c):
    if c["op"] == "tree":
        new, total = _lengths(c)
        pairs = sum(n * (t - n) for n, t in zip(new, total))
        for parents in _parents(c):
            depth = []
            for p in parents:
                depth.append(1 if p < 0 else depth[p] + 1)
            pairs += sum(depth)
        rows = sum(new) * c["Hq"]
        masks = sum(new) * 4 * -(-c["n"] // 32)
        return {"bytes": 4 * sum(total) * c["Hk"] * c["d"] + 4 * rows * c["d"] + 4 * rows + masks,
                "flops": 4 * c["d"] * c["Hq"] * pairs}
    if c["op"] == "compact":
        moved = sum(i != k for kept in _kept(c) for i, k in enumerate(kept))
        return {"bytes": moved * (8 * c["Hk"] * c["d"] + 4) + 12 * c["B"], "flops": 0}
    if c["op"] == "copy":
        pages = max(1, int(c["pairs"] * c["share"]))
        return {"bytes": pages * 8 * c["Hk"] * c["page"] * c["d"] + 8 * c["pairs"], "flops": 0}
    if c["op"] == "fork":
        held, source = _held(c), _sources(c)
        entries = [-(-t // c["page"]) for t in held]
        children = [0] * c["B"]
        for s in source:
            children[s] += 1
        # entries read and written by the sequences that change, counts of pages whose holders do
        return {"bytes": sum(8 * entries[s] for b, s in enumerate(source) if s != b)
                + sum(8 * e for e, k in zip(entries, children) if k != 1) + 12 * c["B"], "flops": 0}
    before, after, _ = _seated(c)
    pages = [(-(-a // c["page"]), -(-z // c["page"])) for a, z in zip(before, after)]
    # entries and counts of the pages given out and given back
    return {"bytes": sum(12 * abs(a - z) for a, z in pages) + 16 * c["B"], "flops": 0}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    s = {"case": c}

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def caches(pages):
        shape = (pages, c["Hk"], c["page"], c["d"])
        for t in ("k_cache", "v_cache"):
            s[t] = torch.randn(shape, generator=gen, device=dev, dtype=DTYPES[c["dtype"]])

    if c["op"] in ("tree", "compact"):
        new, total = _lengths(c)
        width = -(-max(total) // c["page"])
        pages = sum(-(-t // c["page"]) for t in total) + 3
        caches(pages)
        s["block_table"] = _deal(c, total, width, torch.randperm(pages, generator=gen, device=dev).to(torch.int32))
        s["kv_lens"] = ints(total)
        s["cu_seqlens"] = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
        s["max_new"], s["max_len"], s["tokens"] = max(new), max(total), sum(new)
        if c["op"] == "tree":
            s["tree_mask"] = torch.from_numpy(_masks(c)).to(dev)
            s["q"] = torch.randn(sum(new), c["Hq"], c["d"], generator=gen, device=dev, dtype=DTYPES[c["dtype"]])
            s["scale"] = 1 / math.sqrt(c["d"])
        else:
            lists = _kept(c)
            s["num_kept"] = ints([len(k) for k in lists])
            s["kept"] = ints([k + [0] * (c["kept"] - len(k)) for k in lists])
    elif c["op"] == "copy":
        pages = 2 * c["pairs"] + 3
        caches(pages)
        pairs = torch.randperm(pages, generator=gen, device=dev)[:2 * c["pairs"]].view(-1, 2).to(torch.int32)
        order = torch.randperm(c["pairs"], generator=gen, device=dev)
        pairs[order[max(1, int(c["pairs"] * c["share"])):]] = -1  # sequences that have nothing to copy
        s["pairs"] = pairs
    elif c["op"] == "fork":
        held = _held(c)
        pages = sum(-(-t // c["page"]) for t in held) + 100
        width = -(-c["L"] // c["page"])
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        s["block_table"] = _deal(c, held, width, order)
        s["kv_lens"], s["source"] = ints(held), ints(_sources(c))
        s["page_refs"] = torch.zeros(pages + 1, dtype=torch.int32, device=dev)
        s["page_refs"][s["block_table"].long().flatten()] = 1  # (-1: the last one)
        s["page_refs"] = s["page_refs"][:pages].contiguous()
    else:
        before, after, shared = _seated(c)
        width = -(-c["L"] // c["page"])
        count = [-(-a // c["page"]) for a in before]
        grow = sum(max(0, -(-z // c["page"]) - n) for z, n in zip(after, count)) + c["B"]
        pages = sum(count) + (c["spare"] if c["full"] else grow + c["spare"])
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        table = _deal(c, before, width, order)
        for b in range(1, c["B"]):
            if shared[b]:
                table[b] = table[b - 1]
        s["block_table"] = table
        refs = torch.zeros(pages + 1, dtype=torch.int32, device=dev)
        at = torch.where(table < 0, pages, table).long().flatten()
        refs.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
        s["page_refs"] = refs[:pages].contiguous()
        s["kv_lens"] = ints(before)
        s["lengths"], s["turn"] = [ints(after), ints(before)], 0  # a step there, the next one back
    return s


def _deal(c, lengths, width, order):
    """Tables whose pages come in the given order; -1 where there is none."""
    table = torch.full((c["B"], width), -1, dtype=torch.int32, device=order.device)
    at = 0
    for b, t in enumerate(lengths):
        p = -(-t // c["page"])
        table[b, :p] = order[at:at + p]
        at += p
    return table


def _masks(c):
    """A drafted token sees its ancestors and itself: bit t % 32 of word t / 32."""
    words = -(-c["n"] // 32)
    rows = []
    for parents in _parents(c):
        seen = np.zeros((len(parents), words), dtype=np.uint32)
        for i, p in enumerate(parents):
            if p >= 0:
                seen[i] = seen[p]
            seen[i, i // 32] |= np.uint32(1 << (i % 32))
        rows.append(seen)
    return np.concatenate(rows).view(np.int32)


# ---------------------------------------------------------------- run
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _status(s):
    from attention_kl_loss_gb300 import new_status

    if "status" not in s:  # kept by the caller from step to step
        s["status"] = new_status()
    return s["status"]


def _own_tree(s):
    from attention_kl_loss_gb300 import streamkl_paged_tree_attn, streamkl_paged_tree_attn_workspace_size

    c = s["case"]
    if "workspace" not in s:
        need = streamkl_paged_tree_attn_workspace_size(c["B"], s["tokens"], c["Hq"], c["Hk"], c["d"], s["max_new"],
                                                       s["max_len"])
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return streamkl_paged_tree_attn(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], s["tree_mask"],
                                    cu_seqlens=s["cu_seqlens"], max_seqlen_q=s["max_new"], max_kv_len=s["max_len"],
                                    scale=s["scale"], workspace=s["workspace"], dev_status=_status(s))


def _own_compact(s):
    from attention_kl_loss_gb300 import streamkl_paged_compact

    return streamkl_paged_compact(s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], s["cu_seqlens"], s["kept"],
                                  s["num_kept"], dev_status=_status(s))


def _own_copy(s):
    from attention_kl_loss_gb300 import streamkl_paged_copy

    return streamkl_paged_copy(s["k_cache"], s["v_cache"], s["pairs"], dev_status=_status(s))


def _own_fork(s):
    from attention_kl_loss_gb300 import streamkl_paged_fork

    return streamkl_paged_fork(s["page_refs"], s["block_table"], s["kv_lens"], s["source"], dev_status=_status(s))


def _own_resize(s):
    from attention_kl_loss_gb300 import streamkl_paged_resize

    new_lens, s["turn"] = s["lengths"][s["turn"]], 1 - s["turn"]
    copies = streamkl_paged_resize(s["page_refs"], s["block_table"], s["kv_lens"], new_lens, s["case"]["page"],
                                   dev_status=_status(s))
    return s["page_refs"], s["block_table"], s["kv_lens"], copies


_own = {"tree": _own_tree, "compact": _own_compact, "copy": _own_copy, "fork": _own_fork, "resize": _own_resize}


# ---------------------------------------------------------------- plain forms
def _plain_tree(s):
    c = s["case"]
    dev = s["q"].device
    B, n, group = c["B"], s["max_new"], c["Hq"] // c["Hk"]
    table, lens, cu = s["block_table"].clamp(min=0).long(), s["kv_lens"].long(), s["cu_seqlens"].long()
    k, v = (t[table].permute(0, 2, 1, 3, 4).flatten(2, 3).float() for t in (s["k_cache"], s["v_cache"]))
    token = torch.arange(s["tokens"], device=dev)
    seq = torch.searchsorted(cu, token, right=True) - 1
    row = token - cu[seq]
    q = torch.zeros(B, n, c["Hk"], group, c["d"], device=dev)
    q[seq, row] = s["q"].float().unflatten(1, (c["Hk"], group))
    # the masks' bits [B, n, drafted token], and which of them key j is
    bits = torch.zeros(B, n, 32 * s["tree_mask"].shape[1], dtype=torch.bool, device=dev)
    bits[seq, row] = (s["tree_mask"][:, :, None] >> torch.arange(32, device=dev, dtype=torch.int32) & 1).flatten(1).bool()
    keys = torch.arange(k.shape[2], device=dev)
    drafted = keys - (lens - (cu[1:] - cu[:-1]))[:, None]
    seen = bits.gather(2, drafted.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, n, -1)) | (drafted < 0)[:, None]
    there = keys < lens[:, None]
    seen &= there[:, None]
    v = torch.where(there[:, None, :, None], v, 0)  # what lies past the end of a sequence
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


def _plain_compact(s):
    page, table = s["case"]["page"], s["block_table"].long()
    cu = s["cu_seqlens"].long()
    first = (s["kv_lens"].long() - (cu[1:] - cu[:-1]))[:, None]
    place = torch.arange(s["kept"].shape[1], device=table.device)[None]
    there = place < s["num_kept"][:, None]
    to = first + place
    source = torch.where(there, first + s["kept"].long(), to)
    to, source = (torch.minimum(p, s["kv_lens"].long()[:, None] - 1) for p in (to, source))
    # (what does not move is written where it was: the last position may be written more than once, with itself)
    end = to >= first + s["num_kept"][:, None]
    source = torch.where(end, to, source)
    rows = torch.arange(table.shape[0], device=table.device)[:, None]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[table[rows, to // page], :, to % page] = cache[table[rows, source // page], :, source % page]
    return s["k_cache"], s["v_cache"]


def _plain_copy(s):
    pairs = s["pairs"].long()
    # pairs that copy nothing copy the first one's page once more
    first = torch.argmax((pairs[:, 0] >= 0).to(torch.int32))
    pairs = torch.where(pairs[:, :1] >= 0, pairs, pairs[first])
    for cache in (s["k_cache"], s["v_cache"]):
        cache[pairs[:, 1]] = cache[pairs[:, 0]]
    return s["k_cache"], s["v_cache"]


def _plain_fork(s):
    table, refs, source = s["block_table"], s["page_refs"], s["source"].long()
    children = torch.zeros_like(s["kv_lens"]).index_add_(0, source, torch.ones_like(s["kv_lens"]))
    more = torch.where(table < 0, 0, (children - 1)[:, None])
    refs.index_add_(0, table.clamp(min=0).long().flatten(), more.flatten())
    table.copy_(table[source])
    s["kv_lens"].copy_(s["kv_lens"][source])
    return refs, table, s["kv_lens"]


def _plain_resize(s):
    page, table, refs = s["case"]["page"], s["block_table"], s["page_refs"]
    new, s["turn"] = s["lengths"][s["turn"]].long(), 1 - s["turn"]
    old = s["kv_lens"].long()
    have, need = ((t + page - 1) // page for t in (old, new))
    place = torch.arange(table.shape[1], device=table.device)
    # given back
    back = (place >= need[:, None]) & (place < have[:, None])
    refs.index_add_(0, table.clamp(min=0).long().flatten(), -back.flatten().to(torch.int32))
    table.masked_fill_(back, -1)
    # a last page that others hold is replaced, unless all others before it have left it
    grows = (new > old) & (old % page != 0)
    at = (old // page).clamp(max=table.shape[1] - 1)[:, None]
    last = table.long().gather(1, at)[:, 0].clamp(min=0)
    same = (last[:, None] == last) & grows[:, None] & grows
    held = refs[last].long()
    copy = grows & (held - same.tril(-1).sum(1) > 1)
    want = (need - have).clamp(min=0) + copy
    ends = want.cumsum(0)
    free = refs == 0
    rank = free.cumsum(0) - 1
    served = (ends <= free.sum()) | ((want == 0) & ~(grows & (held > 1)))
    pages = torch.full((refs.shape[0] + 1,), 0, dtype=torch.int64, device=refs.device)
    pages.scatter_(0, torch.where(free, rank, refs.shape[0]), torch.arange(refs.shape[0], device=refs.device))
    start = ends - want
    copy &= served
    given = (place >= have[:, None]) & (place < need[:, None]) & served[:, None]
    slot = (start + copy)[:, None] + place - have[:, None]
    table.copy_(torch.where(given, pages[slot.clamp(0, refs.shape[0])], table))
    copies = torch.where(copy[:, None], torch.stack((last, pages[start.clamp(max=refs.shape[0])]), 1), -1).to(torch.int32)
    table.scatter_(1, at, torch.where(copy[:, None], copies[:, 1:], table.gather(1, at)))
    refs.masked_fill_(free & (rank < torch.where(served & (want > 0), ends, 0).amax()), 1)
    refs.index_add_(0, last, -copy.to(torch.int32))
    s["kv_lens"].copy_(torch.where(served, new, old))
    return refs, table, s["kv_lens"], copies


_plain = {"tree": _plain_tree, "compact": _plain_compact, "copy": _plain_copy, "fork": _plain_fork,
          "resize": _plain_resize}


# ---------------------------------------------------------------- from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "compact": _exact_compact, "copy": _exact_copy, "fork": lambda s: None,
            "resize": lambda s: None}[case["op"]](s)


def _exact_tree(s):
    c = s["case"]
    if work(c)["flops"] > 1.5e13:  # at about 1 TFLOP/s in 64 bits
        return None
    cu, lens, group = s["cu_seqlens"].tolist(), s["kv_lens"].tolist(), c["Hq"] // c["Hk"]
    parents = _parents(c)
    dev = s["q"].device
    o = torch.zeros(s["tokens"], c["Hq"], c["d"], dtype=torch.float64, device=dev)
    lse = torch.zeros(s["tokens"], c["Hq"], dtype=torch.float64, device=dev)
    for b in range(c["B"]):
        a, e, length = cu[b], cu[b + 1], lens[b]
        pages = s["block_table"][b, :-(-length // c["page"])].long()
        ks, vs = (t[pages].movedim(1, 0).flatten(1, 2)[:, :length].double() for t in (s["k_cache"], s["v_cache"]))
        bias = torch.full((e - a, length), -math.inf, dtype=torch.float64)
        bias[:, :length - (e - a)] = 0
        for i in range(e - a):  # up from the token to the root
            t = i
            while t >= 0:
                bias[i, length - (e - a) + t] = 0
                t = parents[b][t]
        bias = bias.to(dev)
        for h in range(c["Hq"]):
            x = s["q"][a:e, h].double() @ ks[h // group].T * s["scale"] + bias
            z = torch.logsumexp(x, -1, keepdim=True)
            o[a:e, h] = (x - z).exp() @ vs[h // group]
            lse[a:e, h] = z[:, 0]
    return o, lse


def _exact_compact(s):
    c = s["case"]
    new, total = _lengths(c)
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    for b, kept in enumerate(_kept(c)):
        pages = s["block_table"][b].long()
        source = torch.tensor(kept, dtype=torch.int64, device=pages.device) + total[b] - new[b]
        to = torch.arange(len(kept), device=pages.device) + total[b] - new[b]
        for cache in caches:
            rows = cache[pages[source // c["page"]], :, source % c["page"]].clone()
            cache[pages[to // c["page"]], :, to % c["page"]] = rows
    return tuple(caches)


def _exact_copy(s):
    pairs = [p for p in s["pairs"].tolist() if p[0] >= 0]
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    for source, to in pairs:
        for cache in caches:
            cache[to] = cache[source]
    return tuple(caches)
