"""Pages of a cache: given out and back, shared, copied, compacted. All results
are whole numbers or moved bytes, so every comparison is exact."""
import ctypes

import numpy as np
import pytest
import torch

import attention_kl_loss_gb300 as skl
from attention_kl_loss_gb300 import binding
from oracle import page_ops as orc
from test_paged import Rows, _cu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
NO_PAGES = binding.STREAMKL_ERR_NO_PAGES


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Tables:
    """Counts, tables and lengths on the device beside those of the oracle."""

    def __init__(self, B, width, pages, page, stride=None):
        self.page, self.width = page, width
        self.refs, self.table, self.lens = np.zeros(pages, np.int32), np.full((B, width), -1, np.int32), np.zeros(B, np.int32)
        self.d_refs, self.d_lens = _dev(self.refs), _dev(self.lens)
        self.whole = torch.full((B, stride or width), -7, dtype=torch.int32, device="cuda")
        self.d_table = self.whole[:, :width]
        self.d_table.copy_(_dev(self.table))
        self.status = binding.new_status()

    def resize(self, new_lens, **kw):
        served = int(self.status.item())
        assert served == 0
        got = skl.streamkl_paged_resize(self.d_refs, self.d_table, self.d_lens, _dev(new_lens), self.page,
                                        dev_status=self.status, **kw)
        copies, all_there = orc.resize(self.refs, self.table, self.lens, np.asarray(new_lens), self.page)
        assert int(self.status.item()) == (0 if all_there else NO_PAGES)
        self.status.zero_()
        assert np.array_equal(got.cpu().numpy(), copies)
        self.check()
        return got

    def fork(self, source, **kw):
        got = skl.streamkl_paged_fork(self.d_refs, self.d_table, self.d_lens, _dev(source), dev_status=self.status, **kw)
        assert got[0] is self.d_refs and got[1] is self.d_table and got[2] is self.d_lens
        orc.fork(self.refs, self.table, self.lens, source)
        assert int(self.status.item()) == 0
        self.check()

    def check(self):
        assert np.array_equal(self.d_lens.cpu().numpy(), self.lens)
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs)
        assert torch.all(self.whole[:, self.width:] == -7)
        orc.check_held(self.refs, self.table, self.lens, self.page)


# ---------------------------------------------------------------- fork, resize
def test_oracle_keeps_the_invariant_and_runs_dry():
    """The oracle itself, on the CPU: random steps keep counts and tables in line; a shortage serves a prefix."""
    rng = np.random.default_rng(0)
    refs, table, lens = np.zeros(24, np.int32), np.full((6, 8), -1, np.int32), np.zeros(6, np.int32)
    short = 0
    for _ in range(300):
        if rng.random() < 0.3:
            orc.fork(refs, table, lens, rng.integers(0, 6, 6))
        else:
            _, fine = orc.resize(refs, table, lens, rng.integers(0, 8 * 16 + 1, 6), 16)
            short += not fine
        orc.check_held(refs, table, lens, 16)
    assert 0 < short < 300
    # three sequences in one shared, partly filled page: two copies, the last keeps it
    refs, table, lens = np.zeros(9, np.int32), np.full((3, 2), -1, np.int32), np.zeros(3, np.int32)
    orc.resize(refs, table, lens, np.array([20, 0, 0]), 16)
    orc.fork(refs, table, lens, [0, 0, 0])
    copies, fine = orc.resize(refs, table, lens, np.array([21, 22, 23]), 16)
    assert fine and copies.tolist() == [[1, 2], [1, 3], [-1, -1]]


@pytest.mark.gpu
@pytest.mark.parametrize("B,width,pages,page,stride", [
    (1, 1, 1, 16, None), (1, 5, 7, 16, 9), (3, 4, 13, 1024, None), (7, 33, 130, 32, 40), (64, 20, 700, 16, None),
    (65, 17, 33001, 64, 19), (300, 9, 1025, 16, None), (1100, 6, 4096, 16, None), (40, 1000, 70003, 16, None),
    (30, 9000, 300001, 16, None),
    (20, 40000, 1100000, 16, None), (4096, 3, 9000, 16, None),
])
def test_random_steps(B, width, pages, page, stride):
    """Sequences grow, shrink, end and go on from one another; some steps ask for more pages than there are."""
    rng = np.random.default_rng(B + pages)
    t = Tables(B, width, pages, page, stride)
    full = width * page
    few = max(1, min(full, pages * page // B))  # what leaves pages over
    for step in range(14):
        what = rng.random()
        if what < 0.25:
            t.fork(rng.integers(0, B, B))
        elif what < 0.35:
            t.fork(rng.permutation(B))
        elif what < 0.6:
            t.resize(np.clip(t.lens + rng.integers(-page - 2, page + 3, B), 0, full))
        elif what < 0.7:
            t.resize(np.where(rng.random(B) < 0.5, 0, t.lens))
        elif what < 0.85:
            t.resize(rng.integers(0, full + 1, B))
        else:
            t.resize(rng.integers(0, few + 1, B))


@pytest.mark.gpu
def test_pages_go_out_lowest_first_and_a_shared_last_page_is_copied():
    t = Tables(4, 4, 10, 16)
    t.resize([40, 16, 0, 0])
    assert t.table[0].tolist() == [0, 1, 2, -1] and t.table[1, 0] == 3
    t.fork([0, 1, 0, 0])                      # three in page 2
    assert t.refs[:4].tolist() == [3, 3, 3, 1]
    got = t.resize([41, 17, 48, 16])          # the last of them shrinks, so one copy is left to make
    assert got.tolist() == [[2, 4], [-1, -1], [-1, -1], [-1, -1]] and t.refs[2] == 1
    got = t.resize([0, 0, 0, 0])
    assert not t.refs.any() and torch.all(got == -1)


@pytest.mark.gpu
def test_too_few_pages_serve_the_first_sequences_and_those_that_ask_for_none():
    t = Tables(5, 8, 6, 16)
    t.resize([16, 20, 20, 0, 5])    # 1 + 2 + 2 + 1: all six
    t.resize([48, 21, 0, 16, 6])    # the third gives two back, the first takes them, the fourth finds none
    assert t.lens.tolist() == [48, 21, 0, 0, 6]
    # a page shared by one that is not served must not be written by the next
    t = Tables(3, 4, 3, 16)
    t.resize([20, 0, 0])
    t.fork([0, 0, 2])
    t.resize([60, 21, 0])           # the first asks for a copy and two more, one is free: neither grows
    assert t.lens.tolist() == [20, 20, 0] and t.refs.tolist() == [2, 2, 0]
    t.resize([20, 21, 0])           # alone it gets its copy
    assert t.lens.tolist() == [20, 21, 0]


@pytest.mark.gpu
def test_bad_numbers_are_reported_and_left_out():
    def fresh():
        t = Tables(4, 4, 16, 16)
        t.resize([20, 30, 40, 0])
        return t

    for place, value in (("new", -1), ("new", 65), ("old", -3), ("old", 1 << 30)):
        t = fresh()
        want = np.array([33, 10, 41, 5])
        if place == "new":
            given = want.copy()
            given[1] = value
        else:
            given = want
            t.d_lens[1] = value
        skl.streamkl_paged_resize(t.d_refs, t.d_table, t.d_lens, _dev(given), 16, dev_status=t.status)
        assert int(t.status.item()) == binding.STREAMKL_ERR_INVALID_ARG
        kept = int(t.d_lens[1])
        assert kept == (30 if place == "new" else value)
        want[1] = t.lens[1]
        orc.resize(t.refs, t.table, t.lens, want, 16)
        t.d_lens[1] = int(t.lens[1])
        t.status.zero_()
        t.check()
    # an entry that is no page: nothing is counted for it
    for entry in (16, -5):
        t = fresh()
        t.d_table[1, 1] = entry
        skl.streamkl_paged_resize(t.d_refs, t.d_table, t.d_lens, _dev([20, 5, 40, 0]), 16, dev_status=t.status)
        assert int(t.status.item()) == binding.STREAMKL_ERR_INVALID_ARG
        assert t.d_lens.tolist() == [20, 5, 40, 0] and t.d_table[1].tolist() == [2, -1, -1, -1]
        assert t.d_refs.tolist() == [1] * 7 + [0] * 9
    t = fresh()
    t.d_table[1, 1] = 77
    skl.streamkl_paged_resize(t.d_refs, t.d_table, t.d_lens, _dev([20, 31, 40, 0]), 16, dev_status=t.status)
    assert int(t.status.item()) == binding.STREAMKL_ERR_INVALID_ARG and t.d_lens.tolist() == [20, 31, 40, 0]
    # sources that are no sequences stay
    for s in (-1, 4, 1 << 30):
        t = fresh()
        skl.streamkl_paged_fork(t.d_refs, t.d_table, t.d_lens, _dev([0, s, 0, 2]), dev_status=t.status)
        assert int(t.status.item()) == binding.STREAMKL_ERR_INVALID_ARG
        orc.fork(t.refs, t.table, t.lens, [0, 1, 0, 2])
        t.status.zero_()
        t.check()


@pytest.mark.gpu
def test_captured_steps_replay():
    """Resize and fork change their arguments in place, so a graph's replays go on from where the last one left them."""
    t = Tables(8, 12, 200, 16)
    t.resize([50, 0, 70, 33, 16, 0, 5, 100])
    new, source = _dev(np.arange(8) * 20), _dev([0, 0, 2, 2, 4, 5, 7, 7])
    skl.streamkl_paged_resize(t.d_refs, t.d_table, t.d_lens, t.d_lens.clone(), 16)  # (the first call sets attributes)
    skl.streamkl_paged_fork(t.d_refs, t.d_table, t.d_lens, _dev(np.arange(8)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        copies = skl.streamkl_paged_resize(t.d_refs, t.d_table, t.d_lens, new, 16, dev_status=t.status)
        skl.streamkl_paged_fork(t.d_refs, t.d_table, t.d_lens, source, dev_status=t.status)
    rng = np.random.default_rng(1)
    for _ in range(4):
        to = rng.integers(0, 12 * 16, 8)
        new.copy_(_dev(to))
        graph.replay()
        want, fine = orc.resize(t.refs, t.table, t.lens, to, 16)
        assert fine and np.array_equal(copies.cpu().numpy(), want)
        orc.fork(t.refs, t.table, t.lens, source.tolist())
        t.check()


@pytest.mark.gpu
def test_captured_steps_of_large_tables_replay():
    """Two kernels, the second launched beside the first's end, and a cluster of sixteen blocks, in a graph."""
    B, width, page = 20, 40000, 16
    t = Tables(B, width, 700000, page)
    rng = np.random.default_rng(3)
    t.resize(rng.integers(0, width * page // 2, B))
    new, source = _dev(t.lens), _dev(np.arange(B))
    step = torch.empty_like(new)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        copies = skl.streamkl_paged_resize(t.d_refs, t.d_table, t.d_lens, new, page, dev_status=t.status, step_lens=step)
        skl.streamkl_paged_fork(t.d_refs, t.d_table, t.d_lens, source, dev_status=t.status)
    for i in range(6):
        to = rng.integers(0, width * page + 1, B) if i % 2 else np.clip(t.lens + rng.integers(-200000, 200000, B), 0, width * page)
        beams = np.arange(B) if i % 3 == 0 else rng.integers(0, B, B)
        new.copy_(_dev(to))
        source.copy_(_dev(beams))
        graph.replay()
        want, fine = orc.resize(t.refs, t.table, t.lens, to, page)
        assert np.array_equal(copies.cpu().numpy(), want) and int(t.status.item()) == (0 if fine else NO_PAGES)
        assert np.array_equal(step.cpu().numpy(), np.where(t.lens == to, to, 0))
        t.status.zero_()
        orc.fork(t.refs, t.table, t.lens, beams.tolist())
        t.check()


@pytest.mark.gpu
@pytest.mark.parametrize("way", ["native", "ctypes"])
@pytest.mark.parametrize("B,width,pages", [(1, 4, 3), (6, 8, 20), (300, 9, 1025), (1100, 6, 3001), (30, 9000, 100001)])
def test_step_lens_are_the_new_lengths_or_zero(B, width, pages, way, monkeypatch):
    """The lengths for the step's calls: what was asked for, 0 where there were no places or numbers do not fit."""
    if way == "ctypes":
        monkeypatch.setattr(binding.load(), "native", None)
    rng = np.random.default_rng(B)
    t = Tables(B, width, pages, 16)
    step = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    short = 0
    for _ in range(8):
        if rng.random() < 0.4:
            t.fork(rng.integers(0, B, B))
        new = rng.integers(0, width * 16 + 1, B) if rng.random() < 0.5 else np.clip(t.lens + rng.integers(-9, 20, B), 0, width * 16)
        t.resize(new, step_lens=step)
        served = t.lens == new
        short += not served.all()
        assert np.array_equal(step.cpu().numpy(), np.where(served, new, 0))
    assert short or B == 1
    bad = t.lens.copy()
    bad[0] = -1
    skl.streamkl_paged_resize(t.d_refs, t.d_table, t.d_lens, _dev(bad), 16, dev_status=t.status, step_lens=step)
    assert int(t.status.item()) == binding.STREAMKL_ERR_INVALID_ARG
    assert step.tolist() == [0] + t.lens[1:].tolist()
    for wrong in (t.d_lens, step.long(), torch.zeros(B + 1, dtype=torch.int32, device="cuda")):
        with pytest.raises((ValueError, binding.StreamKLError), match="step_lens"):
            skl.streamkl_paged_resize(t.d_refs, t.d_table, t.d_lens, _dev(t.lens), 16, step_lens=wrong)


# ---------------------------------------------------------------- copy, compact
def _caches(pages, HK, page, d, dt, layout, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if layout == "heads":
        return [torch.randn(pages, HK, page, d, generator=g, device="cuda").to(dt) for _ in range(2)]
    both = torch.randn(pages, 2, page, HK, d, generator=g, device="cuda").to(dt)
    return [both[:, i].transpose(1, 2) for i in range(2)]


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("n,HK,page,d,dtype,layout", [(1, 1, 16, 64, "bf16", "heads"), (9, 3, 32, 128, "fp16", "slots"),
                                                      (40, 8, 16, 128, "bf16", "heads"), (5, 7, 1024, 64, "fp16", "slots"),
                                                      (700, 2, 64, 64, "bf16", "heads"), (33, 5, 128, 128, "bf16", "slots")])
def test_copy_moves_whole_pages_and_nothing_else(n, HK, page, d, dtype, layout):
    pages = 2 * n + 2
    k, v = _caches(pages, HK, page, d, TYPES[dtype], layout)
    k[0, 0, 0, 0] = float("nan")  # bytes are moved, whatever they are
    rng = np.random.default_rng(n)
    pairs = rng.permutation(pages)[:2 * n].reshape(n, 2)
    pairs[rng.random(n) < 0.3] = -1
    if n > 5:
        pairs[2] = -3, -9
        pairs[4, 1] = pairs[4, 0]  # onto itself
    want = [t.clone() for t in (k, v)]
    for s, t in pairs:
        if s >= 0:
            for w in want:
                w[t] = w[s]
    st = binding.new_status()
    out = skl.streamkl_paged_copy(k, v, _dev(pairs), dev_status=st)
    binding.raise_on_device_status(st)
    assert out[0] is k and out[1] is v and _same(k, want[0]) and _same(v, want[1])


@pytest.mark.gpu
def test_copy_reports_pairs_that_are_none_and_copies_the_rest():
    k, v = _caches(8, 2, 16, 64, torch.bfloat16, "heads")
    want = [t.clone() for t in (k, v)]
    for w in want:
        w[3] = w[1]
    for bad in ((-1, 5), (5, -1), (8, 5), (5, 8)):
        st = binding.new_status()
        skl.streamkl_paged_copy(k, v, _dev([(1, 3), bad]), dev_status=st)
        assert int(st.item()) == binding.STREAMKL_ERR_INVALID_ARG and _same(k, want[0]) and _same(v, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("number", [8, 1 << 30, 2 ** 31 - 1])
def test_copy_reports_a_number_that_is_no_page_onto_itself(number):
    k, v = _caches(8, 2, 16, 64, torch.bfloat16, "heads")
    want = [t.clone() for t in (k, v)]
    for w in want:
        w[3] = w[1]
    st = binding.new_status()
    skl.streamkl_paged_copy(k, v, _dev([(number, number), (5, 5), (1, 3)]), dev_status=st)
    assert int(st.item()) == binding.STREAMKL_ERR_INVALID_ARG and _same(k, want[0]) and _same(v, want[1])
    st.zero_()
    skl.streamkl_paged_copy(k, v, _dev([(5, 5), (1, 3)]), dev_status=st)
    assert int(st.item()) == 0


COMPACT = [
    # lens, drafted, kept lists (None: random), HK, page, d, type, layout, most
    ([1], [1], [[0]], 1, 16, 64, "bf16", "heads", 1),
    ([20], [7], [[1, 3, 6]], 2, 16, 128, "fp16", "slots", 4),
    ([40, 33, 16, 9], [12, 0, 16, 9], [[], [], [15], [0, 1, 2, 3, 4, 5, 6, 7, 8]], 3, 16, 64, "bf16", "heads", 20),
    ([300, 64, 70], [64, 64, 33], None, 8, 32, 128, "bf16", "heads", 32),
    ([300, 64, 70], [64, 64, 33], None, 5, 16, 64, "fp16", "slots", 40),
    ([3000, 1500, 700], [3000, 1100, 700], None, 4, 64, 128, "bf16", "slots", 2000),
    ([5000, 4100], [5000, 4100], None, 2, 16, 64, "fp16", "heads", 4100),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new,lists,HK,page,d,dtype,layout,most", COMPACT)
def test_compact_moves_the_kept_rows_in_place(lens, new, lists, HK, page, d, dtype, layout, most):
    rng = np.random.default_rng(sum(lens))
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    k, v = _caches(pages, HK, page, d, TYPES[dtype], layout)
    k[pages - 1] = float("nan")
    order = rng.permutation(pages)
    table = np.full((len(lens), max(need)), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    if lists is None:
        lists = [sorted(rng.choice(n, min(n, most) if b == 0 else rng.integers(0, min(n, most) + 1), replace=False).tolist())
                 for b, n in enumerate(new)]
    kept = np.full((len(lens), most + 3), 99, np.int32)  # rows further apart than they are long
    for b, l in enumerate(lists):
        kept[b, :len(l)] = l
    want = [t.contiguous().view(torch.int16).cpu().numpy().copy() for t in (k, v)]
    for b, l in enumerate(lists):
        for w in want:
            orc.compact(w, table[b], lens[b], new[b], l)
    st = binding.new_status()
    out = skl.streamkl_paged_compact(k, v, _dev(table), _dev(lens), _cu(new), _dev(kept)[:, :most], _dev([len(l) for l in lists]),
                                     dev_status=st)
    binding.raise_on_device_status(st)
    assert out[0] is k and out[1] is v
    for t, w in zip((k, v), want):
        assert np.array_equal(t.contiguous().view(torch.int16).cpu().numpy(), w)


@pytest.mark.gpu
@pytest.mark.parametrize("most", [6, 50])
def test_compact_reports_lists_that_do_not_fit_and_does_the_others(most):
    lens, new = [40, 60, 50], [20, 20, 20]
    table = np.arange(12).reshape(3, 4)
    good = [3, 5, 9, 19]
    for what in ("order", "twice", "range", "negative", "many", "length", "offsets", "page"):
        k, v = _caches(13, 2, 16, 64, torch.bfloat16, "heads")
        lists, count, ls, cu, tab = [good] * 3, [4, 4, 4], list(lens), [0, 20, 40, 60], table.copy()
        if what == "order":
            lists = [good, [3, 9, 5, 19], good]
        elif what == "twice":
            lists = [good, [3, 5, 5, 19], good]
        elif what == "range":
            lists = [good, [3, 5, 9, 20], good]
        elif what == "negative":
            lists = [good, [-1, 5, 9, 19], good]
        elif what == "many":
            count[1] = most + 1
        elif what == "length":
            ls[1] = 19
        elif what == "offsets":
            cu = [0, 20, 10, 30]
        else:
            tab[1] = [4, 5, 13, -1]  # the pages of the last 20
        want = [t.contiguous().view(torch.int16).cpu().numpy().copy() for t in (k, v)]
        for b in (0, 2):
            for w in want:
                orc.compact(w, table[b], lens[b], new[b], good)
        kept = np.zeros((3, most), np.int32)
        kept[:, :4] = lists
        st = binding.new_status()
        skl.streamkl_paged_compact(k, v, _dev(tab), _dev(ls), _dev(cu), _dev(kept), _dev(count), dev_status=st)
        assert int(st.item()) == binding.STREAMKL_ERR_INVALID_ARG, what
        for t, w in zip((k, v), want):
            assert np.array_equal(t.contiguous().view(torch.int16).cpu().numpy(), w), what


@pytest.mark.gpu
def test_pages_past_32_bits():
    """Pages whose offset in elements, and in 16-byte vectors, does not fit 32 bits: 2^32 elements and more."""
    page_elems = 64 * 1024 * 128
    pages = (1 << 32) // page_elems + 3
    k = torch.zeros(pages, 64, 1024, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(1, 64, 1024, 128, dtype=torch.bfloat16, device="cuda").expand(pages, -1, -1, -1)
    with pytest.raises(binding.StreamKLError):  # pages that are one another
        skl.streamkl_paged_copy(k, v, _dev([(0, 1)]))
    v = torch.zeros_like(k)
    last = pages - 1
    k[last] = torch.randn(64, 1024, 128, device="cuda").to(torch.bfloat16)
    v[1] = torch.randn(64, 1024, 128, device="cuda").to(torch.bfloat16)
    st = binding.new_status()
    skl.streamkl_paged_copy(k, v, _dev([(last, 0), (1, last - 1)]), dev_status=st)
    binding.raise_on_device_status(st)
    assert torch.equal(k[0], k[last]) and torch.equal(v[last - 1], v[1]) and not v[0].any() and not k[1].any()
    skl.streamkl_paged_compact(k, v, _dev([[last]]), _dev([1024]), _cu([1024]), _dev([[7, 1000]]), _dev([2]), dev_status=st)
    binding.raise_on_device_status(st)
    assert torch.equal(k[last, :, 0], k[0, :, 7]) and torch.equal(k[last, :, 1], k[0, :, 1000])
    assert torch.equal(k[last, :, 2:], k[0, :, 2:])


@pytest.mark.gpu
def test_on_another_stream_and_both_ways_to_the_library(monkeypatch):
    """The way through ctypes does what the native one does; a given stream is the one that is used."""
    lib = binding.load()
    assert lib.native is not None
    results = []
    for way in ("native", "ctypes", "stream"):
        if way == "ctypes":
            monkeypatch.setattr(lib, "native", None)
        side = torch.cuda.Stream() if way == "stream" else None
        t = Tables(6, 10, 70, 16)
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
        k, v = _caches(70, 2, 16, 64, torch.bfloat16, "heads")
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
        new, source = [_dev(x) for x in ([40, 33, 0, 16, 7, 100], [50, 40, 60, 17, 8, 99])], _dev([0, 1, 0, 3, 3, 5])
        torch.cuda.synchronize()
        kw = dict(dev_status=t.status, stream=side)
        skl.streamkl_paged_resize(t.d_refs, t.d_table, t.d_lens, new[0], 16, **kw)
        skl.streamkl_paged_fork(t.d_refs, t.d_table, t.d_lens, source, **kw)
        out = torch.empty(6, 2, dtype=torch.int32, device="cuda") if way == "ctypes" else None
        copies = skl.streamkl_paged_resize(t.d_refs, t.d_table, t.d_lens, new[1], 16, out=out, **kw)
        skl.streamkl_paged_copy(k, v, copies, **kw)
        skl.streamkl_paged_compact(k, v, t.d_table, t.d_lens, _cu([10, 10, 20, 1, 2, 30]), _dev([[0, 3]] * 6),
                                   _dev([2, 1, 2, 1, 0, 2]), **kw)
        torch.cuda.synchronize()
        binding.raise_on_device_status(t.status)
        results.append([x.clone() for x in (t.d_refs, t.d_table, t.d_lens, copies, k.view(torch.int16), v.view(torch.int16))])
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    from attention_kl_loss_gb300 import build
    build.build()
    return binding.load()


def _struct(name, *fields):
    kinds = {"P": ctypes.c_void_p, "q": ctypes.c_longlong, "i": ctypes.c_int, "N": ctypes.c_size_t, "R": Rows}
    return type(name, (ctypes.Structure,), {"_fields_": [("struct_size", ctypes.c_size_t)] + [
        (n, kinds[k]) for k, names in fields for n in names.split()]})


CompactArgs = _struct("CompactArgs", ("R", "k_cache v_cache"), ("P", "block_table"), ("q", "table_stride"),
                      ("P", "kv_lens cu_seqlens kept"), ("q", "kept_stride"), ("P", "num_kept dev_status"),
                      ("i", "dtype B HK d page_size num_pages max_pages max_kept"))
CopyArgs = _struct("CopyArgs", ("R", "k_cache v_cache"), ("P", "pairs dev_status"), ("i", "dtype n HK d page_size num_pages"))
ForkArgs = _struct("ForkArgs", ("P", "page_refs block_table"), ("q", "table_stride"), ("P", "kv_lens source dev_status"),
                   ("i", "B num_pages max_pages"))
ResizeArgs = _struct("ResizeArgs", ("P", "page_refs block_table"), ("q", "table_stride"),
                     ("P", "kv_lens new_lens copies dev_status"), ("i", "B num_pages max_pages page_size"))


def _raw(cls, over):
    """Arguments that only the host looks at: a refused call never uses its addresses."""
    a = cls(struct_size=ctypes.sizeof(cls))
    base = dict(table_stride=4, kept_stride=4, dtype=0, B=2, n=2, HK=2, d=64, page_size=16, num_pages=9, max_pages=4,
                max_kept=4, k_cache=Rows(4096, (2048, 1024, 64)), v_cache=Rows(4096, (2048, 1024, 64)))
    for n, kind in cls._fields_[1:]:
        setattr(a, n, base.get(n, 4096 if kind is ctypes.c_void_p else 0))
    for n, v in over.items():
        rows, _, field = n.partition("__")
        if not field:
            setattr(a, n, v)
        elif field == "data":
            getattr(a, rows).data = v
        else:
            getattr(a, rows).stride[:] = v
    return ctypes.byref(a)


CACHES = [(dict(struct_size=8), 1), (dict(dtype=2), 2), (dict(d=80), 2), (dict(HK=0), 1), (dict(num_pages=0), 1),
          (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=2048), 2), (dict(k_cache__data=None), 1),
          (dict(v_cache__data=4100), 1), (dict(k_cache__stride=(2048, 1024, 60)), 1), (dict(v_cache__stride=(0, 1024, 64)), 1),
          (dict(k_cache__stride=(1024, 1024, 64)), 1), (dict(dev_status=None), 1)]
TABLES = [(dict(struct_size=8), 1), (dict(B=0), 1), (dict(B=4097), 2), (dict(num_pages=0), 1), (dict(num_pages=(1 << 23) + 1), 2), (dict(max_pages=0), 1),
          (dict(max_pages=1 << 30, table_stride=1 << 30), 2), (dict(page_refs=None), 1), (dict(block_table=None), 1),
          (dict(kv_lens=None), 1), (dict(table_stride=3), 1), (dict(dev_status=None), 1)]


@pytest.mark.parametrize("over,status", CACHES + [
    (dict(B=0), 1), (dict(max_pages=1 << 27), 2), (dict(table_stride=-1), 1), (dict(block_table=None), 1),
    (dict(kv_lens=None), 1), (dict(cu_seqlens=None), 1), (dict(kept=None), 1), (dict(num_kept=None), 1), (dict(max_kept=0), 1),
    (dict(kept_stride=3), 1), (dict(kept_stride=-1, B=1), 1), (dict(B=1 << 28, HK=8, k_cache__stride=(8192, 1024, 64),
                                                                   v_cache__stride=(8192, 1024, 64)), 2),
    (dict(B=(1 << 25) + 1), 2)])
def test_compact_c_call_refuses(lib, over, status):
    assert lib.streamkl_paged_compact(_raw(CompactArgs, over), None) == status and lib.streamkl_last_error()


@pytest.mark.parametrize("over,status", CACHES + [(dict(n=0), 1), (dict(pairs=None), 1), (dict(pairs=4100), 1),
                                                  (dict(HK=65536), 2), (dict(n=1 << 30, HK=4096), 2),
                                                  (dict(n=(1 << 30) + 1, HK=1), 2), (dict(n=1 << 28, HK=17), 2)])
def test_copy_c_call_refuses(lib, over, status):
    assert lib.streamkl_paged_copy(_raw(CopyArgs, over), None) == status and lib.streamkl_last_error()


@pytest.mark.parametrize("over,status", TABLES + [(dict(source=None), 1)])
def test_fork_c_call_refuses(lib, over, status):
    assert lib.streamkl_paged_fork(_raw(ForkArgs, over), None) == status and lib.streamkl_last_error()


@pytest.mark.parametrize("over,status", TABLES + [
    (dict(new_lens=None), 1), (dict(copies=None), 1), (dict(copies=4100), 1), (dict(page_refs=4104), 1),
    (dict(page_size=24), 2), (dict(page_size=1024, max_pages=1 << 21, table_stride=1 << 21), 2)])
def test_resize_c_call_refuses(lib, over, status):
    assert lib.streamkl_paged_resize(_raw(ResizeArgs, over), None) == status and lib.streamkl_last_error()


def test_resize_takes_its_struct_with_and_without_step_lens(lib):
    long = _struct("LongResizeArgs", *[(k[0], k[1]) for k in (
        ("P", "page_refs block_table"), ("q", "table_stride"), ("P", "kv_lens new_lens copies dev_status"),
        ("i", "B num_pages max_pages page_size"), ("P", "step_lens"))])
    for over, status, text in ((dict(page_size=24, step_lens=8192), 2, b"page size"), (dict(), 1, b"step_lens"),  # (kv_lens)
                               (dict(kv_lens=8192), 1, b"step_lens"), (dict(struct_size=ctypes.sizeof(long) + 8), 1, b"struct_size"),
                               (dict(struct_size=ctypes.sizeof(long) - 16), 1, b"struct_size")):
        assert lib.streamkl_paged_resize(_raw(long, over), None) == status and text in lib.streamkl_last_error()
    assert ctypes.sizeof(long) == ctypes.sizeof(ResizeArgs) + 8
    assert lib.streamkl_paged_resize(_raw(ResizeArgs, dict(page_size=24)), None) == 2


def test_native_calls_leave_what_they_do_not_know(lib):
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    for call in (lib.native.tree_attn, lib.native.compact, lib.native.copy, lib.native.fork, lib.native.resize):
        assert call() is None and call(None) is None
        assert all(call(*[a] * n) is None for n in range(3, 16) for a in (x, None, 1, "text"))


@pytest.mark.gpu
def test_python_calls_refuse():
    k, v = _caches(8, 2, 16, 64, torch.bfloat16, "heads")
    i = _dev
    table, lens, cu, kept, count = i([[0, 1], [2, 3]]), i([20, 30]), _cu([5, 5]), i([[0, 1]] * 2), i([2, 2])
    refs, pairs = i([1] * 4 + [0] * 4), i([[0, 5]])
    for match, call, args in [
        ("cu_seqlens", skl.streamkl_paged_compact, (k, v, table, lens, None, kept, count)),
        ("cu_seqlens", skl.streamkl_paged_compact, (k, v, table, lens, cu[:2], kept, count)),
        ("kept", skl.streamkl_paged_compact, (k, v, table, lens, cu, kept[:1], count)),
        ("kept", skl.streamkl_paged_compact, (k, v, table, lens, cu, kept.long(), count)),
        ("num_kept", skl.streamkl_paged_compact, (k, v, table, lens, cu, kept, None)),
        ("num_kept", skl.streamkl_paged_compact, (k, v, table, lens, cu, kept, count[:1])),
        ("both", skl.streamkl_paged_compact, (k, v[1:], table, lens, cu, kept, count)),
        ("unsupported", skl.streamkl_paged_copy, (k.float(), v.float(), pairs)),
        ("both", skl.streamkl_paged_copy, (k, v[1:], pairs)),
        ("pairs", skl.streamkl_paged_copy, (k, v, pairs.long())),
        ("pairs", skl.streamkl_paged_copy, (k, v, i([[0, 5, 1]]))),
        ("pairs", skl.streamkl_paged_copy, (k, v, i([[0, 5], [1, 6]]).t().contiguous().t())),
        ("page_refs", skl.streamkl_paged_fork, (refs.long(), table, lens, count)),
        ("page_refs", skl.streamkl_paged_fork, (refs[None], table, lens, count)),
        ("block_table", skl.streamkl_paged_fork, (refs, table[0], lens, count)),
        ("kv_lens", skl.streamkl_paged_fork, (refs, table, lens[:1], count)),
        ("kv_lens", skl.streamkl_paged_fork, (refs, table, None, count)),
        ("source", skl.streamkl_paged_fork, (refs, table, lens, count[:1])),
        ("source", skl.streamkl_paged_fork, (refs, table, lens, None)),
        ("new_lens", skl.streamkl_paged_resize, (refs, table, lens, None, 16)),
        ("new_lens", skl.streamkl_paged_resize, (refs, table, lens, count.long(), 16)),
        ("out of range", skl.streamkl_paged_resize, (refs, table, lens, count, "16")),
    ]:
        with pytest.raises(ValueError, match=match):
            call(*args)
    with pytest.raises(ValueError, match="out"):
        skl.streamkl_paged_resize(refs, table, lens, lens.clone(), 16, out=torch.empty(2, 2, device="cuda"))
    with pytest.raises(binding.StreamKLError):
        skl.streamkl_paged_resize(refs, table, lens, lens.clone(), 20)
    none = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    assert skl.streamkl_paged_resize(refs, none, lens[:0], lens[:0], 16).shape == (0, 2)
    skl.streamkl_paged_fork(refs, none, lens[:0], lens[:0])
    skl.streamkl_paged_copy(k, v, none)
    skl.streamkl_paged_compact(k, v, table, lens, cu, kept[:, :0], count)


@pytest.mark.parametrize("call,args", [
    ("rope_fwd", ("q", "q", "q", "q")), ("rope_bwd", ("q",) * 6), ("append", ("q",) * 6), ("attn", ("q",) * 5), ("tree_attn", ("q",) * 6),
    ("compact", ("q",) * 7), ("copy", ("q",) * 3), ("fork", ("q",) * 4), ("resize", ("q",) * 4 + (16,))])
def test_a_failed_launch_is_raised_and_not_made_again(lib, call, args, monkeypatch):
    """The native way says that its launch failed: the call may have begun, and ctypes must not begin it again."""
    name = {"rope_fwd": "streamkl_qk_norm_rope_fwd", "rope_bwd": "streamkl_qk_norm_rope_bwd"}.get(call, "streamkl_paged_" + call)

    class Native:
        def __getattr__(self, _):
            return lambda *a: binding.STREAMKL_ERR_CUDA

    def again(*a):
        raise AssertionError("the call was made again")

    monkeypatch.setattr(lib, "native", Native())
    monkeypatch.setattr(lib, name, again)
    x = torch.zeros(2, 2, 2, dtype=torch.int32)
    with pytest.raises(binding.StreamKLError) as e:
        getattr(skl, name)(*[x if a == "q" else a for a in args])
    assert e.value.status == binding.STREAMKL_ERR_CUDA and name in str(e.value)


@pytest.mark.gpu
def test_the_native_way_returns_the_status_of_a_failed_launch(tmp_path):
    """The entries of a library that refuses, or whose launches fail: None for the one, the status for the other, one
    call each."""
    import functools
    import importlib.util
    import subprocess
    from attention_kl_loss_gb300 import build
    names = [n for n in binding._SIGNATURES if n.startswith(("streamkl_paged", "streamkl_qk"))]
    source = tmp_path / "entries.c"
    source.write_text("int result, calls;\n" + "\n".join(
        f"unsigned long {n}(void) {{ return 0; }}" if n.endswith("_size") else f"int {n}(void) {{ ++calls; return result; }}"
        for n in names))
    so = str(tmp_path / "entries.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", so, str(source)], check=True)
    stub = ctypes.CDLL(so)
    spec = importlib.util.spec_from_file_location("_marshal", build.marshal_path())
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    entries = module.entries(so)
    k, v = _caches(8, 2, 16, 64, torch.bfloat16, "heads")
    table, lens, cu, kept = _dev([[0, 1], [2, 3]]), _dev([20, 30]), _cu([5, 5]), _dev([[0, 1]] * 2)
    refs, mask, q = _dev([1] * 4 + [0] * 4), torch.ones(10, 1, dtype=torch.int32, device="cuda"), torch.zeros(
        10, 2, 64, dtype=torch.bfloat16, device="cuda")
    calls = [functools.partial(getattr(module, n), entries, *a) for n, a in (
        ("append", (q, q, k, v, table, lens, cu, None, None, None, 1e-6, False, None)),
        ("attn", (q, k, v, table, lens, cu, 5, 32, None, True, 0, None, None)),
        ("tree_attn", (q, k, v, table, lens, mask, cu, 5, 32, None, None, None)),
        ("compact", (k, v, table, lens, cu, kept, _dev([2, 2]), None)), ("copy", (k, v, _dev([[0, 5]]), None)),
        ("fork", (refs, table, lens, _dev([0, 1]), None)), ("resize", (refs, table, lens, lens.clone(), 16, None, None)))]
    for status in range(6):
        for i, call in enumerate(calls):
            ctypes.c_int.in_dll(stub, "result").value = status
            ctypes.c_int.in_dll(stub, "calls").value = 0
            got = call()
            assert ctypes.c_int.in_dll(stub, "calls").value == 1, i
            if status == binding.STREAMKL_OK:
                assert got is not None and type(got) is not int, i
            elif status == binding.STREAMKL_ERR_CUDA:
                assert got == status and type(got) is int, i
            else:
                assert got is None, (i, status)
