"""GPU: page tables (reserve, fork, free, compact) against plain Python lists, exactly, and
the row copies bit for bit."""
import random

import pytest
import torch

import gated_delta_rule_102_b200 as gdn
from attn_reference import Tables

pytestmark = pytest.mark.gpu
I32 = torch.int32
DEV = "cuda"


def dev(x):
    return torch.as_tensor(x, dtype=I32).to(DEV)


class Pool:
    def __init__(self, rows, width, pages, ps, offset=0):
        # counters that are not 16-byte aligned when offset is set
        self.ps, self.rows = ps, rows
        self.table = torch.full((rows, width), -1, dtype=I32, device=DEV)
        self.lens = torch.zeros(rows, dtype=I32, device=DEV)
        self.refs = torch.zeros(pages + offset, dtype=I32, device=DEV)[offset:]
        self.err = dev([0])
        self.model = Tables(self.table, self.lens, self.refs, ps)

    def check(self):
        self.model.same(self.table, self.lens, self.refs)

    def reserve(self, slots, counts, as_tensor=True):
        gdn.gdn_pages_reserve(self.ps, dev(slots), dev(counts) if as_tensor else counts[0], self.table, self.lens, self.refs, self.err)
        return self.model.reserve(slots, counts)

    def grow(self, slots, counts):
        self.lens.index_add_(0, dev(slots), dev(counts))
        for s, c in zip(slots, counts):
            self.model.lens[s] += c

    def fork(self, src, dst):
        a, z = dev([-9] * len(src)), dev([-9] * len(src))
        gdn.gdn_pages_fork(self.ps, dev(src), dev(dst), self.table, self.lens, self.refs, a, z, self.err)
        assert list(zip(a.tolist(), z.tolist())) == self.model.fork(src, dst)

    def free(self, slots):
        gdn.gdn_pages_free(dev(slots), self.table, self.lens, self.refs, self.err)
        self.model.free(dict.fromkeys(slots))

    def compact(self):
        P = self.refs.shape[0]
        a, z, n, remap = dev([0] * P), dev([0] * P), dev([7]), dev([0] * P)
        gdn.gdn_pages_compact(self.table, self.refs, a, z, n, remap, self.err)
        movers, holes, want = self.model.compact()
        k = len(movers)
        assert int(n) == k and a.tolist() == movers + [-1] * (P - k) and z.tolist() == holes + [-1] * (P - k)
        assert remap.tolist() == want
        return a, z, n


@pytest.mark.parametrize("rows,width,pages,ps,offset", [(6, 9, 40, 4, 1), (40, 70, 1200, 1, 3), (300, 20, 9000, 16, 0), (20, 2100, 20000, 2, 2)])
def test_random_histories(rows, width, pages, ps, offset):
    """Reserve, grow, fork, free and compact in random order: every table, length, counter,
    copy list and flag equal to the plain model's."""
    rng = random.Random(rows)
    p = Pool(rows, width, pages, ps, offset)
    for step in range(40):
        busy = [s for s in range(rows) if p.model.lens[s] or p.model.table[s][0] >= 0]
        idle = [s for s in range(rows) if s not in busy]
        what = rng.choice(["reserve", "reserve", "fork", "free", "compact"])
        if what == "reserve":
            slots = rng.sample(range(rows), rng.randint(1, rows))
            room = [width * ps - p.model.lens[s] for s in slots]
            one = rng.random() < 0.3
            top = min(room) if one else 0
            counts = [rng.randint(0, min(top, 40 * ps))] * len(slots) if one else [rng.randint(0, min(r, 40 * ps)) for r in room]
            flagged = p.reserve(slots, counts, as_tensor=not one)
            assert int(p.err) == (gdn.GDN_DEVICE_ERR_PAGE if flagged else 0)
            if not flagged:
                p.grow(slots, [rng.randint(0, c) for c in counts])
        elif what == "fork" and busy and idle:
            dst = rng.sample(idle, rng.randint(1, min(len(idle), 30)))
            src = [rng.choice(busy) for _ in dst]  # a parent may appear many times
            p.fork(src, dst)
        elif what == "free" and busy:
            slots = rng.sample(busy, rng.randint(1, len(busy)))
            p.free(slots + slots[:1])              # listed twice: released once
        elif what == "compact":
            p.compact()
        p.err.zero_()
        p.check()


def test_flags():
    p = Pool(6, 4, 8, 4)
    p.reserve([0, 1], [6, 3])
    p.grow([0, 1], [6, 3])
    p.check()
    before = [x.clone() for x in (p.table, p.lens, p.refs)]

    def same(flag):
        assert int(p.err) == flag
        assert all(torch.equal(a, b) for a, b in zip(before, (p.table, p.lens, p.refs)))
        p.err.zero_()
    gdn.gdn_pages_reserve(4, dev([-1, 6]), 3, p.table, p.lens, p.refs, p.err)
    same(gdn.GDN_DEVICE_ERR_SLOT_RANGE)
    gdn.gdn_pages_reserve(4, dev([0, 2]), dev([11, -1]), p.table, p.lens, p.refs, p.err)   # 17 tokens in 16 places; a negative count
    same(gdn.GDN_DEVICE_ERR_SEQLEN)
    a, z = dev([0] * 3), dev([0] * 3)
    gdn.gdn_pages_fork(4, dev([0, 9, 2]), dev([7, 3, 2]), p.table, p.lens, p.refs, a, z, p.err)
    same(gdn.GDN_DEVICE_ERR_SLOT_RANGE)
    assert a.tolist() == [-1] * 3 and z.tolist() == [-2] * 3
    gdn.gdn_pages_fork(4, dev([0]), dev([1]), p.table, p.lens, p.refs, a[:1], z[:1], p.err)   # the child's row is in use
    same(gdn.GDN_DEVICE_ERR_PAGE)
    gdn.gdn_pages_free(dev([-3, 77]), p.table, p.lens, p.refs, p.err)
    same(gdn.GDN_DEVICE_ERR_SLOT_RANGE)
    # no page left for the second child: it stays empty, the first is complete
    p.reserve([2], [16]); p.grow([2], [16])
    p.check()
    p.fork([0, 0], [3, 4])
    assert int(p.err) == gdn.GDN_DEVICE_ERR_PAGE
    p.check()
    # too few pages: the first sequence gets all of its pages, the second none
    p = Pool(3, 8, 5, 1)
    assert p.reserve([2, 0, 1], [3, 4, 1]) and int(p.err) == gdn.GDN_DEVICE_ERR_PAGE
    p.check()


@pytest.mark.parametrize("row_bytes", [16, 4096, 4112, 100000, 1 << 21])
def test_copy_rows(row_bytes):
    rows, n = 12, 5
    gen = torch.Generator(device=DEV).manual_seed(row_bytes)
    bufs = [torch.randint(0, 256, (rows, b), generator=gen, device=DEV, dtype=torch.uint8) for b in (row_bytes, 48, row_bytes)]
    want = [b.clone() for b in bufs]
    src, dst = [3, 7, -1, 3, 11], [0, 9, 4, 1, -1]
    for w in want:
        for a, z in zip(src, dst):
            if a >= 0 and z >= 0:
                w[z] = w[a]
    err = dev([0])
    gdn.gdn_copy_rows(bufs, dev(src), dev(dst), err_flag=err)
    assert int(err) == 0 and all(torch.equal(a, b) for a, b in zip(bufs, want))
    gdn.gdn_copy_rows(bufs, dev([12, 0]), dev([2, 12]), err_flag=err)                   # out of range: skipped
    assert int(err) == gdn.GDN_DEVICE_ERR_SLOT_RANGE and all(torch.equal(a, b) for a, b in zip(bufs, want))
    err.zero_()
    gdn.gdn_copy_rows(bufs, dev([5, 6]), dev([2, 8]), n_dev=dev([1]), err_flag=err)     # the first pair only
    for w in want:
        w[2] = w[5]
    assert int(err) == 0 and all(torch.equal(a, b) for a, b in zip(bufs, want))
    for bad in (-1, 3):
        gdn.gdn_copy_rows(bufs, dev([5, 6]), dev([2, 8]), n_dev=dev([bad]), err_flag=err)
        assert int(err) == gdn.GDN_DEVICE_ERR_BATCH and all(torch.equal(a, b) for a, b in zip(bufs, want))
        err.zero_()


def test_forked_and_compacted_caches_hold_the_same_tokens():
    """Sequences are written, forked, some dropped, the pool compacted: every sequence still
    reads its own tokens through its table, in every layer and in the GDN state pool."""
    ps, rows, width, pages, d = 8, 10, 12, 90, 64
    p = Pool(rows, width, pages, ps)
    layers = [torch.zeros(pages, ps, 1, d, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    state = torch.randn(rows, 4, 16, 16, device=DEV)
    lens = {0: 50, 1: 8, 2: 33, 3: 79}
    p.reserve(list(lens), list(lens.values()))
    p.grow(list(lens), list(lens.values()))
    text = {s: torch.randn(len(layers), n, d, device=DEV).to(torch.bfloat16) for s, n in lens.items()}

    def read(s):
        n = int(p.lens[s])
        ids = p.table[s, :-(-n // ps)].long()
        return torch.stack([x[ids].reshape(-1, d)[:n] for x in layers])
    for s, n in lens.items():
        pos = torch.arange(n, device=DEV)
        for x, t in zip(layers, text[s]):
            x[p.table[s, (pos // ps)].long(), pos % ps, 0] = t
    src, dst = [0, 0, 2, 1], [5, 9, 6, 7]
    a, z = dev([0] * 4), dev([0] * 4)
    gdn.gdn_pages_fork(ps, dev(src), dev(dst), p.table, p.lens, p.refs, a, z, p.err)
    gdn.gdn_copy_rows(layers, a, z, err_flag=p.err)
    gdn.gdn_copy_rows([state], dev(src), dev(dst), err_flag=p.err)
    for x, y in zip(src, dst):
        text[y] = text[x]
        assert torch.equal(state[x], state[y])
    # a child's own tokens do not reach its parent
    last = int(p.lens[5]) - 1
    for i, x in enumerate(layers):
        x[int(p.table[5, last // ps]), last % ps, 0] += 1
    text[5] = text[5].clone()
    text[5][:, last] += 1
    for s in text:
        assert torch.equal(read(s), text[s]), s
    gone = dev([0, 3])
    gdn.gdn_pages_free(gone, p.table, p.lens, p.refs, p.err)
    P = pages
    cs, cd, n, remap = dev([0] * P), dev([0] * P), dev([0]), dev([0] * P)
    gdn.gdn_pages_compact(p.table, p.refs, cs, cd, n, remap, p.err)
    gdn.gdn_copy_rows(layers, cs, cd, n_dev=n, err_flag=p.err)
    assert int(p.err) == 0 and int(n) > 0
    live = int((p.refs > 0).sum())
    assert bool((p.refs[:live] > 0).all()) and int(p.table.max()) < live
    for s in text:
        if s not in (0, 3):
            assert torch.equal(read(s), text[s]), s


def test_reserve_more_than_can_be_counted():
    """Wishes whose sum passes 2^31 pages: the first sequences get theirs, the call is flagged."""
    n, width = 2048, (1 << 20) + 8
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(100, dtype=torch.int32, device="cuda")
    counts = torch.full((n,), width, dtype=torch.int32, device="cuda")
    counts[0] = 3
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_pages_reserve(1, torch.arange(n, dtype=torch.int32, device="cuda"), counts, table, lens, refs, err)
    assert int(err) == gdn.GDN_DEVICE_ERR_PAGE
    assert table[0, :4].tolist() == [0, 1, 2, -1] and refs[:4].tolist() == [1, 1, 1, 0] and int(refs.sum()) == 3
    assert int(table[1:, :128].max()) == -1
