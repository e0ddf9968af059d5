"""The page operations on the GPU against the oracle's one-by-one account: every
table, count, list and error word is equal."""

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


class Pool:
    """A table and its counts, on the host (oracle) and on the device."""

    def __init__(self, n_slots, max_pages, n_pages, page_rows, seed=0):
        import int8_kv_decode_gb300 as K
        self.r = np.random.default_rng(seed)
        self.P = page_rows
        self.table = np.full((n_slots, max_pages), -1, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        self.ws = K.alloc_page_workspace(n_slots, n_pages)
        self.sync()

    def sync(self):
        self.t, self.c = dev(self.table), dev(self.refs)

    def fill(self, share):
        """Random rows: pages in shuffled order, some shared."""
        S, mp = self.table.shape
        order = self.r.permutation(len(self.refs))[:int(len(self.refs) * share)]
        at = 0
        for s in self.r.permutation(S):
            n = int(min(self.r.integers(0, mp + 1), len(order) - at))
            self.table[s, :n] = order[at:at + n]
            at += n
            if n and s:
                self.table[s, 0] = max(self.table[s, 0], self.table[s - 1, 0])
        self.refs[:] = np.bincount(self.table[self.table >= 0], minlength=len(self.refs))
        self.sync()

    def check(self, err):
        import int8_kv_decode_gb300 as K
        assert np.array_equal(self.t.cpu().numpy(), self.table)
        assert np.array_equal(self.c.cpu().numpy(), self.refs)
        assert K.get_device_status(self.ws) == err
        # claims and marks are back to zero for the next call
        assert int(self.ws[256:256 + 2 * (-(-4 * len(self.table) // 256) * 256)].max()) == 0

    def reserve(self, seqs, lens):
        import int8_kv_decode_gb300 as K
        K.reserve_pages(self.t, self.c, dev(seqs), dev(lens), self.P, workspace=self.ws)
        self.check(oracle.pages.reserve(self.table, self.refs, seqs, lens, self.P))

    def free(self, seqs):
        import int8_kv_decode_gb300 as K
        K.free_sequences(self.t, self.c, dev(seqs), workspace=self.ws)
        self.check(oracle.pages.free(self.table, self.refs, seqs))

    def fork(self, parents, children, lens):
        import int8_kv_decode_gb300 as K
        src, dst = K.fork_sequences(self.t, self.c, dev(parents), dev(children), dev(lens), self.P,
                                    workspace=self.ws)
        err, s, d = oracle.pages.fork(self.table, self.refs, parents, children, lens, self.P)
        assert np.array_equal(src.cpu().numpy(), s) and np.array_equal(dst.cpu().numpy(), d)
        self.check(err)
        return src, dst

    def compact(self, in_place):
        import int8_kv_decode_gb300 as K
        kw = dict(table_out=self.t, ref_out=self.c) if in_place else {}
        t, c, src, dst, counts = K.compact_pages(self.t, self.c, workspace=self.ws, **kw)
        err, table, refs, s, d, n = oracle.pages.compact(self.table, self.refs)
        assert np.array_equal(src.cpu().numpy(), s) and np.array_equal(dst.cpu().numpy(), d)
        assert np.array_equal(counts.cpu().numpy(), n)
        if not in_place:                  # the inputs stay as they were
            assert np.array_equal(self.t.cpu().numpy(), self.table)
            assert np.array_equal(self.c.cpu().numpy(), self.refs)
        self.t, self.c, self.table, self.refs = t, c, table, refs
        self.check(err)
        return src, dst, counts


@pytest.mark.parametrize("S,mp,n", [(1, 1, 1), (3, 2, 5), (7, 5, 40), (64, 33, 1000), (300, 40, 8192),
                                    (1500, 70, 70001)])
def test_reserve_free_and_compact(S, mp, n):
    p = Pool(S, mp, n, 32, seed=S)
    r = p.r
    p.fill(0.4)
    for _ in range(3):
        m = int(r.integers(1, S + 1))
        seqs = r.permutation(S)[:m]
        p.reserve(seqs, r.integers(0, mp * 32 + 1, m))       # may or may not fit the pool
        p.free(r.permutation(S)[:max(1, S // 3)])
        p.reserve(seqs[:1], [min(mp, 1) * 32])
        p.compact(in_place=bool(r.integers(2)))


@pytest.mark.parametrize("S,mp,n,m", [(2, 1, 3, 1), (8, 4, 64, 3), (100, 20, 3000, 40),
                                      (1200, 30, 40000, 500)])
def test_fork(S, mp, n, m):
    p = Pool(S, mp, n, 64, seed=n)
    p.fill(0.5)
    r = p.r
    for _ in range(3):
        slots = r.permutation(S)
        children, parents = slots[:m], slots[m:][r.integers(0, S - m, m)]
        held = (p.table[parents] >= 0).sum(1)
        lens = np.maximum(0, held * 64 - r.integers(0, 64, m))
        lens[r.random(m) < 0.2] //= 2                        # a branch from further back
        lens[r.random(m) < 0.2] = 0
        p.fork(parents, children, lens)
        p.free(r.permutation(S)[:S // 4])


def test_fork_children_reuse_what_the_call_released():
    # the pool is full but for what the children hold
    p = Pool(4, 2, 4, 32)
    p.reserve([0, 1], [64, 64])
    p.fork([0], [1], [40])                # child 1 gives its two pages back and takes one
    assert p.refs.tolist() == [2, 1, 1, 0]
    p.fork([0], [1], [40])                # and again: the same result
    assert p.refs.tolist() == [2, 1, 1, 0]


def test_pool_without_room():
    p = Pool(6, 4, 10, 32)
    p.reserve([0, 1], [128, 128])
    p.reserve([2, 3], [32, 64])           # 3 wanted, 2 left: nothing is given
    p.reserve([2], [64])
    p.reserve([4], [1])                   # none left
    p.reserve([4, 0], [0, 100])           # nothing wanted
    p.free([2])
    p.fork([0, 0, 1, 1], [2, 3, 4, 5], [33, 34, 64, 1])      # two tails fit, the third does not


def test_lists_that_break_the_rules():
    p = Pool(8, 4, 40, 32)
    p.reserve([0, 1, 2, 3], [100, 32, 64, 128])
    p.reserve([4, 4, -1, 8, 5, 6], [32, 64, 32, 32, -5, 129])   # twice, outside, bad lengths
    p.free([2, 2, 9, -3])
    p.fork([0, 1, 0, 2, 0, 3, -2, 0], [5, 5, 1, 6, 0, 7, 6, 8], [10, 10, 10, 10, 10, 129, 1, 1])
    p.fork([1], [6], [33])                # more rows than the parent holds
    p.fork([0, 3], [4, 0], [5, 5])        # child 0 is a parent of the call


@pytest.mark.parametrize("m", [64, 65, 1024, 1025, 2100])
def test_long_lists_that_break_the_rules(m):
    # slots named again near and far, slots outside, children that are parents of the
    # call: lists on both sides of each of the plan's limits
    p = Pool(2100, 6, 30000, 32, seed=m)
    p.fill(0.3)
    r = p.r
    for _ in range(2):
        seqs = r.permutation(2100)[:m]
        again = r.integers(1, m, m // 8)
        seqs[again] = seqs[r.integers(0, again)]
        seqs[r.integers(0, m, 3)] = [-1, 2100, 2**31 - 1]
        seqs[-1] = seqs[0]
        lens = r.integers(0, 6 * 32 + 1, m) // 4
        lens[r.integers(0, m, 2)] = [-1, 6 * 32 + 1]
        p.reserve(seqs, lens)
        slots = r.permutation(2100)
        children, parents = slots[:m], slots[-(m // 2 + 1):][r.integers(0, m // 2 + 1, m)]
        children[-1], parents[0] = children[0], children[m // 3]
        parents[m // 2] = -7
        held = (p.table[np.clip(parents, 0, 2099)] >= 0).sum(1)
        p.fork(parents, children, np.maximum(0, held * 32 - r.integers(0, 32, m)))
        p.free(seqs[:m // 2])


def test_damaged_tables_stay_inside_the_pool():
    p = Pool(6, 3, 12, 32)
    p.reserve([0, 1, 2], [96, 64, 32])
    p.table[1, 0] = 99
    p.table[2, 1] = 11                    # names a free page
    p.table[3] = [-5, -1, 12]
    p.sync()
    p.fork([1], [4], [40])                # an entry outside the pool
    p.compact(in_place=False)
    p.free([1, 2, 3])
    p.fork([0], [5], [90])


def test_compaction_extremes():
    for n, live in ((5, []), (5, [0, 1, 2, 3, 4]), (5, [4]), (6, [3, 4, 5]), (9000, [8999]),
                    (9000, list(range(4500, 9000)))):
        p = Pool(3, 4500, n, 32)
        p.table[1, :len(live)] = live
        p.refs[live] = 1
        p.sync()
        p.compact(in_place=True)
        assert sorted(p.table[1, :len(live)].tolist()) == list(range(len(live)))


@pytest.mark.parametrize("Hkv,P,n,m", [(1, 32, 3, 1), (2, 32, 50, 20), (3, 64, 200, 99), (4, 128, 40, 7),
                                       (8, 256, 24, 12), (2, 1024, 8, 3)])
def test_copy_pages(Hkv, P, n, m):
    import torch
    import int8_kv_decode_gb300 as K
    r = np.random.default_rng(n)
    k = torch.randint(-127, 128, (Hkv, n * P, 128), dtype=torch.int8, device="cuda")
    v = torch.randint(-127, 128, (Hkv, n * P, 128), dtype=torch.int8, device="cuda")
    ks, vs = torch.rand((Hkv, n * P), device="cuda"), torch.rand((Hkv, n * P), device="cuda")
    pages = r.permutation(n)
    dst = pages[:m].copy()
    src = pages[m:][r.integers(0, n - m, m)]
    for count in (None, 0, m // 2, m + 5, -1):
        s, d = src.copy(), dst.copy()
        s[::4], d[2::5] = -1, -1
        ws = K.alloc_page_workspace(1, n)
        want = [t.clone() for t in (k, ks, v, vs)]
        take = m if count is None else max(0, min(m, count))
        for a, b in list(zip(s, d))[:take]:
            if a >= 0 and b >= 0:
                for t in want:
                    t[:, b * P:(b + 1) * P] = t[:, a * P:(a + 1) * P]
        K.copy_pages(k, ks, v, vs, dev(s), dev(d), P, workspace=ws,
                     count=None if count is None else dev([count]))
        for got, w in zip((k, ks, v, vs), want):
            assert torch.equal(got, w)
        assert K.get_device_status(ws) == 0
    ws = K.alloc_page_workspace(1, n)
    before = [t.clone() for t in (k, ks, v, vs)]
    K.copy_pages(k, ks, v, vs, dev([n, 0]), dev([0, n + 3]), P, workspace=ws)
    assert K.get_device_status(ws) == K.DEVERR_BAD_PAGE
    assert all(torch.equal(a, b) for a, b in zip(before, (k, ks, v, vs)))


def test_compaction_moves_the_rows_of_every_sequence():
    import torch
    import int8_kv_decode_gb300 as K
    p = Pool(40, 9, 500, 32, seed=2)
    p.fill(0.5)
    p.free(list(range(0, 40, 3)))
    k = torch.randint(-127, 128, (2, 500 * 32, 128), dtype=torch.int8, device="cuda")
    v, ks = k.flip(1).contiguous(), torch.rand((2, 500 * 32), device="cuda")
    vs = ks.flip(1).contiguous()
    old = p.table.copy()
    rows = [k.view(2, 500, -1)[:, e].clone() for e in old[old >= 0]]
    scales = [vs.view(2, 500, -1)[:, e].clone() for e in old[old >= 0]]
    src, dst, counts = p.compact(in_place=False)
    K.copy_pages(k, ks, v, vs, src, dst, 32, count=counts[1:], workspace=p.ws)
    for e, a, b in zip(p.table[old >= 0], rows, scales):
        assert torch.equal(k.view(2, 500, -1)[:, e], a) and torch.equal(vs.view(2, 500, -1)[:, e], b)
    assert p.table.max() < int(counts[0])
    assert not p.refs[int(counts[0]):].any()


@pytest.mark.parametrize("n_pages", [100, 20000])
def test_graph_replay_of_a_turnover(n_pages):
    # free and reserve captured once and replayed: every replay frees what the one
    # before gave and takes the same pages again (one block, and a cluster)
    import torch
    import int8_kv_decode_gb300 as K
    p = Pool(16, 8, n_pages, 32, seed=5)
    p.reserve(list(range(8)), [100] * 8)
    seqs, lens = dev([1, 3, 5, 9]), dev([200, 31, 64, 1])
    K.free_sequences(p.t, p.c, seqs, workspace=p.ws)         # warm-up outside the capture
    K.reserve_pages(p.t, p.c, seqs, lens, 32, workspace=p.ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.free_sequences(p.t, p.c, seqs, workspace=p.ws)
        K.reserve_pages(p.t, p.c, seqs, lens, 32, workspace=p.ws)
    for _ in range(3):
        oracle.pages.free(p.table, p.refs, [1, 3, 5, 9])
        oracle.pages.reserve(p.table, p.refs, [1, 3, 5, 9], [200, 31, 64, 1], 32)
        g.replay()
        p.check(0)


def test_unaligned_arrays():
    # tables and counts need no more than their element's alignment
    import torch
    import int8_kv_decode_gb300 as K
    buf = torch.zeros(1 + 6 * 5, dtype=torch.int32, device="cuda")
    table = buf[1:].view(6, 5)
    table.fill_(-1)
    refs = torch.zeros(42, dtype=torch.int32, device="cuda")[1:]
    host, counts = np.full((6, 5), -1, np.int32), np.zeros(41, np.int32)
    ws = K.alloc_page_workspace(6, 41)
    K.reserve_pages(table, refs, dev([0, 2, 5]), dev([160, 33, 64]), 32, workspace=ws)
    assert oracle.pages.reserve(host, counts, [0, 2, 5], [160, 33, 64], 32) == 0
    K.free_sequences(table, refs, dev([2]), workspace=ws)
    oracle.pages.free(host, counts, [2])
    out = K.compact_pages(table, refs, workspace=ws)
    want = oracle.pages.compact(host, counts)
    for a, b in zip(out, want[1:]):
        assert np.array_equal(a.cpu().numpy(), b)
    assert K.get_device_status(ws) == 0


@pytest.mark.parametrize("n_pages", [12, 6000])
@pytest.mark.parametrize("in_place", [False, True])
def test_compaction_flags_entries_that_name_a_free_page(n_pages, in_place):
    # a damaged row names a page of count 0 below the live count: another sequence's page
    # moves there, so the row would answer with that sequence's keys
    p = Pool(6, 3, n_pages, 32)
    p.reserve([0, 1, 2], [96, 64, 32])
    p.free([0])                           # pages 0, 1, 2 are free, 3, 4, 5 move there
    p.compact(in_place=False)
    p.reserve([0], [96])
    p.free([1])                           # live: 2 (slot 2), 3, 4, 5 (slot 0); free: 0, 1
    p.table[4] = [-1, 1, 4]               # a free page, and one of slot 0's
    p.sync()
    p.compact(in_place)
    assert p.table[4, 1] == 1             # kept, and flagged


@pytest.mark.parametrize("n_pages", [12, 20000])
def test_reserve_flags_entries_outside_the_pool(n_pages):
    p = Pool(4, 300, n_pages, 32)
    p.reserve([0, 1], [64, 32])
    p.table[0, 1] = n_pages
    p.table[2, 0] = 2**31 - 1
    p.sync()
    p.reserve([1], [64])                  # other rows
    p.reserve([0], [32])                  # the entry lies past what the length needs
    p.reserve([0, 3], [96, 32])           # flagged; the others of the row get theirs
    p.reserve([2], [64])
