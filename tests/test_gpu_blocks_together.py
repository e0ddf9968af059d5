"""The operators of a block-scaled cache in one run, as a serving loop uses them: pages
reserved, ragged prompts written with their rotation, decode steps (norm in 8 bits, a
projection, rows written and queries turned in one call, attention), draft columns that
are partly taken back, a branch with its page copies, a prefix read back, sequences
ended, the pool compacted.  Every attention is held to the oracle, whose cache takes the
same rows in the same order, and moving pages changes no byte.
"""

import numpy as np
import pytest

import oracle
from test_gpu_blocks import Cache, check_attend, i32, same, torch_angles

pytestmark = pytest.mark.gpu

P, HKV, HQ, D, WIDTH, SLOTS, MAX_PAGES, N_PAGES, ROT = 64, 2, 8, 128, 256, 6, 12, 48, 64


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


class Server:
    def __init__(self, code, R):
        import torch
        import int8_kv_decode_gb300 as K
        self.g = torch.Generator(device="cuda").manual_seed(3)
        self.c = Cache(HKV, N_PAGES, P, R, code)
        self.table = torch.full((SLOTS, MAX_PAGES), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(N_PAGES, dtype=torch.int32, device="cuda")
        self.ws = K.alloc_page_workspace(SLOTS, N_PAGES)
        self.angles = torch_angles(MAX_PAGES * P, ROT)
        self.w = torch.randn((WIDTH, (HQ + 2 * HKV) * D), generator=self.g, device="cuda") * WIDTH ** -0.5
        self.gain = 1 + 0.1 * torch.randn(WIDTH, generator=self.g, device="cuda")
        self.held = {}                        # slot -> rows

    def rand(self, *shape):
        import torch
        return torch.randn(shape, generator=self.g, device="cuda")

    def project(self, x):
        """The fused projection of the 8-bit norm of x, as rows of bf16 heads."""
        import int8_kv_decode_gb300 as K
        codes, scales = K.rms_norm_quant(x, self.gain)
        return ((codes.float() * scales[:, None]) @ self.w).bfloat16().view(len(x), HQ + 2 * HKV, D)

    def write(self, slots, lens, x):
        """Rows of the slots into the cache; the turned queries."""
        import torch
        import int8_kv_decode_gb300 as K
        ends = [self.held.get(s, 0) + n for s, n in zip(slots, lens)]
        K.reserve_pages(self.table, self.refs, i32(slots), i32(ends), P, workspace=self.ws)
        start = [self.held.get(s, 0) for s in slots]
        cu = np.concatenate([[0], np.cumsum(lens)])
        y = self.project(x)
        table = self.table[torch.tensor(slots, device="cuda")].contiguous()
        q = K.append_blocks(y[:, HQ:HQ + HKV], y[:, HQ + HKV:], i32(cu), i32(start), *self.c.args, table, P,
                            table=self.angles, q=y[:, :HQ], workspace=self.c.ws)
        assert K.get_device_status(self.c.ws) == 0 and K.get_device_status(self.ws) == 0
        host, th, ang = y.float().cpu().numpy(), table.cpu().numpy(), self.angles.cpu().numpy()
        for i, s in enumerate(slots):
            rows = host[cu[i]:cu[i + 1]]
            pos = np.arange(start[i], ends[i])
            k = oracle.blocks.rotate(rows[:, HQ:HQ + HKV], ang[pos], False)
            oracle.blocks.append(self.c.host, "k", k, start[i], th[i], P)
            oracle.blocks.append(self.c.host, "v", rows[:, HQ + HKV:], start[i], th[i], P)
            self.held[s] = ends[i]
        return q

    def attend(self, slots, q, M=1, check=True):
        """Column 0 of each slot sees its rows but the last M - 1."""
        import torch
        import int8_kv_decode_gb300 as K
        table = self.table[torch.tensor(slots, device="cuda")].contiguous()
        ctx = np.array([self.held[s] - M + 1 for s in slots])
        out = K.decode_blocks(q.view(len(slots), M, HQ, D), *self.c.args, table, P, i32(ctx), int(ctx.max()))
        if check:
            check_attend(self.c, table.cpu().numpy(), ctx, q.view(len(slots), M, HQ, D), out)
        return out

    def books(self):
        import int8_kv_decode_gb300 as K
        t = self.table.cpu().numpy()
        assert np.array_equal(np.bincount(t[t >= 0], minlength=N_PAGES), self.refs.cpu().numpy())
        assert K.get_device_status(self.ws) == 0
        self.c.check()


@pytest.mark.parametrize("code,R", [("int8", 32), ("e4m3", 64)])
def test_a_serving_loop(code, R):
    import torch
    import int8_kv_decode_gb300 as K
    s = Server(code, R)
    lens = [150, 1, 63, 200]
    q = s.write([0, 1, 2, 3], lens, s.rand(sum(lens), WIDTH))
    last = np.cumsum(lens) - 1
    s.attend([0, 1, 2, 3], q[torch.from_numpy(last).cuda()].contiguous())
    s.books()
    for _ in range(3):                        # decode steps
        s.attend([0, 1, 2, 3], s.write([0, 1, 2, 3], [1] * 4, s.rand(4, WIDTH)))
    # drafts: four columns, then all but the first of each are taken back and written again
    s.attend([0, 2], s.write([0, 2], [4, 4], s.rand(8, WIDTH)), M=4)
    for slot in (0, 2):
        s.held[slot] -= 3
    s.attend([0, 2], s.write([0, 2], [1, 1], s.rand(2, WIDTH)))
    s.books()
    # slot 0 branches twice, slot 2 once
    ends = [s.held[p] for p in (0, 0, 2)]
    src, dst = K.fork_sequences(s.table, s.refs, i32([0, 0, 2]), i32([4, 5, 1]), i32(ends), P, workspace=s.ws)
    K.copy_pages(*s.c.args, src, dst, P, workspace=s.c.ws)
    for a, b in zip(src.tolist(), dst.tolist()):
        if a >= 0:
            per = P // R
            for n in ("k", "v"):
                s.c.host[n][:, b * P:(b + 1) * P] = s.c.host[n][:, a * P:(a + 1) * P]
                s.c.host[n + "s"][:, b * per:(b + 1) * per] = s.c.host[n + "s"][:, a * per:(a + 1) * per]
    s.held.update({4: ends[0], 5: ends[1], 1: ends[2]})
    s.books()
    q = s.rand(6, 1, HQ, D).bfloat16()
    q[4] = q[5] = q[0]
    q[1] = q[2]
    out = s.attend([0, 1, 2, 3, 4, 5], q)
    assert same(out[0], out[4]) and same(out[0], out[5]) and same(out[1], out[2])
    for _ in range(2):                        # the branches go their own ways
        s.attend([0, 1, 2, 4, 5], s.write([0, 1, 2, 4, 5], [1] * 5, s.rand(5, WIDTH)))
    s.books()
    # a prefix read back: the values that attention sees
    n = s.held[3]
    k, v = K.read_blocks(*s.c.args, s.table[3:4].contiguous(), P, i32([0, n]), i32([0]), n, dtype=torch.float32)
    rows = oracle.blocks.rows_of(s.table[3].cpu().numpy(), P, np.arange(n))
    for got, name in ((k, "k"), (v, "v")):
        want = oracle.blocks.values(s.c.host, name, rows).transpose(1, 0, 2)
        assert (np.abs(got.cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want)).all()
    # sequences end, the pool is compacted beside the running table
    K.free_sequences(s.table, s.refs, i32([3, 4]), workspace=s.ws)
    q = s.rand(4, 1, HQ, D).bfloat16()
    before = s.attend([0, 1, 2, 5], q)
    table, refs, src, dst, counts = K.compact_pages(s.table, s.refs, workspace=s.ws)
    K.copy_pages(*s.c.args, src, dst, P, count=counts[1:], workspace=s.c.ws)
    assert int(counts[1]) > 0
    assert same(before, s.attend([0, 1, 2, 5], q, check=False))    # the old table still answers
    s.table, s.refs = table, refs
    assert same(before, s.attend([0, 1, 2, 5], q, check=False))
