"""The operators around the cache in one run, as a serving loop uses them: pages
reserved for prompts, a sequence branched, decode steps of a differential
attention layer (norm in 8 bits, projections, K/V append, paged differential
decode, head norm in 8 bits), sequences ended, the pool compacted.  Every step's
attention is held to the oracle on host copies of the same rows, and moving pages
changes no byte.
"""

import numpy as np
import pytest

import oracle
from test_gpu_diff import TOL

pytestmark = pytest.mark.gpu

P, HKV, HQ, D, WIDTH, SLOTS, MAX_PAGES, N_PAGES = 64, 4, 16, 128, 512, 8, 12, 60


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


class Server:
    def __init__(self):
        import torch
        import int8_kv_decode_gb300 as K
        g = torch.Generator(device="cuda").manual_seed(3)
        self.table = torch.full((SLOTS, MAX_PAGES), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(N_PAGES, dtype=torch.int32, device="cuda")
        self.ws = K.alloc_page_workspace(SLOTS, N_PAGES)
        self.k = torch.zeros((HKV, N_PAGES * P, D), dtype=torch.int8, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.ks = torch.zeros((HKV, N_PAGES * P), device="cuda")
        self.vs = torch.zeros_like(self.ks)
        self.w = (torch.randn((WIDTH, (HQ + 2 * HKV) * D), generator=g, device="cuda") * WIDTH ** -0.5)
        self.gain = 1 + 0.1 * torch.randn(WIDTH, generator=g, device="cuda")
        self.head_gain = 0.2 * (1 + 0.1 * torch.randn(2 * D, generator=g, device="cuda"))
        self.lam = torch.linspace(0.2, 0.8, HQ // 2, device="cuda")
        self.rows = {}                    # slot -> K and V rows appended so far (host, float32)

    def lens(self, slots):
        import torch
        return torch.tensor([len(self.rows[s][0]) for s in slots], dtype=torch.int32, device="cuda")

    def slots(self, slots):
        import torch
        return torch.tensor(slots, dtype=torch.int32, device="cuda")

    def append(self, slots, k_rows, v_rows):
        """k_rows, v_rows: per slot, [n][HKV][D] on the device."""
        import torch
        import int8_kv_decode_gb300 as K
        old = {s: len(self.rows.setdefault(s, ([], []))[0]) for s in slots}
        for s, kr, vr in zip(slots, k_rows, v_rows):
            self.rows[s][0].extend(kr.cpu().numpy())
            self.rows[s][1].extend(vr.cpu().numpy())
        K.reserve_pages(self.table, self.refs, self.slots(slots), self.lens(slots), P, workspace=self.ws)
        dst = []
        for s in slots:
            t = torch.arange(old[s], len(self.rows[s][0]), device="cuda")
            dst.append(self.table[s].long()[t // P] * P + t % P)
        dst = torch.cat(dst)
        K.quantize_kv_rows(torch.cat(list(k_rows)).contiguous(), dst, self.k, self.ks)
        K.quantize_kv_rows(torch.cat(list(v_rows)).contiguous(), dst, self.v, self.vs)

    def decode(self, slots, q):
        import int8_kv_decode_gb300 as K
        ctx = self.lens(slots)
        return K.decode_diff_paged(q, self.k, self.ks, self.v, self.vs,
                                   self.table[self.slots(slots).long()].contiguous(), P, ctx,
                                   int(ctx.max()), self.lam)

    def check(self, slots, q, out):
        """The oracle on its own contiguous caches of the slots' rows."""
        kr = np.concatenate([np.stack(self.rows[s][0]) for s in slots])
        vr = np.concatenate([np.stack(self.rows[s][1]) for s in slots])
        n = [len(self.rows[s][0]) for s in slots]
        start = np.concatenate([[0], np.cumsum(n)[:-1]])
        k8, ks = oracle.quant.quantize_kv(kr)
        v8, vs = oracle.quant.quantize_kv(vr)
        want, mass = oracle.diff.decode(q.cpu().numpy(), k8, ks, v8, vs,
                                        [a + np.arange(c) for a, c in zip(start, n)], n,
                                        self.lam.cpu().numpy())
        assert (np.abs(out.cpu().numpy() - want) <= TOL * mass).all()

    def step(self, slots, x, residual):
        """One decode step of the layer for the slots; x, residual [n][WIDTH]."""
        import torch
        import int8_kv_decode_gb300 as K
        codes, scales = K.rms_norm_quant(x, self.gain, residual=residual)
        h = (codes.float() * scales[:, None]) @ self.w
        n = len(slots)
        q = h[:, :HQ * D].reshape(n, 1, HQ, D).contiguous()
        k = h[:, HQ * D:(HQ + HKV) * D].reshape(n, 1, HKV, D)
        v = h[:, (HQ + HKV) * D:].reshape(n, 1, HKV, D)
        self.append(slots, k, v)
        out = self.decode(slots, q)
        self.check(slots, q, out)
        hc, hs = K.rms_norm_quant(out, self.head_gain, group=128)
        want, scale = oracle.norm.rms_norm_quant(out.reshape(-1, 2 * D).cpu().numpy(),
                                                 self.head_gain.cpu().numpy(), group=128)
        assert np.array_equal(hc.cpu().numpy().reshape(want.shape), want)
        assert np.allclose(hs.cpu().numpy().reshape(scale.shape), scale, rtol=1e-5)
        return out

    def books(self):
        """Counts equal the entries that name a page."""
        import int8_kv_decode_gb300 as K
        t = self.table.cpu().numpy()
        assert np.array_equal(np.bincount(t[t >= 0], minlength=N_PAGES), self.refs.cpu().numpy())
        assert K.get_device_status(self.ws) == 0


def test_a_serving_loop():
    import copy
    import torch
    import int8_kv_decode_gb300 as K
    s = Server()
    g = torch.Generator(device="cuda").manual_seed(4)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    prompts = {0: 150, 1: 63, 2: 300}
    s.append(list(prompts), [rand(n, HKV, D) for n in prompts.values()],
             [rand(n, HKV, D) for n in prompts.values()])
    s.books()
    residual = rand(5, WIDTH)
    s.step([0, 1, 2], rand(3, WIDTH), residual[:3].clone())
    # slot 0 branches twice, slot 1 (64 rows: a full page) once
    src, dst = K.fork_sequences(s.table, s.refs, s.slots([0, 0, 1]), s.slots([3, 4, 5]),
                                s.lens([0, 0, 1]), P, workspace=s.ws)
    K.copy_pages(s.k, s.ks, s.v, s.vs, src, dst, P, workspace=s.ws)
    for child, parent in ((3, 0), (4, 0), (5, 1)):
        s.rows[child] = copy.deepcopy(s.rows[parent])
    assert int(src[2]) == -1 and len({int(d) for d in dst[:2]}) == 2
    s.books()
    q = rand(5, 1, HQ, D)
    q[3] = q[4] = q[0]
    out = s.decode([0, 1, 2, 3, 4], q)    # a branch answers as its parent
    assert torch.equal(out[0], out[3]) and torch.equal(out[0], out[4])
    # the branches go their own ways, and the parents keep theirs
    for _ in range(3):
        s.step([0, 1, 2, 3, 4], rand(5, WIDTH), residual)
    s.step([5], rand(1, WIDTH), residual[:1].clone())
    s.books()
    # the long sequence ends, the pool is compacted beside the running table
    K.free_sequences(s.table, s.refs, s.slots([2, 3]), workspace=s.ws)
    s.books()
    q = rand(4, 1, HQ, D)
    before = s.decode([0, 1, 4, 5], q)
    table, refs, src, dst, counts = K.compact_pages(s.table, s.refs, workspace=s.ws)
    K.copy_pages(s.k, s.ks, s.v, s.vs, src, dst, P, count=counts[1:], workspace=s.ws)
    assert int(counts[1]) > 0
    assert torch.equal(before, s.decode([0, 1, 4, 5], q))          # the old table still answers
    s.table, s.refs = table, refs
    s.books()
    after = s.decode([0, 1, 4, 5], q)
    assert torch.equal(before, after)
    s.check([0, 1, 4, 5], q, after)
    s.step([0, 1, 4, 5], rand(4, WIDTH), residual[:4])
    s.books()
