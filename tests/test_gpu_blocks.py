"""Rotary positions and the block-scaled cache on the GPU against the oracle.

rope, append_blocks and read_blocks are defined by float32 operations that are each
rounded once, so their results are held to the oracle's bits.

decode_blocks, per channel: |error| <= tol * mass + tail + half a step of the output's
type, with mass = sum w |V|.  A weight's relative error, and that of the row sum, is at
most e, so the quotient's is 2 e, where e adds up
  * the score S c: products exact, 8 tensor-core additions of 16 channels, each off by up
    to 2^-22 of sum |q K| (float32 queries: twice as many, and their elements held to
    2^-22), three roundings of c, one of S c - m: (8 + 4) 2^-22 of the size, or (16 + 1 +
    4) 2^-22; a base-2 exponent, so times log2(e) ln(2) = 1;
  * the rounding of an exponent up to 16 away from the reference, and 2 ulp of the
    exponential: 2^-20 + 2^-22 (further weights are below 2^-16 of the largest, and an
    exponent of size 2^k rounds to 2^(k - 24) while the weight falls by 2^(2^k));
  * the weight's own rounding: 2^-11, for float32 queries 2^-22;
  * sums: 2 tensor-core additions a step (2^-21), 8 steps of a window, 64 + 8 windows'
    additions for up to 512 windows and 8 roundings besides, 2^-24 each: below 2^-17.
tail: a weight below 2^-14 is held to 2^-25, where the row's largest is 2^9 or more: up to
2^-34 of the largest value for each key, once in the sum over V and once in the row sum.
"""

import numpy as np
import pytest

import oracle

D = 128
HALF_STEP = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


gpu = pytest.mark.gpu


def dtype_of(name):
    import torch
    return getattr(torch, name)


def bits(t):
    t = t.detach().cpu().contiguous()
    import torch
    return t.view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()]).numpy()


def same(a, b):
    return np.array_equal(bits(a), bits(b))


# ------------------------------------------------------------------- rope

def torch_angles(n, rot, base=10000.0):
    import torch
    import int8_kv_decode_gb300 as K
    return torch.from_numpy(oracle.blocks.angles(K.rope_frequencies(rot, base), np.arange(n))).cuda()


@gpu
@pytest.mark.parametrize("rot", [8, 64, 96, 128])
def test_rope_table(rot):
    # the angles and functions are float64: what is left is one rounding to float32 of a
    # cosine or sine that float64 gives to 2^-52, and the oracle's own
    import int8_kv_decode_gb300 as K
    got = K.rope_table(5000, rot, base=500000.0).cpu().numpy()
    want = oracle.blocks.angles(K.rope_frequencies(rot, 500000.0), np.arange(5000))
    assert got.shape == want.shape == (5000, rot // 2, 2)
    assert (np.abs(got.astype(np.float64) - want) <= 2.0 ** -24 + 1e-9).all()
    # far positions, one at a time through scaled frequencies
    far = K.rope_table(2, rot, frequencies=[w * 1e6 for w in K.rope_frequencies(rot)]).cpu().numpy()
    want = oracle.blocks.angles([w * 1e6 for w in K.rope_frequencies(rot)], [0, 1])
    assert (np.abs(far.astype(np.float64) - want) <= 2.0 ** -24 + 1e-9).all()


@gpu
@pytest.mark.parametrize("dtype,out", [("float32", "float32"), ("bfloat16", "bfloat16"), ("float16", "float16"),
                                       ("bfloat16", "float32"), ("float16", "float32")])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (96, True), (96, False),
                                             (8, False), (8, True)])
def test_rope_matches_the_oracle(dtype, out, rot, interleaved):
    import torch
    import int8_kv_decode_gb300 as K
    table = torch_angles(300, rot)
    g = torch.Generator(device="cuda").manual_seed(rot)
    for rows, heads in ((1, 1), (3, 4), (37, 5), (64, 9)):
        wide = torch.randn((rows, heads + 3, D), generator=g, device="cuda").to(dtype_of(dtype))
        x = wide[:, 1:1 + heads]                             # among other heads
        pos = torch.randint(0, 300, (rows,), generator=g, device="cuda", dtype=torch.int32)
        pos[0] = 299
        got = K.rope(x, pos, table, interleaved=interleaved, out_dtype=dtype_of(out))
        want = oracle.blocks.rotate(x.float().cpu().numpy(), table.cpu().numpy()[pos.cpu().numpy()], interleaved)
        assert same(got, torch.from_numpy(want).to(dtype_of(out)))


@gpu
def test_rope_in_place_padding_and_positions_past_the_table():
    import torch
    import int8_kv_decode_gb300 as K
    table = torch_angles(50, 64)
    x = torch.randn((6, 3, D), device="cuda")
    want = K.rope(x, torch.tensor([4, 49, 0, 7, 8, 9], dtype=torch.int32, device="cuda"), table)
    pos = torch.tensor([4, 49, -1, 50, 8, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    y = x.clone()
    assert K.rope(y, pos, table, out=y) is y
    assert same(y[[0, 1, 4]], want[[0, 1, 4]])
    assert same(y[2], x[2])                                  # padding: as it was
    assert torch.isnan(y[3]).all() and torch.isnan(y[5]).all()
    assert K.rope(x[:0], pos[:0], table).shape == (0, 3, D)
    # a slice of one row, in place
    z = torch.randn((6, 5, D), device="cuda")
    w = K.rope(z[2:3, 1:4], pos[:1], table)
    K.rope(z[2:3, 1:4], pos[:1], table, out=z[2:3, 1:4])
    assert same(z[2:3, 1:4], w)


# ------------------------------------------------------- write and read back

class Cache:
    """A paged block-scaled cache on the device with the oracle's beside it."""

    def __init__(self, Hkv, pages, page, R, code, seed=0):
        import torch
        self.Hkv, self.page, self.R, self.e4m3, self.n_pages = Hkv, page, R, code == "e4m3", pages
        self.type = torch.float8_e4m3fn if self.e4m3 else torch.int8
        r = np.random.default_rng(seed)
        cap = pages * page
        self.host = {"R": R, "e4m3": self.e4m3}
        for n in ("k", "v"):
            x = r.standard_normal((Hkv, cap, D)).astype(np.float32)
            c = oracle.blocks.round_codes(x * np.float32(100 if self.e4m3 else 30), self.e4m3)
            self.host[n] = c
            self.host[n + "s"] = (r.uniform(0.5, 1.5, (Hkv, cap // R)) / (100 if self.e4m3 else 30)).astype(np.float32)
            setattr(self, n, torch.from_numpy(c.astype(np.float32)).cuda().to(self.type))
            setattr(self, n + "s", torch.from_numpy(self.host[n + "s"].copy()).cuda())
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    @property
    def args(self):
        return self.k, self.ks, self.v, self.vs

    def check(self):
        import torch
        for n in ("k", "v"):
            got = getattr(self, n).float().cpu().numpy()
            assert np.array_equal(got, self.host[n].astype(np.float32)), n
            assert same(getattr(self, n + "s"), torch.from_numpy(self.host[n + "s"])), n


def tables(lens, page, n_pages, seed=0, spare=1):
    """Shuffled pages for `lens` keys of each sequence; -1 past them."""
    r = np.random.default_rng(seed)
    need = [-(-int(n) // page) for n in lens]
    t = np.full((len(lens), max(need + [1]) + spare), -1, np.int32)
    order = r.permutation(n_pages)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    assert at <= n_pages
    return t


def i32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def append(c, table, start, lens, seed, dtype="float32", rot=None, interleaved=False, Hq=0, gain=1.0):
    """One call on the device and on the oracle's cache; returns (q_out, oracle's)."""
    import torch
    import int8_kv_decode_gb300 as K
    r = np.random.default_rng(seed)
    T = int(sum(lens))
    wide = torch.from_numpy(r.standard_normal((T, Hq + 2 * c.Hkv, D)).astype(np.float32) * np.float32(gain))
    wide = wide.cuda().to(dtype_of(dtype))
    q, kn, vn = wide[:, :Hq], wide[:, Hq:Hq + c.Hkv], wide[:, Hq + c.Hkv:]
    cu = np.concatenate([[0], np.cumsum(lens)])
    ang = torch_angles(int(max(s + n for s, n in zip(start, lens))), rot) if rot else None
    got = K.append_blocks(kn, vn, i32(cu), i32(start), *c.args, i32(table), c.page, table=ang,
                          interleaved=interleaved, q=q if Hq else None, workspace=c.ws)
    assert K.get_device_status(c.ws) == 0
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(start, lens)]).astype(np.int64)
    turn = (lambda x: oracle.blocks.rotate(x, ang.cpu().numpy()[pos], interleaved)) if rot else (lambda x: x)
    kh, vh = turn(kn.float().cpu().numpy()), vn.float().cpu().numpy()
    for b, n in enumerate(lens):
        if n:
            for name, x in (("k", kh), ("v", vh)):
                oracle.blocks.append(c.host, name, x[cu[b]:cu[b + 1]], int(start[b]), table[b], c.page)
    if Hq:
        assert same(got, torch.from_numpy(turn(q.float().cpu().numpy())).to(dtype_of(dtype)))
    return cu


@gpu
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("R,page", [(32, 32), (32, 128), (64, 64), (128, 256)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_append_matches_the_oracle(code, R, page, dtype):
    # lengths and starts around the blocks' edges, an empty sequence, spans over many blocks
    lens = [1, 0, R, R - 1, R + 1, 3 * R + 5, 2, 7]
    start = [0, 5, 0, 1, R - 1, R // 2, 2 * R - 1, 3 * R + 3]
    ends = [s + n for s, n in zip(start, lens)]
    c = Cache(3, sum(-(-e // page) for e in ends) + 2, page, R, code, seed=R)
    table = tables(ends, page, c.n_pages, seed=1)
    append(c, table, start, lens, seed=2, dtype=dtype, rot=128, Hq=6)
    c.check()
    # and again behind them: larger rows (the kept ones are coded again), then smaller ones
    ends2 = [e + 5 for e in ends]
    table2 = tables(ends2, page, 64 + c.n_pages, seed=1)
    table2[:, :table.shape[1]] = np.where(table >= 0, table, -1)
    fresh = [p for p in range(c.n_pages) if p not in set(table[table >= 0])]
    lens2 = []
    for b, (e, e2) in enumerate(zip(ends, ends2)):
        lens2.append(5 if -(-e2 // page) == -(-e // page) else 0)
        table2[b, -(-e // page):] = -1
    assert fresh and sum(lens2) > 0
    for gain in (8.0, 0.01):
        append(c, table2, ends, lens2, seed=3, dtype=dtype, rot=64, interleaved=True, gain=gain)
        c.check()


@gpu
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_one_row_at_a_time(code):
    # a block filled by single rows of growing and falling size, twice over
    R = 32
    c = Cache(2, 4, 64, R, code)
    table = tables([100, 60], 64, 4)
    for t in range(70):
        lens = [1, 1 if t < 60 else 0]
        append(c, table, [t, t], lens, seed=t, gain=float(2.0 ** ((t * 7) % 11 - 5)), rot=32)
    c.check()


@gpu
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_zero_rows_equal_rows_and_extremes(code):
    import torch
    import int8_kv_decode_gb300 as K
    R = 32
    c = Cache(1, 4, 32, R, code)
    table = tables([96], 32, 4)
    x = np.zeros((64, 1, D), np.float32)
    x[5, 0, 3], x[6, 0, 4] = 1e-38, -3e38                    # scale spans float32
    x[40] = 2.5                                              # ties: codes exact
    for name in ("k", "v"):
        oracle.blocks.append(c.host, name, x, 0, table[0], 32)
    t = torch.from_numpy(x).cuda()
    K.append_blocks(t, t, i32([0, 64]), i32([0]), *c.args, i32(table), 32)
    c.check()
    # a block of zeros alone: scale 0, codes 0; then a row beside them
    z = np.zeros((20, 1, D), np.float32)
    one = np.full((1, 1, D), -0.75, np.float32)
    for start, rows in ((64, z), (84, one)):
        for name in ("k", "v"):
            oracle.blocks.append(c.host, name, rows, start, table[0], 32)
        t = torch.from_numpy(rows).cuda()
        K.append_blocks(t, t, i32([0, len(rows)]), i32([start]), *c.args, i32(table), 32)
        c.check()


@gpu
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("R,page", [(32, 64), (128, 128)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_read_back(code, R, page, dtype):
    import torch
    import int8_kv_decode_gb300 as K
    lens, start = [1, 0, 33, 200, 5, 64, 1, 1], [0, 3, 31, 17, 127, 64, 300, 5]
    ends = [s + n for s, n in zip(start, lens)]
    c = Cache(3, sum(-(-e // page) for e in ends) + 1, page, R, code)
    table = tables(ends, page, c.n_pages, seed=4)
    cu = np.concatenate([[0], np.cumsum(lens)])
    n = int(cu[-1]) + 9                                      # rows behind the last sequence
    out = [torch.full((n, 3, D), 7.0, device="cuda", dtype=dtype_of(dtype)) for _ in "kv"]
    got = K.read_blocks(*c.args, i32(table), page, i32(cu), i32(start), n, out_k=out[0], out_v=out[1],
                        workspace=c.ws)
    assert K.get_device_status(c.ws) == 0
    rows = np.concatenate([oracle.blocks.rows_of(table[b], page, np.arange(start[b], ends[b]))
                           for b in range(len(lens))])
    for name, y in zip("kv", got):
        # code * scale in float32, rounded once more to the type
        want = (c.host[name][:, rows].astype(np.float32)
                * c.host[name + "s"][:, rows // R][..., None]).astype(np.float32).transpose(1, 0, 2)
        assert same(y[:len(rows)], torch.from_numpy(want.copy()).to(dtype_of(dtype)))
        assert (y[len(rows):] == 7.0).all()


@gpu
def test_many_short_sequences():
    # more sequences than a warp's search sees in two steps, several of them empty
    import int8_kv_decode_gb300 as K
    r = np.random.default_rng(0)
    B, R = 1500, 32
    lens = r.integers(0, 4, B)
    start = r.integers(0, 60, B)
    c = Cache(1, 2 * B, 32, R, "int8")
    table = tables([64] * B, 32, 2 * B, spare=0)
    cu = append(c, table, start, lens, seed=1, rot=128, Hq=1)
    c.check()
    k, _ = K.read_blocks(*c.args, i32(table), 32, i32(cu), i32(start), int(cu[-1]), workspace=c.ws)
    rows = np.concatenate([oracle.blocks.rows_of(table[b], 32, np.arange(start[b], start[b] + lens[b]))
                           for b in range(B)])
    want = oracle.blocks.values(c.host, "k", rows).transpose(1, 0, 2)
    err = np.abs(k.float().cpu().numpy() - want)
    assert (err <= 2.0 ** -8 * 1.001 * np.abs(want)).all()


@gpu
def test_bad_spans_and_pages_are_skipped():
    import torch
    import int8_kv_decode_gb300 as K
    c = Cache(2, 8, 32, 32, "int8")
    table = tables([64, 64, 64], 32, 8, spare=0)
    before = [t.clone() for t in c.args]
    x = torch.randn((30, 2, D), device="cuda")
    ang = torch_angles(40, 128)
    q = torch.randn((30, 1, D), device="cuda")

    def run(cu, start, tab, **kw):
        for t, b in zip(c.args, before):
            t.copy_(b)
        out = torch.full_like(q, 7.0)
        K.append_blocks(x, x, i32(cu), i32(start), *c.args, i32(tab), 32, table=ang, q=q, q_out=out,
                        workspace=c.ws, **kw)
        back = torch.full((30, 2, D), 7.0, device="cuda")
        K.read_blocks(*c.args, i32(tab), 32, i32(cu), i32(start), 30, out_k=back, out_v=back.clone(),
                      workspace=c.ws)
        return out, back, K.get_device_status(c.ws)

    good, _, st = run([0, 10, 20, 30], [0, 0, 0], table)
    assert st == 0
    for cu, start in (([0, 10, 20, 30], [0, -1, 0]),         # a negative start
                      ([0, 10, 20, 30], [0, 60, 0]),         # past the table's row
                      ([0, 10, 20, 30], [0, 2 ** 31 - 3, 0])):
        out, back, st = run(cu, start, table)
        assert st == K.DEVERR_BAD_SEQUENCE
        assert same(out[:10], good[:10]) and same(out[20:], good[20:]) and torch.isnan(out[10:20]).all()
        assert (back[10:20] == 7.0).all() and (back[:10] != 7.0).all()
        rows = oracle.blocks.rows_of(table[1], 32, np.arange(64))
        assert same(c.k[:, rows], before[0][:, rows])
    _, _, st = run([0, 10, 20, 30], [0, 31, 0], table)       # keys past the angles (40): not written
    assert st == K.DEVERR_BAD_SEQUENCE
    for cu in ([0, 10, 20, 31], [0, 20, 10, 30], [-5, 10, 20, 30], [0, 2 ** 31 - 1, 5, 30]):
        assert run(cu, [0, 0, 0], table)[2] & K.DEVERR_BAD_SEQUENCE
    bad = table.copy()
    bad[1, 0] = 8
    out, back, st = run([0, 10, 20, 30], [0, 0, 0], bad)
    assert st == K.DEVERR_BAD_PAGE and same(out, good)
    assert (back[10:20] == 7.0).all() and (back[:10] != 7.0).all()


@gpu
def test_rows_of_no_sequence_and_queries_in_place():
    # rows before the first sequence and behind the last are left as they are, in a call with
    # its queries turned in place inside the fused rows
    import torch
    import int8_kv_decode_gb300 as K
    c = Cache(2, 6, 64, 32, "int8")
    table = tables([100, 70], 64, 6)
    ang = torch_angles(128, 96)
    y = torch.randn((80, 7, D), device="cuda").bfloat16()
    before, cu, start = y.clone(), [3, 63, 70], [40, 63]
    pos = np.zeros(80, np.int64)
    pos[3:63], pos[63:70] = np.arange(40, 100), np.arange(63, 70)
    want = K.rope(y[:, :3].contiguous(), i32(pos), ang)
    for i, (a, b) in enumerate(((3, 63), (63, 70))):
        rows = before[a:b].float().cpu().numpy()
        k = oracle.blocks.rotate(rows[:, 3:5], ang.cpu().numpy()[pos[a:b]], False)
        oracle.blocks.append(c.host, "k", k, start[i], table[i], 64)
        oracle.blocks.append(c.host, "v", rows[:, 5:], start[i], table[i], 64)
    got = K.append_blocks(y[:, 3:5], y[:, 5:], i32(cu), i32(start), *c.args, i32(table), 64, table=ang,
                          q=y[:, :3], q_out=y[:, :3], workspace=c.ws)
    assert got.data_ptr() == y.data_ptr() and K.get_device_status(c.ws) == 0
    c.check()
    assert same(y[3:70, :3], want[3:70]) and same(y[:, 3:], before[:, 3:])
    assert same(y[:3], before[:3]) and same(y[70:], before[70:])


@gpu
def test_offsets_past_32_bits():
    # a plane of more than 2^31 bytes and values: the last pages written, read, copied and
    # attended to
    import torch
    import int8_kv_decode_gb300 as K
    pages, page, R = 36000, 512, 64                          # 18.4 M rows of 128: 2.4 GB in each plane
    k = torch.zeros((1, pages * page, D), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.zeros((1, pages * page // R), device="cuda")
    vs = torch.zeros_like(ks)
    host = {"R": R, "e4m3": False, "k": np.zeros((1, 1024, D)), "v": np.zeros((1, 1024, D)),
            "ks": np.zeros((1, 16), np.float32), "vs": np.zeros((1, 16), np.float32)}
    r = np.random.default_rng(0)
    x = r.standard_normal((700, 1, D)).astype(np.float32)
    t = torch.from_numpy(x).cuda()
    table, far = np.array([[1, 0]]), i32([[pages - 1, pages - 2]])
    for n in ("k", "v"):
        oracle.blocks.append(host, n, x, 0, table[0], page)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    K.append_blocks(t, t, i32([0, 700]), i32([0]), k, ks, v, vs, far, page, workspace=ws)
    back, _ = K.read_blocks(k, ks, v, vs, far, page, i32([0, 700]), i32([0]), 700, dtype=torch.float32, workspace=ws)
    rows = oracle.blocks.rows_of(table[0], page, np.arange(700))
    want = oracle.blocks.values(host, "k", rows).transpose(1, 0, 2)
    assert (np.abs(back.cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want)).all()
    q = torch.randn((1, 1, 4, D), device="cuda")
    out = K.decode_blocks(q, k, ks, v, vs, far, page, i32([700]), 700)
    from types import SimpleNamespace
    check_attend(SimpleNamespace(host=host, page=page), table, np.array([700]), q, out)
    K.copy_pages(k, ks, v, vs, i32([pages - 1, pages - 2]), i32([0, pages - 3]), page, workspace=ws)
    assert same(out, K.decode_blocks(q, k, ks, v, vs, i32([[0, pages - 3]]), page, i32([700]), 700))
    assert K.get_device_status(ws) == 0


@gpu
def test_copy_pages_of_a_block_scaled_cache():
    import torch
    import int8_kv_decode_gb300 as K
    for code, R, page in (("int8", 32, 128), ("e4m3", 64, 64), ("int8", 128, 256)):
        c = Cache(3, 6, page, R, code)
        want = {n: getattr(c, n).clone() for n in ("k", "v", "ks", "vs")}
        for a, b in ((0, 4), (0, 1), (5, 3)):
            for n in ("k", "v"):
                want[n].view(torch.uint8)[:, b * page:(b + 1) * page] = \
                    want[n].view(torch.uint8)[:, a * page:(a + 1) * page]
                per = page // R
                want[n + "s"][:, b * per:(b + 1) * per] = want[n + "s"][:, a * per:(a + 1) * per]
        K.copy_pages(*c.args, i32([0, -1, 0, 5]), i32([4, 2, 1, 3]), page, workspace=c.ws)
        assert K.get_device_status(c.ws) == 0
        for n in want:
            assert same(getattr(c, n), want[n]), n


# -------------------------------------------------------------- attention

def tolerance(dtype, size):
    own = 2.0 ** -22 if dtype == "float32" else 2.0 ** -11
    score = ((21 if dtype == "float32" else 12) * 2.0 ** -22) * size
    return 2 * (score + 2.0 ** -20 + 2.0 ** -22 + own) + 2.0 ** -17


def attend_inputs(B, M, Hq, Hkv, ctx, R=32, page=64, code="int8", dtype="float32", seed=0, gain=1.5):
    import torch
    ctx = np.asarray([ctx] * B if np.isscalar(ctx) else ctx, np.int64)
    keys = np.where(ctx > 0, ctx + M - 1, 0)
    pages = int((-(-keys // page)).sum()) + 2
    c = Cache(Hkv, pages, page, R, code, seed=seed)
    table = tables(keys, page, pages, seed=seed)
    r = np.random.default_rng(seed + 1)
    q = torch.from_numpy((gain * r.standard_normal((B, M, Hq, D))).astype(np.float32)).cuda().to(dtype_of(dtype))
    return c, table, ctx, q


def attend(c, table, ctx, q, **kw):
    import int8_kv_decode_gb300 as K
    return K.decode_blocks(q, *c.args, i32(table), c.page, i32(ctx), kw.pop("max_ctx", int(max(1, ctx.max()))), **kw)


def check_attend(c, table, ctx, q, got, **kw):
    dtype = str(q.dtype).replace("torch.", "")
    want, mass, size = oracle.blocks.decode(q.float().cpu().numpy(), c.host, table, c.page, ctx, **kw)
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    top = max(np.abs(oracle.blocks.values(c.host, "v", np.arange(c.host["v"].shape[1]))).max(), 1e-30)
    tail = 2 * max(int(ctx.max()), 1) * 2.0 ** -34 * top
    tol = tolerance(dtype, size)[..., None] * mass + tail
    tol += HALF_STEP[dtype] * (np.abs(want) + tol) + 2.0 ** -25        # (and below the type's least step)
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1, worst


SHAPES = [
    (1, 1, 1, 1, 1),                      # one key, one head
    (1, 1, 8, 2, 2),
    (3, 1, 8, 2, [31, 32, 33]),           # the 32-key step's edges
    (4, 2, 6, 2, [127, 128, 129, 126]),   # the first window's edges, GQA 3
    (4, 3, 8, 4, [1023, 1024, 1025, 1022]),      # where the windows become longer
    (5, 2, 8, 2, [255, 256, 257, 254, 383]),
    (2, 8, 16, 2, [5, 700]),              # 8 columns, 64 rows per head
    (2, 5, 32, 4, [1500, 1281]),          # 40 rows per head: row groups of 16
    (1, 1, 32, 4, 5000),
    (5, 1, 10, 2, [1, 2000, 64, 600, 3]),
    (3, 1, 16, 1, [300, 900, 17]),        # 16 rows
    (4, 1, 7, 7, [0, 40, 0, 300]),        # empty slots
    (1, 1, 4, 2, 20000),                  # more than 64 windows
]


@gpu
@pytest.mark.parametrize("B,M,Hq,Hkv,ctx", SHAPES)
@pytest.mark.parametrize("dtype,code,R,page", [("float32", "int8", 32, 32), ("bfloat16", "int8", 64, 64),
                                               ("float16", "e4m3", 32, 128), ("float32", "e4m3", 128, 128)])
def test_attention_matches_the_oracle(B, M, Hq, Hkv, ctx, dtype, code, R, page):
    x = attend_inputs(B, M, Hq, Hkv, ctx, R, page, code, dtype, seed=B * 100 + M * 10 + Hq)
    got = attend(*x)
    check_attend(*x, got)
    assert (got[x[2] == 0] == 0).all()


@gpu
@pytest.mark.parametrize("seed", range(8))
def test_attention_random_shapes(seed):
    r = np.random.default_rng(177 + seed)
    M, Hkv = int(r.integers(1, 9)), int(r.integers(1, 5))
    g = int(r.choice([n for n in range(1, 17) if n * M <= 64]))
    B = int(r.integers(1, 7))
    ctx = np.exp(r.uniform(0, np.log(2500), B)).astype(np.int64)
    x = attend_inputs(B, M, g * Hkv, Hkv, ctx, int(r.choice([32, 64, 128])), 128, str(r.choice(["int8", "e4m3"])),
                      str(r.choice(["float32", "bfloat16", "float16"])), seed=seed)
    check_attend(*x, attend(*x, sm_scale=0.05), sm_scale=0.05)


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_scales_and_scores_of_any_size(dtype):
    # value scales over 30 decimal powers between blocks, scores in the hundreds whose
    # largest lies anywhere, queries of very different size, zero blocks
    c, table, ctx, q = attend_inputs(3, 2, 8, 2, [900, 257, 40], dtype=dtype, code="int8", seed=5)
    r = np.random.default_rng(9)
    c.host["vs"] *= (10.0 ** r.uniform(-15, 15, c.host["vs"].shape)).astype(np.float32)
    c.host["vs"][:, ::5] = 0
    c.host["ks"][:, 1::7] = 0
    c.host["ks"] *= r.uniform(0.01, 12, c.host["ks"].shape).astype(np.float32)
    import torch
    c.vs.copy_(torch.from_numpy(c.host["vs"]))
    c.ks.copy_(torch.from_numpy(c.host["ks"]))
    q[0, 0] *= 2.0 ** -9
    q[1, 0, :4] = 0
    if dtype != "float16":
        q[2] *= 2.0 ** 40
        q[2, 1] *= 2.0 ** -90
        q[2, 0] *= 2.0 ** -38
    got = attend(c, table, ctx, q)
    want, mass, size = oracle.blocks.decode(q.float().cpu().numpy(), c.host, table, c.page, ctx)
    got = got.float().cpu().numpy().astype(np.float64)
    # (the tail's weights: the largest value of the row's own head and sequence, not of the cache)
    tol = tolerance(dtype, size)[..., None]
    top = np.zeros(mass.shape[:3])
    for b in range(3):
        V = np.abs(oracle.blocks.values(c.host, "v", oracle.blocks.rows_of(table[b], c.page, np.arange(ctx[b] + 1))))
        top[b] = np.repeat(V.max((1, 2)), 4)[None]
    # rows beyond float16's range come out infinite on both sides
    lim = tol * mass + 2 * 1000 * 2.0 ** -34 * top[..., None]
    lim = lim + HALF_STEP[dtype] * (np.abs(want) + lim) + 2.0 ** -25
    ok = np.abs(got - want) <= lim
    if dtype == "float16":
        ok |= np.isinf(got) & (np.abs(want) + lim >= 65504.0) & (np.sign(got) == np.sign(want))
    assert ok.all(), (np.abs(got - want) / lim)[~ok].max()


@gpu
@pytest.mark.parametrize("M,g", [(2, 12), (8, 4), (5, 8), (6, 8), (8, 7), (8, 8), (3, 7), (1, 16)])
@pytest.mark.parametrize("dtype,code", [("bfloat16", "int8"), ("float16", "e4m3"), ("float32", "int8"),
                                        ("float32", "e4m3")])
def test_units_of_any_size_give_the_same_bytes(M, g, dtype, code):
    # the limit max_ctx chooses how many rows go together (a large one: many); lengths that
    # leave warps of a block without keys, end inside steps, and move references late
    c, table, ctx, q = attend_inputs(5, M, 2 * g, 2, [40, 700, 513, 1200, 97], 32, 64, code, dtype,
                                     seed=M * 10 + g, gain=6.0)
    few = attend(c, table, ctx, q)
    check_attend(c, table, ctx, q, few)
    for limit in (4000, 20000, 60000):
        assert same(few, attend(c, table, ctx, q, max_ctx=limit)), limit


@gpu
@pytest.mark.parametrize("dtype,code", [("bfloat16", "int8"), ("float32", "e4m3")])
@pytest.mark.parametrize("gain", [1e3, 1e6, 1e9, 1e12])
def test_scores_of_any_size(dtype, code, gain):
    # scores whose float32 neighbours lie whole powers of two apart: a key then takes all of
    # a row's weight, unless others lie within the scores' rounding (the tolerance grows with
    # the size of the scores and leaves those rows to the finiteness alone)
    c, table, ctx, q = attend_inputs(4, 2, 8, 2, [5, 130, 600, 1500], 32, 64, code, dtype, seed=12, gain=gain)
    got = attend(c, table, ctx, q)
    check_attend(c, table, ctx, q, got)
    assert same(got, attend(c, table, ctx, q, max_ctx=60000))
    assert same(got[:, 1:], attend(c, table, ctx + 1, q[:, 1:].contiguous()))


@gpu
@pytest.mark.parametrize("dtype,code", [("bfloat16", "int8"), ("float32", "e4m3")])
def test_columns_and_batches_have_the_bytes_of_a_row_alone(dtype, code):
    import torch
    B, M, Hq, Hkv = 4, 5, 24, 2                              # 60 rows per head: groups of 16
    c, table, ctx, q = attend_inputs(B, M, Hq, Hkv, [125, 1022, 3, 640], 32, 64, code, dtype, seed=3, gain=4.0)
    whole = attend(c, table, ctx, q)
    for j in range(M):
        alone = attend(c, table, ctx + j, q[:, j:j + 1].contiguous())
        assert same(whole[:, j:j + 1], alone), j
    for b in range(B):
        assert same(whole[b:b + 1], attend(c, table[b:b + 1], ctx[b:b + 1], q[b:b + 1].contiguous(), max_ctx=5000))
    # one query head of a group alone, through a cache of its plane
    from types import SimpleNamespace
    one = SimpleNamespace(page=c.page, args=tuple(t[1:2].contiguous() for t in c.args))
    assert same(whole[:, :, 17:18], attend(one, table, ctx, q[:, :, 17:18].contiguous()))
    assert same(whole, attend(c, table, ctx, q))
    assert torch.isfinite(whole.float()).all()


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_codes_that_are_no_numbers_stay_where_they_are(dtype):
    # e4m3 NaN codes in rows past a sequence's keys, and in draft rows that a column does
    # not see; scales that are not finite in blocks of those alone
    import torch
    c, table, ctx, q = attend_inputs(2, 3, 8, 2, [94, 161], 32, 64, "e4m3", dtype, seed=8)
    want = attend(c, table, ctx, q)
    for b in range(2):
        n = int(ctx[b])
        past = oracle.blocks.rows_of(table[b], 64, np.arange(n + 2, -(-(n + 2) // 64) * 64))
        for t in (c.k, c.v):
            t.view(torch.uint8)[:, past] = 0x7f
    assert same(want, attend(c, table, ctx, q))
    # ctx 94: column 2 sees keys 94, 95 as well; ctx 94 + 3 would reach block 3
    for b in range(2):
        rows = oracle.blocks.rows_of(table[b], 64, np.arange(int(ctx[b]), int(ctx[b]) + 2))
        for t in (c.k, c.v):
            t.view(torch.uint8)[:, rows] = 0xff
    got = attend(c, table, ctx, q)
    assert same(want[:, 0], got[:, 0])
    # ctx 96: the drafts' rows begin a block of their own
    c, table, ctx, q = attend_inputs(2, 3, 8, 2, [96, 160], 32, 64, "e4m3", dtype, seed=8)
    want = attend(c, table, ctx, q)
    for b in range(2):
        at = int(oracle.blocks.rows_of(table[b], 64, [int(ctx[b])])[0]) // 32
        for t, bad in ((c.ks, float("nan")), (c.vs, float("inf"))):
            t[:, at] = bad
    got = attend(c, table, ctx, q)
    assert same(want[:, 0], got[:, 0])


@gpu
def test_bad_sequences_and_pages():
    import torch
    import int8_kv_decode_gb300 as K
    c, table, ctx, q = attend_inputs(5, 2, 8, 2, [70, 300, 50, 90, 260], seed=2)
    ws = K.alloc_blocks_workspace(5, 2, 8, 300)
    want = attend(c, table, ctx, q, workspace=ws)
    assert K.get_device_status(ws) == 0
    for bad in (-1, 301, 2 ** 31 - 1, -2 ** 31):
        x = ctx.copy()
        x[1] = bad
        got = attend(c, table, x, q, workspace=ws, max_ctx=300)
        assert K.get_device_status(ws) == K.DEVERR_BAD_SEQUENCE
        assert torch.isnan(got[1]).all() and same(got[[0, 2, 3, 4]], want[[0, 2, 3, 4]])
    # more keys than the table's row has pages
    got = attend(c, table[:, :3].copy(), ctx, q, workspace=ws)
    assert K.get_device_status(ws) == K.DEVERR_BAD_SEQUENCE
    assert torch.isnan(got[[1, 4]]).all() and same(got[[0, 2, 3]], want[[0, 2, 3]])
    t = table.copy()
    t[4, 1] = c.n_pages
    got = attend(c, t, ctx, q, workspace=ws)
    assert K.get_device_status(ws) == K.DEVERR_BAD_PAGE and same(got[:4], want[:4])
    x = np.zeros(5, np.int64)
    assert (attend(c, table, x, q, workspace=ws) == 0).all()


@gpu
def test_more_sequences_than_the_prefix_has_groups():
    import torch
    B = 700
    r = np.random.default_rng(0)
    ctx = r.integers(0, 200, B)
    c, table, ctx, q = attend_inputs(B, 1, 4, 2, ctx, 32, 32, "int8", "bfloat16", seed=6)
    got = attend(c, table, ctx, q)
    for b in list(range(0, B, 97)) + [B - 1]:
        check_attend(c, table[b:b + 1], ctx[b:b + 1], q[b:b + 1], got[b:b + 1])
    assert torch.isfinite(got.float()).all()


@gpu
def test_streams_graphs_and_devices():
    # a step captured once and replayed on new lengths and rows; two calls on two streams
    # with workspaces of their own
    import torch
    import int8_kv_decode_gb300 as K
    c, table, ctx, q = attend_inputs(4, 1, 8, 2, [60, 500, 1, 1200], 32, 64, "int8", "bfloat16", seed=4)
    tab, cu = i32(table), i32(np.arange(5))
    start, length = i32(ctx - 1), i32(ctx)
    kn = torch.randn((4, 2, D), device="cuda").bfloat16()
    vn = torch.randn((4, 2, D), device="cuda").bfloat16()
    ang = K.rope_table(2000)
    qin = q.view(4, 8, D)
    qout, out = torch.empty_like(qin), torch.empty_like(q)
    ws = K.alloc_blocks_workspace(4, 1, 8, 1300)

    def step():
        K.append_blocks(kn, vn, cu, start, *c.args, tab, 64, table=ang, q=qin, q_out=qout, workspace=ws)
        K.decode_blocks(qout.view(4, 1, 8, D), *c.args, tab, 64, length, 1300, out=out, workspace=ws)

    state = [t.clone() for t in c.args]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        kn.normal_()
        qin.normal_()
        start.copy_(i32(np.maximum(ctx - 2 - i, 0)))
        length.copy_(i32(np.maximum(ctx - 1 - i, 1)))
        for t, s in zip(c.args, state):
            t.copy_(s)
        graph.replay()
        got, after = out.clone(), [t.clone() for t in c.args]
        for t, s in zip(c.args, state):
            t.copy_(s)
        step()
        assert same(out, got)
        assert all(same(a, t) for a, t in zip(after, c.args))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    w2 = [K.alloc_blocks_workspace(4, 1, 8, 1300) for _ in range(2)]
    want = attend(c, table, ctx, q)
    torch.cuda.synchronize()
    res = []
    for s, w in zip((a, b), w2):
        with torch.cuda.stream(s):
            for _ in range(5):
                r = attend(c, table, ctx, q, workspace=w)
            res.append(r)
    torch.cuda.synchronize()
    assert same(res[0], want) and same(res[1], want)


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("sm_scale", [-0.11, 0.5])
def test_other_scales_of_the_scores(dtype, sm_scale):
    # a negative one is the positive one with the queries' signs turned
    c, table, ctx, q = attend_inputs(3, 2, 8, 2, [33, 600, 1], 32, 64, "int8", dtype, seed=15)
    got = attend(c, table, ctx, q, sm_scale=sm_scale)
    check_attend(c, table, ctx, q if sm_scale > 0 else -q, got, sm_scale=abs(sm_scale))


@gpu
@pytest.mark.parametrize("M,g,dtype", [(1, 4, "bfloat16"), (3, 7, "float32"), (5, 8, "float16")])
def test_queries_that_are_no_numbers_stay_in_their_row(M, g, dtype):
    import torch
    for ctx in (1, 32, 500, 9000):
        c, table, n, q = attend_inputs(2, M, 2 * g, 2, ctx, 32, 64, "int8", dtype, seed=16)
        want = attend(c, table, n, q)
        for bad in (float("nan"), float("inf")):
            x = q.clone()
            x[0, M - 1, g - 1, 5] = bad
            got = attend(c, table, n, x)
            assert torch.isnan(got[0, M - 1, g - 1]).all()
            got[0, M - 1, g - 1] = want[0, M - 1, g - 1]
            assert same(want, got), (ctx, bad)


@gpu
def test_one_call_of_many_sequences_is_many_calls_of_few():
    # so many that the search for a row's sequence goes three steps, runs of them empty
    import torch
    import int8_kv_decode_gb300 as K
    r = np.random.default_rng(3)
    B, per = 5000, 50
    lens = r.integers(0, 3, B)
    lens[700:1400] = 0
    lens[4990:] = 0
    start = r.integers(0, 30, B)
    cu = np.concatenate([[0], np.cumsum(lens)])
    n = int(cu[-1])
    caches = [Cache(1, B, 32, 32, "int8") for _ in range(2)]
    table = i32(r.permutation(B)[:, None])
    x = torch.randn((n, 3, D), device="cuda")
    ang = K.rope_table(64)

    def run(c, a, b):
        rows = x[cu[a]:cu[b]]
        args = (i32(cu[a:b + 1] - cu[a]), i32(start[a:b]))
        turned = K.append_blocks(rows[:, 1:2], rows[:, 2:], *args, *c.args, table[a:b], 32, table=ang,
                                 q=rows[:, :1], workspace=c.ws)
        back = K.read_blocks(*c.args, table[a:b], 32, *args, int(cu[b] - cu[a]), workspace=c.ws)
        return (turned, *back)

    whole = run(caches[0], 0, B)
    parts = [run(caches[1], a, a + per) for a in range(0, B, per) if cu[a + per] > cu[a]]
    for i, t in enumerate(whole):
        assert same(t, torch.cat([p[i] for p in parts]))
    for a, b in zip(caches[0].args, caches[1].args):
        assert same(a, b)
    assert K.get_device_status(caches[0].ws) == 0


@gpu
def test_only_keys_or_only_values_read_back():
    import torch
    import int8_kv_decode_gb300 as K
    from int8_kv_decode_gb300 import _lib
    c = Cache(3, 4, 64, 32, "int8")
    table = i32(tables([120, 70], 64, 4, spare=0))
    cu, start = i32([0, 90, 130]), i32([20, 30])
    want = K.read_blocks(*c.args, table, 64, cu, start, 140, dtype=torch.float32, workspace=c.ws)
    for one in (0, 1):
        out = torch.full((140, 3, D), 7.0, device="cuda")
        ptr = [None, None]
        ptr[one] = out.data_ptr()
        k, ks, v, vs = c.args
        status = _lib.load().kattn_read_blocks(
            k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr(), 0, 3, D, k.shape[1], 32, table.data_ptr(),
            table.shape[1], 64, cu.data_ptr(), start.data_ptr(), 2, 140, *ptr, 0, c.ws.data_ptr(), c.ws.numel(),
            torch.cuda.current_stream().cuda_stream)
        assert status == 0 and K.get_device_status(c.ws) == 0
        assert same(out[:130], want[one][:130]) and (out[130:] == 7.0).all()


@gpu
def test_captures_with_other_work_before_and_beside():
    # a step whose rows come from a copy, a fill and another stream's kernel in the capture,
    # and whose outputs another stream takes
    import torch
    import int8_kv_decode_gb300 as K
    c, table, ctx, q = attend_inputs(3, 1, 8, 2, [40, 300, 900], 32, 64, "int8", "bfloat16", seed=17)
    tab, cu, start, length = i32(table), i32(np.arange(4)), i32(ctx - 1), i32(ctx)
    ang = K.rope_table(1000)
    src = torch.randn((3, 12, D), device="cuda").bfloat16()
    rows, qout, out = torch.zeros_like(src), torch.empty_like(q), torch.empty_like(q)
    both = torch.empty((2, *out.shape), device="cuda", dtype=out.dtype)
    side = torch.cuda.Stream()
    ws = K.alloc_blocks_workspace(3, 1, 8, 900)

    def step():
        main = torch.cuda.current_stream()
        rows.zero_()
        rows[:, :8].copy_(src[:, :8])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.add(src[:, 8:], 1.0, out=rows[:, 8:])
        main.wait_stream(side)
        K.append_blocks(rows[:, 8:10], rows[:, 10:], cu, start, *c.args, tab, 64, table=ang, q=rows[:, :8],
                        q_out=qout.view(3, 8, D), workspace=ws)
        K.decode_blocks(qout, *c.args, tab, 64, length, 900, out=out, workspace=ws)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            both[0].copy_(out)
        K.decode_blocks(qout, *c.args, tab, 64, length, 900, out=both[1], workspace=ws)
        main.wait_stream(side)

    step()
    torch.cuda.synchronize()
    state = [t.clone() for t in c.args]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        src.normal_()
        for t, s in zip(c.args, state):
            t.copy_(s)
        step()
        want = [t.clone() for t in (out, both, qout, *c.args)]
        out.zero_()
        both.zero_()
        for t, s in zip(c.args, state):
            t.copy_(s)
        graph.replay()
        assert all(same(a, b) for a, b in zip(want, (out, both, qout, *c.args)))
        assert same(both[0], both[1])
    assert K.get_device_status(ws) == 0


@gpu
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_large_reads_have_the_values_of_small_ones(code):
    # 16-bit rows of large reads go through warps of more rows: ragged sequences, some empty,
    # with rows between none of them, against the float32 rows rounded once and single reads
    import torch
    import int8_kv_decode_gb300 as K
    r = np.random.default_rng(7)
    B, H = 230, 5
    lens = r.integers(0, 90, B)
    lens[40:110] = r.integers(0, 3, 70)
    start = r.integers(0, 128 - 90, B)
    c = Cache(H, 2 * B, 64, 32, code, seed=5)
    table = i32(tables([128] * B, 64, 2 * B, spare=0))
    cu = np.concatenate([[7], 7 + np.cumsum(lens)])
    n = int(cu[-1]) + 9
    assert n * 2 * H > 32768
    args = (*c.args, table, 64, i32(cu), i32(start), n)
    wide = K.read_blocks(*args, dtype=torch.float32, workspace=c.ws)
    for dtype in (torch.bfloat16, torch.float16):
        out = [torch.full((n, H, D), 7.0, device="cuda", dtype=dtype) for _ in range(2)]
        K.read_blocks(*args, out_k=out[0], out_v=out[1], workspace=c.ws)
        for o, w in zip(out, wide):
            assert same(o[7:n - 9], w[7:n - 9].to(dtype))
            assert (o[:7] == 7.0).all() and (o[n - 9:] == 7.0).all()
        for b in (0, 45, 113, B - 1):
            m = int(lens[b])
            alone = K.read_blocks(*c.args, table[b:b + 1], 64, i32([0, m]), i32(start[b:b + 1]), m, dtype=dtype,
                                  workspace=c.ws)
            for o, a in zip(out, alone):
                assert same(o[cu[b]:cu[b + 1]], a)
    assert K.get_device_status(c.ws) == 0
