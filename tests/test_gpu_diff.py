"""Differential decode attention on the GPU against the float64 oracle.

Tolerance, per channel: |error| <= 2^-16 * (sum w_0 |V| + |lam| sum w_1 |V|).
The query codes, the integer scores and the float32 scores are the oracle's own, so
the error is that of the weights and sums, relative to the terms added:
  * a weight 2^(s log2 e - m): the constant log2 e (2^-26) and the rounding of the
    exponent x (2^-24 |x|, and |x| 2^-x is at most 0.53, above the reference x is
    below 5.8), the exponential 2 ulp: below 2^-21 of the largest weight, once in
    the numerator and once in the row sum; the reference m is common to both;
  * weight times scale held in 22 bits (2^-22);
  * 16 tensor-core additions of 16 keys to a 256-key window, each off by up to 2^-22;
  * 8 rescalings of a window, 64 + 8 roundings of the window merge for up to 512
    windows, the division, the product with lam and the difference, 2^-24 each.
The sum is below (2 * 2 + 1 + 16) * 2^-22 + 84 * 2^-24 = 42 * 2^-22 < 2^-16.
"""

import numpy as np
import pytest

import oracle
from synth.paging import page_layout, paged_copy

TOL = 2.0 ** -16


def inputs(B, M, Hq, Hkv, ctx, seed=0, per_row=False, q_gain=2.0, outliers=False):
    """Host arrays of a ragged contiguous cache with random rows between the
    sequences."""
    r = np.random.default_rng(seed)
    ctx = np.asarray([ctx] * B if np.isscalar(ctx) else ctx, np.int32)
    gaps = r.integers(0, 4, B)
    n = ctx.astype(np.int64) + M - 1 + gaps
    start = np.concatenate([[0], np.cumsum(n)[:-1]]).astype(np.int64)
    cap = int(n.sum())
    x = {"ctx": ctx, "start": start, "cap": cap, "M": M,
         "q": (q_gain * r.standard_normal((B, M, Hq, 128))).astype(np.float32)}
    for name in ("k", "v"):
        rows = r.standard_normal((cap, Hkv, 128)).astype(np.float32)
        if outliers:
            rows[:, :, r.integers(0, 128, 4)] *= 20
        x[name + "8"], x[name + "s"] = oracle.quant.quantize_kv(rows)
    H = Hq // 2
    x["lam"] = r.uniform(-0.5, 1.2, (B, M, H) if per_row else (H,)).astype(np.float32)
    return x


def device(x):
    import torch
    return {n: torch.from_numpy(np.ascontiguousarray(a)).cuda() for n, a in x.items()
            if isinstance(a, np.ndarray)}


def run(x, t=None, **kw):
    import int8_kv_decode_gb300 as K
    t = t or device(x)
    return K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"],
                         int(x["ctx"].max()), t["lam"], **kw)


def expected(x, **kw):
    rows = [np.arange(int(c) + x["M"] - 1) + s for c, s in zip(x["ctx"], x["start"])]
    return oracle.diff.decode(x["q"], x["k8"], x["ks"], x["v8"], x["vs"], rows, x["ctx"], x["lam"],
                              **kw)


def check(got, want, mass):
    err = np.abs(got.astype(np.float64) - want)
    assert np.all(np.isfinite(got))
    worst = (err / np.maximum(mass, 1e-30)).max()
    assert worst <= TOL, worst


def bits(t):
    return t.cpu().numpy().view(np.uint32)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("B,M,Hq,Hkv,ctx", [
    (1, 1, 2, 2, 1),                      # one key, one head
    (1, 1, 8, 2, 2),
    (3, 1, 8, 2, [31, 32, 33]),           # the 32-key block's edges
    (3, 2, 6, 2, [127, 128, 129]),        # the first window's edges, GQA 3
    (4, 3, 8, 4, [511, 512, 513, 510]),   # the 256-key windows' edges, drafts across them
    (5, 2, 8, 2, [255, 256, 257, 254, 383]),
    (2, 8, 16, 2, [5, 700]),              # 8 columns, 64 rows per map
    (2, 5, 32, 4, [1500, 1025]),
    (1, 1, 32, 4, 5000),
    (5, 1, 10, 2, [1, 2000, 64, 600, 3]),  # GQA 5
    (2, 4, 64, 4, [300, 900]),            # 64 rows per map
    (1, 1, 4, 2, 40000),                  # more than 64 windows
])
@pytest.mark.parametrize("per_row", [False, True])
def test_matches_the_oracle(B, M, Hq, Hkv, ctx, per_row):
    x = inputs(B, M, Hq, Hkv, ctx, seed=B * 1000 + M * 100 + Hq, per_row=per_row)
    want, mass = expected(x)
    check(run(x).cpu().numpy(), want, mass)


@gpu
@pytest.mark.parametrize("seed", range(6))
def test_random_shapes(seed):
    r = np.random.default_rng(77 + seed)
    M, Hkv = int(r.integers(1, 9)), 2 * int(r.integers(1, 4))
    g = int(r.choice([n for n in range(1, 17) if n * M <= 64]))
    B = int(r.integers(1, 7))
    ctx = np.exp(r.uniform(0, np.log(3000), B)).astype(np.int32)
    x = inputs(B, M, g * Hkv, Hkv, np.maximum(ctx, 1), seed=seed, per_row=bool(seed % 2))
    want, mass = expected(x, sm_scale=0.05)
    check(run(x, sm_scale=0.05).cpu().numpy(), want, mass)


@gpu
def test_outlier_channels_and_large_scores():
    x = inputs(2, 2, 16, 2, [700, 90], seed=5, outliers=True, q_gain=8.0)
    want, mass = expected(x)
    check(run(x).cpu().numpy(), want, mass)


@gpu
def test_zero_and_extreme_scales():
    # rows of zeros (scale 0), rows with scales 2^-30 of the others and a query of
    # zeros: the weights are then 1 / L each
    x = inputs(2, 1, 8, 2, [600, 40], seed=6)
    x["vs"][:, ::3] = 0
    x["v8"][:, ::3] = 0
    x["vs"][:, 1::3] *= np.float32(2.0 ** -30)
    x["ks"][:, 5] = 0
    x["q"][0, 0, 2:4] = 0
    want, mass = expected(x)
    check(run(x).cpu().numpy(), want, mass)


@gpu
def test_lam_zero_leaves_one_map_and_equal_maps_cancel():
    import torch
    x = inputs(2, 2, 8, 2, [200, 65], seed=7)
    t = device(x)
    t["lam"].zero_()
    one = run(x, t)
    x["lam"][:] = 0
    want, mass = expected(x)
    check(one.cpu().numpy(), want, mass)
    # the same keys and queries on both maps, lam = 1: exactly zero
    t["q"][:, :, 1::2] = t["q"][:, :, 0::2]
    t["k8"][1::2], t["ks"][1::2] = t["k8"][0::2], t["ks"][0::2]
    t["lam"].fill_(1.0)
    assert torch.count_nonzero(run(x, t)) == 0


@gpu
@pytest.mark.parametrize("M,Hq,Hkv", [(4, 8, 2), (8, 16, 2), (3, 12, 2), (5, 32, 4)])
def test_column_j_equals_a_single_column_call(M, Hq, Hkv):
    x = inputs(3, M, Hq, Hkv, [510, 1300, 30], seed=8, per_row=True)
    t = device(x)
    full = run(x, t)
    import int8_kv_decode_gb300 as K
    for j in range(M):
        col = K.decode_diff(t["q"][:, j:j + 1].contiguous(), t["k8"], t["ks"], t["v8"], t["vs"],
                            t["start"], t["ctx"] + j, int(x["ctx"].max()) + j,
                            t["lam"][:, j:j + 1].contiguous())
        assert np.array_equal(bits(full[:, j:j + 1]), bits(col)), j


@gpu
def test_bytes_do_not_depend_on_the_batch():
    x = inputs(40, 1, 16, 2, np.random.default_rng(1).integers(1, 2500, 40), seed=9)
    t = device(x)
    full = bits(run(x, t))
    for b in (0, 7, 39):
        y = dict(x, ctx=x["ctx"][b:b + 1])
        one = run(y, {**t, "q": t["q"][b:b + 1], "start": t["start"][b:b + 1], "ctx": t["ctx"][b:b + 1]})
        assert np.array_equal(full[b:b + 1], bits(one))
    assert np.array_equal(full, bits(run(x, t)))


@gpu
@pytest.mark.parametrize("M,Hq", [(1, 8), (5, 16)])
def test_bytes_do_not_depend_on_max_ctx(M, Hq):
    # the join of the windows has other shapes for longer limits
    import int8_kv_decode_gb300 as K
    x = inputs(4, M, Hq, 2, [300, 5000, 257, 1], seed=10)
    t = device(x)
    got = [bits(K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"], limit,
                              t["lam"]))
           for limit in (5000, 8190, 8200, 65000, 70000)]
    for other in got[1:]:
        assert np.array_equal(got[0], other)


@gpu
def test_a_row_of_more_than_256_windows():
    x = inputs(2, 2, 4, 2, [70000, 900], seed=11)
    want, mass = expected(x)
    check(run(x).cpu().numpy(), want, mass)


# Many rows per map over many windows have a kernel of their own; the length limit of
# a call decides (more windows at most), so a small batch reaches it with a large one.
MANY = 80000


@gpu
@pytest.mark.parametrize("M,Hq", [(1, 34), (3, 16), (3, 14), (4, 16), (3, 26), (5, 16), (6, 16), (5, 22),
                                  (8, 14), (8, 16)])
@pytest.mark.parametrize("q_gain", [2.0, 30.0])          # 30: references move in most windows
def test_many_rows_over_many_windows(M, Hq, q_gain):
    import int8_kv_decode_gb300 as K
    x = inputs(4, M, Hq, 2, [1, 300, 1400, 120], seed=M * 100 + Hq, per_row=True, q_gain=q_gain)
    t = device(x)
    got = K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"], MANY, t["lam"])
    if q_gain == 2.0:
        want, mass = expected(x)
        check(got.cpu().numpy(), want, mass)
    assert np.array_equal(bits(got), bits(run(x, t)))
    for j in (0, M - 1):
        col = K.decode_diff(t["q"][:, j:j + 1].contiguous(), t["k8"], t["ks"], t["v8"], t["vs"],
                            t["start"], t["ctx"] + j, 1400 + j, t["lam"][:, j:j + 1].contiguous())
        assert np.array_equal(bits(got[:, j:j + 1]), bits(col)), j


@gpu
@pytest.mark.parametrize("B,M,Hq,Hkv,top", [(300, 3, 16, 2, 700), (70, 5, 32, 4, 3000), (3, 8, 16, 2, 70000)])
def test_many_rows_in_more_units_than_blocks(B, M, Hq, Hkv, top):
    ctx = np.exp(np.random.default_rng(B).uniform(0, np.log(top), B)).astype(np.int32)
    ctx[:2] = [top, 1]
    x = inputs(B, M, Hq, Hkv, ctx, seed=B, q_gain=6.0)
    t = device(x)
    full = bits(run(x, t))
    assert np.array_equal(full, bits(run(x, t)))
    for b in range(0, B, max(1, B // 12)):               # alone: row groups
        y = dict(x, ctx=np.minimum(x["ctx"][b:b + 1], 70000))
        one = run(y, {**t, "q": t["q"][b:b + 1], "start": t["start"][b:b + 1], "ctx": t["ctx"][b:b + 1]})
        assert np.array_equal(full[b:b + 1], bits(one)), b


@gpu
@pytest.mark.parametrize("P", [32, 128])
def test_many_rows_paged_and_bad_sequences(P):
    import torch
    import int8_kv_decode_gb300 as K
    x = inputs(5, 4, 16, 2, [900, 1, 64, 2000, 31], seed=P)
    t = device(x)
    want = bits(run(x, t))
    L = page_layout(x["ctx"], x["start"], 4, P, seed=P)
    kp, ksp, vp, vsp = paged_copy(L, t["k8"], t["ks"], t["v8"], t["vs"], seed=1)
    table = torch.from_numpy(L.block_table).cuda()
    ws = K.alloc_diff_workspace(5, 4, 16, MANY)

    def paged(ctx, table):
        return K.decode_diff_paged(t["q"], kp, ksp, vp, vsp, table, P, ctx, MANY, t["lam"], workspace=ws)

    assert np.array_equal(bits(paged(t["ctx"], table)), want)
    assert K.get_device_status(ws) == 0
    ctx = t["ctx"].clone()
    ctx[1], ctx[3] = 0, MANY + 1
    got = paged(ctx, table)
    assert torch.isnan(got[[1, 3]]).all()
    assert np.array_equal(bits(got[[0, 2, 4]]), want[[0, 2, 4]])
    assert K.get_device_status(ws) == K.DEVERR_BAD_SEQUENCE
    broken = table.clone()
    broken[0, 1] = L.n_pages + 7
    got = paged(t["ctx"], broken)
    assert K.get_device_status(ws) == K.DEVERR_BAD_PAGE
    assert np.array_equal(bits(got[1:]), want[1:])


@gpu
def test_many_rows_two_streams_and_a_graph():
    import torch
    import int8_kv_decode_gb300 as K
    x = inputs(6, 5, 16, 2, [3000, 700, 1, 256, 2222, 1500], seed=21)
    t = device(x)
    want = bits(run(x, t))
    args = (t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"], MANY, t["lam"])
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [K.alloc_diff_workspace(6, 5, 16, MANY) for _ in streams]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for s, w in zip(streams, spaces):
            with torch.cuda.stream(s):
                outs.append(K.decode_diff(*args, workspace=w))
    torch.cuda.synchronize()
    assert all(np.array_equal(bits(o), want) for o in outs)
    out = torch.empty_like(outs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.decode_diff(*args, out=out, workspace=spaces[0])
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), want)
    assert all(K.get_device_status(w) == 0 for w in spaces)


@gpu
@pytest.mark.parametrize("P", [32, 64, 256])
@pytest.mark.parametrize("M,Hq,Hkv,ctx", [(1, 8, 2, [1, 33, 900]), (5, 32, 4, [700, 1, 64]),
                                          (2, 64, 2, [2000, 513, 40])])
def test_paged_equals_contiguous_bytes(P, M, Hq, Hkv, ctx):
    import torch
    import int8_kv_decode_gb300 as K
    x = inputs(3, M, Hq, Hkv, ctx, seed=P)
    t = device(x)
    want = bits(run(x, t))
    L = page_layout(x["ctx"], x["start"], M, P, seed=P)
    kp, ksp, vp, vsp = paged_copy(L, t["k8"], t["ks"], t["v8"], t["vs"], seed=1)
    bt = torch.from_numpy(L.block_table).cuda()
    ws = K.alloc_diff_workspace(3, M, Hq, int(max(ctx)))
    got = K.decode_diff_paged(t["q"], kp, ksp, vp, vsp, bt, P, t["ctx"], int(max(ctx)), t["lam"],
                              workspace=ws)
    assert np.array_equal(bits(got), want)
    assert K.get_device_status(ws) == 0


@gpu
@pytest.mark.parametrize("M,Hq", [(1, 8), (4, 32)])
def test_bad_sequences_give_nan_and_leave_the_others(M, Hq):
    import int8_kv_decode_gb300 as K
    x = inputs(5, M, Hq, 2, [100, 600, 40, 700, 9], seed=11)
    t = device(x)
    ws = K.alloc_diff_workspace(5, M, Hq, 700)
    clean = run(x, t, workspace=ws).cpu().numpy()
    assert K.get_device_status(ws) == 0
    t["ctx"][0] = 0                       # no key
    t["ctx"][2] = 701                     # above max_ctx
    t["start"][4] = x["cap"] - 3          # past the cache
    out = run(x, t, workspace=ws).cpu().numpy()
    assert np.isnan(out[[0, 2, 4]]).all()
    assert np.array_equal(out[[1, 3]].view(np.uint32), clean[[1, 3]].view(np.uint32))
    assert K.get_device_status(ws) == K.DEVERR_BAD_SEQUENCE
    assert K.get_device_status(ws) == 0


@gpu
def test_bad_table_entries_are_flagged():
    import torch
    import int8_kv_decode_gb300 as K
    x = inputs(3, 1, 8, 2, [300, 700, 64], seed=12)
    t = device(x)
    L = page_layout(x["ctx"], x["start"], 1, 64, seed=2)
    kp, ksp, vp, vsp = paged_copy(L, t["k8"], t["ks"], t["v8"], t["vs"])
    bt = torch.from_numpy(L.block_table).cuda()
    ws = K.alloc_diff_workspace(3, 1, 8, 700)

    def go(table):
        return K.decode_diff_paged(t["q"], kp, ksp, vp, vsp, table, 64, t["ctx"], 700, t["lam"],
                                   workspace=ws).cpu().numpy()
    clean = go(bt)
    bad = bt.clone()
    bad[1, 3], bad[1, 10] = L.n_pages, -7
    out = go(bad)
    assert np.array_equal(out[[0, 2]].view(np.uint32), clean[[0, 2]].view(np.uint32))
    assert np.isfinite(out[1]).all()
    assert K.get_device_status(ws) == K.DEVERR_BAD_PAGE
    narrow = go(bt[:, :5].contiguous())
    assert np.isnan(narrow[1]).all() and np.isfinite(narrow[[0, 2]]).all()
    assert K.get_device_status(ws) == K.DEVERR_BAD_SEQUENCE


@gpu
def test_graph_replay_side_stream_and_two_calls_at_once():
    import torch
    import int8_kv_decode_gb300 as K
    x, y = inputs(4, 2, 16, 2, [900, 30, 513, 64], seed=13), inputs(2, 1, 8, 2, [2000, 5], seed=14)
    a, b = device(x), device(y)
    wa, wb = bits(run(x, a)), bits(run(y, b))
    ws = K.alloc_diff_workspace(4, 2, 16, 900)
    out = torch.empty((4, 2, 8, 256), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(x, a, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(x, a, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        with torch.cuda.stream(s):        # another call, its own workspace, meanwhile
            other = run(y, b)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), wa) and np.array_equal(bits(other), wb)
    q2 = torch.randn_like(a["q"])         # new inputs in the captured buffers
    a["q"].copy_(q2)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(out), bits(run(x, a)))


@gpu
def test_many_short_sequences():
    r = np.random.default_rng(3)
    x = inputs(3000, 1, 4, 2, r.integers(1, 40, 3000), seed=15)
    t = device(x)
    got = run(x, t).cpu().numpy()
    pick = [0, 1, 1499, 2999]
    rows = [np.arange(int(x["ctx"][b])) + x["start"][b] for b in pick]
    want, mass = oracle.diff.decode(x["q"][pick], x["k8"], x["ks"], x["v8"], x["vs"], rows,
                                    x["ctx"][pick], x["lam"])
    check(got[pick], want, mass)


@gpu
def test_offsets_past_32_bits():
    # a cache of 2^24 + rows per plane: byte offsets of plane 1 pass 2^31, the
    # sequence sits at the very end
    import torch
    import int8_kv_decode_gb300 as K
    x = inputs(1, 1, 4, 2, [700], seed=16)
    want = bits(run(x))
    t = device(x)
    cap = (1 << 24) + 4096
    big = {n: torch.zeros((2, cap, 128), dtype=torch.int8, device="cuda") for n in ("k8", "v8")}
    big.update({n: torch.zeros((2, cap), device="cuda") for n in ("ks", "vs")})
    for n in big:
        big[n][:, cap - 700:] = t[n][:, :700]
    got = K.decode_diff(t["q"], big["k8"], big["ks"], big["v8"], big["vs"], t["start"] + (cap - 700),
                        t["ctx"], 700, t["lam"])
    assert np.array_equal(bits(got), want)


# ------------------------------------------- keys that a column does not see

def columns_alone(x, t, full, limit=None):
    """Every column of `full` has the bytes of a single-column call (which has no
    hidden key)."""
    import int8_kv_decode_gb300 as K
    for j in range(x["M"]):
        col = K.decode_diff(t["q"][:, j:j + 1].contiguous(), t["k8"], t["ks"], t["v8"], t["vs"],
                            t["start"], t["ctx"] + j, limit or int(x["ctx"].max()) + j, t["lam"])
        assert np.array_equal(bits(full[:, j:j + 1]), bits(col)), j


# M, Hq and the limit: up to 4 rows per map, 8 rows and more, and the kernel of many rows
HIDING = [(2, 4, None), (4, 2, None), (8, 2, None), (2, 16, None), (3, 12, 80000), (8, 16, 80000)]


@gpu
@pytest.mark.parametrize("M,Hq,limit", HIDING)
def test_large_drafts_behind_zero_or_tiny_rows(M, Hq, limit):
    # what a column sees in a window is all zeros, or tiny, and a draft key behind it has
    # a large scale: 2^E of the small scales times the hidden one would leave float32
    import int8_kv_decode_gb300 as K
    x = inputs(4, M, Hq, 2, [1, 128, 300, 40], seed=31)
    at = x["start"]
    drafts = [np.arange(int(c), int(c) + M - 1) + int(s) for c, s in zip(x["ctx"], at)]
    x["v8"][:, at[0]], x["vs"][:, at[0]] = 0, 0                     # the only key of column 0
    x["vs"][:, at[2] + 256:at[2] + 300] = np.float32(2.0 ** -118)
    x["vs"][:, at[3]:at[3] + 40] = np.float32(2.0 ** -126)
    for d in drafts:
        x["vs"][:, d] = 8.0
    x["v8"][:, drafts[1][0]], x["vs"][:, drafts[1][0]] = 0, 0       # a window begins with a draft of zeros
    t = device(x)
    full = K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"],
                         limit or 300, t["lam"])
    want, mass = expected(x)
    check(full.cpu().numpy(), want, mass)
    columns_alone(x, t, full)


@gpu
@pytest.mark.parametrize("M,Hq,limit", HIDING)
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_hidden_scale_that_is_no_number(M, Hq, limit, value):
    # the last draft key's scales: the columns before the last do not see it
    import int8_kv_decode_gb300 as K
    x = inputs(3, M, Hq, 2, [5, 255, 600], seed=32)
    t = device(x)
    args = (t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"], limit or 600, t["lam"])
    want = bits(K.decode_diff(*args))
    for b in range(3):
        last = int(x["start"][b] + x["ctx"][b]) + M - 2
        t["ks"][:, last] = value
        t["vs"][:, last] = value
    assert np.array_equal(bits(K.decode_diff(*args))[:, :M - 1], want[:, :M - 1])


# -------------------------------------------- value scales that differ widely

def sink(x, b, key, v_scale, score=68.0):
    """Key `key` of sequence b takes nearly all of the weight of both maps, with the
    value scale v_scale and no zero among its values: its score is about `score`, those
    of the others are within +-10."""
    r = np.random.default_rng(key)
    at, Hkv = int(x["start"][b]) + key, x["k8"].shape[0]
    g = x["q"].shape[2] // Hkv
    for plane in range(Hkv):
        base = r.standard_normal(128).astype(np.float32)
        base *= np.float32(np.sqrt(128.0) / np.linalg.norm(base))
        heads = 2 * (plane // 2 * g + np.arange(g)) + plane % 2
        x["q"][b][:, heads] = 2 * base + 0.02 * x["q"][b][:, heads]
        k = base * np.float32(score / (2 * np.sqrt(128.0)))
        x["ks"][plane, at] = np.abs(k).max() / np.float32(127)
        x["k8"][plane, at] = np.rint(k / x["ks"][plane, at])
    x["v8"][:, at] = r.integers(64, 128, (Hkv, 128)) * r.choice([-1, 1], (Hkv, 128))
    x["vs"][:, at] = v_scale


SPREAD = [(1, 4, None), (4, 2, None), (1, 16, None), (2, 16, None), (3, 12, 80000), (8, 16, 80000)]


@gpu
@pytest.mark.parametrize("M,Hq,limit", SPREAD)
@pytest.mark.parametrize("down", [5, 7, 20, 34, 60, 100])
def test_the_weight_on_a_key_of_small_scale(M, Hq, limit, down):
    # one key has nearly all the weight and a value scale 2^-down of the others': a
    # product of weight and scale is held relative to the largest product of its row,
    # not to the largest scale.  First, middle and last key of a window, and a draft key.
    # The tolerance is the file's: products are off by 2^-22 of themselves, or by 2^-27 of
    # the row's largest, 256 of them times 127 to the 64 of the sink's own values: 2^-18 of
    # the mass when all err alike.
    import int8_kv_decode_gb300 as K
    ctx = [400, 256, 700, 90, 511]
    x = inputs(5, M, Hq, 2, ctx, seed=33)
    small = np.float32(2.0 ** -down / 40)
    for b, key in enumerate((0, 255, 300, 89, 511 + M - 2)):
        sink(x, b, key, small)
    t = device(x)
    full = K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"], limit or 700,
                         t["lam"])
    want, mass = expected(x)
    check(full.cpu().numpy(), want, mass)
    columns_alone(x, t, full)
    assert np.array_equal(bits(full), bits(run(x, t)))


@gpu
@pytest.mark.parametrize("M,Hq,limit", SPREAD)
def test_the_weight_on_a_value_row_of_zeros(M, Hq, limit):
    # the same with a value row of zeros: what is left of the sum are weights of about
    # e^-25, whose exponents are rounded to 2^-19 (the others' bound leaves that room)
    import int8_kv_decode_gb300 as K
    x = inputs(3, M, Hq, 2, [200, 256, 600], seed=34)
    for b, key in enumerate((0, 128, 599)):
        sink(x, b, key, 0.0, score=25.0)
        x["v8"][:, int(x["start"][b]) + key] = 0
    t = device(x)
    full = K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"], limit or 600,
                         t["lam"])
    want, mass = expected(x)
    check(full.cpu().numpy(), want, mass)
    columns_alone(x, t, full)


@gpu
@pytest.mark.parametrize("M,Hq,limit", SPREAD)
@pytest.mark.parametrize("seed", range(4))
def test_scales_over_the_whole_range(M, Hq, limit, seed):
    # scales over 2^-60 .. 2^20 and rows of zeros, references that move in most blocks
    # (weights below 2^-126 are 0, 2^-46 of the sum at most)
    import int8_kv_decode_gb300 as K
    x = inputs(4, M, Hq, 2, [33, 129, 900, 300], seed=40 + seed, q_gain=[2.0, 30.0][seed % 2])
    r = np.random.default_rng(seed)
    x["vs"] *= (2.0 ** r.integers(-60, 20, x["vs"].shape)).astype(np.float32)
    zero = r.random(x["vs"].shape) < 0.1
    x["vs"][zero] = 0
    x["v8"][zero] = 0
    x["v8"][(x["v8"] == 0) & ~zero[..., None]] = 1
    t = device(x)
    full = K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"], limit or 900,
                         t["lam"])
    assert np.isfinite(full.cpu().numpy()).all()
    columns_alone(x, t, full)
    # relative to the channel of the largest mass: a channel may be 1 where another is 127
    want, mass = expected(x)
    err = np.abs(full.cpu().numpy().astype(np.float64) - want).reshape(4, M, Hq // 2, 2, 128)
    most = mass.reshape(4, M, Hq // 2, 2, 128).max(-1, keepdims=True)
    assert (err <= TOL * most).all()


@gpu
@pytest.mark.parametrize("M,Hq,limit", SPREAD)
@pytest.mark.parametrize("plane", [0, 1])
def test_one_plane_of_the_two_has_such_a_key(M, Hq, limit, plane):
    # the two planes of a pair go their own ways, and so do windows and columns
    import int8_kv_decode_gb300 as K
    x = inputs(3, M, Hq, 2, [300, 120, 1000], seed=35)
    other = x["vs"][1 - plane].copy()
    for b, key in enumerate((0, 119 + M - 1, 700)):
        sink(x, b, key, np.float32(2.0 ** -30))
    x["vs"][1 - plane] = other
    t = device(x)
    full = K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"], limit or 1000,
                         t["lam"])
    want, mass = expected(x)
    check(full.cpu().numpy(), want, mass)
    columns_alone(x, t, full)
    # the other plane's channels are those of a cache without the small scales
    t["vs"][plane] = t["vs"][1 - plane]
    same = K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"], limit or 1000,
                         t["lam"])
    c = slice(128 * (1 - plane), 128 * (2 - plane))
    assert np.array_equal(bits(full[..., c].contiguous()), bits(same[..., c].contiguous()))


# --------------------------------------------------------------- large scores

@gpu
@pytest.mark.parametrize("M,Hq,limit", SPREAD)
@pytest.mark.parametrize("size", [1e3, 1e7, 1e8, 3e9, 1e12, 1e20])
def test_scores_of_any_size(M, Hq, limit, size):
    # scores are finite float32 values of any size: differences are taken first, where
    # they are exact near the largest, and a row's weights do not depend on where its
    # scores lie.  Keys 3, 40, 300 and 555 are the same, so that large scores tie.
    import int8_kv_decode_gb300 as K
    x = inputs(3, M, Hq, 2, [600, 45, 1400], seed=36)
    for b in range(3):
        at = int(x["start"][b])
        for key in (40, 300, 555):
            if key < x["ctx"][b]:
                x["k8"][:, at + key], x["ks"][:, at + key] = x["k8"][:, at + 3], x["ks"][:, at + 3]
    x["q"] *= np.float32(np.sqrt(size))
    x["ks"] *= np.float32(np.sqrt(size))
    t = device(x)
    full = K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"], limit or 1400,
                         t["lam"])
    got = full.cpu().numpy()
    want, mass = expected(x)
    assert np.all(np.isfinite(got))
    # (a channel may be 0 where all the weight is: relative to the row's largest)
    most = mass.max(-1, keepdims=True)
    assert (np.abs(got.astype(np.float64) - want) <= TOL * most).all()
    columns_alone(x, t, full)
