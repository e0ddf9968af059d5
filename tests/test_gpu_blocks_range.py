"""Values at the ends of float32's range, and values that are no numbers, through the
operators on block-scaled caches; the Python calls without the compiled binding.

Tolerances are those of test_gpu_blocks.py; what is left beside them is a share of the
row's own largest value (the tail) and float32's least steps, never a fixed number.
"""

import numpy as np
import pytest

import oracle
from test_gpu_blocks import (Cache, D, HALF_STEP, attend, attend_inputs, built, dtype_of, i32, same, tables,  # noqa: F401
                             tolerance, torch_angles)

gpu = pytest.mark.gpu


def set_scales(c, name, a):
    import torch
    c.host[name] = a.astype(np.float32)
    getattr(c, name).copy_(torch.from_numpy(c.host[name]))


def check_row_by_row(c, table, ctx, q, got):
    """As check_attend, with a tail of the row's own values: 2 * keys * 2^-34 of the largest
    |V| that it sees, and 2^-146 for results below float32's normal numbers (a float32 sum of
    weights up to 2^15 times such values, divided by 2^9 or more, is off by single steps of
    2^-149)."""
    dtype = str(q.dtype).replace("torch.", "")
    want, mass, size = oracle.blocks.decode(q.float().cpu().numpy(), c.host, table, c.page, ctx)
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    top = np.zeros(mass.shape[:3])
    B, M, Hq = top.shape
    for b in range(B):
        for j in range(M):
            V = oracle.blocks.values(c.host, "v", oracle.blocks.rows_of(table[b], c.page, np.arange(ctx[b] + j)))
            top[b, j] = np.repeat(np.abs(V).max((1, 2)), Hq // V.shape[0])
    lim = tolerance(dtype, size)[..., None] * mass + (2 * (np.asarray(ctx) + M)[:, None, None] * 2.0 ** -34 * top)[..., None]
    lim = lim + HALF_STEP[dtype] * (np.abs(want) + lim) + (2.0 ** -25 if dtype == "float16" else 2.0 ** -146)
    worst = (np.abs(got - want) / lim).max()
    assert worst <= 1, worst


# Scales of V: all near the top of the range (values to 1e37 and more), all near its bottom,
# over the whole of it from block to block, and ordinary ones with single blocks at the top.
def value_scales(kind, shape, r):
    if kind == "large":
        return 10.0 ** r.uniform(34.5, 35.5, shape)
    if kind == "largest":
        return np.full(shape, 7e35)                          # 448 times that is 3.1e38
    if kind == "tiny":
        return 10.0 ** r.uniform(-37.5, -36.5, shape)
    if kind == "small":
        return 10.0 ** r.uniform(-31, -29, shape)
    if kind == "any":
        return 10.0 ** r.uniform(-34, 35, shape)
    return np.where(r.random(shape) < 0.1, 1e35, 1.0) * r.uniform(0.5, 1.5, shape)


@gpu
@pytest.mark.parametrize("kind", ["large", "largest", "tiny", "small", "any", "single"])
@pytest.mark.parametrize("dtype,code", [("bfloat16", "int8"), ("float32", "e4m3"), ("bfloat16", "e4m3")])
@pytest.mark.parametrize("M,g,ctx", [(1, 4, [1, 33, 500, 9000]), (3, 7, [5, 510, 1500]), (5, 8, [700, 64]),
                                     (2, 24, [40, 2000])])
def test_value_scales_of_any_size(kind, dtype, code, M, g, ctx):
    c, table, ctx, q = attend_inputs(len(ctx), M, 2 * g, 2, ctx, 32, 64, code, dtype, seed=M + g)
    r = np.random.default_rng(M * 100 + g)
    set_scales(c, "vs", value_scales(kind, c.host["vs"].shape, r))
    got = attend(c, table, ctx, q)
    check_row_by_row(c, table, ctx, q, got)
    # the bytes of a row: under any limit, in any batch, as the only column
    assert same(got, attend(c, table, ctx, q, max_ctx=60000))
    for b in range(len(ctx)):
        assert same(got[b:b + 1], attend(c, table[b:b + 1], ctx[b:b + 1], q[b:b + 1].contiguous(), max_ctx=9000))
    for j in range(M):
        assert same(got[:, j:j + 1], attend(c, table, ctx + j, q[:, j:j + 1].contiguous()))


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,g", [(2, 4), (4, 8), (5, 8)])
def test_large_values_that_a_column_does_not_see(dtype, M, g):
    # a block of draft rows with the largest scales behind contexts of the smallest
    c, table, ctx, q = attend_inputs(3, M, 2 * g, 2, [96, 640, 1600], 32, 64, "int8", dtype, seed=3)
    set_scales(c, "vs", c.host["vs"] * np.float32(2.0 ** -118))
    want = attend(c, table, ctx, q)
    scales = c.host["vs"].copy()
    for b in range(3):
        scales[:, int(oracle.blocks.rows_of(table[b], 64, [int(ctx[b])])[0]) // 32] = 1e35
    set_scales(c, "vs", scales)
    got = attend(c, table, ctx, q)
    assert same(want[:, 0], got[:, 0])
    check_row_by_row(c, table, ctx, q, got)


@gpu
@pytest.mark.parametrize("at", [100, 35000, 69900])
def test_a_large_block_in_a_long_context(at):
    # more windows than the join of a row weighs at a time, by every number of warps
    c, table, ctx, q = attend_inputs(2, 2, 4, 1, [70000, 20000], 32, 64, "int8", "float32", seed=6)
    scales = c.host["vs"].copy()
    scales[:, int(oracle.blocks.rows_of(table[0], 64, [at])[0]) // 32] = 1e35
    want = attend(c, table, ctx, q)
    set_scales(c, "vs", scales)
    got = attend(c, table, ctx, q)
    check_row_by_row(c, table, ctx, q, got)
    assert same(want[1], got[1])
    assert same(got, attend(c, table, ctx, q, max_ctx=200000))
    # a window with the block alone, and a row that begins and ends with it
    c, table, ctx, q = attend_inputs(1, 1, 4, 1, [600], 32, 64, "int8", "float32", seed=7)
    set_scales(c, "vs", np.full(c.host["vs"].shape, 1e-30 if at == 100 else 1.0))
    scales = c.host["vs"].copy()
    scales[:, int(oracle.blocks.rows_of(table[0], 64, [at % 600])[0]) // 32] = 1e35
    set_scales(c, "vs", scales)
    check_row_by_row(c, table, ctx, q, attend(c, table, ctx, q))


# ------------------------------------------------------------- no numbers

@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,g,gain", [(1, 4, 1.5), (1, 4, 40.0), (3, 7, 6.0), (5, 8, 1.5)])
def test_keys_that_are_no_numbers_reach_the_rows_that_see_them(dtype, M, g, gain):
    # an e4m3 NaN in one key, in steps that move references and in steps that do not; the
    # rows of the other head keep their bytes
    import torch
    c, table, ctx, q = attend_inputs(2, M, 2 * g, 2, [1500, 700], 32, 64, "e4m3", dtype, seed=8, gain=gain)
    want = attend(c, table, ctx, q)
    keys = c.k.view(torch.uint8).clone()
    for t in (0, 5, 31, 130, 300, 520, 699, 700 + M - 2):
        row = int(oracle.blocks.rows_of(table[1], 64, [t])[0])
        c.k.view(torch.uint8)[1, row, 77] = 0x7f
        got = attend(c, table, ctx, q)
        for j in range(M):
            if t < 700 + j:
                assert torch.isnan(got[1, j, g:].float()).all(), (t, j)
            else:
                assert same(got[1, j], want[1, j]), (t, j)
        assert same(got[0], want[0]) and same(got[1, :, :g], want[1, :, :g])
        assert same(got, attend(c, table, ctx, q, max_ctx=60000))
        c.k.view(torch.uint8).copy_(keys)
    # every key of a warp's first step, and of a whole first window
    for keys_of in (np.arange(32), np.arange(512)):
        c.k.view(torch.uint8)[1, oracle.blocks.rows_of(table[1], 64, keys_of)] = 0xff
        got = attend(c, table, ctx, q)
        assert torch.isnan(got[1, :, g:].float()).all() and same(got[0], want[0])
        c.k.view(torch.uint8).copy_(keys)
    # a scale that is no number
    c.ks[1, int(oracle.blocks.rows_of(table[1], 64, [32])[0]) // 32] = float("nan")
    got = attend(c, table, ctx, q)
    assert torch.isnan(got[1, :, g:].float()).all() and same(got[0], want[0]) and same(got[1, :, :g], want[1, :, :g])


@gpu
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("rot", [None, 64])
def test_rows_that_are_not_finite_do_not_spoil_their_block(code, dtype, rot):
    import torch
    import int8_kv_decode_gb300 as K
    c = Cache(2, 6, 64, 32, code, seed=2)
    start, lens = [20, 0], [50, 33]                          # the first goes on inside a block
    table = tables([70, 33], 64, 6)
    r = np.random.default_rng(1)
    kn, vn = (torch.from_numpy(r.standard_normal((83, 2, D)).astype(np.float32)).cuda().to(dtype_of(dtype))
              for _ in "kv")
    for x in (kn, vn):
        x[2, 0, 3], x[3, 0, 5], x[4, 0, 100] = float("inf"), float("nan"), -float("inf")
        x[13, 1, 6] = float("nan")                           # beside a finite neighbour near a border
        x[50:82, 1, 9] = float("inf")                        # in every row of a block
        x[82, 0] = float("nan")                              # a block of nothing else
    ang = torch_angles(80, rot) if rot else None
    cu = np.array([0, 50, 83])
    K.append_blocks(kn, vn, i32(cu), i32(start), *c.args, i32(table), 64, table=ang, workspace=c.ws)
    assert K.get_device_status(c.ws) == K.DEVERR_NOT_FINITE
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(start, lens)])
    with np.errstate(invalid="ignore"):
        kh = kn.float().cpu().numpy()
        kh = oracle.blocks.rotate(kh, ang.cpu().numpy()[pos], False) if rot else kh
        for b in range(2):
            for name, x in (("k", kh), ("v", vn.float().cpu().numpy())):
                oracle.blocks.append(c.host, name, x[cu[b]:cu[b + 1]], start[b], table[b], 64)
    for name in ("k", "v"):
        got = getattr(c, name).float().cpu().numpy()
        assert np.array_equal(got, c.host[name].astype(np.float32), equal_nan=True), name
        assert same(getattr(c, name + "s"), torch.from_numpy(c.host[name + "s"])), name
        assert np.isfinite(c.host[name + "s"]).all()
    # finite rows flag nothing
    K.append_blocks(kn[5:12], vn[5:12], i32([0, 7, 7]), i32([0, 0]), *c.args, i32(table), 64, workspace=c.ws)
    assert K.get_device_status(c.ws) == 0


def test_the_error_bit_is_the_headers():
    import os
    import re
    import int8_kv_decode_gb300 as K
    with open(os.path.join(os.path.dirname(__file__), "..", "include", "kattn.h"), encoding="utf-8") as f:
        bit = int(re.search(r"#define KATTN_DEVERR_NOT_FINITE (0x[0-9a-f]+)u", f.read()).group(1), 16)
    assert bit == K.DEVERR_NOT_FINITE
    assert bit & (K.DEVERR_BAD_SEQUENCE | K.DEVERR_TIMEOUT | K.DEVERR_BAD_PAGE | K.DEVERR_NO_PAGES) == 0


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_queries_of_sequences_that_leave_the_call_are_nan(dtype):
    import torch
    import int8_kv_decode_gb300 as K
    c = Cache(2, 8, 32, 32, "int8")
    table = tables([64, 64, 64], 32, 8, spare=0)
    x = torch.randn((30, 2, D), device="cuda").to(dtype_of(dtype))
    q = torch.randn((30, 9, D), device="cuda").to(dtype_of(dtype))
    ang = torch_angles(64, 128)

    def run(cu):
        out = torch.full_like(q, 7.0)
        K.append_blocks(x, x, i32(cu), i32([0, 0, 0]), *c.args, i32(table), 32, table=ang, q=q, q_out=out,
                        workspace=c.ws)
        return out, K.get_device_status(c.ws)

    good, st = run([0, 10, 20, 30])
    assert st == 0
    got, st = run([0, 10, 20, 31])                           # one row behind the arrays
    assert st == K.DEVERR_BAD_SEQUENCE
    assert same(got[:20], good[:20]) and torch.isnan(got[20:].float()).all()
    got, st = run([-5, 10, 20, 30])                          # rows before them
    assert st == K.DEVERR_BAD_SEQUENCE
    assert same(got[10:], good[10:]) and torch.isnan(got[:10].float()).all()
    got, st = run([2, 10, 20, 28])                           # rows of no sequence stay
    assert st == 0 and (got[:2] == 7.0).all() and (got[28:] == 7.0).all()
    assert same(got[10:20], good[10:20])


# ----------------------------------------------- without the compiled binding

@gpu
def test_calls_without_the_compiled_binding(monkeypatch):
    import sys
    import torch
    import int8_kv_decode_gb300 as K
    from int8_kv_decode_gb300 import api

    def run():
        c, table, ctx, q = attend_inputs(2, 2, 8, 2, [100, 300], dtype="bfloat16", seed=1)
        ang = torch_angles(400, 128)
        x = torch.randn((9, 12, D), device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
        got = [K.rope(x, i32(np.arange(9)), ang, out=torch.empty_like(x))]
        q_out = torch.empty_like(x[:, :8])
        K.append_blocks(x[:, 8:10], x[:, 10:], i32([0, 5, 9]), i32([96, 1]), *c.args, i32(table), c.page, table=ang,
                        q=x[:, :8], q_out=q_out, workspace=c.ws)
        back = [torch.empty((9, 2, D), device="cuda") for _ in "kv"]
        K.read_blocks(*c.args, i32(table), c.page, i32([0, 5, 9]), i32([96, 1]), 9, out_k=back[0], out_v=back[1],
                      workspace=c.ws)
        out = attend(c, table, ctx, q, out=torch.empty_like(q), workspace=K.alloc_blocks_workspace(2, 2, 8, 300))
        assert K.get_device_status(c.ws) == 0
        return got + [q_out] + back + [out]

    want = run()
    monkeypatch.setattr(api, "_plain", None)
    monkeypatch.setitem(sys.modules, "int8_kv_decode_gb300._bind", None)       # its import fails
    monkeypatch.delattr(K, "_bind", raising=False)
    with pytest.warns(RuntimeWarning, match="binding"):
        got = run()
    assert all(same(a, b) for a, b in zip(want, got))
