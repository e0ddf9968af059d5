"""Differential decode, the 8-bit norm and the page operations without a GPU:
what the C ABI and the binding refuse before anything is enqueued, the
workspace sizes, and pins of their oracles against something else than
themselves.
"""

import numpy as np
import pytest

import oracle

INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = -1, -2, -3, -4
FAKE = 0x100000                           # never dereferenced: validation comes first
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from int8_kv_decode_gb300 import _lib
    return _lib.load()


def call(fn, defaults, **changes):
    args = dict(defaults, **changes)
    assert set(args) == set(defaults), changes
    return fn(*args.values())


DIFF = dict(q=FAKE, k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, rs=FAKE, ctx=FAKE, lam=FAKE, per_row=0, B=2, M=1,
            Hq=8, Hkv=2, d=128, cap=4096, max_ctx=1000, scale=0.0, out=FAKE, ws=FAKE, ws_bytes=0,
            stream=None)
DIFF_PAGED = dict(q=FAKE, k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, bt=FAKE, max_pages=16, page_rows=64,
                  ctx=FAKE, lam=FAKE, per_row=0, B=2, M=1, Hq=8, Hkv=2, d=128, cap=4096, max_ctx=1000,
                  scale=0.0, out=FAKE, ws=FAKE, ws_bytes=0, stream=None)


@pytest.mark.parametrize("paged", [False, True])
def test_diff_refusals(lib, paged):
    fn = lib.kattn_decode_diff_paged if paged else lib.kattn_decode_diff
    base = DIFF_PAGED if paged else DIFF
    # every call below fails: with valid arguments, ws_bytes = 0 is the error
    assert call(fn, base) == WORKSPACE
    need = lib.kattn_diff_workspace_size(2, 1, 8, 1000)
    assert call(fn, base, ws_bytes=need - 1) == WORKSPACE
    assert call(fn, base, ws_bytes=BIG, ws=FAKE + 128) == WORKSPACE
    assert call(fn, base, ws_bytes=BIG, ws=None) == WORKSPACE
    for name in ("q", "k", "ks", "v", "vs", "ctx", "lam", "out"):
        assert call(fn, base, **{name: None}) == INVALID, name
        assert call(fn, base, **{name: FAKE + 2}) == MISALIGNED, name
    assert call(fn, base, out=FAKE + 8) == MISALIGNED
    for bad in (dict(Hkv=1, Hq=8), dict(Hkv=3, Hq=9), dict(Hq=7), dict(B=-1), dict(M=0),
                dict(max_ctx=0), dict(cap=0), dict(per_row=2), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(B=65536)):
        assert call(fn, base, **bad) == INVALID, bad
    for bad in (dict(d=64), dict(M=9), dict(Hq=130, Hkv=2), dict(Hq=32, M=5, Hkv=2)):
        assert call(fn, base, **bad) == UNSUPPORTED, bad
    assert call(fn, base, B=65535, max_ctx=2 ** 29, Hkv=64, Hq=64, cap=64 * 1024) == UNSUPPORTED
    assert call(fn, base, B=0, ws=None) == 0
    if paged:
        assert call(fn, base, page_rows=16) == UNSUPPORTED
        assert call(fn, base, page_rows=96) == UNSUPPORTED
        assert call(fn, base, page_rows=0) == INVALID
        assert call(fn, base, max_pages=0) == INVALID
        assert call(fn, base, cap=4100) == INVALID
        assert call(fn, base, bt=None) == INVALID


def test_diff_workspace_size(lib):
    size = lib.kattn_diff_workspace_size
    assert size(1, 1, 2, 1) >= 256
    assert size(4, 8, 64, 9000) >= size(4, 1, 64, 9000) >= size(2, 1, 64, 9000) > 0
    assert size(0, 1, 2, 1) == size(1, 0, 2, 1) == size(1, 9, 2, 1) == size(1, 1, 0, 1) == size(1, 1, 2, 0) == 0


NORM = dict(x=FAKE, res=FAKE, w=FAKE, x_type=0, rows=4, d=256, xs=256, rs=256, ros=256, eps=1e-6, group=0,
            code=0, res_out=FAKE, codes=FAKE, scales=FAKE, stream=None)


def test_norm_refusals(lib):
    fn = lib.kattn_rms_norm_quant
    for bad in (dict(x=None), dict(w=None), dict(codes=None), dict(scales=None), dict(res=None),
                dict(res_out=None), dict(x_type=3), dict(x_type=-1), dict(code=2), dict(rows=-1), dict(d=0),
                dict(d=(1 << 24) + 1, xs=1 << 25), dict(xs=255), dict(rs=255), dict(ros=255),
                dict(eps=float("nan")), dict(eps=-1.0), dict(group=128, d=200, xs=200, rs=200, ros=200),
                dict(rs=512)):
        assert call(fn, NORM, **bad) == INVALID, bad
    for bad in (dict(group=64), dict(rows=1 << 31)):
        assert call(fn, NORM, **bad) == UNSUPPORTED, bad
    for name in ("x", "res", "w", "res_out", "scales"):
        assert call(fn, NORM, **{name: FAKE + 2}) == MISALIGNED, name
        assert call(fn, dict(NORM, x_type=1), **{name: FAKE + 1}) == MISALIGNED, name
    assert call(fn, NORM, rows=0, x=None) == 0


RESERVE = dict(table=FAKE, S=8, mp=4, refs=FAKE, n_pages=64, P=32, seqs=FAKE, lens=FAKE, n=3, ws=FAKE,
               ws_bytes=0, stream=None)
FREE = dict(table=FAKE, S=8, mp=4, refs=FAKE, n_pages=64, seqs=FAKE, n=3, ws=FAKE, ws_bytes=0, stream=None)
FORK = dict(table=FAKE, S=8, mp=4, refs=FAKE, n_pages=64, P=32, parents=FAKE, children=FAKE, lens=FAKE, n=3,
            src=FAKE, dst=FAKE, ws=FAKE, ws_bytes=0, stream=None)
COMPACT = dict(table=FAKE, S=8, mp=4, refs=FAKE, n_pages=64, table_out=FAKE, ref_out=FAKE, src=FAKE, dst=FAKE,
               counts=FAKE, ws=FAKE, ws_bytes=0, stream=None)
COPY = dict(k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, Hkv=2, d=128, cap=4096, P=32, src=FAKE, dst=FAKE, n=3,
            count=None, ws=FAKE, ws_bytes=0, stream=None)


@pytest.mark.parametrize("name,base", [("reserve_pages", RESERVE), ("free_sequences", FREE),
                                       ("fork_sequences", FORK), ("compact_pages", COMPACT)])
def test_page_operation_refusals(lib, name, base):
    fn = getattr(lib, "kattn_" + name)
    assert call(fn, base) == WORKSPACE
    assert call(fn, base, ws_bytes=lib.kattn_page_workspace_size(8, 64) - 1) == WORKSPACE
    assert call(fn, base, ws_bytes=BIG, ws=FAKE + 64) == WORKSPACE
    ok = dict(base, ws_bytes=BIG)
    for arg, value in base.items():
        if value == FAKE and arg != "ws":
            assert call(fn, ok, **{arg: None}) == INVALID, arg
            assert call(fn, ok, **{arg: FAKE + 2}) == MISALIGNED, arg
    for arg in ("S", "mp", "n_pages"):
        assert call(fn, ok, **{arg: 0}) == INVALID, arg
    if "n" in base:
        assert call(fn, ok, n=-1) == INVALID
        assert call(fn, ok, n=9) == INVALID            # more entries than slots
        assert call(fn, ok, n=0) == 0
    if "P" in base:
        assert call(fn, ok, P=0) == INVALID
        assert call(fn, ok, P=48) == UNSUPPORTED
        assert call(fn, ok, P=16) == UNSUPPORTED


def test_copy_pages_refusals(lib):
    fn = lib.kattn_copy_pages
    assert call(fn, COPY) == WORKSPACE
    ok = dict(COPY, ws_bytes=256)
    assert call(fn, ok, ws=None) == WORKSPACE
    for arg in ("k", "ks", "v", "vs", "src", "dst"):
        assert call(fn, ok, **{arg: None}) == INVALID, arg
        assert call(fn, ok, **{arg: FAKE + 2}) == MISALIGNED, arg
    assert call(fn, ok, ks=FAKE + 8) == MISALIGNED
    assert call(fn, ok, count=FAKE + 2) == MISALIGNED
    for bad in (dict(Hkv=0), dict(cap=0), dict(n=-1), dict(P=0), dict(cap=4100)):
        assert call(fn, ok, **bad) == INVALID, bad
    for bad in (dict(d=64), dict(P=40), dict(P=16)):
        assert call(fn, ok, **bad) == UNSUPPORTED, bad
    assert call(fn, ok, n=0) == 0


def test_page_workspace_size(lib):
    size = lib.kattn_page_workspace_size
    assert size(0, 1) == size(1, 0) == 0
    assert size(1, 1) > 256 and size(4096, 100000) > 4 * (100000 + 4096)


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    import int8_kv_decode_gb300 as K
    f, i = torch.zeros(2, 3), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        K.rms_norm_quant(f, torch.ones(3))
    with pytest.raises(TypeError):
        K.rms_norm_quant(f.double(), torch.ones(3))
    with pytest.raises(TypeError):
        K.rms_norm_quant(None, torch.ones(3))
    with pytest.raises(ValueError):
        K.free_sequences(torch.zeros((2, 2), dtype=torch.int32), i, i)
    with pytest.raises(TypeError):
        K.reserve_pages(torch.zeros((2, 2), dtype=torch.int64), i, i, i, 32)
    with pytest.raises(ValueError):
        K.decode_diff(f, None, None, None, None, None, None, 1, f)
    with pytest.raises(TypeError):
        K.decode_diff(f, None, None, None, None, None, None, 1, None)
    with pytest.raises(TypeError):
        K.copy_pages(None, f, f, f, i, i, 32)


def test_no_pages_bit_matches_header():
    import os
    import re
    from conftest import ROOT
    from int8_kv_decode_gb300 import api
    text = open(os.path.join(ROOT, "include", "kattn.h"), encoding="utf-8").read()
    assert int(re.search(r"#define KATTN_DEVERR_NO_PAGES (0x[0-9a-f]+)u", text).group(1), 16) == api.DEVERR_NO_PAGES
    assert (oracle.pages.BAD_SEQUENCE, oracle.pages.BAD_PAGE, oracle.pages.NO_PAGES) == \
        (api.DEVERR_BAD_SEQUENCE, api.DEVERR_BAD_PAGE, api.DEVERR_NO_PAGES)


# ------------------------------------------------------------ oracle pins

def test_diff_oracle_against_two_plain_decodes():
    # with lam = 0 the first 128 channels are a plain decode of heads 0, 2, ... whose
    # kv planes are (2p, 2p); with lam = 1 and equal maps the difference is 0
    r = np.random.default_rng(0)
    q = r.standard_normal((2, 2, 8, 128)).astype(np.float32)
    k8, ks = oracle.quant.quantize_kv(r.standard_normal((60, 4, 128)).astype(np.float32))
    v8, vs = oracle.quant.quantize_kv(r.standard_normal((60, 4, 128)).astype(np.float32))
    rows, ctx = [np.arange(20), np.arange(20, 60)], np.array([19, 39])
    out, _ = oracle.diff.decode(q, k8, ks, v8, vs, rows, ctx, np.zeros(4))
    for c in (0, 1):
        plain = oracle.attention.decode(q[:, :, 0::2], k8[0::2], ks[0::2], v8[c::2], vs[c::2],
                                        np.array([0, 20]), ctx)
        assert np.allclose(out[..., 128 * c:128 * c + 128], plain, rtol=1e-5, atol=1e-5)
    q[:, :, 1::2] = q[:, :, 0::2]
    k8[1::2], ks[1::2] = k8[0::2], ks[0::2]
    out, mass = oracle.diff.decode(q, k8, ks, v8, vs, rows, ctx, np.ones(4))
    assert np.abs(out).max() < 1e-12 and mass.min() > 0


def test_norm_oracle_reconstructs_the_norm():
    r = np.random.default_rng(1)
    h, w = r.standard_normal((7, 256)).astype(np.float32), r.uniform(0.5, 2, 256).astype(np.float32)
    want = h / np.sqrt((h.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-6) * w
    for group in (0, 128):
        c, s = oracle.norm.rms_norm_quant(h, w, group=group)
        got = (c.reshape(7, -1, group or 256) * s[..., None]).reshape(7, 256)
        # half a step of the row's scale
        assert (np.abs(got - want) <= 0.5001 * np.repeat(s, group or 256, axis=1)).all()
        c, s = oracle.norm.rms_norm_quant(h, w, group=group, e4m3=True)
        got = (c.reshape(7, -1, group or 256) * s[..., None]).reshape(7, 256)
        # 2^-4 of the value, or half the smallest step 2^-9
        assert (np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -4,
                                                 2.0 ** -10 * np.repeat(s, group or 256, axis=1)) * 1.0001).all()
    c, s = oracle.norm.rms_norm_quant(np.zeros((1, 4)), np.ones(4))
    assert not c.any() and not s.any()


def test_page_oracle_keeps_its_books():
    # counts equal the entries that name a page, whatever is called
    r = np.random.default_rng(2)
    table, refs = np.full((12, 6), -1, np.int32), np.zeros(40, np.int32)
    for step in range(200):
        kind = r.integers(4)
        slots = r.permutation(12)
        if kind == 0:
            oracle.pages.reserve(table, refs, slots[:3], r.integers(0, 193, 3), 32)
        elif kind == 1:
            oracle.pages.free(table, refs, slots[:2])
        elif kind == 2:
            held = (table[slots[4:6]] >= 0).sum(1) * 32
            _, src, dst = oracle.pages.fork(table, refs, slots[4:6], slots[:2],
                                            np.maximum(0, held - r.integers(0, 32, 2)), 32)
            assert len(set(dst[dst >= 0])) == (dst >= 0).sum() and not set(dst[dst >= 0]) & set(src[src >= 0])
        else:
            _, table, refs, src, dst, counts = oracle.pages.compact(table, refs)
            assert (refs[:counts[0]] > 0).all() and not refs[counts[0]:].any()
        assert np.array_equal(refs, np.bincount(table[table >= 0], minlength=40))


# -------------------------------------------------- sizes past the kernels' 32-bit counts

@pytest.mark.parametrize("name,base", [("reserve_pages", RESERVE), ("free_sequences", FREE),
                                       ("fork_sequences", FORK), ("compact_pages", COMPACT)])
def test_page_operations_refuse_counts_past_32_bits(lib, name, base):
    # run on the host alone: the refusal comes before anything is enqueued
    fn = getattr(lib, "kattn_" + name)
    ok = dict(base, ws_bytes=BIG)
    for arg in ("S", "mp", "n_pages"):
        for size in ((1 << 30) + 1, (1 << 31) - 1):
            assert call(fn, ok, **{arg: size}) == UNSUPPORTED, (arg, size)


def test_diff_workspace_size_of_a_limit_that_the_call_refuses(lib):
    size = lib.kattn_diff_workspace_size
    top = (1 << 31) - 1
    for max_ctx, M in ((top, 1), (top, 8), (top - 6, 8), (top // 2 + 1, 1), (top // 2 - 6, 8)):
        assert size(1, M, 2, max_ctx) == 0, (max_ctx, M)
        assert call(lib.kattn_decode_diff, DIFF, max_ctx=max_ctx, M=M, ws_bytes=BIG) == INVALID
    assert size(1, 8, 2, top // 2 - 7) > 0
