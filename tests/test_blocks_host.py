"""Rotary positions and the block-scaled cache without a GPU: what the C ABI and the
binding refuse before anything is enqueued, workspace sizes, frequencies, and pins of
the oracle against something else than itself.
"""

import math

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


# Every call of a refusal test fails, or has nothing to do: with valid arguments the
# workspace (or, for rope, a null pointer) is the error.
TABLE = dict(freq=FAKE, n=100, rot=128, table=None, stream=None)
ROPE = dict(x=FAKE, x_type=0, rows=4, heads=3, d=128, xs=384, pos=None, table=FAKE, n_pos=100, rot=128,
            inter=0, out=FAKE, out_type=0, os=384, stream=None)
APPEND = dict(kn=FAKE, vn=FAKE, x_type=0, rows=4, n_kv=2, d=128, ks_=256, vs_=256, cu=FAKE, start=FAKE, B=2,
              k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, code=0, cap=4096, R=32, bt=FAKE, mp=8, page=64, table=FAKE,
              n_pos=100, rot=128, inter=0, q=FAKE, Hq=4, qs=512, q_out=FAKE, qos=512, ws=FAKE, ws_bytes=0,
              stream=None)
READ = dict(k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, code=0, Hkv=2, d=128, cap=4096, R=32, bt=FAKE, mp=8, page=64,
            cu=FAKE, start=FAKE, B=2, rows=4, out_k=FAKE, out_v=FAKE, out_type=0, ws=FAKE, ws_bytes=0,
            stream=None)
DECODE = dict(q=FAKE, q_type=0, k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, code=0, cap=4096, R=32, bt=FAKE, mp=16,
              page=64, ctx=FAKE, B=2, M=1, Hq=8, Hkv=2, d=128, max_ctx=1000, scale=0.0, out=FAKE, ws=FAKE,
              ws_bytes=0, stream=None)
COPY = dict(k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, Hkv=2, d=128, cap=4096, page=64, R=32, src=FAKE, dst=FAKE, n=3,
            count=None, ws=FAKE, ws_bytes=0, stream=None)


def refused(fn, base, invalid=(), unsupported=()):
    for bad in invalid:
        assert call(fn, base, **bad) == INVALID, bad
    for bad in unsupported:
        assert call(fn, base, **bad) == UNSUPPORTED, bad


def test_rope_refusals(lib):
    t = lib.kattn_rope_table
    assert call(t, TABLE) == INVALID and call(t, TABLE, n=0) == 0
    refused(t, TABLE, [dict(n=-1), dict(rot=0), dict(freq=None, table=FAKE)], [dict(rot=12), dict(rot=136), dict(rot=2)])
    assert call(t, TABLE, table=FAKE + 8) == MISALIGNED and call(t, TABLE, freq=FAKE + 4, table=FAKE) == MISALIGNED
    f = lib.kattn_rope
    assert call(f, ROPE) == INVALID                        # positions missing
    assert call(f, ROPE, rows=0) == call(f, ROPE, heads=0) == 0
    ok = dict(ROPE, pos=FAKE + 2)                          # misaligned positions, the last check
    assert call(f, ok) == MISALIGNED
    refused(f, ok, [dict(x=None), dict(out=None), dict(table=None), dict(x_type=3), dict(x_type=1, out_type=2),
                    dict(out_type=1), dict(rows=-1), dict(heads=-1), dict(xs=380), dict(os=383), dict(n_pos=0),
                    dict(rot=0), dict(inter=2), dict(os=512), dict(x_type=1)],
            [dict(d=64), dict(rot=10), dict(rot=256), dict(rows=2 ** 31 - 1, heads=8)])
    for bad in (dict(x=FAKE + 8), dict(out=FAKE + 8), dict(table=FAKE + 8), dict(xs=386), dict(out=2 * FAKE, os=386)):
        assert call(f, ok, **bad) == MISALIGNED, bad
    half = dict(ok, x_type=1, out=2 * FAKE, out_type=1)    # 16-bit elements: 8 bytes
    assert call(f, half, pos=FAKE + 2, x=FAKE + 4) == MISALIGNED


CACHE_INVALID = [dict(k=None), dict(ks=None), dict(v=None), dict(vs=None), dict(bt=None), dict(code=2),
                 dict(code=-1), dict(cap=0), dict(cap=4100), dict(mp=0), dict(page=0), dict(B=-1), dict(B=65536),
                 dict(R=128)]
CACHE_UNSUPPORTED = [dict(d=64), dict(R=16), dict(R=48), dict(R=256, page=256), dict(page=96), dict(page=16),
                     dict(cap=2 ** 30)]


def test_append_refusals(lib):
    f = lib.kattn_append_blocks
    assert call(f, APPEND) == call(f, APPEND, ws=None, ws_bytes=BIG) == call(f, APPEND, ws=FAKE + 128, ws_bytes=BIG) == WORKSPACE
    assert call(f, APPEND, B=0, k=None) == call(f, APPEND, rows=0, kn=None) == 0
    refused(f, APPEND, CACHE_INVALID + [
        dict(kn=None), dict(vn=None), dict(cu=None), dict(start=None), dict(x_type=3), dict(rows=-1), dict(n_kv=0),
        dict(ks_=252), dict(vs_=255), dict(q=None), dict(q_out=None), dict(table=None), dict(Hq=0), dict(Hq=5),
        dict(qos=508), dict(inter=-1), dict(n_pos=0), dict(rot=0), dict(qs=1024)],
        CACHE_UNSUPPORTED + [dict(rot=20), dict(rot=132), dict(rows=2 ** 31 - 1, n_kv=64, ks_=8192, vs_=8192)])
    for bad in ("kn", "vn", "q_out", "k", "v", "table"):
        assert call(f, APPEND, **{bad: FAKE + 8}) == MISALIGNED, bad
    for bad in ("cu", "start", "ks", "vs", "bt"):
        assert call(f, APPEND, **{bad: FAKE + 2}) == MISALIGNED, bad
    assert call(f, APPEND, ks_=258) == call(f, APPEND, vs_=258) == call(f, APPEND, q=2 * FAKE, qs=514) == MISALIGNED
    # without a table, its arguments are not looked at
    assert call(f, APPEND, table=None, q=None, q_out=None, rot=3, n_pos=-1, inter=9) == WORKSPACE


def test_read_refusals(lib):
    f = lib.kattn_read_blocks
    assert call(f, READ) == call(f, READ, ws=None, ws_bytes=BIG) == WORKSPACE
    assert call(f, READ, B=0, k=None) == call(f, READ, rows=0, out_k=None) == 0
    assert call(f, READ, out_k=None) == call(f, READ, out_v=None) == WORKSPACE
    refused(f, READ, CACHE_INVALID + [dict(Hkv=0), dict(out_type=3), dict(rows=-1), dict(out_k=None, out_v=None),
                                      dict(cu=None), dict(start=None)],
            CACHE_UNSUPPORTED + [dict(rows=2 ** 31 - 1, Hkv=64)])
    for bad in ("out_k", "out_v", "k", "v"):
        assert call(f, READ, **{bad: FAKE + 8}) == MISALIGNED, bad
    for bad in ("cu", "start", "ks", "vs", "bt"):
        assert call(f, READ, **{bad: FAKE + 2}) == MISALIGNED, bad


def test_decode_refusals(lib):
    f = lib.kattn_decode_blocks
    need = lib.kattn_blocks_workspace_size(2, 1, 8, 1000)
    assert call(f, DECODE) == call(f, DECODE, ws_bytes=need - 1) == WORKSPACE
    assert call(f, DECODE, ws_bytes=BIG, ws=FAKE + 128) == call(f, DECODE, ws_bytes=BIG, ws=None) == WORKSPACE
    assert call(f, DECODE, B=0, ws=None) == 0
    refused(f, DECODE, CACHE_INVALID + [
        dict(q=None), dict(out=None), dict(ctx=None), dict(q_type=-1), dict(M=0), dict(Hq=0), dict(Hkv=0),
        dict(Hq=7), dict(max_ctx=0), dict(max_ctx=2 ** 30 + 1), dict(scale=float("nan")), dict(scale=float("inf"))],
        CACHE_UNSUPPORTED + [dict(M=9), dict(Hq=130), dict(Hq=32, M=5),
                             dict(B=65535, max_ctx=2 ** 29, Hkv=64, Hq=64, cap=64 * 1024)])
    for bad in ("q", "out", "k", "v"):
        assert call(f, DECODE, **{bad: FAKE + 8}) == MISALIGNED, bad
    for bad in ("ctx", "ks", "vs", "bt"):
        assert call(f, DECODE, **{bad: FAKE + 2}) == MISALIGNED, bad


def test_copy_refusals(lib):
    f = lib.kattn_copy_block_pages
    assert call(f, COPY) == WORKSPACE
    ok = dict(COPY, ws_bytes=256)
    assert call(f, ok, n=0) == 0
    for arg in ("k", "ks", "v", "vs", "src", "dst"):
        assert call(f, ok, **{arg: None}) == INVALID, arg
        assert call(f, ok, **{arg: FAKE + 2}) == MISALIGNED, arg
    refused(f, ok, [dict(Hkv=0), dict(cap=0), dict(n=-1), dict(page=0), dict(cap=4100), dict(page=32, R=64)],
            [dict(d=64), dict(page=96), dict(R=1), dict(R=16)])


def test_workspace_size(lib):
    size = lib.kattn_blocks_workspace_size
    assert size(1, 1, 1, 1) >= 256
    assert size(4, 8, 64, 9000) >= size(4, 1, 64, 9000) >= size(2, 1, 64, 9000) > 0
    top = (1 << 31) - 1
    for B, M, Hq, ctx in ((0, 1, 2, 1), (1, 0, 2, 1), (1, 9, 2, 1), (1, 1, 0, 1), (1, 1, 2, 0), (1, 1, 2, top),
                          (1, 8, 2, top // 2 - 6)):
        assert size(B, M, Hq, ctx) == 0
    assert size(1, 8, 2, top // 2 - 7) > 0


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    import int8_kv_decode_gb300 as K
    x, i = torch.zeros(2, 3, 128), torch.zeros(2, dtype=torch.int32)
    k, s = torch.zeros((3, 64, 128), dtype=torch.int8), torch.zeros(3, 2)
    cache = (k, s, k, s)
    for bad in (x, x.double(), None):
        with pytest.raises((ValueError, TypeError)):
            K.rope(bad, i, torch.zeros(5, 64, 2))
    with pytest.raises(TypeError):
        K.append_blocks(x.double(), x, i, i, *cache, i, 64)
    with pytest.raises(ValueError):
        K.append_blocks(x, x, i, i, *cache, i, 64)
    with pytest.raises(TypeError):
        K.read_blocks(k.float(), s, k, s, i, 64, i, i, 2)
    with pytest.raises(ValueError):
        K.read_blocks(*cache, i, 64, i, i, 2)
    with pytest.raises(ValueError):
        K.decode_blocks(x[None], *cache, i, 64, i, 1)
    with pytest.raises(TypeError):
        K.decode_blocks(None, *cache, i, 64, i, 1)
    with pytest.raises(ValueError):
        K.alloc_blocks_workspace(1, 9, 8, 100)
    for bad in (dict(rot_dim=12), dict(rot_dim=256), dict(linear=2.0, extend=2.0), dict(base=0.0),
                dict(parts=(4.0, 100, 3, 3))):
        with pytest.raises(ValueError):
            K.rope_frequencies(**bad)


# ------------------------------------------------------------ frequencies

def test_rope_frequencies():
    import int8_kv_decode_gb300 as K
    plain = K.rope_frequencies(64, 10000.0)
    assert len(plain) == 32 and plain[0] == 1.0 and math.isclose(plain[16], 0.01, rel_tol=1e-12)
    assert np.allclose(K.rope_frequencies(64, linear=4.0), np.array(plain) / 4, rtol=1e-15)
    ext = K.rope_frequencies(64, extend=8.0)
    assert ext[0] == 1.0 and math.isclose(ext[-1], plain[-1] / 8, rel_tol=1e-12)
    parts = K.rope_frequencies(128, parts=(8.0, 4096, 1.0, 32.0))
    base = K.rope_frequencies(128)
    turns = [4096 * w / (2 * math.pi) for w in base]
    for p, w, t in zip(parts, base, turns):
        if t >= 32:
            assert p == w
        elif t <= 1:
            assert math.isclose(p, w / 8, rel_tol=1e-12)
        else:
            assert w / 8 < p < w
    assert all(a > b for a, b in zip(parts, parts[1:]))


# ------------------------------------------------------------ oracle pins

@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_is_a_rotation_by_the_positions_difference(interleaved):
    # lengths are kept, and products of rotated rows depend on the distance alone
    r = np.random.default_rng(0)
    freq = [10000.0 ** (-i / 64) for i in range(0, 64, 2)]
    x, y = r.standard_normal((2, 1, 1, 128))

    def at(v, p):
        return oracle.blocks.rotate(v, oracle.blocks.angles(freq, [p]), interleaved, np.float64)[0, 0]
    assert np.isclose(np.linalg.norm(at(x, 70)), np.linalg.norm(x), rtol=1e-6)
    for p, s in ((0, 5), (100, 7), (31, 900)):
        assert np.isclose(at(x, p) @ at(y, p + 11), at(x, s) @ at(y, s + 11), atol=1e-4)
    assert np.array_equal(at(x, 90)[64:], x[0, 0, 64:])
    pair = [0, 1] if interleaved else [0, 32]
    one = np.zeros((1, 1, 128))
    one[0, 0, pair[0]] = 1.0
    z = at(one, 1)
    assert np.allclose(z[pair], [np.cos(1), np.sin(1)], atol=1e-6) and np.count_nonzero(z) == 2


@pytest.mark.parametrize("e4m3", [False, True])
def test_oracle_cache_holds_the_rows(e4m3):
    # written at once, each value is within half a step of its block's scale; row by row,
    # within half a step for each time that it was coded
    r = np.random.default_rng(1)
    x = r.standard_normal((70, 2, 128)).astype(np.float32)
    table = np.array([2, 0, 3, 1])

    def fresh():
        c = {"R": 32, "e4m3": e4m3}
        for n in "kv":
            c[n], c[n + "s"] = np.zeros((2, 128, 128)), np.zeros((2, 4), np.float32)
        return c
    a, b = fresh(), fresh()
    oracle.blocks.append(a, "k", x, 3, table, 32)
    for i in range(70):
        oracle.blocks.append(b, "k", x[i:i + 1], 3 + i, table, 32)
    rows = oracle.blocks.rows_of(table, 32, np.arange(3, 73))
    want = x.transpose(1, 0, 2).astype(np.float64)
    step = np.abs(want) * 2.0 ** -3 if e4m3 else 0.0
    for c, times in ((a, 1), (b, 8)):
        s = c["ks"][:, rows // 32].astype(np.float64)[..., None]
        half = np.maximum(step / 2, s * 2.0 ** -10) if e4m3 else s / 2
        assert (np.abs(oracle.blocks.values(c, "k", rows) - want) <= times * half * 1.001).all()
    assert np.array_equal(a["ks"][:, [2, 0, 3]], b["ks"][:, [2, 0, 3]])


def test_oracle_attention_against_the_row_scaled_oracle():
    # equal scales in every row: both caches hold the same values; queries that int8 holds
    r = np.random.default_rng(2)
    k8, v8 = r.integers(-127, 128, (2, 2, 64, 128)).astype(np.int8)
    q = r.integers(-127, 128, (1, 2, 4, 128)).astype(np.float32)
    q[..., 0] = 127
    ks, vs = np.full((2, 64), 0.001, np.float32), np.full((2, 64), 0.5, np.float32)
    want = oracle.attention.decode(q, k8, ks, v8, vs, np.array([0]), np.array([50]))
    c = {"R": 32, "e4m3": False, "k": k8.astype(np.float64), "v": v8.astype(np.float64), "ks": ks[:, ::32],
         "vs": vs[:, ::32]}
    out, mass, size = oracle.blocks.decode(q, c, np.array([[0, 1]]), 32, [50])
    assert np.allclose(out, want, rtol=1e-4, atol=1e-4 * mass.max())
    assert (mass >= np.abs(out) - 1e-12).all() and (size > 0).all()


def test_sizes_whose_products_pass_32_bits(lib):
    huge = 2 ** 31 - 1
    # g * M = 2^32, more heads than a grid's axis numbers
    assert call(lib.kattn_decode_blocks, DECODE, M=8, Hq=2 ** 29, Hkv=1, ws_bytes=BIG) == UNSUPPORTED
    for heads in (huge, huge - 3, 2 ** 28):
        wide = dict(rows=8, heads=heads, pos=FAKE + 2, xs=heads * 128 + 512, os=heads * 128 + 512)
        assert call(lib.kattn_rope, ROPE, **wide) == UNSUPPORTED, heads
        assert call(lib.kattn_append_blocks, APPEND, rows=8, Hq=heads, qs=heads * 128 + 512,
                    qos=heads * 128 + 512) == UNSUPPORTED, heads
    # a workspace for no call: 0
    size = lib.kattn_blocks_workspace_size
    for sizes in ((65536, 1, 8, 100), (1, 1, huge, 100), (huge, 8, huge, 2 ** 29), (65535, 8, 2 ** 22, 2 ** 29),
                  (65535, 1, 64, 2 ** 29)):
        assert size(*sizes) == 0, sizes
    # the largest that a call takes: its bytes count past 32 bits
    assert size(65535, 8, 8, 4089) == 256 + 65535 * 8 * 8 * (8 * 130 + 3) * 4
