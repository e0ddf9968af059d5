"""The norm with 8-bit output on the GPU against the oracle.

The codes and the stored residual are defined by single float32 roundings, so
they are equal to the oracle's.  The scales carry the float32 sum of d squares:
a thread's own run of at most ceil(d / 32) additions, 10 more across threads,
half of it after the square root, and 5 further roundings, 2^-24 each.
"""

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

TYPES = ["float32", "bfloat16", "float16"]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def make(rows, d, dtype, residual, seed=0, gain=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    t = getattr(torch, dtype)
    x = (gain * torch.randn((rows, d), generator=g)).to(t)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(t)
    res = (2 * torch.randn((rows, d), generator=g)).to(t) if residual else None
    return x, w, res


def check(x, w, res, codes, scales, res_out, group, eps=1e-6):
    """x, w, res on the host; codes, scales, res_out from the GPU."""
    import torch
    h = x
    if res is not None:
        h = (x.float() + res.float()).to(x.dtype)
        assert torch.equal(res_out.cpu().view(torch.uint8), h.view(torch.uint8))
    e4m3 = codes.dtype == torch.float8_e4m3fn
    rows, d = x.shape
    want, scale = oracle.norm.rms_norm_quant(h.float().numpy(), w.float().numpy(), eps, group, e4m3)
    got = codes.float().cpu().numpy().reshape(rows, d)
    assert np.array_equal(got, want)
    s = scales.cpu().numpy().reshape(scale.shape).astype(np.float64)
    tol = ((-(-d // 32) + 10) / 2 + 5) * 2.0 ** -24
    assert (np.abs(s - scale) <= tol * scale + 2.0 ** -149).all()


@pytest.mark.parametrize("d", [1, 2, 7, 31, 32, 33, 127, 128, 255, 256, 257, 1000, 1024, 2047, 2048,
                               2560, 4096, 5000, 8192, 16384, 20001, 40000])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_codes_equal_the_oracle(d, dtype, residual):
    import torch
    import int8_kv_decode_gb300 as K
    x, w, res = make(5, d, dtype, residual, seed=d)
    for out_dtype in (torch.int8, torch.float8_e4m3fn):
        for group in (0, 128) if d % 128 == 0 else (0,):
            rc = None if res is None else res.cuda()
            codes, scales = K.rms_norm_quant(x.cuda(), w.cuda(), residual=rc, group=group,
                                             out_dtype=out_dtype)
            assert scales.shape == ((5, d // 128) if group else (5,))
            check(x, w, res, codes, scales, rc, group)


@pytest.mark.parametrize("rows,d", [(1, 2048), (3, 256), (1000, 256), (301, 2048), (2, 4096), (700, 96)])
@pytest.mark.parametrize("dtype", TYPES)
def test_row_counts_and_residual_out(rows, d, dtype):
    import torch
    import int8_kv_decode_gb300 as K
    x, w, res = make(rows, d, dtype, True, seed=rows)
    rc = res.cuda()
    out = torch.empty_like(rc)
    codes, scales = K.rms_norm_quant(x.cuda(), w.cuda(), residual=rc, residual_out=out, eps=1e-5)
    assert torch.equal(rc.cpu(), res)
    check(x, w, res, codes, scales, out, 0, eps=1e-5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,stride,offset", [(256, 300, 0), (256, 257, 1), (1000, 1024, 8), (2048, 4096, 2048),
                                             (128, 136, 3), (4096, 4104, 0)])
def test_strided_rows_and_odd_offsets(dtype, d, stride, offset):
    import torch
    import int8_kv_decode_gb300 as K
    x, w, res = make(9, d, dtype, True, seed=d + stride)

    def spread(t):
        buf = torch.full((9 * stride + offset,), 99.0, dtype=t.dtype, device="cuda")
        view = buf[offset:].view(9, stride)[:, :d]
        view.copy_(t)
        return buf, view
    _, xv = spread(x)
    rbuf, rv = spread(res)
    codes, scales = K.rms_norm_quant(xv, w.cuda(), residual=rv)
    check(x, w, res, codes, scales, rv, 0)
    rest = rbuf[offset:].view(9, stride)[:, d:]
    assert (rest == 99).all() and (rbuf[:offset] == 99).all()      # nothing between the rows
    if d % 128 == 0:
        for t in (torch.int8, torch.float8_e4m3fn):
            out = torch.empty_like(rv.contiguous())
            rv.copy_(res)
            codes, scales = K.rms_norm_quant(xv, w.cuda(), residual=rv, residual_out=out, group=128,
                                             out_dtype=t)
            check(x, w, res, codes, scales, out, 128)
            assert torch.equal(rv.cpu(), res)


@pytest.mark.parametrize("group", [0, 128])
def test_zero_rows_ties_and_saturation(group):
    # a row of zeros: codes 0, scale 0; halves round to even; the largest element
    # is +-127 (448); a zero group beside others
    import torch
    import int8_kv_decode_gb300 as K
    d = 256
    x = torch.zeros((4, d))
    x[1, :128] = torch.arange(128) - 63.5
    x[1, 0] = -127.0
    x[2] = torch.linspace(-1, 1, d)
    x[3, 5] = -3.0
    w = torch.ones(d)
    for t in (torch.int8, torch.float8_e4m3fn):
        codes, scales = K.rms_norm_quant(x.cuda(), w.cuda(), group=group, out_dtype=t)
        check(x, w, None, codes, scales, None, group)
        assert torch.count_nonzero(codes[0].float()) == 0 and float(scales.reshape(4, -1)[0].sum()) == 0
        assert float(codes[3, 5].float()) == (-127 if t == torch.int8 else -448)


@pytest.mark.parametrize("gain", [2.0 ** -60, 2.0 ** -10, 2.0 ** 10])
def test_small_and_large_values(gain):
    import int8_kv_decode_gb300 as K
    x, w, _ = make(6, 512, "float32", False, gain=gain)
    codes, scales = K.rms_norm_quant(x.cuda(), w.cuda())
    check(x, w, None, codes, scales, None, 0)


def test_many_values_at_the_rounding_borders():
    # quotients within a few float32 steps of n + 1/2 (and of the e4m3 midpoints):
    # the codes are still those of the exact float32 division
    import torch
    import int8_kv_decode_gb300 as K
    r = np.random.default_rng(4)
    rows, d = 64, 4096
    amax = r.uniform(1, 3, (rows, 1)).astype(np.float32)
    for top, t in ((127.0, torch.int8), (448.0, torch.float8_e4m3fn)):
        s0 = (amax / np.float32(top)).astype(np.float32)
        if t == torch.int8:
            mid = r.integers(-126, 126, (rows, d)) + 0.5
        else:
            e = r.integers(-9, 9, (rows, d))
            mid = (1 + (2 * r.integers(0, 8, (rows, d)) + 1) / 16) * 2.0 ** np.maximum(e, -6)
            mid = np.where(e < -6, (r.integers(0, 8, (rows, d)) + 0.5) * 2.0 ** -9, mid)
            mid = np.minimum(mid, 440) * r.choice([-1, 1], (rows, d))
        x = (mid.astype(np.float32) * s0).astype(np.float32)
        x = (x.view(np.int32) + r.integers(-2, 3, x.shape).astype(np.int32)).view(np.float32)
        x[:, 0] = amax[:, 0]
        x = torch.from_numpy(np.clip(x, -amax, amax))
        w = torch.ones(d)
        for group in (0, 128):
            codes, scales = K.rms_norm_quant(x.cuda(), w.cuda(), group=group, out_dtype=t)
            check(x, w, None, codes, scales, None, group)


def test_leading_dimensions_given_outputs_and_graph():
    import torch
    import int8_kv_decode_gb300 as K
    x, w, res = make(24, 256, "bfloat16", True)
    xd, wd, rd = x.cuda().view(2, 3, 4, 256), w.cuda(), res.cuda().view(2, 3, 4, 256)
    codes, scales = K.rms_norm_quant(xd, wd, residual=rd)
    assert codes.shape == (2, 3, 4, 256) and scales.shape == (2, 3, 4)
    check(x, w, res, codes, scales, rd.view(24, 256), 0)
    ro = torch.empty_like(rd)
    rd.copy_(res.view(2, 3, 4, 256))
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    K.rms_norm_quant(xd, wd, residual=rd, residual_out=ro, out=c2, out_scale=s2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.rms_norm_quant(xd, wd, residual=rd, residual_out=ro, out=c2, out_scale=s2)
    c2.zero_(), s2.zero_(), ro.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    x3, _, _ = make(0, 64, "float32", False)
    codes, scales = K.rms_norm_quant(x3.cuda(), torch.ones(64).cuda())
    assert codes.shape == (0, 64) and scales.shape == (0,)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,stride,group", [(256, 257, 0), (256, 257, 128), (255, 255, 0), (256, 256, 0),
                                            (256, 264, 128), (1024, 1025, 0), (4096, 4100, 0), (4097, 4097, 0)])
def test_a_row_alone_has_the_bytes_it_has_in_a_batch(dtype, d, stride, group):
    # a slice of one row keeps the row stride of its buffer
    import torch
    import int8_kv_decode_gb300 as K
    n = 96
    x, w, res = make(n, d, dtype, True, seed=d + stride)

    def spread(t):
        view = torch.zeros((n, stride), dtype=t.dtype, device="cuda")[:, :d]
        view.copy_(t)
        return view
    xv, wc, rv = spread(x), w.cuda(), spread(res)
    out = torch.empty_like(rv)
    codes, scales = K.rms_norm_quant(xv, wc, residual=rv, residual_out=out, group=group)
    check(x, w, res, codes, scales, out, group)
    for i in range(n):
        c, s = K.rms_norm_quant(xv[i:i + 1], wc, residual=rv[i:i + 1],
                                residual_out=torch.empty_like(rv[i:i + 1]), group=group)
        assert torch.equal(c, codes[i:i + 1]) and torch.equal(s, scales[i:i + 1]), i


def test_one_row_views_of_any_stride():
    # a single row whose stride says nothing (a column's transpose, an expanded row), and
    # the same memory as residual and residual_out through views of different strides
    import torch
    import int8_kv_decode_gb300 as K
    x, w, res = make(1, 256, "bfloat16", True, seed=3)
    buf = torch.zeros((4, 257), dtype=torch.bfloat16, device="cuda")
    buf[2, :256] = res[0]
    for xv in (x.cuda(), x.cuda().reshape(256, 1).t(), x.cuda()[0].expand(1, 256),
               x.cuda().as_strided((1, 256), (0, 1))):
        assert xv.shape == (1, 256)
        rv = buf[2:3, :256]
        rv.copy_(res)
        codes, scales = K.rms_norm_quant(xv, w.cuda(), residual=rv, residual_out=rv.view(1, 256))
        check(x, w, res, codes, scales, rv, 0)
        rv.copy_(res)
        codes, scales = K.rms_norm_quant(xv, w.cuda(), residual=rv,
                                         residual_out=rv.as_strided((1, 256), (256, 1)))
        check(x, w, res, codes, scales, rv, 0)
