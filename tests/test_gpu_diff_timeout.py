"""decode_diff's bounded waits, made to run out on purpose.

The two warps of a pair wait for their own copies and for each other's weights; a
warp whose copy never arrives tells the other at their next exchange, sets
KATTN_DEVERR_TIMEOUT and leaves, and the other leaves too.  Separate builds of the
library (build.py, build_diff_timeout_variant) find no copy ready after a number of
stages, at once and with nothing left in flight: on map 1 alone at the first, on map
0 alone in the middle of a window, on both, and late, after whole units.  The call
returns, the bit is set, and the ordinary library answers on the same inputs.
"""

import concurrent.futures
import ctypes

import numpy as np
import pytest

from test_gpu_diff import bits, check, device, expected, inputs

pytestmark = pytest.mark.gpu

VARIANTS = [(0, 2), (3, 1), (4, 3), (21, 2)]


@pytest.fixture(scope="module")
def libs():
    from int8_kv_decode_gb300 import _lib, build
    build.build()
    with concurrent.futures.ThreadPoolExecutor(4) as ex:
        paths = list(ex.map(lambda v: build.build_diff_timeout_variant(*v), VARIANTS))
    out = []
    for path in paths:
        lib = ctypes.CDLL(path)                   # its own handle: not the package's library
        for name in ("kattn_decode_diff", "kattn_get_device_status"):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = _lib.SIGNATURES[name]
        out.append(lib)
    return out


@pytest.mark.parametrize("variant", range(len(VARIANTS)))
@pytest.mark.parametrize("B,M,Hq,Hkv,ctx", [(2, 1, 8, 2, [120, 300]), (3, 2, 16, 2, [1500, 100, 600]),
                                            (30, 1, 16, 2, 9000), (30, 3, 16, 2, 16000),
                                            (12, 8, 16, 2, 9000)])
def test_waits_that_run_out_set_the_bit_and_end(libs, variant, B, M, Hq, Hkv, ctx):
    import torch
    import int8_kv_decode_gb300 as K
    x = inputs(B, M, Hq, Hkv, ctx, seed=B)
    t = device(x)
    lib, top = libs[variant], int(x["ctx"].max())
    ws = K.alloc_diff_workspace(B, M, Hq, top)
    out = torch.full((B, M, Hq // 2, 256), 7.0, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.kattn_decode_diff(
        t["q"].data_ptr(), t["k8"].data_ptr(), t["ks"].data_ptr(), t["v8"].data_ptr(),
        t["vs"].data_ptr(), t["start"].data_ptr(), t["ctx"].data_ptr(), t["lam"].data_ptr(), 0, B, M,
        Hq, Hkv, 128, x["cap"], top, 0.0, out.data_ptr(), ws.data_ptr(), ws.numel(), stream) == 0
    torch.cuda.synchronize()
    err = ctypes.c_int()
    assert lib.kattn_get_device_status(ws.data_ptr(), ws.numel(), ctypes.byref(err), stream) == 0
    limit = VARIANTS[variant][0]
    if limit < 16 or B == 30:                     # (21 stages: more than these small calls have)
        assert err.value == K.DEVERR_TIMEOUT
    if limit == 0:                                # no unit was finished: single windows unwritten
        one = [b for b in range(B) if x["ctx"][b] + M - 1 <= 128]
        assert (out[one] == 7.0).all()
    # the context is unharmed: the library proper, on the same workspace
    good = K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"], t["start"], t["ctx"], top, t["lam"],
                         workspace=ws)
    assert K.get_device_status(ws) == 0
    if B < 30:
        want, mass = expected(x)
        check(good.cpu().numpy(), want, mass)
    assert np.array_equal(bits(good), bits(K.decode_diff(t["q"], t["k8"], t["ks"], t["v8"], t["vs"],
                                                         t["start"], t["ctx"], top, t["lam"])))
