"""decode_blocks' bounded waits, made to run out on purpose.

A warp whose copy never arrives sets KATTN_DEVERR_TIMEOUT and a flag in shared memory;
the four warps of its block leave at their next barrier, after a bounded wait for what
each has in flight, and tensor memory is given back.  Separate builds of the library
(build.py, build_blocks_timeout_variant) find no copy ready after a number of copies:
one warp at once, another in the middle of a window, all four, and late, after whole
units.  The call returns, the bit is set, and the ordinary library answers on the same
inputs.
"""

import concurrent.futures
import ctypes

import pytest

from test_gpu_blocks import attend, attend_inputs, check_attend, i32, same

pytestmark = pytest.mark.gpu

# Copies taken, warps.  A warp takes 8 copies in a full window (K and V of 4 steps); the
# large calls have 1440 and 1080 units for 456 blocks, so 3 or 4 and 2 or 3 each: 24 copies
# or more in some blocks, which is past the last limit; the others have a unit a block.
VARIANTS = [(0, 2), (3, 1), (4, 15), (21, 8)]


@pytest.fixture(scope="module")
def libs():
    from int8_kv_decode_gb300 import _lib, build
    build.build()
    with concurrent.futures.ThreadPoolExecutor(4) as ex:
        paths = list(ex.map(lambda v: build.build_blocks_timeout_variant(*v), VARIANTS))
    out = []
    for path in paths:
        lib = ctypes.CDLL(path)                   # its own handle: not the package's library
        for name in ("kattn_decode_blocks", "kattn_get_device_status"):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = _lib.SIGNATURES[name]
        out.append(lib)
    return out


@pytest.mark.parametrize("variant", range(len(VARIANTS)))
@pytest.mark.parametrize("B,M,Hq,Hkv,ctx,limit", [
    (2, 1, 8, 2, [120, 300], 300), (3, 2, 16, 2, [1500, 100, 600], 1500), (40, 1, 16, 2, 9000, 9000),
    (30, 5, 16, 2, 9000, 9000), (3, 5, 16, 2, [1500, 700, 2000], 60000)])   # the last two: sums in tensor memory
def test_waits_that_run_out_set_the_bit_and_end(libs, variant, B, M, Hq, Hkv, ctx, limit):
    import torch
    import int8_kv_decode_gb300 as K
    c, table, ctx, q = attend_inputs(B, M, Hq, Hkv, ctx, 32, 64, "int8", "bfloat16", seed=B)
    lib, t, n = libs[variant], i32(table), i32(ctx)
    ws = K.alloc_blocks_workspace(B, M, Hq, limit)
    out = torch.full_like(q, 7.0)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.kattn_decode_blocks(
        q.data_ptr(), 1, c.k.data_ptr(), c.ks.data_ptr(), c.v.data_ptr(), c.vs.data_ptr(), 0, c.k.shape[1], 32,
        t.data_ptr(), table.shape[1], 64, n.data_ptr(), B, M, Hq, Hkv, 128, limit, 0.0, out.data_ptr(),
        ws.data_ptr(), ws.numel(), stream) == 0
    torch.cuda.synchronize()
    err = ctypes.c_int()
    assert lib.kattn_get_device_status(ws.data_ptr(), ws.numel(), ctypes.byref(err), stream) == 0
    if VARIANTS[variant][0] < 8 or B >= 30:
        assert err.value == K.DEVERR_TIMEOUT
    if VARIANTS[variant][0] == 0:                 # no unit of two steps or more was finished
        one = [b for b in range(B) if 32 < ctx[b] and ctx[b] + M - 1 <= 512]
        assert (out[one] == 7.0).all()
    # the context is unharmed: the library proper, on the same workspace
    good = attend(c, table, ctx, q, workspace=ws, max_ctx=limit)
    assert K.get_device_status(ws) == 0
    if B < 30:
        check_attend(c, table, ctx, q, good)
    assert same(good, attend(c, table, ctx, q, max_ctx=limit))
