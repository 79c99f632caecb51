"""A CTA of a cluster that comes late: the others wait for it, end, and the next step is right.

The checked build (waits of about a millisecond) never asks for one tile of a pair's first split.  That split leaves its
own waits after a few milliseconds, which is past the limit of its peers' wait for it.  One of these has a block to round
into the ring at its end."""
import ctypes
import os

import numpy as np
import pytest
import torch

import sliding_window_gqa_chunk_b200 as swa
from oracle import q8
from sliding_window_gqa_chunk_b200.csrc import build as swa_build

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def checked():
    so = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libswa_q8_late.so")
    swa_build.build(force=True, defines=["SWA_TEST_FAULTS", "SWA_WAIT_LIMIT_CYCLES=2000000LL"], out=so)
    lib = ctypes.CDLL(so)
    P, D, C = ctypes.c_void_p, ctypes.POINTER(swa._CDims), ctypes.POINTER(swa._CCacheQ8)
    lib.swa_q8_decode.argtypes = [D, P, P, P, P, C, P, P, ctypes.c_size_t, P]
    lib.swa_device_status.argtypes = [P]
    lib.swa_debug_set_trace.argtypes = [P]
    lib.swa_debug_set_trace.restype = None
    return lib


def test_peers_of_a_late_cta_end_together(checked):
    B, Hq, H, d, W = 2, 4, 2, 64, 1200             # 19 blocks: splits of 7, 7 and 5
    dims = swa.Dims(B, Hq, H, d, W, 0.125, "f32")
    g = torch.Generator().manual_seed(5)
    pos = [W + 9 * 64 + 63, 1023]                  # the last row of a block of the second and of the third split
    cache, ref = swa.new_cache_q8(dims, "e4m3", DEV), q8.RollingCacheQ8(B, H, W, d, "e4m3")

    def rows(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    for s in range(0, max(pos), 400):
        n = [max(0, min(400, p - s)) for p in pos]
        k, v = rows(B, 400, H, d), rows(B, 400, H, d)
        swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([s] * B), i32(n))
        q8.append(ref, k, v, [s] * B, n)
    q, k, v = rows(B, Hq, d), rows(B, H, d), rows(B, H, d)
    qd, kd, vd, pd, ws = q.to(DEV), k.to(DEV), v.to(DEV), i32(pos), swa.decode_workspace_q8(dims, DEV)
    out = torch.zeros((B, Hq, d), device=DEV)

    def step():
        return checked.swa_q8_decode(ctypes.byref(dims._record), out.data_ptr(), qd.data_ptr(), kd.data_ptr(), vd.data_ptr(),
                                     ctypes.byref(cache._record.c), pd.data_ptr(), ws.data_ptr(), ws.numel(), None)

    flag = torch.full((1,), 2, dtype=torch.int32, device=DEV)
    checked.swa_debug_set_trace(flag.data_ptr())
    try:
        for _ in range(3):                         # the row is taken in again, where it already is
            torch.cuda.synchronize()
            assert step() == swa.SWA_OK
            torch.cuda.synchronize()
            assert checked.swa_device_status(None) == swa.SWA_ERR_TIMEOUT
            assert checked.swa_device_status(None) == swa.SWA_OK
        flag.zero_()
        torch.cuda.synchronize()
        assert step() == swa.SWA_OK
        torch.cuda.synchronize()
        assert checked.swa_device_status(None) == swa.SWA_OK
    finally:
        checked.swa_debug_set_trace(None)
    want, spread = q8.decode(ref, q, k, v, pos, dims.scale)
    # weights in f16 and fp32 sums: 2^-10 of the weighted mean of |v| (tests/test_gpu_q8.py)
    assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -10 * spread).all()
    for name in ("k", "v"):                        # the blocks that the late calls filled up
        got = getattr(cache, name).float().double().cpu().numpy()
        held = np.broadcast_to((ref.held >= 0)[:, None, :, None], got.shape)
        np.testing.assert_array_equal(np.where(held, got, 0), np.where(held, getattr(ref, name + "8"), 0))
        np.testing.assert_array_equal(getattr(cache, name + "_scale").cpu().double().numpy(), getattr(ref, name + "_scale"))
