"""A step over the 8-bit cache computes the same bits every time: its sums have one order, so any difference between two
runs on the same inputs is a race (a copy into shared memory ahead of the reads of what was there)."""
import math

import pytest
import torch

import sliding_window_gqa_chunk_b200 as swa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def full(dims, fmt, g):
    """A cache of random bytes and scales, as full sequences hold them; positions of one more token."""
    B, H, W, d = dims.batch, dims.n_kv_heads, dims.window, dims.head_dim
    cache = swa.new_cache_q8(dims, fmt, DEV)
    for x in (cache.k, cache.v):
        y = torch.randn(x.shape, generator=g, device=DEV) * (100.0 if fmt == "e4m3" else 40.0)
        x.copy_(y.clamp(-448, 448).to(x.dtype) if fmt == "e4m3" else y.clamp(-127, 127).round().to(x.dtype))
    for s in (cache.k_scale, cache.v_scale):
        s.copy_(torch.exp2(torch.randint(-8, -5, s.shape, generator=g, device=DEV).float()))
    for t in (cache.k_tail, cache.v_tail):
        t.copy_(torch.randn(t.shape, generator=g, device=DEV))
    pos = torch.randint(W, 8 * W, (B,), generator=g, device=DEV, dtype=torch.int32)
    return cache, pos


# several blocks to each place of the rings, one and several waves of CTAs, each kind of CTA
SHAPES = [(100, 32, 8, 128, 4096), (200, 32, 8, 128, 1000), (64, 64, 4, 128, 4096), (60, 32, 8, 64, 8192), (1, 32, 8, 128, 16384),
          (1, 4, 1, 128, 65536 * 3)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,Hq,H,d,W", SHAPES)
def test_a_decode_step_repeats_itself(B, Hq, H, d, W, fmt):
    g = torch.Generator(device=DEV).manual_seed(B)
    dims = swa.Dims(B, Hq, H, d, W, 1.0 / math.sqrt(d), "f32")
    cache, pos = full(dims, fmt, g)
    q, k, v = (torch.randn(B, h, d, generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, H, H))
    ws = swa.decode_workspace_q8(dims, DEV)
    outs = [torch.empty(B, Hq, d, device=DEV) for _ in range(2)]
    swa.decode_q8(dims, outs[0], q, k, v, cache, pos, ws)
    off = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(60):
        swa.decode_q8(dims, outs[1], q, k, v, cache, pos, ws)        # the row is already there
        off += (outs[1].view(torch.int32) != outs[0].view(torch.int32)).sum()
    assert int(off) == 0
    swa.device_status()


@pytest.mark.parametrize("B,T,Hq,H,d,W", [(64, 4, 32, 8, 128, 4096), (16, 4, 32, 8, 128, 4096), (1, 500, 1, 1, 128, 4096)])
def test_a_few_row_chunk_repeats_itself(B, T, Hq, H, d, W):
    g = torch.Generator(device=DEV).manual_seed(B + T)
    dims = swa.Dims(B, Hq, H, d, W, 1.0 / math.sqrt(d), "f32")
    cache, start = full(dims, "e4m3", g)
    q, k, v = (torch.randn(B, T, h, d, generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, H, H))
    n = torch.full((B,), T, dtype=torch.int32, device=DEV)
    ws = swa.prefill_workspace_q8(dims, T, DEV)
    outs = [torch.empty(B, T, Hq, d, device=DEV) for _ in range(2)]
    swa.prefill_chunk_q8(dims, outs[0], q, k, v, cache, start, n, ws)
    off = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(60):
        swa.prefill_chunk_q8(dims, outs[1], q, k, v, cache, start, n, ws)
        off += (outs[1].view(torch.int32) != outs[0].view(torch.int32)).sum()
    assert int(off) == 0
    swa.device_status()
