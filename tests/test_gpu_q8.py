"""The 8-bit rolling cache on the GPU, against the float64 oracle (oracle/q8.py).

The cache's contents (8-bit numbers, scales, tails) are compared exactly: scales
are powers of two and every rounding is to nearest even, so there is one right
answer.  Attention outputs are held to bounds that follow from the arithmetic:

* decode (and a chunk of few rows) rounds the weights to f16 (half a step: 2^-11 of the
  weight, or 2^-25 where it is subnormal, the largest being 2^15 or 2^14 at least), and does
  the rest in fp32: the scores (d products, d 2^-24 of their sizes' sum), exp2 (2^-22) and
  the sums.  For the scores here (|x| below 2^4) these stay within another 2^-11.  So
  |out - ref| <= 2^-10 S, with S the weighted mean of |v|, plus n 2^-23 of the largest |v|
  for the subnormal weights (a weight is relative to the largest product of weight and value
  scale, and no value exceeds 448 / 224 times what its block's largest one says; 2^-37 would do).
* prefill rounds the weights to bf16 (2^-8), the rest as above: (2^-8 + 2^-10) S.
* bf16 output adds half a step, 2^-8 of the output.
"""
import math

import numpy as np
import pytest
import torch

import sliding_window_gqa_chunk_b200 as swa
from oracle import q8

pytestmark = pytest.mark.gpu
DEV = "cuda"
DECODE_REL, PREFILL_REL = 2.0 ** -10, 2.0 ** -8 + 2.0 ** -10


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def rows(g, *shape, spread=1.0):
    """bf16 rows whose sizes differ from row to row and with a few large channels."""
    x = torch.randn(shape, generator=g) * torch.exp2(spread * torch.randn(shape[:-1] + (1,), generator=g))
    x[..., 0] *= 5.0
    return x.to(torch.bfloat16)


def make(B, Hq, H, d, W, fmt, out="f32", scale=None):
    dims = swa.Dims(B, Hq, H, d, W, scale or 1.0 / math.sqrt(d), out)
    return dims, swa.new_cache_q8(dims, fmt, DEV), q8.RollingCacheQ8(B, H, W, d, fmt)


def same_cache(cache, ref, what=""):
    """The tensors that a later call may read hold what the oracle's do."""
    for name in ("k", "v"):
        got, want = getattr(cache, name).float().cpu().double().numpy(), getattr(ref, name + "8")
        used = np.broadcast_to((ref.held >= 0)[:, None, :, None], got.shape)
        np.testing.assert_array_equal(np.where(used, got, 0), np.where(used, want, 0), err_msg=f"{what} {name}")
        np.testing.assert_array_equal(getattr(cache, name + "_scale").cpu().double().numpy(),
                                      getattr(ref, name + "_scale"), err_msg=f"{what} {name}_scale")
        tail = getattr(cache, name + "_tail").cpu().double().numpy()
        for b, n in enumerate(ref.next % ref.W % q8.BLOCK):     # rows of the block being filled
            np.testing.assert_array_equal(tail[b, :, :n], getattr(ref, name + "_tail")[b, :, :n],
                                          err_msg=f"{what} {name}_tail of sequence {b}")


def close(got, ref, spread, rel, small, what, out="f32"):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    tol = rel * spread + small + (2.0 ** -8 * np.abs(ref) if out == "bf16" else 0.0)
    worst = float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max())
    assert worst <= 1.0, f"{what}: {worst:.2f} of the bound"


def fill(dims, cache, ref, lengths, g, chunk):
    """Appends lengths[b] tokens to each sequence in chunks, to the cache and to the oracle."""
    B, H, d = dims.batch, dims.n_kv_heads, dims.head_dim
    done = [0] * B
    while any(done[b] < lengths[b] for b in range(B)):
        n = [min(chunk, lengths[b] - done[b]) for b in range(B)]
        k, v = rows(g, B, chunk, H, d), rows(g, B, chunk, H, d)
        swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32(done), i32(n))
        q8.append(ref, k, v, done, n)
        done = [a + c for a, c in zip(done, n)]
    return done


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,H,d,W,lengths,chunk", [
    (1, 1, 16, 1, [3], 1),                       # one slot: every token fills its block
    (2, 2, 16, 4, [0, 9], 3),                    # blocks of 4, an empty sequence
    (1, 2, 64, 64, [130], 64),                   # one whole block
    (2, 1, 128, 65, [64, 200], 65),              # a last block of one slot
    (3, 2, 128, 100, [63, 64, 333], 100),        # chunks of a whole ring: its first block comes round twice
    (2, 3, 64, 200, [500, 37], 29),              # odd chunks
    (1, 2, 128, 192, [192 * 2 + 5], 192),
])
def test_append_matches_the_oracle_exactly(fmt, B, H, d, W, lengths, chunk):
    g = torch.Generator().manual_seed(W * 7 + chunk)
    dims, cache, ref = make(B, H, H, d, W, fmt)
    fill(dims, cache, ref, lengths, g, chunk)
    same_cache(cache, ref, f"W={W} chunk={chunk}")
    swa.device_status()


def test_append_does_not_depend_on_the_chunking():
    g = torch.Generator().manual_seed(3)
    dims, one, _ = make(1, 2, 2, 64, 150, "e4m3")
    _, many, _ = make(1, 2, 2, 64, 150, "e4m3")
    k, v = rows(g, 1, 470, 2, 64).to(DEV), rows(g, 1, 470, 2, 64).to(DEV)
    for cache, step in ((one, 150), (many, 7)):
        for s in range(0, 470, step):
            n = min(step, 470 - s)
            swa.cache_append_q8(dims, cache, k[:, s:s + n].contiguous(), v[:, s:s + n].contiguous(), i32([s]), i32([n]))
    for a, b in zip((one.k, one.v), (many.k, many.v)):
        assert torch.equal(a.view(torch.int8), b.view(torch.int8))
    for a, b in zip((one.k_scale, one.v_scale), (many.k_scale, many.v_scale)):
        assert torch.equal(a, b)
    r = 470 % 150 % 64
    assert torch.equal(one.k_tail[:, :, :r], many.k_tail[:, :, :r])
    assert torch.equal(one.v_tail[:, :, :r], many.v_tail[:, :, :r])


@pytest.mark.parametrize("fmt,top", [("e4m3", 448.0), ("int8", 127.0)])
def test_scale_at_its_borders(fmt, top):
    """Largest magnitudes on, just above and far from a power of two times the format's top; zeros; tiny."""
    peaks = [top, top * 2 ** -3, (top + (2 if fmt == "e4m3" else 1)) * 2 ** -3, 1.0, 2.0 ** -30, 2.0 ** -110, 0.0, 3e38]
    B = len(peaks)
    dims, cache, ref = make(B, 1, 1, 16, 64, fmt)
    g = torch.Generator().manual_seed(1)
    k = (torch.rand(B, 64, 1, 16, generator=g) - 0.5)
    k = k * torch.tensor(peaks).view(B, 1, 1, 1)
    k[:, 17, 0, 5] = -torch.tensor(peaks)
    k = k.to(torch.bfloat16)
    swa.cache_append_q8(dims, cache, k.to(DEV), k.flip(1).to(DEV), i32([0] * B), i32([64] * B))
    q8.append(ref, k, k.flip(1), [0] * B, [64] * B)
    same_cache(cache, ref)


def test_append_leaves_the_rest_alone():
    """Padding rows, other sequences and rows of the ring that no token reaches keep their bytes."""
    g = torch.Generator().manual_seed(5)
    dims, cache, ref = make(3, 2, 2, 64, 200, "e4m3")
    before = [t.clone() for t in (cache.k.view(torch.int8), cache.k_scale, cache.k_tail)]
    k, v = rows(g, 3, 100, 2, 64), rows(g, 3, 100, 2, 64)
    k[1, 70:], v[1, 70:] = float("nan"), float("nan")
    swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([0, 0, 0]), i32([0, 70, 0]))
    q8.append(ref, k, v, [0] * 3, [0, 70, 0])
    same_cache(cache, ref)
    for now, old in zip((cache.k.view(torch.int8), cache.k_scale, cache.k_tail), before):
        for b in (0, 2):
            assert torch.equal(now[b], old[b])
    assert float(cache.k_tail[1, :, 6:].float().abs().sum()) == 0.0


DECODE = [
    # B, Hq, H, d, W, lengths (positions of the first step), steps
    (1, 4, 2, 16, 4, [0], 9),
    (2, 2, 2, 16, 1, [0, 5], 2),
    (3, 8, 2, 128, 100, [0, 63, 250], 3),
    (2, 14, 2, 64, 130, [127, 400], 4),            # group of 7, a last block of two slots
    (1, 12, 1, 64, 300, [299], 3),                 # group of 12
    (2, 32, 2, 128, 256, [255, 511], 3),           # group of 16, blocks completed by the first step
    (1, 32, 8, 128, 1024, [2047], 2),              # clusters of 8
    (40, 4, 4, 16, 200, [i * 13 for i in range(40)], 2),    # 160 pairs: splits merged through the workspace
    (150, 2, 1, 64, 64, list(range(150)), 2),
    (300, 1, 1, 16, 130, list(range(300)), 2),              # 300 pairs: two CTAs an SM
    (7, 3, 3, 16, 70, [0, 1, 5, 63, 64, 69, 70], 8),        # a last block of 6 slots, filled up and begun
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,Hq,H,d,W,lengths,steps", DECODE)
def test_decode_matches_the_oracle(fmt, B, Hq, H, d, W, lengths, steps):
    out = "bf16" if fmt == "int8" else "f32"
    g = torch.Generator().manual_seed(B * 31 + W)
    dims, cache, ref = make(B, Hq, H, d, W, fmt, out)
    pos = fill(dims, cache, ref, lengths, g, min(W, 64))
    ws = swa.decode_workspace_q8(dims, DEV)
    for i in range(steps):
        q = torch.randn(B, Hq, d, generator=g).to(torch.bfloat16)
        k, v = rows(g, B, H, d), rows(g, B, H, d)
        o = torch.full((B, Hq, d), float("nan"), dtype=dims.torch_out_dtype, device=DEV)
        swa.decode_q8(dims, o, q.to(DEV), k.to(DEV), v.to(DEV), cache, i32(pos), ws)
        want, spread = q8.decode(ref, q, k, v, pos, dims.scale)
        big = max(float(np.abs(ref.v_tail).max()), float((np.abs(ref.v8).max(axis=(2, 3)) * ref.v_scale.max(axis=2)).max()))
        close(o, want, spread, DECODE_REL, W * 2.0 ** -23 * big, f"step {i}", out)
        same_cache(cache, ref, f"step {i}")
        pos = [p + 1 for p in pos]
    swa.device_status()


@pytest.mark.parametrize("scales", ["values far apart", "queries far apart", "tiny", "huge"])
def test_decode_with_values_of_very_different_sizes(scales):
    """Blocks whose values differ by 2^40 (a block with small weights may hold the largest products, and the
    other way round), queries of 2^-60 and 2^60, rows near the ends of bf16's range."""
    B, Hq, H, d, W = 2, 4, 1, 64, 256
    g = torch.Generator().manual_seed(11)
    dims, cache, ref = make(B, Hq, H, d, W, "e4m3")
    k, v = rows(g, B, W, H, d, spread=0.0) * 0.5, rows(g, B, W, H, d, spread=0.0)
    q = torch.randn(B, Hq, d, generator=g)
    if scales == "values far apart":
        v = v * torch.exp2(torch.tensor([-20.0, 20.0, 0.0, -10.0])).repeat_interleave(64).view(1, W, 1, 1)
    elif scales == "queries far apart":
        q, k = q * torch.exp2(torch.tensor([-60.0, 60.0])).view(2, 1, 1), k * torch.exp2(torch.tensor([60.0, -60.0])).view(2, 1, 1, 1)
    elif scales == "tiny":
        v = v * 2.0 ** -90
    else:
        v = v * 2.0 ** 100
    q, k, v = q.to(torch.bfloat16), k.to(torch.bfloat16), v.to(torch.bfloat16)
    n = W - 20
    swa.cache_append_q8(dims, cache, k[:, :n].contiguous().to(DEV), v[:, :n].contiguous().to(DEV), i32([0] * B), i32([n] * B))
    q8.append(ref, k[:, :n], v[:, :n], [0] * B, [n] * B)
    o = torch.empty((B, Hq, d), dtype=torch.float32, device=DEV)
    swa.decode_q8(dims, o, q.to(DEV), k[:, n].to(DEV), v[:, n].to(DEV), cache, i32([n] * B), swa.decode_workspace_q8(dims, DEV))
    want, spread = q8.decode(ref, q, k[:, n], v[:, n], [n] * B, dims.scale)
    big = float(np.abs(v.double().numpy()).max())
    # weights are at most 1 for the largest product of weight and block size: errors of the small ones are relative to it
    close(o, want, spread, DECODE_REL, W * 2.0 ** -23 * float(spread.max()) if scales == "values far apart" else W * 2.0 ** -23 * big, scales)


def test_decode_does_not_read_masked_rows():
    """Rows that no position holds, and what a new block has not been given yet, may be anything, NaN too."""
    B, Hq, H, d, W = 2, 8, 2, 128, 192
    g = torch.Generator().manual_seed(8)
    dims, cache, ref = make(B, Hq, H, d, W, "e4m3")
    cache.k.view(torch.int8).fill_(127)          # NaN in e4m3
    cache.v.view(torch.int8).fill_(127)
    for t in (cache.k_scale, cache.v_scale, cache.k_tail, cache.v_tail):
        t.fill_(float("nan"))
    pos = [0, 70]
    k, v = rows(g, B, 70, H, d), rows(g, B, 70, H, d)
    swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([0, 0]), i32(pos))
    q8.append(ref, k, v, [0, 0], pos)
    ws = swa.decode_workspace_q8(dims, DEV).fill_(255)
    pws = swa.prefill_workspace_q8(dims, 8, DEV)
    for i in range(3):
        q, k1, v1 = torch.randn(B, Hq, d, generator=g).to(torch.bfloat16), rows(g, B, H, d), rows(g, B, H, d)
        qc, kc, vc = (x[:, None].expand(-1, 8, -1, -1).contiguous() for x in (q, k1, v1))
        oc = torch.full((B, 8, Hq, d), 7.0, dtype=torch.float32, device=DEV)
        swa.prefill_chunk_q8(dims, oc, qc.to(DEV), kc.to(DEV), vc.to(DEV), cache, i32(pos), i32([1, 1]), pws)
        o = torch.empty((B, Hq, d), dtype=torch.float32, device=DEV)
        swa.decode_q8(dims, o, q.to(DEV), k1.to(DEV), v1.to(DEV), cache, i32(pos), ws)
        want, spread = q8.decode(ref, q, k1, v1, pos, dims.scale)
        close(o, want, spread, DECODE_REL, W * 2.0 ** -23 * 200, f"decode {i}")
        close(oc[:, 0], want, spread, PREFILL_REL, 0.0, f"one-token chunk {i}")
        assert bool((oc[:, 1:] == 7.0).all())
        pos = [p + 1 for p in pos]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,Hq,H,d,W,T,starts,counts", [
    (1, 4, 2, 16, 4, 4, [0], [4]),
    (1, 4, 2, 16, 4, 3, [6], [3]),
    (3, 8, 2, 128, 200, 77, [0, 63, 500], [77, 1, 40]),
    (2, 6, 2, 64, 320, 320, [321, 64], [320, 0]),      # a chunk of the whole window
    (2, 4, 4, 128, 1000, 130, [130, 990], [130, 130]),
    (4, 16, 2, 128, 640, 4, [1, 639, 640, 1300], [4, 4, 2, 3]),   # a few tokens each
    (3, 14, 2, 64, 300, 9, [0, 5, 700], [9, 9, 9]),
    (2, 2, 2, 64, 64, 64, [64, 31], [64, 64]),              # 64 columns of a window of one block: every row outlives one
    (3, 4, 4, 16, 70, 70, [0, 69, 211], [70, 33, 70]),      # a short last block, rows that see only the chunk's end
    (2, 16, 1, 64, 130, 8, [129, 260], [8, 5]),             # 128 columns: 8 CTAs share them
    (1, 3, 1, 128, 1000, 2, [999], [2]),                    # 6 columns, clusters
    (160, 2, 1, 16, 64, 3, list(range(160)), [i % 4 for i in range(160)]),   # more pairs than SMs, some without rows
    (2, 1, 1, 128, 200, 128, [63, 137], [128, 128]),        # 128 columns
    (2, 1, 1, 128, 200, 129, [63, 137], [129, 129]),        # a ninth CTA for one column
    # over the bytes with several rounds of each warp's ring for the chunk's own rows
    (1, 1, 1, 16, 600, 512, [1234], [512]),
    (1, 3, 1, 64, 700, 300, [330], [299]),
    (2, 2, 1, 128, 520, 400, [519, 1039], [400, 337]),
    (3, 32, 8, 16, 200, 40, [17, 0, 555], [40, 39, 3]),     # two waves
    (3, 12, 12, 128, 130, 33, [64, 500, 129], [33, 0, 30]),
    # written out
    (3, 8, 8, 16, 200, 130, [17, 0, 555], [130, 129, 5]),
    (4, 8, 4, 64, 300, 150, [299, 1, 64, 1000], [150, 128, 129, 77]),
    (3, 16, 8, 128, 260, 77, [259, 12, 640], [77, 77, 1]),
    (1, 1, 1, 128, 700, 513, [365], [513]),
    (1, 4, 1, 64, 1000, 600, [2000], [600]),
])
def test_prefill_matches_the_oracle(fmt, B, Hq, H, d, W, T, starts, counts):
    out = "bf16" if fmt == "int8" else "f32"
    g = torch.Generator().manual_seed(W + T)
    dims, cache, ref = make(B, Hq, H, d, W, fmt, out)
    fill(dims, cache, ref, starts, g, min(W, 64))
    ws = swa.prefill_workspace_q8(dims, T, DEV)
    q = torch.randn(B, T, Hq, d, generator=g).to(torch.bfloat16)
    k, v = rows(g, B, T, H, d), rows(g, B, T, H, d)
    for again in range(2):      # the workspace serves the next call as it is left
        o = torch.full((B, T, Hq, d), 3.0, dtype=dims.torch_out_dtype, device=DEV)
        swa.prefill_chunk_q8(dims, o, q.to(DEV), k.to(DEV), v.to(DEV), cache, i32(starts), i32(counts), ws)
        want, spread = q8.prefill_chunk(ref, q, k, v, starts, counts, dims.scale)
        for b in range(B):
            n = counts[b]
            assert bool((o[b, n:] == 3.0).all())
            if n:
                close(o[b, :n], want[b, :n], spread[b, :n], PREFILL_REL, 1e-6, f"sequence {b}", out)
    same_cache(cache, ref)
    swa.device_status()


@pytest.mark.parametrize("pairs", [1, 14, 15, 16, 18, 19, 22, 23, 26, 27, 33, 34, 45, 46, 74, 75, 147])
def test_pairs_in_clusters_of_every_size(pairs):
    """From one pair in a cluster of 8 to as many as need an SM each, a decode step and a chunk."""
    d, W, pos = 16, 64 * 64, [6000 + 37 * b for b in range(pairs)]
    g = torch.Generator().manual_seed(pairs)
    dims, cache, ref = make(pairs, 1, 1, d, W, "int8")
    fill(dims, cache, ref, pos, g, W)
    q, k, v = torch.randn(pairs, 3, 1, d, generator=g).to(torch.bfloat16), rows(g, pairs, 3, 1, d), rows(g, pairs, 3, 1, d)
    o = torch.empty((pairs, 3, 1, d), dtype=torch.float32, device=DEV)
    swa.prefill_chunk_q8(dims, o, q.to(DEV), k.to(DEV), v.to(DEV), cache, i32(pos), i32([3] * pairs),
                         swa.prefill_workspace_q8(dims, 3, DEV))
    want, spread = q8.prefill_chunk(ref, q, k, v, pos, [3] * pairs, dims.scale)
    close(o, want, spread, DECODE_REL, W * 2.0 ** -37 * 500, "chunk")
    o = torch.empty((pairs, 1, d), dtype=torch.float32, device=DEV)
    q1, k1, v1 = (t[:, 0].contiguous() for t in (q, k, v))
    swa.decode_q8(dims, o, q1.to(DEV), k1.to(DEV), v1.to(DEV), cache, i32(pos), swa.decode_workspace_q8(dims, DEV))
    want, spread = q8.decode(ref, q1, k1, v1, pos, dims.scale)
    # the subnormal weights' part, W 2^-37 of the largest |v| (see above)
    close(o, want, spread, DECODE_REL, W * 2.0 ** -37 * 500, "decode")
    same_cache(cache, ref)
    swa.device_status()


def test_decode_of_a_long_window_goes_over_all_sms():
    """More than 512 blocks and one pair: partials in the workspace, merged by the second kernel."""
    B, Hq, H, d, W = 1, 4, 1, 16, 32768 + 70
    g = torch.Generator().manual_seed(77)
    dims, cache, ref = make(B, Hq, H, d, W, "int8")
    assert swa.decode_workspace_size_q8(dims) > 16
    pos = fill(dims, cache, ref, [W + 100], g, W)
    ws = swa.decode_workspace_q8(dims, DEV).fill_(255)       # what it holds before does not matter
    for i in range(2):
        q, k, v = torch.randn(B, Hq, d, generator=g).to(torch.bfloat16), rows(g, B, H, d), rows(g, B, H, d)
        o = torch.empty((B, Hq, d), dtype=torch.float32, device=DEV)
        swa.decode_q8(dims, o, q.to(DEV), k.to(DEV), v.to(DEV), cache, i32(pos), ws)
        want, spread = q8.decode(ref, q, k, v, pos, dims.scale)
        # the subnormal weights' part, W 2^-37 of the largest |v| (see above)
        close(o, want, spread, DECODE_REL, W * 2.0 ** -37 * 500, f"step {i}")
        pos = [p + 1 for p in pos]
    swa.device_status()


def test_decode_writes_nothing_else():
    """Bytes around every tensor that a step writes, and the rows that it must leave, stay as they were."""
    B, Hq, H, d, W = 3, 4, 2, 64, 100
    dims = swa.Dims(B, Hq, H, d, W, 0.125, "bf16")
    g = torch.Generator(device=DEV).manual_seed(6)
    shapes = [((B, H, W, d), torch.int8), ((B, H, W, d), torch.int8), ((B, H, 2), torch.float32), ((B, H, 2), torch.float32),
              ((B, H, 64, d), torch.bfloat16), ((B, H, 64, d), torch.bfloat16), ((B, Hq, d), torch.bfloat16)]
    guarded = []
    for shape, dtype in shapes:
        n = math.prod(shape)
        whole = torch.full((n + 512,), 1, dtype=dtype, device=DEV)
        guarded.append((whole, whole[256:256 + n].view(shape)))
    cache, out = swa.CacheQ8(*[x[1] for x in guarded[:6]]), guarded[6][1]
    ws = swa.decode_workspace_q8(dims, DEV)
    pos = [0, 63, 250]          # into the tail; fills a block of 64; into the tail of a running ring
    before = [x[0].clone() for x in guarded]
    rnd = lambda h: torch.randn(B, h, d, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    k, v = rnd(H), rnd(H)
    swa.decode_q8(dims, out, rnd(Hq), k, v, cache, i32(pos), ws)
    for i, ((whole, inner), old) in enumerate(zip(guarded, before)):
        n = inner.numel()
        assert torch.equal(whole[:256], old[:256]) and torch.equal(whole[256 + n:], old[256 + n:])
        was = old[256:256 + n].view(inner.shape)
        if i < 2:
            assert torch.equal(inner[0], was[0]) and torch.equal(inner[2], was[2]) and torch.equal(inner[1, :, 64:], was[1, :, 64:])
        elif i < 4:
            assert torch.equal(inner[0], was[0]) and torch.equal(inner[2], was[2]) and torch.equal(inner[1, :, 1], was[1, :, 1])
        elif i < 6:
            new = k if i == 4 else v
            want = was.clone()
            want[0, :, 0], want[2, :, 50] = new[0], new[2]
            assert torch.equal(inner, want)
    swa.device_status()


def test_two_streams_with_their_own_workspaces():
    """Two layers' steps at the same time on two streams give what they give one after the other."""
    B, Hq, H, d, W = 4, 8, 2, 128, 512
    dims = swa.Dims(B, Hq, H, d, W, 0.1, "f32")
    g = torch.Generator(device=DEV).manual_seed(12)

    def layer():
        cache = swa.new_cache_q8(dims, "e4m3", DEV)
        k, v = (torch.randn(B, W, H, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
        swa.cache_append_q8(dims, cache, k, v, i32([0] * B), i32([W] * B))
        q = torch.randn(B, Hq, d, generator=g, device=DEV).to(torch.bfloat16)
        return cache, q, k[:, 3].contiguous(), v[:, 5].contiguous()

    layers, pos = [layer() for _ in range(2)], i32([W] * B)
    alone, together = [], []
    for cache, q, k, v in layers:
        o = torch.empty((B, Hq, d), device=DEV)
        swa.decode_q8(dims, o, q, k, v, cache, pos, swa.decode_workspace_q8(dims, DEV))
        alone.append(o)
    torch.cuda.synchronize()
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [swa.decode_workspace_q8(dims, DEV) for _ in range(2)]
    outs = [torch.empty((B, Hq, d), device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):          # the same step again: the row is already there
        for (cache, q, k, v), s, ws, o in zip(layers, streams, spaces, outs):
            swa.decode_q8(dims, o, q, k, v, cache, pos, ws, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(alone, outs):
        assert torch.equal(a, b)
    swa.device_status()


def test_binding_refuses_what_does_not_fit():
    dims, cache, _ = make(2, 4, 2, 64, 128, "e4m3")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
    ws, pos, o = swa.decode_workspace_q8(dims, DEV), i32([0, 0]), z(2, 4, 64, dt=torch.float32)
    q, k = z(2, 4, 64), z(2, 2, 64)
    good = dict(out=o, q=q, k_new=k, v_new=k.clone(), cache=cache, pos=pos, workspace=ws)
    swa.decode_q8(dims, **good)
    for name, bad in (("out", z(2, 4, 64)), ("q", z(2, 4, 32)), ("q", q.float()), ("k_new", z(2, 4, 64)), ("v_new", z(2, 2, 64).cpu()),
                      ("k_new", z(2, 64, 2).transpose(1, 2)), ("pos", pos.long()), ("pos", i32([0])), ("workspace", ws.cpu())):
        with pytest.raises(ValueError, match=name):
            swa.decode_q8(dims, **{**good, name: bad})
    other = swa.Dims(2, 4, 2, 64, 192, 0.1, "f32")
    with pytest.raises(ValueError, match="cache"):
        swa.decode_q8(other, **good)
    with pytest.raises(ValueError, match="k_scale"):
        swa.CacheQ8(cache.k, cache.v, cache.k_scale[:, :, :1].contiguous(), cache.v_scale, cache.k_tail, cache.v_tail)
    with pytest.raises(ValueError, match="v: "):
        swa.CacheQ8(cache.k, cache.v.view(torch.int8), cache.k_scale, cache.v_scale, cache.k_tail, cache.v_tail)
    with pytest.raises(swa.SwaError) as e:
        swa.prefill_chunk_q8(dims, z(2, 1, 4, 64, dt=torch.float32), z(2, 1, 4, 64), z(2, 1, 2, 64), z(2, 1, 2, 64), cache, pos, pos, ws)
    assert e.value.code == swa.SWA_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(ValueError, match="n_tokens"):
        swa.cache_append_q8(dims, cache, z(2, 1, 2, 64), z(2, 1, 2, 64), pos, i32([1]))
    with pytest.raises(swa.SwaError):
        swa.cache_append_q8(dims, cache, z(2, 129, 2, 64), z(2, 129, 2, 64), pos, pos)
    spec = swa.new_rope(64, device=DEV)
    x, y = z(2, 3, 4, 64), z(2, 3, 2, 64)
    with pytest.raises(ValueError, match="k and k_out"):
        swa.rope(dims, spec, x, None, x, y, pos)
    with pytest.raises(ValueError, match="q: "):
        swa.rope(dims, spec, x, y, z(2, 3, 4, 128)[..., ::2], y, pos)
    with pytest.raises(ValueError, match="q_out"):
        swa.rope(dims, spec, z(2, 3, 64, 4).transpose(2, 3), y, x, y, pos)
    with pytest.raises(swa.SwaError):
        swa.rope(dims, swa.new_rope(8, device=DEV), x, y, x, y, pos)
    with pytest.raises(swa.SwaError):      # one row for all tokens: rows on top of one another
        swa.rope(dims, spec, x, y, z(1, 1, 4, 64).expand(2, 3, 4, 64), y, pos)
    swa.device_status()


def test_prefill_append_decode_together_with_rotary_positions():
    """A prompt in chunks, then decode steps, q and k turned to their positions in place: as a model's layer
    uses the calls, captured in a graph for the decode steps, on another stream than the default one."""
    B, Hq, H, d, W, T, chunk, steps = 2, 8, 2, 128, 160, 300, 100, 70
    g = torch.Generator().manual_seed(21)
    dims, cache, ref = make(B, Hq, H, d, W, "e4m3")
    spec = swa.new_rope(64, base=10000.0, scaling="yarn", scale=4.0, original_length=512, device=DEV)
    freq = spec.inv_freq.cpu().numpy()
    lengths = [T, T - 83]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pws, ws = swa.prefill_workspace_q8(dims, chunk, DEV), swa.decode_workspace_q8(dims, DEV)
        for s in range(0, T, chunk):
            n = [max(0, min(chunk, x - s)) for x in lengths]
            q = torch.randn(B, chunk, Hq, d, generator=g).to(torch.bfloat16)
            k, v = rows(g, B, chunk, H, d), rows(g, B, chunk, H, d)
            qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
            swa.rope(dims, spec, qd, kd, qd, kd, i32([s] * B), i32(n))
            o = torch.zeros((B, chunk, Hq, d), dtype=torch.float32, device=DEV)
            swa.prefill_chunk_q8(dims, o, qd, kd, vd, cache, i32([s] * B), i32(n), pws)
            swa.cache_append_q8(dims, cache, kd, vd, i32([s] * B), i32(n))
            at = s + np.arange(chunk)
            for x, y in ((q, qd), (k, kd)):
                for b in range(B):
                    want = q8.rope(x[b, :n[b]], at[:n[b]], freq, False, spec.factor)
                    got = y[b, :n[b]].double().cpu().numpy()
                    size = 2.0 * spec.factor * np.abs(x.double().numpy()[b, :n[b]]).max(axis=-1, keepdims=True) if n[b] else 0
                    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size).all()
            qr, kr = qd.cpu(), kd.cpu()          # the library's own rounding of the turned rows goes to the oracle
            want, spread = q8.prefill_chunk(ref, qr, kr, v, [s] * B, n, dims.scale)
            for b in range(B):
                if n[b]:
                    close(o[b, :n[b]], want[b, :n[b]], spread[b, :n[b]], PREFILL_REL, 1e-6, f"chunk at {s}, sequence {b}")
            q8.append(ref, kr, v, [s] * B, n)
        same_cache(cache, ref, "after the prompt")
        pos = i32(lengths)
        qd = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device=DEV)
        kd, vd = (torch.zeros((B, H, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        qi, ki = torch.zeros_like(qd), torch.zeros_like(kd)
        o = torch.zeros((B, Hq, d), dtype=torch.float32, device=DEV)
        other = swa.new_cache_q8(dims, "e4m3", DEV)      # the kernels' first launches come before the capture
        swa.rope(dims, spec, qd[:, None], kd[:, None], qi[:, None], ki[:, None], pos)
        swa.decode_q8(dims, o, qd, kd, vd, other, torch.zeros_like(pos), ws)
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            swa.rope(dims, spec, qd[:, None], kd[:, None], qi[:, None], ki[:, None], pos)
            swa.decode_q8(dims, o, qd, kd, vd, cache, pos, ws)
            pos.add_(1)
        for i in range(steps):
            q, k, v = torch.randn(B, Hq, d, generator=g).to(torch.bfloat16), rows(g, B, H, d), rows(g, B, H, d)
            qi.copy_(q)
            ki.copy_(k)
            vd.copy_(v)
            graph.replay()
            want, spread = q8.decode(ref, qd.cpu(), kd.cpu(), v, [x + i for x in lengths], dims.scale)
            close(o, want, spread, DECODE_REL, W * 2.0 ** -23 * 200, f"replay {i}")
        same_cache(cache, ref, "after the replays")
    swa.device_status()


def test_many_pairs_and_a_cache_past_32_bits():
    """A ring whose byte offsets pass 2^32: the last sequence's rows, against the same rows in a small cache."""
    B, H, d, W = 33, 1, 128, 1 << 20
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    dims = swa.Dims(B, 4, H, d, W, 1.0 / math.sqrt(d), "f32")
    one = swa.Dims(1, 4, H, d, W, 1.0 / math.sqrt(d), "f32")
    big, small = swa.new_cache_q8(dims, "int8", DEV), swa.new_cache_q8(one, "int8", DEV)
    for c in (big, small):      # the earlier positions' blocks: zeros, whose scale is 1
        c.k_scale.fill_(1.0)
        c.v_scale.fill_(1.0)
    g = torch.Generator(device=DEV).manual_seed(2)
    T, s0 = 300, W - 100
    k, v = (torch.randn(B, T, H, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    n = [0] * (B - 1) + [T]
    swa.cache_append_q8(dims, big, k, v, i32([s0] * B), i32(n))
    swa.cache_append_q8(one, small, k[-1:].contiguous(), v[-1:].contiguous(), i32([s0]), i32([T]))
    assert torch.equal(big.k[-1:], small.k) and torch.equal(big.v[-1:], small.v)
    assert int((big.k[0] != 0).sum()) == 0
    q = torch.randn(B, 4, d, generator=g, device=DEV).to(torch.bfloat16)
    o, o1 = torch.zeros(B, 4, d, device=DEV), torch.zeros(1, 4, d, device=DEV)
    pos = i32([3] * (B - 1) + [s0 + T])
    swa.decode_q8(dims, o, q, k[:, 0].contiguous(), v[:, 0].contiguous(), big, pos, swa.decode_workspace_q8(dims, DEV))
    swa.decode_q8(one, o1, q[-1:].contiguous(), k[-1:, 0].contiguous(), v[-1:, 0].contiguous(), small, i32([s0 + T]),
                  swa.decode_workspace_q8(one, DEV))
    # other splits, so other orders of fp32 sums over the same weights, but some 1e6 of them: W 2^-24 of them at most
    assert float((o[-1] - o1[0]).abs().max()) <= 2.0 ** -10 * float(v.float().abs().max())
    swa.device_status()


def test_bad_device_arguments_skip_the_sequence():
    dims, cache, _ = make(2, 2, 2, 64, 128, "e4m3")
    g = torch.Generator().manual_seed(4)
    k, v, q = (rows(g, 2, 8, 2, 64).to(DEV) for _ in range(3))
    for start, n in (([-1, 0], [4, 4]), ([0, 0], [9, 4]), ([0, 0], [-1, 4])):
        cache.k.view(torch.int8).zero_()
        cache.k_tail.zero_()
        o = torch.full((2, 8, 2, 64), 9.0, device=DEV)
        swa.cache_append_q8(dims, cache, k, v, i32(start), i32(n))
        with pytest.raises(swa.SwaError) as e:
            swa.device_status()
        assert e.value.code == swa.SWA_ERR_DEVICE_ARG
        assert float(cache.k_tail[0].float().abs().sum()) == 0.0 and torch.equal(cache.k_tail[1, :, :4], k[1, :4].transpose(0, 1))
        swa.prefill_chunk_q8(dims, o, q, k, v, cache, i32(start), i32(n), swa.prefill_workspace_q8(dims, 8, DEV))
        with pytest.raises(swa.SwaError):
            swa.device_status()
        assert bool((o[0] == 9.0).all())
    o = torch.full((2, 2, 64), 9.0, device=DEV)
    swa.decode_q8(dims, o, q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), cache, i32([-5, 0]),
                  swa.decode_workspace_q8(dims, DEV))
    with pytest.raises(swa.SwaError):
        swa.device_status()
    assert bool((o[0] == 9.0).all())
    torch.testing.assert_close(o[1], v[1, 0].float(), rtol=2.0 ** -10, atol=0)     # one key: the output is its value


@pytest.mark.parametrize("B,H", [(19, 8), (37, 8), (41, 8), (70, 8), (5, 30)])
def test_decode_in_every_variant_is_the_same_sequence_by_sequence(B, H):
    """Batches that are spread over the SMs in different ways (one to three CTAs an SM, several waves, clusters): a
    sequence's step does not depend on its neighbours beyond the order of fp32 sums."""
    Hq, d, W = 2 * H, 64, 200
    g = torch.Generator(device=DEV).manual_seed(B)
    dims, one = (swa.Dims(n, Hq, H, d, W, 0.125, "f32") for n in (B, 1))
    cache = swa.new_cache_q8(dims, "e4m3", DEV)
    start = torch.randint(0, 500, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    for s in range(0, 500, W):
        n = [max(0, min(W, x - s)) for x in start]
        k, v = (torch.randn(B, W, H, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
        swa.cache_append_q8(dims, cache, k, v, i32([s] * B), i32(n))
    q, k, v = (torch.randn(B, h, d, generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, H, H))
    parts = [cache.k, cache.v, cache.k_scale, cache.v_scale, cache.k_tail, cache.v_tail]
    single = [swa.CacheQ8(*[(t.view(torch.int8) if t.dtype == torch.float8_e4m3fn else t)[b:b + 1].clone().view(t.dtype)
                            for t in parts]) for b in range(B)]
    out = torch.empty(B, Hq, d, device=DEV)
    swa.decode_q8(dims, out, q, k, v, cache, i32(start), swa.decode_workspace_q8(dims, DEV))
    for b in range(B):
        o = torch.empty(1, Hq, d, device=DEV)
        swa.decode_q8(one, o, q[b:b + 1], k[b:b + 1], v[b:b + 1], single[b], i32([start[b]]), swa.decode_workspace_q8(one, DEV))
        # weights of f16, each within 2^-11, twice
        assert float((o[0] - out[b]).abs().max()) <= 2.0 ** -10 * 5.0
        assert torch.equal(single[b].k.view(torch.int8)[0], cache.k.view(torch.int8)[b])
        assert torch.equal(single[b].k_tail[0], cache.k_tail[b]) and torch.equal(single[b].v_scale[0], cache.v_scale[b])
    swa.device_status()


def test_a_wait_that_runs_out_is_reported_and_the_next_step_is_right():
    """The checked build (waits of about a millisecond) never asks for one warp's first tile: the step reports a timeout,
    every warp leaves through the merge, and with the switch off the same library gives the oracle's step."""
    import ctypes
    import os

    from sliding_window_gqa_chunk_b200.csrc import build as swa_build

    so = swa_build.build(force=True, defines=["SWA_TEST_FAULTS", "SWA_WAIT_LIMIT_CYCLES=2000000LL"],
                         out=os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libswa_q8_faults.so"))
    lib = ctypes.CDLL(so)
    P, D, C = ctypes.c_void_p, ctypes.POINTER(swa._CDims), ctypes.POINTER(swa._CCacheQ8)
    lib.swa_q8_decode.argtypes = [D, P, P, P, P, C, P, P, ctypes.c_size_t, P]
    lib.swa_device_status.argtypes = [P]
    lib.swa_debug_set_trace.argtypes = [P]
    lib.swa_debug_set_trace.restype = None
    B, Hq, H, d, W = 2, 4, 2, 64, 1200          # clusters of several CTAs
    g = torch.Generator().manual_seed(9)
    dims, cache, ref = make(B, Hq, H, d, W, "e4m3")
    pos = fill(dims, cache, ref, [W + 30, 900], g, 400)
    q, k, v = torch.randn(B, Hq, d, generator=g).to(torch.bfloat16), rows(g, B, H, d), rows(g, B, H, d)
    qd, kd, vd, pd, ws = q.to(DEV), k.to(DEV), v.to(DEV), i32(pos), swa.decode_workspace_q8(dims, DEV)
    o = torch.zeros((B, Hq, d), device=DEV)

    def step():
        return lib.swa_q8_decode(ctypes.byref(dims._record), o.data_ptr(), qd.data_ptr(), kd.data_ptr(), vd.data_ptr(),
                                 ctypes.byref(cache._record.c), pd.data_ptr(), ws.data_ptr(), ws.numel(), None)

    flag = torch.ones(1, dtype=torch.int32, device=DEV)
    lib.swa_debug_set_trace(flag.data_ptr())
    try:
        torch.cuda.synchronize()
        assert step() == swa.SWA_OK
        torch.cuda.synchronize()
        assert lib.swa_device_status(None) == swa.SWA_ERR_TIMEOUT
        assert lib.swa_device_status(None) == swa.SWA_OK
        flag.zero_()
        torch.cuda.synchronize()
        assert step() == swa.SWA_OK              # the row is taken in again, where it already is
        torch.cuda.synchronize()
        assert lib.swa_device_status(None) == swa.SWA_OK
    finally:
        lib.swa_debug_set_trace(None)
    want, spread = q8.decode(ref, q, k, v, pos, dims.scale)
    close(o, want, spread, DECODE_REL, W * 2.0 ** -23 * 200, "after the timeout")
    same_cache(cache, ref, "after the timeout")
