"""The 8-bit cache's decode steps and few-row chunks where values of one window differ in size, or are zero, against
the float64 oracle (oracle/q8.py).

A weight is held in f16, 2^15 for the row with the largest product p* of softmax weight and value scale: it is off by
2^-11 of itself or, below 2^-14, by 2^-25.  The scores (d products, sizes below 2^4), exp2 and the fp32 sums stay within
another 2^-11.  With S the weighted mean of |v| the first and the last make 2^-10 S.  The second is 2^-40 of p* for each
of n rows, times a number of at most 2^15 where that row's scale makes its largest number 2^6 at least: n 2^-31 of the
row's weight times its largest |v|.  Rows here are at least half as large everywhere as in one place, so that is at most
n 2^-30 S; a row of zeros among others in a ring's block may weigh more than they do by its score, 2^9 at most.  With
n <= 2^16 / 2^9 there and n <= 2^16 elsewhere it stays below 2^-14 S."""
import math

import numpy as np
import pytest
import torch

import sliding_window_gqa_chunk_b200 as swa
from oracle import q8

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 2.0 ** -10 + 2.0 ** -14


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def bf16(x):
    return x.to(torch.bfloat16)


def close(got, want, spread, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    # below fp32's normal numbers an output keeps 2^-150
    worst = float((np.abs(got - want) / (REL * spread + 2.0 ** -149)).max())
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"


# largest sizes of the values of a ring's blocks, in turn (block j: sizes[j % len]); 0: a block of zeros.  Of odd length,
# so that a warp, which takes every eighth or fourth block, meets all of them.
SIZES = {
    "zeros beside 2^-24": [0.0, 2.0 ** -24, 2.0 ** -24],
    "zeros beside 2^-36, 2^-30": [2.0 ** -36, 0.0, 2.0 ** -30],
    "zeros beside 2^-80": [2.0 ** -80, 2.0 ** -80, 0.0],
    "zeros alone": [0.0],
    "zeros beside 2^100": [0.0, 0.0, 2.0 ** 100],
    "2^100 and 2^-60": [2.0 ** 100, 2.0 ** -60, 2.0 ** -60],
    "2^-60 and 2^100": [2.0 ** -60, 2.0 ** -60, 2.0 ** 100],
    "2^-60, zeros and 2^100": [2.0 ** -60, 0.0, 2.0 ** 100],
    "2^-112": [2.0 ** -112],
    "1, zeros and 300": [1.0, 0.0, 300.0],         # a scale of 1 that is not of zeros (e4m3; int8: 100)
}
# B, Hq, H, d, W, first position: warps of one CTA with a block each; a short sequence in the tail alone; several blocks
# to each warp of a cluster of 8, with the open block's old rows; several to a warp of a pair's only CTA
SHAPES = [
    (2, 4, 1, 128, 256, 700),
    (1, 4, 1, 64, 150 * 64, 38),
    (1, 12, 1, 128, 140 * 64, 141 * 64 + 37),
    (1, 3, 1, 64, 150 * 64 - 5, 160 * 64),
    (150, 1, 1, 16, 320, 333),
]


def run(dims, cache, ref, q, k, v, pos, T):
    """A chunk of T rows, then its first row as a decode step; both against the oracle."""
    B, Hq, d = dims.batch, dims.n_q_heads, dims.head_dim
    o = torch.full((B, T, Hq, d), float("nan"), device=DEV)
    swa.prefill_chunk_q8(dims, o, q.to(DEV), k.to(DEV), v.to(DEV), cache, i32(pos), i32([T] * B),
                         swa.prefill_workspace_q8(dims, T, DEV))
    want, spread = q8.prefill_chunk(ref, q, k, v, pos, [T] * B, dims.scale)
    close(o, want, spread, "chunk")
    o = torch.full((B, Hq, d), float("nan"), device=DEV)
    q1, k1, v1 = (x[:, 0].contiguous() for x in (q, k, v))
    swa.decode_q8(dims, o, q1.to(DEV), k1.to(DEV), v1.to(DEV), cache, i32(pos), swa.decode_workspace_q8(dims, DEV))
    want, spread = q8.decode(ref, q1, k1, v1, pos, dims.scale)
    close(o, want, spread, "decode step")
    swa.device_status()


def sized(g, sizes, B, n, H, d, W, start=0):
    """Values of rows start .. start + n - 1, each of its block's size."""
    at = (start + torch.arange(n)) % W // q8.BLOCK
    size = torch.tensor(sizes, dtype=torch.float64)[at % len(sizes)].view(1, n, 1, 1)
    sign = torch.randint(0, 2, (B, n, H, d), generator=g) * 2 - 1
    return bf16((torch.rand(B, n, H, d, generator=g) * 0.5 + 0.5) * sign * size)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,Hq,H,d,W,pos", SHAPES)
@pytest.mark.parametrize("name", list(SIZES))
def test_blocks_of_far_sizes(name, B, Hq, H, d, W, pos, fmt):
    sizes = [min(s, 100.0) if s > 1 and s < 2.0 ** 10 and fmt == "int8" else s for s in SIZES[name]]
    if name == "2^-112":
        pos = min(pos, 63)             # what is in the tail: a ring's scale is 2^-100 at least
    g = torch.Generator().manual_seed(W + d)
    dims = swa.Dims(B, Hq, H, d, W, 1.0 / math.sqrt(d), "f32")
    cache, ref = swa.new_cache_q8(dims, fmt, DEV), q8.RollingCacheQ8(B, H, W, d, fmt)
    for s in range(0, pos, 4096 if W > 4096 else W):
        n = min(4096, W, pos - s)
        k, v = bf16(torch.randn(B, n, H, d, generator=g)), sized(g, sizes, B, n, H, d, W, s)
        swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([s] * B), i32([n] * B))
        q8.append(ref, k, v, [s] * B, [n] * B)
    T = 3
    run(dims, cache, ref, bf16(torch.randn(B, T, Hq, d, generator=g)), bf16(torch.randn(B, T, H, d, generator=g)),
        sized(g, sizes, B, T, H, d, W, pos), [pos] * B, T)


@pytest.mark.parametrize("size", [2.0 ** -28, 2.0 ** 60])
def test_zero_rows_of_the_tail_and_of_the_chunk(size):
    """16 rows of zeros in the block being filled, in the ring's blocks none, and a new row of zeros."""
    B, Hq, H, d, W, pos = 2, 8, 2, 64, 256, 512 + 60
    g = torch.Generator().manual_seed(3)
    dims = swa.Dims(B, Hq, H, d, W, 0.125, "f32")
    cache, ref = swa.new_cache_q8(dims, "e4m3", DEV), q8.RollingCacheQ8(B, H, W, d, "e4m3")
    for s in range(0, pos, 128):
        n = min(128, pos - s)
        k, v = bf16(torch.randn(B, n, H, d, generator=g)), sized(g, [size], B, n, H, d, W)
        if s + n == pos:
            v[:, n - 44:n - 12] = 0.0      # rows 16 .. 47 of the open block
        swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([s] * B), i32([n] * B))
        q8.append(ref, k, v, [s] * B, [n] * B)
    q, k = bf16(torch.randn(B, 2, Hq, d, generator=g)), bf16(torch.randn(B, 2, H, d, generator=g))
    run(dims, cache, ref, q, k, torch.zeros(B, 2, H, d, dtype=torch.bfloat16), [pos] * B, 2)


@pytest.mark.parametrize("sizes", [[2.0 ** 100, 2.0 ** -60, 2.0 ** -60], [1.0, 16.0, 1.0], [0.0, 2.0 ** -30, 2.0 ** -30]])
def test_far_sizes_over_all_sms(sizes):
    """A window whose partial results are merged by a second kernel."""
    B, Hq, H, d, W = 1, 4, 1, 16, 1900 * 64
    g = torch.Generator().manual_seed(5)
    dims = swa.Dims(B, Hq, H, d, W, 0.25, "f32")
    assert swa.decode_workspace_size_q8(dims) > 16
    cache, ref = swa.new_cache_q8(dims, "int8", DEV), q8.RollingCacheQ8(B, H, W, d, "int8")
    k, v = bf16(torch.randn(B, W, H, d, generator=g)), sized(g, sizes, B, W, H, d, W)
    swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([0]), i32([W]))
    q8.append(ref, k, v, [0], [W])
    q, k1 = bf16(torch.randn(B, 1, Hq, d, generator=g)), bf16(torch.randn(B, 1, H, d, generator=g))
    run(dims, cache, ref, q, k1, sized(g, sizes, B, 1, H, d, W), [W], 1)

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("pos", [0, 16, 256 + 19])
def test_rows_of_a_chunk_do_not_see_the_sizes_of_later_ones(pos, fmt):
    """Rows whose keys or values are 2^40 times those of the rows before them, in one group of 16."""
    B, Hq, H, d, W, T = 2, 2, 1, 64, 256, 4
    g = torch.Generator().manual_seed(9)
    dims = swa.Dims(B, Hq, H, d, W, 0.125, "f32")
    cache, ref = swa.new_cache_q8(dims, fmt, DEV), q8.RollingCacheQ8(B, H, W, d, fmt)
    for s in range(0, pos, W):
        n = min(W, pos - s)
        k, v = bf16(torch.randn(B, n, H, d, generator=g)), sized(g, [2.0 ** -20], B, n, H, d, W)
        swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([s] * B), i32([n] * B))
        q8.append(ref, k, v, [s] * B, [n] * B)
    q, k, v = bf16(torch.randn(B, T, Hq, d, generator=g)), bf16(torch.randn(B, T, H, d, generator=g)), sized(g, [2.0 ** -20], B, T, H, d, W)
    k[0, 2:] *= 2.0 ** 40              # sequence 0: keys
    v[1, 2:] *= 2.0 ** 40
    o = torch.full((B, T, Hq, d), float("nan"), device=DEV)
    swa.prefill_chunk_q8(dims, o, q.to(DEV), k.to(DEV), v.to(DEV), cache, i32([pos] * B), i32([T] * B),
                         swa.prefill_workspace_q8(dims, T, DEV))
    want, spread = q8.prefill_chunk(ref, q, k, v, [pos] * B, [T] * B, dims.scale)
    close(o[:, :2], want[:, :2], spread[:, :2], "rows before the large ones")
    close(o[1, 2:], want[1, 2:], spread[1, 2:], "rows of large values")
    with pytest.raises(swa.SwaError) as e:      # sequence 0's last rows have scores of 2^40
        swa.device_status()
    assert e.value.code == swa.SWA_ERR_DEVICE_ARG


def test_a_chunk_over_a_tail_of_far_sizes():
    """A row of the block being filled that has next to no weight, and values 2^45 times the others'."""
    B, Hq, H, d, W, pos, T = 1, 4, 1, 64, 256, 13, 2
    g = torch.Generator().manual_seed(10)
    dims = swa.Dims(B, Hq, H, d, W, 0.125, "f32")
    cache, ref = swa.new_cache_q8(dims, "e4m3", DEV), q8.RollingCacheQ8(B, H, W, d, "e4m3")
    k, v = bf16(0.25 * torch.randn(B, pos, H, d, generator=g)), sized(g, [1.0], B, pos, H, d, W)
    q = bf16(torch.rand(B, T, Hq, d, generator=g) + 0.5)
    k[:, 7], v[:, 7] = -8.0, v[:, 7] * 2.0 ** 45       # a weight below 2^-46 for every query
    swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([0]), i32([pos]))
    q8.append(ref, k, v, [0], [pos])
    kc, vc = bf16(0.25 * torch.randn(B, T, H, d, generator=g)), sized(g, [1.0], B, T, H, d, W)
    o = torch.full((B, T, Hq, d), float("nan"), device=DEV)
    swa.prefill_chunk_q8(dims, o, q.to(DEV), kc.to(DEV), vc.to(DEV), cache, i32([pos]), i32([T]),
                         swa.prefill_workspace_q8(dims, T, DEV))
    want, spread = q8.prefill_chunk(ref, q, kc, vc, [pos], [T], dims.scale)
    close(o, want, spread, "chunk")
    swa.device_status()


@pytest.mark.parametrize("log2_score", [6, 12, 17, 22, 23])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,Hq,H,d,W,pos", [(2, 4, 2, 128, 256, 700), (1, 12, 1, 128, 140 * 64, 9100), (150, 1, 1, 16, 320, 333), (1, 4, 1, 64, 1900 * 64, 4000)])
def test_large_scores(B, Hq, H, d, W, pos, fmt, log2_score):
    """Keys that are whole multiples of the query, with large scores on 16 levels: equal scores share the weight equally,
    and value scales that differ from block to block count in full beside maxima of this size."""
    g = torch.Generator().manual_seed(log2_score)
    u = torch.randint(0, 2, (d,), generator=g) * 2.0 - 1.0
    # u . u = d: level c of 1 .. 16 gives a score of c / 16 2^log2_score
    dims = swa.Dims(B, Hq, H, d, W, 2.0 ** log2_score / (16 * d), "f32")
    cache, ref = swa.new_cache_q8(dims, fmt, DEV), q8.RollingCacheQ8(B, H, W, d, fmt)

    def keys(n):
        return bf16(torch.randint(1, 17, (B, n, H, 1), generator=g) * u)

    for s in range(0, pos, 256):
        n = min(256, pos - s)
        k, v = keys(n), sized(g, [1.0, 2.0 ** -3, 2.0 ** 5], B, n, H, d, W, s)
        swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([s] * B), i32([n] * B))
        q8.append(ref, k, v, [s] * B, [n] * B)
    q = bf16(u.expand(B, 3, Hq, d).contiguous())
    run(dims, cache, ref, q, keys(3), sized(g, [1.0, 2.0 ** -3, 2.0 ** 5], B, 3, H, d, W, pos), [pos] * B, 3)


@pytest.mark.parametrize("log2_score", [24, 40, 100])
@pytest.mark.parametrize("chunk", [False, True])
def test_scores_beyond_the_limit_are_reported(chunk, log2_score):
    """One sequence of two has a row whose largest score, 2^log2_score or its negative, is past 2^23.5; the other is right."""
    B, Hq, H, d, W, pos = 2, 4, 2, 64, 640, 300
    g = torch.Generator().manual_seed(1)
    for sign in (1.0, -1.0):
        dims = swa.Dims(B, Hq, H, d, W, 2.0 ** log2_score / d, "f32")
        cache, ref = swa.new_cache_q8(dims, "e4m3", DEV), q8.RollingCacheQ8(B, H, W, d, "e4m3")
        k, v = torch.ones(B, pos, H, d, dtype=torch.bfloat16), sized(g, [1.0], B, pos, H, d, W)
        swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([0] * B), i32([pos] * B))
        q8.append(ref, k, v, [0] * B, [pos] * B)
        q = torch.full((B, 1, Hq, d), sign, dtype=torch.bfloat16)
        q[1] = 0.0                          # scores of zero
        o = torch.full((B, 1, Hq, d), float("nan"), device=DEV)
        args = q.to(DEV), k[:, :1].contiguous().to(DEV), v[:, :1].contiguous().to(DEV)
        if chunk:
            swa.prefill_chunk_q8(dims, o, *args, cache, i32([pos] * B), i32([1] * B), swa.prefill_workspace_q8(dims, 1, DEV))
        else:
            swa.decode_q8(dims, o.view(B, Hq, d), *(x[:, 0] for x in args), cache, i32([pos] * B), swa.decode_workspace_q8(dims, DEV))
        with pytest.raises(swa.SwaError) as e:
            swa.device_status()
        assert e.value.code == swa.SWA_ERR_DEVICE_ARG
        want, spread = q8.prefill_chunk(ref, q, k[:, :1], v[:, :1], [pos] * B, [1] * B, dims.scale)
        close(o[1:], want[1:], spread[1:], "the other sequence")
