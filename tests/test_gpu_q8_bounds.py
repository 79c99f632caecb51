"""The 8-bit cache's calls held to the bounds that their arithmetic gives, in the forms that other tests of them leave
out: offsets past 32 bits with rows that matter, partial results merged by a second kernel, few-row chunks at each
head dimension.

Decode steps and few-row chunks: weights in f16 (2^-11) and scores, exp2 and fp32 sums (another 2^-11) make 2^-10 S, S
the weighted mean of |v|.  Weights below 2^-14 are off by 2^-25, where the largest product of weight and value scale
has 2^15, times numbers of up to 2^15 where that row's largest is 2^6 at least: n 2^-31 of the largest |v| for n
positions.  A written-out chunk rounds weights to bf16: (2^-8 + 2^-10) S.  bf16 output adds 2^-8 of itself."""
import math

import numpy as np
import pytest
import torch

import sliding_window_gqa_chunk_b200 as swa
from oracle import q8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BYTES, WRITTEN_OUT = 2.0 ** -10, 2.0 ** -8 + 2.0 ** -10


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def rows(g, *shape):
    """bf16 rows whose sizes differ from row to row and with a few large channels."""
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randn(shape[:-1] + (1,), generator=g))
    x[..., 0] *= 5.0
    return x.to(torch.bfloat16)


def close(got, want, spread, rel, small, what, out="f32"):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    tol = rel * spread + small + (2.0 ** -8 * np.abs(want) if out == "bf16" else 0.0)
    worst = float((np.abs(got - want) / np.maximum(tol, 1e-300)).max())
    assert worst <= 1.0, f"{what}: {worst:.2f} of the bound"
    return tol


def fill(dims, cache, ref, lengths, g, chunk):
    B, H, d = dims.batch, dims.n_kv_heads, dims.head_dim
    biggest = 0.0
    for s in range(0, max(lengths), chunk):
        n = [max(0, min(chunk, x - s)) for x in lengths]
        k, v = rows(g, B, chunk, H, d), rows(g, B, chunk, H, d)
        swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([s] * B), i32(n))
        q8.append(ref, k, v, [s] * B, n)
        biggest = max(biggest, float(v.float().abs().max()))
    return biggest


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,Hq,H,d,W,T,starts", [
    (3, 8, 2, 128, 200, 4, [0, 63, 500]),
    (2, 16, 2, 64, 640, 7, [640, 1300]),
    (1, 32, 8, 128, 1024, 16, [2047]),
    (2, 4, 4, 128, 192, 128, [63, 400]),
    (1, 1, 1, 64, 700, 512, [365]),
    (2, 12, 1, 128, 260, 9, [259, 31]),
    (2, 3, 1, 16, 300, 40, [299, 900]),
    (160, 2, 1, 64, 64, 3, list(range(160))),
])
def test_few_row_chunks_and_steps(B, Hq, H, d, W, T, starts, fmt):
    out = "bf16" if fmt == "int8" else "f32"
    g = torch.Generator().manual_seed(W * 3 + T)
    dims = swa.Dims(B, Hq, H, d, W, 1.0 / math.sqrt(d), out)
    cache, ref = swa.new_cache_q8(dims, fmt, DEV), q8.RollingCacheQ8(B, H, W, d, fmt)
    big = fill(dims, cache, ref, starts, g, min(W, 64))
    q, k, v = torch.randn(B, T, Hq, d, generator=g).to(torch.bfloat16), rows(g, B, T, H, d), rows(g, B, T, H, d)
    small = W * 2.0 ** -31 * max(big, float(v.float().abs().max()))
    o = torch.full((B, T, Hq, d), float("nan"), dtype=dims.torch_out_dtype, device=DEV)
    swa.prefill_chunk_q8(dims, o, q.to(DEV), k.to(DEV), v.to(DEV), cache, i32(starts), i32([T] * B),
                         swa.prefill_workspace_q8(dims, T, DEV))
    want, spread = q8.prefill_chunk(ref, q, k, v, starts, [T] * B, dims.scale)
    close(o, want, spread, BYTES, small, "chunk", out)
    ws, pos = swa.decode_workspace_q8(dims, DEV), list(starts)
    for t in range(min(T, 3)):
        o = torch.full((B, Hq, d), float("nan"), dtype=dims.torch_out_dtype, device=DEV)
        q1, k1, v1 = (x[:, t].contiguous() for x in (q, k, v))
        swa.decode_q8(dims, o, q1.to(DEV), k1.to(DEV), v1.to(DEV), cache, i32(pos), ws)
        want, spread = q8.decode(ref, q1, k1, v1, pos, dims.scale)
        close(o, want, spread, BYTES, small, f"step {t}", out)
        pos = [p + 1 for p in pos]
    swa.device_status()


@pytest.mark.parametrize("d,G,fmt,out", [(128, 4, "e4m3", "f32"), (128, 16, "int8", "bf16"), (64, 12, "e4m3", "bf16"), (64, 1, "int8", "f32"),
                                         (16, 9, "e4m3", "f32")])
def test_partial_results_merged_by_a_second_kernel(d, G, fmt, out):
    """A long window and few pairs: a full sequence, a short one (most of its parts are empty), one that is skipped."""
    B, H, W = 3, 1, 512 * 64 + 70
    g = torch.Generator().manual_seed(d + G)
    dims = swa.Dims(B, G * H, H, d, W, 1.0 / math.sqrt(d), out)
    need = swa.decode_workspace_size_q8(dims)
    assert need > 16
    cache, ref = swa.new_cache_q8(dims, fmt, DEV), q8.RollingCacheQ8(2, H, W, d, fmt)
    lengths = [W + 100, 130]
    big = 0.0
    for s in range(0, max(lengths), 4096):
        n = [max(0, min(4096, x - s)) for x in lengths]
        k, v = rows(g, B, 4096, H, d), rows(g, B, 4096, H, d)
        swa.cache_append_q8(dims, cache, k.to(DEV), v.to(DEV), i32([s] * B), i32(n + [0]))
        q8.append(ref, k[:2], v[:2], [s] * 2, n)
        big = max(big, float(v.float().abs().max()))
    whole = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)       # what it holds before does not matter
    ws = whole[256:256 + need]
    for i in range(2):
        q, k, v = torch.randn(B, G * H, d, generator=g).to(torch.bfloat16), rows(g, B, H, d), rows(g, B, H, d)
        o = torch.full((B, G * H, d), 7.0, dtype=dims.torch_out_dtype, device=DEV)
        pos = [x + i for x in lengths]
        swa.decode_q8(dims, o, q.to(DEV), k.to(DEV), v.to(DEV), cache, i32(pos + [-1 - i]), ws)
        with pytest.raises(swa.SwaError) as e:
            swa.device_status()
        assert e.value.code == swa.SWA_ERR_DEVICE_ARG
        assert bool((o[2] == 7.0).all())
        assert bool((whole[:256] == 255).all()) and bool((whole[256 + need:] == 255).all())
        want, spread = q8.decode(ref, q[:2], k[:2], v[:2], pos, dims.scale)
        close(o[:2], want, spread, BYTES, W * 2.0 ** -31 * max(big, float(v.float().abs().max())), f"step {i}", out)


def test_offsets_past_32_bits_with_rows_that_matter():
    """The last sequence of a ring of more than 2^32 bytes: 300 rows whose weights outweigh those of the zeros that the rest
    of the window holds; a decode step, a chunk over the bytes and one that is written out, against float64."""
    B, Hq, H, d, W, T = 33, 4, 1, 128, 1 << 20, 300
    free, _ = torch.cuda.mem_get_info()
    if free < 48 << 30:
        pytest.skip("needs 48 GB of device memory")
    dims = swa.Dims(B, Hq, H, d, W, 1.0 / math.sqrt(d), "f32")
    cache = swa.new_cache_q8(dims, "int8", DEV)
    cache.k_scale.fill_(1.0)                       # blocks of zeros
    cache.v_scale.fill_(1.0)
    g = torch.Generator().manual_seed(2)
    u = torch.randn(d, generator=g)
    u = u * (math.sqrt(d) / u.norm())
    # scores of about 2.2 sqrt(d) = 25: e^25 against 2^20 zeros of weight 1
    k, v = (2.2 * u + 0.2 * torch.randn(T, H, d, generator=g)).to(torch.bfloat16), torch.randn(T, H, d, generator=g).to(torch.bfloat16)
    s0 = W - 100
    n = [0] * (B - 1) + [T]
    kd, vd = (torch.zeros(B, T, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kd[-1], vd[-1] = k.to(DEV), v.to(DEV)
    swa.cache_append_q8(dims, cache, kd, vd, i32([s0] * B), i32(n))
    # the same rows in a short ring whose blocks begin at the same places, after zeros
    short = 1024
    ref = q8.RollingCacheQ8(1, H, short, d, "int8")
    z = np.zeros((1, short - 100, H, d))
    q8.append(ref, z, z, [0], [short - 100])
    q8.append(ref, k[None], v[None], [short - 100], [T])
    held_k, held_v, at = ref.rows(0, short - 100 + T)
    held_k, held_v = held_k[-T:, 0], held_v[-T:, 0]
    assert at[-1] - at[-T] == T - 1

    def want(q, kn, vn):
        """Rows of the chunk (or one step): what is held, the chunk's rows up to their own, zeros for the rest of the window."""
        out, spread = np.zeros(q.shape), np.zeros(q.shape)
        for t in range(q.shape[0]):
            kk = np.concatenate([held_k, kn[:t + 1, 0]])[-W:]
            vv = np.concatenate([held_v, vn[:t + 1, 0]])[-W:]
            for h in range(Hq):
                s = kk @ q[t, h] * dims.scale
                w = np.exp(s - s.max())
                total = w.sum() + (W - len(kk)) * math.exp(-s.max())
                out[t, h], spread[t, h] = w @ vv / total, w @ np.abs(vv) / total
        return out, spread

    def chunk(rows_):
        q = (u + 0.1 * torch.randn(rows_, Hq, d, generator=g)).to(torch.bfloat16)
        kn, vn = (2.2 * u + 0.2 * torch.randn(rows_, H, d, generator=g)).to(torch.bfloat16), torch.randn(rows_, H, d, generator=g).to(torch.bfloat16)
        dense = [torch.zeros(B, rows_, x.shape[1], d, dtype=torch.bfloat16, device=DEV) for x in (q, kn, vn)]
        for a, x in zip(dense, (q, kn, vn)):
            a[-1] = x.to(DEV)
        return dense, want(*(x.double().numpy() for x in (q, kn, vn)))

    pos = i32([3] * (B - 1) + [s0 + T])
    for rows_, rel in ((3, BYTES), (T, WRITTEN_OUT)):
        (qd, kn, vn), (ref_out, spread) = chunk(rows_)
        o = torch.full((B, rows_, Hq, d), 5.0, device=DEV)
        swa.prefill_chunk_q8(dims, o, qd, kn, vn, cache, pos, i32([0] * (B - 1) + [rows_]), swa.prefill_workspace_q8(dims, rows_, DEV))
        tol = close(o[-1], ref_out, spread, rel, 0.0, f"chunk of {rows_}")
        # means of some 300 values of size 1 are about S / 20, and the wider bound is S / 205
        assert np.abs(ref_out).mean() > 8 * tol.mean()
        assert bool((o[:-1] == 5.0).all())
    (qd, kn, vn), (ref_out, spread) = chunk(1)
    o = torch.full((B, Hq, d), 5.0, device=DEV)
    swa.decode_q8(dims, o, qd[:, 0].contiguous(), kn[:, 0].contiguous(), vn[:, 0].contiguous(), cache, pos, swa.decode_workspace_q8(dims, DEV))
    tol = close(o[-1:], ref_out, spread, BYTES, 0.0, "step")
    assert np.abs(ref_out).mean() > 16 * tol.mean()
    swa.device_status()
