"""An 8-bit cache that another program filled: scales that are not powers of two mean the same to every call.

Decode steps and few-row chunks keep the numbers times the scale in full, to 2^-10 of the weighted mean of |v|
(tests/test_gpu_q8.py) and what the logarithm of a scale adds, below 2^-20 of it.  A chunk that is written out rounds
keys and values to bf16: half a step, 2^-9 of each.  That moves a score by at most e = 2^-9 scale |q| . |k| (e < 1 / 8 is
checked), so a softmax weight by a factor of at most exp(2 e) <= 1 + 3 e, and the weights are rounded to bf16 (2^-8 with
the fp32 rest, 2^-10): (3 e + 2^-9 + 2^-8 + 2^-10) S, twice as a weight's error counts in its sum too."""
import math

import numpy as np
import pytest
import torch

import sliding_window_gqa_chunk_b200 as swa
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,Hq,H,d,W,T", [(2, 8, 2, 128, 256, 3), (2, 4, 2, 64, 640, 3), (1, 24, 2, 128, 192, 1), (150, 1, 1, 16, 128, 2),
                                          (2, 8, 2, 64, 256, 200), (1, 8, 8, 128, 640, 520)])
def test_scales_that_are_not_powers_of_two(B, Hq, H, d, W, T, fmt):
    g = torch.Generator().manual_seed(B + W)
    dims = swa.Dims(B, Hq, H, d, W, 0.25 / math.sqrt(d), "f32")
    cache = swa.new_cache_q8(dims, fmt, DEV)
    n = W // swa.Q8_BLOCK
    rows = []
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        # a block's largest number is the format's top, as a quantiser leaves it with amax / top as the scale
        top = 448.0 if fmt == "e4m3" else 127.0
        y = torch.randn(B, H, n, swa.Q8_BLOCK, d, generator=g)
        y = y * (top / y.abs().amax(dim=(-1, -2), keepdim=True))
        y = (y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().to(torch.int8)).view(B, H, W, d)
        scale = torch.rand(B, H, n, generator=g) * 3 / top + 1 / top
        x.copy_(y)
        s.copy_(scale)
        rows.append((y.double() * scale.double().repeat_interleave(swa.Q8_BLOCK, 2)[..., None]).numpy())
    pos = [3 * W] * B                              # whole laps: every slot is held, none in the tail

    def attend(q, k, v, t):
        out, spread, worst = np.zeros((B, t, Hq, d)), np.zeros((B, t, Hq, d)), 0.0
        at = np.arange(pos[0] - W, pos[0] + t)
        for b in range(B):
            kk, vv = (np.concatenate([r[b].transpose(1, 0, 2), x[b, :t].double().numpy()]) for r, x in zip(rows, (k, v)))
            qq = q[b, :t].double().numpy()
            out[b] = oracle.attend(qq, at[W:], kk, vv, at, W, dims.scale)
            spread[b] = oracle.attend(qq, at[W:], kk, np.abs(vv), at, W, dims.scale)
            for h in range(H):
                worst = max(worst, (np.abs(qq[:, h * (Hq // H):(h + 1) * (Hq // H)]) @ np.abs(kk[:, h]).T).max() * dims.scale)
        return out, spread, worst

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    q = torch.randn(B, T, Hq, d, generator=g).to(torch.bfloat16)
    k, v = (torch.randn(B, T, H, d, generator=g).to(torch.bfloat16) for _ in range(2))
    out = torch.full((B, T, Hq, d), float("nan"), device=DEV)
    swa.prefill_chunk_q8(dims, out, q.to(DEV), k.to(DEV), v.to(DEV), cache, i32(pos), i32([T] * B), swa.prefill_workspace_q8(dims, T, DEV))
    want, spread, worst = attend(q, k, v, T)
    exact = 2.0 ** -10 + 2.0 ** -20
    e = 2.0 ** -9 * worst
    assert e < 0.125
    rel = exact if T < 100 else 2 * (3 * e + 2.0 ** -9 + 2.0 ** -8 + 2.0 ** -10)
    off = np.abs(out.double().cpu().numpy() - want)
    assert (off <= rel * spread).all(), float((off / spread).max())
    out = torch.full((B, Hq, d), float("nan"), device=DEV)
    q1, k1, v1 = (x[:, 0].contiguous().to(DEV) for x in (q, k, v))
    swa.decode_q8(dims, out, q1, k1, v1, cache, i32(pos), swa.decode_workspace_q8(dims, DEV))
    want, spread, _ = attend(q, k, v, 1)
    off = np.abs(out.double().cpu().numpy() - want[:, 0])
    assert (off <= exact * spread[:, 0]).all(), float((off / spread[:, 0]).max())
    swa.device_status()
