"""Rotary positions on the GPU against the float64 oracle (angles in extended precision there).

Bound for an element: half a bf16 step of the result (2^-8 of it), and what fp32 adds to a
sum of two products of elements of size a: 3 roundings (2^-24 each), cos and sin (2^-23) and the
angle, off by less than 2^-23 of a turn at positions below 2^31 (2.5 2^-53 of 2^28.35 turns, and
2^-26 for the fraction): together below 2^-19 factor a."""
import numpy as np
import pytest
import torch

import sliding_window_gqa_chunk_b200 as swa
from oracle import q8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def check(got, x, positions, spec, transpose=False):
    x = x.double().cpu().numpy()
    want = q8.rope(x, positions, spec.inv_freq.cpu().numpy(), spec.interleaved, spec.factor, transpose)
    size = spec.factor * np.abs(x).max(axis=-1, keepdims=True)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size).all(), float(err.max())


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,Hq,H,d,r,starts,counts", [
    (1, 1, 4, 2, 16, 16, [0], [1]),
    (1, 1, 32, 8, 128, 128, [2 ** 31 - 2], [1]),
    (3, 7, 6, 2, 64, 32, [0, 5, 100000], [7, 0, 3]),
    (2, 900, 3, 1, 128, 96, [2 ** 24 + 1, 31], [900, 611]),      # 4 tokens a CTA, 4 heads
    (3, 3201, 2, 1, 64, 32, [0, 2 ** 20, 77], [3201, 3200, 17]), # 9 tokens a CTA
    (2, 6300, 1, 1, 16, 16, [5, 10 ** 9], [6300, 6299]),         # two waves of 9
    (2, 601, 7, 7, 64, 64, [2 ** 31 - 700, 9], [601, 601]),
    (70, 1, 9, 3, 128, 48, list(range(0, 7000, 100)), [1] * 70),
    (2, 650, 24, 8, 128, 128, [70, 4000], [650, 649]),           # 32 heads
])
def test_rope_matches_the_oracle(B, T, Hq, H, d, r, starts, counts, interleaved, transpose):
    g = torch.Generator().manual_seed(T + r)
    dims = swa.Dims(B, Hq, H, d, 64, 1.0, "bf16")
    spec = swa.new_rope(r, base=500000.0 if r == 96 else 10000.0, interleaved=interleaved, scaling="yarn" if r == 48 else "none",
                        scale=8.0, device=DEV)
    q, k = torch.randn(B, T, Hq, d, generator=g).to(torch.bfloat16), torch.randn(B, T, H, d, generator=g).to(torch.bfloat16)
    packed = torch.cat([q, k, k], dim=2).to(DEV)                 # heads inside a packed projection
    forms = {"dense": (q.to(DEV), k.to(DEV)), "packed": (packed[:, :, :Hq], packed[:, :, Hq:Hq + H])}
    results = []
    for qi, ki in forms.values():
        qo, ko = (torch.full(s, 3.0, dtype=torch.bfloat16, device=DEV) for s in (q.shape, k.shape))
        swa.rope(dims, spec, qo, ko, qi, ki, i32(starts), i32(counts), transpose=transpose)
        results.append((qo, ko))
    qd, kd = q.to(DEV), k.to(DEV)
    swa.rope(dims, spec, qd, kd, qd, kd, i32(starts), i32(counts), transpose=transpose)   # in place
    for b in range(B):
        n = counts[b]
        at = starts[b] + np.arange(n)
        for x, outs, inplace in ((q, [a[0] for a in results], qd), (k, [a[1] for a in results], kd)):
            check(outs[0][b, :n], x[b, :n], at, spec, transpose)
            assert torch.equal(outs[0][b], outs[1][b])
            assert bool((outs[0][b, n:] == 3.0).all())
            assert torch.equal(inplace[b, :n], outs[0][b, :n]) and torch.equal(inplace[b, n:].cpu(), x[b, n:])
            if r < d:
                assert torch.equal(outs[0][b, :n, :, r:].cpu(), x[b, :n, :, r:])
    swa.device_status()


def test_rope_without_keys_and_without_counts():
    dims = swa.Dims(2, 4, 2, 64, 64, 1.0, "bf16")
    spec = swa.new_rope(64, device=DEV)
    q = torch.randn(2, 5, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device=DEV)
    swa.rope(dims, spec, out, None, q.to(DEV), None, i32([3, 40]))
    for b, s in enumerate((3, 40)):
        check(out[b], q[b], s + np.arange(5), spec)


@pytest.mark.parametrize("interleaved", [False, True])
def test_transpose_is_the_gradient(interleaved):
    """<dy, R x> = <R^T dy, x> with the formula's gradient, and against differences: R is linear, so
    (R(x + e) - R(x - e)) / 2 = R e, whose inner product with dy is the gradient's with e."""
    dims = swa.Dims(1, 2, 2, 64, 64, 1.0, "bf16")
    spec = swa.new_rope(32, interleaved=interleaved, scaling="yarn", scale=4.0, device=DEV)
    g = torch.Generator().manual_seed(7)
    x, e, dy = (torch.randn(1, 40, 2, 64, generator=g).to(torch.bfloat16) for _ in range(3))
    run = {}
    for name, t, tr in (("x", x, False), ("e", e, False), ("dy", dy, True)):
        o, o2 = (torch.zeros(t.shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        swa.rope(dims, spec, o, o2, t.to(DEV), t.to(DEV), i32([1000]), transpose=tr)
        assert torch.equal(o, o2)
        run[name] = o.double().cpu()
    for a, b in (("x", x), ("e", e)):
        left, right = dy.double() * run[a], run["dy"] * b.double()
        # both sides carry half a bf16 step in each of their terms' turned factor
        slack = 2.0 ** -8 * (left.abs().sum() + right.abs().sum()) + 2.0 ** -16
        assert abs(float(left.sum() - right.sum())) <= float(slack)
    xg = x.to(DEV).double().requires_grad_(True)
    pos = (1000 + torch.arange(40, device=DEV)).double()[:, None]
    ang = (pos * spec.inv_freq.double())[None, :, None]
    a, b = (xg[..., 0:32:2], xg[..., 1:32:2]) if interleaved else (xg[..., :16], xg[..., 16:32])
    f = spec.factor
    turned = [f * (a * ang.cos() - b * ang.sin()), f * (b * ang.cos() + a * ang.sin())]
    y = torch.stack(turned, -1).flatten(-2) if interleaved else torch.cat(turned, -1)
    y = torch.cat([y, xg[..., 32:]], -1)
    (grad,) = torch.autograd.grad((y * dy.to(DEV).double()).sum(), xg)
    size = f * dy.double().abs().amax(-1, keepdim=True)
    assert bool(((run["dy"] - grad.cpu()).abs() <= 2.0 ** -8 * grad.cpu().abs() + 2.0 ** -19 * size).all())


def test_bad_device_arguments_skip_the_sequence():
    dims = swa.Dims(2, 2, 2, 64, 64, 1.0, "bf16")
    spec = swa.new_rope(64, device=DEV)
    x = torch.randn(2, 6, 2, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    for start, n in (([-1, 4], [6, 6]), ([0, 4], [7, 6]), ([0, 4], [-2, 6])):
        q, k = (torch.full(x.shape, 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        swa.rope(dims, spec, q, k, x.to(DEV), x.to(DEV), i32(start), i32(n))
        with pytest.raises(swa.SwaError) as e:
            swa.device_status()
        assert e.value.code == swa.SWA_ERR_DEVICE_ARG
        assert bool((q[0] == 5.0).all()) and bool((k[0] == 5.0).all())
        check(q[1], x[1], 4 + np.arange(6), spec)
