"""The 8-bit cache and the rotary positions without a GPU: what the C entry points and the binding
refuse (on the host, before CUDA is touched), and the oracle against other statements of the formulas."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import sliding_window_gqa_chunk_b200 as swa
from oracle import q8
from sliding_window_gqa_chunk_b200.csrc import build as swa_build

FAKE = 0x10000  # aligned, non-null; never dereferenced because validation fails first


@pytest.fixture(scope="module")
def lib():
    swa_build.build()
    return swa.load_library()


def dims(**kw):
    base = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, window=256, scale=0.1, out_dtype="f32")
    base.update(kw)
    return swa.Dims(**base).c()


def P(x=FAKE):
    return ctypes.c_void_p(x)


def cache(**kw):
    c = swa._CCacheQ8(*[FAKE] * 6, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def append(lib, d=None, c=None, k=FAKE, v=FAKE, T=8, s=FAKE, n=FAKE):
    d, c = d or dims(), c or cache()
    return lib.swa_q8_append(ctypes.byref(d), ctypes.byref(c), P(k), P(v), T, P(s), P(n), None)


def prefill(lib, d=None, c=None, ptrs=(FAKE,) * 4, T=8, s=FAKE, n=FAKE, ws=FAKE, size=1 << 40):
    d, c = d or dims(), c or cache()
    return lib.swa_q8_prefill_chunk(ctypes.byref(d), *[P(x) for x in ptrs], T, ctypes.byref(c), P(s), P(n), P(ws), size, None)


def decode(lib, d=None, c=None, ptrs=(FAKE,) * 4, pos=FAKE, ws=FAKE, size=1 << 40):
    d, c = d or dims(), c or cache()
    return lib.swa_q8_decode(ctypes.byref(d), *[P(x) for x in ptrs], ctypes.byref(c), P(pos), P(ws), size, None)


def rope(lib, d=None, spec=None, ptrs=(FAKE,) * 4, qs=8 * 128, ks=2 * 128, T=8, s=FAKE, n=FAKE, tr=0):
    d, spec = d or dims(), spec or swa._CRope(FAKE, 128, 0, 1.0)
    return lib.swa_rope(ctypes.byref(d), ctypes.byref(spec), *[P(x) for x in ptrs], qs, ks, T, P(s), P(n), tr, None)


CALLS = [append, prefill, decode]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,code", [
    (dict(n_q_heads=6, n_kv_heads=4), swa.SWA_ERR_UNSUPPORTED),
    (dict(head_dim=32), swa.SWA_ERR_UNSUPPORTED),
    (dict(n_q_heads=64, n_kv_heads=2), swa.SWA_ERR_UNSUPPORTED),
    (dict(window=0), swa.SWA_ERR_INVALID_ARG),
    (dict(window=(1 << 30) + 1), swa.SWA_ERR_UNSUPPORTED),
    (dict(batch=0), swa.SWA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), swa.SWA_ERR_INVALID_ARG),
])
def test_bad_dims(lib, call, kw, code):
    d = dims(**kw)
    assert call(lib, d=d) == code and lib.swa_last_error()
    assert lib.swa_q8_decode_workspace_size(ctypes.byref(d)) == 0
    assert lib.swa_q8_prefill_workspace_size(ctypes.byref(d), 1) == 0


@pytest.mark.parametrize("call", CALLS)
def test_bad_caches(lib, call):
    for name in ("k", "v", "k_tail", "v_tail"):
        for bad in (None, FAKE + 8):
            assert call(lib, c=cache(**{name: bad})) == swa.SWA_ERR_INVALID_ARG
    for name in ("k_scale", "v_scale"):
        for bad in (None, FAKE + 2):
            assert call(lib, c=cache(**{name: bad})) == swa.SWA_ERR_INVALID_ARG
    for fmt in (-1, 2):
        assert call(lib, c=cache(format=fmt)) == swa.SWA_ERR_INVALID_ARG
        assert b"format" in lib.swa_last_error()


def test_null_cache(lib):
    d = dims()
    p = [P()] * 9
    assert lib.swa_q8_append(ctypes.byref(d), None, p[0], p[1], 8, p[2], p[3], None) == swa.SWA_ERR_INVALID_ARG
    assert lib.swa_q8_decode(ctypes.byref(d), *p[:4], None, p[4], p[5], 1 << 40, None) == swa.SWA_ERR_INVALID_ARG
    assert lib.swa_q8_prefill_chunk(ctypes.byref(d), *p[:4], 8, None, p[4], p[5], p[6], 1 << 40,
                                    None) == swa.SWA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [prefill, decode])
def test_bad_tensors_and_workspaces(lib, call):
    for i in range(4):
        for bad in (None, FAKE + 8):
            assert call(lib, ptrs=[bad if j == i else FAKE for j in range(4)]) == swa.SWA_ERR_INVALID_ARG
    assert call(lib, ws=None) == swa.SWA_ERR_INVALID_ARG
    assert call(lib, ws=FAKE + 4) == swa.SWA_ERR_INVALID_ARG
    assert call(lib, size=8) == swa.SWA_ERR_WORKSPACE_TOO_SMALL
    d = dims()
    need = lib.swa_q8_prefill_workspace_size(ctypes.byref(d), 8)
    assert need >= 2 * 2 * 2 * 256 * 128 * 2 + lib.swa_prefill_workspace_size(ctypes.byref(d), 8)
    assert prefill(lib, size=need - 1) == swa.SWA_ERR_WORKSPACE_TOO_SMALL


def test_bad_counts(lib):
    for T in (0, -1, 257):
        assert append(lib, T=T) == swa.SWA_ERR_INVALID_ARG
        assert prefill(lib, T=T) == swa.SWA_ERR_INVALID_ARG
        assert lib.swa_q8_prefill_workspace_size(ctypes.byref(dims()), T) == 0
    for kw in (dict(k=None), dict(v=FAKE + 2), dict(s=None), dict(n=FAKE + 1)):
        assert append(lib, **kw) == swa.SWA_ERR_INVALID_ARG
    assert prefill(lib, s=None) == swa.SWA_ERR_INVALID_ARG
    assert decode(lib, pos=FAKE + 2) == swa.SWA_ERR_INVALID_ARG
    # more query tiles than the prefill takes: refused before the ring is written out (129 rows, as up to
    # 128 columns go another way)
    big = dims(batch=65535, n_q_heads=16384, n_kv_heads=16384, head_dim=16, window=200)
    assert prefill(lib, d=big, T=129, size=1 << 62) == swa.SWA_ERR_UNSUPPORTED


def test_rope_refusals(lib):
    S = swa._CRope
    for r in (0, 8, 24, 144, -16):
        assert rope(lib, spec=S(FAKE, r, 0, 1.0)) == swa.SWA_ERR_UNSUPPORTED
    for spec in (S(None, 128, 0, 1.0), S(FAKE + 2, 128, 0, 1.0), S(FAKE, 128, 2, 1.0), S(FAKE, 128, 0, 0.0),
                 S(FAKE, 128, 0, float("inf")), S(FAKE, 128, 0, float("nan"))):
        assert rope(lib, spec=spec) == swa.SWA_ERR_INVALID_ARG
    for kw in (dict(ptrs=(None, FAKE, FAKE, FAKE)), dict(ptrs=(FAKE, FAKE, FAKE + 2, FAKE)),
               dict(ptrs=(FAKE, None, FAKE, FAKE)), dict(ptrs=(FAKE, FAKE, FAKE, None)), dict(qs=8 * 128 - 8), dict(qs=8 * 128 + 4),
               dict(ks=0), dict(ks=-256), dict(qs=2048), dict(ks=264), dict(T=0), dict(T=1 << 30), dict(s=None), dict(s=FAKE + 1),
               dict(n=FAKE + 3), dict(tr=2), dict(d=dims(head_dim=64)), dict(d=dims(batch=0))):
        assert rope(lib, **kw) != swa.SWA_OK, kw
        assert lib.swa_last_error()


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    d = swa.Dims(1, 2, 1, 16, 64, 0.25)
    with pytest.raises(ValueError, match="CUDA"):
        swa.new_cache_q8(d, "e4m3", "cpu")
    with pytest.raises(ValueError, match="format"):
        swa.new_cache_q8(d, "fp4", "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        swa.new_rope(16, device="cpu")
    for kw in (dict(scaling="ntk"), dict(base=0.0), dict(scale=-1.0)):
        with pytest.raises(ValueError):
            swa.new_rope(16, device="cpu", **kw)
    with pytest.raises(ValueError):
        swa.new_rope(15, device="cpu")
    z = torch.zeros
    with pytest.raises(ValueError, match="float8"):
        swa.CacheQ8(z(1, 1, 64, 16, dtype=torch.uint8), *[z(1)] * 5)


def test_round_block_against_torch_conversions():
    g = torch.Generator().manual_seed(1)
    for i in range(200):
        x = (torch.randn(5, 16, generator=g) * 2.0 ** float(torch.randint(-40, 40, (1,), generator=g))).to(torch.bfloat16)
        for fmt, top, dtype in (("e4m3", 448.0, torch.float8_e4m3fn), ("int8", 127.0, torch.int8)):
            y, s = q8.round_block(x.double().numpy(), fmt)
            assert np.abs(x.double().numpy()).max() / s <= top < 2 * np.abs(x.double().numpy()).max() / s
            z = x.double() / s
            z = z.float().to(dtype).double() if fmt == "e4m3" else torch.round(z)
            np.testing.assert_array_equal(y, z.numpy())
            # the number stands for a bf16 value
            back = torch.from_numpy(y * s)
            assert torch.equal(back.to(torch.bfloat16).double(), back)


@pytest.mark.parametrize("W", [1, 5, 64, 100, 130])
def test_oracle_cache_is_the_rolling_cache_up_to_its_roundings(W):
    """The same positions are visible as in the bf16 ring's oracle, with rows off by half a step at most."""
    rng = np.random.default_rng(W)
    B, H, d, n = 1, 2, 16, 3 * W + 70
    ref, c = oracle.RollingCache(B, H, W, d), q8.RollingCacheQ8(B, H, W, d, "int8")
    for p in range(n):
        k, v = rng.normal(size=(H, d)), rng.normal(size=(H, d))
        kk, vv, at = c.rows(0, p)
        rk, rv, rp = ref.keys(0)
        window = at > p - W        # the query at p sees these
        assert sorted(at[window]) == sorted(x for x in rp if x >= 0 and x > p - W)
        order = {x: i for i, x in enumerate(rp)}
        for i in np.nonzero(window)[0]:
            got, want = kk[i], rk[order[at[i]]]
            assert np.abs(got - want).max() <= 0.5 * max(c.k_scale.max(), 1e-9)
        ref.write(0, p, k, v)
        c.write(0, p, k, v)


def test_oracle_rope_is_a_complex_product():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(6, 2, 32))
    f = (10000.0 ** (-np.arange(8) / 8)).astype(np.float32)
    pos = np.arange(100, 106)
    turn = np.exp(1j * pos[:, None] * f.astype(np.float64))[:, None]
    for inter in (False, True):
        a, b = (x[..., 0:16:2], x[..., 1:16:2]) if inter else (x[..., :8], x[..., 8:16])
        z = 1.5 * (a + 1j * b) * turn
        y = q8.rope(x, pos, f, inter, 1.5)
        ga, gb = (y[..., 0:16:2], y[..., 1:16:2]) if inter else (y[..., :8], y[..., 8:16])
        np.testing.assert_allclose(ga + 1j * gb, z, rtol=0, atol=1e-12)
        np.testing.assert_array_equal(y[..., 16:], x[..., 16:])
        back = q8.rope(y, pos, f, inter, 1 / 1.5, transpose=True)
        np.testing.assert_allclose(back[..., :16], x[..., :16] , rtol=0, atol=1e-12)


def test_frequencies_of_the_scaled_forms(monkeypatch):
    made = {}
    monkeypatch.setattr(swa, "Rope", lambda f, i, c: made.update(f=f.double().numpy(), c=c))

    def freqs(**kw):
        swa.new_rope(64, device="cpu", **kw)
        return made["f"], made["c"]

    plain, c = freqs()
    i = np.arange(32)
    np.testing.assert_allclose(plain, 10000.0 ** (-i / 32), rtol=2.0 ** -23)
    assert c == 1.0
    np.testing.assert_allclose(freqs(scaling="linear", scale=4.0)[0], plain / 4, rtol=2.0 ** -22)
    f, _ = freqs(scaling="base", scale=4.0)
    np.testing.assert_allclose([f[0], f[-1]], [plain[0], plain[-1] / 4], rtol=1e-6)
    f, c = freqs(scaling="yarn", scale=4.0, original_length=2048)
    turns = 2048 * plain / (2 * math.pi)
    np.testing.assert_allclose(f[turns > 32], plain[turns > 32], rtol=2.0 ** -22)
    np.testing.assert_allclose(f[turns < 1], plain[turns < 1] / 4, rtol=2.0 ** -22)
    assert (turns > 32).any() and (turns < 1).any() and abs(c - (0.1 * math.log(4) + 1)) < 1e-12


def test_dims_copies_make_their_own_records():
    """The address that the binding module reads belongs to one object: copies and pickles do not take it along."""
    import copy
    import pickle

    d = swa.Dims(1, 2, 1, 16, 64, 0.25)
    first = d._dims_addr
    for e in (copy.copy(d), copy.deepcopy(d), pickle.loads(pickle.dumps(d))):
        assert e == d and "_record" not in e.__dict__ and e._dims_addr != first
    assert d._dims_addr == first and hash(d) == hash(swa.Dims(1, 2, 1, 16, 64, 0.25))
