"""The table of the "yarn" form of rotary positions, pair by pair."""
import math

import pytest

import sliding_window_gqa_chunk_b200 as swa


def table(monkeypatch, r, **kw):
    made = {}
    monkeypatch.setattr(swa, "Rope", lambda f, i, c: made.update(f=f.double().tolist(), c=c))
    swa.new_rope(r, device="cpu", scaling="yarn", **kw)
    return made["f"], made["c"]


def test_the_middle_of_the_ramp(monkeypatch):
    # 128, base 10000, 4096: 32 turns at index 64 ln(4096 / 64 pi) / ln 10000 = 20.94, one at 64 ln(4096 / 2 pi) / ln 10000 = 45.03:
    # the ramp goes from 20 to 46, and pair 33 is half slowed
    f, c = table(monkeypatch, 128, scale=8.0, original_length=4096)
    plain = [10000.0 ** (-i / 64) for i in range(64)]
    near = dict(rel=2.0 ** -22)                   # fp32 tables
    assert f[20] == pytest.approx(plain[20], **near) and f[46] == pytest.approx(plain[46] / 8, **near)
    assert f[33] == pytest.approx(plain[33] * (0.5 + 0.5 / 8), **near)
    assert f[27] == pytest.approx(plain[27] * (19 + 7 / 8) / 26, **near)
    assert c == pytest.approx(0.1 * math.log(8) + 1)


@pytest.mark.parametrize("r,base,length,scale", [(16, 10000.0, 4096, 4.0), (96, 500000.0, 8192, 16.0), (64, 1e6, 32768, 2.5), (128, 150.0, 4096, 32.0),
                                                 (64, 10000.0, 100, 4.0), (32, 10000.0, 5, 4.0), (16, 2.0, 100000, 4.0), (2, 10000.0, 4096, 4.0)])
def test_every_pair(monkeypatch, r, base, length, scale):
    f, _ = table(monkeypatch, r, base=base, scale=scale, original_length=length)
    low = max(math.floor(r * math.log(length / (64 * math.pi)) / (2 * math.log(base))), 0)
    high = min(math.ceil(r * math.log(length / (2 * math.pi)) / (2 * math.log(base))), r - 1)
    last = 0.0
    for i in range(r // 2):
        plain = base ** (-2 * i / r)
        turns = length * plain / (2 * math.pi)
        part = 0.0 if turns > 32 else 1.0 if turns < 1 else min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        assert f[i] == pytest.approx(plain * (1 - part) + plain / scale * part, rel=2.0 ** -22)
        assert part >= last
        last = part


def test_a_base_that_does_not_slow_the_pairs_is_refused():
    for base in (1.0, 0.5):
        with pytest.raises(ValueError, match="base"):
            swa.new_rope(32, base=base, scaling="yarn", scale=2.0, device="cpu")
