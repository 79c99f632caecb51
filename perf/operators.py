"""Workloads of the 8-bit rolling cache and of the rotary positions, for measuring them.

Four operators, each with its plain form in elementary torch operations and the call a user makes
of the library (`own`):

* ``rope``    rotary positions on a chunk's q and k (or one token's, in decode), forward and the
              transposed rotation (the gradient);
* ``append``  a chunk's keys and values into the rolling cache held in 8 bits: blocks of 64 slots
              share one power-of-two scale for each kv head, and the block still being filled is
              kept in bf16 (the tail);
* ``prefill`` attention of a chunk over that cache and, causally, over itself;
* ``decode``  one token per sequence over that cache, which takes the token in.

Shapes are the ones the attention calls of this repository are used with: 32 query heads over 8 kv
heads of 128 with a window of 4096, the tiny shape with 16-wide heads, and odd ones around them.
"""
import math
import random

import torch

own = False

BLOCK = 64
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases

def _rope(name, batch, tokens, q_heads, kv_heads, dim, rotary, interleaved, transpose, packed, scaling, far):
    return dict(name=name, op="rope", batch=batch, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                rotary=rotary, interleaved=interleaved, transpose=transpose, packed=packed, scaling=scaling, far=far)


def _cache(op, name, batch, tokens, q_heads, kv_heads, dim, window, fmt, kind):
    return dict(name=name, op=op, batch=batch, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                window=window, fmt=fmt, kind=kind)


def listed():
    return [
        # one sequence's next token: launch latency is all there is
        _rope("rope_decode_b1", 1, 1, 32, 8, 128, 128, False, False, False, "none", False),
        # one prefill chunk of a long prompt, q and k taken out of the packed projection
        _rope("rope_chunk_4096", 1, 4096, 32, 8, 128, 128, False, False, True, "yarn", False),
        # gradient of a ragged batch: pairs side by side, half the head rotated, far positions
        _rope("rope_grad_ragged", 3, 1001, 12, 4, 64, 32, True, True, False, "linear", True),
        # one prefill chunk into an empty or full ring
        _cache("append", "append_chunk_4096", 1, 4096, 32, 8, 128, 4096, "e4m3", "full"),
        # a padded batch of short pieces into small rings whose last block is not whole
        _cache("append", "append_ragged", 8, 333, 16, 4, 64, 1000, "int8", "ragged"),
        # interactive decode, one sequence
        _cache("decode", "decode_b1", 1, 1, 32, 8, 128, 4096, "e4m3", "full"),
        # a medium batch, the other format
        _cache("decode", "decode_b16_int8", 16, 1, 32, 8, 128, 4096, "int8", "full"),
        # the throughput case
        _cache("decode", "decode_b64", 64, 1, 32, 8, 128, 4096, "e4m3", "full"),
        # a mixed batch: short and long sequences, group of 7, odd window
        _cache("decode", "decode_ragged", 37, 1, 14, 2, 64, 1000, "e4m3", "ragged"),
        # a later chunk of a long prompt: the whole window is cached
        _cache("prefill", "prefill_chunk_4096", 1, 4096, 32, 8, 128, 4096, "e4m3", "full"),
        # a padded batch of prompt pieces, some at their start
        _cache("prefill", "prefill_ragged", 6, 500, 32, 8, 128, 2000, "int8", "ragged"),
        # a few tokens for each of several long sequences (drafts to be verified, prompt ends)
        _cache("prefill", "prefill_short", 16, 4, 32, 8, 128, 4096, "e4m3", "full"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "prefill"])
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 4, 7, 8, 12, 16]) if op == "decode" else rng.choice([1, 2, 4, 4, 7, 8])
    dim = rng.choice([16, 64, 128, 128])
    window = _log(rng, 4, 8192)
    fmt = rng.choice(["e4m3", "int8"])
    kind = rng.choice(["full", "ragged"])
    if op == "rope":
        rotary = rng.choice([r for r in (16, 32, 64, 96, 128) if r <= dim])
        tokens = _log(rng, 1, 8192)
        batch = min(_log(rng, 1, 128), max(1, 4096 * 40 * 128 // (tokens * kv * (group + 1) * dim)))
        return _rope_drawn(batch, tokens, kv * group, kv, dim, rotary, rng)
    if op == "append":
        tokens = min(window, _log(rng, 1, 8192))
        batch = min(_log(rng, 1, 64), max(1, 8192 * 8 * 128 // (max(tokens, window // 4) * kv * dim)))
    elif op == "decode":
        tokens = 1
        batch = min(_log(rng, 1, 200), max(1, 64 * 8 * 4096 * 128 // (window * kv * dim)))
    else:
        tokens = min(window, _log(rng, 1, 4096))
        batch = min(_log(rng, 1, 24), max(1, 32 * 4096 * 8192 // (tokens * kv * group * (window + tokens))),
                    max(1, 64 * 8 * 4096 * 128 // (4 * window * kv * dim)))
    c = _cache(op, "", batch, tokens, kv * group, kv, dim, window, fmt, kind)
    del c["name"]
    return c


def _rope_drawn(batch, tokens, q_heads, kv_heads, dim, rotary, rng):
    c = _rope("", batch, tokens, q_heads, kv_heads, dim, rotary, rng.random() < 0.5, rng.random() < 0.4,
              rng.random() < 0.5, rng.choice(["none", "linear", "yarn"]), rng.random() < 0.3)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _counts(case, seed):
    """Each sequence's first position and number of tokens, as lists.

    An append that starts inside a block and ends inside a later one replaces the tail it has read,
    so a second pass over the same state would read other rows: such a start is moved to its
    block's first slot (the others read or leave the tail as it is)."""
    r = random.Random(seed * 7919 + 17)
    W, T, op = case.get("window", 0), case["tokens"], case["op"]
    starts, counts = [], []
    for b in range(case["batch"]):
        if op == "rope":
            s = r.randrange(1 << 20, (1 << 31) - T) if case["far"] else r.randrange(0, 32768)
            n = T if b == 0 or case["batch"] < 3 else r.randint(0, T)
        elif case["kind"] == "full":
            s, n = r.randrange(W, 8 * W + 1), T
        else:
            s = r.choice([0, r.randrange(0, W), r.randrange(W, 8 * W + 1)])
            n = T if b == 0 else r.randint(0 if op != "decode" else 1, T)
        if op == "append" and n:
            row = (s % W) % BLOCK
            last = (s + n - 1) % W
            ends = (last + 1) % BLOCK == 0 or last + 1 == W
            same = row + n <= min(BLOCK, W - (s % W - row))
            if row and not ends and not same:
                s -= row
        starts.append(s)
        counts.append(n)
    return starts, counts


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _quantise(x, fmt):
    """x [..., rows, d] (one block): 8-bit values and the block's scale, the smallest power of two
    that brings the largest magnitude to the format's range (1 for a block of zeros)."""
    top = 448.0 if fmt == "e4m3" else 127.0
    amax = x.abs().amax(dim=(-1, -2))
    m, e = torch.frexp(amax / top)  # amax / top = m 2^e, m in [0.5, 1): the next power of two is 2^e
    e = torch.where(m == 0.5, e - 1, e).clamp(-100, 127)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    y = x / scale[..., None, None]
    y = y.to(FP8) if fmt == "e4m3" else torch.round(y).to(torch.int8)
    return y, scale


def _rows(gen, *shape):
    """Keys or values: normal, with a few channels that are larger than the others, as keys have."""
    x = torch.randn(shape, generator=gen, device="cuda")
    gain = torch.ones(shape[-1], device="cuda")
    gain[torch.randint(0, shape[-1], (max(1, shape[-1] // 32),), generator=gen, device="cuda")] = 6.0
    return (x * gain).to(torch.bfloat16)


def _ring(gen, case):
    B, H, W, d = case["batch"], case["kv_heads"], case["window"], case["dim"]
    n = -(-W // BLOCK)
    q = torch.empty((B, H, W, d), dtype=torch.int8, device="cuda")
    q = q.view(FP8) if case["fmt"] == "e4m3" else q
    scale = torch.empty((B, H, n), device="cuda")
    for b in range(B):
        x = _rows(gen, H, n * BLOCK, d).float()
        # what a sequence holds changes its size slowly: the blocks' scales differ
        x *= torch.exp2(torch.randint(-2, 3, (H, n, 1), generator=gen, device="cuda").float()).repeat_interleave(BLOCK, 1)
        y, s = _quantise(x.view(H, n, BLOCK, d), case["fmt"])
        q.view(torch.int8)[b] = y.view(torch.int8).view(H, n * BLOCK, d)[:, :W]
        scale[b] = s
    return q, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, T, Hq, H, d = (case[k] for k in ("batch", "tokens", "q_heads", "kv_heads", "dim"))
    starts, counts = _counts(case, seed)
    s = dict(case=case, start=_i32(starts), count=_i32(counts))
    if case["op"] == "rope":
        if case["packed"]:
            qkv = torch.randn((B, T, Hq + 2 * H, d), generator=gen, device="cuda").to(torch.bfloat16)
            s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H]
        else:
            s["q"] = torch.randn((B, T, Hq, d), generator=gen, device="cuda").to(torch.bfloat16)
            s["k"] = torch.randn((B, T, H, d), generator=gen, device="cuda").to(torch.bfloat16)
        s["q_out"] = torch.randn((B, T, Hq, d), generator=gen, device="cuda").to(torch.bfloat16)
        s["k_out"] = torch.randn((B, T, H, d), generator=gen, device="cuda").to(torch.bfloat16)
        i = torch.arange(0, case["rotary"], 2, dtype=torch.float64)
        freq = 10000.0 ** (-i / case["rotary"])
        s["factor"] = 1.0
        if case["scaling"] == "linear":
            freq = freq / 4
        elif case["scaling"] == "yarn":  # long waves are stretched, short ones kept, a ramp between
            turns = 4096 * freq / (2 * math.pi)
            keep = ((turns - 1) / 31).clamp(0, 1)
            freq = freq * keep + freq / 8 * (1 - keep)
            s["factor"] = 0.1 * math.log(8) + 1
        s["freq"] = freq.float().cuda()
        if own:
            import sliding_window_gqa_chunk_b200 as swa
            s["dims"] = swa.Dims(B, Hq, H, d, 1, 1.0, "bf16")
            s["rope"] = swa.Rope(s["freq"], case["interleaved"], s["factor"])
        return s
    k8, ks = _ring(gen, case)
    v8, vs = _ring(gen, case)
    s.update(k8=k8, v8=v8, ks=ks, vs=vs, kt=_rows(gen, B, H, BLOCK, d), vt=_rows(gen, B, H, BLOCK, d))
    shape = (B, T) if case["op"] != "decode" else (B,)
    s["k"], s["v"] = _rows(gen, *shape, H, d), _rows(gen, *shape, H, d)
    s["scale"] = d ** -0.5
    if case["op"] != "append":
        s["q"] = torch.randn((*shape, Hq, d), generator=gen, device="cuda").to(torch.bfloat16)
        s["out"] = torch.randn((*shape, Hq, d), generator=gen, device="cuda").to(torch.bfloat16)
    return _handles(s) if own else s


def _handles(s):
    """What a user's program keeps beside its tensors: the dims, the cache's handle and a workspace."""
    import sliding_window_gqa_chunk_b200 as swa
    c = s["case"]
    s["dims"] = swa.Dims(c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["window"], s["scale"], "bf16")
    s["cache"] = swa.CacheQ8(s["k8"], s["v8"], s["ks"], s["vs"], s["kt"], s["vt"])
    if c["op"] == "prefill":
        s["ws"] = swa.prefill_workspace_q8(s["dims"], c["tokens"])
    elif c["op"] == "decode":
        s["ws"] = swa.decode_workspace_q8(s["dims"])
    return s


# ---------------------------------------------------------------- plain forms

def _plain_rope(s):
    c = s["case"]
    T, r = c["tokens"], c["rotary"]
    t = torch.arange(T, device="cuda")
    angle = (s["start"].double()[:, None] + t)[..., None] * s["freq"].double()  # [B, T, r / 2]
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    if c["transpose"]:
        sin = -sin
    live = (t < s["count"][:, None])[..., None, None]

    def turn(x, old):
        y = x.float().clone()
        a, b = (y[..., 0:r:2], y[..., 1:r:2]) if c["interleaved"] else (y[..., : r // 2], y[..., r // 2: r])
        na, nb = (a * cos - b * sin) * s["factor"], (b * cos + a * sin) * s["factor"]
        a.copy_(na)
        b.copy_(nb)
        return old.copy_(torch.where(live, y.to(torch.bfloat16), old))

    return turn(s["q"], s["q_out"]), turn(s["k"], s["k_out"])


def _spread(scale, W):
    return scale.repeat_interleave(BLOCK, dim=-1)[..., :W, None]


def _plain_held(s, q8, scale, tail, filled):
    """The ring's values in fp32: the block being filled has its first rows (slots in `filled`) in the tail."""
    W = q8.shape[2]
    row = (torch.arange(W, device="cuda") % BLOCK)[None, None, :, None].expand(*q8.shape)
    return torch.where(filled[:, None, :, None], tail.float().gather(2, row), q8.float() * _spread(scale, W))


def _plain_store(s, q8, scale, tail, new, start, count):
    """new [B, T, H, d] taken in from position start on: whole blocks in 8 bits, the last one's rows in the tail."""
    B, H, W, d = q8.shape
    n, T = scale.shape[-1], new.shape[1]
    start, end = start.long()[:, None], (start.long() + count.long())[:, None]
    # the blocks that T tokens can reach, from the first token's on
    m = min(n, (T + BLOCK - 2) // BLOCK + 2)
    block = (start % W // BLOCK + torch.arange(m, device="cuda")) % n  # [B, m]
    first = block * BLOCK
    last = (first + BLOCK - 1).clamp(max=W - 1)
    full_at = start + (last - start) % W  # the position that next fills the block up
    done = full_at < end
    # a block's rows; where the ring's last block is short, its last row stands for those it lacks
    row = torch.minimum(torch.arange(BLOCK, device="cuda"), (last - first)[..., None])  # [B, m, 64]
    at = (full_at - (last - first))[..., None] + row
    fresh = (at >= start[..., None])[:, None, ..., None]
    where = (at - start[..., None]).clamp(0, T - 1).view(B, -1, 1, 1).expand(B, m * BLOCK, H, d)
    rows = new.gather(1, where).view(B, m, BLOCK, H, d).permute(0, 3, 1, 2, 4)
    old = tail.gather(2, row.view(B, 1, -1, 1).expand(B, H, m * BLOCK, d)).view(B, H, m, BLOCK, d)
    y, sc = _quantise(torch.where(fresh, rows, old).float(), s["case"]["fmt"])
    slot = (first[..., None] + row).view(B, 1, -1, 1).expand(B, H, m * BLOCK, d)
    held = q8.view(torch.int8)
    y = torch.where(done[:, None, :, None, None], y.view(torch.int8), held.gather(2, slot).view(y.shape))
    held.scatter_(2, slot, y.reshape(slot.shape))
    index = block[:, None].expand(B, H, m)
    scale.scatter_(2, index, torch.where(done[:, None], sc, scale.gather(2, index)))
    # the block that the last token leaves unfilled
    stop = (end - 1) % W
    whole = stop == (stop // BLOCK * BLOCK + BLOCK - 1).clamp(max=W - 1)
    left = end - 1 - stop % BLOCK + torch.arange(BLOCK, device="cuda")  # [B, 64]
    keep = (left >= start) & (left < end) & ~whole
    rows = new.gather(1, (left - start).clamp(0, T - 1)[..., None, None].expand(B, BLOCK, H, d)).permute(0, 2, 1, 3)
    tail.copy_(torch.where(keep[:, None, :, None], rows, tail))


def _plain_append(s):
    _plain_store(s, s["k8"], s["ks"], s["kt"], s["k"], s["start"], s["count"])
    _plain_store(s, s["v8"], s["vs"], s["vt"], s["v"], s["start"], s["count"])
    return _cache_out(s)


def _cache_out(s):
    return [s[k] for k in ("k8", "v8", "ks", "vs", "kt", "vt")]


def _softmax_sum(x, v):
    """softmax over the last axis of x (masked places are -inf) times v, in fp32."""
    x -= x.amax(dim=-1, keepdim=True)
    x.exp_()
    return torch.matmul(x, v) / x.sum(dim=-1, keepdim=True)


def _plain_decode(s):
    W, B = s["case"]["window"], s["case"]["batch"]
    H, d = s["case"]["kv_heads"], s["case"]["dim"]
    slot = torch.arange(W, device="cuda")
    pos = s["start"].long()[:, None]
    at = pos % W
    filled = (slot >= at - at % BLOCK) & (slot < at)
    new, seen = slot == at, (slot <= pos)[:, None, None]
    k = _plain_held(s, s["k8"], s["ks"], s["kt"], filled)
    v = _plain_held(s, s["v8"], s["vs"], s["vt"], filled)
    k = torch.where(new[:, None, :, None], s["k"].float()[:, :, None], k)
    v = torch.where(new[:, None, :, None], s["v"].float()[:, :, None], v)
    q = s["q"].float().view(B, H, -1, d) * s["scale"]
    x = torch.matmul(q, k.transpose(-1, -2)).masked_fill_(~seen, -math.inf)
    s["out"].copy_(_softmax_sum(x, v).reshape(B, -1, d))
    one = torch.ones_like(s["start"])
    _plain_store(s, s["k8"], s["ks"], s["kt"], s["k"][:, None], s["start"], one)
    _plain_store(s, s["v8"], s["vs"], s["vt"], s["v"][:, None], s["start"], one)
    return [s["out"], *_cache_out(s)]


def _plain_prefill(s):
    c = s["case"]
    B, T, W, H, d = c["batch"], c["tokens"], c["window"], c["kv_heads"], c["dim"]
    slot, t = torch.arange(W, device="cuda"), torch.arange(T, device="cuda")
    start = s["start"].long()[:, None]
    at = start % W
    filled = (slot >= at - at % BLOCK) & (slot < at)
    held = start - 1 - (start - 1 - slot) % W  # [B, W]: the position that each slot holds (below 0: none)
    k = torch.cat([_plain_held(s, s["k8"], s["ks"], s["kt"], filled), s["k"].float().transpose(1, 2)], dim=2)
    v = torch.cat([_plain_held(s, s["v8"], s["vs"], s["vt"], filled), s["v"].float().transpose(1, 2)], dim=2)
    at_key = torch.cat([held, start + t], dim=1)[:, None]  # [B, 1, W + T]
    at_row = (start + t)[..., None]
    seen = (at_key >= 0) & (at_key <= at_row) & (at_key > at_row - W)  # [B, T, W + T]
    q = s["q"].float().view(B, T, H, -1, d).permute(0, 2, 3, 1, 4) * s["scale"]  # [B, H, G, T, d]
    x = torch.matmul(q, k[:, :, None].transpose(-1, -2)).masked_fill_(~seen[:, None, None], -math.inf)
    y = _softmax_sum(x, v[:, :, None]).permute(0, 3, 1, 2, 4).reshape(B, T, -1, d)
    live = (t < s["count"][:, None])[..., None, None]
    return s["out"].copy_(torch.where(live, y.to(torch.bfloat16), s["out"]))


# ---------------------------------------------------------------- the pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill}[c["op"]](s)
    import sliding_window_gqa_chunk_b200 as swa
    if c["op"] == "rope":
        swa.rope(s["dims"], s["rope"], s["q_out"], s["k_out"], s["q"], s["k"], s["start"], s["count"], transpose=c["transpose"])
        return s["q_out"], s["k_out"]
    if c["op"] == "append":
        swa.cache_append_q8(s["dims"], s["cache"], s["k"], s["v"], s["start"], s["count"])
        return _cache_out(s)
    if c["op"] == "prefill":
        swa.prefill_chunk_q8(s["dims"], s["out"], s["q"], s["k"], s["v"], s["cache"], s["start"], s["count"], s["ws"])
        return s["out"]
    swa.decode_q8(s["dims"], s["out"], s["q"], s["k"], s["v"], s["cache"], s["start"], s["ws"])
    return [s["out"], *_cache_out(s)]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    B, T, Hq, H, d = (c[k] for k in ("batch", "tokens", "q_heads", "kv_heads", "dim"))
    starts, counts = _counts(c, 0)
    n = sum(counts)
    if c["op"] == "rope":
        return {"bytes": n * (Hq + H) * d * 4 + c["rotary"] * 2, "flops": n * (Hq + H) * c["rotary"] * 3}
    W = c["window"]
    if c["op"] == "append":
        return {"bytes": n * H * d * 2 * 3, "flops": n * H * d * 2 * 2}
    pairs = held = 0
    for s, m in zip(starts, counts):
        if c["op"] == "decode":
            held += min(s, W - 1)
            pairs += min(s + 1, W)
        elif m:
            held += min(s, W - 1)
            pairs += sum(min(s + t + 1, W) for t in range(m))
    return {"bytes": held * H * d * 2 + n * (2 * Hq + 2 * H) * d * 2, "flops": pairs * Hq * d * 4}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "decode": _exact_decode, "prefill": _exact_prefill}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    r, sign = c["rotary"], -1.0 if c["transpose"] else 1.0
    outs = []
    for name in ("q", "k"):
        y = s[name + "_out"].double()
        for b, (p, n) in enumerate(zip(s["start"].tolist(), s["count"].tolist())):
            x = s[name][b, :n].double()
            y[b, :n] = x
            for i, f in enumerate(s["freq"].double().tolist()):
                at = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
                turn = sign * f * torch.arange(p, p + n, dtype=torch.float64, device="cuda")[:, None]
                z = torch.complex(x[..., at[0]], x[..., at[1]]) * torch.polar(torch.full_like(turn, s["factor"]), turn)
                y[b, :n, :, at[0]], y[b, :n, :, at[1]] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _exact_round(x, fmt):
    """x [rows, d] of one block in 64 bits: the 8-bit values, as numbers, and the scale."""
    amax, top = float(x.abs().max()), 448.0 if fmt == "e4m3" else 127.0
    scale = 1.0
    if amax > 0:
        scale = 2.0 ** max(-100, math.ceil(math.log2(amax)) - 12)
        while amax > scale * top:
            scale *= 2
    y = x / scale
    if fmt == "int8":
        return torch.round(y), scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, scale


def _exact_take(s, start, new_k, new_v, counts):
    """The cache after new_k[b], new_v[b] [T, H, d] from position start[b] on, token by token."""
    c = s["case"]
    W = c["window"]
    out = []
    for q8, scale, tail, new in (("k8", "ks", "kt", new_k), ("v8", "vs", "vt", new_v)):
        q8, scale, tail = s[q8].double(), s[scale].double(), s[tail].double()
        for b, (p0, n) in enumerate(zip(start, counts)):
            for h in range(c["kv_heads"]):
                room = tail[b, h].clone()
                p = p0
                while p < p0 + n:
                    row = (p % W) % BLOCK
                    j = (p % W) // BLOCK
                    size = min(BLOCK, W - j * BLOCK)
                    m = min(size - row, p0 + n - p)
                    room[row:row + m] = new[b, p - p0:p - p0 + m, h].double()
                    p += m
                    if row + m == size:
                        y, a = _exact_round(room[:size], c["fmt"])
                        q8[b, h, j * BLOCK:j * BLOCK + size], scale[b, h, j] = y, a
                    else:
                        tail[b, h, row:row + m] = room[row:row + m]
        out.append((q8, scale, tail))
    (a, b, e), (f, g, i) = out
    if c["fmt"] == "int8":
        a, f = None, None  # whole numbers: held to be equal to the plain form's
    return [a, f, b, g, e, i]


def _exact_append(s):
    if s["case"]["batch"] * s["case"]["kv_heads"] * (s["case"]["tokens"] / BLOCK + 2) > 40000:
        return None
    return _exact_take(s, s["start"].tolist(), s["k"], s["v"], s["count"].tolist())


def _exact_ring(s, b, p):
    """Sequence b's keys, values [H, n, d] and positions [n] before position p, oldest first."""
    W = s["case"]["window"]
    at = list(range(max(0, p - W + 1), p))
    idx = torch.tensor([x % W for x in at], dtype=torch.long, device="cuda")
    row, block = idx % BLOCK, idx // BLOCK
    # positions of the block that p falls into, once p is in it, are in the tail
    begin = p - (p % W) % BLOCK
    open_ = torch.tensor([x >= begin for x in at], dtype=torch.bool, device="cuda")[None, :, None]
    got = []
    for q8, scale, tail in (("k8", "ks", "kt"), ("v8", "vs", "vt")):
        packed = s[q8][b].view(torch.int8)[:, idx]
        x = (packed.view(FP8) if s["case"]["fmt"] == "e4m3" else packed).double() * s[scale][b].double()[:, block, None]
        got.append(torch.where(open_, s[tail][b].double()[:, row], x))
    return got[0], got[1], torch.tensor(at, dtype=torch.long, device="cuda")


def _exact_attend(s, b, p, q, k_new, v_new):
    """Rows q [n, Hq, d] at positions p.. over the ring before p and the new keys [n, H, d]."""
    c = s["case"]
    W, n = c["window"], q.shape[0]
    k, v, at = _exact_ring(s, b, p)
    here = p + torch.arange(n, device="cuda")
    at = torch.cat([at, here])
    see = (at[None] <= here[:, None]) & (at[None] > here[:, None] - W)
    y = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for h in range(c["kv_heads"]):
        kk, vv = torch.cat([k[h], k_new[:, h].double()]), torch.cat([v[h], v_new[:, h].double()])
        for g in range(h * (c["q_heads"] // c["kv_heads"]), (h + 1) * (c["q_heads"] // c["kv_heads"])):
            w = (q[:, g].double() @ kk.T) * s["scale"]
            y[:, g] = torch.softmax(w.masked_fill(~see, -math.inf), dim=-1) @ vv
    return y


def _exact_decode(s):
    y = torch.stack([_exact_attend(s, b, p, s["q"][b:b + 1], s["k"][b:b + 1], s["v"][b:b + 1])[0]
                     for b, p in enumerate(s["start"].tolist())])
    return [y, *_exact_take(s, s["start"].tolist(), s["k"][:, None], s["v"][:, None], [1] * s["case"]["batch"])]


def _exact_prefill(s):
    y = s["out"].double()
    for b, (p, n) in enumerate(zip(s["start"].tolist(), s["count"].tolist())):
        if n:
            y[b, :n] = _exact_attend(s, b, p, s["q"][b, :n], s["k"][b, :n], s["v"][b, :n])
    return y
