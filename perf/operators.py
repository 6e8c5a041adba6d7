"""The operators of the 8-bit key/value cache: what is timed, and their plain forms.

Three operators that a serving program calls one after the other:

  slots   block tables and slot maps on the GPU from request lengths
  append  new K and V rows into the E4M3 cache, a scale per (block, head)
  attend  attention of each request's newest tokens over that cache

``own`` chooses between the plain forms below (elementary torch operations in
32 bits) and the framework's kernels.  A case is a dict of plain values; the
lengths of its requests follow from the case alone, the data from the seed.

The cache: codes uint8 [blocks, Hkv, P, d] for K and for V, scales fp32
[blocks, Hkv]; the value a code stands for is E4M3(code) * scale.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a few users decoding: the smallest call of a step, pure latency
        dict(name="slots decode 8", op="slots", requests=8, low=100, high=4000, new_low=1, new_high=1, block=16,
             mix=1),
        # a full decode batch: every request one token, some need a block
        dict(name="slots decode 1000", op="slots", requests=1000, low=1, high=8192, new_low=1, new_high=1, block=64,
             mix=2),
        # a wave of prompts of very different lengths, some behind a cached prefix
        dict(name="slots prompts 64", op="slots", requests=64, low=0, high=2000, new_low=1, new_high=4000, block=32,
             mix=3),
        # one layer's K and V of a small decode batch
        dict(name="append decode 32", op="append", requests=32, low=0, high=4096, new_low=1, new_high=1, block=64,
             heads_kv=8, d=128, mix=4),
        # a large decode batch, small head dim, small blocks
        dict(name="append decode 500 d64", op="append", requests=500, low=0, high=2048, new_low=1, new_high=1,
             block=16, heads_kv=16, d=64, mix=5),
        # ragged prompts, some continuing in a partly filled block
        dict(name="append prompts", op="append", requests=24, low=0, high=500, new_low=1, new_high=4096, block=64,
             heads_kv=8, d=128, mix=6),
        # one user, a short conversation: latency
        dict(name="attend decode 1", op="attend", requests=1, low=1000, high=1000, new_low=1, new_high=1, block=16,
             heads=32, heads_kv=8, d=128, mix=7),
        # the d = 64 batch of 32 heads, a head of its own for each query head
        dict(name="attend decode 16 d64", op="attend", requests=16, low=1, high=1024, new_low=1, new_high=1,
             block=32, heads=32, heads_kv=32, d=64, mix=8),
        # an ordinary decode batch of ragged lengths
        dict(name="attend decode 64", op="attend", requests=64, low=30, high=8192, new_low=1, new_high=1, block=64,
             heads=32, heads_kv=8, d=128, mix=9),
        # long contexts: the largest read of the cache
        dict(name="attend decode 32K", op="attend", requests=24, low=20000, high=32768, new_low=1, new_high=1,
             block=64, heads=64, heads_kv=8, d=128, mix=10),
        # drafted tokens checked against the cache, a few per request
        dict(name="attend draft 16", op="attend", requests=16, low=500, high=8192, new_low=2, new_high=5, block=128,
             heads=32, heads_kv=4, d=128, mix=11),
        # prompts, or chunks of them behind a cached prefix
        dict(name="attend prompts", op="attend", requests=3, low=700, high=10000, new_low=1500, new_high=4096,
             block=64, heads=32, heads_kv=8, d=128, mix=12),
    ]


def _logint(rng, low, high):
    """An integer of [low, high], spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(("slots", "append", "attend", "attend"))
    c = dict(op=op, block=rng.choice((16, 32, 64, 128)), mix=rng.randrange(1 << 20))
    if op == "slots":
        prompts = rng.random() < 0.5
        c.update(requests=_logint(rng, 1, 100 if prompts else 2000), low=rng.choice((0, 1, 300)),
                 high=_logint(rng, 300, 9000), new_low=rng.choice((0, 1)),
                 new_high=_logint(rng, 2, 3000) if prompts else 1)
        return c
    c["d"] = rng.choice((64, 128))
    if op == "append":
        c["heads_kv"] = rng.choice((1, 2, 4, 5, 8, 16))
        prompts = rng.random() < 0.5
        c.update(requests=_logint(rng, 1, 20 if prompts else 600), low=0, high=_logint(rng, 20, 4000),
                 new_low=1, new_high=_logint(rng, 2, 2500) if prompts else 1)
        return c
    c["heads_kv"] = rng.choice((1, 2, 4, 5, 8))
    c["heads"] = c["heads_kv"] * rng.choice((1, 2, 3, 4, 7, 8, 16))
    kind = rng.choice(("decode", "decode", "draft", "prompts"))
    high = _logint(rng, 40, 20000)
    c.update(low=max(1, high // rng.choice((1, 3, 40))), high=high)
    if kind == "prompts":
        c.update(requests=_logint(rng, 1, 4), new_low=1, new_high=_logint(rng, 50, 2500))
        c["low"], c["high"] = c["low"] % 4000, max(c["low"] % 4000, c["high"] % 6000)
        c["heads"] = min(c["heads"], 40 // c["heads_kv"] * c["heads_kv"])
    else:
        c.update(requests=_logint(rng, 1, max(2, 500000 // high) if high < 5000 else 24), new_low=1,
                 new_high=1 if kind == "decode" else rng.randint(2, 8))
        c["requests"] = min(c["requests"], 300)
    return c


def _lengths(case):
    """Tokens cached before the call and new tokens of each request; the last request is the longest."""
    rng = random.Random(case["mix"])
    R = case["requests"]
    held = [rng.randint(case["low"], case["high"]) for _ in range(R)]
    new = [rng.randint(case["new_low"], case["new_high"]) for _ in range(R)]
    held[-1], new[-1] = case["high"], case["new_high"]
    return held, new


def work(case):
    held, new = _lengths(case)
    R, P, T = case["requests"], case["block"], sum(new)
    up = lambda a: -(-a // P)  # noqa: E731
    if case["op"] == "slots":
        granted = sum(up(h + n) - up(h) for h, n in zip(held, new))
        started = sum(1 for h in held if h % P)
        return {"bytes": 8 * R + 4 * (granted + started) + 8 * T + 4 * granted + 8 * R + 12, "flops": 0}
    H, d = case["heads_kv"], case["d"]
    if case["op"] == "append":
        blocks = sum(up(h + n) - h // P for h, n in zip(held, new) if n)
        return {"bytes": 6 * T * H * d + 8 * T + 8 * blocks * H, "flops": 4 * T * H * d}
    Hq, total = case["heads"], [h + n for h, n in zip(held, new)]
    seen = sum(n * h + n * (n + 1) // 2 for h, n in zip(held, new))
    cache = sum(2 * t * H * d + (8 * H + 4) * up(t) for t in total)
    return {"bytes": cache + T * Hq * (4 * d + 4) + 8 * R, "flops": 4 * d * Hq * seen}


# ------------------------------------------------------------------ inputs

def _table(R, M, blocks, gen, want):
    """Block tables [R, M] of distinct blocks in no order, -1 behind each request's own."""
    perm = torch.randperm(blocks, generator=gen, device="cuda", dtype=torch.int32)
    want = torch.tensor(want, device="cuda")
    first = torch.cumsum(want, 0) - want
    j = torch.arange(M, device="cuda")
    at = (first[:, None] + j).clamp(max=blocks - 1)
    return torch.where(j < want[:, None], perm[at], perm.new_tensor(-1)).contiguous(), perm, int(sum(want.tolist()))


def _codes(x):
    """Codes and power-of-two scales of x [blocks, H, P, d]: how the cache comes to hold such values."""
    a = x.abs().amax(dim=(2, 3))
    s = torch.exp2(torch.ceil(torch.log2(a / 448)).clamp(-100, 120))
    return (x / s[:, :, None, None]).to(E4M3).view(torch.uint8), s


def _fill(blocks, H, P, d, gen):
    """A cache's codes and scales, blocks of different magnitude, made piece by piece."""
    c8 = torch.empty(blocks, H, P, d, dtype=torch.uint8, device="cuda")
    s = torch.empty(blocks, H, device="cuda")
    size = torch.exp2(torch.randint(-3, 2, (blocks, H), generator=gen, device="cuda").float())
    step = max(1, (1 << 27) // (H * P * d))
    for b in range(0, blocks, step):
        e = min(blocks, b + step)
        x = torch.randn(e - b, H, P, d, generator=gen, device="cuda") * size[b:e, :, None, None]
        c8[b:e], s[b:e] = _codes(x)
    return c8, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    held, new = _lengths(case)
    R, P, T = case["requests"], case["block"], sum(new)
    up = lambda a: -(-a // P)  # noqa: E731
    total = [h + n for h, n in zip(held, new)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    M = max(up(t) for t in total) + 1
    state = dict(op=case["op"], P=P, T=T, most=max(new))
    if case["op"] == "slots":
        blocks = sum(up(t) for t in total) + R + 7
        table, perm, used = _table(R, M, blocks, gen, [up(h) for h in held])
        state.update(table=table, lens=i32(held), new=i32(new), free=perm, used=i32([used]), T=T + 5)
        return state
    H, d = case["heads_kv"], case["d"]
    blocks = sum(up(t) for t in total) + 3
    table, _, _ = _table(R, M, blocks, gen, [up(t) for t in total])
    k8, ks = _fill(blocks, H, P, d, gen)
    v8, vs = _fill(blocks, H, P, d, gen)
    state.update(table=table, k8=k8, v8=v8, ks=ks, vs=vs, lens=i32(total), cu=i32(cu))
    if case["op"] == "append":
        # K and V as one projection leaves them: rows of K heads, then V heads
        size = torch.exp2(torch.randint(-2, 3, (T, 2 * H, 1), generator=gen, device="cuda").float())
        kv = (torch.randn(T, 2 * H, d, generator=gen, device="cuda") * size).to(torch.bfloat16)
        pos = torch.cat([torch.arange(h, h + n) for h, n in zip(held, new)]).cuda()
        row = torch.repeat_interleave(torch.arange(R), torch.tensor(new)).cuda()
        slots = table[row, pos // P].long() * P + pos % P
        state.update(k=kv[:, :H], v=kv[:, H:], slots=slots)
        return state
    # behind a request's last token its block holds whatever was there, NaN codes too
    last, off = [t // P for t in total], [t % P for t in total]
    for c8 in (k8, v8):
        for r in range(R):
            if off[r]:
                c8[table[r, last[r]].long(), :, off[r]:] = 0x7F
    q = torch.randn(T, case["heads"], d, generator=gen, device="cuda")
    q *= torch.exp2(torch.randint(-1, 2, (T, case["heads"], 1), generator=gen, device="cuda").float())
    state.update(q=q.to(torch.bfloat16), scale=1.0 / math.sqrt(d))
    return state


# --------------------------------------------------------------------- run

def run(s):
    if s["op"] == "slots":
        return _run_slots(s)
    return _run_append(s) if s["op"] == "append" else _run_attend(s)


def _cache(fa, s):
    return fa.CacheE4M3(s["k8"], s["v8"], s["ks"], s["vs"])


def _run_slots(s):
    table, lens, new, free, used, P, T = (s[k] for k in ("table", "lens", "new", "free", "used", "P", "T"))
    if own:
        import exact_attention_forward_04_gb300 as fa
        cu, slots, lens2, used2 = fa.cache_slots(table, lens, new, free, used, P, T)
        return dict(table=table, cu=cu, slots=slots, lens=lens2, used=used2)
    R, M = table.shape
    lens_l, new_l = lens.long(), new.long()
    cu = torch.zeros(R + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.cumsum(new_l, 0)
    held = (lens_l + P - 1) // P
    want = (lens_l + new_l + P - 1) // P
    fits = (want <= M) & (cu[1:] <= T)
    need = torch.where(fits, want - held, 0)
    end = torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (end <= free.numel() - used.long()))
    need = torch.where(ok, need, 0)
    first = used.long() + end - need
    j = torch.arange(M, device="cuda")
    fresh = (j >= held[:, None]) & (j < want[:, None]) & ok[:, None]
    at = (first[:, None] + j - held[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[at], table))
    t = torch.arange(T, device="cuda")
    row = torch.searchsorted(cu, t, right=True) - 1
    inside = row < R
    row = row.clamp(max=R - 1)
    pos = lens_l[row] + t - cu[row]
    inside = inside & ok[row]
    slot = table[row, (pos // P).clamp(max=M - 1)].long() * P + pos % P
    slots = torch.where(inside, slot, -1)
    lens2 = (lens_l + torch.where(ok, new_l, 0)).int()
    return dict(table=table, cu=cu.int(), slots=slots, lens=lens2, used=(used.long() + need.sum()).int())


def _run_append(s):
    k, v, slots, P = s["k"], s["v"], s["slots"], s["P"]
    if own:
        import exact_attention_forward_04_gb300 as fa
        fa.cache_append_e4m3(k, v, _cache(fa, s), slots)
    else:
        _append_plain(k, s["k8"], s["ks"], slots, P)
        _append_plain(v, s["v8"], s["vs"], slots, P)
    return dict(k=s["k8"].view(E4M3), v=s["v8"].view(E4M3), k_scale=s["ks"], v_scale=s["vs"])


def _append_plain(x, c8, scale, slots, P):
    T, H, d = x.shape
    x = x.float()
    block, off = slots // P, slots % P
    uniq, inv = torch.unique(block, return_inverse=True)
    n = uniq.numel()
    amax = torch.zeros(n, H, device="cuda").scatter_reduce(0, inv[:, None].expand(T, H), x.abs().amax(-1), "amax")
    first = torch.full((n,), P, dtype=torch.int64, device="cuda").scatter_reduce(0, inv, off, "amin")
    # the smallest power of two that takes the largest value to 448 at most
    frac, exp = torch.frexp(amax / 448)
    exp = torch.where(frac == 0.5, exp - 1, exp).clamp(-100, 120)
    want = torch.ldexp(torch.ones_like(amax), exp)
    old = scale[uniq]
    now = torch.where(first[:, None] > 0, torch.maximum(old, want), want)
    kept = torch.arange(P, device="cuda") < first[:, None]
    have = c8[uniq].view(E4M3).float()
    again = (have * (old / now)[:, :, None, None]).to(E4M3).view(torch.uint8)
    grown = kept[:, None, :] & (now > old)[:, :, None]
    c8[uniq] = torch.where(grown[..., None], again, c8[uniq])
    scale[uniq] = now
    c8[block, :, off] = (x / now[inv][:, :, None]).to(E4M3).view(torch.uint8)


def _run_attend(s):
    q, table, lens, cu, P = s["q"], s["table"], s["lens"], s["cu"], s["P"]
    if own:
        import exact_attention_forward_04_gb300 as fa
        o, lse = fa.cache_forward_e4m3(q, _cache(fa, s), table, lens, cu, scale=s["scale"])
        return dict(o=o, lse=lse)
    T, Hq, d = q.shape
    R, M = table.shape
    H = s["ks"].shape[1]
    g, n = Hq // H, s["most"]
    at = table.clamp(min=0).long()
    seen = torch.arange(M * P, device="cuda") < lens[:, None]

    def values(c8, sc):
        x = c8[at].view(E4M3).float() * sc[at][..., None, None]             # [R, M, H, P, d]
        x = x.permute(0, 2, 1, 3, 4).reshape(R, H, M * P, d)
        return torch.where(seen[:, None, :, None], x, 0)

    k, v = values(s["k8"], s["ks"]), values(s["v8"], s["vs"])
    count = (cu[1:] - cu[:-1]).long()
    i = torch.arange(n, device="cuda")
    rows = (cu[:-1, None] + i).clamp(max=T - 1).long()                      # [R, n]
    x = q.float()[rows].view(R, n, H, g, d).permute(0, 2, 1, 3, 4).reshape(R, H, n * g, d)
    sc = torch.matmul(x, k.transpose(2, 3)).mul_(s["scale"])
    pos = (lens.long() - count)[:, None] + i                                # [R, n]
    hide = torch.arange(M * P, device="cuda") > pos.repeat_interleave(g, 1)[..., None]
    sc.masked_fill_((hide | ~seen[:, None, :])[:, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(m).exp_()
    tot = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / tot
    lse = (m + torch.log(tot)).squeeze(-1)
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(cu, t, right=True) - 1
    o = o.view(R, H, n, g, d).permute(0, 2, 1, 3, 4).reshape(R, n, Hq, d)[r, t - cu[r]]
    lse = lse.view(R, H, n, g).permute(0, 2, 1, 3).reshape(R, n, Hq)[r, t - cu[r]]
    return dict(o=o.to(torch.bfloat16), lse=lse)


# ------------------------------------------------------------------- exact

def _value64(c8):
    """The value of each code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F is NaN."""
    c = torch.arange(256, dtype=torch.int64, device="cuda")
    e, m = (c >> 3) & 15, (c & 7).double()
    val = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e.double() - 7))
    val = torch.where((c & 127) == 127, math.nan, val) * torch.where(c >= 128, -1.0, 1.0)
    return val[c8.long()]


def _round64(y):
    """Nearest E4M3 value, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _scale64(a):
    """The smallest power of two s with a <= 448 s, its exponent within [-100, 120]."""
    s = torch.exp2(torch.round(torch.log2(a.clamp(min=2.0 ** -120) / 448)))
    s = torch.where(a > 448 * s, 2 * s, s)
    s = torch.where(a <= 224 * s, s / 2, s)
    return s.clamp(2.0 ** -100, 2.0 ** 120)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "slots":
        return None
    P, H = s["P"], s["ks"].shape[1]
    if case["op"] == "append":
        out = {}
        held, new = _lengths(case)
        table = s["table"].tolist()
        for name, x, c8, sc in (("k", s["k"], s["k8"], s["ks"]), ("v", s["v"], s["v8"], s["vs"])):
            val, sc, x = _value64(c8), sc.double(), x.double()
            t = 0
            for r, (h, n) in enumerate(zip(held, new)):
                while n > 0:                                               # block by block
                    b, off = table[r][h // P], h % P
                    m = min(n, P - off)
                    part = x[t:t + m].transpose(0, 1)                      # [H, m, d]
                    want = _scale64(part.abs().amax((1, 2)))
                    if off:
                        was, want = sc[b].clone(), torch.maximum(sc[b], want)
                        ratio = (was / want)[:, None, None]
                        val[b, :, :off] = torch.where(ratio < 1, _round64(val[b, :, :off] * ratio), val[b, :, :off])
                    sc[b] = want
                    val[b, :, off:off + m] = _round64(part / want[:, None, None])
                    t, h, n = t + m, h + m, n - m
            out[name], out[name + "_scale"] = val, sc
        return out
    if work(case)["flops"] > 6e12:
        return None
    T, Hq, d = s["q"].shape
    g = Hq // H
    o = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, Hq, dtype=torch.float64, device="cuda")
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].long()
    for r in range(len(lens)):
        n, N = cu[r + 1] - cu[r], lens[r]
        if n == 0:
            continue
        at = table[r, :-(-N // P)]
        later = torch.arange(N, device="cuda") > (N - n + torch.arange(n, device="cuda"))[:, None]
        for h in range(H):
            k = (_value64(s["k8"][at, h]) * s["ks"][at, h].double()[:, None, None]).reshape(-1, d)[:N]
            v = (_value64(s["v8"][at, h]) * s["vs"][at, h].double()[:, None, None]).reshape(-1, d)[:N]
            for j in range(h * g, h * g + g):
                z = s["q"][cu[r]:cu[r + 1], j].double() @ k.T * s["scale"]
                z[later] = -math.inf
                lse[cu[r]:cu[r + 1], j] = torch.logsumexp(z, -1)
                o[cu[r]:cu[r + 1], j] = torch.softmax(z, -1) @ v
    return dict(o=o, lse=lse)
