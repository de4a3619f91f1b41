"""The operators of the paged MXFP4 KV cache: what is measured, their plain forms and their values in 64 bits.

A KV cache holds keys and values in pages of P tokens. Per page and KV head there are two chunks, K
then V, of P * 17 d / 32 bytes: P rows of d/2 code bytes (E2M1, two per byte), then P rows of d/32
scale bytes (E8M0). Blocks of 32 run along d. The cache is one uint8 tensor
[pages, Hkv, 2, P, 17 d / 32]. Inside a chunk the bytes are interleaved:

* a K row holds word w (4 bytes, 8 codes) of block b at byte w * (d/8) + 4 b,
* a V row holds half-word h (2 bytes, 4 codes) of block b at byte h * (d/16) + 2 b,
* the scale rows of each 16 tokens are in another order: token i at (i % 8) * 2 + i / 8 for K, and
  at ((i % 8) / 2) * 4 + (i / 8) * 2 + i % 2 for V.

Four operators:

* plan: block tables and slot maps of a batch from its requests' lengths,
* append: quantize the new tokens' K and V into their slots (then read the slots back),
* attend: causal attention of a chunk of new tokens over the paged cache (one token each: decoding),
* cross: attention to an encoder's cached states of another length, with no causal mask.
"""
import math
import random

import torch

own = False

UOS, OCP = 1, 0
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _device():
    return torch.device("cuda", torch.cuda.current_device())


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decoding step of a batch: one token each, most pages already there
        {"name": "plan_decode_256", "op": "plan", "requests": 256, "ctx": 8192, "new": 1, "page": 16, "ragged": True},
        # a prefill batch: ragged prompts, every slot of about 65 thousand tokens
        {"name": "plan_prefill_64", "op": "plan", "requests": 64, "ctx": 0, "new": 2048, "page": 64, "ragged": True},
        # the tokens of one decoding step of 64 requests
        {"name": "append_decode_64", "op": "append", "tokens": 64, "kv_heads": 8, "d": 128, "page": 16, "uos": True},
        # an odd chunk of a prompt, small heads, the OCP exponent rule
        {"name": "append_odd_4099", "op": "append", "tokens": 4099, "kv_heads": 5, "d": 64, "page": 32, "uos": False},
        # a whole prefill of 4 x 8192 tokens
        {"name": "append_prefill_32768", "op": "append", "tokens": 32768, "kv_heads": 8, "d": 128, "page": 64, "uos": True},
        # the smallest call of a chat: one request, one token, a short context
        {"name": "decode_1x1000", "op": "attend", "requests": 1, "ctx": 1000, "new": 1, "heads": 32, "kv_heads": 8, "d": 128, "page": 16, "ragged": False},
        # a serving batch with ragged contexts, one token each
        {"name": "decode_64x8192", "op": "attend", "requests": 64, "ctx": 8191, "new": 1, "heads": 32, "kv_heads": 8, "d": 128, "page": 16, "ragged": True},
        # two long documents, four tokens each (drafted tokens to verify)
        {"name": "verify_2x131072", "op": "attend", "requests": 2, "ctx": 131068, "new": 4, "heads": 32, "kv_heads": 8, "d": 128, "page": 64, "ragged": False},
        # ragged chunks over ragged contexts, an odd group, small heads
        {"name": "chunk_7x777", "op": "attend", "requests": 7, "ctx": 3001, "new": 777, "heads": 15, "kv_heads": 3, "d": 64, "page": 32, "ragged": True},
        # a chunk of a long prompt: 2048 new tokens over 30 thousand
        {"name": "chunk_2048_over_30720", "op": "attend", "requests": 1, "ctx": 30720, "new": 2048, "heads": 32, "kv_heads": 8, "d": 128, "page": 64, "ragged": False},
        # two prompts of odd lengths attended to from a small latent
        {"name": "cross_2x1560", "op": "cross", "requests": 2, "ctx": 77, "new": 1560, "heads": 24, "kv_heads": 24, "d": 64, "page": 16, "ragged": True},
        # all latent tokens of a video attending to its prompt
        {"name": "cross_32760x512", "op": "cross", "requests": 1, "ctx": 512, "new": 32760, "heads": 40, "kv_heads": 40, "d": 128, "page": 64, "ragged": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend", "cross"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        new = rng.choice([1, 1, _log_int(rng, 2, 2048)])
        requests = min(_log_int(rng, 1, 1024), max(1, 65536 // new))
        return {"op": op, "requests": requests, "ctx": rng.choice([0, _log_int(rng, 1, 16384)]), "new": new, "page": page, "ragged": rng.random() < 0.8}
    d = rng.choice([64, 128])
    if op == "append":
        return {"op": op, "tokens": _log_int(rng, 1, 32768), "kv_heads": rng.choice([1, 2, 3, 4, 5, 8]), "d": d, "page": page, "uos": rng.random() < 0.5}
    if op == "cross":
        heads = rng.choice([1, 3, 8, 24, 40])
        requests = rng.randint(1, 4)
        return {"op": op, "requests": requests, "ctx": _log_int(rng, 1, 512), "new": _log_int(rng, 1, 32760 // requests), "heads": heads, "kv_heads": heads, "d": d,
                "page": page, "ragged": rng.random() < 0.5}
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    new = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 2, 1024)])
    requests = min(_log_int(rng, 1, 64), max(1, 4096 // new))
    most = min(65536, 400_000_000 // (requests * kv_heads * d), 2_000_000_000 // (requests * heads * new))
    ctx = rng.choice([0, _log_int(rng, 1, most), _log_int(rng, 1, most), rng.randint(most // 4, most)])
    return {"op": op, "requests": requests, "ctx": ctx, "new": new, "heads": heads, "kv_heads": kv_heads, "d": d, "page": page, "ragged": rng.random() < 0.7}


def _lengths(case):
    """(context length, new tokens) of each request: the same for every seed, but for their order."""
    rng = random.Random("%s %s %s %s" % (case["op"], case["requests"], case["ctx"], case["new"]))
    got = []
    for r in range(case["requests"]):
        ctx, new = case["ctx"], case["new"]
        if case["ragged"] and r > 0:  # one request has the full lengths
            ctx = rng.randint(0, ctx)
            if case["op"] != "cross":  # an encoder's states of another length; the queries of a batch are alike
                new = rng.randint(0 if new > 1 else 1, new)  # a request may sit a step out
        got.append((ctx, new))
    return got


# ------------------------------------------------------------------ the cache's bytes


def _order(values, device):
    return torch.tensor(values, device=device)


def _scale_order(which, device):
    """Position of token i's scale row among those of its 16 tokens."""
    if which == 0:
        return _order([(i % 8) * 2 + i // 8 for i in range(16)], device)
    return _order([((i % 8) // 2) * 4 + (i // 8) * 2 + i % 2 for i in range(16)], device)


def _encode(x, uos):
    """Codes [.., d] (0..15) and scale bytes [.., d/32] of x [.., d]."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    mant, e = torch.frexp(amax)  # amax = mant 2^e with mant in [1/2, 1)
    e = e - 3 + (mant > 0.90625).int() * int(uos)  # 7.25 / 8 = 0.90625
    e = torch.where(amax > 0, e, -127).clamp(-127, 127)
    y = torch.ldexp(b.abs().double(), -e.unsqueeze(-1))
    k = (y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
    return (k + 8 * torch.signbit(b).int()).flatten(-2).to(torch.uint8), (e + 127).to(torch.uint8)


def _pages_of(codes, scales, which):
    """One chunk a page, [.., P * 17 d / 32] bytes, of codes [.., P, d] and scales [.., P, d/32]."""
    P, d = codes.shape[-2:]
    nb, lead = d // 32, codes.shape[:-2]
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    parts = (4, 4) if which == 0 else (8, 2)
    packed = packed.reshape(*lead, P, nb, *parts).transpose(-3, -2).reshape(*lead, P * d // 2)
    at = _scale_order(which, codes.device)
    s = torch.empty_like(scales).reshape(*lead, P // 16, 16, nb)
    s[..., at, :] = scales.reshape(*lead, P // 16, 16, nb)
    return torch.cat([packed, s.reshape(*lead, P * nb)], -1)


def _values_of(chunk, P, which):
    """fp32 values [.., P, d] of chunks [.., P, 17 d / 32]."""
    d = chunk.shape[-1] * 32 // 17
    nb, lead = d // 32, chunk.shape[:-2]
    flat = chunk.reshape(*lead, P * nb * 17)
    parts = (4, 4) if which == 0 else (8, 2)
    packed = flat[..., : P * nb * 16].reshape(*lead, P, parts[0], nb, parts[1]).transpose(-3, -2).reshape(*lead, P, d // 2)
    s = flat[..., P * nb * 16 :].reshape(*lead, P // 16, 16, nb)[..., _scale_order(which, chunk.device), :].reshape(*lead, P, nb)
    codes = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=chunk.device)
    scale = torch.exp2(s.double() - 127.0).float()
    return (table[codes.int()].unflatten(-1, (nb, 32)) * scale.unsqueeze(-1)).flatten(-2)


# ------------------------------------------------------------------ inputs


def _batch(case, g, dev, seed):
    """Lengths, block table, free pages and pool size of a batch: every request's pages are random ones of the pool."""
    lens = _lengths(case)
    random.Random(seed).shuffle(lens)
    P = case["page"]
    held = [-(-c // P) for c, _ in lens]
    full = [-(-(c + n) // P) for c, n in lens] if case["op"] != "cross" else held
    width = max(max(full), 1)
    n_pages = sum(full) + 8
    pool = torch.randperm(n_pages, generator=g, device=dev).int()
    return lens, held, full, width, n_pages, pool


def _ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _table(counts, width, pool, dev):
    """A block table whose row r holds the next counts[r] pages of the pool, the rest -1."""
    c = _ints(counts, dev).long()
    first = c.cumsum(0) - c
    j = torch.arange(width, device=dev)
    at = (first[:, None] + j).clamp(max=pool.numel() - 1)
    return torch.where(j < c[:, None], pool[at], -1).int()


def _like_keys(shape, g, dev):
    """Rows as attention sees them: a few strong channels, and now and then an outlier."""
    x = torch.randn(shape, generator=g, device=dev)
    x[..., :4] *= 4.0
    x *= 1.0 + 15.0 * (torch.rand(shape[:-1], generator=g, device=dev) < 0.002).unsqueeze(-1)
    return x.bfloat16()


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    P = case["page"]
    if case["op"] == "append":
        T, H, d = case["tokens"], case["kv_heads"], case["d"]
        n_pages = -(-T // P) + 8
        slots = torch.randperm(n_pages, generator=g, device=dev)[:, None] * P + torch.arange(P, device=dev)
        return {"op": "append", "uos": case["uos"], "k": _like_keys((T, H, d), g, dev), "v": torch.randn(T, H, d, generator=g, device=dev).bfloat16(),
                "slots": slots.reshape(-1)[:T].contiguous(),  # the tokens follow one another through their pages
                "cache": torch.zeros(n_pages, H, 2, P, 17 * d // 32, dtype=torch.uint8, device=dev)}
    lens, held, full, width, n_pages, pool = _batch(case, g, dev, seed)
    ctx, new = _ints([c for c, _ in lens], dev), _ints([n for _, n in lens], dev)
    T = sum(n for _, n in lens)
    if case["op"] == "plan":
        return {"op": "plan", "ctx": ctx, "new": new, "table": _table(held, width, pool, dev), "free": pool[sum(held):].contiguous(), "page": P, "tokens": T}
    H, G, d = case["kv_heads"], case["heads"] // case["kv_heads"], case["d"]
    causal = case["op"] == "attend"
    k, v = (_like_keys((n_pages, H, P, d), g, dev), torch.randn(n_pages, H, P, d, generator=g, device=dev).bfloat16())
    cache = torch.stack([_pages_of(*_encode(k, True), 0), _pages_of(*_encode(v, True), 1)], 2).unflatten(-1, (P, 17 * d // 32)).contiguous()
    del k, v
    start = torch.zeros(len(lens) + 1, dtype=torch.int32, device=dev)
    start[1:] = new.cumsum(0)
    return {"op": case["op"], "q": torch.randn(T, H * G, d, generator=g, device=dev).bfloat16(), "cache": cache, "table": _table(full, width, pool, dev), "start": start,
            "kv": ctx + new if causal else ctx, "max_new": max(n for _, n in lens), "max_kv": max(c + n if causal else c for c, n in lens), "page": P}


# ------------------------------------------------------------------ one pass


def _plan(s):
    """Block table with the new pages, first token and length of each request, slot of each new token, and [new tokens, pages taken, requests refused, 0]."""
    ctx, new, P = s["ctx"].long(), s["new"].long(), s["page"]
    dev, T = ctx.device, s["tokens"]
    held, full = (ctx + P - 1) // P, (ctx + new + P - 1) // P
    need = full - held
    first = need.cumsum(0) - need  # of the free pages, this request's first
    start = torch.zeros(ctx.numel() + 1, dtype=torch.int64, device=dev)
    start[1:] = new.cumsum(0)
    j = torch.arange(s["table"].shape[1], device=dev)
    at = (first[:, None] + j - held[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where((j >= held[:, None]) & (j < full[:, None]), s["free"][at], s["table"])
    s["table"].copy_(table)
    t = torch.arange(T, device=dev)
    r = torch.searchsorted(start, t, right=True) - 1
    pos = ctx[r] + t - start[r]
    slots = table[r, pos // P].long() * P + pos % P
    zero = torch.zeros_like(start[-1])
    return {"table": s["table"], "start": start.int(), "kv": (ctx + new).int(), "slots": slots, "info": torch.stack([start[-1], need.sum(), zero, zero]).int()}


def _append(s):
    """The values that the slots hold once the new tokens are in the cache."""
    n_pages, H, _, P, row = s["cache"].shape
    nb = row // 17
    slots, got = s["slots"], []
    page, off = slots // P, slots % P
    flat = s["cache"].view(n_pages, H, 2, P * row)
    h = torch.arange(H, device=slots.device)
    for which, x in ((0, s["k"]), (1, s["v"])):
        codes, scales = _encode(x, s["uos"])
        packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
        parts = (4, 4) if which == 0 else (8, 2)
        packed = packed.unflatten(-1, (nb,) + parts).transpose(-3, -2).flatten(-3)
        i = off % 16
        row_of = off - i + _scale_order(which, slots.device)[i]
        at_codes = off[:, None] * (nb * 16) + torch.arange(nb * 16, device=slots.device)
        at_scales = P * nb * 16 + row_of[:, None] * nb + torch.arange(nb, device=slots.device)
        flat[page[:, None, None], h[:, None], which, at_codes[:, None, :]] = packed
        flat[page[:, None, None], h[:, None], which, at_scales[:, None, :]] = scales
        back = flat[page[:, None, None], h[:, None], which, at_codes[:, None, :]]
        back = back.unflatten(-1, (parts[0], nb, parts[1])).transpose(-3, -2).flatten(-3)
        held = torch.stack([back & 15, back >> 4], -1).flatten(-2)
        scale = torch.exp2(flat[page[:, None, None], h[:, None], which, at_scales[:, None, :]].double() - 127.0).float()
        table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=slots.device)
        got.append((table[held.int()].unflatten(-1, (nb, 32)) * scale.unsqueeze(-1)).flatten(-2).bfloat16())
    return {"k": got[0], "v": got[1]}


def _attend(s, causal):
    """softmax(q k^T / sqrt d) v of each request's new tokens over its pages, in 32 bits."""
    q, cache, table, start, kv = s["q"], s["cache"], s["table"].long().clamp(min=0), s["start"].long(), s["kv"].long()
    T, Hq, d = q.shape
    H, P = cache.shape[1], cache.shape[3]
    n, L = s["max_new"], table.shape[1] * P
    pages = cache[table]  # [R, width, H, 2, P, row]
    k = _values_of(pages[:, :, :, 0], P, 0).transpose(1, 2).flatten(2, 3)  # [R, H, L, d]
    i = torch.arange(n, device=q.device)
    new = start[1:] - start[:-1]
    rows = (start[:-1, None] + i).clamp(max=T - 1)
    qr = q[rows].float().unflatten(2, (H, Hq // H)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [R, H, G n, d]
    score = torch.matmul(qr, k.transpose(-1, -2)) * d ** -0.5
    del k
    j = torch.arange(L, device=q.device)
    last = (kv[:, None] - new[:, None] + i if causal else kv[:, None].expand(-1, n)).minimum(kv[:, None] - 1)
    seen = (j <= last[:, :, None]).repeat(1, Hq // H, 1)[:, None]  # [R, 1, G n, L]
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    v = _values_of(pages[:, :, :, 1], P, 1).transpose(1, 2).flatten(2, 3)
    o = torch.matmul(score, v) / torch.where(total > 0, total, 1.0)
    o = o.unflatten(2, (Hq // H, n)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [R, n, Hq, d]
    return o[i < new[:, None]].to(q.dtype)  # the rows of each request after one another


def run(state):
    s = state
    if own:
        from mxfp4_microscaled_bit_quantize_b200 import api

        if s["op"] == "plan":
            start, kv, slots, info = api.mxattn_cache_plan(s["ctx"], s["new"], s["table"], s["free"], s["page"], s["tokens"])
            return {"table": s["table"], "start": start, "kv": kv, "slots": slots, "info": info}
        if s["op"] == "append":
            api.mxattn_cache_append(s["k"], s["v"], s["slots"], s["cache"], scale_mode=api.SCALE_UOS if s["uos"] else api.SCALE_OCP)
            k, v = api.mxattn_cache_read(s["cache"], s["slots"])
            return {"k": k, "v": v}
        return api.mxattn_paged_forward(s["q"], s["cache"], s["table"], s["start"], s["kv"], max_new=s["max_new"], max_kv=s["max_kv"], causal=s["op"] == "attend")
    if s["op"] == "plan":
        return _plan(s)
    if s["op"] == "append":
        return _append(s)
    return _attend(s, s["op"] == "attend")


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    if case["op"] == "append":
        # bf16 in, codes and scales out; the same back
        values = 2 * case["tokens"] * case["kv_heads"] * case["d"]
        return {"bytes": 2 * values * (2 + 17 / 32) + 2 * 8 * case["tokens"], "flops": 0}
    lens = _lengths(case)
    P, R, T = case["page"], len(lens), sum(n for _, n in lens)
    if case["op"] == "plan":
        taken = sum(-(-(c + n) // P) - -(-c // P) for c, n in lens)
        return {"bytes": 8 * R + 8 * R + 4 + 8 * T + 8 * taken + 16, "flops": 0}
    causal = case["op"] == "attend"
    Hq, H, d = case["heads"], case["kv_heads"], case["d"]
    keys = sum(c + n if causal else c for c, n in lens)
    pairs = sum(n * c + (n * (n + 1) // 2 if causal else 0) for c, n in lens)
    return {"bytes": 2 * 2 * T * Hq * d + keys * H * d * 17 / 16 + 4 * -(-keys // P) + 8 * R, "flops": 4 * Hq * d * pairs}


# ------------------------------------------------------------------ the definition in 64 bits


def _nearest(x, uos):
    """MXFP4 values of x [.., d], by search: the smallest allowed exponent, and the nearest magnitude of the even code."""
    b = x.double().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    some = torch.where(amax > 0, amax, 1.0)
    if uos:
        e = torch.ceil(torch.log2(some / 7.25))
        e = torch.where(some > 7.25 * torch.exp2(e), e + 1, e)
        e = torch.where(some <= 7.25 * torch.exp2(e - 1), e - 1, e)
    else:
        e = torch.floor(torch.log2(some))
        e = torch.where(torch.exp2(e) > some, e - 1, e)
        e = torch.where(torch.exp2(e + 1) <= some, e + 1, e) - 2
    unit = torch.exp2(e.clamp(-127, 127))
    y = (b.abs() / unit).clamp(max=6.0)
    best, far = torch.zeros_like(y), y.clone()
    for k in (2, 4, 6, 1, 3, 5, 7):  # even codes first: a tie stays with them
        here = (y - MAGNITUDES[k]).abs()
        best, far = torch.where(here < far, MAGNITUDES[k], best), torch.minimum(far, here)
    return (torch.copysign(best, b) * unit).flatten(-2)


def _plain_rows(cache, pages, head, which, count):
    """The first `count` rows of one head's K or V on these pages, from the bytes, in 64 bits."""
    P, row = cache.shape[3], cache.shape[4]
    nb = row // 17
    chunk = cache[pages, head, which].reshape(len(pages), P * row)
    t, c = torch.arange(P, device=cache.device), torch.arange(nb * 32, device=cache.device)
    b, e = c // 32, c % 32
    byte = (e // 8) * (4 * nb) + 4 * b + (e % 8) // 2 if which == 0 else (e // 4) * (2 * nb) + 2 * b + (e % 4) // 2
    i = t % 16
    place = (i % 8) * 2 + i // 8 if which == 0 else (i % 8) // 2 * 4 + i // 8 * 2 + i % 2
    raw = chunk[:, t[:, None] * (16 * nb) + byte].long()
    code = torch.where(e % 2 == 0, raw % 16, raw // 16)
    scale = chunk[:, 16 * nb * P + (t - i + place)[:, None] * nb + b].double()
    mag = code % 8
    value = torch.where(mag < 2, mag * 0.5, (1 + (mag % 2) * 0.5) * torch.exp2((mag // 2 - 1).double())) * torch.exp2(scale - 127)
    return torch.where(code >= 8, -value, value).reshape(len(pages) * P, nb * 32)[:count]


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "plan":  # whole numbers: written out one request after another
        P, ctx, new, free = s["page"], s["ctx"].tolist(), s["new"].tolist(), s["free"].tolist()
        table, start, slots, taken = s["table"].tolist(), [0], [], 0
        for r, (c, n) in enumerate(zip(ctx, new)):
            for j in range(-(-c // P), -(-(c + n) // P)):
                table[r][j] = free[taken]
                taken += 1
            slots += [table[r][p // P] * P + p % P for p in range(c, c + n)]
            start.append(start[-1] + n)
        return {"table": torch.tensor(table, dtype=torch.int32), "start": torch.tensor(start, dtype=torch.int32),
                "kv": torch.tensor([c + n for c, n in zip(ctx, new)], dtype=torch.int32), "slots": torch.tensor(slots), "info": torch.tensor([start[-1], taken, 0, 0], dtype=torch.int32)}
    if s["op"] == "append":
        return {"k": _nearest(s["k"], s["uos"]), "v": _nearest(s["v"], s["uos"])}
    q, cache, causal = s["q"], s["cache"], s["op"] == "attend"
    T, Hq, d = q.shape
    H, P = cache.shape[1], cache.shape[3]
    start, kv = s["start"].tolist(), s["kv"].tolist()
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device=q.device)
    for r, L in enumerate(kv):
        n = start[r + 1] - start[r]
        pages = s["table"][r, : -(-L // P)].long()
        for h in range(H) if L else ():
            k, v = (_plain_rows(cache, pages, h, which, L) for which in (0, 1))
            for hq in range(h * (Hq // H), (h + 1) * (Hq // H)):
                for a in range(0, n, 8192):
                    rows = slice(start[r] + a, start[r] + min(n, a + 8192))
                    x = q[rows, hq].double() @ k.T / math.sqrt(d)
                    if causal:
                        i = torch.arange(a, min(n, a + 8192), device=q.device)
                        x = x.masked_fill(torch.arange(L, device=q.device) > (L - n + i)[:, None], -math.inf)
                    out[rows, hq] = torch.softmax(x, -1) @ v
    return out
