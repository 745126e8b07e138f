"""Cases that measure three operators of a serving step over a paged KV cache.

norm_rope        RMS norm of every query and key head, the position rotation and
                 the cache write in one pass
block_scatter    the cache write into 8-bit (E4M3) pages with one power-of-two
                 scale per (page, KV head)
block_attention  attention over such pages, for steps that mix decode tokens and
                 chunked-prefill chunks

`run` computes them from elementary torch operations, or, with `own` set, with
the calls of the paged-attention library.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
CODE_MAX = 448.0      # largest E4M3 magnitude
MIN_SCALE_EXP = -64   # smallest scale of a page: 2^-64


def listed():
    gqa = dict(heads=32, kv_heads=8, head_dim=128, dtype="bf16", block_size=16)
    return [
        # one token of one request: the latency of a single-stream decode
        dict(name="norm_rope one token", op="norm_rope", tokens=1, rotary_dim=128, neox=True, cache="16", **gqa),
        # a decode step of 256 requests
        dict(name="norm_rope decode 256", op="norm_rope", tokens=256, rotary_dim=128, neox=True, cache="16", **gqa),
        # a continuous-batching step: 16 chunks of 512 tokens and 240 decode tokens
        dict(name="norm_rope step of 8432", op="norm_rope", tokens=8432, rotary_dim=128, neox=True, cache="16", **gqa),
        # part of each head rotated, adjacent pairs, rows handed on without a cache write
        dict(name="norm_rope fp16 d96 partial", op="norm_rope", tokens=1001, heads=16, kv_heads=4, head_dim=96,
             dtype="fp16", block_size=16, rotary_dim=64, neox=False, cache="none"),
        # one new row per request, into pages that are part full
        dict(name="block_scatter decode 256", op="block_scatter", chunks=0, chunk=1, decodes=256, context=256, **gqa),
        # the rows of 16 chunks of 512 tokens and 240 decode tokens
        dict(name="block_scatter step of 8432", op="block_scatter", chunks=16, chunk=512, decodes=240, context=256,
             **gqa),
        # ragged chunks into short pages, one KV head per query head
        dict(name="block_scatter fp16 d64 ragged", op="block_scatter", chunks=3, chunk=333, decodes=29, context=100,
             heads=16, kv_heads=16, head_dim=64, dtype="fp16", block_size=8),
        # one request of a single-stream decode
        dict(name="block_attention one request", op="block_attention", chunks=0, chunk=1, decodes=1, context=700,
             spread="fixed", **gqa),
        # a decode step of 256 requests whose lengths are spread as in a serving mix
        dict(name="block_attention decode 256", op="block_attention", chunks=0, chunk=1, decodes=256, context=1024,
             spread="lognormal", **gqa),
        # long contexts, eight query heads per KV head
        dict(name="block_attention long 8", op="block_attention", chunks=0, chunk=1, decodes=8, context=32767,
             spread="fixed", heads=64, kv_heads=8, head_dim=128, dtype="bf16", block_size=16),
        # chunked prefill beside decode tokens
        dict(name="block_attention chunks 16x512", op="block_attention", chunks=16, chunk=512, decodes=48,
             context=2048, spread="uniform", **gqa),
        # short ragged chunks, small heads, short pages
        dict(name="block_attention fp16 d64 ragged", op="block_attention", chunks=7, chunk=131, decodes=21,
             context=1500, spread="uniform", heads=8, kv_heads=4, head_dim=64, dtype="fp16", block_size=8),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm_rope", "block_scatter", "block_attention"])
    group = rng.choice([1, 2, 4, 8])
    kv_heads = rng.choice([1, 2, 4, 8, 5])
    c = dict(op=op, heads=group * kv_heads, kv_heads=kv_heads, head_dim=rng.choice([64, 80, 96, 128, 256]),
             dtype=rng.choice(["bf16", "fp16"]), block_size=rng.choice([8, 16, 32]))
    if op == "norm_rope":
        c["tokens"] = _log_int(rng, 1, 4000)
        c["rotary_dim"] = 16 * rng.randint(1, c["head_dim"] // 16)
        c["neox"] = rng.random() < 0.5
        c["cache"] = rng.choice(["16", "fp8", "none"])
        return c
    c["chunks"] = rng.randint(0, 6)
    c["chunk"] = _log_int(rng, 2, 400) if c["chunks"] else 1
    c["decodes"] = _log_int(rng, 1, 60)
    if op == "block_scatter":
        c["context"] = _log_int(rng, 1, 300)
        return c
    c["context"] = _log_int(rng, 1, 2000)
    c["spread"] = rng.choice(["fixed", "uniform"] if c["chunks"] else ["fixed", "uniform", "lognormal"])
    return c


# ---- inputs ---------------------------------------------------------------

def _lengths(case):
    """Context and query length of every request: a function of the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["chunks"] + case["decodes"]
    spread, c = case.get("spread", "uniform"), case["context"]
    if spread == "fixed":
        ctx = [c] * n
    elif spread == "uniform":
        ctx = [rng.randint(0, c) for _ in range(n)]
    else:  # median c, clipped to [c / 64, 8 c]
        ctx = [min(8 * c, max(c // 64, round(c * math.exp(rng.gauss(0.0, 1.0))))) for _ in range(n)]
    query = [case["chunk"]] * case["chunks"] + [1] * case["decodes"]
    order = list(range(n))
    rng.shuffle(order)
    return [ctx[i] for i in order], [query[i] for i in order]


def _pages(ctx, query, bs, gen):
    """Block tables over a shuffled pool, and the lengths, on the GPU."""
    need = [(c + q + bs - 1) // bs for c, q in zip(ctx, query)]
    total, widest = sum(need), max(need) + 1
    pool = torch.randperm(total + 3, generator=gen)[:total].to(torch.int32)
    tables = torch.full((len(need), widest), -1, dtype=torch.int32)
    have = torch.arange(widest)[None, :] < torch.tensor(need)[:, None]
    tables[have] = pool
    starts = torch.tensor([0] + query).cumsum(0).to(torch.int32)
    lens = torch.tensor([c + q for c, q in zip(ctx, query)], dtype=torch.int32)
    return total + 3, tables.cuda(), lens.cuda(), starts.cuda()


def _codes(shape, gen):
    return (torch.randn(shape, device="cuda", generator=gen) * 64.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(
        torch.uint8)


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    H, Hkv, D, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    s = {"case": case, "scale": 1.0 / math.sqrt(D)}
    if case["op"] == "norm_rope":
        T, rot = case["tokens"], case["rotary_dim"]
        qkv = (randn(T, H + 2 * Hkv, D) * 2.0).to(dt)  # the output of a fused projection
        s["q"], s["key"], s["value"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        s["q_weight"], s["k_weight"] = (1.0 + 0.2 * randn(D)).to(dt), (1.0 + 0.2 * randn(D)).to(dt)
        max_position = 8192
        angle = torch.arange(max_position, dtype=torch.float64)[:, None] * 10000.0 ** (
            -2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)[None, :]
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        s["positions"] = torch.randint(0, max_position, (T,), generator=host).cuda()
        s["q_out"] = torch.empty((T, H, D), dtype=dt, device="cuda")
        if case["cache"] == "none":
            s["key_out"] = torch.empty((T, Hkv, D), dtype=dt, device="cuda")
            return s
        blocks = (T + bs - 1) // bs + 2
        slots = torch.randperm(blocks * bs, generator=host)[:T]
        if T > 4:
            slots[torch.randperm(T, generator=host)[:T // 50 + 1]] = -1  # padding tokens
        s["slots"] = slots.cuda()
        if case["cache"] == "16":
            s["key_cache"] = randn(blocks, bs, Hkv, D).to(dt)
            s["value_cache"] = randn(blocks, bs, Hkv, D).to(dt)
        else:
            s["key_cache"], s["value_cache"] = _codes((blocks, bs, Hkv, D), gen), _codes((blocks, bs, Hkv, D), gen)
            s["k_scale"], s["v_scale"] = 0.03, 0.02
        return s

    ctx, query = _lengths(case)
    blocks, s["tables"], s["lens"], s["starts"] = _pages(ctx, query, bs, host)
    s["max_query"], s["max_len"] = max(query), max(c + q for c, q in zip(ctx, query))
    T = sum(query)
    s["key_cache"], s["value_cache"] = _codes((blocks, bs, Hkv, D), gen), _codes((blocks, bs, Hkv, D), gen)
    for name, low, high in (("k_scales", -7, -5), ("v_scales", -8, -4)):  # values near 1 in magnitude
        s[name] = torch.exp2(torch.randint(low, high + 1, (blocks, Hkv), device="cuda", generator=gen).float())
    if case["op"] == "block_scatter":
        rows = randn(T, 2 * Hkv, D) * torch.exp(randn(T, 2 * Hkv, 1))  # magnitudes differ from token to token
        rows = rows.to(dt)
        s["key"], s["value"] = rows[:, :Hkv], rows[:, Hkv:]
    else:
        s["q"] = randn(T, H, D).to(dt)
        s["out"] = torch.empty((T, H, D), dtype=dt, device="cuda")
    return s


# ---- one pass -------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_norm_rope(s):
    from paged_kv_cache_55_gb300 import binding as B
    c = s["case"]
    if c["cache"] == "none":
        B.pa_norm_rope(s["q"], s["key"], s["q_weight"], s["k_weight"], EPS, s["positions"], s["table"], s["q_out"],
                       s["key_out"], is_neox=c["neox"])
        return s["q_out"], s["key_out"]
    if c["cache"] == "fp8":
        B.pa_norm_rope_reshape_and_cache_fp8(s["q"], s["key"], s["value"], s["q_weight"], s["k_weight"], EPS,
                                             s["key_cache"], s["value_cache"], s["slots"], s["positions"],
                                             s["table"], s["k_scale"], s["v_scale"], s["q_out"], is_neox=c["neox"])
        return s["q_out"], s["key_cache"].view(torch.float8_e4m3fn), s["value_cache"].view(torch.float8_e4m3fn)
    B.pa_norm_rope_reshape_and_cache(s["q"], s["key"], s["value"], s["q_weight"], s["k_weight"], EPS, s["key_cache"],
                                     s["value_cache"], s["slots"], s["positions"], s["table"], s["q_out"],
                                     is_neox=c["neox"])
    return s["q_out"], s["key_cache"], s["value_cache"]


def _own_block_scatter(s):
    from paged_kv_cache_55_gb300 import binding as B
    B.pa_reshape_and_cache_fp8_block(s["key"], s["value"], s["key_cache"], s["value_cache"], s["k_scales"],
                                     s["v_scales"], s["tables"], s["lens"], s["starts"], s["max_query"])
    return (s["key_cache"].view(torch.float8_e4m3fn), s["value_cache"].view(torch.float8_e4m3fn), s["k_scales"],
            s["v_scales"])


def _own_block_attention(s):
    from paged_kv_cache_55_gb300 import binding as B
    c = s["case"]
    if "workspace" not in s:  # a serving loop keeps one
        n = B.pa_attention_workspace_size(s["lens"].numel(), s["q"].shape[0], s["max_query"], s["max_len"],
                                          c["heads"], c["kv_heads"], c["head_dim"], c["block_size"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    B.pa_attention_varlen_fp8_block(s["q"], s["key_cache"], s["value_cache"], s["k_scales"], s["v_scales"],
                                    s["tables"], s["lens"], s["starts"], s["max_query"], s["max_len"], s["scale"],
                                    s["out"], s["workspace"])
    return s["out"]


_OWN = {"norm_rope": _own_norm_rope, "block_scatter": _own_block_scatter, "block_attention": _own_block_attention}


def _norm_rope_rows(x, weight, cos, sin, rot, neox):
    """Rows [T, heads, D] in 32 bits: norm over D, then rotation of the first `rot` elements."""
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if neox else (y[..., 0:rot:2], y[..., 1:rot:2])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([c, d], -1) if neox else torch.stack([c, d], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_norm_rope(s):
    c, dt = s["case"], s["q"].dtype
    rot = c["rotary_dim"]
    rows = s["table"][s["positions"]][:, None, :]
    cos, sin = rows[..., :rot // 2], rows[..., rot // 2:]
    q = _norm_rope_rows(s["q"], s["q_weight"], cos, sin, rot, c["neox"]).to(dt)
    k = _norm_rope_rows(s["key"], s["k_weight"], cos, sin, rot, c["neox"]).to(dt)
    if c["cache"] == "none":
        return q, k
    kept = s["slots"] >= 0
    slots = s["slots"][kept]
    k, v = k[kept], s["value"][kept]
    shape = s["key_cache"].shape
    if c["cache"] == "fp8":
        k = (k.float() / s["k_scale"]).clamp(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v.float() / s["v_scale"]).clamp(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    s["key_cache"].view(-1, *shape[2:])[slots] = k
    s["value_cache"].view(-1, *shape[2:])[slots] = v
    if c["cache"] == "fp8":
        return q, s["key_cache"].view(torch.float8_e4m3fn), s["value_cache"].view(torch.float8_e4m3fn)
    return q, s["key_cache"], s["value_cache"]


def _needed_scale(amax):
    """The smallest power of two (not below 2^MIN_SCALE_EXP) by which amax does not exceed the largest code."""
    fraction, exponent = torch.frexp(amax)  # amax = fraction * 2^exponent, 0.5 <= fraction < 1
    e = exponent - 9 + (fraction > 0.875).int()  # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_SCALE_EXP)).clamp(min=MIN_SCALE_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _plain_block_scatter(s):
    bs = s["case"]["block_size"]
    lens, starts, tables = s["lens"].long(), s["starts"].long(), s["tables"].long()
    query = starts[1:] - starts[:-1]
    context = lens - query
    first = context // bs  # the first page that gets a new row
    pages = torch.arange((s["max_query"] + bs - 2) // bs + 1, device="cuda")
    logical = first[:, None] + pages[None, :]  # [B, P]
    touched = (logical * bs < lens[:, None]) & (query > 0)[:, None]
    position = logical[..., None] * bs + torch.arange(bs, device="cuda")  # [B, P, bs]
    new = touched[..., None] & (position >= context[:, None, None]) & (position < lens[:, None, None])
    old = touched[..., None] & (position < context[:, None, None])
    token = (starts[:-1, None, None] + position - context[:, None, None]).clamp(0, int(s["key"].shape[0]) - 1)
    page = tables.gather(1, logical.clamp(max=tables.shape[1] - 1))[touched]  # [N]
    new, old, token = new[touched], old[touched], token[touched]  # [N, bs]
    fresh = ~old.any(1)
    for rows, cache, scales in ((s["key"], s["key_cache"], s["k_scales"]),
                                (s["value"], s["value_cache"], s["v_scales"])):
        x = rows[token].float()  # [N, bs, Hkv, D]
        magnitude = torch.where(new[:, :, None, None] & torch.isfinite(x), x.abs(), torch.zeros_like(x))
        before = torch.where(fresh[:, None], torch.zeros_like(scales[page]), scales[page])
        after = torch.maximum(before, _needed_scale(magnitude.amax((1, 3))))  # [N, Hkv]
        held = cache[page]
        wide = after[:, None, :, None]
        codes = (x / wide).clamp(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        kept = held.view(torch.float8_e4m3fn).float() * (before / after)[:, None, :, None]
        kept = kept.to(torch.float8_e4m3fn).view(torch.uint8)
        cache[page] = torch.where(new[:, :, None, None], codes, torch.where(old[:, :, None, None], kept, held))
        scales[page] = after
    return (s["key_cache"].view(torch.float8_e4m3fn), s["value_cache"].view(torch.float8_e4m3fn), s["k_scales"],
            s["v_scales"])


def _plain_block_attention(s):
    c = s["case"]
    H, Hkv, D, bs = c["heads"], c["kv_heads"], c["head_dim"], c["block_size"]
    G = H // Hkv
    lens, starts = s["lens"].long(), s["starts"].long()
    B, Q, L = lens.numel(), s["max_query"], s["max_len"]
    n = (L + bs - 1) // bs
    pages = s["tables"][:, :n].long().clamp(min=0)  # [B, n]
    real = torch.arange(n * bs, device="cuda")[None, :] < lens[:, None]  # [B, n bs]

    def values(cache, scales):  # [B, Hkv, n bs, D] in 32 bits; rows past the length are zero
        x = cache[pages].view(torch.float8_e4m3fn).float() * scales[pages][:, :, None, :, None]
        x = x.view(B, n * bs, Hkv, D)
        return torch.where(real[:, :, None, None], x, torch.zeros((), device="cuda")).transpose(1, 2)

    query = starts[1:] - starts[:-1]
    i = torch.arange(Q, device="cuda")
    row = (starts[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)  # [B, Q]
    q = s["q"][row].float().view(B, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    scores = torch.matmul(q, values(s["key_cache"], s["k_scales"]).transpose(2, 3)).mul_(s["scale"])
    seen = torch.arange(n * bs, device="cuda")[None, None, :] <= ((lens - query)[:, None] + i[None, :])[:, :, None]
    scores.view(B, Hkv, G, Q, n * bs).masked_fill_(~(seen & real[:, None, :])[:, None, None], -math.inf)
    scores = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    out = torch.matmul(scores, values(s["value_cache"], s["v_scales"])) / scores.sum(-1, keepdim=True)
    out = out.view(B, Hkv, G, Q, D).permute(0, 3, 1, 2, 4).reshape(B, Q, H, D)
    return out[i[None, :] < query[:, None]].to(s["q"].dtype)


_PLAIN = {"norm_rope": _plain_norm_rope, "block_scatter": _plain_block_scatter,
          "block_attention": _plain_block_attention}


# ---- what a pass cannot do without ----------------------------------------

def work(case):
    H, Hkv, D, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    if case["op"] == "norm_rope":
        T, rot = case["tokens"], case["rotary_dim"]
        rows = T * (H + Hkv)
        moved = 2 * 2 * T * H * D + 2 * T * Hkv * D + 4 * min(T, 8192) * rot + 8 * T + 4 * D
        if case["cache"] == "none":
            moved += 2 * T * Hkv * D
        else:
            moved += 2 * T * Hkv * D + 8 * T + 2 * T * Hkv * D * (2 if case["cache"] == "16" else 1)
        return {"bytes": moved, "flops": rows * (4 * D + 3 * rot)}
    ctx, query = _lengths(case)
    T, B = sum(query), len(query)
    if case["op"] == "block_scatter":
        touched = sum((c + q - 1) // bs - c // bs + 1 for c, q in zip(ctx, query))
        kept = sum(1 for c in ctx if c % bs)  # pages whose scale is read before it is written
        moved = 2 * T * Hkv * D * (2 + 1) + 2 * 4 * Hkv * (touched + kept) + 4 * touched + 4 * (2 * B + 1)
        return {"bytes": moved, "flops": 2 * T * Hkv * D * 2}
    keys = sum(c + q for c, q in zip(ctx, query))
    pages = sum((c + q + bs - 1) // bs for c, q in zip(ctx, query))
    pairs = sum(q * c + q * (q + 1) // 2 for c, q in zip(ctx, query))
    moved = 2 * keys * Hkv * D + 2 * 4 * pages * Hkv + 2 * 2 * T * H * D + 4 * pages + 4 * (2 * B + 1)
    return {"bytes": moved, "flops": 4 * pairs * H * D}


# ---- the definitions, in 64 bits ------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "block_scatter": _exact_block_scatter,
            "block_attention": _exact_block_attention}[case["op"]](case, s)


def _nearest_code(x):
    """The E4M3 value nearest to x, ties to the even fraction, in 64 bits."""
    x = x.double().clamp(-448.0, 448.0)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_norm_rope(case, s):
    D, rot, T = case["head_dim"], case["rotary_dim"], case["tokens"]
    table = s["table"].double()

    def rows(x, weight):
        x = x.double()
        y = x / ((x * x).sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
        z = y.clone()
        for t0 in range(0, T, 1024):
            part = slice(t0, min(T, t0 + 1024))
            turn = torch.complex(table[s["positions"][part], :rot // 2], table[s["positions"][part], rot // 2:])[:, None]
            if case["neox"]:
                w = torch.complex(y[part, :, :rot // 2], y[part, :, rot // 2:rot]) * turn
                z[part, :, :rot // 2], z[part, :, rot // 2:rot] = w.real, w.imag
            else:
                w = torch.complex(y[part, :, 0:rot:2], y[part, :, 1:rot:2]) * turn
                z[part, :, 0:rot:2], z[part, :, 1:rot:2] = w.real, w.imag
        return z

    q, k = rows(s["q"], s["q_weight"]), rows(s["key"], s["k_weight"])
    if case["cache"] == "none":
        return q, k
    if case["cache"] == "16":
        kc, vc, v = s["key_cache"].double(), s["value_cache"].double(), s["value"].double()
    else:
        kc = s["key_cache"].view(torch.float8_e4m3fn).double()
        vc = s["value_cache"].view(torch.float8_e4m3fn).double()
        k, v = _nearest_code(k / s["k_scale"]), _nearest_code(s["value"].double() / s["v_scale"])
    flat_k, flat_v = kc.flatten(0, 1), vc.flatten(0, 1)
    written = torch.nonzero(s["slots"] >= 0).flatten()
    flat_k.index_copy_(0, s["slots"][written], k[written])
    flat_v.index_copy_(0, s["slots"][written], v[written])
    return q, kc, vc


def _exact_block_scatter(case, s):
    bs, Hkv = case["block_size"], case["kv_heads"]
    lens, starts, tables = s["lens"].tolist(), s["starts"].tolist(), s["tables"].tolist()
    got = []
    for rows, cache, scales in ((s["key"], s["key_cache"], s["k_scales"]),
                                (s["value"], s["value_cache"], s["v_scales"])):
        rows = rows.double()
        held = cache.view(torch.float8_e4m3fn).double()
        power = scales.double()
        peak = rows.abs().amax(-1).cpu()  # [T, Hkv]
        was = scales.double().cpu()
        for b, (length, t0, t1) in enumerate(zip(lens, starts, starts[1:])):
            context = length - (t1 - t0)
            for page in range(context // bs, (length - 1) // bs + 1):
                low, high = max(context, page * bs), min(length, (page + 1) * bs)
                where, t = tables[b][page], t0 + low - context
                amax = peak[t:t + high - low].amax(0)
                scale = []
                for h in range(Hkv):
                    a, e = float(amax[h]), MIN_SCALE_EXP
                    if a > 0:
                        e = max(e, math.frexp(a)[1] - 10)
                        while a > 448.0 * 2.0 ** e:
                            e += 1
                    before = float(was[where, h]) if low > page * bs else 0.0
                    scale.append(max(2.0 ** e, before))
                wide = torch.tensor(scale, dtype=torch.float64, device="cuda")[:, None]
                if low > page * bs:
                    kept = held[where, :low - page * bs]
                    held[where, :low - page * bs] = _nearest_code(kept * power[where][:, None] / wide)
                held[where, low - page * bs:high - page * bs] = _nearest_code(rows[t:t + high - low] / wide)
                power[where] = wide[:, 0]
        got.append((held, power))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def _exact_block_attention(case, s):
    H, Hkv, D, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    G = H // Hkv
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (length, t0, t1) in enumerate(zip(lens, starts, starts[1:])):
        pages = s["tables"][b, :(length + bs - 1) // bs].long()

        def rows(cache, scales):
            x = cache[pages].view(torch.float8_e4m3fn).double() * scales[pages].double()[:, None, :, None]
            return x.flatten(0, 1)[:length]

        k, v = rows(s["key_cache"], s["k_scales"]), rows(s["value_cache"], s["v_scales"])
        q = s["q"][t0:t1].double()
        last = length - (t1 - t0) + torch.arange(t1 - t0, device="cuda")
        hidden = torch.arange(length, device="cuda")[None, :] > last[:, None]
        for h in range(Hkv):
            heads = q[:, h * G:(h + 1) * G]
            logits = torch.einsum("tgd,kd->tgk", heads, k[:, h]) / math.sqrt(D)
            p = torch.softmax(logits.masked_fill(hidden[:, None, :], -math.inf), -1)
            out[t0:t1, h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", p, v[:, h])
    return out
