"""The operators around a shared prefix, as they are measured: rotation of the
position dims, appending tokens to the paged latent cache, expanding a shared
prefix into per-head keys and values, and attention over that prefix.

`run` computes each operator either in its plain form (elementary torch
operations in 32 bits, one rounding at the end) or, where `own` is true, by the
calls a user makes of mla_latent_kv_09_gb300.  `exact` gives the same results
from the definitions in 64 bits.
"""

import math

import torch

own = False

LATENT = 512     # latent dims of a cached token
ROPE = 64        # its position dims
NOPE = 128       # dims of a head without position, and of its values
PAGE = 64        # tokens in a page
FP8_ROW = 656    # bytes of an FP8 cache row: 512 codes, 4 scale bytes, 12 unused, 64 bf16
BASE = 10000.0   # base of the rotation's frequencies
EPS = 1e-6       # of the latent's norm


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the query's position dims of one decode step of 64 requests, 128 heads: a call bound by latency
        {"name": "rope-decode", "op": "rope", "tokens": 64, "heads": 128, "dim": 64, "offset": 0, "rope": 64,
         "half": False, "inverse": False, "yarn": False, "far": 8192},
        # the same dims for a step that checks 4 draft tokens of 333 requests, 64 index heads of 128 dims of which the first half turns, back again
        {"name": "rope-part", "op": "rope", "tokens": 1332, "heads": 64, "dim": 128, "offset": 0, "rope": 64,
         "half": True, "inverse": True, "yarn": False, "far": 65536},
        # a prefill chunk of 8192 tokens, whole 192-dim heads, positions of a context stretched to a million tokens
        {"name": "rope-prefill", "op": "rope", "tokens": 8192, "heads": 128, "dim": 192, "offset": 128, "rope": 64,
         "half": False, "inverse": False, "yarn": True, "far": 1 << 20},
        # the new tokens of one decode step of 64 requests
        {"name": "append-decode", "op": "append", "tokens": 64, "requests": 64, "fp8": False, "norm": True, "half": False},
        # a prefill chunk of 8192 tokens of 7 requests of uneven lengths
        {"name": "append-prefill", "op": "append", "tokens": 8192, "requests": 7, "fp8": False, "norm": True, "half": False},
        # a chunk into an FP8 cache
        {"name": "append-fp8", "op": "append", "tokens": 4099, "requests": 33, "fp8": True, "norm": True, "half": True},
        # a short system prompt on one shard of 16 heads, FP8 cache
        {"name": "expand-short", "op": "expand", "prefix": 1000, "heads": 16, "fp8": True},
        # a long shared document, all heads
        {"name": "expand-long", "op": "expand", "prefix": 8192, "heads": 128, "fp8": False},
        # one request alone on a short prefix: the smallest call
        {"name": "attend-one", "op": "attend", "tokens": 1, "prefix": 777, "heads": 128, "partial": False, "suffix": False, "spiked": False},
        # 64 requests, one token each, joined with what each attended to on its own
        {"name": "attend-decode", "op": "attend", "tokens": 64, "prefix": 8192, "heads": 128, "partial": False, "suffix": True, "spiked": False},
        # 128 requests with two tokens each, some of which share only a part of the prefix, peaked softmax
        {"name": "attend-mtp", "op": "attend", "tokens": 256, "prefix": 16384, "heads": 128, "partial": True, "suffix": True, "spiked": True},
        # a prefill chunk behind the prefix, one shard of 16 heads
        {"name": "attend-prefill", "op": "attend", "tokens": 2048, "prefix": 4096, "heads": 16, "partial": False, "suffix": True, "spiked": False},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "expand", "attend", "attend"])
    if op == "rope":
        dim, offset, rope = rng.choice([(64, 0, 64), (128, 0, 64), (128, 0, 128), (192, 128, 64), (128, 64, 32)])
        heads = rng.choice([1, 3, 16, 64, 128])
        return {"op": op, "tokens": _spread(rng, 1, 8192), "heads": heads, "dim": dim, "offset": offset, "rope": rope,
                "half": rng.random() < 0.5, "inverse": rng.random() < 0.3, "yarn": rng.random() < 0.5,
                "far": rng.choice([1, 4096, 131072, 1 << 20])}
    if op == "append":
        tokens = _spread(rng, 1, 8192)
        return {"op": op, "tokens": tokens, "requests": _spread(rng, 1, min(tokens, 256)), "fp8": rng.random() < 0.5,
                "norm": rng.random() < 0.8, "half": rng.random() < 0.5}
    heads = rng.choice([1, 5, 8, 16, 32, 64, 128])
    if op == "expand":
        return {"op": op, "prefix": _spread(rng, 1, 8192), "heads": heads, "fp8": rng.random() < 0.5}
    prefix = _spread(rng, 1, 16384)
    tokens = _spread(rng, 1, max(1, min(2048, 256 * 16384 * 128 // (prefix * heads))))
    return {"op": op, "tokens": tokens, "prefix": prefix, "heads": heads, "partial": rng.random() < 0.4,
            "suffix": rng.random() < 0.6, "spiked": rng.random() < 0.3}


# ------------------------------------------------------------------ inputs

def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _frequencies(rope, yarn):
    """Radians per position of each pair, in 64 bits, and the factor on the turned dims.  Stretched by
    YaRN from 4096 to 40 times that: pairs of few turns over the old length are slowed down, the others kept."""
    inv = BASE ** (-torch.arange(0, rope, 2, dtype=torch.float64) / rope)
    if not yarn:
        return inv.cuda(), 1.0
    factor, length = 40.0, 4096
    at = lambda turns: rope * math.log(length / (2 * math.pi * turns)) / (2 * math.log(BASE))  # noqa: E731
    low, high = max(0, math.floor(at(32.0))), min(rope - 1, math.ceil(at(1.0)))
    slow = ((torch.arange(rope // 2, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
    return (inv / factor * slow + inv * (1 - slow)).cuda(), 0.1 * math.log(factor) + 1.0


def _fp8_pool(pages, g):
    """FP8 rows of N(0, 1) values: codes, one power-of-two scale byte for 128 dims, position dims in bf16."""
    pool = torch.zeros((pages, PAGE, FP8_ROW), dtype=torch.uint8, device="cuda")
    shift = torch.randint(0, 3, (pages, PAGE, 4), generator=g, device="cuda")
    x = torch.randn((pages, PAGE, 4, 128), generator=g, device="cuda") * torch.exp2(6.0 - shift)[..., None]
    pool[..., :LATENT] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(2)
    pool[..., LATENT:LATENT + 4] = (121 + shift).to(torch.uint8)
    pool[..., 528:] = _normal((pages, PAGE, ROPE), g).view(torch.uint8)
    return pool


def _pool(pages, fp8, g):
    return _fp8_pool(pages, g) if fp8 else _normal((pages, PAGE, LATENT + ROPE), g)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    s = dict(case)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "rope":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        # heads of 64 dims are the last ones of a 192-dim projection and go to the last ones of the 576-dim query
        if D == 64:
            s["x"] = _normal((T, H, 192), g)[..., 128:]
            s["out"] = torch.zeros((T, H, 576), dtype=torch.bfloat16, device="cuda")[..., 512:]
        else:
            s["x"], s["out"] = _normal((T, H, D), g), torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"], s["factor"] = _frequencies(case["rope"], case["yarn"])
    elif case["op"] == "append":
        T, B = case["tokens"], case["requests"]
        # every request has some new tokens; they follow up to two pages of older ones
        cuts = (torch.randperm(T - 1, generator=g, device="cuda")[:B - 1] + 1).sort().values
        zero, end = cuts.new_zeros(1), cuts.new_full((1,), T)
        start = torch.cat([zero, cuts])
        count = torch.cat([cuts, end]) - start
        old = torch.randint(0, 2 * PAGE, (B,), generator=g, device="cuda")
        request = torch.repeat_interleave(torch.arange(B, device="cuda"), count)
        s["requests"] = request.to(torch.int32)
        s["positions"] = (torch.arange(T, device="cuda") - start[request] + old[request]).to(torch.int32)
        held = (old + count + PAGE - 1) // PAGE
        width, pages = int(held.max()), 3 * B + T // PAGE + 1  # some pages of the pool stay free
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        page = torch.randperm(pages, generator=g, device="cuda")[:int(held.sum())].to(torch.int32)
        table[torch.arange(width, device="cuda")[None] < held[:, None]] = page
        s["table"], s["cache"] = table, _pool(pages, case["fp8"], g)
        # a projection's output: the latent, then the dims that turn
        x = _normal((T, LATENT + ROPE), g)
        s["latent"], s["k_pe"] = x[:, :LATENT], x[:, LATENT:]
        s["weight"] = (1 + 0.1 * torch.randn(LATENT, generator=g, device="cuda")).to(torch.bfloat16) if case["norm"] else None
        s["inv_freq"], s["factor"] = _frequencies(ROPE, False)
    elif case["op"] == "expand":
        P, H = case["prefix"], case["heads"]
        pages = (P + PAGE - 1) // PAGE
        s["cache"] = _pool(pages + 3, case["fp8"], g)
        s["table"] = torch.randperm(pages + 3, generator=g, device="cuda")[:pages].to(torch.int32)
        s["w_uk"] = _normal((H, LATENT, NOPE), g) * LATENT ** -0.5
        s["w_uv"] = _normal((H, LATENT, NOPE), g) * LATENT ** -0.5
        s["k_nope"] = torch.zeros((H, P, NOPE), dtype=torch.bfloat16, device="cuda")
        s["k_pe"] = torch.zeros((P, ROPE), dtype=torch.bfloat16, device="cuda")
        s["v"] = torch.zeros((H, P, NOPE), dtype=torch.float16, device="cuda")
    else:
        T, P, H = case["tokens"], case["prefix"], case["heads"]
        q = _normal((T, H, NOPE + ROPE), g)
        s["q_nope"], s["q_pe"] = q[..., :NOPE], q[..., NOPE:]
        s["k_nope"], s["k_pe"] = _normal((H, P, NOPE), g), _normal((P, ROPE), g)
        if case["spiked"]:  # a few rows of large keys make the softmax peaked
            s["k_nope"] *= torch.where(torch.rand(P, generator=g, device="cuda") < 0.05, 8.0, 1.0)[None, :, None].to(torch.bfloat16)
        s["v"] = _normal((H, P, NOPE), g, torch.float16)
        s["visible"] = None
        if case["partial"]:  # a quarter of the tokens see a part of the prefix, a few see nothing
            cut = torch.randint(0, P + 1, (T,), generator=g, device="cuda")
            kind = torch.rand(T, generator=g, device="cuda")
            s["visible"] = torch.where(kind < 0.25, cut, torch.full_like(cut, P)).masked_fill(kind > 0.95, 0).to(torch.int32)
        s["suffix_out"] = _normal((T, H, NOPE), g) if case["suffix"] else None
        s["suffix_lse"] = math.log(P) + torch.randn((T, H), generator=g, device="cuda") if case["suffix"] else None
        s["scale"] = (NOPE + ROPE) ** -0.5
        s["out"] = torch.zeros((T, H, NOPE), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros((T, H), dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def _turned(x, cos, sin, half):
    """x [..., R] with pair i turned by the angle whose cosine and sine are given (they broadcast)."""
    R = x.shape[-1]
    a, b = (x[..., :R // 2], x[..., R // 2:]) if half else (x[..., 0::2], x[..., 1::2])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"]  # 64 bits: far positions
    if s["inverse"]:
        angle = -angle
    cos = (angle.cos() * s["factor"]).float()[:, None]
    sin = (angle.sin() * s["factor"]).float()[:, None]
    x, o, r = s["x"].float(), s["offset"], s["rope"]
    return torch.cat([x[..., :o], _turned(x[..., o:o + r], cos, sin, s["half"]), x[..., o + r:]], -1).to(torch.bfloat16)


def _plain_append(s):
    x = s["latent"].float()
    if s["weight"] is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    pe = _turned(s["k_pe"].float(), angle.cos().float(), angle.sin().float(), s["half"]).to(torch.bfloat16)
    at = s["positions"].long()
    page, row = s["table"][s["requests"].long(), at // PAGE].long(), at % PAGE
    cache = s["cache"]
    if not s["fp8"]:
        cache[page, row] = torch.cat([x.to(torch.bfloat16), pe], -1)
        return cache
    # the smallest power of two that brings a group of 128 dims within the largest code, 448
    group = x.view(-1, 4, 128)
    most = group.abs().amax(-1)
    m, e = torch.frexp(most)                  # most = m 2^e, m in [1/2, 1); 448 = (7/8) 2^9
    e = e - 9 + (m > 0.875)
    e = torch.where(most == 0, torch.zeros_like(e), e).clamp(-127, 127)
    codes = torch.ldexp(group, -e[..., None]).to(torch.float8_e4m3fn)
    new = torch.zeros((x.shape[0], FP8_ROW), dtype=torch.uint8, device=x.device)
    new[:, :LATENT] = codes.view(torch.uint8).flatten(1)
    new[:, LATENT:LATENT + 4] = (e + 127).to(torch.uint8)
    new[:, 528:] = pe.view(torch.uint8)
    cache[page, row] = new
    return _fp8_values(cache)


def _fp8_values(cache):
    """An FP8 cache as what its bytes stand for: codes, power-of-two scales, position dims."""
    return {"codes": cache[..., :LATENT].view(torch.float8_e4m3fn),
            "scales": cache[..., LATENT:LATENT + 4].view(torch.float8_e8m0fnu),
            "position": cache[..., 528:].view(torch.bfloat16)}


def _rows(cache, fp8, dtype):
    """Latent and position dims of every row of a pool."""
    if not fp8:
        return cache[..., :LATENT].to(dtype), cache[..., LATENT:]
    scale = torch.exp2(cache[..., LATENT:LATENT + 4].to(dtype) - 127.0)
    codes = cache[..., :LATENT].view(torch.float8_e4m3fn).to(dtype)
    return (codes.unflatten(-1, (4, 128)) * scale[..., None]).flatten(-2), cache[..., 528:].view(torch.bfloat16)


def _plain_expand(s):
    P = s["prefix"]
    rows, pe = _rows(s["cache"][s["table"].long()], s["fp8"], torch.float32)
    rows = rows.flatten(0, 1)[:P]
    return {"k_nope": torch.matmul(rows, s["w_uk"].float()).to(torch.bfloat16), "k_pe": pe.flatten(0, 1)[:P].contiguous(),
            "v": torch.matmul(rows, s["w_uv"].float()).to(torch.float16)}


def _plain_attend(s):
    qn, qp = s["q_nope"].float().transpose(0, 1), s["q_pe"].float().transpose(0, 1)
    x = torch.matmul(qn, s["k_nope"].float().transpose(1, 2))
    x += torch.matmul(qp, s["k_pe"].float().t())
    x *= s["scale"]
    if s["visible"] is not None:
        hidden = torch.arange(s["prefix"], device=x.device)[None] >= s["visible"][:, None]
        x.masked_fill_(hidden[None], -math.inf)
    most = x.amax(-1, keepdim=True)
    x -= torch.where(most == -math.inf, torch.zeros_like(most), most)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x, s["v"].float()) / total.clamp_min(1e-38)
    lse = (total.log() + most)[..., 0].t()
    out = out.transpose(0, 1)
    if s["suffix_out"] is not None:
        both = torch.logaddexp(lse, s["suffix_lse"])
        out = torch.exp(lse - both)[..., None] * out + torch.exp(s["suffix_lse"] - both)[..., None] * s["suffix_out"].float()
        lse = both
    return {"out": out.to(torch.bfloat16), "lse": lse}


def run(state):
    s = state
    if own:
        import mla_latent_kv_09_gb300 as m
        if s["op"] == "rope":
            return m.rope(s["x"], s["positions"], s["inv_freq"], offset=s["offset"], half=s["half"], inverse=s["inverse"],
                          scale=s["factor"], out=s["out"])
        if s["op"] == "append":
            m.cache_append(s["latent"], s["k_pe"], s["cache"], s["table"], s["positions"], request_ids=s["requests"],
                           norm_weight=s["weight"], eps=EPS, inv_freq=s["inv_freq"], half=s["half"], status=s["status"])
            return _fp8_values(s["cache"]) if s["fp8"] else s["cache"]
        if s["op"] == "expand":
            k_nope, k_pe, v = m.prefix_expand(s["cache"], s["table"], s["prefix"], s["w_uk"], s["w_uv"],
                                              out=(s["k_nope"], s["k_pe"], s["v"]), status=s["status"])
            return {"k_nope": k_nope, "k_pe": k_pe, "v": v}
        out, lse = m.prefix_attend(s["q_nope"], s["q_pe"], s["k_nope"], s["k_pe"], s["v"], s["scale"], visible=s["visible"],
                                   suffix_out=s["suffix_out"], suffix_lse=s["suffix_lse"], out=s["out"], lse=s["lse"],
                                   status=s["status"])
        return {"out": out, "lse": lse}
    return {"rope": _plain_rope, "append": _plain_append, "expand": _plain_expand, "attend": _plain_attend}[s["op"]](s)


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * case["dim"] + 4 * case["tokens"] + 4 * case["rope"], "flops": 3 * n * case["rope"]}
    if case["op"] == "append":
        T = case["tokens"]
        row = FP8_ROW - 12 if case["fp8"] else 2 * (LATENT + ROPE)
        return {"bytes": T * (2 * (LATENT + ROPE) + row + 8), "flops": T * (4 * LATENT + 3 * ROPE)}
    P, H = case["prefix"], case["heads"]
    if case["op"] == "expand":
        row = FP8_ROW - 12 if case["fp8"] else 2 * (LATENT + ROPE)
        return {"bytes": P * (row + 2 * ROPE) + 4 * H * LATENT * NOPE + 4 * P * H * NOPE, "flops": 4 * P * H * LATENT * NOPE}
    T = case["tokens"]
    # a quarter of the tokens of a partly shared prefix see half of it on average, one in twenty nothing
    seen = T * P * (1 - 0.25 / 2 - 0.05 if case["partial"] else 1)
    bytes_ = 4 * P * H * NOPE + 2 * P * ROPE + 2 * T * H * (NOPE + ROPE) + T * H * (2 * NOPE + 4) * (2 if case["suffix"] else 1)
    return {"bytes": bytes_, "flops": 2 * seen * H * (2 * NOPE + ROPE)}


# ------------------------------------------------------------------ definitions, in 64 bits

def _rotation(x, positions, inv, half, sign, factor):
    """Rows x [T, n, R] as complex numbers, each pair times factor * e^(i sign position inv)."""
    T, n, R = x.shape
    pair = x.double().view(T, n, 2, R // 2).transpose(2, 3) if half else x.double().view(T, n, R // 2, 2)
    z = torch.view_as_complex(pair.contiguous())
    turn = torch.polar(torch.full((T, R // 2), float(factor), dtype=torch.float64, device=x.device),
                       sign * positions.double()[:, None] * inv[None])
    y = torch.view_as_real(z * turn[:, None])
    return (y.transpose(2, 3) if half else y).reshape(T, n, R)


def _exact_append(s):
    x = s["latent"].double()
    if s["weight"] is not None:
        x = x / ((x * x).sum(1, keepdim=True) / LATENT + EPS).sqrt() * s["weight"].double()
    pe = _rotation(s["k_pe"].contiguous()[:, None], s["positions"], s["inv_freq"], s["half"], 1.0, 1.0)[:, 0]
    flat = (s["table"].long()[s["requests"].long(), (s["positions"] // PAGE).long()] * PAGE + s["positions"].long() % PAGE)
    pages = s["cache"].shape[0]
    if not s["fp8"]:
        cache = s["cache"].double().view(pages * PAGE, -1)
        cache[flat] = torch.cat([x, pe], 1)
        return cache.view(pages, PAGE, -1)
    was = _fp8_values(s["cache"])
    codes = was["codes"].to(torch.float64).reshape(pages * PAGE, 4, 128)
    scales = torch.exp2(s["cache"][..., LATENT:LATENT + 4].double() - 127).reshape(pages * PAGE, 4)
    place = was["position"].double().reshape(pages * PAGE, ROPE)
    group = x.view(-1, 4, 128)
    most = group.abs().amax(2)
    power = torch.ceil(torch.log2(torch.where(most > 0, most, torch.full_like(most, 448.0)) / 448.0)).clamp(-127, 127)
    codes[flat], scales[flat], place[flat] = group / torch.exp2(power)[..., None], torch.exp2(power), pe
    return {"codes": codes.view(pages, PAGE, LATENT), "scales": scales.view(pages, PAGE, 4), "position": place.view(pages, PAGE, ROPE)}


def _exact_attend(s):
    T, H, P = s["tokens"], s["heads"], s["prefix"]
    out = torch.empty((T, H, NOPE), dtype=torch.float64, device="cuda")
    lse = torch.empty((T, H), dtype=torch.float64, device="cuda")
    seen = torch.full((T,), P, device="cuda") if s["visible"] is None else s["visible"].long()
    for h in range(H):
        key = torch.cat([s["k_nope"][h], s["k_pe"]], 1).double()
        query = torch.cat([s["q_nope"][:, h], s["q_pe"][:, h]], 1).double()
        x = (query @ key.t()) * s["scale"]
        x = x.masked_fill(torch.arange(P, device="cuda")[None] >= seen[:, None], -math.inf)
        lse[:, h] = torch.logsumexp(x, 1)
        weight = torch.exp(x - lse[:, h, None]).nan_to_num(0.0)
        out[:, h] = weight @ s["v"][h].double()
    if s["suffix_out"] is not None:
        total = torch.stack([lse, s["suffix_lse"].double()]).logsumexp(0)
        share = torch.exp(lse - total)[..., None]
        out = share * out + (1 - share) * s["suffix_out"].double()
        lse = total
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        x, o, r = s["x"], s["offset"], s["rope"]
        y = x.double().clone()
        y[..., o:o + r] = _rotation(x[..., o:o + r].contiguous(), s["positions"], s["inv_freq"], s["half"],
                                    -1.0 if s["inverse"] else 1.0, s["factor"])
        return y
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "expand":
        rows, pe = _rows(s["cache"][s["table"].long()], s["fp8"], torch.float64)
        rows = rows.reshape(-1, LATENT)[:s["prefix"]]
        up = lambda w: torch.einsum("pc,hcd->hpd", rows, w.double())  # noqa: E731
        return {"k_nope": up(s["w_uk"]), "k_pe": pe.reshape(-1, ROPE)[:s["prefix"]].double(), "v": up(s["w_uv"])}
    return _exact_attend(s)
