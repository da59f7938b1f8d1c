"""The operators of a cache that prompts enter in chunks and that shrinks by what was attended to, as they are
measured: attention of a chunk of new tokens over the paged latent cache, the attention weight that each cached
row received, the choice of the rows to keep, and their move to pages of their own.

`run` computes each operator either in its plain form (elementary torch operations in 32 bits, one rounding at the
end) or, where `own` is true, by the calls a user makes of mla_latent_kv_09_gb300.  `exact` gives the same results
from the definitions in 64 bits.
"""

import math

import torch

own = False

HEADS = 128      # query heads of a token
LATENT = 512     # latent dims of a cached token, which are its value
ROPE = 64        # its position dims
ROW = LATENT + ROPE
INDEX = 128      # dims of an index key
PAGE = 64        # tokens in a page
FP8_ROW = 656    # bytes of an FP8 cache row: 512 codes, 4 scale bytes, 12 unused, 64 bf16
SCALE = 192 ** -0.5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one request checks a tree of 16 draft tokens on a short context: the smallest call
        {"name": "chunk-draft", "op": "chunk", "requests": 1, "tokens": 16, "longest": 777, "fp8": False, "causal": True, "spiked": False},
        # the next turns of 13 conversations, some tens of tokens each, uneven
        {"name": "chunk-turns", "op": "chunk", "requests": 13, "tokens": 611, "longest": 4096, "fp8": False, "causal": True, "spiked": True},
        # a chunk of 1024 tokens of one long prompt
        {"name": "chunk-prompt", "op": "chunk", "requests": 1, "tokens": 1024, "longest": 8192, "fp8": False, "causal": True, "spiked": False},
        # chunks of 7 prompts over an FP8 cache
        {"name": "chunk-fp8", "op": "chunk", "requests": 7, "tokens": 333, "longest": 8192, "fp8": True, "causal": True, "spiked": False},
        # what one decode step of 64 requests attended to, added to the weights so far
        {"name": "weights-step", "op": "weights", "requests": 64, "tokens": 64, "longest": 8192, "fp8": False, "decay": 1.0},
        # the last 32 tokens of a prompt as the window that says which of its rows matter
        {"name": "weights-window", "op": "weights", "requests": 1, "tokens": 32, "longest": 16384, "fp8": False, "decay": 0.0},
        # two tokens of each of 33 requests over an FP8 cache, older weights fading
        {"name": "weights-fp8", "op": "weights", "requests": 33, "tokens": 66, "longest": 4099, "fp8": True, "decay": 0.97},
        # 64 requests brought back to 4096 rows
        {"name": "select-step", "op": "select", "requests": 64, "longest": 8192, "keep": 4096, "sinks": 4, "recent": 256, "ties": False},
        # one request of 131072 rows brought back to a quarter, many of its weights equal
        {"name": "select-long", "op": "select", "requests": 1, "longest": 131072, "keep": 32768, "sinks": 4, "recent": 1024, "ties": True},
        # the latent rows that 64 requests keep
        {"name": "compact-step", "op": "compact", "requests": 64, "longest": 8192, "keep": 4096, "rows": "bf16"},
        # the FP8 rows of 5 long requests
        {"name": "compact-fp8", "op": "compact", "requests": 5, "longest": 65536, "keep": 16384, "rows": "fp8"},
        # the index keys of 9 requests
        {"name": "compact-index", "op": "compact", "requests": 9, "longest": 5000, "keep": 1111, "rows": "index"},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "weights", "weights", "select", "compact"])
    if op == "chunk":
        longest = _spread(rng, 1, 16384)
        tokens = _spread(rng, 1, min(1024, 1024 * 8192 // longest))
        return {"op": op, "requests": _spread(rng, 1, min(tokens, 64)), "tokens": tokens, "longest": longest,
                "fp8": rng.random() < 0.4, "causal": rng.random() < 0.8, "spiked": rng.random() < 0.3}
    if op == "weights":
        longest = _spread(rng, 1, 16384)
        requests = _spread(rng, 1, min(128, max(1, 48 * 8192 // longest)))
        tokens = requests * _spread(rng, 1, max(1, min(64, 2048 // requests, 64 * 8192 // (requests * longest))))
        return {"op": op, "requests": requests, "tokens": tokens, "longest": longest, "fp8": rng.random() < 0.4,
                "decay": rng.choice([0.0, 0.9, 1.0])}
    longest = _spread(rng, 1, 131072)
    requests = _spread(rng, 1, min(256, max(1, 48 * 8192 // longest)))
    keep = max(1, int(longest * rng.uniform(0.05, 0.9)))
    if op == "select":
        return {"op": op, "requests": requests, "longest": longest, "keep": keep, "sinks": min(keep, 4) if rng.random() < 0.7 else 0,
                "recent": (keep - min(keep, 4)) // rng.choice([2, 8, 32]), "ties": rng.random() < 0.4}
    return {"op": op, "requests": requests, "longest": longest, "keep": keep, "rows": rng.choice(["bf16", "fp8", "index"])}


def _lengths(case):
    """New tokens and cached rows (these tokens among them) of each request: uneven, and the same for every seed."""
    B, longest = case["requests"], case["longest"]
    part = [(b * 0.6180339887) % 1.0 for b in range(B)]
    N = case.get("tokens", 0)
    share = [0.2 + p for p in part]
    counts = [1 + int((N - B) * s / sum(share)) for s in share] if N else [0] * B
    if N:
        counts[0] += N - sum(counts)
    if case["op"] == "weights":  # a step has equally many tokens of every request
        counts = [N // B] * B
    lens = [max(1, n, round(longest * (1 - 0.75 * p))) for n, p in zip(counts, part)]
    return counts, lens


# ------------------------------------------------------------------ inputs

def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _fp8_pool(pages, g):
    """FP8 rows of N(0, 1) values: codes, one power-of-two scale byte for 128 dims, position dims in bf16."""
    pool = torch.zeros((pages, PAGE, FP8_ROW), dtype=torch.uint8, device="cuda")
    shift = torch.randint(0, 3, (pages, PAGE, 4), generator=g, device="cuda")
    x = torch.randn((pages, PAGE, 4, 128), generator=g, device="cuda") * torch.exp2(6.0 - shift)[..., None]
    pool[..., :LATENT] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(2)
    pool[..., LATENT:LATENT + 4] = (121 + shift).to(torch.uint8)
    pool[..., 528:] = _normal((pages, PAGE, ROPE), g).view(torch.uint8)
    return pool


def _paged(lens, g, spare=0):
    """A block table of shuffled pages for these lengths (-1 where a request has none), and, behind it in the same
    pool, the pages of a second one that holds `spare` rows of each request."""
    held = [(n + PAGE - 1) // PAGE for n in lens]
    kept = [(min(n, spare) + PAGE - 1) // PAGE for n in lens]
    order = torch.randperm(sum(held) + sum(kept) + 3, generator=g, device="cuda").to(torch.int32)  # some pages stay free
    tables, at = [], 0
    for counts in (held, kept):
        table = torch.full((len(lens), max(max(counts), 1)), -1, dtype=torch.int32, device="cuda")
        for b, n in enumerate(counts):
            table[b, :n] = order[at:at + n]
            at += n
        tables.append(table)
    return tables[0], tables[1], order.numel()


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    s = dict(case)
    counts, lens = _lengths(case)
    s["counts"], s["host_lens"], s["lens"] = counts, lens, _ints(lens)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    B, longest = case["requests"], max(lens)
    if case["op"] in ("chunk", "weights"):
        s["table"], _, pages = _paged(lens, g)
        s["cache"] = _fp8_pool(pages, g) if case["fp8"] else _normal((pages, PAGE, ROW), g)
        if case.get("spiked") and not case["fp8"]:  # a few rows of large dims make the softmax peaked
            s["cache"] *= torch.where(torch.rand((pages, PAGE, 1), generator=g, device="cuda") < 0.05, 6.0, 1.0).to(s["cache"].dtype)
        s["host_starts"] = _starts(counts)
        s["starts"] = _ints(s["host_starts"])
        s["q"] = _normal((sum(counts), HEADS, ROW), g)
        s["causal"] = case.get("causal", True)
    if case["op"] == "chunk":
        s["out"] = torch.zeros((sum(counts), HEADS, LATENT), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros((sum(counts), HEADS), dtype=torch.float32, device="cuda")
    elif case["op"] == "weights":
        # the softmax's logarithm of each (token, head), as the attention before this call returned it
        s["lse"] = torch.cat([torch.logsumexp(x, 2).t() for x in _scores(s, torch.float32)])
        s["weights"] = torch.rand((B, longest), generator=g, device="cuda") ** 8
        s["new"] = torch.zeros((B, longest), dtype=torch.float32, device="cuda")
    elif case["op"] == "select":
        # a few rows have most of the weight
        w = torch.exp(2.0 * torch.randn((B, longest), generator=g, device="cuda"))
        s["weights"] = torch.floor(w * 8) / 8 if case["ties"] else w
        s["kept"] = torch.zeros((B, case["keep"]), dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["new"] = torch.zeros((B, longest), dtype=torch.float32, device="cuda")
    else:
        keep, rows = case["keep"], case["rows"]
        s["table"], s["out_table"], pages = _paged(lens, g, keep)
        s["cache"] = (_fp8_pool(pages, g) if rows == "fp8" else _normal((pages, PAGE, INDEX if rows == "index" else ROW), g))
        # any increasing choice of each request's rows
        s["kept"] = torch.full((B, keep), -1, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            k = min(n, keep)
            s["kept"][b, :k] = torch.randperm(n, generator=g, device="cuda")[:k].sort().values.to(torch.int32)
        s["new_lens"] = _ints([min(n, keep) for n in lens])
    return s


# ------------------------------------------------------------------ one pass

def _rows(cache, dtype):
    """The 576 dims of cache rows [..., 576] bf16 or [..., 656] FP8."""
    if cache.dtype != torch.uint8:
        return cache.to(dtype)
    scale = torch.exp2(cache[..., LATENT:LATENT + 4].to(dtype) - 127.0)
    codes = cache[..., :LATENT].view(torch.float8_e4m3fn).to(dtype)
    latent = (codes.unflatten(-1, (4, 128)) * scale[..., None]).flatten(-2)
    return torch.cat([latent, cache[..., 528:].view(torch.bfloat16).to(dtype)], -1)


def _held(s, b, dtype):
    """Request b's cached rows in order."""
    n = s["host_lens"][b]
    return _rows(s["cache"][s["table"][b, :(n + PAGE - 1) // PAGE].long()], dtype).flatten(0, 1)[:n]


def _scores(s, dtype):
    """Each request's scores [heads, tokens, rows], -inf where a token does not see a row."""
    for b, (n, L) in enumerate(zip(s["counts"], s["host_lens"])):
        q = s["q"][s["host_starts"][b]:s["host_starts"][b] + n].to(dtype)
        x = torch.matmul(q.transpose(0, 1), _held(s, b, dtype).t())
        x *= SCALE
        if s["causal"]:
            seen = torch.arange(L - n + 1, L + 1, device=x.device)
            x.masked_fill_(torch.arange(L, device=x.device) >= seen[:, None], -math.inf)
        yield x


def _plain_chunk(s):
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    for b, x in enumerate(_scores(s, torch.float32)):
        part = slice(s["host_starts"][b], s["host_starts"][b + 1])
        most = x.amax(-1, keepdim=True)
        x -= torch.where(most == -math.inf, torch.zeros_like(most), most)
        x.exp_()
        total = x.sum(-1, keepdim=True)
        o = torch.matmul(x, _held(s, b, torch.float32)[:, :LATENT]) / total.clamp_min(1e-38)
        out[part] = o.transpose(0, 1).to(torch.bfloat16)
        lse[part] = (total.log() + most)[..., 0].t()
    return {"out": out, "lse": lse}


def _plain_weights(s):
    new = s["new"]
    for b, x in enumerate(_scores(s, torch.float32)):
        lse = s["lse"][s["host_starts"][b]:s["host_starts"][b + 1]].t()[..., None]
        x -= torch.where(lse == -math.inf, torch.full_like(lse, math.inf), lse)
        L = s["host_lens"][b]
        new[b, :L] = s["decay"] * s["weights"][b, :L] + x.exp_().sum((0, 1))
    return new


def _choice(weights, lens, keep, sinks, recent):
    """Which rows stay, [B, width]: the protected ones, then the heaviest, of equal ones the first."""
    B, width = weights.shape
    at = torch.arange(width, device=weights.device)[None]
    lens = lens[:, None]
    weights = torch.where(weights.isnan() | (at >= lens), torch.full_like(weights, -math.inf), weights)
    group = ((at < sinks) | (at >= lens - recent)).int() + (at < lens).int()  # 2: protected, 1: others, 0 and 1 beyond the end
    group = torch.where(at < lens, group, torch.zeros_like(group))
    order = weights.sort(dim=1, descending=True, stable=True).indices
    order = order.gather(1, group.gather(1, order).sort(dim=1, descending=True, stable=True).indices)
    stay = torch.zeros((B, width), dtype=torch.bool, device=weights.device)
    stay.scatter_(1, order, at < torch.minimum(lens, torch.full_like(lens, keep)))
    return stay


def _plain_select(s):
    keep, w = s["keep"], s["weights"]
    B, width = w.shape
    stay = _choice(w, s["lens"].long(), keep, s["sinks"], s["recent"])
    place = stay.long().cumsum(1) - 1
    where = torch.where(stay, place, torch.full_like(place, width))
    at = torch.arange(width, device=w.device).expand(B, width)
    kept = torch.full((B, width + 1), -1, dtype=torch.int64, device=w.device).scatter_(1, where, at)[:, :keep]
    new = torch.zeros((B, width + 1), dtype=torch.float32, device=w.device).scatter_(1, where, w)[:, :width].contiguous()
    return {"kept": kept.to(torch.int32), "lens": stay.sum(1).to(torch.int32), "weights": new}


def _values(cache):
    """A cache as what its bytes stand for."""
    if cache.dtype != torch.uint8:
        return cache
    return {"codes": cache[..., :LATENT].view(torch.float8_e4m3fn),
            "scales": cache[..., LATENT:LATENT + 4].view(torch.float8_e8m0fnu),
            "position": cache[..., 528:].view(torch.bfloat16)}


def _plain_compact(s):
    cache, kept = s["cache"], s["kept"].long()
    request, place = (kept >= 0).nonzero(as_tuple=True)
    row = kept[request, place]
    page = s["table"].long()[request, row // PAGE]
    cache[s["out_table"].long()[request, place // PAGE], place % PAGE] = cache[page, row % PAGE]
    return _values(cache)


def run(state):
    s = state
    if own:
        import mla_latent_kv_09_gb300 as m
        if s["op"] == "chunk":
            out, lse = m.chunk_attend(s["q"], s["cache"], s["table"], s["lens"], SCALE, token_starts=s["starts"],
                                      causal=s["causal"], out=s["out"], lse=s["lse"], status=s["status"])
            return {"out": out, "lse": lse}
        if s["op"] == "weights":
            return m.attention_weights(s["q"], s["lse"], s["cache"], s["table"], s["lens"], SCALE, s["weights"], causal=True,
                                       decay=s["decay"], out=s["new"], status=s["status"])
        if s["op"] == "select":
            kept, lens, new = m.evict_select(s["weights"], s["lens"], s["keep"], sinks=s["sinks"], recent=s["recent"],
                                             out=(s["kept"], s["new_lens"], s["new"]), status=s["status"])
            return {"kept": kept, "lens": lens, "weights": new}
        return _values(m.cache_compact(s["cache"], s["table"], s["kept"], s["new_lens"], s["out_table"], status=s["status"]))
    return {"chunk": _plain_chunk, "weights": _plain_weights, "select": _plain_select, "compact": _plain_compact}[s["op"]](s)


def work(case):
    counts, lens = _lengths(case)
    rows, B = sum(lens), case["requests"]
    if case["op"] in ("chunk", "weights"):
        pairs = 0  # (token, row it sees)
        for n, L in zip(counts, lens):
            first = L - n + 1 if case.get("causal", True) else L
            pairs += sum(max(0, min(L, first + i)) for i in range(n))
        row, N = FP8_ROW - 12 if case["fp8"] else 2 * ROW, sum(counts)
        if case["op"] == "chunk":
            return {"bytes": rows * row + N * HEADS * (2 * ROW + 2 * LATENT + 4), "flops": 2 * pairs * HEADS * (ROW + LATENT)}
        return {"bytes": rows * row + N * HEADS * (2 * ROW + 4) + rows * (8 if case["decay"] else 4),
                "flops": 2 * pairs * HEADS * ROW}
    kept = sum(min(n, case["keep"]) for n in lens)
    if case["op"] == "select":
        return {"bytes": 4 * rows + 4 * B * (case["keep"] + max(lens)), "flops": rows}
    row = {"bf16": 2 * ROW, "fp8": FP8_ROW - 12, "index": 2 * INDEX}[case["rows"]]
    return {"bytes": kept * (2 * row + 4), "flops": 0}


# ------------------------------------------------------------------ definitions, in 64 bits

def _exact_attention(s, weights):
    """Row by row of the definition, a token at a time: softmax over the rows that it sees."""
    N = s["q"].shape[0]
    out = torch.zeros((N, HEADS, LATENT), dtype=torch.float64, device="cuda")
    lse = torch.full((N, HEADS), -math.inf, dtype=torch.float64, device="cuda")
    total = s["weights"].double() * s["decay"] if weights else None
    t = 0
    for b, (n, L) in enumerate(zip(s["counts"], s["host_lens"])):
        place = torch.arange(L, device="cuda")
        row = s["cache"].flatten(0, 1)[s["table"][b].long()[place // PAGE] * PAGE + place % PAGE]
        if s["fp8"]:
            power = row[:, LATENT:LATENT + 4].double() - 127
            latent = row[:, :LATENT].view(torch.float8_e4m3fn).double() * torch.pow(2.0, power).repeat_interleave(128, 1)
            key = torch.cat((latent, row[:, 528:].contiguous().view(torch.bfloat16).double()), 1)
        else:
            key = row.double()
        for i in range(n):
            seen = max(0, L - n + 1 + i) if s["causal"] else L
            score = SCALE * (s["q"][t].double() @ key[:seen].t())
            if weights:
                total[b, :seen] += (score - s["lse"][t].double()[:, None]).exp().sum(0)
            elif seen:
                lse[t] = score.logsumexp(1)
                out[t] = score.softmax(1) @ key[:seen, :LATENT]
            t += 1
    if not weights:
        return {"out": out, "lse": lse}
    # behind a request's rows the new weights are as they were
    behind = torch.arange(total.shape[1], device="cuda")[None] >= s["lens"].long()[:, None]
    return torch.where(behind, s["new"].double(), total)


def exact(case, seed):
    if case["op"] in ("chunk", "weights"):
        if work(case)["flops"] > 8e12:  # 64 bits run at about 1 TFLOP/s
            return None
        return _exact_attention(prepare(case, seed), case["op"] == "weights")
    s = prepare(case, seed)
    if case["op"] == "select":
        keep, width = case["keep"], s["weights"].shape[1]
        kept = torch.full((case["requests"], keep), -1, dtype=torch.int64)
        new = torch.zeros((case["requests"], width), dtype=torch.float64)
        for b, (L, w) in enumerate(zip(s["host_lens"], s["weights"].double().cpu())):
            if L <= keep:
                stay = list(range(L))
            else:
                fixed = set(range(min(case["sinks"], L))) | set(range(max(0, L - case["recent"]), L))
                value = w[:L].tolist()
                rest = sorted((i for i in range(L) if i not in fixed), key=lambda i: (-value[i], i))
                stay = sorted(list(fixed) + rest[:keep - len(fixed)])
            kept[b, :len(stay)] = torch.tensor(stay)
            new[b, :len(stay)] = w[stay]
        return {"kept": kept.to(torch.int32), "lens": torch.tensor([min(L, keep) for L in s["host_lens"]], dtype=torch.int32),
                "weights": new}
    # the rows in their new places, whatever they hold
    cache = s["cache"]
    flat = cache.flatten(0, 1).clone()
    for b, L in enumerate(s["new_lens"].tolist()):
        place = torch.arange(L, device="cuda")
        kept = s["kept"][b, :L].long()
        old = s["table"][b].long()[kept // PAGE] * PAGE + kept % PAGE
        flat[s["out_table"][b].long()[place // PAGE] * PAGE + place % PAGE] = cache.flatten(0, 1)[old]
    moved = flat.view_as(cache)
    if case["rows"] != "fp8":
        return moved.double()
    v = _values(moved)
    return {"codes": v["codes"].double(), "scales": torch.exp2(moved[..., LATENT:LATENT + 4].double() - 127),
            "position": v["position"].double()}
