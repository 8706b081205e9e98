"""The 4-bit key/value cache, attention over it, and the router's balance loss,
as cases to measure.

listed() / draw(rng) give cases, prepare(case, seed) the inputs a program has
in hand, run(state) one pass, work(case) what a pass cannot do without, and
exact(case, seed) the same outputs from the definitions in 64 bits.  With
own = False run() computes the plain form in elementary torch operations;
with own = True it makes the library's calls.

The cache: pages of page_size tokens; of each page and head the codes
[page_size, head_dim / 2] (two E2M1 codes a byte, the even element in the low
nibble) and the scale bytes [head_dim / 32, page_size] (one UE8M0 byte for 32
elements of a token), for keys and for values.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SIGNS = 0x9A3C61E5          # of the randomized Hadamard transform, a bit an element of 32


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _cache(tokens, heads, dim, dtype, rht, page, way="both"):
    return dict(op="cache", tokens=tokens, heads=heads, dim=dim, dtype=dtype, rht=rht, page=page, way=way)


def _attention(seqs, longest, heads, group, dim, page, dtype="bf16", rht=False, queries=1, window=0, sinks=False,
               lse=False, ragged=1):
    """seqs sequences of up to `longest` tokens in the cache (ragged: the seed
    of their lengths, 0: all of them that long), each with up to `queries`
    queries at its end."""
    return dict(op="attention", seqs=seqs, longest=longest, heads=heads, group=group, dim=dim, page=page, dtype=dtype,
                rht=rht, queries=queries, window=window, sinks=sinks, lse=lse, ragged=ragged)


def _balance(tokens, experts, k, dtype, score="softmax", accumulate=False, ld=0):
    return dict(op="balance", tokens=tokens, experts=experts, k=k, dtype=dtype, score=score, accumulate=accumulate,
                ld=ld or experts)


def listed():
    return [
        # the new tokens of eight requests that are being decoded: latency alone
        dict(_cache(8, 8, 64, "bf16", False, 16), name="cache few tokens"),
        # a long prompt's keys and values, spread by the Hadamard transform before they are rounded
        dict(_cache(16384, 8, 128, "bf16", True, 64), name="cache prompt"),
        # odd sizes in fp32, some tokens padding
        dict(_cache(1537, 5, 96, "f32", False, 32), name="cache odd"),
        # one request, a short context, sinks: latency again
        dict(_attention(1, 777, 8, 8, 64, 16, sinks=True, ragged=0), name="attention one request"),
        # a batch being decoded, every request with a length of its own
        dict(_attention(64, 16384, 8, 4, 128, 64, rht=True), name="attention batch"),
        # one very long context: few rows, the key axis has to be shared out
        dict(_attention(1, 262144, 8, 8, 128, 256, ragged=0), name="attention long context"),
        # layers that see the last 128 tokens only, with sinks
        dict(_attention(128, 8192, 8, 8, 64, 32, window=128, sinks=True), name="attention window"),
        # several drafted tokens a request, odd heads, fp32, with the log of the sum of exponentials
        dict(_attention(16, 4096, 5, 3, 96, 16, dtype="f32", queries=5, lse=True), name="attention drafts"),
        # a prompt of two requests behind what their caches hold
        dict(_attention(2, 8192, 8, 4, 128, 64, queries=4096), name="attention prompt"),
        # the expert layer's training step: 16384 tokens, 32 experts, top 4
        dict(_balance(16384, 32, 4, "bf16"), name="balance step"),
        # an odd batch, padded rows
        dict(_balance(1001, 60, 6, "f32", ld=64), name="balance odd"),
        # many experts, normalised sigmoid scores, added to the router's own gradient
        dict(_balance(65536, 256, 8, "f32", score="sigmoid", accumulate=True), name="balance many experts"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "attention", "attention", "attention", "balance"])
    if op == "balance":
        experts = rng.choice([8, 16, 24, 32, 60, 64, 96, 128, 160, 256])
        return _balance(_log(rng, 1, 65536), experts, rng.choice([1, 2, 3, 4, 6, 8]), rng.choice(["bf16", "f32"]),
                        rng.choice(["softmax", "sigmoid"]), rng.random() < 0.4, experts + rng.choice([0, 0, 3, 8]))
    heads, dim = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([32, 64, 64, 96, 128, 128, 192, 256])
    page, rht = rng.choice([16, 32, 64, 128, 256]), rng.random() < 0.5
    if op == "cache":
        return _cache(_log(rng, 1, 16384), min(heads, 1024 // dim), dim, rng.choice(["bf16", "bf16", "f32"]), rht,
                      page, rng.choice(["both", "both", "read"]))
    group, dtype = rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice(["bf16", "bf16", "bf16", "f32"])
    window, sinks = rng.choice([0, 0, 0, 100, 128, 1000]), rng.random() < 0.3
    kind = rng.choice(["decode", "decode", "drafts", "prompt"])
    if kind == "prompt":
        longest = _log(rng, 64, 4096)
        return _attention(rng.randint(1, 2), longest, heads, min(group, 32 // heads), min(dim, 128), page, dtype, rht,
                          rng.randint(17, longest), window, sinks, rng.random() < 0.3, rng.randint(1, 10 ** 6))
    seqs = _log(rng, 1, 128)
    longest = _log(rng, 16, min(65536, (1 << 29) // (seqs * heads * dim)))
    queries = 1 if kind == "decode" else rng.randint(2, 8)
    return _attention(seqs, longest, heads, group, dim, page, dtype, rht, queries, window, sinks, rng.random() < 0.3,
                      rng.choice([0, rng.randint(1, 10 ** 6)]))


def _lengths(case):
    """Tokens in the cache and queries of each sequence."""
    n, longest, queries = case["seqs"], case["longest"], case["queries"]
    if not case["ragged"]:
        return [longest] * n, [min(queries, longest)] * n
    r = random.Random(case["ragged"])
    lengths = [longest] + [r.randint(1, longest) for _ in range(n - 1)]
    return lengths, [min(v, queries if i == 0 else r.randint(1, queries)) for i, v in enumerate(lengths)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _new_cache(pages, heads, page, dim):
    """Codes and scales of keys, then of values."""
    shape_c, shape_s = (pages, heads, page, dim // 2), (pages, heads, dim // 32, page)
    return [torch.zeros(s, device="cuda", dtype=torch.uint8) for s in (shape_c, shape_s) * 2]


def _tokens(shape, gen):
    """Keys or values [tokens, heads, dim]: some channels are far larger than others."""
    channel = torch.exp(0.6 * torch.randn(shape[1:], device="cuda", generator=gen))
    return channel * torch.randn(shape, device="cuda", generator=gen)


def _fill(cache, case, gen):
    """A cache with tokens in every slot."""
    pages, heads, page, half = cache[0].shape
    step = max(1, (1 << 28) // (heads * page * half * 2))
    for codes, scales in (cache[:2], cache[2:]):
        for p in range(0, pages, step):
            n = min(step, pages - p)
            x = _tokens((n * page, heads, 2 * half), gen)
            c, s = _quantize(_hadamard(x) if case["rht"] else x)
            codes[p:p + n] = c.view(n, page, heads, half).transpose(1, 2)
            scales[p:p + n] = s.view(n, page, heads, half // 16).permute(0, 2, 3, 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "balance":
        t, e = case["tokens"], case["experts"]
        popular = -1.1 * torch.log(torch.arange(1, e + 1, device="cuda", dtype=torch.float32))
        wide = torch.zeros((t, case["ld"]), device="cuda", dtype=TYPES[case["dtype"]])
        wide[:, :e] = 1.5 * torch.randn((t, e), device="cuda", generator=gen) + 0.3 * popular
        logits, padding = wide[:, :e], t // 64      # (tokens at the end of the batch that go to no expert)
        ids = logits.float().topk(min(case["k"], e), dim=1).indices.to(torch.int32)
        logits[t - padding:], ids[t - padding:] = -math.inf, -1
        before = None
        if case["accumulate"]:                      # the router's own gradient
            before = (1e-7 * torch.randn((t, e), device="cuda", generator=gen)).to(logits.dtype)
        return dict(case=case, logits=logits, ids=ids, weight=0.01, dloss=torch.tensor(0.5, device="cuda"),
                    before=before)
    heads, dim, page = case["heads"], case["dim"], case["page"]
    if case["op"] == "cache":
        t = case["tokens"]
        pages = -(-t // page) + 3
        cache = _new_cache(pages, heads, page, dim)
        # whole pages in any order, the tokens in order within them; the last page is nobody's
        order = torch.randperm(pages - 1, device="cuda", generator=gen)
        at = torch.arange(t, device="cuda")
        slots = (order[at // page] * page + at % page).to(torch.int32)
        state = dict(case=case, cache=cache, slots=slots)
        if case["way"] == "read":
            _fill(cache, case, gen)
            return state
        # keys and values side by side, as one projection writes them
        both = torch.cat([_tokens((t, heads, dim), gen) for _ in range(2)], 1).to(TYPES[case["dtype"]])
        slots[t - t // 50:] = -1                    # padding at the batch's end
        return dict(state, k=both[:, :heads], v=both[:, heads:])
    lengths, queries = _lengths(case)
    used = [-(-n // page) for n in lengths]
    cache = _new_cache(sum(used) + 2, heads, page, dim)
    _fill(cache, case, gen)
    # pages in any order, as requests come and go
    order = torch.randperm(sum(used) + 2, device="cuda", generator=gen).to(torch.int32)
    starts = torch.tensor([sum(used[:i]) for i in range(len(used))], device="cuda")
    column = torch.arange(max(used), device="cuda")
    held = column < torch.tensor(used, device="cuda")[:, None]
    table = torch.where(held, order[(starts[:, None] + column).clamp(max=len(order) - 1)], -1).contiguous()
    rows, qheads = sum(queries), heads * case["group"]
    q = 1.2 * torch.randn((rows, qheads, dim), device="cuda", generator=gen) / 1.43     # scores of about 1.2
    offsets = None
    if case["queries"] > 1:
        offsets = torch.tensor([0] + [sum(queries[:i + 1]) for i in range(len(queries))], device="cuda",
                               dtype=torch.int32)
    sinks = torch.randn((qheads,), device="cuda", generator=gen) if case["sinks"] else None
    return dict(case=case, cache=cache, q=q.to(TYPES[case["dtype"]]), table=table, offsets=offsets, sinks=sinks,
                lengths=torch.tensor(lengths, device="cuda", dtype=torch.int32))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    if c["op"] == "cache":
        return _plain_cache(state, c)
    if c["op"] == "attention":
        return _plain_attention(state, c)
    return _plain_balance(state, c)


def _own(state, c):
    from mxfp4_precision_numerics_amd import mx
    if c["op"] == "balance":
        score = mx.SOFTMAX if c["score"] == "softmax" else mx.SIGMOID
        loss, counts, slope = mx.balance(state["logits"], state["ids"], score=score)
        dlogits = mx.balance_bwd(state["logits"], slope, score=score, dloss=state["dloss"], scale=state["weight"],
                                 add=state["before"])
        return {"loss": loss, "counts": counts, "dlogits": dlogits}
    if "handle" not in state:               # a program makes it once, with the cache
        state["handle"] = mx.KVCache(*state["cache"], use_rht=c["rht"], sign_mask=SIGNS if c["rht"] else 0)
    cache = state["handle"]
    if c["op"] == "cache":
        if c["way"] == "both":
            mx.cache_write(cache, state["k"], state["v"], state["slots"])
        k, v = mx.cache_read(cache, state["slots"], out_dtype=TYPES[c["dtype"]])
        return {"k": k, "v": v}
    out, lse = mx.cache_attention(cache, state["q"], state["table"], state["lengths"], q_offsets=state["offsets"],
                                  max_queries=c["queries"], window=c["window"], sinks=state["sinks"],
                                  need_lse=c["lse"])
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def _butterflies(x):
    """The 32-point Walsh-Hadamard transform of the last axis's blocks, stage by
    stage (1, 2, 4, 8, 16), times 2^-2.5."""
    y = x.reshape(-1, 1, 32)
    y = torch.stack((y[..., 0::2] + y[..., 1::2], y[..., 0::2] - y[..., 1::2]), -1)
    y = y.view(-1, 8, 2, 2)
    y = torch.stack((y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]), 2).view(-1, 4, 2, 4)
    y = torch.stack((y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]), 2).view(-1, 2, 2, 8)
    y = torch.stack((y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]), 2).view(-1, 2, 16)
    y = torch.stack((y[:, 0] + y[:, 1], y[:, 0] - y[:, 1]), 1)
    return (y * 2.0 ** -2.5).view(x.shape)


def _signs(x):
    bit = torch.arange(x.shape[-1], device="cuda") % 32
    return 1.0 - 2.0 * ((SIGNS >> bit) & 1).to(x.dtype)


def _hadamard(x):
    return _butterflies(x * _signs(x))


def _hadamard_back(y):
    return _butterflies(y) * _signs(y)


def _quantize(x):
    """Codes [..., n / 2] and scale bytes [..., n / 32] of x [..., n] in fp32."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    byte = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)
    v = torch.ldexp(b, (127 - byte)[..., None])
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    m = (torch.round(v.abs() / step) * step).clamp(max=6.0)         # (ties to the even multiple: the even code)
    code = torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(v).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], byte.to(torch.uint8)


def _decode(codes, scales):
    """Values in fp32 of codes [..., n / 2] and scale bytes [..., n / 32]."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    m = (n & 7).float()
    m = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2, 2 * m - 8))
    m = torch.where(n > 7, -m, m).unflatten(-1, (-1, 32))
    return torch.ldexp(m, scales.int()[..., None] - 127).flatten(-2)


def _plain_cache(state, c):
    slots, page, dt = state["slots"].long(), c["page"], TYPES[c["dtype"]]
    there = slots >= 0
    # (padding goes to the page that is nobody's)
    at = torch.where(there, slots, state["cache"][0].shape[0] * page - 1)
    p, o = at // page, at % page
    out = {}
    for name, (codes, scales) in {"k": state["cache"][:2], "v": state["cache"][2:]}.items():
        if c["way"] == "both":
            x = state[name].float()
            codes[p, :, o], scales[p, :, :, o] = _quantize(_hadamard(x) if c["rht"] else x)
        y = _decode(codes[p, :, o], scales[p, :, :, o])
        y = _hadamard_back(y) if c["rht"] else y
        out[name] = torch.where(there[:, None, None], y, 0.0).to(dt)
    return out


def _plain_attention(state, c):
    table, lengths, q = state["table"].long(), state["lengths"].long(), state["q"].float()
    s, h, g, d, n = c["seqs"], c["heads"], c["group"], c["dim"], c["queries"]
    at = table.clamp(min=0)
    keys, values = (_decode(codes[at], scales[at].transpose(-1, -2)).transpose(1, 2).reshape(s, h, -1, d)
                    for codes, scales in (state["cache"][:2], state["cache"][2:]))
    # queries padded to the longest
    off = torch.arange(s + 1, device="cuda") if state["offsets"] is None else state["offsets"].long()
    count = off[1:] - off[:-1]
    i = torch.arange(n, device="cuda")
    row = (off[:-1, None] + i).clamp(max=q.shape[0] - 1)
    x = (_hadamard(q) if c["rht"] else q)[row].view(s, n, h, g, d).permute(0, 2, 1, 3, 4).reshape(s, h, n * g, d)
    scores = (x @ keys.transpose(2, 3)) * d ** -0.5
    pos = (lengths - count)[:, None] + i
    key = torch.arange(keys.shape[2], device="cuda")
    seen = key <= pos[:, :, None]
    if c["window"]:
        seen &= key > pos[:, :, None] - c["window"]
    seen = seen[:, None, :, None].expand(s, 1, n, g, -1).reshape(s, 1, n * g, -1)
    scores = scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(3, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    if c["sinks"]:
        sink = state["sinks"].view(1, h, 1, g).expand(s, h, n, g).reshape(s, h, n * g, 1)
        top = torch.maximum(top, sink)
    p = scores.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    if c["sinks"]:
        total = total + (sink - top).exp()
    y = (p @ values) / total.clamp(min=1e-30)
    y = _hadamard_back(y) if c["rht"] else y
    # back to the rows there are
    r = torch.arange(q.shape[0], device="cuda")
    of = (r[:, None] >= off[None, 1:]).sum(1)
    y = y.view(s, h, n, g, d).permute(0, 2, 1, 3, 4).reshape(s, n, h * g, d)
    out = {"out": y[of, r - off[of]].to(state["q"].dtype)}
    if c["lse"]:
        lse = (top + total.log()).view(s, h, n, g).permute(0, 2, 1, 3).reshape(s, n, h * g)
        out["lse"] = lse[of, r - off[of]]
    return out


def _plain_balance(state, c):
    l, ids, e = state["logits"].float(), state["ids"].long(), c["experts"]
    used = (l > -math.inf).any(1)
    if c["score"] == "softmax":
        s = torch.exp(l - l.amax(1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
    else:
        s = 1 / (1 + torch.exp(-l))
    sig, total = s, s.sum(1, keepdim=True).clamp(min=1e-30)
    s = s / total
    counts = (ids[:, :, None] == torch.arange(e, device="cuda")).sum((0, 1)).to(torch.int32)
    slope = e * counts.float() / (counts.sum() * used.sum()).clamp(min=1).float()
    loss = (slope * s.double().sum(0).float()).sum()
    factor = state["weight"] * state["dloss"]
    dl = factor * s * (slope - (s * slope).sum(1, keepdim=True))
    dl = dl * (1 - sig) if c["score"] == "sigmoid" else dl
    if c["accumulate"]:
        dl = dl + state["before"].float()
    return {"loss": loss, "counts": counts, "dlogits": dl.to(state["logits"].dtype)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "balance":
        t, e, size = case["tokens"], case["experts"], SIZE[case["dtype"]]
        return {"bytes": t * e * size * (3 if case["accumulate"] else 2) + t * case["k"] * 4, "flops": 8 * t * e}
    h, d, size = case["heads"], case["dim"], SIZE[case["dtype"]]
    token = h * (d // 2 + d // 32) * 2          # codes and scales of a token's keys and values
    if case["op"] == "cache":
        t, both = case["tokens"], case["way"] == "both"
        return {"bytes": t * (token + 2 * h * d * size) * (2 if both else 1), "flops": 0}
    lengths, queries = _lengths(case)
    w = case["window"] or math.inf
    keys = sum(min(n, m + w - 1) for n, m in zip(lengths, queries))
    pairs = sum(min(n - m + i + 1, w) for n, m in zip(lengths, queries) for i in range(m))
    rows = sum(queries) * h * case["group"]
    return {"bytes": keys * token + rows * (2 * d * size + (4 if case["lse"] else 0)),
            "flops": 4 * d * h * case["group"] * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "balance":
            return _exact_balance(case, state)
        if case["op"] == "cache":
            return _exact_cache(case, state)
        return _exact_attention(case, state)


def _exact_matrix(case):
    """The transform of a head as a matrix: y = M x."""
    i = torch.arange(32, device="cuda")
    both = i[:, None] & i
    odd = sum((both >> b) & 1 for b in range(5)) % 2
    sign = torch.tensor([-1.0 if (SIGNS >> b) & 1 else 1.0 for b in range(32)], dtype=torch.float64, device="cuda")
    block = (1.0 - 2.0 * odd.double()) * sign / math.sqrt(32)
    return torch.block_diag(*[block] * (case["dim"] // 32))


def _exact_values(codes, scales):
    """Codes [..., n / 2] and scales [..., n / 32] as they are read."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device="cuda")
    low, high = grid[(codes % 16).int()], grid[torch.div(codes, 16, rounding_mode="floor").int()]
    v = torch.stack((low, high), -1).flatten(-2)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_rounded(x):
    """x [rows, n], each block of 32 as its nearest values on the grid."""
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    out = torch.empty_like(x)
    for b in range(0, x.shape[1], 32):
        y = x[:, b:b + 32]
        top = y.abs().amax(1, keepdim=True)
        unit = torch.exp2((torch.frexp(top).exponent - 3).clamp(min=-127).double())
        y = y / unit
        far = (y.abs().clamp(max=6.0)[:, :, None] - grid).abs()
        least = far.amin(2, keepdim=True)
        # of two that are as near the one with the even index
        rank = torch.where(far == least, torch.arange(8, device="cuda") % 2, 9)
        out[:, b:b + 32] = grid[rank.argmin(2)] * torch.sign(y) * unit
    return out


def _exact_cache(case, state):
    slots = state["slots"].tolist()
    there = torch.tensor([s >= 0 for s in slots], device="cuda")
    matrix = _exact_matrix(case) if case["rht"] else None
    out = {}
    for name, at in (("k", 0), ("v", 2)):
        if case["way"] == "read":
            p = torch.tensor([s // case["page"] for s in slots], device="cuda")
            o = torch.tensor([s % case["page"] for s in slots], device="cuda")
            y = _exact_values(state["cache"][at][p, :, o], state["cache"][at + 1][p, :, :, o])
        else:
            x = state[name].double()
            x = x @ matrix.t() if case["rht"] else x
            y = torch.cat([_exact_rounded(x[t:t + 512].reshape(-1, case["dim"])) for t in range(0, len(slots), 512)])
            y = y.view(x.shape)
        y = y @ matrix if case["rht"] else y
        out[name] = y * there[:, None, None]
    return out


def _exact_attention(case, state):
    lengths, queries = _lengths(case)
    page, group, matrix = case["page"], case["group"], _exact_matrix(case)
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(state["q"].shape[:2], dtype=torch.float64, device="cuda")
    first = 0
    for s, (length, n) in enumerate(zip(lengths, queries)):
        pages = state["table"][s, :-(-length // page)].long()
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")
        hidden = key > pos
        if case["window"]:
            hidden = hidden | (key <= pos - case["window"])
        low = max(0, length - n - case["window"] + 1) if case["window"] else 0      # none sees a key before it
        for h in range(case["heads"]):
            k, v = (_exact_values(state["cache"][a][pages, h].reshape(-1, case["dim"] // 2)[low:length],
                                  state["cache"][a + 1][pages, h].transpose(1, 2).reshape(-1, case["dim"] // 32)
                                  [low:length]) for a in (0, 2))
            for j in range(h * group, (h + 1) * group):
                q = state["q"][first:first + n, j].double()
                z = (q @ matrix.t() if case["rht"] else q) @ k.t() / math.sqrt(case["dim"])
                z = z.masked_fill(hidden[:, low:], -math.inf)
                if case["sinks"]:
                    z = torch.cat((z, state["sinks"][j].double().expand(n, 1)), 1)
                total = torch.logsumexp(z, 1)
                w = torch.exp(z - total[:, None])[:, :length - low]
                y = w @ v
                out[first:first + n, j] = y @ matrix if case["rht"] else y
                lse[first:first + n, j] = total
        first += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_balance(case, state):
    l, e = state["logits"].double(), case["experts"]
    live = ~torch.isneginf(l).all(1)
    sig = torch.softmax(l[live], 1) if case["score"] == "softmax" else torch.sigmoid(l[live])
    s = sig / sig.sum(1, keepdim=True)
    counts = torch.bincount(state["ids"].flatten().long() + 1, minlength=e + 1)[1:]
    made, used = int(counts.sum()), int(live.sum())
    slope = e * counts.double() / (made * used) if made * used else torch.zeros(e, dtype=torch.float64, device="cuda")
    loss = (s.mean(0) * counts * e / made).sum() if made * used else slope.sum()
    ds = state["weight"] * state["dloss"].double() * slope
    dl = torch.zeros_like(l)
    if case["score"] == "softmax":
        dl[live] = s * ds - s * (s * ds).sum(1, keepdim=True)
    else:       # through the sum, then through each sigmoid
        dsig = (ds - (ds * s).sum(1, keepdim=True)) / sig.sum(1, keepdim=True)
        dl[live] = dsig * sig * (1 - sig)
    if case["accumulate"]:
        dl += state["before"].double()
    return {"loss": loss, "counts": counts.to(torch.int32), "dlogits": dl}
