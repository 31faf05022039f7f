"""Operators on the paged K/V cache: what is measured, and their plain forms.

`kv_matmul_paged` fills a paged cache of keys and values; these operators go with it:

  rope       `kv_rope_paged`: new queries and keys turned by their positions, one position for
             every axis (time, height, width) and an axis for every pair of columns; keys and
             values stored in the paged cache
  attention  `kv_attention_paged`: new tokens of every request (a chunk, or one token) over the
             request's cached keys and values and the new ones up to their own, heads in groups
             that share keys
  window     `kv_window_attention_paged`: the same over the last `window` positions and the
             first `sinks` positions of the request alone

A case holds sizes only; request lengths follow from its `shape` number and the values from the
seed that `prepare` is given.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def _attention(batch, heads, kv_heads, size, ctx, new, page, window=0, sinks=0, shape=1):
    """`new` tokens a request over `ctx` cached ones; a window of 0 is none."""
    return {"kind": "window" if window else "attention", "batch": batch, "heads": heads,
            "kv_heads": kv_heads, "size": size, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "new_lo": new[0], "new_hi": new[1], "page": page, "window": window, "sinks": sinks,
            "shape": shape}


def _rope(batch, heads, kv_heads, size, rope, axes, woven, half, ctx, new, page, shape=1):
    """`woven`: the axes take turns over the pairs of columns, else each has a run of them."""
    return {"kind": "rope", "batch": batch, "heads": heads, "kv_heads": kv_heads, "size": size,
            "rope": rope, "axes": axes, "woven": woven, "half": half, "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "new_lo": new[0], "new_hi": new[1], "page": page, "shape": shape}


def listed():
    return [
        # one user, one token, a short history: latency alone
        dict(_attention(1, 32, 8, 128, (500, 500), (1, 1), 64, shape=11), name="token_one_user"),
        # a full decode batch, one token each
        dict(_attention(64, 32, 8, 128, (512, 4096), (1, 1), 128, shape=12), name="token_batch"),
        # few users with long histories: the key axis has to be split
        dict(_attention(4, 32, 8, 128, (65536, 65536), (1, 1), 64, shape=13), name="token_long"),
        # prompts of many lengths, nothing cached
        dict(_attention(6, 32, 8, 128, (0, 0), (1, 4096), 128, shape=81), name="prompts"),
        # a chunk of a long prompt, most of which is cached
        dict(_attention(1, 32, 8, 128, (16384, 16384), (2048, 2048), 128, shape=15), name="chunk_long"),
        # a mixed step: single tokens and odd chunks, an odd group of heads, small pages
        dict(_attention(33, 20, 4, 64, (0, 3000), (1, 97), 16, shape=16), name="mixed_small_pages"),
        # a decode batch of a layer with a window: the history's middle is not read
        dict(_attention(64, 64, 8, 64, (8192, 32768), (1, 1), 64, 1024, 4, shape=17), name="window_tokens"),
        # a chunk in such a layer
        dict(_attention(2, 64, 8, 64, (5000, 12000), (2048, 4096), 128, 1024, 4, shape=18), name="window_chunk"),
        # one image's worth of odd rows for one user: three axes, a run of pairs each
        dict(_rope(1, 32, 8, 128, 128, 3, False, True, (77, 77), (37, 37), 64, shape=21), name="rope_image"),
        # prompts of several users: three axes that take turns
        dict(_rope(8, 32, 8, 128, 128, 3, True, True, (0, 4096), (256, 1024), 128, shape=22), name="rope_prompts"),
        # a decode batch of text, one axis, part of the columns, interleaved layout
        dict(_rope(64, 32, 8, 128, 64, 1, False, False, (512, 4096), (1, 1), 16, shape=23), name="rope_tokens"),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw_one(rng):
    shape = rng.randrange(1 << 30)
    kind = rng.choice(["attention", "attention", "window", "rope"])
    page = rng.choice([8, 12, 16, 24, 32, 64, 96, 128, 256])
    heads, kv_heads = rng.choice([(32, 8), (32, 8), (64, 8), (32, 32), (8, 1), (20, 4), (6, 2),
                                  (28, 4), (71, 1), (12, 3)])
    size = rng.choice([64, 128, 128])
    batch = _log_int(rng, 1, 64)
    ctx = _log_int(rng, 1, 65536 if kind != "rope" else 4096)
    ctx = (rng.randint(0, ctx), ctx)
    if kind == "rope":
        new = _log_int(rng, 1, 1024)
        axes = rng.choice([1, 3, 3, 2])
        rope = rng.choice([size, size, size // 2])
        return _rope(batch, heads, kv_heads, size, rope, axes, axes > 1 and rng.random() < 0.5,
                     rng.random() < 0.5, ctx, (rng.randint(1, new), new), page, shape)
    new = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4096)
    window, sinks = (_log_int(rng, 1, 4096), rng.choice([0, 1, 4, 130])) if kind == "window" else (0, 0)
    return _attention(batch, heads, kv_heads, size, ctx, (rng.randint(1, new), new), page, window,
                      sinks, shape)


def _padded(case):
    """Values of the largest tensor that the plain form holds at once."""
    if case["kind"] == "rope":
        return 0
    return max(n * (c + n) for c, n in zip(*_lengths(case))) * case["heads"]


def _in_all(case):
    """Scores that the plain form computes, masked ones among them."""
    if case["kind"] == "rope":
        return 0
    return sum(n * (c + n) for c, n in zip(*_lengths(case))) * case["heads"] * case["size"]


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["kind"] == "rope", {"bytes": 0, "flops": 0, "padded": 0, "all": 0})
        now = {"bytes": w["bytes"], "flops": w["flops"], "padded": _padded(c), "all": _in_all(c)}
        for k in m:
            m[k] = max(m[k], now[k])
    while True:
        c = _draw_one(rng)
        w, m = work(c), most[c["kind"] == "rope"]
        if w["bytes"] <= m["bytes"] and w["flops"] <= m["flops"] and _padded(c) <= m["padded"] \
                and _in_all(c) <= m["all"]:
            return c


# ---------------------------------------------------------------------------------------
# shapes that follow from a case
# ---------------------------------------------------------------------------------------

def _lengths(case):
    """Cached tokens and new tokens of every request."""
    rng = random.Random(case["shape"])
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    return ctx, new


def _pair_axes(case):
    """The axis of every pair of columns: by turns, or runs of which the first axis's is the
    shortest."""
    pairs, axes = case["rope"] // 2, case["axes"]
    if case["woven"]:
        return [j % axes for j in range(pairs)]
    first = pairs // 4 if axes > 1 else pairs
    rest = -(-(pairs - first) // max(axes - 1, 1))
    return [0] * first + [1 + j // rest for j in range(pairs - first)]


def _seen(case, p):
    """Positions that a token at position p attends."""
    if not case["window"]:
        return p + 1
    return min(p + 1, case["window"]) + min(case["sinks"], max(p + 1 - case["window"], 0))


def _pairs(case, c, n):
    """Sum of _seen over the positions c .. c + n - 1, and the positions that any of them
    attends."""
    if not case["window"]:
        return n * c + n * (n + 1) // 2, c + n
    pairs = sum(_seen(case, p) for p in range(c, c + n))
    first = max(c + 1 - case["window"], 0)
    return pairs, c + n - first + min(case["sinks"], first)


def work(case):
    ctx, new = _lengths(case)
    rows, h, kv, d = sum(new), case["heads"], case["kv_heads"], case["size"]
    if case["kind"] == "rope":
        # queries, keys and values in and out; positions, and the factors of the pairs
        return {"bytes": rows * (4 * d * (h + 2 * kv) + 4 * case["axes"] + 4 * case["rope"]),
                "flops": 3 * rows * (h + kv) * case["rope"]}
    both = [_pairs(case, c, n) for c, n in zip(ctx, new)]
    return {"bytes": sum(k for _, k in both) * kv * d * 4 + rows * h * (4 * d + 4),
            "flops": 4 * d * h * sum(p for p, _ in both)}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _normal(g, *size):
    return torch.randn(size, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _paging(case, g, ctx, new):
    """A shuffled page table and its page count: pages for every cached and new token."""
    need = [(c + n + case["page"] - 1) // case["page"] for c, n in zip(ctx, new)]
    order = torch.randperm(sum(need) + 1, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda")
    column = torch.arange(max(need), device="cuda")
    inside = column[None] < torch.tensor(need, device="cuda")[:, None]
    table = order[(at[:, None] + column[None]).clamp(max=sum(need) - 1)]
    return torch.where(inside, table, torch.zeros_like(table)).contiguous(), sum(need) + 1


def _freqs(positions, rope, base=1000000.0):
    """(cos, sin) pairs [positions, rope]."""
    pairs = torch.arange(rope // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * base ** (-2 * pairs / rope)
    return torch.stack([angle.cos(), angle.sin()], -1).reshape(positions, rope).float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ctx, new = _lengths(case)
    h, kv, d = case["heads"], case["kv_heads"], case["size"]
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    rows = offsets[-1]
    table, pages = _paging(case, g, ctx, new)
    # keys and values of a page side by side: [layers, pages, planes, slots, columns]
    cache = _normal(g, 1, pages, 2, case["page"], kv * d)
    s = {"case": case, "ctx": ctx, "new": new, "first": offsets, "table": table, "cache": cache,
         "lengths": _int32(ctx), "offsets": _int32(offsets)}
    if case["kind"] == "rope":
        # out of one projection: a row's queries, keys and values side by side
        x = _normal(g, rows, (h + 2 * kv) * d)
        q, k, v = x.split([h * d, kv * d, kv * d], 1)
        s.update(q=q.unflatten(1, (h, d)), k=k.unflatten(1, (kv, d)), v=v.unflatten(1, (kv, d)),
                 turned=torch.empty(rows, h, d, dtype=torch.bfloat16, device="cuda"),
                 axes=_pair_axes(case), freqs=_freqs(max(c + n for c, n in zip(ctx, new)), case["rope"]))
        # the first axis counts the tokens, the others lie on a grid behind a common start
        at = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)]).cuda()
        grid = torch.stack([at - torch.randint(0, 1 + int(at.min()) // 2, (rows,), generator=g, device="cuda")
                            for _ in range(case["axes"] - 1)]) if case["axes"] > 1 else at[:0].view(0, rows)
        s["positions"] = torch.cat([at[None], grid]).to(torch.int32).contiguous()
        return s
    s.update(q=_normal(g, rows, h, d), scale=1.0 / math.sqrt(d),
             out=torch.empty(rows, h, d, dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty(rows, h, dtype=torch.float32, device="cuda"))
    return s


# ---------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------

def _handle(s):
    """What a user's program keeps beside its tensors: the cache descriptor, the workspace."""
    import paged_kv_mla_gb300 as pkm
    case, cache = s["case"], s["cache"]
    s["handle"] = pkm.PagedCache(
        data=cache, page_table=s["table"], layer_stride=cache.stride(0), page_stride=cache.stride(1),
        kv_stride=cache.stride(2), slot_stride=cache.stride(3), num_layers=cache.shape[0],
        num_pages=cache.shape[1], page_size=cache.shape[3], row_elems=cache.shape[4],
        cache_lengths=s["lengths"])
    if case["kind"] != "rope":
        s["workspace"] = torch.empty(pkm.kv_attention_paged_workspace_size(
            s["q"].shape[0], case["heads"], case["kv_heads"], case["size"]), dtype=torch.uint8, device="cuda")
    return s["handle"]


def _own(s):
    import paged_kv_mla_gb300 as pkm
    case = s["case"]
    cache = s.get("handle") or _handle(s)
    if case["kind"] == "rope":
        pkm.kv_rope_paged(s["offsets"], s["positions"], s["freqs"], cache, 0, case["kv_heads"],
                          q=s["q"], q_out=s["turned"], k=s["k"], v=s["v"], pair_axes=s["axes"],
                          half=case["half"])
        return [s["turned"], s["cache"]]
    if case["kind"] == "window":
        pkm.kv_window_attention_paged(s["q"], s["offsets"], s["scale"], case["window"], case["sinks"],
                                      cache, 0, s["out"], s["workspace"], lse=s["lse"])
    else:
        pkm.kv_attention_paged(s["q"], s["offsets"], s["scale"], cache, 0, s["out"], s["workspace"],
                               lse=s["lse"])
    return [s["out"], s["lse"]]


# ---------------------------------------------------------------------------------------
# plain forms: elementary torch operations in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------------------

def _rotate(x, c, sn, half):
    """The first 2 * pairs columns of x [..., D] turned by c, sn [..., pairs], in 32 bits; the
    others as they are."""
    p = c.shape[-1]
    x, rest = x.float().split([2 * p, x.shape[-1] - 2 * p], -1)
    a, b = (x[..., :p], x[..., p:]) if half else (x[..., 0::2], x[..., 1::2])
    u, w = a * c - b * sn, a * sn + b * c
    turned = torch.cat([u, w], -1) if half else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([turned, rest], -1).bfloat16()


def _plain_rope(s):
    case = s["case"]
    page = case["page"]
    axes = torch.tensor(s["axes"], device="cuda")
    pair = torch.arange(len(s["axes"]), device="cuda")
    turns = s["freqs"].unflatten(1, (-1, 2))[s["positions"].long()[axes].T, pair]
    c, sn = turns[:, None, :, 0], turns[:, None, :, 1]
    s["turned"].copy_(_rotate(s["q"], c, sn, case["half"]))
    r = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["offsets"].long(), r, right=True) - 1
    at = s["lengths"].long()[b] + r - s["offsets"].long()[b]
    where = s["table"].long()[b, at // page]
    s["cache"][0, where, 0, at % page] = _rotate(s["k"], c, sn, case["half"]).flatten(1)
    s["cache"][0, where, 1, at % page] = s["v"].flatten(1)
    return [s["turned"], s["cache"]]


def _plain_attention(s):
    """Request by request, the heads of a group side by side."""
    case = s["case"]
    h, kv, d, page = case["heads"], case["kv_heads"], case["size"], case["page"]
    for b, (c, n) in enumerate(zip(s["ctx"], s["new"])):
        t = torch.arange(c + n, device="cuda")
        rows = s["cache"][0, s["table"][b].long()[t // page], :, t % page].float().unflatten(-1, (kv, d))
        keys, values = rows[:, 0].transpose(0, 1), rows[:, 1].transpose(0, 1)
        r0 = s["first"][b]
        q = s["q"][r0:r0 + n].float().unflatten(1, (kv, h // kv)).transpose(0, 1).flatten(1, 2)
        score = torch.bmm(q, keys.transpose(1, 2)).mul_(s["scale"]).unflatten(1, (n, h // kv))
        p = torch.arange(c, c + n, device="cuda")[:, None]
        seen = t[None] <= p
        if case["window"]:
            seen = seen & ((t[None] > p - case["window"]) | (t[None] < case["sinks"]))
        score.masked_fill_(~seen[None, :, None], -math.inf)
        top = score.amax(-1, keepdim=True)
        weight = score.sub_(top).exp_()
        total = weight.sum(-1)
        out = torch.bmm(weight.flatten(1, 2), values).unflatten(1, (n, h // kv)) / total[..., None]
        s["out"][r0:r0 + n] = out.transpose(0, 1).reshape(n, h, d).bfloat16()
        s["lse"][r0:r0 + n] = (top[..., 0] + total.log()).transpose(0, 1).reshape(n, h)
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _own(state)
    return _plain_rope(state) if state["case"]["kind"] == "rope" else _plain_attention(state)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, head by head
# ---------------------------------------------------------------------------------------

def _exact_turn(x, angle_of, half):
    """x [rows, heads, D] in 64 bits; angle_of(j): (cos, sin) of pair j for every row."""
    y = x.clone()
    pairs = angle_of.shape[1]
    for j in range(pairs):
        i, k = (j, j + pairs) if half else (2 * j, 2 * j + 1)
        c, sn = angle_of[:, j, 0, None], angle_of[:, j, 1, None]
        y[..., i] = x[..., i] * c - x[..., k] * sn
        y[..., k] = x[..., k] * c + x[..., i] * sn
    return y


def _exact_rope(s, case):
    angle = torch.stack([s["freqs"][s["positions"][a].long(), 2 * j:2 * j + 2]
                         for j, a in enumerate(_pair_axes(case))], 1).double()
    cache, r = s["cache"].double(), 0
    keys = _exact_turn(s["k"].double(), angle, case["half"]).flatten(1)
    for b, (c, n) in enumerate(zip(s["ctx"], s["new"])):
        at = torch.arange(c, c + n, device="cuda")
        held = s["table"][b].long()[at // case["page"]]
        cache[0, held, 0, at % case["page"]] = keys[r:r + n]
        cache[0, held, 1, at % case["page"]] = s["v"][r:r + n].flatten(1).double()
        r += n
    return [_exact_turn(s["q"].double(), angle, case["half"]), cache]


def _exact_attention(s, case):
    group, page, d = case["heads"] // case["kv_heads"], case["page"], case["size"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    r = 0
    for b, (c, n) in enumerate(zip(s["ctx"], s["new"])):
        t = torch.arange(c + n, device="cuda")
        held = s["table"][b].long()[t // page]
        # how far back a key lies from each new token
        back = torch.arange(c, c + n, device="cuda")[:, None] - t[None]
        hidden = back < 0
        if case["window"]:
            hidden = hidden | ((back >= case["window"]) & (t >= case["sinks"])[None])
        for h in range(case["heads"]):
            cols = slice(h // group * d, (h // group + 1) * d)
            keys = s["cache"][0, held, 0, t % page, cols].double()
            score = s["q"][r:r + n, h].double() @ keys.T * s["scale"]
            score[hidden] = -math.inf
            lse[r:r + n, h] = torch.logsumexp(score, 1)
            weight = (score - lse[r:r + n, h, None]).exp()
            out[r:r + n, h] = weight @ s["cache"][0, held, 1, t % page, cols].double()
        r += n
    return [out, lse]


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s, case) if case["kind"] == "rope" else _exact_attention(s, case)
