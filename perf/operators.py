"""The speculative-decoding operators of the MLA cache: what is measured, and their plain forms.

Four operators that a serving step with drafted tokens runs one after the other on the paged
latent cache:

  attention   `mla_tree_attention_paged` (and `_qcache`): absorbed MLA attention of the new
              tokens of every request (one token, a chain, or a tree given by a mask) over
              the request's cached latent rows and the new tokens' own rows
  rope        `mla_rope_heads`: the position rotation of the queries' rope columns at given
              positions, interleaved or half layout, out of one strided tensor into another
  write       `mla_cache_write_paged_at` (and `_qcache_at`): RMSNorm + RoPE of new latent
              rows whose rotary position differs from their cache position (a tree's depth)
  compact     `mla_cache_compact_paged` (and `_qcache`): the accepted path's rows move to the
              front of the drafted region in every layer, and the lengths grow by its length

A case holds sizes only; request lengths and tree shapes follow from its `shape` number and
the values from the seed that `prepare` is given.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def _attention(batch, heads, ctx, new, page, tree, quantised=False, rank=512, rope=64, shape=1):
    return {"kind": "attention", "batch": batch, "heads": heads, "rank": rank, "rope": rope,
            "page": page, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0],
            "new_hi": new[1], "tree": tree, "quantised": quantised, "shape": shape}


def _rope(rows, heads, nope, rank, rope, half, positions, shape=1):
    return {"kind": "rope", "rows": rows, "heads": heads, "nope": nope, "rank": rank,
            "rope": rope, "half": half, "positions": positions, "shape": shape}


def _write(batch, ctx, new, page, rank=512, rope=64, shape=1):
    return {"kind": "write", "batch": batch, "rank": rank, "rope": rope, "page": page,
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0], "new_hi": new[1],
            "shape": shape}


def _compact(batch, layers, ctx, new, kept, page, rank=512, rope=64, shape=1):
    return {"kind": "compact", "batch": batch, "layers": layers, "rank": rank, "rope": rope,
            "page": page, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0],
            "new_hi": new[1], "kept": kept, "shape": shape}


def listed():
    return [
        # one user, one token, an eighth of the heads (a tensor-parallel share): latency alone
        dict(_attention(1, 16, (500, 500), (1, 1), 64, False, shape=11), name="token_one_user"),
        # a full decode batch, one token each, all 128 heads of the benchmark's model
        dict(_attention(64, 128, (512, 4096), (1, 1), 128, False, shape=12), name="token_batch"),
        # few users with long histories: the key axis has to be split
        dict(_attention(4, 128, (32768, 32768), (1, 1), 128, False, shape=13), name="token_long"),
        # verification of drafted trees, all heads: bound by the tensor cores
        dict(_attention(16, 128, (512, 4096), (16, 64), 128, True, shape=14), name="tree_batch"),
        # ragged trees over small pages, a share of the heads, some histories near empty
        dict(_attention(33, 16, (0, 2047), (1, 23), 16, True, shape=15), name="tree_ragged"),
        # short chains over the quantised cache
        dict(_attention(32, 128, (512, 4096), (1, 4), 128, False, True, shape=16), name="chain_qcache"),
        # queries of one drafted tree, a share of the heads, half layout
        dict(_rope(37, 16, 128, 512, 64, True, 163840, shape=21), name="rope_tree"),
        # queries of a prefill chunk, all heads, interleaved layout
        dict(_rope(4096, 128, 128, 512, 64, False, 163840, shape=22), name="rope_prefill"),
        # a few drafted trees written to a small cache
        dict(_write(5, (0, 600), (3, 17), 16, shape=31), name="write_trees"),
        # a large batch of drafted trees
        dict(_write(256, (0, 1024), (48, 64), 128, shape=32), name="write_batch"),
        # one user's accepted path, a model of few layers
        dict(_compact(1, 8, (100, 100), (24, 24), 4, 64, shape=45), name="compact_one_user"),
        # the accepted paths of a batch in all layers
        dict(_compact(128, 16, (0, 128), (33, 64), 8, 64, shape=42), name="compact_batch"),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw_one(rng):
    shape = rng.randrange(1 << 30)
    kind = rng.choice(["attention", "attention", "attention", "rope", "write", "compact"])
    page = rng.choice([8, 12, 16, 32, 40, 64, 96, 128, 256])
    rank, rope = rng.choice([(512, 64), (512, 64), (512, 64), (256, 64), (128, 32), (384, 48), (64, 16)])
    if kind == "attention":
        quantised = rng.random() < 0.3 and rank % 128 == 0
        tree = rng.random() < 0.5
        new = _log_int(rng, 1, 64) if tree or rng.random() < 0.5 else 1
        ctx = _log_int(rng, 1, 32768)
        return _attention(_log_int(rng, 1, 64), rng.choice([1, 3, 8, 16, 20, 32, 64, 96, 128, 128]),
                          (rng.randint(0, ctx), ctx), (rng.randint(1, new), new), page, tree,
                          quantised, rank, rope, shape)
    if kind == "rope":
        return _rope(_log_int(rng, 1, 4096), rng.choice([1, 3, 8, 16, 20, 64, 96, 128]),
                     rng.choice([64, 128]), rank, rope, rng.random() < 0.5,
                     rng.choice([4096, 32768, 163840]), shape)
    new = _log_int(rng, 2, 64)
    ctx = _log_int(rng, 1, 1024 if kind == "write" else 128)
    if kind == "write":
        return _write(_log_int(rng, 1, 256), (rng.randint(0, ctx), ctx), (rng.randint(1, new), new),
                      page, rank, rope, shape)
    return _compact(_log_int(rng, 1, 128), _log_int(rng, 1, 16), (rng.randint(0, ctx), ctx),
                    (rng.randint(2, new), new), rng.randint(1, 8), min(page, 64), rank, rope, shape)


def _padded(case):
    """Values of the largest tensor that the plain form holds at once."""
    if case["kind"] != "attention":
        return 0
    ctx, new = _lengths(case)
    longest = max(c + n for c, n in zip(ctx, new))
    return case["batch"] * longest * max(max(new) * case["heads"], case["rank"] + case["rope"])


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["kind"], {"bytes": 0, "flops": 0, "padded": 0})
        most[c["kind"]] = {"bytes": max(m["bytes"], w["bytes"]), "flops": max(m["flops"], w["flops"]),
                           "padded": max(m["padded"], _padded(c))}
    while True:
        c = _draw_one(rng)
        w, m = work(c), most[c["kind"]]
        if w["bytes"] <= m["bytes"] and w["flops"] <= m["flops"] and _padded(c) <= m["padded"]:
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


def _parents(case):
    """Parent of every drafted token of every request (-1: none)."""
    _, new = _lengths(case)
    rng = random.Random(case["shape"] + 1)
    return [[-1] + [rng.randint(max(0, i - 8), i - 1) for i in range(1, n)] for n in new]


def _ancestors(parents):
    """Bit j of entry i: token j is i itself or one of its ancestors."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
    return bits


def _depths(parents):
    depth = []
    for p in parents:
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return depth


def _kept(case):
    """The accepted path of every request: token 0 and then tokens from the tree's end, so
    that running the call again on its own result changes nothing."""
    _, new = _lengths(case)
    rng = random.Random(case["shape"] + 2)
    paths = []
    for n in new:
        m = rng.randint(1, min(case["kept"], (n + 1) // 2))
        paths.append([0] + sorted(rng.sample(range(m, n), m - 1)))
    return paths


def work(case):
    if case["kind"] == "rope":
        n = case["rows"] * case["heads"] * case["rope"]
        return {"bytes": 4 * n + 4 * case["rows"] * (1 + case["rope"]), "flops": 3 * n}
    cols = case["rank"] + case["rope"]
    ctx, new = _lengths(case)
    if case["kind"] == "write":
        rows = sum(new)
        return {"bytes": rows * (4 * cols + 4 * case["rope"] + 4),
                "flops": rows * (4 * case["rank"] + 3 * case["rope"])}
    if case["kind"] == "compact":
        moves = sum(sum(1 for j, t in enumerate(p) if t != j) for p in _kept(case))
        return {"bytes": moves * case["layers"] * 4 * cols + 12 * case["batch"], "flops": 0}
    rows, h = sum(new), case["heads"]
    slot = cols * 2 if not case["quantised"] else case["rank"] + 2 * case["rope"] + case["rank"] // 32
    if case["tree"]:
        own_pairs = [sum(bin(b).count("1") for b in _ancestors(p)) for p in _parents(case)]
    else:
        own_pairs = [n * (n + 1) // 2 for n in new]
    pairs = sum(c * n + o for c, n, o in zip(ctx, new, own_pairs))
    mask = rows * 4 * ((max(new) + 31) // 32) if case["tree"] else 0
    return {"bytes": sum(c + n for c, n in zip(ctx, new)) * slot + mask
            + rows * h * (2 * cols + 2 * case["rank"] + 4),
            "flops": 2 * pairs * h * (cols + case["rank"])}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _normal(g, *size, dtype=torch.bfloat16):
    return torch.randn(size, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _int32(values):
    return torch.tensor(values, dtype=torch.int64).to(torch.int32).cuda()


def _paging(case, g, ctx, new):
    """A shuffled page table and its page count: pages for every cached and new token."""
    need = [(c + n + case["page"] - 1) // case["page"] for c, n in zip(ctx, new)]
    order = torch.randperm(sum(need) + 1, generator=g, device="cuda").to(torch.int32)
    width = max(max(need), 1)
    at = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda")
    column = torch.arange(width, device="cuda")
    inside = column[None] < torch.tensor(need, device="cuda")[:, None]
    table = order[(at[:, None] + column[None]).clamp(max=sum(need) - 1)]
    return torch.where(inside, table, torch.zeros_like(table)).contiguous(), sum(need) + 1


def _offsets(new):
    total = [0]
    for n in new:
        total.append(total[-1] + n)
    return total


def _freqs(positions, rope, base=10000.0, factor=40.0, trained=4096):
    """(cos, sin) pairs [positions, rope], the slow frequencies stretched for long contexts:
    those that turn less than once over the trained length by `factor`, those that turn more
    than 32 times not at all, a ramp between."""
    pairs = torch.arange(rope // 2, device="cuda", dtype=torch.float64)
    inv = base ** (-2 * pairs / rope)
    turns = trained * inv / (2 * math.pi)
    ramp = ((turns - 1) / 31).clamp(0, 1)
    inv = inv * (ramp + (1 - ramp) / factor)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.stack([angle.cos(), angle.sin()], -1).reshape(positions, rope).float().contiguous()


def _quantised(g, pages, case):
    """Slots of a quantised cache: e4m3 codes, bf16 rope columns, fp32 block scales."""
    rank, rope, page = case["rank"], case["rope"], case["page"]
    x = _normal(g, pages, page, rank // 128, 128, dtype=torch.float32)
    scale = x.abs().amax(-1) / 448.0
    codes = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(pages, page, rank)
    k_rope = _normal(g, pages, page, rope).view(torch.uint8)
    payload = torch.cat([codes, k_rope, scale.contiguous().view(torch.uint8)], -1)
    slot = (payload.shape[-1] + 15) // 16 * 16
    return torch.nn.functional.pad(payload, (0, slot - payload.shape[-1])).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    rope, rank = case["rope"], case["rank"]
    cols = rank + rope
    if case["kind"] == "rope":
        x = _normal(g, case["rows"], case["heads"], case["nope"] + rope)
        q = _normal(g, case["rows"], case["heads"], cols)
        s.update(x=x[..., case["nope"]:], y=q[..., rank:], freqs=_freqs(case["positions"], rope),
                 positions=torch.randint(0, case["positions"], (case["rows"],), generator=g,
                                         device="cuda").to(torch.int32))
        return s
    ctx, new = _lengths(case)
    table, pages = _paging(case, g, ctx, new)
    s.update(table=table, pages=pages, lengths=_int32(ctx), offsets=_int32(_offsets(new)))
    if case["kind"] == "write":
        depths = [_depths(p) for p in _parents(case)]
        s.update(cache=_normal(g, 1, pages, case["page"], cols), latent=_normal(g, sum(new), cols),
                 gamma=_normal(g, rank, dtype=torch.float32).mul_(0.1).add_(1.0),
                 positions=_int32([c + d for c, ds in zip(ctx, depths) for d in ds]),
                 freqs=_freqs(max(c + n for c, n in zip(ctx, new)), rope))
        return s
    if case["kind"] == "compact":
        kept = _kept(case)
        s.update(cache=_normal(g, case["layers"], pages, case["page"], cols),
                 kept=_int32([p + [0] * (case["kept"] - len(p)) for p in kept]),
                 counts=_int32([len(p) for p in kept]),
                 new_lengths=torch.zeros(case["batch"], dtype=torch.int32, device="cuda"))
        return s
    words = (max(new) + 31) // 32
    s.update(mask=None, width=max(new), longest=max(c + n for c, n in zip(ctx, new)))
    if case["tree"]:
        bits = [b for p in _parents(case) for b in _ancestors(p)]
        flat = [(b >> (32 * w)) & 0xFFFFFFFF for b in bits for w in range(words)]
        s["mask"] = _int32(flat).view(-1, words)
    rows = sum(new)
    s.update(q=_normal(g, rows, case["heads"], cols), scale=1.0 / math.sqrt(128 + rope),
             cache=_quantised(g, pages, case)[None] if case["quantised"]
             else _normal(g, 1, pages, case["page"], cols),
             out=torch.empty(rows, case["heads"], rank, dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty(rows, case["heads"], dtype=torch.float32, device="cuda"))
    return s


# ---------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------

def _handle(s):
    """What a user's program keeps beside its tensors: the cache descriptor, the workspace."""
    import paged_kv_mla_gb300 as pkm
    case, cache = s["case"], s["cache"]
    sizes = dict(data=cache, page_table=s["table"], layer_stride=cache.stride(0),
                 page_stride=cache.stride(1), slot_stride=cache.stride(2),
                 num_layers=cache.shape[0], num_pages=cache.shape[1], page_size=cache.shape[2],
                 cache_lengths=s["lengths"])
    if cache.dtype == torch.uint8:
        s["handle"] = pkm.QuantCache(kv_lora_rank=case["rank"], rope_dim=case["rope"], **sizes)
    else:
        s["handle"] = pkm.PagedCache(row_elems=case["rank"] + case["rope"], **sizes)
    if case["kind"] == "attention":
        s["workspace"] = torch.empty(pkm.mla_tree_attention_paged_workspace_size(
            s["q"].shape[0], case["heads"], case["rank"]), dtype=torch.uint8, device="cuda")
    return s["handle"]


def _own(s):
    import paged_kv_mla_gb300 as pkm
    case = s["case"]
    if case["kind"] == "rope":
        pkm.mla_rope_heads(s["x"], s["positions"], s["freqs"], s["y"], half=case["half"])
        return s["y"]
    cache = s.get("handle") or _handle(s)
    if case["kind"] == "write":
        pkm.mla_cache_write_paged_at(s["latent"], s["offsets"], s["positions"], s["gamma"], 1e-6,
                                     s["freqs"], cache, 0, case["rank"], case["rope"])
        return s["cache"]
    if case["kind"] == "compact":
        pkm.mla_cache_compact_paged(cache, 0, case["layers"], s["kept"], s["counts"],
                                    s["new_lengths"])
        return [s["cache"], s["new_lengths"]]
    if case["quantised"]:
        pkm.mla_tree_attention_paged_qcache(s["q"], s["offsets"], s["scale"], cache, 0, s["out"],
                                            s["workspace"], tree_mask=s["mask"], lse=s["lse"])
    else:
        pkm.mla_tree_attention_paged(s["q"], s["offsets"], s["scale"], cache, 0, case["rank"],
                                     case["rope"], s["out"], s["workspace"], tree_mask=s["mask"],
                                     lse=s["lse"])
    return [s["out"], s["lse"]]


# ---------------------------------------------------------------------------------------
# plain forms: elementary torch operations in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------------------

def _rotate(x, cs, half):
    """x [..., P] rotated by the (cos, sin) pairs cs [..., P], in 32 bits."""
    pairs = cs.unflatten(-1, (-1, 2))
    c, sn = pairs[..., 0], pairs[..., 1]
    p = x.shape[-1] // 2
    x = x.float()
    a, b = (x[..., :p], x[..., p:]) if half else (x[..., 0::2], x[..., 1::2])
    u, v = a * c - b * sn, a * sn + b * c
    return torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)


def _plain_rope(s):
    cs = s["freqs"][s["positions"].long()][:, None]
    s["y"].copy_(_rotate(s["x"], cs, s["case"]["half"]))
    return s["y"]


def _request_of_rows(s, rows):
    """Request of every row, and the row's place in it."""
    r = torch.arange(rows, device="cuda")
    b = torch.searchsorted(s["offsets"].long(), r, right=True) - 1
    return b, r - s["offsets"].long()[b]


def _plain_write(s):
    case = s["case"]
    rank, page = case["rank"], case["page"]
    x = s["latent"].float()
    nope = x[:, :rank]
    nope = nope * s["gamma"] / torch.sqrt((nope * nope).mean(-1, keepdim=True) + 1e-6)
    turned = _rotate(x[:, rank:], s["freqs"][s["positions"].long()], False)
    b, i = _request_of_rows(s, x.shape[0])
    at = s["lengths"].long()[b] + i
    s["cache"][0, s["table"].long()[b, at // page], at % page] = torch.cat([nope, turned], -1).bfloat16()
    return s["cache"]


def _plain_compact(s):
    case = s["case"]
    page, table = case["page"], s["table"].long()
    j = torch.arange(case["kept"], device="cuda")
    live = j[None] < s["counts"][:, None]
    # a place without an accepted token takes its request's first one, which does not move
    to = s["lengths"].long()[:, None] + torch.where(live, j[None], 0)
    fro = s["lengths"].long()[:, None] + torch.where(live, s["kept"].long(), 0)
    b = torch.arange(case["batch"], device="cuda")[:, None]
    s["cache"][:, table[b, to // page], to % page] = s["cache"][:, table[b, fro // page], fro % page]
    s["new_lengths"].copy_(s["lengths"] + s["counts"])
    return [s["cache"], s["new_lengths"]]


def _rows_of(case, cells):
    """Latent rows in 32 bits; codes times scales are rounded to bf16, as the cache's other
    readers round them."""
    if not case["quantised"]:
        return cells.float()
    rank, rope = case["rank"], case["rope"]
    codes = cells[..., :rank].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128))
    k_rope = cells[..., rank:rank + 2 * rope].contiguous().view(torch.bfloat16).float()
    scale = cells[..., rank + 2 * rope:rank + 2 * rope + rank // 32].contiguous().view(torch.float32)
    return torch.cat([(codes * scale[..., None]).flatten(-2).bfloat16().float(), k_rope], -1)


def _plain_attention(s):
    case = s["case"]
    h, rank, page = case["heads"], case["rank"], case["page"]
    width, longest = s["width"], s["longest"]
    lengths, offsets = s["lengths"].long(), s["offsets"].long()
    at = torch.arange(longest, device="cuda")
    i = torch.arange(width, device="cuda")
    held = s["table"].long()[:, (at // page).clamp(max=s["table"].shape[1] - 1)]
    keys = _rows_of(case, s["cache"][0][held, (at % page)[None]])
    rows = (offsets[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().flatten(1, 2)
    j = at[None] - lengths[:, None]
    if s["mask"] is None:
        seen = j[:, None] <= i[None, :, None]
    else:
        word = s["mask"].long()[rows]
        place = j.clamp(min=0, max=32 * word.shape[-1] - 1)
        picked = torch.gather(word, 2, (place // 32)[:, None].expand(-1, width, -1))
        seen = (picked >> (place % 32)[:, None]) & 1 == 1
        seen = seen & (j < 32 * word.shape[-1])[:, None]
    count = offsets[1:] - offsets[:-1]
    seen = ((j < 0)[:, None] | seen) & (j < count[:, None])[:, None]
    score = torch.bmm(q, keys.transpose(1, 2)).mul_(s["scale"]).unflatten(1, (width, h))
    score.masked_fill_(~seen[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1)
    out = torch.bmm(weight.flatten(1, 2), keys[..., :rank]).unflatten(1, (width, h))
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    lse = top[..., 0] + total.log()
    b, place = _request_of_rows(s, s["q"].shape[0])
    return [out[b, place].bfloat16(), lse[b, place]]


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "rope": _plain_rope, "write": _plain_write,
            "compact": _plain_compact}[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, request by request
# ---------------------------------------------------------------------------------------

def _exact_turn(x, cs, half):
    c, sn = cs[..., 0::2], cs[..., 1::2]
    y = torch.empty_like(x)
    p = x.shape[-1] // 2
    for k in range(p):
        i, j = (k, k + p) if half else (2 * k, 2 * k + 1)
        y[..., i] = x[..., i] * c[..., k] - x[..., j] * sn[..., k]
        y[..., j] = x[..., j] * c[..., k] + x[..., i] * sn[..., k]
    return y


def _exact_attention(s, case, ctx, new):
    rank, page, h = case["rank"], case["page"], case["heads"]
    parents = _parents(case)
    outs, lses, first = [], [], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        t = torch.arange(c + n, device="cuda")
        cells = s["cache"][0, s["table"][b].long()[t // page], t % page]
        if case["quantised"]:
            value = cells[:, :rank].contiguous().view(torch.float8_e4m3fn).double()
            scale = cells[:, rank + 2 * case["rope"]:][:, :rank // 32].contiguous().view(torch.float32)
            value = (value * scale.double().repeat_interleave(128, 1)).float().bfloat16().double()
            part = cells[:, rank:rank + 2 * case["rope"]].contiguous().view(torch.bfloat16).double()
            keys = torch.cat([value, part], 1)
        else:
            keys = cells.double()
        seen = torch.zeros(n, c + n, dtype=torch.bool)
        seen[:, :c] = True
        if case["tree"]:
            for i, bits in enumerate(_ancestors(parents[b])):
                seen[i, c:] = torch.tensor([bool(bits >> j & 1) for j in range(n)])
        else:
            seen[:, c:] = torch.ones(n, n, dtype=torch.bool).tril()
        score = torch.einsum("nhc,tc->nht", s["q"][first:first + n].double(), keys) * s["scale"]
        score = torch.where(seen.cuda()[:, None], score, -math.inf)
        lses.append(torch.logsumexp(score, -1))
        outs.append(torch.einsum("nht,tr->nhr", (score - lses[-1][..., None]).exp(), keys[:, :rank]))
        first += n
    return [torch.cat(outs), torch.cat(lses)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rope":
        return _exact_turn(s["x"].double(), s["freqs"].double()[s["positions"].long()][:, None], case["half"])
    ctx, new = _lengths(case)
    if case["kind"] == "attention":
        return _exact_attention(s, case, ctx, new)
    page, rank = case["page"], case["rank"]
    cache = s["cache"].double()
    first = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        held = s["table"][b].long()
        if case["kind"] == "write":
            x = s["latent"][first:first + n].double()
            size = (x[:, :rank].square().sum(1, keepdim=True) / rank + 1e-6).sqrt()
            at = torch.arange(c, c + n, device="cuda")
            turned = _exact_turn(x[:, rank:], s["freqs"].double()[s["positions"][first:first + n].long()], False)
            cache[0, held[at // page], at % page] = torch.cat([x[:, :rank] / size * s["gamma"].double(), turned], 1)
        else:
            path = _kept(case)[b]
            for j, t in enumerate(path):
                cache[:, held[(c + j) // page], (c + j) % page] = cache[:, held[(c + t) // page], (c + t) % page].clone()
        first += n
    if case["kind"] == "write":
        return cache
    return [cache, None]
