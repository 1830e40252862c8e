"""Measured cases of the operators that a serving step needs around the
quantized products and the paged cache.

plan     page tables, positions and cache slots of a step's new tokens, built on
         the GPU from the requests' lengths
norm     the norm after a block, its gate and residual scale, and the norm before
         the next block in one pass, the result in a float type or as the int8
         activations that the products take
sample   temperature, top-k, top-p and min-p from given random numbers: the tokens,
         or the distribution itself (what the verification of drafts takes)
bounds   the smallest and largest key of each page and head, in int8 blocks
sparse   attention over the pages of the cache whose bounds promise the most, with
         the bounds of the new tokens' pages brought up to date

Each has a plain form in elementary torch operations (own = False) and the
calls of this package's entry points (own = True).
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _tq():
    import block_quantized_matmul_repack_amd as tq
    return tq


def _ctype(case):
    tq = _tq()
    return {"q8_0": tq.Q8_0, "q4_0": tq.Q4_0}[case["ctype"]]


# --------------------------------------------------------------------------
# cases

def listed():
    heads = {"hq": 32, "hkv": 8, "d": 128}       # 4096-wide model, grouped queries
    return [
        # one new token for each of 64 users: all launch latency
        dict(name="plan_decode", op="plan", b=64, most=1, ctx=16384, page=64),
        # prompt chunks beside single tokens, many requests, small pages
        dict(name="plan_mixed", op="plan", b=511, most=1500, ctx=8192, page=16),
        # one token of one user, straight into the next product's activations
        dict(name="norm_token", op="norm", t=1, n=4096, ydtype="fp32", dtype="bf16", post=False,
             gate="none", out="q8"),
        # a long prompt chunk, norms on both sides and a gate for each channel
        dict(name="norm_prompt", op="norm", t=8191, n=4096, ydtype="bf16", dtype="bf16", post=True,
             gate="channel", out="same"),
        # one user, all filters
        dict(name="sample_one", op="sample", rows=1, vocab=128001, dtype="fp32", top_k=40,
             top_p=0.95, min_p=0.05, temp=0.8, probs=False),
        # 64 users, nucleus sampling over the whole vocabulary
        dict(name="sample_batch", op="sample", rows=64, vocab=128001, dtype="fp32", top_k=0,
             top_p=0.95, min_p=0.0, temp=1.0, probs=False),
        # the target's distribution at every node of drafted trees
        dict(name="sample_probs", op="sample", rows=128, vocab=128001, dtype="bf16", top_k=50,
             top_p=0.9, min_p=0.0, temp=0.7, probs=True),
        # the pages that one new token of 64 users lies on
        dict(heads, name="bounds_step", op="bounds", b=64, ctx=1024, ragged=True, nodes=1, page=64,
             ctype="q8_0"),
        # all pages of two prompts
        dict(heads, name="bounds_prompt", op="bounds", b=2, ctx=0, ragged=False, nodes=8191,
             page=64, ctype="q8_0"),
        # one user, a very long cache, one page in 30 read
        dict(heads, name="sparse_long", op="sparse", b=1, ctx=131000, ragged=False, nodes=1,
             page=64, ctype="q8_0", dtype="bf16", keep=64),
        # 64 users of unlike lengths
        dict(heads, name="sparse_batch", op="sparse", b=64, ctx=16384, ragged=True, nodes=1,
             page=64, ctype="q8_0", dtype="bf16", keep=24),
        # trees of drafted tokens over a 4-bit cache of small pages
        dict(heads, name="sparse_tree", op="sparse", b=4, ctx=20011, ragged=True, nodes=31,
             page=32, ctype="q4_0", dtype="fp16", keep=50),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "norm", "norm", "sample", "sample", "bounds", "sparse", "sparse"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "plan":
        b = _log_int(rng, 1, 1024)
        return dict(op=op, b=b, most=_log_int(rng, 1, min(8192, 750 * 511 // b)),
                    ctx=_log_int(rng, 16, 32768), page=rng.choice([16, 32, 64, 128, 256]))
    if op == "norm":
        out = rng.choice(["same", "same", "q8"])
        n = _log_int(rng, 64, 16384)
        n = -(-n // 32) * 32 if out == "q8" else n
        return dict(op=op, t=_log_int(rng, 1, min(8191, 8191 * 4096 // n)), n=n,
                    ydtype=rng.choice([dtype, "fp32"]), dtype=rng.choice([dtype, dtype, "fp32"]),
                    post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token"]), out=out)
    if op == "sample":
        probs = rng.random() < 0.3
        vocab = _log_int(rng, 33, 262144)
        rows = _log_int(rng, 1, min(128, 128 * 128001 // vocab))
        return dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice([dtype, "fp32", "fp32"]),
                    top_k=rng.choice([0, 0, 1, _log_int(rng, 2, 1000)]),
                    top_p=rng.choice([1.0, 0.95, rng.uniform(0.05, 1.0)]),
                    min_p=rng.choice([0.0, 0.0, 0.05, rng.uniform(0.0, 0.5)]),
                    temp=rng.choice([1.0, 0.7, rng.uniform(0.2, 2.0)]), probs=probs)
    d = rng.choice([64, 96, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 4, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    ctype = rng.choice(["q8_0", "q4_0"])
    if op == "bounds":
        b = _log_int(rng, 1, 64)
        nodes = rng.choice([1, _log_int(rng, 2, max(2, 2 * 8191 * 8 * 128 // (b * hkv * d)))])
        nodes = min(nodes, 8191)
        most = max(2, 64 * 1024 * 8 * 128 // (b * hkv * d) - nodes)
        return dict(op=op, hq=hq, hkv=hkv, d=d, b=b, ctx=_log_int(rng, 1, min(most, 32768)),
                    ragged=rng.random() < 0.6, nodes=nodes, page=page, ctype=ctype)
    nodes = rng.choice([1, 1, 1, _log_int(rng, 2, 32)])
    b = _log_int(rng, 1, 64)
    most = min(64 * 16384 * 8 * 128 // (2 * b * hkv * d), 131000)
    return dict(op=op, hq=hq, hkv=hkv, d=d, b=b, ctx=_log_int(rng, 1, most),
                ragged=rng.random() < 0.6, nodes=nodes, page=page, ctype=ctype, dtype=dtype,
                keep=_log_int(rng, 1, max(2, 2048 // page)))


# --------------------------------------------------------------------------
# inputs, from the seed alone

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(nodes):
    out = [0]
    for n in nodes:
        out.append(out[-1] + n)
    return out


def _plan_counts(case):
    """Host lengths: (cached tokens, new tokens, pages owned) of each request."""
    rng = random.Random(case["b"] * 7919 + case["most"])
    page, lens, new, owned = case["page"], [], [], []
    for i in range(case["b"]):
        n = 1 if rng.random() < 0.5 else rng.randint(1, case["most"])
        c = 0 if n > 1 and rng.random() < 0.3 else rng.randint(1, case["ctx"])
        lens.append(c)
        new.append(n)
        # a request may still own pages of drafted tokens that were refused
        owned.append(-(-c // page) + (rng.random() < 0.1))
    return lens, new, owned


def _plan_inputs(case, seed):
    g = _gen(seed)
    lens, new, owned = _plan_counts(case)
    page = case["page"]
    width = -(-(case["ctx"] + case["most"]) // page) + 1
    grow = sum(max(0, -(-(c + n) // page) - o) for c, n, o in zip(lens, new, owned))
    pages = sum(owned) + grow + 37
    order = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.full((case["b"], width), -1, dtype=torch.int32, device="cuda")
    have = torch.arange(width, device="cuda") < _int32(owned)[:, None]
    table[have] = order[:sum(owned)]
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:pages - sum(owned)] = order[sum(owned):]
    return {"lens": _int32(lens), "new": _int32(new), "owned": _int32(owned), "table": table,
            "free": free, "count": _int32([pages - sum(owned)]), "tokens": sum(new) + 5}


def _norm_inputs(case, seed):
    g = _gen(seed)
    t, n, dt = case["t"], case["n"], _DT[case["dtype"]]

    def rand(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    s = {"y": (0.5 * rand(t, n)).to(_DT[case["ydtype"]]), "x": rand(t, n).to(dt),
         "pre": (1 + 0.2 * rand(n)).to(dt), "post": None, "gate": None, "scale": 1.0}
    # a few loud channels, as residual streams have
    s["x"][:, ::97] *= 20
    if case["post"]:
        s["post"] = (1 + 0.2 * rand(n)).to(dt)
    if case["gate"] != "none":
        s["gate"] = (0.3 * rand(*((n,) if case["gate"] == "channel" else (t, n)))).to(dt)
        s["scale"] = 0.9
    return s


def _sample_inputs(case, seed):
    g = _gen(seed)
    shape = (case["rows"], case["vocab"])
    s = {"logits": (2.5 * torch.randn(shape, device="cuda", generator=g)).to(_DT[case["dtype"]]),
         "u": torch.rand(case["rows"], device="cuda", generator=g)}

    def rows(x, dtype):
        return torch.full((case["rows"],), x, dtype=dtype, device="cuda")

    # each request has settings of its own
    s["temp"] = rows(case["temp"], torch.float32)
    s["top_k"] = rows(case["top_k"], torch.int32) if case["top_k"] else None
    s["top_p"] = rows(case["top_p"], torch.float32) if case["top_p"] < 1 else None
    s["min_p"] = rows(case["min_p"], torch.float32) if case["min_p"] > 0 else None
    return s


def _counts(case):
    """Host lengths of the case: (cached tokens, new tokens) of each sequence."""
    b = case["b"]
    rng = random.Random(b * 7919 + case["nodes"])
    if not case["ragged"]:
        return [case["ctx"]] * b, [case["nodes"]] * b
    ctx = [max(1, int(case["ctx"] * rng.uniform(0.1, 1.0))) for _ in range(b)]
    nodes = [rng.randint((case["nodes"] + 1) // 2, case["nodes"]) for _ in range(b)]
    return ctx, nodes


def _kv(n, case, g):
    """Keys with a few loud channels that drift from page to page, as models
    have, and even values."""
    hkv, d = case["hkv"], case["d"]
    loud = 1.0 + 4.0 * (torch.rand(d, device="cuda", generator=g) > 0.95)
    drift = torch.randn((-(-n // case["page"]), hkv, d), device="cuda", generator=g)
    k = torch.randn((n, hkv, d), device="cuda", generator=g)
    k = (k + drift.repeat_interleave(case["page"], 0)[:n]) * loud
    v = torch.randn((n, hkv, d), device="cuda", generator=g)
    return k.bfloat16(), v.bfloat16()


def _parents(n, rng):
    """A tree of n nodes in the order they were drafted; node 0 is the root."""
    return [-1] + [rng.randint(max(0, (i - 1) // 3 - 1), i - 1) for i in range(1, n)]


def _cache_inputs(case, seed):
    """Pages, lengths and (sparse) queries; the cache's contents follow from
    `gen` by _fill_chunks."""
    g = _gen(seed)
    rng = random.Random(seed * 31 + 5)
    ctx, nodes = _counts(case)
    page, b = case["page"], case["b"]
    length = [c + n for c, n in zip(ctx, nodes)]
    per = [(n + page - 1) // page for n in length]
    pages = sum(per) + 1
    order = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.full((b, max(per)), -1, dtype=torch.int32, device="cuda")
    have = torch.arange(max(per), device="cuda") < _int32(per)[:, None]
    table[have] = order[:sum(per)]
    s = {"table": table, "ctx": ctx, "nodes": nodes, "ctx_dev": _int32(ctx),
         "len_dev": _int32(length), "starts": _int32(_starts(nodes)), "pages": pages, "gen": g}
    if case["op"] == "sparse":
        q = torch.randn((sum(nodes), case["hq"], case["d"]), device="cuda", generator=g)
        s["q"], s["scale"], s["mask"] = q.to(_DT[case["dtype"]]), case["d"] ** -0.5, None
        if case["nodes"] > 1:
            rows = []
            for n in nodes:
                par, seen = _parents(n, rng), []
                for i in range(n):
                    seen.append((seen[par[i]] if par[i] >= 0 else 0) | (1 << i))
                rows += [[m - ((1 << 32) if m >> 31 else 0)] for m in seen]
            s["mask"] = _int32(rows)
    return s


def _fill_chunks(case, s):
    """The cache's contents, some pages at a time: (first slot, k, v)."""
    page, g = case["page"], s["gen"]
    step = max(1, (1 << 25) // (page * case["hkv"] * case["d"]))
    for p0 in range(0, s["pages"], step):
        n = min(step, s["pages"] - p0) * page
        k, v = _kv(n, case, g)
        yield p0 * page, k, v


def prepare(case, seed):
    op = case["op"]
    if op in ("plan", "norm", "sample"):
        s = {"plan": _plan_inputs, "norm": _norm_inputs, "sample": _sample_inputs}[op](case, seed)
        s["case"] = case
        return s
    s = _cache_inputs(case, seed)
    s["case"] = case
    blocks = (s["pages"], case["hkv"], case["d"] // 32)
    s["bq"] = torch.zeros((*blocks, 2, 32), dtype=torch.int8, device="cuda")
    s["bd"] = torch.zeros(blocks, dtype=torch.float16, device="cuda")
    if own:
        tq = _tq()
        n = tq.cache_bytes(_ctype(case), s["pages"], case["page"], case["hkv"], case["d"])
        s["kc"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        s["vc"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        for at, k, v in _fill_chunks(case, s):
            where = torch.arange(at, at + k.shape[0], dtype=torch.int32, device="cuda")
            tq.cache_write(_ctype(case), k, v, s["kc"], s["vc"], where, case["page"])
    else:
        parts = [(_quantize(case["ctype"], k), _quantize(case["ctype"], v))
                 for _, k, v in _fill_chunks(case, s)]
        s["kq"], s["kd"] = (torch.cat([p[0][i] for p in parts]) for i in (0, 1))
        s["vq"], s["vd"] = (torch.cat([p[1][i] for p in parts]) for i in (0, 1))
    del s["gen"]
    if op == "sparse":                           # the bounds of what is cached already
        _bounds(s, torch.zeros_like(s["ctx_dev"]), s["len_dev"], case["ctx"] + case["nodes"])
    return s


# --------------------------------------------------------------------------
# plain forms

def _round_away(y):
    """Nearest whole number, halves away from zero."""
    n = y.abs().floor()
    return torch.copysign(n + (y.abs() - n >= 0.5), y)


def _quantize(ctype, x):
    """x [.., D] -> (codes int8, fp16 scales [.., D/32]); each step in fp32."""
    b = x.float().unflatten(-1, (-1, 32))
    if ctype == "q8_0":
        d = b.abs().amax(-1, keepdim=True)
        d = d / torch.full_like(d, 127.0)
        inv = torch.where(d != 0, torch.ones_like(d) / d, torch.zeros_like(d))
        q = _round_away(b * inv)
    else:
        far = b.abs().argmax(-1, keepdim=True)        # the first of the largest
        d = b.gather(-1, far) * -0.125
        inv = torch.where(d != 0, torch.ones_like(d) / d, torch.zeros_like(d))
        q = (b * inv + 8.5).floor().clamp(0, 15) - 8
    return q.to(torch.int8).flatten(-2), d.squeeze(-1).half()


def _values(q, d):
    return (q.unflatten(-1, (-1, 32)).float() * d.float().unsqueeze(-1)).flatten(-2)


def _plain_plan(s):
    case, page = s["case"], s["case"]["page"]
    lens, new, owned = s["lens"].long(), s["new"].long(), s["owned"].long()
    b, width = s["table"].shape
    starts = torch.cat((torch.zeros_like(new[:1]), new.cumsum(0)))
    want = ((lens + new + page - 1) // page).clamp(max=width)
    grow = (want - owned).clamp(min=0)
    off = grow.cumsum(0) - grow
    avail = s["count"].long()
    at = torch.arange(width, device="cuda")
    i = off[:, None] + at - owned[:, None]
    fresh = (at >= owned[:, None]) & (at < (owned + grow)[:, None])
    top = avail - 1 - i
    page_id = torch.where(top >= 0, s["free"][top.clamp(min=0)], torch.full_like(top, -1).int())
    s["table"].copy_(torch.where(fresh, page_id, s["table"]))
    got = torch.minimum((avail - off).clamp(min=0), grow)
    t = torch.arange(s["tokens"], device="cuda")
    seq = (torch.searchsorted(starts, t, right=True) - 1).clamp(max=b - 1)
    live = t < starts[-1]
    pos = torch.where(live, lens[seq] + t - starts[seq], torch.zeros_like(t))
    entry = s["table"][seq, (pos // page).clamp(max=width - 1)].long()
    slot = torch.where(live & (entry >= 0) & (pos // page < width), entry * page + pos % page,
                       torch.full_like(t, -1))
    return [starts.int(), pos.int(), slot.int(), (lens + new).int(), (owned + got).int(),
            (avail - grow.sum()).int(), s["table"]]


def _plain_norm(s):
    case = s["case"]
    y, w = s["y"].float(), s["post"]
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    x = (s["x"].float() * s["scale"] + y).to(s["x"].dtype)
    z = x.float()
    z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 1e-6) * s["pre"].float()
    if case["out"] == "q8":
        q, d = _quantize("q8_0", z)
        z = q.unflatten(-1, (-1, 32)) * d[..., None]
    return [x, z.to(x.dtype) if case["out"] == "same" else z]


def _weight_bits(vocab):
    """Weights are whole multiples of 2^-this, so that their sums do not
    depend on the order: 2^62 holds `vocab` of them."""
    return min(45, 62 - (vocab - 1).bit_length())


def _plain_sample(s):
    case = s["case"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    unit = 2.0 ** _weight_bits(case["vocab"])
    w = (torch.exp((x - top) / s["temp"].double()[:, None]) * unit).round().long()
    # by falling logit, ties by rising index
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    ws = w.gather(-1, order)
    keep = torch.ones_like(ws, dtype=torch.bool)
    if s["top_k"] is not None:
        keep &= torch.arange(case["vocab"], device="cuda") < s["top_k"][:, None]
    if s["top_p"] is not None:
        left = torch.where(keep, ws, torch.zeros_like(ws))
        before = left.cumsum(-1) - left
        want = s["top_p"].double()[:, None] * left.sum(-1, keepdim=True).double()
        keep &= before.double() < want
        keep[:, 0] = True
    if s["min_p"] is not None:
        keep &= ws.double() >= s["min_p"].double()[:, None] * unit
    kept = torch.zeros_like(w).scatter_(-1, order, torch.where(keep, ws, torch.zeros_like(ws)))
    if case["probs"]:
        return (kept.double() / kept.sum(-1, keepdim=True).double()).float()
    run_sum = kept.cumsum(-1)
    hit = run_sum.double() > s["u"].double()[:, None] * run_sum[:, -1:].double()
    return hit.int().argmax(-1).int()


def _plain_bounds(s, begin, end, most):
    """Smallest and largest key of every page that holds a position in
    [begin, end) of its sequence, over its positions before `end`."""
    page, width = s["case"]["page"], s["table"].shape[1]
    for b in range(len(s["ctx"])):
        lo, hi = int(begin[b]), int(end[b])
        for j0 in range(lo // page, min(-(-hi // page), width), 256):
            j = torch.arange(j0, min(j0 + 256, -(-hi // page), width), device="cuda")
            ids = s["table"][b, j].long()
            pos = j[:, None] * page + torch.arange(page, device="cuda")
            slots = ids[:, None] * page + torch.arange(page, device="cuda")
            k = _values(s["kq"][slots], s["kd"][slots])              # [pages, page, hkv, d]
            there = (pos < hi)[:, :, None, None]
            up = k.masked_fill(~there, float("-inf")).amax(1)
            down = k.masked_fill(~there, float("inf")).amin(1)
            both = torch.stack((up.unflatten(-1, (-1, 32)), down.unflatten(-1, (-1, 32))), 3)
            d = both.abs().amax((3, 4), keepdim=True)
            d = d / torch.full_like(d, 127.0)
            inv = torch.where(d != 0, torch.ones_like(d) / d, torch.zeros_like(d))
            s["bq"][ids] = _round_away(both * inv).to(torch.int8)
            s["bd"][ids] = d[..., 0, 0].half()


def _bounds(s, begin, end, most):
    case = s["case"]
    if own:
        _tq().cache_bounds(_ctype(case), s["kc"], s["table"], begin, end, case["hkv"], case["d"],
                           case["page"], s["bq"], s["bd"], max_new=most)
    else:
        _plain_bounds(s, begin.tolist(), end.tolist(), most)


FIRST, LAST = 1, 1                  # pages always read: the first, and before the newest


def _width(case, table_pages):
    new = (case["nodes"] + case["page"] - 2) // case["page"] + 1
    return min(FIRST + LAST + case["keep"] + new, table_pages)


def _plain_select(s):
    """For each sequence and key head the pages to read, and the cached tokens
    on them."""
    case, page = s["case"], s["case"]["page"]
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    tables = torch.full((case["b"], hkv, _width(case, s["table"].shape[1])), -1,
                        dtype=torch.int32, device="cuda")
    ctx_out, row = [], 0
    for b, (ctx, n) in enumerate(zip(s["ctx"], s["nodes"])):
        new, total = ctx // page, -(-(ctx + n) // page)
        first = min(FIRST, max(new - LAST, 0))
        cand = torch.arange(first, max(new - LAST, first), device="cuda")
        keep = min(case["keep"], len(cand))
        ids = s["table"][b, :total].long()
        if keep < len(cand):
            q = s["q"][row:row + n].float().unflatten(1, (hkv, g)).unflatten(-1, (-1, 32))
            dq = q.abs().amax(-1, keepdim=True)
            dq = dq / torch.full_like(dq, 127.0)
            inv = torch.where(dq > 2.0 ** -100, torch.ones_like(dq) / dq, torch.zeros_like(dq))
            q = _round_away(q * inv).double()                        # [n, hkv, g, blocks, 32]
            dots = torch.cat((q.clamp(min=0), q.clamp(max=0)), -1).permute(1, 3, 0, 2, 4)
            dots = dots.flatten(2, 3).contiguous()                   # [hkv, blocks, rows, 64]
            dq = dq.squeeze(-1).double().permute(1, 3, 0, 2).flatten(2)[..., None]
            bq = s["bq"][ids[cand]].double().flatten(3).permute(1, 2, 3, 0).contiguous()
            bd = s["bd"][ids[cand]].double().permute(1, 2, 0)[:, :, None]
            score = (torch.matmul(dots, bq) * (dq * bd)).sum(1).amax(1).float()
            best = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :keep]
            best = cand[best].sort(-1).values
        else:
            best = cand.expand(hkv, -1)
        tail = torch.arange(max(new - LAST, first), total, device="cuda")
        pages = torch.cat((torch.arange(first, device="cuda").expand(hkv, -1), best,
                           tail.expand(hkv, -1)), -1)
        tables[b, :, :pages.shape[1]] = ids[pages].int()
        ctx_out.append(ctx - page * (len(cand) - keep))
        row += n
    return tables, _int32(ctx_out), ctx_out


def _plain_sparse(s):
    case = s["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    tables, ctx_dev, ctxs = _plain_select(s)
    out = torch.empty_like(s["q"])
    row = 0
    for b, (ctx, n) in enumerate(zip(ctxs, s["nodes"])):
        pos = torch.arange(ctx + n, device="cuda")
        slots = tables[b][:, pos // page].long() * page + pos % page             # [hkv, keys]
        head = torch.arange(hkv, device="cuda")[:, None]
        k, v = (_values(s[c + "q"][slots, head], s[c + "d"][slots, head]) for c in "kv")
        q = s["q"][row:row + n].float().unflatten(1, (hkv, hq // hkv))
        q = q.permute(1, 2, 0, 3).flatten(1, 2)                         # [hkv, g * n, d]
        score = torch.matmul(q, k.transpose(1, 2).contiguous()) * s["scale"]
        if s["mask"] is not None:
            node = torch.arange(n, device="cuda")
            bit = (s["mask"][row:row + n, node // 32] >> (node % 32)) & 1
            see = torch.ones((n, ctx + n), dtype=torch.bool, device="cuda")
            see[:, ctx:] = bit.bool()
            score = score.masked_fill(~see.repeat(hq // hkv, 1), float("-inf"))
        p = torch.exp(score - score.amax(-1, keepdim=True))
        o = torch.matmul(p, v.contiguous()) / p.sum(-1, keepdim=True)
        o = o.unflatten(1, (hq // hkv, n)).permute(2, 0, 1, 3).flatten(1, 2)
        out[row:row + n] = o.to(out.dtype)
        row += n
    return [tables, ctx_dev, out]


def run(state):
    case = state["case"]
    op = case["op"]
    if op in ("bounds", "sparse"):
        _bounds(state, state["ctx_dev"], state["len_dev"], case["nodes"])
        if op == "bounds":
            return state["bq"] * state["bd"][..., None, None]        # the values, in fp16
    if not own:
        return {"plan": _plain_plan, "norm": _plain_norm, "sample": _plain_sample,
                "sparse": _plain_sparse}[op](state)
    tq = _tq()
    if op == "plan":
        return [*tq.plan_step(state["lens"], state["new"], state["owned"], state["table"],
                              state["free"], state["count"], case["page"], state["tokens"]),
                state["table"]]
    if op == "norm":
        x, z = tq.residual_norm(state["y"], state["x"], state["pre"], post_weight=state["post"],
                                gate=state["gate"], scale=state["scale"], eps=1e-6,
                                quantize=case["out"] == "q8")
        if case["out"] == "q8":
            z = z[0].unflatten(-1, (-1, 32)) * z[1][..., None]       # the values, in fp16
        return [x, z]
    if op == "sample":
        settings = {k: state[k] for k in ("top_k", "top_p", "min_p")}
        if case["probs"]:
            return tq.sample_probs(state["logits"], temperature=state["temp"], **settings)
        return tq.sample(state["logits"], state["u"], temperature=state["temp"], **settings)
    tables, ctx = tq.select_pages(
        state["q"], state["bq"], state["bd"], state["table"], state["ctx_dev"], state["starts"],
        case["page"], case["keep"], first=FIRST, last=LAST, max_nodes=case["nodes"],
        max_ctx=case["ctx"])
    out = tq.tree_attention(
        _ctype(case), state["q"], state["kc"], state["vc"], tables, ctx, state["starts"],
        case["hkv"], case["page"], max_nodes=case["nodes"], scale=state["scale"],
        max_ctx=min(case["ctx"], tables.shape[2] * case["page"]), mask=state["mask"])
    return [tables, ctx, out]


# --------------------------------------------------------------------------
# what a pass cannot do without

def _size(dtype):
    return torch.finfo(_DT[dtype]).bits // 8


def work(case):
    op = case["op"]
    if op == "plan":
        lens, new, owned = _plan_counts(case)
        page = case["page"]
        grow = sum(max(0, -(-(c + n) // page) - o) for c, n, o in zip(lens, new, owned))
        return {"bytes": 24 * case["b"] + 8 * grow + 8 * sum(new),
                "flops": 8 * case["b"] + 4 * sum(new)}
    if op == "norm":
        n = case["t"] * case["n"]
        out = 1 + 2 / 32 if case["out"] == "q8" else _size(case["dtype"])
        gate = _size(case["dtype"]) if case["gate"] == "token" else 0
        return {"bytes": n * (_size(case["ydtype"]) + 2 * _size(case["dtype"]) + out + gate),
                "flops": 10 * n}
    if op == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (_size(case["dtype"]) + (4 if case["probs"] else 0)), "flops": 4 * n}
    ctx, nodes = _counts(case)
    page, hkv, d = case["page"], case["hkv"], case["d"]
    block = 34 if case["ctype"] == "q8_0" else 18
    token, bound = hkv * (d // 32) * block, hkv * (d // 32) * 66
    fresh = sum(-(-(c + n) // page) - c // page for c, n in zip(ctx, nodes))
    if op == "bounds":
        # the keys of the new tokens' pages (what lies on them before those, too)
        keys = sum(c % page + n for c, n in zip(ctx, nodes))
        return {"bytes": keys * token + fresh * bound, "flops": 2 * keys * hkv * d}
    keys = pairs = scored = 0
    for c, n in zip(ctx, nodes):
        cand = max(c // page - FIRST - LAST, 0)
        drop = max(cand - case["keep"], 0)
        keys += c - drop * page + n
        pairs += n * (c - drop * page + n)
        scored += cand if drop else 0
    return {"bytes": 2 * keys * token + (scored + fresh) * bound
            + 2 * _size(case["dtype"]) * sum(nodes) * case["hq"] * d,
            "flops": 4 * pairs * case["hq"] * d + 4 * scored * case["hq"] * d}


# --------------------------------------------------------------------------
# the definitions in 64 bits

def _f32(x):
    """A 64-bit value rounded to the 32-bit grid, where a definition says so."""
    return x.float().double()


def _exact_blocks(ctype, x):
    """Values of the blocks that x [.., D] is stored as.  The formats define
    their codes by 32-bit steps: the scale, its reciprocal, the product."""
    x = x.double().reshape(*x.shape[:-1], -1, 32)
    if ctype == "q8_0":
        d = _f32(x.abs().max(-1, keepdim=True).values / 127.0)
    else:
        hi, lo = x.max(-1, keepdim=True).values, x.min(-1, keepdim=True).values
        # both signs at the largest magnitude: the earlier element decides
        first_hi = (x == hi).int().argmax(-1, keepdim=True)
        first_lo = (x == lo).int().argmax(-1, keepdim=True)
        up = (hi > -lo) | ((hi == -lo) & (first_hi < first_lo))
        d = torch.where(up, hi, lo) / -8.0
    inv = torch.where(d != 0, _f32(1.0 / d), torch.zeros_like(d))
    y = _f32(x * inv)
    if ctype == "q8_0":
        code = torch.where(y >= 0, (y + 0.5).floor(), (y - 0.5).ceil())
    else:
        code = _f32(y + 8.5).floor().clamp(0, 15) - 8
    return (code * d.float().half().double()).reshape(*x.shape[:-2], -1)


def _exact_plan(case, seed):
    s = _plan_inputs(case, seed)
    page, table, free = case["page"], s["table"].tolist(), s["free"].tolist()
    lens, new, owned = _plan_counts(case)
    left = int(s["count"])
    pos, slot, got = [], [], []
    for c, n, o, row in zip(lens, new, owned, table):
        while o * page < c + n:
            left -= 1
            row[o] = free[left]
            o += 1
        got.append(o)
        for p in range(c, c + n):
            pos.append(p)
            slot.append(row[p // page] * page + p % page)
    rest = s["tokens"] - len(pos)
    return [_int32(_starts(new)), _int32(pos + [0] * rest), _int32(slot + [-1] * rest),
            _int32([c + n for c, n in zip(lens, new)]), _int32(got), _int32([left]), _int32(table)]


def _exact_sample(case, seed):
    s = _sample_inputs(case, seed)
    unit, vocab = 2.0 ** _weight_bits(case["vocab"]), case["vocab"]
    tokens = torch.empty(case["rows"], dtype=torch.int32, device="cuda")
    probs = torch.zeros((case["rows"], vocab), dtype=torch.float64, device="cuda") \
        if case["probs"] else None
    for r in range(case["rows"]):
        x = s["logits"][r].double()
        z = (x - x.max()) / float(s["temp"][r])
        order = torch.argsort(-x, stable=True)
        w = torch.floor(z.exp() * unit + 0.5)[order]
        if s["top_k"] is not None:
            w[int(s["top_k"][r]):] = 0
        if s["top_p"] is not None:
            upto = torch.cumsum(w, 0)            # whole numbers below 2^53 here, or near
            n = 1 + int((upto < float(s["top_p"][r]) * float(w.sum())).sum())
            w[n:] = 0
        if s["min_p"] is not None:
            w[w < float(s["min_p"][r]) * unit] = 0
        back = torch.zeros_like(w)
        back[order] = w
        if case["probs"]:
            probs[r] = back / back.sum()
        else:
            run_sum = torch.cumsum(back, 0)
            tokens[r] = int((run_sum <= float(s["u"][r]) * float(run_sum[-1])).sum())
    return probs if case["probs"] else tokens


def _exact_cache(case, seed):
    """Keys and values [slots, hkv, d] (32 bits: exact) and the inputs."""
    s = _cache_inputs(case, seed)
    chunks = []
    for _, k, v in _fill_chunks(case, s):
        chunks.append((_exact_blocks(case["ctype"], k).float(),
                       _exact_blocks(case["ctype"], v).float()))
    return s, *(torch.cat([c[i] for c in chunks]) for i in (0, 1))


def _exact_bounds(case, s, kall, begin, end):
    """int8 codes [pages, hkv, blocks, 64] and fp16 scales as 64-bit numbers."""
    page, hkv, nb = case["page"], case["hkv"], case["d"] // 32
    codes = torch.zeros((s["pages"], hkv, nb, 64), dtype=torch.float64, device="cuda")
    scale = torch.zeros((s["pages"], hkv, nb), dtype=torch.float64, device="cuda")
    for b, (lo, hi) in enumerate(zip(begin, end)):
        ids = s["table"][b].tolist()
        for j in range(lo // page, -(-hi // page)):
            n = min(page, hi - j * page)
            k = kall[ids[j] * page:ids[j] * page + n].double().reshape(n, hkv, nb, 32)
            both = torch.cat((k.max(0).values, k.min(0).values), -1)
            d = _f32(both.abs().max(-1, keepdim=True).values / 127.0)
            y = _f32(both * torch.where(d != 0, _f32(1.0 / d), torch.zeros_like(d)))
            codes[ids[j]] = torch.where(y >= 0, (y + 0.5).floor(), (y - 0.5).ceil())
            scale[ids[j]] = d[..., 0].float().half().double()
    return codes, scale


def _exact_sparse(case, seed):
    s, kall, vall = _exact_cache(case, seed)
    length = [c + n for c, n in zip(s["ctx"], s["nodes"])]
    codes, scale = _exact_bounds(case, s, kall, [0] * case["b"], length)
    g, page, nb = case["hq"] // case["hkv"], case["page"], case["d"] // 32
    tables = torch.full((case["b"], case["hkv"], _width(case, s["table"].shape[1])), -1,
                        dtype=torch.int32, device="cuda")
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    ctxs, row = [], 0
    for b, (ctx, n) in enumerate(zip(s["ctx"], s["nodes"])):
        ids = s["table"][b].long()
        total, new = -(-(ctx + n) // page), ctx // page
        cand = list(range(FIRST, new - LAST))
        drop = max(0, len(cand) - case["keep"])
        c2 = ctx - drop * page
        ctxs.append(c2)
        allow = torch.ones((n, c2 + n), dtype=torch.bool, device="cuda")
        if s["mask"] is not None:
            words = s["mask"][row:row + n].long() & 0xFFFFFFFF
            for j in range(n):
                allow[:, c2 + j] = (words[:, j // 32] >> (j % 32)) % 2 == 1
        for h in range(case["hkv"]):
            read = list(range(total))
            if drop:
                at = ids[torch.tensor(cand, device="cuda")]
                score = torch.full((len(cand),), -math.inf, dtype=torch.float64, device="cuda")
                for r in range(n):
                    for e in range(g):
                        q = s["q"][row + r, h * g + e].double().reshape(nb, 32)
                        d = _f32(q.abs().max(-1, keepdim=True).values / 127.0)
                        y = _f32(q * torch.where(d > 2.0 ** -100, _f32(1.0 / d), 0 * d))
                        y = torch.where(y >= 0, (y + 0.5).floor(), (y - 0.5).ceil())
                        best = torch.maximum(y * codes[at, h, :, :32], y * codes[at, h, :, 32:])
                        score = torch.maximum(
                            score, (best.sum(-1) * (d[:, 0] * scale[at, h])).sum(-1))
                by = torch.argsort(-_f32(score), stable=True)[:case["keep"]]
                kept = sorted(cand[i] for i in by.tolist())
                read = list(range(FIRST)) + kept + list(range(new - LAST, total))
            pages = ids[torch.tensor(read, device="cuda")]
            tables[b, h, :len(read)] = pages.int()
            slots = (pages[:, None] * page + torch.arange(page, device="cuda")).flatten()[:c2 + n]
            k, v = kall[slots, h].double(), vall[slots, h].double()
            for e in range(g):
                a = (s["q"][row:row + n, h * g + e].double() @ k.t()) * s["scale"]
                a = torch.where(allow, a, torch.full_like(a, -math.inf))
                out[row:row + n, h * g + e] = torch.softmax(a, -1) @ v
        row += n
    return [tables, _int32(ctxs), out]


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return _exact_plan(case, seed)
    if op == "norm":
        s = _norm_inputs(case, seed)
        y = s["y"].double()
        if s["post"] is not None:
            y = s["post"].double() * y / torch.sqrt(y.square().sum(-1, keepdim=True) / case["n"]
                                                    + 1e-6)
        gate = 1.0 if s["gate"] is None else s["gate"].double()
        x = s["scale"] * s["x"].double() + gate * y
        r = x.to(s["x"].dtype).double()          # the norm is of what is stored
        z = r / torch.sqrt(r.square().sum(-1, keepdim=True) / case["n"] + 1e-6) * s["pre"].double()
        if case["out"] == "q8":
            z = _exact_blocks("q8_0", _f32(z)).unflatten(-1, (-1, 32))
        return [x, z]
    if op == "sample":
        return _exact_sample(case, seed)
    if op == "bounds":
        s, kall, _ = _exact_cache(case, seed)
        length = [c + n for c, n in zip(s["ctx"], s["nodes"])]
        codes, scale = _exact_bounds(case, s, kall, s["ctx"], length)
        return (codes * scale[..., None]).unflatten(-1, (2, 32))
    return _exact_sparse(case, seed)
