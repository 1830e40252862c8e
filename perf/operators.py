"""Measured cases of the speculative-decoding operators over a block-quantized cache.

Four operators that a decode loop runs one after another:

norm_rope   per-head RMS norm of queries and keys and their position rotation, one pass
cache       keys and values quantized into Q8_0 / Q4_0 blocks of a paged cache, and read back
attention   attention of one token, a chain or a tree of drafted tokens over that cache
verify      drafted tokens accepted or replaced from the target's probabilities and given
            random numbers

Each has a plain form in elementary torch operations (own = False) and the
call of this package's entry point (own = True).
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_LIMIT = 65472.0                    # largest magnitude a cache block stands for


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
        # one token of one user: all launch latency
        dict(heads, name="norm_rope_token", op="norm_rope", t=1, rot=128, dtype="bf16",
             interleaved=False, norm=True, far=4096),
        # a long prompt chunk, far positions
        dict(heads, name="norm_rope_prompt", op="norm_rope", t=8192, rot=128, dtype="bf16",
             interleaved=False, norm=True, far=131072),
        # narrow heads, half of each rotated, neighbouring pairs, odd count of tokens
        dict(name="norm_rope_partial", op="norm_rope", hq=12, hkv=3, d=96, t=777, rot=48,
             dtype="fp16", interleaved=True, norm=True, far=32768),
        # one new token for each of 64 users
        dict(heads, name="cache_step", op="cache", t=64, page=64, ctype="q8_0", dtype="bf16"),
        # a prompt chunk stored and read back
        dict(heads, name="cache_prompt", op="cache", t=8192, page=64, ctype="q8_0",
             dtype="bf16"),
        # 4-bit cache, small pages, odd count of tokens
        dict(name="cache_q4", op="cache", hq=12, hkv=12, d=64, t=1501, page=16, ctype="q4_0",
             dtype="fp16"),
        # one user, one token: few rows, the long axis has to be split
        dict(heads, name="attention_token", op="attention", b=1, ctx=8191, ragged=False,
             nodes=1, page=64, ctype="q8_0", dtype="bf16"),
        # 64 users of unlike lengths, one token each: cache bandwidth
        dict(heads, name="attention_batch", op="attention", b=64, ctx=16384, ragged=True,
             nodes=1, page=64, ctype="q8_0", dtype="bf16"),
        # trees of 63 drafted tokens over a 4-bit cache: matrix work counts
        dict(heads, name="attention_tree", op="attention", b=4, ctx=20011, ragged=True,
             nodes=63, page=32, ctype="q4_0", dtype="bf16"),
        # a small tree over a very long cache
        dict(heads, name="attention_long", op="attention", b=1, ctx=131000, ragged=False,
             nodes=13, page=128, ctype="q8_0", dtype="fp16"),
        # one user, a chain of four drafted tokens with the draft's probabilities
        dict(name="verify_chain", op="verify", b=1, nodes=5, vocab=128001, tree=False,
             draft=True),
        # 32 users, trees of most likely tokens (no draft probabilities), ragged
        dict(name="verify_trees", op="verify", b=32, nodes=31, vocab=128001, tree=True,
             draft=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "cache", "attention", "attention", "verify"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    d = rng.choice([64, 96, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 4, 7, 8])
    if op == "norm_rope":
        most = 8192 * 40 * 128 // ((hq + hkv) * d)
        return dict(op=op, hq=hq, hkv=hkv, d=d, t=_log_int(rng, 1, min(most, 8192)),
                    rot=rng.choice([d, d, d // 2]), dtype=rng.choice([dtype, dtype, "fp32"]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.8,
                    far=_log_int(rng, 64, 1 << 20))
    ctype = rng.choice(["q8_0", "q4_0"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "cache":
        most = 8192 * 8 * 128 // (hkv * d)
        return dict(op=op, hq=hq, hkv=hkv, d=d, t=_log_int(rng, 1, min(most, 8192)), page=page,
                    ctype=ctype, dtype=rng.choice([dtype, dtype, "fp32"]))
    if op == "attention":
        nodes = rng.choice([1, 1, 1, _log_int(rng, 2, 128), _log_int(rng, 2, 128)])
        b = _log_int(rng, 1, 64)
        # no more cache or matrix work than the largest listed cases
        most = min(64 * 16384 * 8 * 128 // (2 * b * hkv * d),
                   4 * 20011 * 63 * 32 * 128 // (b * nodes * hq * d), 131000)
        return dict(op=op, hq=hq, hkv=hkv, d=d, b=b, ctx=_log_int(rng, 1, max(most, 2)),
                    ragged=rng.random() < 0.6, nodes=nodes, page=page, ctype=ctype, dtype=dtype)
    tree = rng.random() < 0.5
    draft = rng.random() < 0.6
    nodes = _log_int(rng, 1, 31) if tree else _log_int(rng, 1, 9)
    b = _log_int(rng, 1, 32)
    most = 32 * 31 * 128001 // (b * nodes * (2 if draft else 1))
    return dict(op=op, b=b, nodes=nodes, vocab=_log_int(rng, 33, min(most, 262144)), tree=tree,
                draft=draft)


# --------------------------------------------------------------------------
# inputs, from the seed alone

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _counts(case):
    """Host lengths of the case: (cached tokens, new tokens) of each sequence."""
    b = case["b"]
    rng = random.Random(b * 7919 + case["nodes"])
    if not case.get("ragged", case.get("tree", False)):
        return [case.get("ctx", 0)] * b, [case["nodes"]] * b
    ctx = [max(1, int(case.get("ctx", 0) * rng.uniform(0.1, 1.0))) for _ in range(b)]
    nodes = [rng.randint((case["nodes"] + 1) // 2, case["nodes"]) for _ in range(b)]
    return ctx, nodes


def _parents(n, rng):
    """A tree of n nodes in the order they were drafted; node 0 is the root."""
    return [-1] + [rng.randint(max(0, (i - 1) // 3 - 1), i - 1) for i in range(1, n)]


def _starts(nodes):
    out = [0]
    for n in nodes:
        out.append(out[-1] + n)
    return out


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _kv(n, case, g):
    """Keys with a few loud channels, as models have, and even values."""
    shape = (n, case["hkv"], case["d"])
    loud = 1.0 + 4.0 * (torch.rand(case["d"], device="cuda", generator=g) > 0.95)
    k = torch.randn(shape, device="cuda", generator=g) * loud
    v = torch.randn(shape, device="cuda", generator=g)
    return k.to(_DT[case["dtype"]]), v.to(_DT[case["dtype"]])


def _norm_rope_inputs(case, seed):
    g = _gen(seed)
    dt, t, d = _DT[case["dtype"]], case["t"], case["d"]
    hq, hkv = case["hq"], case["hkv"]
    # queries, keys and values lie in one fused projection's rows
    qkv = torch.randn((t, (hq + 2 * hkv) * d), device="cuda", generator=g).to(dt)
    s = {"q": qkv[:, :hq * d].unflatten(1, (hq, d)),
         "k": qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
         "wq": None, "wk": None}
    if case["norm"]:
        s["wq"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt)
        s["wk"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt)
    first = int(torch.randint(0, case["far"], (1,), device="cuda", generator=g))
    s["pos"] = torch.arange(first, first + t, dtype=torch.int32, device="cuda")
    half = case["rot"] // 2
    s["freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
                 ).float()
    return s


def _cache_inputs(case, seed):
    g = _gen(seed)
    t, page = case["t"], case["page"]
    pages = 2 * ((t + page - 1) // page) + 3
    k, v = _kv(t, case, g)
    # the tokens of whole pages in order, the pages anywhere
    order = torch.randperm(pages, device="cuda", generator=g)
    at = torch.arange(t, device="cuda") + page // 3
    slots = (order[at // page] * page + at % page).int()
    return {"k": k, "v": v, "slots": slots, "pages": pages}


def _attention_inputs(case, seed):
    g = _gen(seed)
    rng = random.Random(seed * 31 + 5)
    ctx, nodes = _counts(case)
    page, b = case["page"], case["b"]
    length = [c + n for c, n in zip(ctx, nodes)]
    per = [(n + page - 1) // page for n in length]
    pages = sum(per) + 1
    order = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.full((b, max(per)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i in range(b):
        table[i, :per[i]] = order[at:at + per[i]]
        at += per[i]
    total = sum(nodes)
    q = torch.randn((total, case["hq"], case["d"]), device="cuda", generator=g)
    mask = None
    if case["nodes"] > 1:
        words = (case["nodes"] + 31) // 32
        rows = []
        for n in nodes:
            par, seen = _parents(n, rng), []
            for i in range(n):
                seen.append((seen[par[i]] if par[i] >= 0 else 0) | (1 << i))
            for m in seen:
                rows.append([((m >> (32 * w)) & 0xFFFFFFFF) - (
                    (1 << 32) if (m >> (32 * w + 31)) & 1 else 0) for w in range(words)])
        mask = _int32(rows)
    return {"q": q.to(_DT[case["dtype"]]), "table": table, "ctx": ctx, "nodes": nodes,
            "ctx_dev": _int32(ctx), "starts": _int32(_starts(nodes)), "mask": mask,
            "pages": pages, "scale": case["d"] ** -0.5, "gen": g}


def _fill_chunks(case, s):
    """The cache's contents, some pages at a time: (first slot, k, v)."""
    page, g = case["page"], s["gen"]
    step = max(1, (1 << 25) // (page * case["hkv"] * case["d"]))
    for p0 in range(0, s["pages"], step):
        n = min(step, s["pages"] - p0) * page
        k, v = _kv(n, case, g)
        yield p0 * page, k, v


def _verify_inputs(case, seed):
    g = _gen(seed)
    rng = random.Random(seed * 131 + 9)
    _, nodes = _counts(case)
    total, vocab = sum(nodes), case["vocab"]
    logits = 3.0 * torch.randn((total, vocab), device="cuda", generator=g)
    target = torch.softmax(logits, -1)
    parents, rows = [], []
    base = 0
    for n in nodes:
        par = _parents(n, rng) if case["tree"] else list(range(-1, n - 1))
        parents += par
        rows += [base + max(p, 0) for p in par]
        base += n
    from_row = torch.tensor(rows, device="cuda")
    s = {"target": target, "draft": None}
    if case["draft"]:
        s["draft"] = torch.softmax(
            logits + 0.7 * torch.randn((total, vocab), device="cuda", generator=g), -1)
        del logits
        tokens = torch.cat([torch.multinomial(s["draft"][r:r + 1], 1, generator=g)[0]
                            for r in rows])
    else:
        # the parent's most likely tokens, one rank further for each sibling
        seen, rank = {}, []
        for r in rows:
            rank.append(seen.get(r, 0))
            seen[r] = rank[-1] + 1
        top = torch.topk(target, min(max(rank) + 1, vocab), dim=-1).indices
        tokens = top[from_row, torch.tensor(rank, device="cuda").clamp(max=top.shape[1] - 1)]
    s["tokens"] = tokens.int()
    s["u"] = torch.rand(total, device="cuda", generator=g)
    s["r"] = torch.rand(case["b"], device="cuda", generator=g)
    s["starts"] = _int32(_starts(nodes))
    s["parents"] = _int32(parents) if case["tree"] else None
    s["parents_host"], s["nodes"] = parents, nodes
    return s


def prepare(case, seed):
    op = case["op"]
    if op == "norm_rope":
        s = _norm_rope_inputs(case, seed)
    elif op == "cache":
        s = _cache_inputs(case, seed)
        if own:
            tq = _tq()
            n = tq.cache_bytes(_ctype(case), s["pages"], case["page"], case["hkv"], case["d"])
            s["kc"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
            s["vc"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        else:
            slots = s["pages"] * case["page"]
            for c in "kv":
                s[c + "q"] = torch.zeros((slots, case["hkv"], case["d"]), dtype=torch.int8,
                                         device="cuda")
                s[c + "d"] = torch.zeros((slots, case["hkv"], case["d"] // 32),
                                         dtype=torch.float16, device="cuda")
    elif op == "attention":
        s = _attention_inputs(case, seed)
        slots = s["pages"] * case["page"]
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
    else:
        s = _verify_inputs(case, seed)
    s["case"] = case
    return s


# --------------------------------------------------------------------------
# plain forms

def _quantize(ctype, x):
    """x [.., D] -> (codes int8, fp16 scales [.., D/32]); each step in fp32."""
    b = x.float().nan_to_num(nan=0.0, posinf=_LIMIT, neginf=-_LIMIT)
    b = b.clamp(-_LIMIT, _LIMIT).unflatten(-1, (-1, 32))
    if ctype == "q8_0":
        d = b.abs().amax(-1, keepdim=True)
        d = d / torch.full_like(d, 127.0)
        inv = torch.where(d != 0, torch.ones_like(d) / d, torch.zeros_like(d))
        y = b * inv
        # nearest whole number, halves away from zero
        n = y.abs().floor()
        n = n + (y.abs() - n >= 0.5)
        q = torch.copysign(n, y)
    else:
        far = b.abs().argmax(-1, keepdim=True)        # the first of the largest
        d = b.gather(-1, far) * -0.125
        inv = torch.where(d != 0, torch.ones_like(d) / d, torch.zeros_like(d))
        q = (b * inv + 8.5).floor().clamp(0, 15) - 8
    return q.to(torch.int8).flatten(-2), d.squeeze(-1).half()


def _values(q, d):
    return (q.unflatten(-1, (-1, 32)).float() * d.float().unsqueeze(-1)).flatten(-2)


def _plain_norm_rope(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    angle = s["pos"].double()[:, None] * s["freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        if case["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:rot]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        out.append(torch.cat((turned, y[..., rot:]), -1).to(x.dtype))
    return out


def _plain_cache(s):
    case, slots = s["case"], s["slots"].long()
    out = []
    for c in "kv":
        q, d = _quantize(case["ctype"], s[c])
        s[c + "q"][slots] = q
        s[c + "d"][slots] = d
        out.append(_values(s[c + "q"][slots], s[c + "d"][slots]).to(s[c].dtype))
    return out


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    out = torch.empty_like(s["q"])
    row = 0
    for b, (ctx, n) in enumerate(zip(s["ctx"], s["nodes"])):
        pos = torch.arange(ctx + n, device="cuda")
        slots = s["table"][b, pos // page].long() * page + pos % page
        k = _values(s["kq"][slots], s["kd"][slots]).transpose(0, 1)     # [hkv, keys, d]
        v = _values(s["vq"][slots], s["vd"][slots]).transpose(0, 1)
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
    return out


def _plain_verify(s):
    """One sweep over the nodes in order, all sequences at once: node i is
    tried where its parent is the node reached so far."""
    case = s["case"]
    b, width, vocab = case["b"], case["nodes"], case["vocab"]
    starts = s["starts"].long()
    first, count = starts[:-1], starts[1:] - starts[:-1]
    seq = torch.arange(b, device="cuda")
    cur = torch.zeros(b, dtype=torch.long, device="cuda")
    taken = torch.zeros(b, dtype=torch.long, device="cuda")
    nodes = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    tokens = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    chain, draft = s["parents"] is None, s["draft"]
    one = torch.ones(b, dtype=torch.float64, device="cuda")
    a, c, left = one.clone(), torch.zeros_like(one), one.clone()
    gone = torch.zeros((b, vocab), dtype=torch.bool, device="cuda") if draft is None else None
    last = s["target"].shape[0] - 1
    for i in range(1, width):
        at = (first + i).clamp(max=last)
        parent = torch.full_like(cur, i - 1) if chain else s["parents"][at].long()
        trying = (i < count) & (parent == cur)
        x, u = s["tokens"][at].long(), s["u"][at].double()
        p = s["target"][first + cur, x].double()
        if draft is None:
            p = p.masked_fill(gone[seq, x], 0.0)
            good = trying & (u * left < p)
            bad = trying & ~good
            left = torch.where(bad, left - p, left)
            gone[seq, x] |= bad
            left = torch.where(good, one, left)
            gone &= ~good[:, None]
        else:
            q = draft[first + cur, x].double()
            good = trying & (u * q < (a * p - c * q).clamp(min=0))
            bad = trying & ~good
            rows = first + cur
            z = (a[:, None] * s["target"][rows].double()
                 - (c + 1)[:, None] * draft[rows].double()).clamp(min=0).sum(-1)
            bad = bad & (z > 0)
            a, c = (torch.where(bad, a / z, torch.where(good, one, a)),
                    torch.where(bad, (c + 1) / z, torch.where(good, 0 * one, c)))
        w = taken.clamp(max=width - 1)
        nodes[seq, w] = torch.where(good, torch.full_like(w, i).int(), nodes[seq, w])
        tokens[seq, w] = torch.where(good, x.int(), tokens[seq, w])
        cur = torch.where(good, torch.full_like(cur, i), cur)
        taken = taken + good
    rows = first + cur
    if draft is None:
        weight = s["target"][rows].double().masked_fill(gone, 0.0)
    else:
        weight = (a[:, None] * s["target"][rows].double()
                  - c[:, None] * draft[rows].double()).clamp(min=0)
    cdf = weight.cumsum(-1)
    hit = cdf > (s["r"].double() * cdf[:, -1])[:, None]
    tokens[seq, taken] = hit.int().argmax(-1).int()
    return [taken.int(), tokens, nodes]


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"norm_rope": _plain_norm_rope, "cache": _plain_cache,
                "attention": _plain_attention, "verify": _plain_verify}[op](state)
    tq = _tq()
    if op == "norm_rope":
        return list(tq.qk_norm_rope(state["q"], state["k"], state["pos"], state["freq"],
                                    state["wq"], state["wk"], eps=1e-6,
                                    interleaved=case["interleaved"]))
    if op == "cache":
        tq.cache_write(_ctype(case), state["k"], state["v"], state["kc"], state["vc"],
                       state["slots"], case["page"])
        return list(tq.cache_read(_ctype(case), state["kc"], state["vc"], state["slots"],
                                  case["hkv"], case["d"], case["page"],
                                  dtype=state["k"].dtype))
    if op == "attention":
        return tq.tree_attention(_ctype(case), state["q"], state["kc"], state["vc"],
                                 state["table"], state["ctx_dev"], state["starts"],
                                 case["hkv"], case["page"], max_nodes=case["nodes"],
                                 max_ctx=case["ctx"], scale=state["scale"],
                                 mask=state["mask"])
    return list(tq.verify_draft(state["target"], state["tokens"], state["starts"], state["u"],
                                state["r"], draft=state["draft"], parents=state["parents"],
                                max_nodes=case["nodes"]))


# --------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "norm_rope":
        size = torch.finfo(_DT[case["dtype"]]).bits // 8
        n = case["t"] * (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": 2 * n * size + 4 * case["t"], "flops": 9 * n}
    if op == "cache":
        size = torch.finfo(_DT[case["dtype"]]).bits // 8
        n = 2 * case["t"] * case["hkv"] * case["d"]
        block = 34 if case["ctype"] == "q8_0" else 18
        # read, stored as blocks; the blocks read again, written out
        return {"bytes": 2 * n * size + 2 * (n // 32) * block + 8 * case["t"], "flops": 6 * n}
    if op == "attention":
        ctx, nodes = _counts(case)
        block = 34 if case["ctype"] == "q8_0" else 18
        keys = sum(c + n for c, n in zip(ctx, nodes))
        pairs = sum(n * (c + n) for c, n in zip(ctx, nodes))
        return {"bytes": 2 * keys * case["hkv"] * (case["d"] // 32) * block
                + 4 * sum(nodes) * case["hq"] * case["d"],
                "flops": 4 * pairs * case["hq"] * case["d"]}
    # two numbers a drafted token, and the rows that the last token is drawn from
    _, nodes = _counts(case)
    rows = case["b"] * (2 if case["draft"] else 1)
    return {"bytes": 4 * rows * case["vocab"] + 20 * sum(nodes),
            "flops": 3 * rows * case["vocab"]}


# --------------------------------------------------------------------------
# the definitions in 64 bits

def _f32(x):
    """A 64-bit value rounded to the 32-bit grid, where a definition says so."""
    return x.float().double()


def _exact_blocks(ctype, x):
    """Values of the blocks that x [.., D] is stored as.  The formats define
    their codes by 32-bit steps: the scale, its reciprocal, the product."""
    x = torch.where(x.isnan(), torch.zeros_like(x), x).double()
    x = torch.minimum(torch.maximum(x, torch.full_like(x, -_LIMIT)), torch.full_like(x, _LIMIT))
    x = x.reshape(*x.shape[:-1], -1, 32)
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


def _exact_attention(case, seed):
    s = _attention_inputs(case, seed)
    chunks = []
    for _, k, v in _fill_chunks(case, s):
        chunks.append((_exact_blocks(case["ctype"], k).float(),     # 19 bits at most: exact
                       _exact_blocks(case["ctype"], v).float()))
    kall, vall = (torch.cat([c[i] for c in chunks]) for i in (0, 1))
    del chunks
    g, page = case["hq"] // case["hkv"], case["page"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (ctx, n) in enumerate(zip(s["ctx"], s["nodes"])):
        pages = s["table"][b, :(ctx + n + page - 1) // page].long()
        slots = (pages[:, None] * page + torch.arange(page, device="cuda")).flatten()[:ctx + n]
        allow = torch.ones((n, ctx + n), dtype=torch.bool, device="cuda")
        if s["mask"] is not None:
            words = s["mask"][row:row + n].long() & 0xFFFFFFFF
            for j in range(n):
                allow[:, ctx + j] = (words[:, j // 32] >> (j % 32)) % 2 == 1
        for h in range(case["hq"]):
            k, v = kall[slots, h // g].double(), vall[slots, h // g].double()
            e = (s["q"][row:row + n, h].double() @ k.t()) * s["scale"]
            e = torch.where(allow, e, torch.full_like(e, -math.inf))
            out[row:row + n, h] = torch.softmax(e, -1) @ v
        row += n
    return out


def _exact_verify(case, seed):
    s = _verify_inputs(case, seed)
    u, r = s["u"].double().tolist(), s["r"].double().tolist()
    tok, base = s["tokens"].tolist(), 0
    width, b = case["nodes"], case["b"]
    taken = torch.zeros(b, dtype=torch.int32)
    tokens = torch.full((b, width), -1, dtype=torch.int32)
    path = torch.full((b, width), -1, dtype=torch.int32)
    for i, n in enumerate(s["nodes"]):
        par = s["parents_host"][base:base + n]
        at, k = 0, 0
        while True:
            w = s["target"][base + at].double()
            q = s["draft"][base + at].double() if case["draft"] else None
            left, go = 1.0, None
            for c in (c for c in range(at + 1, n) if par[c] == at):
                x = tok[base + c]
                p = float(w[x])
                if q is None:
                    if u[base + c] * left < p:
                        go = c
                        break
                    left -= p
                    w = w.clone()
                    w[x] = 0.0
                else:
                    if u[base + c] * float(q[x]) < p:
                        go = c
                        break
                    rest = torch.relu(w - q)
                    if float(rest.sum()) > 0:
                        w = rest / rest.sum()
            if go is None:
                break
            at = go
            path[i, k], tokens[i, k] = go, tok[base + go]
            k += 1
        cdf = torch.cumsum(w, 0)
        tokens[i, k] = int((cdf <= r[i] * float(cdf[-1])).sum())
        taken[i] = k
        base += n
    return [taken.cuda(), tokens.cuda(), path.cuda()]


def exact(case, seed):
    op = case["op"]
    if op == "norm_rope":
        s = _norm_rope_inputs(case, seed)
        half, out = case["rot"] // 2, []
        turn = torch.polar(torch.ones((case["t"], half), dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * s["freq"].double())[:, None]
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            y = x.double()
            if w is not None:
                y = y * w.double() / torch.sqrt(y.square().sum(-1, keepdim=True) / case["d"]
                                                + 1e-6)
            z = y[..., :case["rot"]]
            z = z.unflatten(-1, (half, 2)) if case["interleaved"] else \
                z.unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z if case["interleaved"] else z.transpose(-1, -2)
            out.append(torch.cat((z.flatten(-2), y[..., case["rot"]:]), -1))
        return out
    if op == "cache":
        s = _cache_inputs(case, seed)
        return [_exact_blocks(case["ctype"], s[c]) for c in "kv"]
    if op == "attention":
        return _exact_attention(case, seed)
    return _exact_verify(case, seed)
