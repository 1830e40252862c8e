"""Plain 64-bit forms of the serving-step operators, written from their
definitions (numpy on the CPU), for the tests of the HIP kernels."""
import numpy as np

from decode_ref import cache_values  # noqa: F401  (blocks of the cache)


def f32(x):
    return np.float32(x).astype(np.float64)


# ---- pages, positions, slots ------------------------------------------------

def plan(lens, new, owned, table, free, count, page, tokens):
    """tq_plan_step on lists; table (a numpy array) is written in place."""
    width = table.shape[1]
    count = min(max(count, 0), len(free))
    starts, pos, slot, lens_out, owned_out, taken = [0], [], [], [], [], 0
    for b, (c, n, o) in enumerate(zip(lens, new, owned)):
        c, o = max(c, 0), min(max(o, 0), width)
        n = min(max(n, 0), tokens - starts[-1])
        want = min(-(-(c + n) // page), width)
        got = 0
        for j in range(o, want):
            taken += 1
            there = taken <= count
            got += there
            table[b, j] = free[count - taken] if there else -1
        for p in range(c, c + n):
            pos.append(p)
            e = int(table[b, p // page]) if p // page < width else -1
            slot.append(e * page + p % page if e >= 0 else -1)
        starts.append(starts[-1] + n)
        lens_out.append(c + n)
        owned_out.append(o + got)
    rest = tokens - len(pos)
    return (starts, pos + [0] * rest, slot + [-1] * rest, lens_out, owned_out, [count - taken])


def release(done, owned, table, free, count):
    """tq_release_pages; table and free are written in place."""
    width = table.shape[1]
    count, out = min(max(count, 0), len(free)), []
    for b, (d, o) in enumerate(zip(done, owned)):
        o = min(max(o, 0), width)
        if d:
            for j in range(o):
                if count < len(free):
                    free[count] = table[b, j]
                    count += 1
                table[b, j] = -1
            o = 0
        out.append(o)
    return out, [count]


# ---- norms around a block ---------------------------------------------------

def rms(x, w, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def residual(y, x, post, gate, scale, eps):
    """x' before its rounding, and the size of its terms."""
    p = y if post is None else rms(y, post, eps)
    g = 1.0 if gate is None else gate
    return scale * x + g * p, np.abs(scale * x) + np.abs(g * p)


# ---- sampling ----------------------------------------------------------------

def weight_bits(vocab):
    return min(45, 62 - (vocab - 1).bit_length())


def weights(x, temp, vocab):
    """A row's weights as whole numbers (python's exp in fp64)."""
    top = np.max(x[~np.isnan(x)], initial=-np.inf)
    if top == -np.inf:
        return np.zeros(len(x), np.int64)
    with np.errstate(all="ignore"):
        z = np.where(x == top, 0.0, (x - top) / temp)
        w = np.where((x == -np.inf) | np.isnan(x), 0.0, np.exp(z))
    w = np.where(x == top, 1.0, w)
    return np.rint(w * 2.0 ** weight_bits(vocab)).astype(np.int64)


def kept(x, temp, top_k, top_p, min_p):
    """What is kept of a row's weights, int64 [V].  x fp64."""
    V = len(x)
    unit = 2.0 ** weight_bits(V)
    out = np.zeros(V, np.int64)
    x = np.where(np.isnan(x), -np.inf, x)
    if x.max() == -np.inf:
        return out
    if not temp > 0:
        out[np.argmax(x)] = 1
        return out
    w = weights(x, temp, V)
    order = np.argsort(-x, kind="stable")
    n = V
    if top_k is not None and top_k > 0:
        n = min(n, top_k)
    if top_p is not None and top_p < 1:
        ws = w[order[:n]]
        total, before, m = sum(int(v) for v in ws), 0, 0
        want = float(np.float32(top_p)) * total
        while m < n and (m == 0 or before < want):
            before += int(ws[m])
            m += 1
        n = m
    out[order[:n]] = w[order[:n]]
    if min_p is not None and min_p > 0:
        out[out < float(np.float32(min(min_p, 1.0))) * unit] = 0
    return out


def sample(w, u):
    total = int(w.sum())
    if total == 0:
        return -1
    u = min(max(float(u), 0.0), 1.0)
    thr = min(int(u * total), total - 1)
    return int(np.argmax(np.cumsum(w) > thr))


# ---- bounds of pages and their choice -----------------------------------------

def q8_codes(x):
    """Q8_0's steps in fp32 for blocks [..., n]: (codes, fp32 d)."""
    x = np.asarray(x, np.float32)
    d = (np.abs(x).max(-1, keepdims=True) / np.float32(127)).astype(np.float32)
    with np.errstate(all="ignore"):
        inv = np.where(d != 0, np.float32(1) / d, np.float32(0)).astype(np.float32)
    y = (x * inv).astype(np.float64)
    return np.sign(y) * np.floor(np.abs(y) + 0.5), d


def bounds(keys, n):
    """Codes [D/32, 2, 32] and fp16 scales of the first n keys [n, D]."""
    k = np.asarray(keys[:n], np.float64).reshape(n, -1, 32)
    both = np.concatenate((k.max(0), k.min(0)), -1)
    codes, d = q8_codes(both)
    return codes.reshape(-1, 2, 32), d[:, 0].astype(np.float16)


def score(q, codes, scale):
    """Score of one page for the query rows q [rows, D] (fp32 values)."""
    q = np.clip(np.nan_to_num(q, nan=0.0, posinf=3e38, neginf=-3e38), -3e38, 3e38)
    qb = q.reshape(len(q), -1, 32).astype(np.float32)
    c, d = q8_codes(qb)
    c = np.where(d > np.float32(2.0 ** -100), c, 0.0)
    dots = np.maximum(c * codes[None, :, 0], c * codes[None, :, 1]).sum(-1)
    s = (dots * (d[..., 0].astype(np.float64) * scale.astype(np.float64))).sum(-1)
    return np.float32(s.max())


def select(q, codes, scales, table, n_pages, ctx, T, page, first, last, keep, group, width):
    """tables [heads, width] and ctx_out of one sequence; q [T, Hq, D] fp32."""
    H = codes.shape[1]
    total = min(-(-(ctx + T) // page), len(table))
    fresh = min(ctx // page, total)
    tail = max(fresh - last, 0)
    head = min(first, tail)
    out = np.full((H, width), -1, np.int32)
    cand = list(range(head, tail))
    for h in range(H):
        pages = cand
        if keep < len(cand):
            rows = q[:, h * group:(h + 1) * group].reshape(-1, q.shape[-1])
            s = []
            for p in cand:
                e = table[p]
                s.append(-np.inf if not 0 <= e < n_pages else float(score(rows, codes[e, h], scales[e, h])))
            miss = [not 0 <= table[p] < n_pages for p in cand]
            by = sorted(range(len(cand)), key=lambda i: (miss[i], -s[i], i))[:keep]
            pages = sorted(cand[i] for i in by)
        pages = list(range(head)) + pages + list(range(tail, total))
        out[h, :len(pages)] = [table[p] for p in pages]
    return out, ctx - page * (len(cand) - min(keep, len(cand)))
