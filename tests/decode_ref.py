"""Plain 64-bit forms of the decode-step operators, written from their
definitions (numpy / torch on the CPU), for the tests of the HIP kernels."""
import numpy as np
import torch

LIMIT = 65472.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(dtype):
    """The relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


# ---- norm and rotation ----------------------------------------------------

def norm_rope(x, w, eps, pos, freq, interleaved):
    """x [T, H, D] -> fp64; also the magnitudes |a| + |b| that an output is
    combined from."""
    x = x.double()
    D, half = x.shape[-1], len(freq)
    rot = 2 * half
    if w is not None:
        x = x * w.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    ang = pos.double()[:, None] * freq.double()
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    y, mag = x.clone(), x.abs()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


# ---- cache blocks ----------------------------------------------------------

def cache_values(kind, x):
    """fp64 values of the blocks that x [..., D] (fp32 numpy) is stored as;
    the format's own fp32 steps are taken in fp32."""
    x = np.asarray(x, np.float32)
    x = np.where(np.isnan(x), np.float32(0), np.clip(x, -LIMIT, LIMIT)).astype(np.float32)
    b = x.reshape(-1, 32)
    out = np.zeros(b.shape, np.float64)
    with np.errstate(all="ignore"):
        for i, blk in enumerate(b):
            big = blk[np.argmax(np.abs(blk))]               # the first of the largest
            d = np.float32(abs(big)) / np.float32(127) if kind == "q8_0" \
                else big * np.float32(-0.125)
            dh = np.float64(np.float16(d))
            if dh == 0.0:
                continue
            y = blk * (np.float32(1) / d)
            if kind == "q8_0":
                q = np.sign(y) * np.floor(np.abs(y.astype(np.float64)) + 0.5)
            else:
                q = np.minimum(15, np.trunc(y + np.float32(8.5))) - 8
            out[i] = dh * q
    return out.reshape(x.shape)


# ---- attention -------------------------------------------------------------

def attention(q, k, v, see, scale):
    """One sequence: q [T, Hq, D], k, v [L, Hkv, D] fp64, see [T, L] bool.
    Returns out [T, Hq, D], sum p |v| and the largest sum |q||k| * scale over
    the keys seen, [T, Hq, 1]."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    mag = torch.zeros_like(out)
    span = torch.zeros((T, Hq, 1), dtype=torch.float64)
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        s = (q[:, h].double() @ kh.T) * scale
        s = s.masked_fill(~see, float("-inf"))
        m = s.max(1, keepdim=True).values
        p = torch.where(see, torch.exp(s - torch.where(m.isinf(), torch.zeros_like(m), m)),
                        torch.zeros_like(s))
        tot = p.sum(1, keepdim=True)
        p = torch.where(tot > 0, p / tot, torch.zeros_like(p))
        out[:, h], mag[:, h] = p @ vh, p @ vh.abs()
        a = (q[:, h].double().abs() @ kh.abs().T) * scale
        span[:, h, 0] = a.masked_fill(~see, 0.0).max(1).values
    return out, mag, span


def attention_bound(out, mag, span, keys, dtype, vsum):
    """How far the kernel's output may be from `out`.  Half a step of the
    output's type; 2^-11 relative for each value (code * scale to fp16) and
    each probability; a key's rounding, 2^-11 of each |q||k| term, changes the
    exponent of its probability by at most 2^-11 * span, which moves the
    weighted mean by twice that at most; fp32 sums of `keys` terms, and the
    exponent's own fp32 error (2^-22 of its size), which enters likewise.
    Below fp16's normal numbers the errors are absolute: half a subnormal
    step, 2^-25, of a value, and of a probability that was taken times 2^10
    or more of the largest (`vsum`: sum of |v| over the keys)."""
    h = 2.0 ** -11
    rel = 2 * h + 2 * (h + 2.0 ** -21) * span + (keys + 64) * 2.0 ** -24
    return half_step(dtype) * out.abs() + rel * mag * 1.01 + 2.0 ** -25 + 2.0 ** -35 * vsum


# ---- verification ----------------------------------------------------------

def verify(target, draft, tokens, parents, u, r, width):
    """One sequence, fp64: (accepted, tokens row, nodes row)."""
    n, V = target.shape
    out_t, out_n = [-1] * width, [-1] * width
    if n == 0:
        return 0, out_t, out_n
    pos = lambda x: np.where(x > 0, x, 0.0)                 # noqa: E731
    at, k = 0, 0
    while True:
        w = pos(target[at].astype(np.float64))
        q = None if draft is None else draft[at].astype(np.float64)
        left, step = 1.0, None
        for c in range(1, n):
            x = int(tokens[c])
            par = c - 1 if parents is None else int(parents[c])
            if par != at or par >= c or x < 0 or x >= V:
                continue
            if q is None:
                if w[x] > 0 and float(u[c]) * left < w[x]:
                    step = c
                    break
                left -= w[x]
                w[x] = 0.0
            else:
                if float(u[c]) * q[x] < w[x]:
                    step = c
                    break
                rest = pos(w - q)
                if rest.sum() > 0:
                    w = rest / rest.sum()
        if step is None:
            break
        at = step
        out_n[k], out_t[k] = step, int(tokens[step])
        k += 1
    cdf = np.cumsum(w)
    hit = np.nonzero(cdf > float(r) * cdf[-1])[0]
    live = np.nonzero(w > 0)[0]
    out_t[k] = int(hit[0]) if len(hit) else (int(live[-1]) if len(live) else -1)
    return k, out_t, out_n
