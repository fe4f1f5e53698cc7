"""fp64 references of cross attention, of the norm and rotation of queries and keys, and of gradient clipping, with
error bounds; each returns {output: (value, bound)}, fp64 tensors on the CPU, for linear_ref.check.

What a bound counts: the rounding of the output (half a step of its type); fp32 arithmetic as (number of roundings) x
2^-24 x (sum of the magnitudes that enter); a tensor-core product as 2^-23 of the magnitudes for every 16 terms (its sums
may drop up to a unit); with bf16 the rounding of each weight and of each dS by half a step, 2^-8 of itself.
"""
import math

import numpy as np
import torch

from linear_ref import U32, d, half_step

TC = 2.0 ** -23


def cuts(off, n):
    return [0, n] if off is None else [int(x) for x in off.cpu()]


def _dot(a, b, f32):
    """Error of the products <a_i, b_j> of [h][n][c] and [h][m][c]."""
    c = a.shape[-1]
    mag = a.abs() @ b.abs().transpose(-1, -2)
    return mag * ((c + 4) * U32 if f32 else (math.ceil(c / 16) + 2) * TC)


def _pieces(q, k, q_off, kv_off):
    cq, ck = cuts(q_off, q.shape[0]), cuts(kv_off, k.shape[0])
    return list(zip(cq[:-1], cq[1:], ck[:-1], ck[1:]))


def _heads(t, a, b, share=1):
    return d(t[a:b]).transpose(0, 1).repeat_interleave(share, 0)


def attn_fwd(q, k, v, q_off=None, kv_off=None, mask=None, scale=None):
    f32, h, nq, c = q.dtype == torch.float32, q.shape[1], q.shape[0], q.shape[2]
    share, scale = h // k.shape[1], 1.0 / math.sqrt(c) if scale is None else scale
    o, bo = torch.zeros(nq, h, c, dtype=torch.float64), torch.zeros(nq, h, c, dtype=torch.float64)
    lse, bl = torch.full((h, nq), -math.inf, dtype=torch.float64), torch.zeros(h, nq, dtype=torch.float64)
    for a, b, ka, kb in _pieces(q, k, q_off, kv_off):
        seen = torch.ones(kb - ka, dtype=torch.bool) if mask is None else mask[ka:kb].cpu().bool()
        if not seen.any() or a == b:
            continue
        qs, ks, vs = _heads(q, a, b), _heads(k, ka, kb, share)[:, seen], _heads(v, ka, kb, share)[:, seen]
        n = ks.shape[1]
        s = scale * qs @ ks.transpose(1, 2)
        top = s.amax(-1, keepdim=True)
        # the exponent: the product's error, the rounding of s c - base c (both factors of c counted), ex2 itself
        e = scale * _dot(qs, ks, f32) + 4 * U32 * (s.abs() + top.abs()) + 4 * U32
        p = torch.softmax(s, -1)
        out = p @ vs
        w = e + (0.0 if f32 else half_step(torch.bfloat16))
        # sums over n keys; the joins of parts and the raised bases add a few roundings each
        steps = (n + 80) * U32 if f32 else (math.ceil(n / 16) + 80) * TC
        err = (p * w) @ vs.abs() + out.abs() * (p * e).sum(-1, keepdim=True) + steps * (p @ vs.abs()) \
            + (n + 80) * U32 * out.abs()
        o[a:b] = out.transpose(0, 1)
        bo[a:b] = (err + (half_step(q.dtype) + U32) * out.abs()).transpose(0, 1)
        l = torch.logsumexp(s, -1)
        lse[:, a:b] = l
        bl[:, a:b] = (p * e).sum(-1) + (n + 80) * U32 + 4 * U32 * (l.abs() + top[..., 0].abs())
    return {"o": (o, bo), "lse": (lse, bl)}


def attn_bwd(q, k, v, o, do, lse, q_off=None, kv_off=None, mask=None, scale=None):
    f32, h, hk, c = q.dtype == torch.float32, q.shape[1], k.shape[1], q.shape[2]
    share, scale = h // hk, 1.0 / math.sqrt(c) if scale is None else scale
    half = 0.0 if f32 else half_step(torch.bfloat16)
    z = {"dq": torch.zeros(q.shape, dtype=torch.float64), "dk": torch.zeros(k.shape, dtype=torch.float64),
         "dv": torch.zeros(k.shape, dtype=torch.float64)}
    e = {n: torch.zeros_like(t) for n, t in z.items()}
    for a, b, ka, kb in _pieces(q, k, q_off, kv_off):
        seen = torch.ones(kb - ka, dtype=torch.bool) if mask is None else mask[ka:kb].cpu().bool()
        if not seen.any() or a == b:
            continue
        at = torch.arange(ka, kb)[seen]
        qs, ds_, os = _heads(q, a, b), _heads(do, a, b), _heads(o, a, b)
        ks, vs = _heads(k, ka, kb, share)[:, seen], _heads(v, ka, kb, share)[:, seen]
        l = d(lse)[:, a:b, None]
        s = scale * qs @ ks.transpose(1, 2)
        p = torch.exp(s - l)
        ep = p * (scale * _dot(qs, ks, f32) + 4 * U32 * (s.abs() + l.abs()) + 4 * U32)
        dp = ds_ @ vs.transpose(1, 2)
        delta = (ds_ * os).sum(-1, keepdim=True)
        ed = _dot(ds_, vs, f32) + (c + 8) * U32 * (ds_ * os).abs().sum(-1, keepdim=True)
        g = p * (dp - delta)
        eg = ep * ((dp - delta).abs() + ed) + p * ed + 3 * U32 * p * (dp.abs() + delta.abs())
        ep, eg = ep + half * (p + ep), eg + half * (g.abs() + eg)
        n, m = ks.shape[1], qs.shape[1] * share

        def steps(x):
            return (x + 80) * U32 if f32 else (math.ceil(x / 16) + 80) * TC

        def add(name, rows, value, err):
            if name != "dq":
                value, err = value.unflatten(0, (hk, share)).sum(1), err.unflatten(0, (hk, share)).sum(1)
            z[name][rows] = value.transpose(0, 1)
            e[name][rows] = (err + (half_step(q.dtype) + 2 * U32) * value.abs()).transpose(0, 1)

        mag = scale * g.abs() @ ks.abs()
        add("dq", torch.arange(a, b), scale * g @ ks, scale * eg @ ks.abs() + steps(n) * mag)
        gt_, pt = g.transpose(1, 2), p.transpose(1, 2)
        add("dk", at, scale * gt_ @ qs, scale * eg.transpose(1, 2) @ qs.abs() + steps(m) * scale * gt_.abs() @ qs.abs())
        add("dv", at, pt @ ds_, ep.transpose(1, 2) @ ds_.abs() + steps(m) * pt @ ds_.abs())
    return {n: (z[n], e[n]) for n in z}


# ---------------------------------------------------------------------------- norm and rotation

_PI = np.longdouble("3.14159265358979323846264338327950288")


def angles(pos, freq, n):
    """cos and sin of pos * freq, [n][len(freq)], the product and its remainder in extended precision."""
    p = np.arange(n) if pos is None else pos.cpu().numpy()
    a = p.astype(np.longdouble)[:, None] * freq.cpu().numpy().astype(np.longdouble)[None, :]
    a = (a - np.round(a / (2 * _PI)) * 2 * _PI).astype(np.float64)
    return torch.from_numpy(np.cos(a)), torch.from_numpy(np.sin(a))


def turn(t, pos, freq, pairs, back=False):
    """R t, or R^T t, of t [n][h][c] in fp64"""
    if freq is None:
        return t.clone()
    c, s = (x[:, None] for x in angles(pos, freq, t.shape[0]))
    s = -s if back else s
    rot = 2 * freq.numel()
    a, b = (t[..., 0:rot:2], t[..., 1:rot:2]) if pairs else (t[..., :rot // 2], t[..., rot // 2:rot])
    out = t.clone()
    x, y = a * c - b * s, a * s + b * c
    if pairs:
        out[..., 0:rot:2], out[..., 1:rot:2] = x, y
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = x, y
    return out


def _pair_size(t, freq, pairs):
    """|a| + |b| of each channel's pair (twice |t| past the turning channels)"""
    rot = 0 if freq is None else 2 * freq.numel()
    out = 2 * t.abs()
    if rot:
        a, b = (t[..., 0:rot:2], t[..., 1:rot:2]) if pairs else (t[..., :rot // 2], t[..., rot // 2:rot])
        m = a.abs() + b.abs()
        if pairs:
            out[..., 0:rot:2], out[..., 1:rot:2] = m, m
        else:
            out[..., :rot // 2], out[..., rot // 2:rot] = m, m
    return out


# cos and sin are 6 x 2^-24 off: the angle in turns is rounded (half a step of at most half a turn), the functions are 2 units
_TURN = 9 * U32       # with the two products and the sum of a turn


def qk_fwd(x, gain, freq, pos, pairs, eps, out_dtype):
    xd, g, c = d(x), d(gain), x.shape[-1]
    r = ((xd * xd).mean(-1, keepdim=True) + eps) ** -0.5
    w = xd * r * g
    ew = ((c + 4) / 2 + 6) * U32 * w.abs()
    y = turn(w, pos, freq, pairs)
    return {"y": (y, _pair_size(w, freq, pairs) * _TURN + _pair_size(ew, freq, pairs) + (half_step(out_dtype) + U32) * y.abs())}


def qk_bwd(dy, x, gain, freq, pos, pairs, eps):
    xd, gd, c = d(x), d(gain), x.shape[-1]
    n = x.shape[0] * x.shape[1]
    r = ((xd * xd).mean(-1, keepdim=True) + eps) ** -0.5
    er = ((c + 4) / 2 + 6) * U32
    g = turn(d(dy), pos, freq, pairs, back=True)
    eg = _pair_size(d(dy), freq, pairs) * _TURN
    w, ew = gd * g, gd.abs() * eg + U32 * (gd * g).abs()
    dot = (w * xd).sum(-1, keepdim=True)
    edot = (ew * xd.abs()).sum(-1, keepdim=True) + (c + 4) * U32 * (w * xd).abs().sum(-1, keepdim=True)
    back = xd * r * r * dot / c
    eback = back.abs() * (2 * er + 8 * U32) + xd.abs() * r * r * edot / c
    dx = r * (w - back)
    edx = r * (ew + eback + 2 * U32 * (w.abs() + back.abs())) + (er + 2 * U32) * dx.abs()
    part = g * xd * r
    epart = eg * xd.abs() * r + part.abs() * (er + 3 * U32)
    dg = part.sum((0, 1))
    # a thread adds its share of the heads, then come at most 256 groups, 32 x 19 partial rows
    adds = n / 64 + 1024
    return {"dx": (dx, edx + (half_step(x.dtype) + U32) * dx.abs()),
            "dgain": (dg, epart.sum((0, 1)) + adds * U32 * part.abs().sum((0, 1)))}


# ---------------------------------------------------------------------------- clipping

def clip(grads, max_norm, out_dtypes):
    """A lane adds 64 squares in four chains of 16; what follows is fp64: 20 roundings of positive terms, halved by the
    root, and that of the norm; the factor's and the product's."""
    total = math.fsum(float((d(g) ** 2).sum()) for g in grads)
    norm = math.sqrt(total)
    factor = 1.0 if norm <= max_norm or math.isinf(max_norm) else max_norm / norm
    ref = {"norm": (torch.tensor([norm], dtype=torch.float64), torch.tensor([norm * 12 * U32], dtype=torch.float64))}
    for i, (g, t) in enumerate(zip(grads, out_dtypes)):
        v = d(g) * factor
        off = half_step(t) + U32 + (0.0 if factor == 1.0 else 14 * U32)
        ref[f"out{i}"] = (v, v.abs() * off)
    return ref
