"""fp64 references of the LayerNorm and linear-layer operators with error bounds.

Each reference returns {output: (value, bound)}, both fp64 tensors on the CPU.  A bound counts:
the rounding of the output (half a step of its type, relative to the value), and fp32
arithmetic as (number of roundings) x 2^-24 x (sum of the magnitudes that enter).
"""
import math

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def d(t):
    return t.detach().cpu().double()


def ln_fwd(x, gain, shift, eps, out_dtype):
    """A sum over c features takes at most 32 additions in a thread and 5 + 16 across threads (64 counted)."""
    x, g, s = d(x), d(gain), d(shift)
    mean = x.mean(1, keepdim=True)
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    y = (x - mean) * rstd * g + s
    ax = x.abs() + x.abs().mean(1, keepdim=True)
    # the mean is off by dm; a centred square by 2 |x - mean| dm + its own rounding; 1/sqrt halves that
    dm = 64 * U32 * x.abs().mean(1, keepdim=True)
    dvar = 64 * U32 * var + 2 * dm * (x - mean).abs().mean(1, keepdim=True) + dm ** 2 + 2 * U32 * (ax * (x - mean).abs()).mean(1, keepdim=True)
    drel = 0.5 * dvar / (var + eps) + 4 * U32
    by = half_step(out_dtype) * y.abs() + g.abs() * rstd * (dm + 2 * U32 * ax) + (g * (x - mean) * rstd).abs() * drel \
        + 4 * U32 * ((g * (x - mean) * rstd).abs() + s.abs())
    return {"y": (y, by), "mean": (mean[:, 0], dm[:, 0] + U32 * mean[:, 0].abs()),
            "rstd": (rstd[:, 0], rstd[:, 0] * (drel[:, 0] + U32))}


def ln_bwd(dy, x, gain, mean, rstd, dres):
    """Column sums: a thread adds n / (row groups of the grid) rows, then at most 32 + 304 / 8 + 8 partial sums."""
    n, c = x.shape
    dyd, xd, g, mu, r = d(dy), d(x), d(gain), d(mean)[:, None], d(rstd)[:, None]
    xh = (xd - mu) * r
    axh = 3 * U32 * (xd.abs() + mu.abs()) * r.abs()          # error of xh
    dd = dyd * g
    m1, m2 = dd.mean(1, keepdim=True), (dd * xh).mean(1, keepdim=True)
    dx = r * (dd - m1 - xh * m2)
    bm1 = 64 * U32 * dd.abs().mean(1, keepdim=True)
    bm2 = 66 * U32 * (dd * xh).abs().mean(1, keepdim=True) + (dd.abs() * axh).mean(1, keepdim=True)
    bdx = r.abs() * (4 * U32 * (dd.abs() + m1.abs() + (xh * m2).abs()) + bm1 + xh.abs() * bm2 + axh * (m2.abs() + bm2))
    if dres is not None:
        dx = dx + d(dres)
        bdx = bdx + 2 * U32 * d(dres).abs()
    bdx = bdx + half_step(x.dtype) * dx.abs() + U32 * dx.abs()
    adds = n / 128 + 128
    dg, ds = (dyd * xh).sum(0), dyd.sum(0)
    return {"dx": (dx, bdx),
            "dgain": (dg, adds * U32 * (dyd * xh).abs().sum(0) + (dyd.abs() * axh).sum(0) + U32 * dg.abs()),
            "dshift": (ds, adds * U32 * dyd.abs().sum(0) + U32 * ds.abs())}


def product_bound(a, b, f32):
    """Error of a tensor-core product of |a| [m][k] and |b| [k][n]: the products of bf16 values are exact in
    fp32; every 16 of them are added to the accumulator, which may drop up to a whole unit (2^-23) of it each
    time, and 16 aligned terms with it.  fp32 operands: six such products, and three dropped terms of at most
    2^-24 of the whole each."""
    k = a.shape[1]
    mag = a.abs() @ b.abs()
    steps = math.ceil(k / 16) * (6 if f32 else 1) + 160
    return mag * (steps * 2.0 ** -23 + (3 * U32 if f32 else 0.0))


def phi(a):
    return torch.special.ndtr(a)


def gelu_slope(a):
    return phi(a) + a * torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi)


def linear_fwd(x, w, b, gelu, r, out_dtype):
    f32 = x.dtype == torch.float32
    xd, wd = d(x), d(w)
    a = xd @ wd
    ba = product_bound(xd, wd, f32)
    if b is not None:
        a = a + d(b)
    ba = ba + 2 * U32 * a.abs()
    y, by = a, ba
    if gelu:
        # |gelu'| <= 1.13; the CDF is 1.5e-7 off by its formula and a few roundings by its arithmetic
        y, by = a * phi(a), 1.13 * ba + a.abs() * (1.5e-7 + 12 * U32)
    if r is not None:
        y = y + d(r)
        by = by + U32 * d(r).abs()
    return {"y": (y, by + (U32 + half_step(out_dtype)) * y.abs()), "pre": (a, ba + half_step(x.dtype) * a.abs())}


def linear_bwd(dy, x, w, pre, gelu, add, has_bias=True):
    f32 = x.dtype == torch.float32
    xd, wd, da = d(x), d(w), d(dy)
    bda = torch.zeros_like(da)
    if gelu:
        slope = gelu_slope(d(pre))
        # slope: CDF as above, a phi(a) a few roundings
        bda = da.abs() * (1.5e-7 + 16 * U32 * (1 + d(pre).abs()))
        da = da * slope
        bda = bda + 2 * U32 * da.abs()
    m = da.shape[0]
    bdb = bda.sum(0) + (m / 128 + 128) * U32 * da.abs().sum(0)
    db = da.sum(0)
    bq = bda if f32 or (dy.dtype == torch.bfloat16 and not gelu) else bda + half_step(torch.bfloat16) * da.abs()
    dx = da @ wd.t()
    bdx = product_bound(da.abs() + bq, wd.t(), f32) + bq @ wd.t().abs()
    if add is not None:
        dx = dx + d(add)
        bdx = bdx + U32 * d(add).abs()
    dw = xd.t() @ da
    bdw = product_bound(xd.t(), da.abs() + bq, f32) + xd.t().abs() @ bq
    h = half_step(x.dtype) + U32
    return {"dx": (dx, bdx + h * dx.abs()), "dw": (dw, bdw + h * dw.abs()), "db": (db, bdb + U32 * db.abs())}


def check(got, ref, floor=1e-30):
    for name, t in got.items():
        value, bound = ref[name]
        t = d(t)
        assert t.shape == value.shape, (name, t.shape, value.shape)
        off = (t - value).abs()
        bad = ~(off <= bound + floor)
        assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                               f"{float((off / (bound + floor)).nan_to_num(nan=1e9).max()):.3g} times it")
