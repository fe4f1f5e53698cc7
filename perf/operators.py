"""Timed cases of the LayerNorm and linear-layer operators (gt_layer_norm_fwd / _bwd, gt_linear_fwd / _bwd).

    LayerNorm   y = gain (x - mean) rstd + shift, statistics over the c features of a node
    linear      y = act(x W + b) + r, x [m][k], W [k][n] (in x out), act none or GELU(a) = a Phi(a)

`run` makes one pass of one operator: with `own` false in a plain form (elementary torch operations in fp32,
rounded once at the end), with `own` true through the library.  `exact` gives the same outputs in fp64.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
_EPS = 1e-5


def _ln(name, op, n, c, xt, yt, res=False):
    return dict(name=name, op=op, n=n, c=c, x=xt, y=yt, res=res)


def _lin(name, op, m, k, n, xt, yt, act, bias=True, res=False, pre=False, pad=0):
    return dict(name=name, op=op, m=m, k=k, n=n, x=xt, y=yt, act=act, bias=bias, res=res, pre=pre, pad=pad)


def listed():
    return [
        # the 512-node fp32 graph at the width of the fused layer: the smallest training call, launch latency
        _ln("ln fwd 512x64 f32", "ln_fwd", 512, 64, "f32", "f32"),
        # a wide layer's norm over the largest graph: fp32 residual stream in, bf16 for the products out
        _ln("ln fwd 32768x1024 f32-bf16", "ln_fwd", 32768, 1024, "f32", "bf16"),
        # one layer of the 16-layer, 6800-node model: the norm's gradients, the residual's added
        _ln("ln bwd 6800x64 f32", "ln_bwd", 6800, 64, "f32", "f32", res=True),
        # the same in a wide bf16 layer of the 32768-node graph
        _ln("ln bwd 32768x1024 bf16", "ln_bwd", 32768, 1024, "bf16", "bf16", res=True),
        # one new node through the first FFN product (inference): all of W for one row
        _lin("linear fwd 1x512x2048 bf16", "lin_fwd", 1, 512, 2048, "bf16", "bf16", "gelu"),
        # the q | k | v projection of the 6800-node model in fp32
        _lin("linear fwd 6800x64x192 f32", "lin_fwd", 6800, 64, 192, "f32", "f32", "none"),
        # ragged in every size, contiguous rows that are no multiple of 16 bytes, fp32 residual stream
        _lin("linear fwd 4099x321x1001 bf16", "lin_fwd", 4099, 321, 1001, "bf16", "f32", "none", res=True),
        # first FFN product of a wide layer in training, the pre-activation kept for the backward
        _lin("linear fwd 32768x1024x4096 bf16", "lin_fwd", 32768, 1024, 4096, "bf16", "bf16", "gelu", pre=True),
        # the 512-node fp32 graph's FFN product, backward: latency
        _lin("linear bwd 512x64x64 f32", "lin_bwd", 512, 64, 64, "f32", "f32", "gelu"),
        # a fp32 layer of the 4096-node graph: output projection's gradients, added to a branch's gradient
        _lin("linear bwd 4096x512x512 f32", "lin_bwd", 4096, 512, 512, "f32", "f32", "none", res=True),
        # FFN product of a 256-wide layer over the 6800-node graph
        _lin("linear bwd 6800x256x1024 bf16", "lin_bwd", 6800, 256, 1024, "bf16", "bf16", "gelu"),
        # the wide layer's FFN product, backward
        _lin("linear bwd 32768x1024x4096 bf16", "lin_bwd", 32768, 1024, 4096, "bf16", "bf16", "gelu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "lin_fwd", "lin_bwd", "lin_fwd", "lin_bwd"])
    if op in ("ln_fwd", "ln_bwd"):
        c = _log(rng, 8, 8192)
        n = _log(rng, 1, max(1, min(65536, 32768 * 1024 // c)))
        if rng.random() < 0.5:
            c = max(8, c // 8 * 8)
        return dict(op=op, n=n, c=c, x=rng.choice(["f32", "bf16"]), y=rng.choice(["f32", "bf16"]),
                    res=op == "ln_bwd" and rng.random() < 0.5)
    xt = rng.choice(["f32", "bf16", "bf16"])
    k, n = _log(rng, 16, 4096), _log(rng, 16, 4096)
    if rng.random() < 0.6:
        k, n = max(16, k // 8 * 8), max(16, n // 8 * 8)
    most = 32768 * 1024 * 4096 // (8 if xt == "f32" else 1)
    m = _log(rng, 1, max(1, min(32768, most // (k * n))))
    act = rng.choice(["none", "gelu"])
    return dict(op=op, m=m, k=k, n=n, x=xt, y="f32" if xt == "f32" else rng.choice(["f32", "bf16"]), act=act,
                bias=rng.random() < 0.8, res=rng.random() < 0.5,
                pre=op == "lin_fwd" and act == "gelu" and rng.random() < 0.5, pad=rng.choice([0, 0, 8, 5]))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype="f32", std=1.0, mean=0.0, scale=None):
        t = torch.randn(*shape, generator=g, device="cuda") * std + mean
        return (t if scale is None else t * scale).to(_DT[dtype])

    s = {"case": case}
    if case["op"] in ("ln_fwd", "ln_bwd"):
        n, c = case["n"], case["c"]
        # a residual stream: rows of different size and offset, one feature in 32 much larger than the rest
        feature = 1.0 + 7.0 * (torch.rand(c, generator=g, device="cuda") < 1 / 32)
        row = torch.exp(0.5 * torch.randn(n, 1, generator=g, device="cuda"))
        s["x"] = normal(n, c, dtype=case["x"], mean=0.25, scale=feature * row)
        s["gain"] = normal(c, std=0.1, mean=1.0)
        if case["op"] == "ln_fwd":
            s["shift"] = normal(c, std=0.02)
            return s
        s["dy"] = normal(n, c, dtype=case["y"])
        x = s["x"].double()
        s["mean"] = x.mean(1).float()
        s["rstd"] = (1.0 / torch.sqrt(x.var(1, unbiased=False) + _EPS)).float()
        s["dres"] = normal(n, c, dtype=case["x"]) if case["res"] else None
        return s
    m, k, n = case["m"], case["k"], case["n"]
    # x: normalised activations, a slice of wider rows where pad > 0; W keeps their variance
    s["x"] = normal(m, k + case["pad"], dtype=case["x"])[:, :k]
    s["w"] = normal(k, n, dtype=case["x"], std=1.0 / math.sqrt(k))
    s["b"] = normal(n, std=0.02) if case["bias"] else None
    if case["op"] == "lin_fwd":
        s["r"] = normal(m, n, dtype=case["y"]) if case["res"] else None
        return s
    s["dy"] = normal(m, n, dtype=case["y"])
    # the saved x W + b: unit variance, as the products of these x and W have
    s["pre"] = normal(m, n, dtype=case["x"]) if case["act"] == "gelu" else None
    s["add"] = normal(m, k, dtype=case["x"]) if case["res"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _plain_ln_fwd(s, case):
    x = s["x"].float()
    mean = x.sum(1, keepdim=True) / case["c"]
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).sum(1, keepdim=True) / case["c"] + _EPS)
    y = xc * rstd * s["gain"] + s["shift"]
    return y.to(_DT[case["y"]]), mean[:, 0], rstd[:, 0]


def _plain_ln_bwd(s, case):
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    d = dy * s["gain"]
    m1 = d.sum(1, keepdim=True) / case["c"]
    m2 = (d * xh).sum(1, keepdim=True) / case["c"]
    dx = s["rstd"][:, None] * (d - m1 - xh * m2)
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dx.to(_DT[case["x"]]), (dy * xh).sum(0), dy.sum(0)


def _plain_lin_fwd(s, case):
    a = s["x"].float() @ s["w"].float()
    if s["b"] is not None:
        a = a + s["b"]
    y = 0.5 * a * (1.0 + torch.erf(a * math.sqrt(0.5))) if case["act"] == "gelu" else a
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(_DT[case["y"]]), a.to(_DT[case["x"]]) if case["pre"] else None


def _plain_lin_bwd(s, case):
    da = s["dy"].float()
    if s["pre"] is not None:
        a = s["pre"].float()
        cdf = 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5)))
        da = da * (cdf + a * torch.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi))
    dx = da @ s["w"].float().t()
    if s["add"] is not None:
        dx = dx + s["add"].float()
    dw = s["x"].float().t() @ da
    return dx.to(_DT[case["x"]]), dw.to(_DT[case["x"]]), da.sum(0) if case["bias"] else None


# --------------------------------------------------------------- library calls

def _own(s, case):
    import graph_transformer_attention_gb300 as gt
    op = case["op"]
    if op == "ln_fwd":
        return gt.gt_layer_norm_fwd(s["x"], s["gain"], s["shift"], eps=_EPS, out_dtype=_DT[case["y"]])
    if op == "ln_bwd":
        return gt.gt_layer_norm_bwd(s["dy"], s["x"], s["gain"], s["mean"], s["rstd"], dres=s["dres"])
    act = gt.GT_ACT_GELU if case["act"] == "gelu" else gt.GT_ACT_NONE
    if op == "lin_fwd":
        return gt.gt_linear_fwd(s["x"], s["w"], s["b"], act=act, r=s["r"], out_dtype=_DT[case["y"]],
                                save_pre=case["pre"])
    return gt.gt_linear_bwd(s["dy"], s["x"], s["w"], pre=s["pre"], act=act, dx_add=s["add"], need_db=case["bias"])


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd, "lin_fwd": _plain_lin_fwd,
            "lin_bwd": _plain_lin_bwd}[case["op"]](state, case)


# ----------------------------------------------------------------- fp64 results

def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "ln_fwd":
        var, mean = torch.var_mean(x, dim=1, unbiased=False)
        rstd = torch.pow(var + _EPS, -0.5)
        y = torch.addcmul(s["shift"].double(), (x - mean.unsqueeze(1)).mul(rstd.unsqueeze(1)), s["gain"].double())
        return y, mean, rstd
    if case["op"] == "ln_bwd":
        dy = s["dy"].double()
        r = s["rstd"].double().unsqueeze(1)
        xh = torch.addcmul(-s["mean"].double().unsqueeze(1) * r, x, r)
        dgain = torch.einsum("ij,ij->j", dy, xh)
        dshift = torch.einsum("ij->j", dy)
        proj = torch.einsum("ij,ij,j->i", dy, xh, s["gain"].double()).unsqueeze(1)
        flat = torch.mv(dy, s["gain"].double()).unsqueeze(1)
        dx = r * (dy * s["gain"].double() - (flat + xh * proj) / case["c"])
        return dx if s["dres"] is None else dx + s["dres"].double(), dgain, dshift
    w = s["w"].double()
    if case["op"] == "lin_fwd":
        a = torch.mm(w.t(), x.t()).t()
        if s["b"] is not None:
            a += s["b"].double()
        y = a * torch.special.ndtr(a) if case["act"] == "gelu" else a
        if s["r"] is not None:
            y = y + s["r"].double()
        return y, a if case["pre"] else None
    da = s["dy"].double()
    if s["pre"] is not None:
        a = s["pre"].double()
        da = da * (torch.special.ndtr(a) + a * torch.exp(-a.square() / 2) * (1.0 / math.sqrt(2.0 * math.pi)))
    dx = torch.mm(w, da.t()).t()
    if s["add"] is not None:
        dx = dx + s["add"].double()
    dw = torch.mm(da.t(), x).t()
    return dx, dw, torch.mv(da.t(), torch.ones(case["m"], dtype=torch.float64, device="cuda")) if case["bias"] else None


def work(case):
    """Bytes: every input read once, every output written once.  Flops: the products' (linear), about 8 and 14 per
    element (LayerNorm forward and backward)."""
    ex, ey = _SIZE[case["x"]], _SIZE[case["y"]]
    if case["op"] in ("ln_fwd", "ln_bwd"):
        n, c = case["n"], case["c"]
        if case["op"] == "ln_fwd":
            return {"bytes": n * c * (ex + ey) + 8 * n + 8 * c, "flops": 8 * n * c}
        return {"bytes": n * c * (ey + ex * (3 if case["res"] else 2)) + 8 * n + 12 * c, "flops": 14 * n * c}
    m, k, n = case["m"], case["k"], case["n"]
    bias = 4 * n if case["bias"] else 0
    if case["op"] == "lin_fwd":
        rows = ey * (2 if case["res"] else 1) + (ex if case["pre"] else 0)
        return {"bytes": ex * (m * k + k * n) + bias + rows * m * n, "flops": 2 * m * k * n}
    rows = ey + (ex if case["act"] == "gelu" else 0)
    return {"bytes": ex * (m * k * (3 if case["res"] else 2) + 2 * k * n) + rows * m * n + bias, "flops": 4 * m * k * n}
