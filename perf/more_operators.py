"""Timed cases of cross attention, the norm and rotation of queries and keys, and gradient clipping.

    cross attention   o_i = sum_j softmax_j(scale <q_i, k_j>) v_j over the keys of query i's own sequence: queries
                      [nq][h][d], keys and values [nk][hk][d] packed one sequence after another, h / hk query heads
                      to a key head, optionally keys that no query sees (gt_cross_attn_fwd / _bwd)
    norm, rotation    y = R(pos) (gain x / sqrt(mean x^2 + eps)) of every head of the queries and keys, R turning
                      channel pairs by pos * freq (gt_qk_norm_fwd / _bwd)
    clipping          the norm of all gradients together, and min(1, max_norm / norm) times each (gt_grad_clip)

`run` makes one pass of one operator: with `own` false in a plain form (elementary torch operations in fp32,
rounded once at the end), with `own` true through the library.  `exact` gives the same outputs in fp64.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
_EPS = 1e-6


def _attn(name, op, nq, nk, h, hk, d, t, batch=1, ragged=False, mask=False, fused=False):
    return dict(name=name, op=op, nq=nq, nk=nk, h=h, hk=hk, d=d, t=t, batch=batch, ragged=ragged, mask=mask, fused=fused)


def _norm(name, op, nq, nk, h, hk, d, xt, yt, rot="halves", fused=False, far=0):
    return dict(name=name, op=op, nq=nq, nk=nk, h=h, hk=hk, d=d, x=xt, y=yt, rot=rot, fused=fused, far=far)


def _clip(name, layers, width, t, yt):
    return dict(name=name, op="clip", layers=layers, width=width, t=t, y=yt)


def listed():
    return [
        # one readout query over the 512-node fp32 graph: the smallest call, launch latency
        _attn("xattn fwd 1x512 8x8 f32", "xattn_fwd", 1, 512, 8, 8, 8, "f32"),
        # serving: the next token of each of 16 decoders over its own encoder states, four query heads to a key head
        _attn("xattn fwd 16x1 over 65536 32:8x128 bf16", "xattn_fwd", 16, 65536, 32, 8, 128, "bf16", batch=16, ragged=True),
        # a long decoder over the 32768-node graph
        _attn("xattn fwd 4096x32768 8x64 bf16", "xattn_fwd", 4096, 32768, 8, 8, 64, "bf16"),
        # readout of the 6800-node model in fp32 training: 128 learned queries
        _attn("xattn bwd 128x6800 8x8 f32", "xattn_bwd", 128, 6800, 8, 8, 8, "f32"),
        # a ragged batch of odd lengths, shared heads, keys and values as slices of one projection's rows
        _attn("xattn bwd 4099x20001 16:4x128 bf16", "xattn_bwd", 4099, 20001, 16, 4, 128, "bf16", batch=16, ragged=True,
              fused=True),
        # the long decoder over the 32768-node graph, backward
        _attn("xattn bwd 4096x32768 8x64 bf16", "xattn_bwd", 4096, 32768, 8, 8, 64, "bf16"),
        # the queries and keys of the 512-node fp32 graph: launch latency
        _norm("qk norm fwd 512 8x8 f32", "qkn_fwd", 512, 512, 8, 8, 8, "f32", "f32"),
        # a wide layer over the 32768-node graph: slices of one q | k | v projection
        _norm("qk norm fwd 32768 16:8x64 bf16", "qkn_fwd", 32768, 32768, 16, 8, 64, "bf16", "bf16", fused=True),
        # odd row counts, fewer key heads than query heads, adjacent pairs, positions far out, fp32 projections
        _norm("qk norm bwd 6801,4097 8:2x16 f32", "qkn_bwd", 6801, 4097, 8, 2, 16, "f32", "bf16", rot="pairs", far=1000000),
        # the wide layer, backward
        _norm("qk norm bwd 32768 16:8x64 bf16", "qkn_bwd", 32768, 32768, 16, 8, 64, "bf16", "bf16", fused=True),
        # all gradients of the 16-layer model of width 64: many small tensors
        _clip("clip 16 layers of 64 f32", 16, 64, "f32", "f32"),
        # eight layers of width 2048, more than the cache holds
        _clip("clip 8 layers of 2048 f32", 8, 2048, "f32", "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["xattn_fwd", "xattn_bwd", "xattn_fwd", "xattn_bwd", "qkn_fwd", "qkn_bwd", "clip"])
    if op == "clip":
        t = rng.choice(["f32", "f32", "bf16"])
        return dict(op=op, layers=_log(rng, 1, 32), width=_log(rng, 8, 700), t=t, y=rng.choice([t, "f32"]))
    hk = rng.choice([1, 2, 4, 8])
    h = hk * rng.choice([1, 1, 1, 2, 3, 4])
    if op in ("qkn_fwd", "qkn_bwd"):
        d = 2 * _log(rng, 4, 64)
        if rng.random() < 0.6:
            d = max(8, d // 8 * 8)
        n = _log(rng, 1, min(32768, max(1, 32768 * 2048 // ((h + hk) * d))))
        return dict(op=op, nq=n, nk=rng.choice([n, max(1, n // 3)]), h=h, hk=hk, d=d, x=rng.choice(["f32", "bf16"]),
                    y=rng.choice(["f32", "bf16"]), rot=rng.choice(["halves", "halves", "pairs", "none"]),
                    fused=rng.random() < 0.5, far=rng.choice([0, 0, 1000000]))
    t = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = _log(rng, 8, 128)
    if rng.random() < 0.7:
        d = max(8, d // 8 * 8)
    pairs = 2 ** 30 // (16 if t == "f32" else 1)
    nq = _log(rng, 1, 4096)
    nk = _log(rng, 1, max(1, min(32768, pairs * 8 // (nq * h * max(8, d // 8)))))
    batch = min(nq, nk, _log(rng, 1, 64))
    return dict(op=op, nq=nq, nk=nk, h=h, hk=hk, d=d, t=t, batch=batch, ragged=rng.random() < 0.6,
                mask=rng.random() < 0.3, fused=rng.random() < 0.5)


def _cuts(total, batch, ragged):
    """Where the sequences begin and end: equal shares, or shares between 1/4 and 7/4 of the mean; none is empty."""
    weight = [0.25 + 1.5 * (0.618034 * (b + 1) % 1.0) if ragged else 1.0 for b in range(batch)]
    cuts, run_sum, whole = [0], 0.0, sum(weight)
    for b in range(batch):
        run_sum += weight[b]
        cuts.append(b + 1 + int((total - batch) * run_sum / whole + 0.5))
    cuts[-1] = total
    return cuts


def _grad_shapes(layers, width):
    """The weights of `layers` encoder layers: two norms, q | k | v, output and the two FFN products, with biases."""
    w = width
    return [(w,), (w,), (w, 3 * w), (3 * w,), (w, w), (w,), (w,), (w,), (w, 4 * w), (4 * w,), (4 * w, w), (w,)] * layers


def _numel(shape):
    return shape[0] * (shape[1] if len(shape) > 1 else 1)


def _places(case):
    """The pieces' first elements in the flat buffer, and its size."""
    at = [0]
    for shape in _grad_shapes(case["layers"], case["width"]):
        at.append(at[-1] + (_numel(shape) + 63) // 64 * 64)
    return at


def _pieces(flat, grads, case):
    return [flat[at:at + t.numel()].view(t.shape) for at, t in zip(_places(case), grads)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype="f32", std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(_DT[dtype])

    s = {"case": case}
    if case["op"] == "clip":
        # gradients of different size from weight to weight, together well above the limit of 1; the results are
        # pieces of one flat buffer, as an optimiser keeps it, each from a multiple of 64 elements on
        s["grads"] = [normal(*shape, dtype=case["t"], std=0.01 * (1 + i % 7)) for i, shape in
                      enumerate(_grad_shapes(case["layers"], case["width"]))]
        s["flat"] = torch.zeros(_places(case)[-1], dtype=_DT[case["y"]], device="cuda")
        s["out"] = _pieces(s["flat"], s["grads"], case)
        if own:
            import graph_transformer_attention_gb300 as gt
            s["list"] = gt.gt_tensor_list(s["grads"], s["out"])
        return s
    nq, nk, h, hk, d = case["nq"], case["nk"], case["h"], case["hk"], case["d"]
    if case["op"] in ("qkn_fwd", "qkn_bwd"):
        if case["fused"] and nq == nk:      # slices of one projection's rows q | k | v
            rows = normal(nq, (h + 2 * hk) * d, dtype=case["x"], std=2.0)
            s["q"] = rows[:, :h * d].view(nq, h, d)
            s["k"] = rows[:, h * d:(h + hk) * d].view(nk, hk, d)
        else:
            s["q"], s["k"] = normal(nq, h, d, dtype=case["x"], std=2.0), normal(nk, hk, d, dtype=case["x"], std=2.0)
        s["gq"], s["gk"] = normal(d, std=0.1, mean=1.0), normal(d, std=0.1, mean=1.0)
        if case["rot"] != "none":
            s["freq"] = (10000.0 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) * 2 / d)).float()
            s["pq"] = (torch.arange(nq, device="cuda") + case["far"]).int()
            s["pk"] = torch.randint(0, nk + case["far"], (nk,), generator=g, device="cuda").int()
        else:
            s["freq"] = s["pq"] = s["pk"] = None
        if case["op"] == "qkn_bwd":
            s["dyq"], s["dyk"] = normal(nq, h, d, dtype=case["y"]), normal(nk, hk, d, dtype=case["y"])
        return s
    # normalised queries and keys (scores of unit variance), k and v slices of one projection's rows where fused
    s["q"] = normal(nq, h, d, dtype=case["t"])
    if case["fused"]:
        rows = normal(nk, 2 * hk * d, dtype=case["t"])
        s["k"], s["v"] = rows[:, :hk * d].view(nk, hk, d), rows[:, hk * d:].view(nk, hk, d)
    else:
        s["k"], s["v"] = normal(nk, hk, d, dtype=case["t"]), normal(nk, hk, d, dtype=case["t"])
    s["cq"], s["ck"] = _cuts(nq, case["batch"], case["ragged"]), _cuts(nk, case["batch"], case["ragged"])
    one = case["batch"] == 1
    s["q_off"] = None if one else torch.tensor(s["cq"], dtype=torch.int32, device="cuda")
    s["kv_off"] = None if one else torch.tensor(s["ck"], dtype=torch.int32, device="cuda")
    s["mask"] = None
    if case["mask"]:                        # one key in ten is hidden, never a sequence's first
        s["mask"] = torch.rand(nk, generator=g, device="cuda") >= 0.1
        s["mask"][torch.tensor(s["ck"][:-1], device="cuda")] = True
    if case["op"] == "xattn_bwd":
        s["do"] = normal(nq, h, d, dtype=case["t"])
        s["o"], s["lse"] = _plain_attn_fwd(s, case)
    return s


# ------------------------------------------------------------------ plain forms

def _groups(s, case):
    """(first, past) rows of the queries and of the keys of every sequence."""
    cq, ck, b = s["cq"], s["ck"], case["batch"]
    return [(cq[i], cq[i + 1], ck[i], ck[i + 1]) for i in range(b)]


def _even(s, case):
    b = case["batch"]
    return all(c[i + 1] - c[i] == c[1] for c in (s["cq"], s["ck"]) for i in range(b))


def _rows(t, a, b, n):
    """Rows a .. b - 1, n sequences: [n][heads][rows][d] in fp32."""
    return t[a:b].float().unflatten(0, (n, -1)).transpose(1, 2)


def _plain_pieces(s, case):
    """For each piece of the batch: its rows, the number of sequences, q, k, v in fp32 with the shared heads'
    queries one after another, and the scores."""
    h, hk, d = case["h"], case["hk"], case["d"]
    pieces = [(0, case["nq"], 0, case["nk"], case["batch"])] if _even(s, case) else [p + (1,) for p in _groups(s, case)]
    for a, b, ka, kb, n in pieces:
        q = _rows(s["q"], a, b, n).reshape(n, hk, -1, d)
        k, v = _rows(s["k"], ka, kb, n), _rows(s["v"], ka, kb, n)
        x = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
        if s["mask"] is not None:
            x = x.masked_fill(~s["mask"][ka:kb].view(n, 1, 1, -1), -math.inf)
        yield a, b, ka, kb, n, q, k, v, x


def _packed(t, n, h, d):
    """[n][hk][shared heads * rows][d] as [n * rows][h][d]"""
    return t.reshape(n, h, -1, d).transpose(1, 2).reshape(-1, h, d)


def _plain_attn_fwd(s, case):
    h, d = case["h"], case["d"]
    o, lse = [], []
    for a, b, ka, kb, n, q, k, v, x in _plain_pieces(s, case):
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        z = p.sum(-1, keepdim=True)
        o.append(_packed((p @ v) / z, n, h, d))
        lse.append(_packed(m + torch.log(z), n, h, 1)[..., 0])
    return torch.cat(o).to(_DT[case["t"]]), torch.cat(lse).t().contiguous()


def _plain_attn_bwd(s, case):
    h, hk, d, scale = case["h"], case["hk"], case["d"], 1.0 / math.sqrt(case["d"])
    dq, dk, dv = [], [], []
    for a, b, ka, kb, n, q, k, v, x in _plain_pieces(s, case):
        do = _rows(s["do"], a, b, n).reshape(n, hk, -1, d)
        o = _rows(s["o"], a, b, n).reshape(n, hk, -1, d)
        lse = _rows(s["lse"].t()[..., None], a, b, n).reshape(n, hk, -1, 1)
        p = torch.exp(x - lse)
        ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
        dq.append(_packed(scale * (ds @ k), n, h, d))
        dk.append(_packed(scale * (ds.transpose(-1, -2) @ q), n, hk, d))
        dv.append(_packed(p.transpose(-1, -2) @ do, n, hk, d))
    return tuple(torch.cat(t).to(_DT[case["t"]]) for t in (dq, dk, dv))


def _plain_turn(y, pos, freq, rot, back):
    """The channel pairs of y [n][h][d] turned by pos * freq, or back; the angles in fp64 (positions may be far)."""
    if rot == "none":
        return y
    angle = pos.double()[:, None] * freq.double()
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    s = -s if back else s
    half = y.shape[-1] // 2
    a, b = (y[..., :half], y[..., half:]) if rot == "halves" else (y[..., 0::2], y[..., 1::2])
    a, b = a * c - b * s, a * s + b * c
    return torch.cat((a, b), -1) if rot == "halves" else torch.stack((a, b), -1).flatten(-2)


def _plain_norm_fwd(s, case):
    out = []
    for x, gain, pos in ((s["q"], s["gq"], s["pq"]), (s["k"], s["gk"], s["pk"])):
        x = x.float()
        r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + _EPS)
        out.append(_plain_turn(x * r * gain, pos, s["freq"], case["rot"], False).to(_DT[case["y"]]))
    return tuple(out)


def _plain_norm_bwd(s, case):
    dx, dgain = [], []
    for dy, x, gain, pos in ((s["dyq"], s["q"], s["gq"], s["pq"]), (s["dyk"], s["k"], s["gk"], s["pk"])):
        x = x.float()
        r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + _EPS)
        g = _plain_turn(dy.float(), pos, s["freq"], case["rot"], True)
        w = g * gain
        dx.append((r * (w - x * (r * r * (w * x).sum(-1, keepdim=True) / case["d"]))).to(_DT[case["x"]]))
        dgain.append((g * x * r).sum((0, 1)))
    return tuple(dx) + tuple(dgain)


def _plain_clip(s, case):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in s["grads"]:
        f = t.float()
        total = total + (f * f).sum(dtype=torch.float64)
    norm = torch.sqrt(total).float()
    factor = torch.clamp(1.0 / norm, max=1.0)
    for t, out in zip(s["grads"], s["out"]):
        out.copy_(t.float() * factor)
    return norm.reshape(1), s["flat"]


# --------------------------------------------------------------- library calls

def _own(s, case):
    import graph_transformer_attention_gb300 as gt
    op = case["op"]
    if op == "clip":
        return gt.gt_grad_clip(s["list"], 1.0), s["flat"]
    if op == "xattn_fwd":
        return gt.gt_cross_attn_fwd(s["q"], s["k"], s["v"], q_off=s["q_off"], kv_off=s["kv_off"], key_mask=s["mask"])
    if op == "xattn_bwd":
        return gt.gt_cross_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], q_off=s["q_off"],
                                    kv_off=s["kv_off"], key_mask=s["mask"])
    pairs = gt.GT_ROT_PAIRS if case["rot"] == "pairs" else gt.GT_ROT_HALVES
    if op == "qkn_fwd":
        return gt.gt_qk_norm_fwd(s["q"], s["k"], s["gq"], s["gk"], freq=s["freq"], pos_q=s["pq"], pos_k=s["pk"],
                                 pairs=pairs, eps=_EPS, out_dtype=_DT[case["y"]])
    return gt.gt_qk_norm_bwd(s["dyq"], s["dyk"], s["q"], s["k"], s["gq"], s["gk"], freq=s["freq"], pos_q=s["pq"],
                             pos_k=s["pk"], pairs=pairs, eps=_EPS)


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"xattn_fwd": _plain_attn_fwd, "xattn_bwd": _plain_attn_bwd, "qkn_fwd": _plain_norm_fwd,
            "qkn_bwd": _plain_norm_bwd, "clip": _plain_clip}[case["op"]](state, case)


# ----------------------------------------------------------------- fp64 results

def _exact_attn(s, case):
    h, hk, d = case["h"], case["hk"], case["d"]
    nq, nk, share = case["nq"], case["nk"], case["h"] // case["hk"]
    back = case["op"] == "xattn_bwd"
    f64 = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(nq, h, d, **f64), torch.zeros(h, nq, **f64)
    dq, dk, dv = torch.zeros(nq, h, d, **f64), torch.zeros(nk, hk, d, **f64), torch.zeros(nk, hk, d, **f64)
    for a, b, ka, kb in _groups(s, case):
        seen = torch.ones(kb - ka, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"][ka:kb]
        for j in range(h):
            q, k, v = s["q"][a:b, j].double(), s["k"][ka:kb, j // share].double(), s["v"][ka:kb, j // share].double()
            x = torch.einsum("ic,jc->ij", q, k) / math.sqrt(d)
            x[:, ~seen] = -math.inf
            if not back:
                lse[j, a:b] = torch.logsumexp(x, 1)
                o[a:b, j] = torch.softmax(x, 1) @ v
                continue
            do, saved = s["do"][a:b, j].double(), s["o"][a:b, j].double()
            p = x.sub_(s["lse"][j, a:b].double().unsqueeze(1)).exp_()
            dv[ka:kb, j // share] += torch.einsum("ij,ic->jc", p, do)
            dp = torch.einsum("ic,jc->ij", do, v) - torch.einsum("ic,ic->i", do, saved).unsqueeze(1)
            ds = dp.mul_(p).div_(math.sqrt(d))
            dq[a:b, j] = torch.einsum("ij,jc->ic", ds, k)
            dk[ka:kb, j // share] += torch.einsum("ij,ic->jc", ds, q)
    return (dq, dk, dv) if back else (o, lse)


def _exact_norm(s, case):
    d, rot = case["d"], case["rot"]

    def turn(n, pos, sign):
        """The turn of row i as a complex factor per pair, [n][1][d / 2]"""
        if rot == "none":
            return torch.ones(n, 1, d // 2, dtype=torch.complex128, device="cuda")
        angle = torch.outer(pos.double(), s["freq"].double())
        return torch.polar(torch.ones_like(angle), sign * angle).unsqueeze(1)

    def apply(t, z):
        if rot == "pairs":
            return torch.view_as_real(torch.view_as_complex(t.unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
        w = torch.complex(t[..., :d // 2].contiguous(), t[..., d // 2:].contiguous()) * z
        return torch.cat((w.real, w.imag), -1)

    first, second = [], []
    for side in ("q", "k"):
        x, gain, pos = s[side].double(), s["g" + side].double(), s["p" + side]
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
        if case["op"] == "qkn_fwd":
            y = x * r * gain
            first.append(y if rot == "none" else apply(y, turn(x.shape[0], pos, 1.0)))
            continue
        g = s["dy" + side].double()
        if rot != "none":
            g = apply(g, turn(x.shape[0], pos, -1.0))
        xh = x * r
        proj = torch.einsum("nhc,nhc,c->nh", g, xh, gain).unsqueeze(-1) / d
        first.append(r * (g * gain - xh * proj))
        second.append(torch.einsum("nhc,nhc->c", g, xh))
    return tuple(first + second)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(t.double()) for t in s["grads"]]))
        factor = min(1.0, 1.0 / float(norm))
        flat = torch.zeros(_places(case)[-1], dtype=torch.float64, device="cuda")
        for t, out in zip(s["grads"], _pieces(flat, s["grads"], case)):
            torch.mul(t.double(), factor, out=out)
        return norm.reshape(1), flat
    return _exact_norm(s, case) if case["op"] in ("qkn_fwd", "qkn_bwd") else _exact_attn(s, case)


def work(case):
    """Bytes: every input read once, every output written once.  Flops: the products of the attention (two forward,
    five backward); about 10 and 20 per element (norm and rotation), 3 (clipping)."""
    if case["op"] == "clip":
        n = sum(_numel(shape) for shape in _grad_shapes(case["layers"], case["width"]))
        return {"bytes": n * (_SIZE[case["t"]] + _SIZE[case["y"]]) + 4, "flops": 3 * n}
    nq, nk, h, hk, d = case["nq"], case["nk"], case["h"], case["hk"], case["d"]
    if case["op"] in ("qkn_fwd", "qkn_bwd"):
        ex, ey = _SIZE[case["x"]], _SIZE[case["y"]]
        n = (nq * h + nk * hk) * d
        rows = 8 * d + (0 if case["rot"] == "none" else 4 * (nq + nk) + 2 * d)
        if case["op"] == "qkn_fwd":
            return {"bytes": n * (ex + ey) + rows, "flops": 10 * n}
        return {"bytes": n * (2 * ex + ey) + rows + 8 * d, "flops": 20 * n}
    e = _SIZE[case["t"]]
    cq, ck = _cuts(nq, case["batch"], case["ragged"]), _cuts(nk, case["batch"], case["ragged"])
    pairs = sum((cq[b + 1] - cq[b]) * (ck[b + 1] - ck[b]) for b in range(case["batch"]))
    side = (8 * (case["batch"] + 1) if case["batch"] > 1 else 0) + (nk if case["mask"] else 0) + 4 * nq * h
    if case["op"] == "xattn_fwd":
        return {"bytes": e * d * (2 * nq * h + 2 * nk * hk) + side, "flops": 4 * pairs * h * d}
    return {"bytes": e * d * (4 * nq * h + 4 * nk * hk) + side, "flops": 10 * pairs * h * d}
