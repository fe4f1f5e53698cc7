"""Norm and rotation of queries and keys on the GPU against fp64, within derived bounds."""
import math

import pytest
import torch

import cross_ref as X
import linear_ref as R

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def gt():
    import graph_transformer_attention_gb300 as m
    from graph_transformer_attention_gb300 import build
    build.build()
    m.load_library()
    return m


def _t(shape, dtype, seed, std=1.5, mean=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _gain(c, seed):
    return _t((c,), F, seed, 0.2, 1.0)


def _freq(rot):
    return None if rot == 0 else (10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)).float()


def _both(gt, q, k, gq, gk, freq, pq, pk, pairs, yt):
    """Forward and backward against the reference."""
    yq, yk = gt.gt_qk_norm_fwd(q, k, gq, gk, freq=freq, pos_q=pq, pos_k=pk, pairs=pairs, eps=EPS, out_dtype=yt)
    R.check({"y": yq}, X.qk_fwd(q, gq, freq, pq, pairs, EPS, yt))
    dyq = _t(yq.shape, yt, 91)
    dyk = None if k is None else _t(yk.shape, yt, 92)
    dq, dk, dgq, dgk = gt.gt_qk_norm_bwd(dyq, dyk, q, k, gq, gk, freq=freq, pos_q=pq, pos_k=pk, pairs=pairs, eps=EPS)
    R.check({"dx": dq, "dgain": dgq}, X.qk_bwd(dyq, q, gq, freq, pq, pairs, EPS))
    if k is None:
        assert yk is None and dk is None and dgk is None
        return
    R.check({"y": yk}, X.qk_fwd(k, gk, freq, pk, pairs, EPS, yt))
    R.check({"dx": dk, "dgain": dgk}, X.qk_bwd(dyk, k, gk, freq, pk, pairs, EPS))
    again = gt.gt_qk_norm_bwd(dyq, dyk, q, k, gq, gk, freq=freq, pos_q=pq, pos_k=pk, pairs=pairs, eps=EPS)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dgq, dgk), again))


SHAPES = [(1, 1, 1, 1, 8), (1, 5, 8, 2, 64), (37, 19, 3, 1, 16), (300, 300, 8, 8, 8), (65, 7, 4, 2, 128), (33, 40, 2, 2, 96),
          (20, 20, 5, 5, 24), (11, 13, 2, 1, 256), (700, 90, 8, 4, 32), (9, 9, 2, 2, 6), (17, 5, 3, 3, 62), (8, 3, 2, 1, 130)]


@pytest.mark.parametrize("xt,yt", [(F, F), (F, B), (B, F), (B, B)])
@pytest.mark.parametrize("nq,nk,h,hk,c", SHAPES)
def test_forward_and_backward(gt, nq, nk, h, hk, c, xt, yt):
    q, k, gq, gk = _t((nq, h, c), xt, 1), _t((nk, hk, c), xt, 2), _gain(c, 3), _gain(c, 4)
    pq = torch.arange(nq, device="cuda", dtype=torch.int32) * 7 - 3
    for rot, pairs in ((c, 0), (c, 1), (0, 0)):
        _both(gt, q, k, gq, gk, _freq(rot), pq if rot else None, None, pairs, yt)


@pytest.mark.parametrize("c,rot", [(64, 32), (64, 2), (7, 4), (65, 64), (33, 0), (1, 0), (255, 30), (128, 96), (3, 2)])
@pytest.mark.parametrize("t", [F, B])
def test_some_channels_turn(gt, c, rot, t):
    q, k = _t((29, 3, c), t, 1), _t((31, 1, c), t, 2)
    for pairs in (0, 1):
        _both(gt, q, k, _gain(c, 3), _gain(c, 4), _freq(rot), None, None, pairs, t)
    _both(gt, q, None, _gain(c, 3), None, _freq(rot), None, None, 0, t)


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("c", [16, 64, 100])
def test_strides_and_alignment(gt, c, t):
    """Slices of a fused projection, heads first, a row that starts at any element; the rest of an output as it was."""
    n, h, hk = 45, 4, 2
    fused = _t((n, (h + 2 * hk) * c + 8), t, 1)
    q, k = fused[:, :h * c].view(n, h, c), fused[:, h * c:(h + hk) * c].view(n, hk, c)
    gq, gk = _gain(c + 1, 3)[1:], _gain(c, 4)
    _both(gt, q, k, gq.contiguous(), gk, _freq(c), None, None, 0, t)
    odd = _t((n, h * c + 1), t, 5)[:, 1:].unflatten(1, (h, c))
    first = _t((hk, n, c), t, 6).transpose(0, 1)
    _both(gt, odd, first, gk, gk, _freq(c), None, None, 1, t)
    wide = torch.full((n, h * c + 3), 7.0, dtype=t, device="cuda")
    out = wide[:, 1:1 + h * c].unflatten(1, (h, c))
    y, _ = gt.gt_qk_norm_fwd(q, None, gk, freq=_freq(c), out_q=out)
    R.check({"y": y}, X.qk_fwd(q, gk, _freq(c), None, 0, EPS, t))
    assert y is out and (wide[:, 0] == 7).all() and (wide[:, 1 + h * c:] == 7).all()


@pytest.mark.parametrize("c", [8, 64, 70])
@pytest.mark.parametrize("t", [F, B])
def test_in_place(gt, c, t):
    q, k, g, f = _t((130, 4, c), t, 1), _t((50, 2, c), t, 2), _gain(c, 3), _freq(c)
    yq, yk = gt.gt_qk_norm_fwd(q, k, g, g, freq=f)
    a, b = q.clone(), k.clone()
    assert gt.gt_qk_norm_fwd(a, b, g, g, freq=f, out_q=a, out_k=b)[0] is a
    assert torch.equal(a, yq) and torch.equal(b, yk)
    dyq, dyk = _t(q.shape, t, 5), _t(k.shape, t, 6)
    want = gt.gt_qk_norm_bwd(dyq, dyk, q, k, g, g, freq=f)
    got = gt.gt_qk_norm_bwd(dyq, dyk, q, k, g, g, freq=f, dq=dyq, dk=dyk)
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_positions_far_out(gt):
    """Angles of any int32 position, and frequencies from tiny to large, negative ones too."""
    pos = torch.tensor([0, 1, -1, 2, 100, 65535, 10 ** 6, -10 ** 6, 123456789, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1],
                       dtype=torch.int32, device="cuda")
    freq = torch.tensor([1.0, 0.5, 3.14159274, 1e-4, 2.3e-7, 1e-12, 1e-30, 1e-42, 7.77, 1e6, -0.3, 12345678.0, 0.0, 1.9e-8, 6.2831855,
                         1.5e7], device="cuda")
    c = 2 * freq.numel()
    x, g = _t((pos.numel(), 2, c), F, 1), _gain(c, 2)
    for pairs in (0, 1):
        y, _ = gt.gt_qk_norm_fwd(x, None, g, freq=freq, pos_q=pos, pairs=pairs, eps=EPS)
        R.check({"y": y}, X.qk_fwd(x, g, freq, pos, pairs, EPS, F))
    bad = freq.clone()
    bad[3] = math.inf
    y, _ = gt.gt_qk_norm_fwd(x, None, g, freq=bad, pos_q=pos, eps=EPS)
    hit = [3, 3 + c // 2]
    assert y[..., hit].isnan().all() and not y[..., [i for i in range(c) if i not in hit]].isnan().any()


def test_zero_and_nonfinite_rows(gt):
    x, g = _t((12, 2, 40), F, 1), _gain(40, 2)
    x[3] = 0.0
    x[5, 1, 7] = math.nan
    y, _ = gt.gt_qk_norm_fwd(x, None, g, freq=_freq(40), eps=EPS)
    assert (y[3] == 0).all() and y[5, 1].isnan().all()
    y[5, 1] = 0.0
    assert y.isfinite().all()
    dx = gt.gt_qk_norm_bwd(_t(x.shape, F, 3), None, x, None, g, freq=_freq(40), eps=EPS)[0]
    assert dx[5, 1].isnan().all() and dx[3].isfinite().all()
    dx[5, 1] = 0.0
    assert dx.isfinite().all()


@pytest.mark.parametrize("t", [F, B])
def test_many_rows(gt, t):
    """More rows than one turn of the backward's grid."""
    for n, h, hk, c in ((20000, 4, 4, 16), (9000, 8, 1, 64), (30011, 1, 1, 6)):
        _both(gt, _t((n, h, c), t, 1), _t((n, hk, c), t, 2), _gain(c, 3), _gain(c, 4), _freq(c), None, None, 0, t)


def test_offsets_past_32_bits(gt):
    """More than 2^31 elements: the last rows equal those of a call for them alone."""
    n, h, c, tail = 70001, 240, 128, 50
    x, g, f = _t((n, h, c), B, 1), _gain(c, 2), _freq(c)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    y, _ = gt.gt_qk_norm_fwd(x, None, g, freq=f)
    part, _ = gt.gt_qk_norm_fwd(x[-tail:], None, g, freq=f, pos_q=pos[-tail:].contiguous())
    assert torch.equal(y[-tail:], part)
    dx = gt.gt_qk_norm_bwd(y, None, x, None, g, freq=f)[0]
    part = gt.gt_qk_norm_bwd(y[-tail:], None, x[-tail:], None, g, freq=f, pos_q=pos[-tail:].contiguous())[0]
    assert torch.equal(dx[-tail:], part)


def test_gradients_by_differences(gt):
    q, k, gq, gk = _t((5, 2, 12), F, 1), _t((4, 1, 12), F, 2), _gain(12, 3), _gain(12, 4)
    f, wq, wk = _freq(8), _t((5, 2, 12), F, 5), _t((4, 1, 12), F, 6)

    def loss(q, k, gq, gk):
        return sum(float((X.turn(R.d(x) * ((R.d(x) ** 2).mean(-1, keepdim=True) + EPS) ** -0.5 * R.d(g), None, f, 0) * R.d(w)).sum())
                   for x, g, w in ((q, gq, wq), (k, gk, wk)))

    grads = gt.gt_qk_norm_bwd(wq, wk, q, k, gq, gk, freq=f, eps=EPS)
    args = [t.double() for t in (q, k, gq, gk)]
    for i, got in enumerate(grads):
        for at in range(0, args[i].numel(), 7):
            up, down = ([t.clone() for t in args] for _ in range(2))
            up[i].view(-1)[at] += 1e-5
            down[i].view(-1)[at] -= 1e-5
            want = (loss(*up) - loss(*down)) / 2e-5
            # the difference's own error: third derivatives x 1e-10, fp64 rounding / 1e-5
            assert abs(float(got.view(-1)[at]) - want) <= 2e-5 * max(1.0, abs(want)), (i, at)


def test_streams_and_graphs(gt):
    q, k, g, f = _t((200, 4, 64), B, 1), _t((90, 2, 64), B, 2), _gain(64, 3), _freq(64)
    dyq, dyk = _t(q.shape, B, 4), _t(k.shape, B, 5)
    want = (*gt.gt_qk_norm_fwd(q, k, g, g, freq=f), *gt.gt_qk_norm_bwd(dyq, dyk, q, k, g, g, freq=f))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*gt.gt_qk_norm_fwd(q, k, g, g, freq=f, stream=side), *gt.gt_qk_norm_bwd(dyq, dyk, q, k, g, g, freq=f, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*gt.gt_qk_norm_fwd(q, k, g, g, freq=f), *gt.gt_qk_norm_bwd(dyq, dyk, q, k, g, g, freq=f))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def _tail_and_beginning(n):
    """Rows at the beginning, around 2^30 rows before the end and at the end."""
    return torch.cat([torch.arange(300), torch.arange(n // 2, n // 2 + 100), torch.arange(n - 300, n)]).cuda()


def test_rows_past_2_to_the_30(gt):
    """More than 2^30 rows whose heads do not fill the lanes of a warp, in place: each row once."""
    torch.cuda.empty_cache()
    n, c = 2 ** 30 + 150, 16
    x, g, f = torch.empty(n, 1, c, dtype=B, device="cuda").normal_(), _gain(c, 2), _freq(c)
    at = _tail_and_beginning(n)
    want = X.qk_fwd(x[at], g, f, at.int(), 0, EPS, B)
    gt.gt_qk_norm_fwd(x, None, g, freq=f, eps=EPS, out_q=x)
    R.check({"y": x[at]}, want)
    del x
    torch.cuda.empty_cache()
    # backward: one row of x many times, three heads to a row, dx over its own dy
    h, c = 3, 8
    x, dy, g = _t((1, h, c), B, 3).expand(n, h, c), torch.empty(n, h, c, dtype=B, device="cuda").normal_(), _gain(c, 4)
    want = X.qk_bwd(dy[at], x[at], g, None, None, 0, EPS)
    gt.gt_qk_norm_bwd(dy, None, x, None, g, eps=EPS, dq=dy)
    R.check({"dx": dy[at]}, {"dx": want["dx"]})
    del dy
    torch.cuda.empty_cache()


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("c,rot", [(8, 8), (64, 64), (128, 0), (62, 62), (65, 20), (256, 256), (1, 0)])
@pytest.mark.parametrize("size,eps", [(1e10, 1e-6), (3e18, 1e-6), (2e19, 1e-6), (1e25, 1e-6), (1e38, 1e-6), (1e20, 3e38), (1e-12, 1e-24),
                                      (1e-22, 1e-43), (1e-30, 1e-45)])
def test_the_whole_range_of_fp32(gt, size, eps, c, rot, t):
    """Squares above the largest and below the smallest fp32 number, among rows of ordinary size."""
    eps = float(torch.tensor(eps, dtype=F))
    q, k, gq, gk = _t((70, 3, c), F, 1, 0.5), _t((33, 1, c), F, 2, 0.5), _gain(c, 3), _gain(c, 4)
    for x in (q, k):
        x[::3] *= size
        x[5] = 0
    q, k, f = q.to(t), k.to(t), _freq(rot)
    yq, yk = gt.gt_qk_norm_fwd(q, k, gq, gk, freq=f, eps=eps, out_dtype=F)
    R.check({"y": yq}, X.qk_fwd(q, gq, f, None, 0, eps, F))
    R.check({"y": yk}, X.qk_fwd(k, gk, f, None, 0, eps, F))
    # (dy of the size that makes dx ordinary numbers, and with them their rounding a share of each)
    scale = torch.ones(70, 1, 1, device="cuda")
    scale[::3] = min(max(size, 1.0), 1e9)
    dyq = _t(yq.shape, F, 5) * scale
    dq, _, dgq, _ = gt.gt_qk_norm_bwd(dyq, None, q, None, gq, freq=f, eps=eps)
    want = X.qk_bwd(dyq, q, gq, f, None, 0, eps)
    tiny = 2.0 ** -150 if t == F else 2.0 ** -134      # half of the smallest step there is
    R.check({"dx": dq, "dgain": dgq}, {"dx": (want["dx"][0], want["dx"][1] + tiny), "dgain": want["dgain"]}, floor=0.0)


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("n,h,c", [(1, 1, 8), (1, 1, 6), (1, 3, 64), (2, 1, 128), (5, 2, 62), (9, 4, 16), (3, 2, 65)])
def test_gain_sums_of_few_heads(gt, n, h, c, t):
    """A sum of as many terms as there are heads is rounded at most once for each but the first, wherever they are added
    (the zeros of idle lanes and CTAs add nothing)."""
    x, dy, g, f = _t((n, h, c), t, 1), _t((n, h, c), t, 2), _gain(c, 3), _freq(c // 2 * 2)
    dgain = gt.gt_qk_norm_bwd(dy, None, x, None, g, freq=f, eps=EPS)[2]
    value, bound = X.qk_bwd(dy, x, g, f, None, 0, EPS)["dgain"]
    xd = R.d(x)
    part = X.turn(R.d(dy), None, f, 0, back=True) * xd * ((xd * xd).mean(-1, keepdim=True) + EPS) ** -0.5
    terms = part.abs().sum((0, 1))
    bound = bound - (n * h / 64 + 1024) * R.U32 * terms + (n * h - 1) * R.U32 * terms      # the terms' own errors stay
    R.check({"dgain": dgain}, {"dgain": (value, bound + R.U32 * value.abs())}, floor=1e-38)
