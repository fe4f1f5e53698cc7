"""The linear layer's forward and backward on the GPU against fp64, within derived bounds."""
import math

import pytest
import torch

import linear_ref as R

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def gt():
    import graph_transformer_attention_gb300 as m
    from graph_transformer_attention_gb300 import build
    build.build()
    m.load_library()
    return m


def _mat(rows, cols, dtype, seed, std=1.0, pad=0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(rows, cols + pad + offset, generator=g, device="cuda") * std
    return t.to(dtype)[:, offset:offset + cols]


def _vec(n, seed, std=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, generator=g, device="cuda") * std


def _forward(gt, m, k, n, xt, yt, act, bias=True, res=True, pad=0, offset=0):
    x = _mat(m, k, xt, 1, pad=pad, offset=offset)
    w = _mat(k, n, xt, 2, 1 / math.sqrt(k), pad=pad, offset=offset)
    b = _vec(n, 3) if bias else None
    r = _mat(m, n, yt, 4, pad=pad, offset=offset) if res else None
    y, pre = gt.gt_linear_fwd(x, w, b, act=act, r=r, out_dtype=yt, save_pre=True)
    gt.gt_check_device_status()
    assert y.dtype == yt and pre.dtype == xt
    R.check({"y": y, "pre": pre}, R.linear_fwd(x, w, b, act == gt.GT_ACT_GELU, r, yt))


def _backward(gt, m, k, n, xt, yt, act, add=True, pad=0, offset=0):
    dy = _mat(m, n, yt, 5, pad=pad, offset=offset)
    x = _mat(m, k, xt, 1, pad=pad, offset=offset)
    w = _mat(k, n, xt, 2, 1 / math.sqrt(k), pad=pad, offset=offset)
    gelu = act == gt.GT_ACT_GELU
    pre = _mat(m, n, xt, 6, pad=pad, offset=offset) if gelu else None
    a = _mat(m, k, xt, 7, pad=pad, offset=offset) if add else None
    dx, dw, db = gt.gt_linear_bwd(dy, x, w, pre=pre, act=act, dx_add=a)
    gt.gt_check_device_status()
    R.check({"dx": dx, "dw": dw, "db": db}, R.linear_bwd(dy, x, w, pre, gelu, a))


TYPES = [(B, B), (B, F), (F, F)]
# one row, one feature, tiles exact and one past each of their edges, contractions that end inside a k-block
# and short of one, fp32 sizes on both sides of the one-kernel path (k 64 forward, m 1024 or n 128 backward)
SHAPES = [(1, 1, 1), (1, 64, 64), (2, 8, 200), (128, 64, 64), (129, 65, 65), (127, 63, 129), (64, 16, 256),
          (300, 200, 257), (257, 72, 512), (640, 136, 72), (130, 1000, 40), (17, 520, 1016), (65, 512, 33), (66, 64, 192), (67, 65, 193),
          (1024, 33, 65), (1025, 72, 40), (257, 600, 1025), (1, 777, 1500), (9, 140, 192)]


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("m,k,n", SHAPES)
def test_forward(gt, m, k, n, xt, yt, act):
    _forward(gt, m, k, n, xt, yt, act)


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("m,k,n", SHAPES)
def test_backward(gt, m, k, n, xt, yt, act):
    _backward(gt, m, k, n, xt, yt, act)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (5, 0), (0, 8), (8, 1), (0, 3)])
@pytest.mark.parametrize("m,k,n", [(150, 104, 88), (1100, 520, 88)])
def test_strided_and_unaligned_operands(gt, m, k, n, xt, yt, pad, offset):
    _forward(gt, m, k, n, xt, yt, 1, pad=pad, offset=offset)
    _backward(gt, m, k, n, xt, yt, 1, pad=pad, offset=offset)
    _backward(gt, m, k, n, xt, yt, 0, pad=pad, offset=offset)


@pytest.mark.parametrize("m,k,n,xt,yt", [
    (3000, 256, 1024, B, B),        # more tiles than SMs: the persistent loop, both accumulators
    (20000, 64, 192, B, F),         # the tile group order's tail group
    (5000, 64, 192, F, F),
    (4100, 64, 64, B, B),           # long contraction of dW over few tiles: splits and their join
    (4100, 40, 72, F, F),
    (2, 4000, 24, B, B),            # long contraction of the forward over one tile
    (40, 24, 4000, F, F),           # ... and of dx
])
def test_larger_shapes(gt, m, k, n, xt, yt):
    for act in (0, 1):
        _forward(gt, m, k, n, xt, yt, act, res=act == 0)
        _backward(gt, m, k, n, xt, yt, act, add=act == 0)


@pytest.mark.parametrize("m,k,n,xt,yt", [
    (900, 40, 128, F, F), (900, 40, 129, F, F),       # both sides of the one-kernel path of the backward
    (2000, 300, 600, B, B), (2000, 303, 601, B, B),   # both products in one launch, dW's contraction split
    (2000, 303, 601, B, F), (2000, 303, 601, F, F),
    (777, 1032, 520, B, B),                           # ... dx's contraction split too
    (9000, 520, 264, F, F),                           # several tiles to a pair of SMs in both
])
def test_both_products_in_one_launch(gt, m, k, n, xt, yt):
    for act in (0, 1):
        _backward(gt, m, k, n, xt, yt, act, add=act == 1)
    dy, x, w = _mat(m, n, yt, 1), _mat(m, k, xt, 2), _mat(k, n, xt, 3)
    dx, dw, _ = gt.gt_linear_bwd(dy, x, w)
    assert torch.equal(dx, gt.gt_linear_bwd(dy, x, w, need_dw=False)[0])
    assert torch.equal(dw, gt.gt_linear_bwd(dy, x, w, need_dx=False, need_db=False)[1])


@pytest.mark.parametrize("m,k,n", [(2500, 136, 801), (2499, 75, 1030), (33, 64, 2111)])
@pytest.mark.parametrize("pad", [0, 3])
def test_odd_bf16_rows(gt, m, k, n, pad):
    """Rows that only single elements can reach, each array alone and all, with the residual in place."""
    x, w, b, r = _mat(m, k, B, 1), _mat(k, n, B, 2, 0.1), _vec(n, 3), _mat(m, n, B, 4, pad=pad)
    wide = [torch.full((m + 1, n + 8), 7.0, dtype=B, device="cuda") for _ in range(2)]
    out, pre = (t[:m, 1:n + 1] for t in wide)
    out.copy_(r)
    gt.gt_linear_fwd(x, w, b, act=1, r=out, out=out, pre=pre)
    gt.gt_check_device_status()
    ref = R.linear_fwd(x, w, b, True, r, B)
    R.check({"y": out, "pre": pre}, ref)
    for t in wide:
        assert (t[m] == 7).all() and (t[:, 0] == 7).all() and (t[:, n + 1:] == 7).all()
    y, a = gt.gt_linear_fwd(x, w, b, act=1, r=r, save_pre=True)
    assert torch.equal(y, out) and torch.equal(a, pre)


@pytest.mark.parametrize("xt,k,n", [(B, 24, 2200), (F, 2200, 24), (B, 2200, 24)])
def test_offsets_past_32_bits(gt, xt, k, n):
    """A million rows, whose wide matrix has more than 2^31 elements: its last rows, and sums over all of them."""
    m, tail = 1 << 20, 300
    x, w, dy = _mat(m, k, xt, 1), _mat(k, n, xt, 2, 0.1), _mat(m, n, xt, 3)
    y, pre = gt.gt_linear_fwd(x, w, act=1, save_pre=True)
    dx = gt.gt_linear_bwd(dy, x, w, pre=pre, act=1, need_dw=False, need_db=False)[0]
    gt.gt_check_device_status()
    ref = R.linear_fwd(x[-tail:], w, None, True, None, xt)
    R.check({"y": y[-tail:], "pre": pre[-tail:]}, ref)
    R.check({"dx": dx[-tail:]}, {"dx": R.linear_bwd(dy[-tail:], x[-tail:], w, pre[-tail:], True, None)["dx"]})
    # The sums over rows, of positive terms: an accumulator drops at most 2^-23 of itself in each of 256 steps (six times 4
    # for fp32), m / 64 chunks and a thousand partial sums are added with 2^-24 each.
    del y, pre, dx
    x.abs_(), dy.abs_()
    _, dw, db = gt.gt_linear_bwd(dy, x, w, need_dx=False)
    rows = range(0, m, 1 << 16)
    ref = {"dw": sum(x[i:i + (1 << 16)].double().T @ dy[i:i + (1 << 16)].double() for i in rows),
           "db": sum(dy[i:i + (1 << 16)].double().sum(0) for i in rows)}
    for got, want in ((dw, ref["dw"]), (db, ref["db"])):
        tol = (R.half_step(got.dtype) + 256 * 2 * R.U32 + (m / 64 + 1024) * R.U32) * want
        assert ((got.double() - want).abs() <= tol).all()


def test_without_bias_residual_or_add(gt):
    for xt, yt in TYPES:
        _forward(gt, 70, 90, 110, xt, yt, 1, bias=False, res=False)
        _backward(gt, 70, 90, 110, xt, yt, 0, add=False)


@pytest.mark.parametrize("m,k,n", [(75, 48, 40), (1030, 530, 300)])
def test_outputs_into_slices_leave_the_rest_alone(gt, m, k, n):
    for xt, yt in TYPES:
        for pad in (8, 3):
            x, w, dy = _mat(m, k, xt, 1), _mat(k, n, xt, 2), _mat(m, n, yt, 3)
            buf = {s: torch.full((r, c + 2 * pad), 7.0, dtype=t, device="cuda")
                   for s, r, c, t in (("y", m, n, yt), ("pre", m, n, xt), ("dx", m, k, xt), ("dw", k, n, xt))}
            cut = {s: t[:, pad:-pad] for s, t in buf.items()}
            gt.gt_linear_fwd(x, w, None, act=1, out=cut["y"], pre=cut["pre"])
            R.check({"y": cut["y"], "pre": cut["pre"]}, R.linear_fwd(x, w, None, True, None, yt))
            gt.gt_linear_bwd(dy, x, w, dx=cut["dx"], dw=cut["dw"])
            ref = R.linear_bwd(dy, x, w, None, False, None)
            R.check({"dx": cut["dx"], "dw": cut["dw"]}, ref)
            for t in buf.values():
                assert (t[:, :pad] == 7).all() and (t[:, -pad:] == 7).all()


@pytest.mark.parametrize("fill", [300.0, float("nan")])
def test_margins_of_the_inputs_do_not_count(gt, fill):
    """Inputs whose rows end at odd columns inside 16 bytes, with large values or NaN behind them: read in
    place, what lies behind a row's end must not enter any sum."""
    def odd(rows, cols, seed, std=1.0):
        wide = torch.full((rows + 2, (cols + 7) // 8 * 8 + 8), fill, dtype=B, device="cuda")
        wide[:rows, :cols] = _mat(rows, cols, B, seed, std)
        return wide[:rows, :cols]

    for m, k, n in ((300, 65, 129), (257, 321, 1001), (40, 1003, 67), (3000, 257, 511)):
        x, w, dy, pre, r = odd(m, k, 1), odd(k, n, 2, 1 / math.sqrt(k)), odd(m, n, 3), odd(m, n, 4), odd(m, n, 5)
        y, a = gt.gt_linear_fwd(x, w, act=1, r=r, save_pre=True)
        R.check({"y": y, "pre": a}, R.linear_fwd(x, w, None, True, r, B))
        for p, act in ((None, 0), (pre, 1)):
            dx, dw, db = gt.gt_linear_bwd(dy, x, w, pre=p, act=act)
            R.check({"dx": dx, "dw": dw, "db": db}, R.linear_bwd(dy, x, w, p, act == 1, None))


@pytest.mark.parametrize("k", [200, 5000])        # one accumulator chunk (results leave as TMA boxes), and several
def test_box_edges_leave_the_rest_alone(gt, k):
    """Results whose last columns and rows end inside a tile, in rows of whole 16 bytes with a margin."""
    for m, n in ((600, 300), (257, 1001), (130, 33), (3000, 999)):
        x, w, b = _mat(m, k, B, 1), _mat(k, n, B, 2, 0.1), _vec(n, 3)
        width = (n + 7) // 8 * 8 + 8
        buf = [torch.full((m + 3, width), 7.0, dtype=B, device="cuda") for _ in range(2)]
        y, pre = (t[:m, :n] for t in buf)
        gt.gt_linear_fwd(x, w, b, act=1, out=y, pre=pre)
        R.check({"y": y, "pre": pre}, R.linear_fwd(x, w, b, True, None, B))
        for t in buf:
            assert (t[m:] == 7).all() and (t[:, n:] == 7).all()


@pytest.mark.parametrize("m", [200, 1100])
def test_parts_of_the_backward(gt, m):
    """Each gradient alone equals the one of the whole call."""
    for xt, yt in TYPES:
        dy, x, w, pre = _mat(m, 90, yt, 1), _mat(m, 70, xt, 2), _mat(70, 90, xt, 3), _mat(m, 90, xt, 4)
        for act, p in ((0, None), (1, pre)):
            dx, dw, db = gt.gt_linear_bwd(dy, x, w, pre=p, act=act)
            one = gt.gt_linear_bwd(dy, x, w, pre=p, act=act, need_dw=False, need_db=False)
            two = gt.gt_linear_bwd(dy, x, w, pre=p, act=act, need_dx=False, need_db=False)
            three = gt.gt_linear_bwd(dy, x, w, pre=p, act=act, need_dx=False, need_dw=False)
            assert torch.equal(one[0], dx) and one[1] is None and one[2] is None
            assert torch.equal(two[1], dw) and two[0] is None
            assert torch.equal(three[2], db) and three[0] is None and three[1] is None


@pytest.mark.parametrize("m,k", [(90, 60), (1100, 600), (1100, 603)])
def test_in_place_residual_and_accumulated_gradient(gt, m, k):
    for xt, yt in TYPES:
        x, w, b, r, dy = _mat(m, k, xt, 1), _mat(k, 70, xt, 2), _vec(70, 3), _mat(m, 70, yt, 4), _mat(m, 70, yt, 5)
        want, _ = gt.gt_linear_fwd(x, w, b, act=1, r=r)
        buf = r.clone()
        got, _ = gt.gt_linear_fwd(x, w, b, act=1, r=buf, out=buf)
        assert got is buf and torch.equal(got, want)
        add = _mat(m, k, xt, 6)
        want, _, _ = gt.gt_linear_bwd(dy, x, w, dx_add=add)
        buf = add.clone()
        got, _, _ = gt.gt_linear_bwd(dy, x, w, dx_add=buf, dx=buf)
        assert got is buf and torch.equal(got, want)


def test_same_result_every_time(gt):
    for m, k, n, xt in ((4000, 64, 64, B), (3, 2000, 300, B), (700, 100, 60, F), (3000, 1000, 60, F)):
        x, w, dy = _mat(m, k, xt, 1), _mat(k, n, xt, 2), _mat(m, n, xt, 3)
        y = gt.gt_linear_fwd(x, w)[0]
        g = gt.gt_linear_bwd(dy, x, w)
        for _ in range(3):
            assert torch.equal(gt.gt_linear_fwd(x, w)[0], y)
            assert all(torch.equal(a, b) for a, b in zip(gt.gt_linear_bwd(dy, x, w), g))


@pytest.mark.parametrize("k", [64, 640])
def test_fp32_products_keep_fp32_accuracy(gt, k):
    """Exact cases, for the one-kernel path and the split products."""
    # small whole numbers, whose products and sums are whole
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-2000, 2001, (50, k), generator=g, device="cuda").float()
    w = torch.randint(-12, 13, (k, 30), generator=g, device="cuda").float()
    assert torch.equal(gt.gt_linear_fwd(x, w)[0].double(), x.double() @ w.double())
    # 24-bit values times powers of two: hi, mid and lo all matter, nothing rounds
    x = (torch.randint(2 ** 23, 2 ** 24, (40, k), generator=g, device="cuda").float()
         * 2.0 ** torch.randint(-40, 41, (40, 1), generator=g, device="cuda"))
    w = torch.zeros(k, k, device="cuda")
    w[torch.arange(k), torch.arange(k).flip(0)] = 2.0 ** torch.randint(-20, 21, (k,), generator=g, device="cuda")
    assert torch.equal(gt.gt_linear_fwd(x, w)[0].double(), x.double() @ w.double())
    # the largest finite value is split without overflow
    x = torch.full((2, k), torch.finfo(F).max, device="cuda")
    w = torch.zeros(k, 8, device="cuda")
    w[3] = 0.5
    assert torch.equal(gt.gt_linear_fwd(x, w)[0], torch.full((2, 8), torch.finfo(F).max / 2, device="cuda"))


def test_long_positive_sums(gt):
    """All-positive sums 20000 long, where an accumulator that drops low bits would lag by 1e-4 in fp32: within
    1e-6 (measured 3e-7; two roundings of a sum of 80 chunks, 2^-23 each, and 4.4e-8 per 16-deep step of one chunk)."""
    for xt in (F, B):
        x, w = _mat(300, 20000, F, 1).abs().to(xt), _mat(20000, 200, F, 2).abs().to(xt)
        y, _ = gt.gt_linear_fwd(x, w, out_dtype=F)
        ref = R.d(x) @ R.d(w)
        assert float(((R.d(y) - ref).abs() / ref).max()) < 1e-6
        # dW sums over the 20000 rows
        x, dy = _mat(20000, 130, F, 3).abs().to(xt), _mat(20000, 100, F, 4).abs().to(xt)
        _, dw, _ = gt.gt_linear_bwd(dy, x, _mat(130, 100, xt, 5), need_dx=False)
        ref = R.d(x).t() @ R.d(dy)
        assert float(((R.d(dw) - ref).abs() / ref).max()) < (1e-6 if xt == F else 2.0 ** -8 + 2e-5)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("m,k,n", [(140, 70, 90), (1100, 520, 90)])
def test_nonfinite_inputs_stay_in_their_rows(gt, m, k, n, xt, yt):
    x, w, dy = _mat(m, k, xt, 1), _mat(k, n, xt, 2, 0.1), _mat(m, n, yt, 3)
    x[5, 3] = float("inf")
    x[130, 69] = float("nan")
    fine = [i for i in range(m) if i not in (5, 130)]
    y, _ = gt.gt_linear_fwd(x, w, out_dtype=yt)
    assert not y[5].isfinite().any() and y[130].isnan().all()
    R.check({"y": y[fine]}, R.linear_fwd(x[fine], w, None, False, None, yt))
    dx, dw, db = gt.gt_linear_bwd(dy, x, w)
    ref = R.linear_bwd(dy, x.nan_to_num(0, 0, 0), w, None, False, None)
    R.check({"dx": dx, "db": db}, ref)
    rows = [i for i in range(k) if i not in (3, 69)]
    R.check({"dw": dw[rows]}, {"dw": tuple(t[rows] for t in ref["dw"])})
    assert not dw[3].isfinite().any() and dw[69].isnan().all()


def test_gelu_over_its_range(gt):
    """GELU and its slope from -30 to 30 and at the ends, through one-feature products."""
    a = torch.cat([torch.linspace(-30, 30, 2001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e30, -1e30])]).cuda()[:, None]
    one = torch.ones(1, 1, device="cuda")
    y, pre = gt.gt_linear_fwd(a, one, act=gt.GT_ACT_GELU, save_pre=True)
    assert torch.equal(pre, a)
    R.check({"y": y}, R.linear_fwd(a, one, None, True, None, F))
    dx, _, _ = gt.gt_linear_bwd(torch.ones_like(a), a, one, pre=a, act=gt.GT_ACT_GELU, need_dw=False, need_db=False)
    R.check({"dx": dx}, R.linear_bwd(torch.ones_like(a), a, one, a, True, None))


def test_gradient_against_differences(gt):
    m, k, n = 9, 14, 11
    x, w, b, dy = _mat(m, k, F, 1), _mat(k, n, F, 2, 0.3), _vec(n, 3), _mat(m, n, F, 4)
    y, pre = gt.gt_linear_fwd(x, w, b, act=1, save_pre=True)
    dx, dw, db = (R.d(t) for t in gt.gt_linear_bwd(dy, x, w, pre=pre, act=1))
    xd, wd, bd, dyd = R.d(x), R.d(w), R.d(b), R.d(dy)

    def loss(x_, w_, b_):
        a = x_ @ w_ + b_
        return float((a * R.phi(a) * dyd).sum())

    h = 1e-5
    for i, j in ((0, 0), (4, 7), (8, 10)):
        for name, grad, idx in (("x", dx, (i, j)), ("w", dw, (i, j)), ("b", db, (j,))):
            v = {"x": xd.clone(), "w": wd.clone(), "b": bd.clone()}
            v[name][idx] += h
            up = loss(**{s + "_": t for s, t in v.items()})
            v[name][idx] -= 2 * h
            down = loss(**{s + "_": t for s, t in v.items()})
            assert abs((up - down) / (2 * h) - float(grad[idx])) < 1e-5, name


def test_streams_and_graph(gt):
    """On a side stream, two calls at once, and captured once and replayed on new inputs."""
    m, k, n = 300, 500, 60
    x, w, b, dy = _mat(m, k, B, 1), _mat(k, n, B, 2, 0.05), _vec(n, 3), _mat(m, n, B, 4)

    def both(stream=None):
        y, pre = gt.gt_linear_fwd(x, w, b, act=1, save_pre=True, stream=stream)
        return (y, *gt.gt_linear_bwd(dy, x, w, pre=pre, act=1, stream=stream))

    want = both()
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [both(s) for s in sides]
    for s in sides:
        torch.cuda.current_stream().wait_stream(s)
    for g in got:
        assert all(torch.equal(a, c) for a, c in zip(want, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for t, seed in ((x, 11), (dy, 14)):
        t.copy_(_mat(*t.shape, B, seed))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(held, both()))


def test_two_graphs_share_a_workspace(gt):
    """Two captured calls with one workspace, replayed in turn, leave nothing behind in it."""
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    sets = []
    for seed, (m, k, n, xt) in enumerate(((3000, 64, 72, B), (40, 3000, 96, F))):
        x, w, dy = _mat(m, k, xt, seed), _mat(k, n, xt, seed + 5, 0.1), _mat(m, n, xt, seed + 9)
        call = lambda x=x, w=w, dy=dy: (gt.gt_linear_fwd(x, w, workspace=ws)[0],  # noqa: E731
                                        *gt.gt_linear_bwd(dy, x, w, workspace=ws))
        want = call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = call()
        sets.append((graph, held, want))
    for _ in range(3):
        for graph, held, want in sets:
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.parametrize("width,heads,ffn,t", [(128, 8, 320, F), (96, 8, 200, B), (72, 4, 130, F)])
def test_whole_encoder_layer_at_other_widths(gt, width, heads, ffn, t):
    """LayerNorm, projections, biased attention and FFN together, forward and backward, against the fp64
    layer oracle: fp32 to 1e-4 and bf16 products (fp32 residual stream) to 2e-2 relative L2 per tensor, the
    attention's own tolerances."""
    import numpy as np

    import gt_inputs as gi
    from oracle import layer as L
    from oracle import oracle as O
    O.build()
    n, D = 333, 6
    g = gi.barabasi_albert(n, 3, seed=21)
    spd = O.spd(n, g.indptr, g.indices, D)
    p = gi.make_gt_layer_params(width, ffn, D + 2, heads, seed=5)
    io = gi.make_gt_layer_io(n, width, seed=6)
    dev = torch.device("cuda")
    spd_d = torch.zeros((n, gt.spd_ld(n)), dtype=torch.int8)
    spd_d[:, :n] = torch.from_numpy(spd)
    spd_d = spd_d.to(dev)
    P = {s: torch.from_numpy(v).to(dev) for s, v in p.items()}
    x, dy = torch.from_numpy(io["x"]).to(dev), torch.from_numpy(io["dy"]).to(dev)
    W = {s: P[s].to(t) for s in ("w_qkv", "w_o", "w_1", "w_2")}
    cut = [slice(i * width, (i + 1) * width) for i in range(3)]
    d = width // heads

    u, m1, r1 = gt.gt_layer_norm_fwd(x, P["ln1_g"], P["ln1_b"], out_dtype=t)
    q, k, v = (gt.gt_linear_fwd(u, W["w_qkv"][:, c], P["b_qkv"][c])[0].view(n, heads, d) for c in cut)
    o, lse = gt.gt_bias_attn_fwd(q, k, v, spd_d, P["T"])
    hh, _ = gt.gt_linear_fwd(o.view(n, width), W["w_o"], P["b_o"], r=x)
    z, m2, r2 = gt.gt_layer_norm_fwd(hh, P["ln2_g"], P["ln2_b"], out_dtype=t)
    act, pre = gt.gt_linear_fwd(z, W["w_1"], P["b_1"], act=gt.GT_ACT_GELU, save_pre=True)
    y, _ = gt.gt_linear_fwd(act, W["w_2"], P["b_2"], r=hh)

    gr = {}
    dact, gr["w_2"], gr["b_2"] = gt.gt_linear_bwd(dy, act, W["w_2"])
    dz, gr["w_1"], gr["b_1"] = gt.gt_linear_bwd(dact, z, W["w_1"], pre=pre, act=gt.GT_ACT_GELU)
    dhh, gr["ln2_g"], gr["ln2_b"] = gt.gt_layer_norm_bwd(dz, hh, P["ln2_g"], m2, r2, dres=dy)
    do, gr["w_o"], gr["b_o"] = gt.gt_linear_bwd(dhh, o.view(n, width), W["w_o"])
    dq, dk, dv, gr["T"] = gt.gt_bias_attn_bwd(q, k, v, o, do.view(n, heads, d), lse, spd_d, P["T"])
    dw, db, du = torch.empty_like(W["w_qkv"]), torch.empty_like(P["b_qkv"]), None
    for c, s in zip(cut, (dq, dk, dv)):
        du, _, db[c] = gt.gt_linear_bwd(s.view(n, width), u, W["w_qkv"][:, c], dx_add=du, dw=dw[:, c])
    gr["w_qkv"], gr["b_qkv"] = dw, db
    gr["x"], gr["ln1_g"], gr["ln1_b"] = gt.gt_layer_norm_bwd(du, x, P["ln1_g"], m1, r1, dres=dhh)
    gt.gt_check_device_status()

    fw = L.layer_fwd(io["x"], p, spd, heads)
    ref = L.layer_bwd(io["x"], p, spd, heads, fw, io["dy"])
    tol = 1e-4 if t == F else 2e-2

    def rel(a, c):
        a, c = R.d(a).numpy().ravel(), np.asarray(c, np.float64).ravel()
        return float(np.linalg.norm(a - c) / np.linalg.norm(c))

    errs = {"y": rel(y, fw["y"]), **{s: rel(gr[s], ref[s]) for s in gr}}
    assert all(e <= tol for e in errs.values()), errs


def test_binding_refusals(gt):
    """Shapes, types, strides, devices and streams that the binding turns away before any launch."""
    x, w, b, dy = _mat(6, 8, B, 1), _mat(8, 10, B, 2), _vec(10, 3), _mat(6, 10, B, 4)
    value = (
        lambda: gt.gt_linear_fwd(x[0], w),                                    # one dimension
        lambda: gt.gt_linear_fwd(x, w[0]),
        lambda: gt.gt_linear_fwd(x, w[:7]),                                   # inner sizes differ
        lambda: gt.gt_linear_fwd(x, w, b[:9]),
        lambda: gt.gt_linear_fwd(x, w, b.double()),
        lambda: gt.gt_linear_fwd(x, w, r=dy[:5]),
        lambda: gt.gt_linear_fwd(x, w.t().contiguous().t()),                  # columns not contiguous
        lambda: gt.gt_linear_fwd(x[:1].expand(6, 8), w),                      # rows overlap
        lambda: gt.gt_linear_fwd(x, w.cpu()),
        lambda: gt.gt_linear_fwd(x, w, out=torch.empty(6, 9, dtype=B, device="cuda")),
        lambda: gt.gt_linear_fwd(x, w, workspace=torch.empty(64, dtype=torch.uint8)),
        lambda: gt.gt_linear_bwd(dy[:5], x, w),
        lambda: gt.gt_linear_bwd(dy, x, w, dx_add=x[:, :7]),
        lambda: gt.gt_layer_norm_fwd(x, b, b),
        lambda: gt.gt_layer_norm_fwd(x[0], b[:8], b[:8]),
    )
    for call in value:
        with pytest.raises(ValueError):
            call()
    kind = (
        lambda: gt.gt_linear_fwd(x.half(), w.half()),
        lambda: gt.gt_linear_fwd(x, w.float()),
        lambda: gt.gt_linear_fwd(x, w, r=dy.float(), out_dtype=B),
        lambda: gt.gt_linear_fwd(x, w, out_dtype=torch.float16),
        lambda: gt.gt_linear_bwd(dy.half(), x, w),
        lambda: gt.gt_layer_norm_fwd(x.double(), b[:8].contiguous(), b[:8].contiguous()),
    )
    for call in kind:
        with pytest.raises(TypeError):
            call()
    for call in (lambda: gt.gt_linear_fwd(x.float(), w.float(), out_dtype=B),           # bf16 result of fp32 products
                 lambda: gt.gt_linear_fwd(x, w, act=5),
                 lambda: gt.gt_linear_fwd(x[:0], w),                                    # no rows
                 lambda: gt.gt_linear_bwd(dy, x, w, act=gt.GT_ACT_GELU),                # GELU without pre
                 lambda: gt.gt_linear_bwd(dy, x, w, need_dx=False, need_dw=False, need_db=False),
                 lambda: gt.gt_linear_bwd(dy, x, w, dx_add=x, need_dx=False),
                 lambda: gt.gt_linear_bwd(dy, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                 lambda: gt.gt_layer_norm_fwd(x, b[:8].contiguous(), b[:8].contiguous(), eps=0.0),
                 lambda: gt.gt_layer_norm_fwd(x[:0], b[:8].contiguous(), b[:8].contiguous())):
        with pytest.raises(gt.GtError):
            call()


@pytest.mark.parametrize("m,k,n,xt,yt", [
    (2, 4000, 24, B, B), (2, 4000, 24, F, F),         # the forward's contraction split
    (1100, 520, 89, B, F), (300, 200, 257, F, F),     # fp32 sums of rows that only single elements can reach
    (40, 24, 4000, F, F), (40, 24, 4000, B, B),       # dx's contraction split
    (4100, 64, 64, B, B), (4100, 40, 72, F, F),       # dW's, in a launch of its own or with dx
    (2000, 303, 601, B, F), (2000, 303, 601, F, F),   # both products in one launch, both leave sums
])
def test_workspace_of_any_16_byte_alignment(gt, m, k, n, xt, yt):
    """A workspace 16 bytes past a 32-byte boundary serves as any other: the same results, and nothing outside it written."""
    x, w, dy, b = _mat(m, k, xt, 1), _mat(k, n, xt, 2, 1 / math.sqrt(k)), _mat(m, n, yt, 3), _vec(n, 4)

    def room(need):
        buf = torch.full((need + 64,), 7, dtype=torch.uint8, device="cuda")
        assert buf.data_ptr() % 32 == 0
        return buf, buf[16:16 + need]

    code = gt.GT_F32 if xt == F else gt.GT_BF16
    buf, ws = room(gt.gt_linear_fwd_workspace_size(code, m, k, n, aligned=False))
    got = gt.gt_linear_fwd(x, w, b, out_dtype=yt, workspace=ws)[0]
    assert torch.equal(got, gt.gt_linear_fwd(x, w, b, out_dtype=yt)[0])
    assert (buf[:16] == 7).all() and (buf[16 + ws.numel():] == 7).all()
    buf, ws = room(gt.gt_linear_bwd_workspace_size(code, gt.GT_F32 if yt == F else gt.GT_BF16, m, k, n, aligned=False))
    for parts in ({}, {"need_dw": False}, {"need_dx": False}):
        got = gt.gt_linear_bwd(dy, x, w, workspace=ws, **parts)
        for a, c in zip(got, gt.gt_linear_bwd(dy, x, w, **parts)):
            assert (a is None and c is None) or torch.equal(a, c)
    gt.gt_check_device_status()
    assert (buf[:16] == 7).all() and (buf[16 + ws.numel():] == 7).all()


@pytest.mark.parametrize("pad,offset", [(0, 0), (16, 0), (4, 4), (8, 8), (5, 0), (0, 1)])
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("m,k,n", [(1100, 512, 320), (90, 60, 72), (3, 2000, 304), (2000, 304, 600)])
def test_residual_in_place_at_every_access(gt, m, k, n, xt, yt, pad, offset):
    """r and y, and dx_add and dx, one buffer each, in rows of 32-byte, 16-byte and single-element accesses."""
    x, w, b, dy = _mat(m, k, xt, 1), _mat(k, n, xt, 2, 1 / math.sqrt(k)), _vec(n, 3), _mat(m, n, yt, 4)
    buf, other = _mat(m, n, yt, 5, pad=pad, offset=offset), _mat(m, n, yt, 6, pad=pad, offset=offset)
    r = buf.clone()
    want = gt.gt_linear_fwd(x, w, b, act=1, r=r, out=other)[0]
    got = gt.gt_linear_fwd(x, w, b, act=1, r=buf, out=buf)[0]
    assert got is buf and torch.equal(got, want)
    R.check({"y": got}, R.linear_fwd(x, w, b, True, r, yt))
    buf, other = _mat(m, k, xt, 7, pad=pad, offset=offset), _mat(m, k, xt, 8, pad=pad, offset=offset)
    add = buf.clone()
    want = gt.gt_linear_bwd(dy, x, w, dx_add=add, dx=other)
    got = gt.gt_linear_bwd(dy, x, w, dx_add=buf, dx=buf)
    assert got[0] is buf and all(torch.equal(a, c) for a, c in zip(got, want))
    R.check({"dx": got[0]}, R.linear_bwd(dy, x, w, None, False, add))
    gt.gt_check_device_status()


def _gelu_exact(a):
    """GELU and its slope at the fp64 values a, |a| <= 13, and the bounds of both as fp32 arithmetic makes them from the CDF's tail.
    (Exact values from erfc: torch.special.ndtr is 1/2 + erf / 2, which below -8 has no digit left in fp64 either.)
    The tail: its fit (0.5e-8 / max(1, |a|), 5e-5 of itself at most), and relative roundings: a polynomial of seven
    terms whose magnitudes add up to 2.5 times its value (2 x 7 x 2.5), its argument (four units, which count 3.2 times), two
    products, two units of the power (4), 60 with the rest; the power's own argument a^2 / 2 carries four roundings: 2 a^2.
    """
    x = a.abs()
    tail, dens = 0.5 * torch.special.erfc(x * math.sqrt(0.5)), torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi)
    tail_off = torch.minimum(0.5e-8 / x.clamp(min=1), 5e-5 * tail) + R.U32 * (60 + 2 * a * a) * tail
    cdf = torch.where(a >= 0, 1 - tail, tail)
    cdf_off = tail_off + (a >= 0) * R.U32
    y, slope = a * cdf, cdf + a * dens
    return (y, x * cdf_off + R.U32 * y.abs()), (slope, cdf_off + x * dens * R.U32 * (8 + 2 * a * a) + R.U32 * slope.abs())


@pytest.mark.parametrize("path", ["one kernel", "product", "join", "bf16 operands"])
def test_gelu_keeps_its_relative_accuracy(gt, path):
    """Far below zero too, where 1/2 and the CDF's other half cancel: the epilogues of the forward."""
    a = torch.cat([torch.linspace(-13, 13, 26001), torch.linspace(-0.01, 0.01, 201), torch.tensor([0.0, -0.0])]).cuda()
    k, n, t = {"one kernel": (1, 1, F), "product": (128, 8, F), "join": (128, 3, F), "bf16 operands": (16, 8, B)}[path]
    x = torch.zeros(a.numel(), k, dtype=t, device="cuda")
    x[:, 0] = a
    w = torch.zeros(k, n, dtype=t, device="cuda")
    w[0] = 1
    y, _ = gt.gt_linear_fwd(x, w, act=gt.GT_ACT_GELU, out_dtype=F)
    want, _ = _gelu_exact(R.d(x[:, :1]))
    R.check({"y": y}, {"y": tuple(v.expand(-1, n) for v in want)}, floor=1e-37)


@pytest.mark.parametrize("n", [100, 26203])           # one kernel, and the pass that forms da
def test_gelu_slope_keeps_its_relative_accuracy(gt, n):
    a = torch.cat([torch.linspace(-13, 13, n - 3), torch.tensor([0.0, -0.0, -0.75179])]).cuda()[None, :]
    one = torch.ones(1, 1, device="cuda")
    db = gt.gt_linear_bwd(torch.ones_like(a), one, torch.ones_like(a), pre=a, act=gt.GT_ACT_GELU, need_dx=False, need_dw=False)[2]
    _, want = _gelu_exact(R.d(a[0]))
    R.check({"db": db}, {"db": want}, floor=1e-37)


@pytest.mark.parametrize("t", [F, B])
def test_gelu_of_infinities_and_nan(gt, t):
    """a Phi(a): infinity, and NaN for minus infinity (times 0) and NaN; a / 2 for the smallest, as accurate as the tail."""
    a = torch.tensor([[float("inf")], [float("-inf")], [float("nan")], [1e38], [-1e38], [1e-30], [-1e-30]], dtype=t, device="cuda")
    y, _ = gt.gt_linear_fwd(a, torch.ones(1, 1, dtype=t, device="cuda"), act=gt.GT_ACT_GELU, out_dtype=F)
    y, a = y[:, 0], a[:, 0].float()
    assert y[0] == float("inf") and y[1].isnan() and y[2].isnan()
    assert y[3] == a[3] and y[4] == 0
    assert float((y[5:] / (a[5:] / 2) - 1).abs().max()) <= 62 * R.U32


@pytest.mark.parametrize("m,k,n", [(200, 70, 90), (1100, 70, 90), (2000, 304, 600)])
def test_backward_without_what_it_does_not_read(gt, m, k, n):
    """dx needs no x, dw no w, db one of them: the same results as with both."""
    for xt, yt in TYPES:
        dy, x, w, pre = _mat(m, n, yt, 1), _mat(m, k, xt, 2), _mat(k, n, xt, 3), _mat(m, n, xt, 4)
        for act, p in ((0, None), (1, pre)):
            dx, dw, db = gt.gt_linear_bwd(dy, x, w, pre=p, act=act)
            got = gt.gt_linear_bwd(dy, None, w, pre=p, act=act, need_dw=False)
            assert torch.equal(got[0], dx) and got[1] is None and torch.equal(got[2], db)
            got = gt.gt_linear_bwd(dy, x, None, pre=p, act=act, need_dx=False)
            assert got[0] is None and torch.equal(got[1], dw) and torch.equal(got[2], db)
            for a, c in ((x, None), (None, w)):
                assert torch.equal(gt.gt_linear_bwd(dy, a, c, pre=p, act=act, need_dx=False, need_dw=False)[2], db)
    for call in (lambda: gt.gt_linear_bwd(dy, None, w), lambda: gt.gt_linear_bwd(dy, x, None),
                 lambda: gt.gt_linear_bwd(dy, None, w, need_dw=False, dw=torch.empty_like(w)),
                 lambda: gt.gt_linear_bwd(dy, None, None, need_dx=False, need_dw=False),
                 lambda: gt.gt_linear_bwd(dy, x, w[:, :5], need_dx=False),
                 lambda: gt.gt_linear_bwd(dy, None, w[:, :5], need_dw=False)):
        with pytest.raises(ValueError):
            call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gt.gt_linear_bwd(dy, None, w, pre=pre, act=1, need_dw=False, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, dx)


@pytest.mark.parametrize("xt,yt", TYPES)
def test_column_sums_of_many_rows(gt, xt, yt):
    """db of a million positive rows: 64 additions in a thread (2^20 rows over 512 x 32), 32 in the CTA, 512 / 8 and 8 in the join,
    half a unit each at most; 200 of them counted."""
    m = 1 << 20
    dy, x, w = _mat(m, 64, yt, 1).abs(), _mat(m, 8, xt, 2), _mat(8, 64, xt, 3)
    db = gt.gt_linear_bwd(dy, x, w, need_dx=False, need_dw=False)[2]
    want = dy.double().sum(0)
    assert float(((db.double() - want).abs() / want).max()) <= 200 * R.U32
