"""LayerNorm forward and backward on the GPU against fp64, within derived bounds."""
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


def _rows(n, c, dtype, seed, pad=0, offset=0, mean=0.25):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(n, c + pad + offset, generator=g, device="cuda") * 1.5 + mean
    return t.to(dtype)[:, offset:offset + c]


def _vec(c, seed, std, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(c, generator=g, device="cuda") * std + mean


# widths on both sides of every change of layout, odd ones, rows that fill no CTA
SHAPES = [(1, 1), (3, 8), (5, 64), (37, 63), (300, 64), (33, 65), (9, 256), (70, 257), (129, 512), (20, 513),
          (41, 1024), (7, 1025), (11, 2048), (3, 2049), (5, 4096), (2, 4097), (6, 8192), (2, 8200), (3, 16384)]


@pytest.mark.parametrize("xt,yt", [(F, F), (F, B), (B, F), (B, B)])
@pytest.mark.parametrize("n,c", SHAPES)
def test_forward_and_backward(gt, n, c, xt, yt):
    x, gain, shift = _rows(n, c, xt, 1), _vec(c, 2, 0.1, 1.0), _vec(c, 3, 0.02)
    y, mean, rstd = gt.gt_layer_norm_fwd(x, gain, shift, eps=1e-5, out_dtype=yt)
    assert y.dtype == yt
    R.check({"y": y, "mean": mean, "rstd": rstd}, R.ln_fwd(x, gain, shift, 1e-5, yt))
    dy = _rows(n, c, yt, 4, mean=0.0)
    for dres in (None, _rows(n, c, xt, 5)):
        dx, dg, ds = gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd, dres=dres)
        R.check({"dx": dx, "dgain": dg, "dshift": ds}, R.ln_bwd(dy, x, gain, mean, rstd, dres))


@pytest.mark.parametrize("c,pad,offset", [(64, 8, 0), (64, 5, 0), (64, 8, 8), (64, 0, 1), (1000, 3, 1), (2047, 0, 1)])
@pytest.mark.parametrize("t", [F, B])
def test_strided_and_unaligned_rows(gt, c, pad, offset, t):
    n = 53
    x, dy, dres = (_rows(n, c, t, s, pad, offset) for s in (1, 2, 3))
    gain, shift = _vec(c + 1, 4, 0.1, 1.0)[1:].contiguous(), _vec(c, 5, 0.02)
    wide = torch.full((n, c + pad + offset), 7.0, dtype=t, device="cuda")
    out = wide[:, offset:offset + c]
    y, mean, rstd = gt.gt_layer_norm_fwd(x, gain, shift, out=out)
    assert y is out
    R.check({"y": y}, R.ln_fwd(x, gain, shift, 1e-5, t))
    assert (wide[:, :offset] == 7).all() and (wide[:, offset + c:] == 7).all()    # the rest of the rows as it was
    dwide = torch.full_like(wide, 7.0)
    dx, dg, ds = gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd, dres=dres, dx=dwide[:, offset:offset + c])
    R.check({"dx": dx, "dgain": dg, "dshift": ds}, R.ln_bwd(dy, x, gain, mean, rstd, dres))
    assert (dwide[:, :offset] == 7).all() and (dwide[:, offset + c:] == 7).all()


def test_many_rows(gt):
    """More rows than one turn of the grid, 64-wide and wide."""
    for n, c, t in ((20000, 64, F), (6000, 384, B), (2500, 1500, B)):
        x, gain, shift, dy = _rows(n, c, t, 1), _vec(c, 2, 0.1, 1.0), _vec(c, 3, 0.02), _rows(n, c, t, 4)
        y, mean, rstd = gt.gt_layer_norm_fwd(x, gain, shift)
        R.check({"y": y, "mean": mean, "rstd": rstd}, R.ln_fwd(x, gain, shift, 1e-5, t))
        dx, dg, ds = gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd)
        R.check({"dx": dx, "dgain": dg, "dshift": ds}, R.ln_bwd(dy, x, gain, mean, rstd, None))
        again = gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd)
        assert all(torch.equal(a, b) for a, b in zip((dx, dg, ds), again))


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("n,c", [(5000, 512), (3000, 1000), (1500, 2048), (1300, 2051), (700, 4096), (800, 8192), (400, 12000),
                                 (350, 16384)])
def test_many_wide_rows(gt, n, c, t):
    """Several turns of every CTA in each layout, with the next rows fetched ahead and without."""
    x, gain, shift, dy, dres = _rows(n, c, t, 1), _vec(c, 2, 0.1, 1.0), _vec(c, 3, 0.02), _rows(n, c, t, 4), _rows(n, c, t, 5)
    y, mean, rstd = gt.gt_layer_norm_fwd(x, gain, shift)
    R.check({"y": y, "mean": mean, "rstd": rstd}, R.ln_fwd(x, gain, shift, 1e-5, t))
    want = R.ln_bwd(dy, x, gain, mean, rstd, dres)
    dx, dg, ds = gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd, dres=dres)
    R.check({"dx": dx, "dgain": dg, "dshift": ds}, want)
    assert torch.equal(dx, gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd, dres=dres, dx=dres)[0])


@pytest.mark.parametrize("t", [F, B])
def test_offsets_past_32_bits(gt, t):
    """More than 2^31 elements: the last rows equal those of a call for them alone."""
    n, c, tail = 270000, 8008, 64
    x, gain, shift = _rows(n, c, t, 1), _vec(c, 2, 0.1, 1.0), _vec(c, 3, 0.02)
    y, mean, rstd = gt.gt_layer_norm_fwd(x, gain, shift)
    R.check({"y": y[-tail:], "mean": mean[-tail:], "rstd": rstd[-tail:]}, R.ln_fwd(x[-tail:], gain, shift, 1e-5, t))
    one = gt.gt_layer_norm_bwd(y, x, gain, mean, rstd)[0]
    part = gt.gt_layer_norm_bwd(y[-tail:], x[-tail:], gain, mean[-tail:], rstd[-tail:])[0]
    assert torch.equal(one[-tail:], part)


def test_constant_and_nonfinite_rows(gt):
    """A constant row has variance 0: y is the shift.  A NaN or an infinity stays in its own row of
    y and dx, and in dgain's columns."""
    n, c = 12, 100
    x, gain, shift = _rows(n, c, F, 1), _vec(c, 2, 0.1, 1.0), _vec(c, 3, 0.02)
    x[3] = 2.0
    x[5, 7] = float("nan")
    x[8, 99] = float("inf")
    y, mean, rstd = gt.gt_layer_norm_fwd(x, gain, shift, eps=1e-5)
    assert torch.equal(y[3], shift) and float(mean[3]) == 2.0
    fine = [i for i in range(n) if i not in (5, 8)]
    R.check({"y": y[fine]}, R.ln_fwd(x[fine], gain, shift, 1e-5, F))
    assert y[5].isnan().all() and y[8].isnan().all()
    dy = _rows(n, c, F, 4)
    dx, dg, ds = gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd)
    R.check({"dx": dx[fine]}, R.ln_bwd(dy[fine], x[fine], gain, mean[fine], rstd[fine], None) )
    assert dg.isnan().all() and not ds.isnan().any()


def test_gradient_against_differences(gt):
    """dx, dgain and dshift against central differences of the forward in fp64 of the same formula."""
    n, c = 6, 48
    x, gain, shift, dy = _rows(n, c, F, 1), _vec(c, 2, 0.1, 1.0), _vec(c, 3, 0.02), _rows(n, c, F, 4)
    _, mean, rstd = gt.gt_layer_norm_fwd(x, gain, shift)
    dx, dg, ds = (R.d(t) for t in gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd))
    xd, gd, sd, dyd = R.d(x), R.d(gain), R.d(shift), R.d(dy)

    def loss(x_, g_, s_):
        mu = x_.mean(1, keepdim=True)
        return float((((x_ - mu) * (((x_ - mu) ** 2).mean(1, keepdim=True) + 1e-5) ** -0.5 * g_ + s_) * dyd).sum())

    h = 1e-5
    for i, j in ((0, 0), (3, 17), (5, 47)):
        e = torch.zeros_like(xd)
        e[i, j] = h
        assert abs((loss(xd + e, gd, sd) - loss(xd - e, gd, sd)) / (2 * h) - float(dx[i, j])) < 1e-5
        v = torch.zeros_like(gd)
        v[j] = h
        assert abs((loss(xd, gd + v, sd) - loss(xd, gd - v, sd)) / (2 * h) - float(dg[j])) < 1e-5
        assert abs((loss(xd, gd, sd + v) - loss(xd, gd, sd - v)) / (2 * h) - float(ds[j])) < 1e-5


def test_in_place_residual_gradient(gt):
    n, c = 40, 200
    x, gain, shift, dy, dres = _rows(n, c, B, 1), _vec(c, 2, 0.1, 1.0), _vec(c, 3, 0.02), _rows(n, c, B, 4), _rows(n, c, B, 5)
    _, mean, rstd = gt.gt_layer_norm_fwd(x, gain, shift)
    want, _, _ = gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd, dres=dres)
    buf = dres.clone()
    got, _, _ = gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd, dres=buf, dx=buf)
    assert got is buf and torch.equal(got, want)


def test_streams_and_graph(gt):
    """On a side stream, and captured once and replayed on new inputs, as an eager call gives."""
    n, c = 500, 320
    x, gain, shift, dy = _rows(n, c, B, 1), _vec(c, 2, 0.1, 1.0), _vec(c, 3, 0.02), _rows(n, c, B, 4)

    def both(stream=None):
        y, mean, rstd = gt.gt_layer_norm_fwd(x, gain, shift, stream=stream)
        return (y, *gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd, stream=stream))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    x.copy_(_rows(n, c, B, 11))
    dy.copy_(_rows(n, c, B, 14))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, both()))


@pytest.mark.parametrize("n,c,t", [(300, 64, F), (41, 1000, B), (20, 8192, F)])
def test_workspace_of_any_16_byte_alignment(gt, n, c, t):
    """A workspace 16 bytes past a 32-byte boundary serves as any other."""
    x, gain, shift, dy = _rows(n, c, t, 1), _vec(c, 2, 0.1, 1.0), _vec(c, 3, 0.02), _rows(n, c, t, 4)
    _, mean, rstd = gt.gt_layer_norm_fwd(x, gain, shift)
    need = gt.gt_layer_norm_workspace_size(n, c)
    buf = torch.full((need + 64,), 7, dtype=torch.uint8, device="cuda")
    got = gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd, workspace=buf[16:16 + need])
    assert all(torch.equal(a, b) for a, b in zip(got, gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd)))
    assert (buf[:16] == 7).all() and (buf[16 + need:] == 7).all()


@pytest.mark.parametrize("pad,offset", [(0, 0), (16, 0), (4, 4), (8, 8), (5, 0), (0, 1)])
@pytest.mark.parametrize("n,c,t", [(700, 64, F), (700, 64, B), (6000, 512, B), (2500, 1000, F), (900, 4096, B), (350, 8192, F)])
def test_residual_gradient_in_place_at_every_access(gt, n, c, t, pad, offset):
    """dres and dx one buffer, in rows of 32-byte, 16-byte and single-element accesses, several turns of a CTA."""
    x, gain, shift, dy = _rows(n, c, t, 1), _vec(c, 2, 0.1, 1.0), _vec(c, 3, 0.02), _rows(n, c, t, 4)
    _, mean, rstd = gt.gt_layer_norm_fwd(x, gain, shift)
    buf = _rows(n, c, t, 5, pad, offset)
    kept = buf.clone()
    want = gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd, dres=kept, dx=_rows(n, c, t, 6, pad, offset))
    got = gt.gt_layer_norm_bwd(dy, x, gain, mean, rstd, dres=buf, dx=buf)
    assert got[0] is buf and all(torch.equal(a, b) for a, b in zip(got, want))
    R.check({"dx": buf}, R.ln_bwd(dy, x, gain, mean, rstd, kept))


def test_more_rows_than_32_bits_count_are_refused(gt):
    """2^32 + 5 rows: not the call of 5 rows that the low 32 bits would make."""
    x, one = torch.empty((1 << 32) + 5, 1, dtype=B, device="cuda"), torch.ones(1, device="cuda")
    stats = torch.empty(1, device="cuda").expand(x.shape[0])
    with pytest.raises(ValueError, match="rows"):
        gt.gt_layer_norm_fwd(x, one, one)
    with pytest.raises(ValueError, match="rows"):
        gt.gt_layer_norm_bwd(x, x, one, stats, stats)
    with pytest.raises(ValueError, match="rows"):
        gt.gt_linear_fwd(x, torch.ones(1, 1, dtype=B, device="cuda"))


@pytest.mark.parametrize("c", [64, 512])
@pytest.mark.parametrize("t", [F, B])
def test_column_sums_of_many_rows(gt, c, t):
    """dgain and dshift of many rows of positive terms (mean 0, rstd 1, dy and x positive): the additions of a thread, of
    its CTA's row groups and of the partial rows, half a unit each at most, and one rounding of the product.  64 features:
    304 CTAs of 64 rows at a time make 54 turns of 2 rows, then 32, 10 and 32 additions; 512: 152 CTAs of 16 rows in fp32, 108 turns
    of 4 and 4 + 5 + 32, and 304 of 8 in bf16, 108 of 2 and 4 + 10 + 32."""
    n = 1 << (20 if c == 64 else 18)
    adds = 185 if c == 64 else 476 if t == F else 265
    x, dy = _rows(n, c, t, 1).abs(), _rows(n, c, t, 2).abs()
    mean, rstd = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    dx, dg, ds = gt.gt_layer_norm_bwd(dy, x, torch.ones(c, device="cuda"), mean, rstd)
    for got, want in ((dg, (dy.double() * x.double()).sum(0)), (ds, dy.double().sum(0))):
        assert float(((got.double() - want).abs() / want).max()) <= adds * R.U32
