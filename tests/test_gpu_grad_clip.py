"""Gradient norm and clipping on the GPU against fp64."""
import math

import pytest
import torch

import cross_ref as X
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


def _grads(sizes, types, seed=1, std=0.02):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std * (1 + i % 5)).to(types[i % len(types)])
            for i, n in enumerate(sizes)]


def _check(gt, grads, max_norm, types=None):
    types = types or [g.dtype for g in grads]
    out = [torch.full_like(g, 7.0, dtype=t) for g, t in zip(grads, types)]
    before = [g.clone() for g in grads]
    norm = gt.gt_grad_clip(grads, max_norm, out=out)
    want = X.clip(grads, max_norm, types)
    R.check({"norm": norm, **{f"out{i}": o for i, o in enumerate(out)}}, want)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    again = [torch.empty_like(o) for o in out]
    assert torch.equal(gt.gt_grad_clip(gt.gt_tensor_list(grads, again), max_norm), norm)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    if types == [g.dtype for g in grads]:      # in place: the same values
        assert torch.equal(gt.gt_grad_clip(before, max_norm), norm)
        assert all(torch.equal(a, b) for a, b in zip(out, before))


SIZES = [[1], [2048], [2049, 1, 7], [5, 0, 31, 4096, 100000, 3], [64] * 300, [17] * 256, [1000] * 257,
         [0, 0, 5], [3000001, 12]]


@pytest.mark.parametrize("types", [[F], [B], [F, B, B]])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm_and_clip(gt, sizes, types):
    grads = _grads(sizes, types)
    norm = math.sqrt(math.fsum(float((R.d(g) ** 2).sum()) for g in grads))
    for limit in (norm / 3, norm * 2, math.inf, 0.0):
        _check(gt, grads, limit)


@pytest.mark.parametrize("gtype,otype", [(F, B), (B, F)])
def test_other_type_out(gt, gtype, otype):
    grads = _grads([5000, 33, 2048, 1], [gtype])
    for limit in (0.01, 1e9):
        _check(gt, grads, limit, [otype] * len(grads))


def test_unaligned_and_transposed(gt):
    base = _grads([9001], [F])[0]
    wide = _grads([5000], [B], seed=3)[0]
    t = _grads([96 * 40], [F], seed=4)[0].view(96, 40).t()
    _check(gt, [base[1:8001], wide[3:4000], t, base[8003:9000]], 0.1)
    with pytest.raises(ValueError, match="piece of memory"):
        gt.gt_grad_clip([base.view(-1)[::2]], 1.0)


@pytest.mark.parametrize("size", [1e-30, 1e-22, 3e-13, 1e15, 2e19, 1e30])
def test_the_whole_range_of_fp32(gt, size):
    """Squares below the smallest and above the largest fp32 number."""
    grads = [g / 0.02 * size for g in _grads([3000, 5, 70000], [F])]
    grads[1].zero_()
    _check(gt, grads, size)
    _check(gt, [g.to(B) for g in grads], size)


def test_small_beside_large(gt):
    grads = [torch.full((4096,), 1e-24, device="cuda"), torch.full((10,), 1e-3, device="cuda"),
             torch.zeros(2048, device="cuda"), torch.full((4096,), 1e-21, device="cuda")]
    _check(gt, grads, 1e-4)
    _check(gt, [grads[0], grads[3]], 1e-22)


def test_an_output_listed_twice_is_refused(gt):
    g = _grads([50], [F])[0]
    with pytest.raises(ValueError, match="twice"):
        gt.gt_grad_clip([g, g], 1.0)
    norm = gt.gt_grad_clip([g, g], 1.0, out=[torch.empty_like(g) for _ in range(2)])      # two outputs: it counts twice
    R.check({"norm": norm}, X.clip([g, g], 1.0, [F, F]))


def test_nonfinite(gt):
    for bad in (math.nan, math.inf):
        g = _grads([3000, 40], [F])
        g[1][7] = bad
        keep = [t.clone() for t in g]
        norm = gt.gt_grad_clip(g, math.inf)
        assert math.isnan(float(norm)) if math.isnan(bad) else math.isinf(float(norm))
        assert torch.equal(g[0], keep[0]) and torch.equal(g[1][:7], keep[1][:7])      # only measured
        gt.gt_grad_clip(g, 1.0)
        if math.isnan(bad):
            assert all(t.isnan().all() for t in g)
        else:
            assert (g[0] == 0).all() and g[1][7].isnan() and (g[1][:7] == 0).all()


def test_no_element_past_the_end(gt):
    for n in (1, 7, 8, 2047, 2049):
        buf = torch.full((n + 64,), 3.0, device="cuda")
        gt.gt_grad_clip([buf[:n]], 0.5)
        assert (buf[n:] == 3.0).all() and (buf[:n] < 3.0).all()


def test_offsets_past_32_bits(gt):
    """One bf16 tensor of more than 2^31 elements."""
    n = 2 ** 31 + 4099
    g = torch.zeros(n, dtype=B, device="cuda")
    g[-1], g[0], g[2 ** 31 - 1] = 3.0, 4.0, 12.0
    norm = gt.gt_grad_clip([g], 1.3)
    assert float(norm) == 13.0
    assert [float(x) for x in (g[-1], g[0], g[2 ** 31 - 1])] == [float(torch.tensor(v * 0.1, dtype=F).to(B))
                                                                 for v in (3.0, 4.0, 12.0)]
    assert int(torch.count_nonzero(g)) == 3


def test_streams_and_graphs(gt):
    grads = _grads([5000, 300, 70001], [F, B])
    out = [torch.empty_like(g) for g in grads]
    handle = gt.gt_tensor_list(grads, out)
    want = gt.gt_grad_clip(handle, 0.3).clone()
    ref = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for o in out:
        o.zero_()
    side.wait_stream(torch.cuda.current_stream())
    norm = gt.gt_grad_clip(handle, 0.3, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, ref))
    # two graphs that share a workspace and run one after the other
    work = torch.empty(gt.gt_grad_clip_workspace_size(3), dtype=torch.uint8, device="cuda")
    n1, n2 = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    graphs = []
    for n, limit in ((n1, 0.3), (n2, math.inf)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gt.gt_grad_clip(handle, limit, norm=n, workspace=work)
        graphs.append(graph)
    for o in out:
        o.zero_()
    for graph in graphs * 2:
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(n1, want) and torch.equal(n2, want)
    assert all(torch.equal(o, g) for o, g in zip(out, grads))      # the second only copies
    grads[0].mul_(2.0)                                             # a replay reads what is there then
    graphs[0].replay()
    R.check({"norm": n1}, X.clip(grads, 0.3, [g.dtype for g in grads]))


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("size,limit", [(1e30, 1e-16), (1e36, 1.0), (1e36, 1e-3), (1e36, 1e-12), (1e38, 1.0), (1e38, 1e-3),
                                        (3e38, 1e-20)])
def test_large_gradients_and_a_small_limit(gt, size, limit, t):
    """max_norm / norm below the smallest normal fp32 number, or below all of them; the results are ordinary numbers."""
    for n in (1, 4096, 70001):
        g = (torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda") * 0.5 + 0.5) * size
        grads = [g.to(t), (g[:n // 2 + 1] * -1e-2).to(t)]
        # past fp32's range the norm reads infinity; the gradients are scaled by what it is
        fits = float(X.clip(grads, limit, [t, t])["norm"][0]) <= torch.finfo(F).max
        for types in ([F, F], [B, B]):
            out = [torch.full_like(x, 7.0, dtype=y) for x, y in zip(grads, types)]
            norm = gt.gt_grad_clip(grads, limit, out=out)
            ref = X.clip(grads, limit, types)
            assert fits or math.isinf(float(norm))
            got = {"norm": norm} if fits else {}
            R.check({**got, "out0": out[0], "out1": out[1]}, {m: ref[m] for m in (*got, "out0", "out1")}, floor=0.0)


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("n", [1, 100, 1024, 70001])
def test_the_norm_within_its_own_roundings(gt, n, t):
    """A lane adds 32 squares of positive sign in four chains of 8 and joins these in two steps: 10 roundings at most, half
    of that after the root.  A lane's units are added in two fp32 words and the rest in fp64 (2^-40 and less), then the norm
    is rounded, or the factor and each product."""
    grads = _grads([n, n // 3 + 1], [t])
    limit = 0.5 * math.sqrt(math.fsum(float((R.d(g) ** 2).sum()) for g in grads))
    out = [torch.empty_like(g) for g in grads]
    norm = gt.gt_grad_clip(grads, limit, out=out)
    ref, off = X.clip(grads, limit, [t, t]), (5 + 2.0 ** -10) * R.U32
    bounds = {"norm": off + R.U32, "out0": off + 2 * R.U32 + (R.half_step(t) if t == B else 0.0)}
    bounds["out1"] = bounds["out0"]
    R.check({"norm": norm, "out0": out[0], "out1": out[1]}, {m: (ref[m][0], ref[m][0].abs() * bounds[m]) for m in bounds})
