"""Cross attention on the GPU against fp64, within derived bounds."""
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


def _t(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _off(*cuts):
    return torch.tensor(cuts, dtype=torch.int32, device="cuda")


def _both(gt, q, k, v, q_off=None, kv_off=None, mask=None, scale=None, out=None):
    """Forward and backward against the reference; returns the results."""
    o, lse = gt.gt_cross_attn_fwd(q, k, v, q_off, kv_off, mask, scale, out=out)
    rows = slice(None) if q_off is None else slice(int(q_off[0]), int(q_off[-1]))
    keys = slice(None) if kv_off is None else slice(int(kv_off[0]), int(kv_off[-1]))
    ref = X.attn_fwd(q, k, v, q_off, kv_off, mask, scale)
    empty = ref["lse"][0][:, rows] == -math.inf
    assert ((lse[:, rows].cpu() == -math.inf) == empty).all()
    assert (o[rows].cpu()[empty.t()] == 0).all()
    R.check({"o": o[rows], "lse": lse[:, rows].cpu().masked_fill(empty, 0)},
            {"o": tuple(t[rows] for t in ref["o"]),
             "lse": (ref["lse"][0][:, rows].masked_fill(empty, 0), ref["lse"][1][:, rows])})
    do = _t(q.shape, q.dtype, 77)
    saved = ref["o"][0].to(q.dtype).cuda()          # what the forward would have kept, exactly rounded
    lse64 = ref["lse"][0].float().cuda()
    got = gt.gt_cross_attn_bwd(q, k, v, saved, do, lse64, q_off, kv_off, mask, scale)
    want = X.attn_bwd(q, k, v, saved, do, lse64, q_off, kv_off, mask, scale)
    for name, t, part in zip(("dq", "dk", "dv"), got, (rows, keys, keys)):
        R.check({name: t[part]}, {name: tuple(x[part] for x in want[name])})
    return (o, lse, *got)


# one row to many, odd counts, every head width's layout, shared heads, splits over either side
SHAPES = [(1, 1, 1, 1, 8), (1, 512, 8, 8, 8), (3, 5, 2, 1, 16), (65, 129, 4, 4, 32), (130, 200, 2, 2, 64), (77, 300, 6, 2, 24),
          (129, 65, 3, 1, 40), (40, 1000, 8, 1, 128), (200, 131, 4, 2, 96), (64, 64, 1, 1, 72), (1, 3000, 4, 1, 64),
          (2000, 3, 2, 2, 16), (33, 257, 5, 5, 120), (5, 70, 64, 1, 16), (3, 66, 48, 1, 8), (700, 1100, 2, 1, 128)]


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("nq,nk,h,hk,c", SHAPES)
def test_forward_and_backward(gt, nq, nk, h, hk, c, t):
    q, k, v = _t((nq, h, c), t, 1), _t((nk, hk, c), t, 2), _t((nk, hk, c), t, 3)
    first = _both(gt, q, k, v)
    do = _t(q.shape, t, 77)
    again = gt.gt_cross_attn_bwd(q, k, v, first[0], do, first[1])
    assert all(torch.equal(a, b) for a, b in zip(gt.gt_cross_attn_bwd(q, k, v, first[0], do, first[1]), again))
    assert all(torch.equal(a, b) for a, b in zip(gt.gt_cross_attn_fwd(q, k, v), first))


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("c", [1, 2, 7, 17, 33, 63, 65, 100, 127])
def test_odd_widths(gt, c, t):
    _both(gt, _t((70, 4, c), t, 1), _t((140, 2, c), t, 2), _t((140, 2, c), t, 3))


BATCHES = [
    ([0, 5, 9], [0, 70, 71]),
    ([0, 0, 130, 131], [0, 64, 300, 301]),            # a sequence without queries
    ([0, 3, 64, 200], [0, 0, 129, 130]),              # one without keys
    ([0, 0, 0, 7, 7], [0, 0, 9, 9, 300]),
    ([2, 40, 41, 170], [3, 131, 259, 260]),           # rows in front of the first sequence and behind the last
    (list(range(0, 34)), [9 * i for i in range(34)]),
    ([0, 128, 256, 384], [0, 128, 256, 384]),
]


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("h,hk,c", [(4, 4, 16), (6, 2, 64), (4, 1, 128)])
@pytest.mark.parametrize("cq,ck", BATCHES, ids=str)
def test_packed_sequences(gt, cq, ck, h, hk, c, t):
    nq, nk = cq[-1] + 5, ck[-1] + 3
    q, k, v = _t((nq, h, c), t, 1), _t((nk, hk, c), t, 2), _t((nk, hk, c), t, 3)
    # what belongs to no sequence is not a number, and stays out of every result
    for x, cuts in ((q, cq), (k, ck), (v, ck)):
        x[:cuts[0]] = math.nan
        x[cuts[-1]:] = math.inf
    out = torch.full_like(q, 7.0)
    _both(gt, q, k, v, _off(*cq), _off(*ck), out=out)
    assert (out[:cq[0]] == 7).all() and (out[cq[-1]:] == 7).all()
    do, lse = _t(q.shape, t, 5), torch.full((h, nq), 7.0, device="cuda")
    o, lse = gt.gt_cross_attn_fwd(q, k, v, _off(*cq), _off(*ck), lse=lse)
    assert (lse[:, :cq[0]] == 7).all() and (lse[:, cq[-1]:] == 7).all()
    do[:cq[0]], do[cq[-1]:], lse[:, cq[-1]:] = math.nan, math.inf, math.nan
    grads = [torch.full_like(x, 7.0) for x in (q, k, v)]
    gt.gt_cross_attn_bwd(q, k, v, o, do, lse, _off(*cq), _off(*ck), dq=grads[0], dk=grads[1], dv=grads[2])
    for g, cuts in zip(grads, (cq, ck, ck)):
        assert (g[:cuts[0]] == 7).all() and (g[cuts[-1]:] == 7).all() and g[cuts[0]:cuts[-1]].isfinite().all()


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("h,hk,c", [(4, 4, 16), (6, 2, 64), (4, 2, 128)])
@pytest.mark.parametrize("keep", [0.0, 0.02, 0.5, 0.97])
def test_hidden_keys(gt, keep, h, hk, c, t):
    """Hidden keys that are not numbers, whole tiles of them, and sequences without any other."""
    cq, ck = [0, 40, 200, 207], [0, 400, 900, 1003]
    q, k, v = _t((207, h, c), t, 1), _t((1003, hk, c), t, 2), _t((1003, hk, c), t, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    mask = torch.rand(1003, generator=g, device="cuda") < keep
    mask[500:700] = False
    k[~mask], v[~mask] = math.nan, math.inf
    for offs in ((_off(*cq), _off(*ck)), (None, None)):
        r = _both(gt, q, k, v, *offs, mask=mask)
        assert (r[3][~mask] == 0).all() and (r[4][~mask] == 0).all()
        same = gt.gt_cross_attn_fwd(q, k, v, *offs, mask.to(torch.uint8) * 3)
        assert torch.equal(same[0], r[0])


@pytest.mark.parametrize("t", [F, B])
def test_padded_batch(gt, t):
    """[batch][longest] rows with hidden padding equal the packed sequences, a length of 0 among them."""
    lens, top, h, hk, c, nq = [50, 0, 128, 1, 77], 128, 4, 2, 64, 9
    k, v = _t((5 * top, hk, c), t, 2), _t((5 * top, hk, c), t, 3)
    mask = torch.cat([torch.arange(top, device="cuda") < n for n in lens])
    k[~mask], v[~mask] = math.nan, math.nan
    q = _t((5 * nq, h, c), t, 1)
    qo = _off(*range(0, 5 * nq + 1, nq))
    a = gt.gt_cross_attn_fwd(q, k, v, qo, _off(*range(0, 5 * top + 1, top)), mask)
    ko = _off(*[sum(lens[:i]) for i in range(6)])
    b = gt.gt_cross_attn_fwd(q, k[mask].contiguous(), v[mask].contiguous(), qo, ko)
    for x, y in zip(a, b):
        assert torch.equal(x.isinf(), y.isinf())
        # (tiles and parts fall differently: fp32 sums in another order, and a bf16 step of the results)
        x, y = x.float().nan_to_num(neginf=0.0), y.float().nan_to_num(neginf=0.0)
        assert float((x - y).abs().max()) <= (2e-5 if t == F else 2.0 ** -6)
    assert (a[0][nq:2 * nq] == 0).all() and (a[1][:, nq:2 * nq] == -math.inf).all()


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("c", [16, 64, 72, 128, 20])
def test_strides_and_alignment(gt, c, t):
    nq, nk, h, hk = 67, 150, 4, 2
    fused = _t((nk, 2 * hk * c), t, 2)
    k, v = fused[:, :hk * c].unflatten(1, (hk, c)), fused[:, hk * c:].unflatten(1, (hk, c))
    q = _t((h, nq, c), t, 1).transpose(0, 1)                        # heads first
    _both(gt, q, k, v)
    odd = _t((nk, hk * c + 3), t, 4)[:, 1:1 + hk * c].unflatten(1, (hk, c))      # any base, any row stride
    _both(gt, _t((nq + 1, h, c + 1), t, 5)[1:, :, 1:], odd, v)
    shared = _t((nk, 1, c), t, 6).expand(nk, hk, c)                 # a stride of 0: the heads' gradients still apart
    _both(gt, q, shared, odd)
    _both(gt, q, _t((1, hk, c), t, 7).expand(nk, hk, c), v)         # one key many times
    # results as slices of wider rows, the rest as it was
    wq, wk = (torch.full((n, heads * c + 5), 7.0, dtype=t, device="cuda") for n, heads in ((nq, h), (nk, hk)))
    dq, dk = wq[:, 2:2 + h * c].unflatten(1, (h, c)), wk[:, 1:1 + hk * c].unflatten(1, (hk, c))
    o, lse = gt.gt_cross_attn_fwd(q, k, v)
    assert torch.equal(gt.gt_cross_attn_fwd(q, k, v, out=dq)[0], o)
    assert (wq[:, :2] == 7).all() and (wq[:, 2 + h * c:] == 7).all()
    do = _t(q.shape, t, 9)
    want = gt.gt_cross_attn_bwd(q, k, v, o, do, lse)
    got = gt.gt_cross_attn_bwd(q, k, v, o, do, lse, dq=dq, dk=dk)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert (wq[:, :2] == 7).all() and (wk[:, :1] == 7).all() and (wk[:, 1 + hk * c:] == 7).all()


@pytest.mark.parametrize("t", [F, B])
def test_scores_of_any_size(gt, t):
    """Large scores in rising, falling and alternating order (raised bases), equal ones, tiny ones."""
    nq, nk, c = 40, 700, 64
    v = _t((nk, 1, c), t, 3)
    ramp = torch.linspace(-30, 30, nk, device="cuda")
    for row in (ramp, -ramp, ramp * torch.where(torch.arange(nk, device="cuda") % 2 == 0, 1, -1), ramp * 0, ramp * 1e-20):
        k = torch.zeros(nk, 1, c, device="cuda")
        k[:, 0, 0] = row
        q = torch.zeros(nq, 1, c, device="cuda")
        q[:, 0, 0] = torch.linspace(-3, 3, nq, device="cuda")
        _both(gt, q.to(t), k.to(t), v, scale=1.0)


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("c", [64, 128])
def test_raised_bases_over_many_tiles(gt, c, t):
    """Scores that rise by more than the slack of a base from tile to tile, or jump late, in sequences of many tiles whose
    heads fill the SMs, so that one CTA sees all of them."""
    batch, lq, lk, h = 40, 33, 700, 8
    offs = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    v = _t((batch * lk, h, c), t, 3)
    q, k = torch.zeros(batch * lq, h, c, device="cuda"), torch.zeros(batch * lk, h, c, device="cuda")
    q[:, :, 0] = torch.linspace(0.5, 3, batch * lq, device="cuda")[:, None]
    for row in (torch.linspace(-60, 60, lk), torch.where(torch.arange(lk) == lk - 2, 40.0, torch.linspace(3, -3, lk))):
        k[:, :, 0] = row.cuda().repeat(batch)[:, None]
        _both(gt, q.to(t), k.to(t), v, offs * lq, offs * lk, scale=1.0)


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("nk", [31, 47, 48, 63, 64, 65, 95, 96, 97, 127, 128, 191, 192, 193, 289])
@pytest.mark.parametrize("c", [40, 64, 128])
def test_ends_of_tiles(gt, nk, c, t):
    """Keys that fill tiles of any of the kernels' sizes, all but one of one, or one more."""
    _both(gt, _t((35, 2, c), t, 1), _t((nk, 2, c), t, 2), _t((nk, 2, c), t, 3))


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("scale", [1e-30, 0.01, 2.5])
def test_scales(gt, scale, t):
    _both(gt, _t((50, 2, 32), t, 1), _t((200, 2, 32), t, 2), _t((200, 2, 32), t, 3), scale=scale)


@pytest.mark.parametrize("t", [F, B])
def test_nonfinite_values_stay_where_they_belong(gt, t):
    """A NaN in a query spoils its own rows only; one in a value, every query of its sequence and no other."""
    q, k, v = _t((30, 2, 16), t, 1), _t((90, 2, 16), t, 2), _t((90, 2, 16), t, 3)
    qo, ko = _off(0, 10, 30), _off(0, 50, 90)
    clean = gt.gt_cross_attn_fwd(q, k, v, qo, ko)[0]
    q2, v2 = q.clone(), v.clone()
    q2[3, 1, 0] = math.nan
    o = gt.gt_cross_attn_fwd(q2, k, v, qo, ko)[0]
    assert o[3, 1].isnan().all()
    o[3, 1] = clean[3, 1]
    assert torch.equal(o, clean)
    v2[60, 0, 5] = math.nan
    o = gt.gt_cross_attn_fwd(q, k, v2, qo, ko)[0]
    assert o[10:, 0, 5].isnan().all()
    o[10:, 0, 5] = clean[10:, 0, 5]
    assert torch.equal(o, clean)


def test_gradients_by_differences(gt):
    qo, ko, mask = _off(0, 3, 7), _off(0, 6, 11), torch.ones(11, dtype=torch.bool, device="cuda")
    mask[4] = False
    q, k, v, w = _t((7, 4, 5), F, 1), _t((11, 2, 5), F, 2), _t((11, 2, 5), F, 3), _t((7, 4, 5), F, 4)

    def loss(q, k, v):
        return float((X.attn_fwd(q, k, v, qo, ko, mask)["o"][0] * R.d(w)).sum())

    o, lse = gt.gt_cross_attn_fwd(q, k, v, qo, ko, mask)
    grads = gt.gt_cross_attn_bwd(q, k, v, o, w, lse, qo, ko, mask)
    args = [t.double() for t in (q, k, v)]
    for i, got in enumerate(grads):
        for at in range(0, args[i].numel(), 5):
            up, down = ([t.clone() for t in args] for _ in range(2))
            up[i].view(-1)[at] += 1e-5
            down[i].view(-1)[at] -= 1e-5
            want = (loss(*up) - loss(*down)) / 2e-5
            # the difference's own error: third derivatives x 1e-10, fp64 rounding / 1e-5; the kernels' fp32
            assert abs(float(got.view(-1)[at]) - want) <= 2e-5 * max(1.0, abs(want)), (i, at)


@pytest.mark.parametrize("t", [F, B])
def test_offsets_outside_the_rows_are_cut(gt, t):
    q, k, v = _t((60, 2, 64), t, 1), _t((300, 2, 64), t, 2), _t((300, 2, 64), t, 3)
    do = _t(q.shape, t, 4)
    good, wide = (_off(0, 20, 60), _off(0, 100, 300)), (_off(-7, 20, 2 ** 31 - 1), _off(-2 ** 31, 100, 1000))
    a, b = gt.gt_cross_attn_fwd(q, k, v, *good), gt.gt_cross_attn_fwd(q, k, v, *wide)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    a, b = (gt.gt_cross_attn_bwd(q, k, v, a[0], do, a[1], *offs) for offs in (good, wide))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("t", [F, B])
def test_many_short_sequences(gt, t):
    """More sequences than one look at the offsets covers, most of them of no row, one or two."""
    n = 1500
    lq, lk = [(i * 7) % 3 for i in range(n)], [(i * 5) % 4 for i in range(n)]
    lq[700], lk[700] = 300, 200
    cq, ck = ([0] + torch.tensor(x).cumsum(0).tolist() for x in (lq, lk))
    _both(gt, _t((cq[-1], 4, 32), t, 1), _t((ck[-1], 2, 32), t, 2), _t((ck[-1], 2, 32), t, 3), _off(*cq), _off(*ck))


@pytest.mark.parametrize("t", [F, B])
def test_long_sides(gt, t):
    """Long keys for few queries, long queries for few keys: the split forms, against fp64 on some of the heads."""
    for nq, nk, h, hk, c in ((4, 20011, 4, 2, 64), (5003, 70, 2, 2, 32), (1, 9001, 16, 2, 128), (300, 4099, 1, 1, 16)):
        _both(gt, _t((nq, h, c), t, 1), _t((nk, hk, c), t, 2), _t((nk, hk, c), t, 3))


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("share", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("c", [5, 8, 16, 30, 64, 100, 128])
def test_single_queries(gt, c, share, t):
    """The next token of each of some decoders: ragged keys, an empty side, a sequence with more queries than most."""
    ck = [0, 0, 1, 70, 571, 640, 2000]
    cq = [0, 1, 2, 3, 3, 4, 6 + 2]
    hk = 2
    q, k, v = _t((cq[-1], share * hk, c), t, 1), _t((2004, hk, c), t, 2), _t((2004, hk, c), t, 3)
    mask = torch.arange(2004, device="cuda") % 7 != 3
    k[2000:], v[2000:], k[~mask] = math.nan, math.inf, math.nan
    qo, ko = _off(*cq), _off(*ck)
    o, lse = gt.gt_cross_attn_fwd(q, k, v, qo, ko, mask)
    ref = X.attn_fwd(q, k, v, qo, ko, mask)
    empty = ref["lse"][0] == -math.inf
    assert ((lse.cpu() == -math.inf) == empty).all() and bool(empty[:, 0].all()) and (o.cpu()[empty.t()] == 0).all()
    R.check({"o": o, "lse": lse.cpu().masked_fill(empty, 0)},
            {"o": ref["o"], "lse": (ref["lse"][0].masked_fill(empty, 0), ref["lse"][1])})
    assert all(torch.equal(a, b) for a, b in zip(gt.gt_cross_attn_fwd(q, k, v, qo, ko, mask), (o, lse)))


def test_offsets_past_32_bits(gt):
    """Keys and values of more than 2^31 elements each: the last sequence as a call for it alone."""
    nk, hk, c, tail = 140001, 128, 128, 700
    k, v = _t((nk, hk, c), B, 2), _t((nk, hk, c), B, 3)
    q, do = _t((40, hk, c), B, 1), _t((40, hk, c), B, 4)
    ko, qo = _off(0, nk - tail, nk), _off(0, 20, 40)
    o, lse = gt.gt_cross_attn_fwd(q, k, v, qo, ko)
    alone = gt.gt_cross_attn_fwd(q[20:], k[-tail:], v[-tail:])
    assert float((o[20:].float() - alone[0].float()).abs().max()) <= 2.0 ** -6
    assert float((lse[:, 20:] - alone[1]).abs().max()) <= 1e-5
    dq, dk, dv = gt.gt_cross_attn_bwd(q, k, v, o, do, lse, qo, ko)
    one = gt.gt_cross_attn_bwd(q[20:], k[-tail:], v[-tail:], o[20:], do[20:], lse[:, 20:].contiguous())
    for a, b in zip((dq[20:], dk[-tail:], dv[-tail:]), one):
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -6 * max(1.0, float(b.float().abs().max()))


def test_streams_graphs_and_shared_workspaces(gt):
    q, k, v, do = _t((300, 4, 64), B, 1), _t((900, 2, 64), B, 2), _t((900, 2, 64), B, 3), _t((300, 4, 64), B, 4)
    o, lse = gt.gt_cross_attn_fwd(q, k, v)
    want = (o, lse, *gt.gt_cross_attn_bwd(q, k, v, o, do, lse))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = gt.gt_cross_attn_fwd(q, k, v, stream=side)
    got = (*a, *gt.gt_cross_attn_bwd(q, k, v, o, do, lse, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    work = torch.empty(max(gt.gt_cross_attn_workspace_size(1, 300, 900, 4, 2, 64, backward=b) for b in (False, True)),
                       dtype=torch.uint8, device="cuda")
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        fwd = gt.gt_cross_attn_fwd(q, k, v, workspace=work)
    with torch.cuda.graph(two):
        bwd = gt.gt_cross_attn_bwd(q, k, v, *(fwd[0], do, fwd[1]), workspace=work)
    for _ in range(3):
        work.fill_(255)
        one.replay()
        two.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, (*fwd, *bwd)))
    gt.gt_check_device_status()


def test_two_calls_at_once(gt):
    """Two streams, a workspace each."""
    q, k, v = _t((500, 4, 64), B, 1), _t((3000, 4, 64), B, 2), _t((3000, 4, 64), B, 3)
    want = gt.gt_cross_attn_fwd(q, k, v)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [gt.gt_cross_attn_fwd(q, k, v, stream=streams[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(want, r))


@pytest.mark.parametrize("t", [F, B])
def test_a_step_of_a_cross_attention_layer(gt, t):
    """Projections, norm and rotation, attention, their backward and the clipping of all gradients, as one step runs
    them, against autograd of the same layer in fp64 on the GPU."""
    nq, nk, h, hk, c, width = 37, 150, 4, 2, 16, 48
    x, y = _t((nq, width), t, 1), _t((nk, width), t, 2)
    wq, wkv, wo = (_t(s, t, i, 0.15) for i, s in ((3, (width, h * c)), (4, (width, 2 * hk * c)), (5, (h * c, width))))
    gq, gk, f, do = _t((c,), F, 6) * 0.1 + 1, _t((c,), F, 7) * 0.1 + 1, torch.linspace(1, 0.01, c // 2, device="cuda"), _t((nq, width), t, 8)
    qo, ko = _off(0, 20, 37), _off(0, 90, 150)

    a, _ = gt.gt_linear_fwd(x, wq)
    b, _ = gt.gt_linear_fwd(y, wkv)
    qr, kr, vr = a.view(nq, h, c), b[:, :hk * c].unflatten(1, (hk, c)), b[:, hk * c:].unflatten(1, (hk, c))
    qn, kn = gt.gt_qk_norm_fwd(qr, kr, gq, gk, freq=f)
    o, lse = gt.gt_cross_attn_fwd(qn, kn, vr, qo, ko)
    do_, dwo, _ = gt.gt_linear_bwd(do, o.view(nq, h * c), wo, need_db=False)
    db = torch.empty_like(b)
    dqn, dkn, _ = gt.gt_cross_attn_bwd(qn, kn, vr, o, do_.view(nq, h, c), lse, qo, ko, dv=db[:, hk * c:].unflatten(1, (hk, c)))
    da, _, dgq, dgk = gt.gt_qk_norm_bwd(dqn, dkn, qr, kr, gq, gk, freq=f, dk=db[:, :hk * c].unflatten(1, (hk, c)))
    dx, dwq, _ = gt.gt_linear_bwd(da.view(nq, h * c), x, wq, need_db=False)
    dy, dwkv, _ = gt.gt_linear_bwd(db, y, wkv, need_db=False)
    grads = [dwq, dwkv, dwo, dgq, dgk]
    norm = gt.gt_grad_clip(grads, 0.5)

    leaves = [u.double().requires_grad_() for u in (x, y, wq, wkv, wo, gq, gk)]
    X_, Y_, WQ, WKV, WO, GQ, GK = leaves
    def rotate(u):
        ang = torch.arange(u.shape[0], device="cuda").double()[:, None] * f.double()
        cs, sn = ang.cos()[:, None], ang.sin()[:, None]
        p, r = u[..., :c // 2], u[..., c // 2:]
        return torch.cat((p * cs - r * sn, p * sn + r * cs), -1)
    def norm_of(u, g):
        return rotate(u * (u.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * g)
    Q = norm_of((X_ @ WQ).view(nq, h, c), GQ)
    KV = Y_ @ WKV
    K, V = norm_of(KV[:, :hk * c].reshape(nk, hk, c), GK), KV[:, hk * c:].reshape(nk, hk, c)
    outs = []
    for (i, j), (m, n) in (((0, 20), (0, 90)), ((20, 37), (90, 150))):
        s = torch.einsum("ihc,jhc->hij", Q[i:j], K[m:n].repeat_interleave(h // hk, 1)) / math.sqrt(c)
        outs.append(torch.einsum("hij,jhc->ihc", s.softmax(-1), V[m:n].repeat_interleave(h // hk, 1)))
    ((torch.cat(outs).reshape(nq, h * c) @ WO) * do.double()).sum().backward()
    total = math.sqrt(sum(float(u.grad.square().sum()) for u in leaves[2:]))
    # fp32: products and sums of up to 150 terms, a chain of seven of them; bf16: each of the chain's tensors is rounded,
    # 2^-8 of itself at most, and what follows carries that on: in norm, where the roundings are independent
    tol = 2e-5 if t == F else 12 * 2.0 ** -8
    assert abs(float(norm) - total) <= tol * total
    for got, leaf in zip((*grads, dx, dy), (*leaves[2:], X_, Y_)):
        want = leaf.grad * (0.5 / total if leaf is not X_ and leaf is not Y_ else 1.0)
        assert float((got.double() - want).norm()) <= tol * float(want.norm())


def test_query_and_head_rows_past_32_bits(gt):
    """More than 2^31 (query, head) rows on one key head, in fp32 of one channel: dO is 0 but for a few rows from both ends
    and the middle, against fp64 of these (what the others add is exactly 0)."""
    torch.cuda.empty_cache()
    nq, h, nk = 2 ** 25 + 1003, 64, 5
    q, k, v = _t((nq, h, 1), F, 1), _t((nk, 1, 1), F, 2), _t((nk, 1, 1), F, 3)
    rows = torch.tensor([0, 1, 77, 2 ** 24 - 1, 2 ** 24, 2 ** 25 - 1, 2 ** 25, 2 ** 25 + 63, nq - 2, nq - 1], device="cuda")
    do = torch.zeros(nq, h, 1, device="cuda")
    do[rows] = _t((rows.numel(), h, 1), F, 4)
    o, lse = gt.gt_cross_attn_fwd(q, k, v)
    R.check({"o": o[rows], "lse": lse[:, rows]}, X.attn_fwd(q[rows], k, v))
    dq, dk, dv = gt.gt_cross_attn_bwd(q, k, v, o, do, lse)
    want = X.attn_bwd(q[rows], k, v, o[rows], do[rows], lse[:, rows])
    R.check({"dq": dq[rows], "dk": dk, "dv": dv}, want)
    dq[rows] = 0
    assert int(torch.count_nonzero(dq)) == 0
    del q, do, o, lse, dq
    torch.cuda.empty_cache()


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("h,hk,c", [(4, 4, 8), (3, 1, 16), (3, 1, 40), (4, 2, 64), (3, 1, 128)])
@pytest.mark.parametrize("nq", [1, 37, 64, 131])
def test_infinities_in_visible_keys(gt, nq, h, hk, c, t):
    """Keys whose score is -infinity with every query weigh nothing, their gradients are 0, and whether the queries fill
    their tiles makes no difference; against the same call with those keys hidden."""
    q, k, v, do = _t((nq, h, c), t, 1), _t((200, hk, c), t, 2), _t((200, hk, c), t, 3), _t((nq, h, c), t, 4)
    q[..., 0] = q[..., 0].abs() + 1
    far = torch.zeros(200, dtype=torch.bool, device="cuda")
    far[[0, 77, 130, 199]] = True
    k[far, :, 0] = -math.inf
    cut = nq // 3
    for offs in ((None, None), (_off(0, cut, nq), _off(0, 90, 200))):
        o, lse = gt.gt_cross_attn_fwd(q, k, v, *offs)
        R.check({"o": o, "lse": lse}, X.attn_fwd(q, k, v, *offs, mask=~far))
        dq, dk, dv = gt.gt_cross_attn_bwd(q, k, v, o, do, lse, *offs)
        assert (dk[far] == 0).all() and (dv[far] == 0).all()
        want = X.attn_bwd(q, k, v, o, do, lse, *offs, mask=~far)
        # (channel 0 of dq is a sum with 0 x infinity in it, in the formula too)
        R.check({"dk": dk, "dv": dv, "dq": dq[..., 1:]},
                {"dk": want["dk"], "dv": want["dv"], "dq": tuple(x[..., 1:] for x in want["dq"])})


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("h,hk,c", [(4, 4, 8), (3, 1, 16), (3, 1, 40), (4, 2, 64), (3, 1, 128)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_hidden_keys_have_no_gradient_whatever_the_queries_hold(gt, bad, h, hk, c, t):
    """A query, or its dO, that is not a number spoils the keys that it sees, and those only."""
    cq, ck = [0, 70, 110], [0, 150, 290]
    q, k, v, do = _t((110, h, c), t, 1), _t((290, hk, c), t, 2), _t((290, hk, c), t, 3), _t((110, h, c), t, 4)
    mask = torch.arange(290, device="cuda") % 5 != 2
    mask[64:140] = False
    offs = _off(*cq), _off(*ck)
    o, lse = gt.gt_cross_attn_fwd(q, k, v, *offs, mask)
    clean = gt.gt_cross_attn_bwd(q, k, v, o, do, lse, *offs, mask)
    for x in (q, do):
        kept = x[5].clone()
        x[5] = bad
        o2 = o.clone()      # (an infinity may raise the bases of other rows, and with that their roundings)
        o2[5] = gt.gt_cross_attn_fwd(q, k, v, *offs, mask)[0][5]
        dq, dk, dv = gt.gt_cross_attn_bwd(q, k, v, o2, do, lse, *offs, mask)
        assert (dk[~mask] == 0).all() and (dv[~mask] == 0).all()
        assert torch.equal(dk[150:], clean[1][150:]) and torch.equal(dv[150:], clean[2][150:])
        dq[5] = clean[0][5]
        assert torch.equal(dq, clean[0])
        x[5] = kept


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("h,hk,c", [(4, 4, 8), (2, 1, 8), (3, 1, 16), (4, 4, 16), (3, 1, 40), (4, 2, 64), (3, 1, 128)])
@pytest.mark.parametrize("lq", [1, 45])
def test_queries_that_see_no_key_whatever_they_hold(gt, lq, h, hk, c, t):
    """Sequences whose keys are all hidden, or that have none: o = 0, lse = -infinity and dq = 0 for queries, and with dO,
    that are not numbers; with keys enough for several parts."""
    lens = [300, 700, 0, 130]
    ck = [sum(lens[:i]) for i in range(5)]
    nq, nk = 4 * lq, ck[-1]
    q, k, v, do = _t((nq, h, c), t, 1), _t((nk, hk, c), t, 2), _t((nk, hk, c), t, 3), _t((nq, h, c), t, 4)
    mask = torch.ones(nk, dtype=torch.bool, device="cuda")
    mask[ck[1]:ck[2]] = False
    k[~mask] = math.nan
    offs = _off(*range(0, nq + 1, lq)), _off(*ck)
    clean = gt.gt_cross_attn_fwd(q, k, v, *offs, mask)
    grads = gt.gt_cross_attn_bwd(q, k, v, clean[0], do, clean[1], *offs, mask)
    empty = slice(lq, 3 * lq)
    for bad in (math.nan, math.inf, -math.inf):
        q[empty, :, c // 2] = bad
        do[empty, :, c - 1] = bad
        o, lse = gt.gt_cross_attn_fwd(q, k, v, *offs, mask)
        assert (o[empty] == 0).all() and (lse[:, empty] == -math.inf).all()
        assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])
        got = gt.gt_cross_attn_bwd(q, k, v, o, do, lse, *offs, mask)
        assert (got[0][empty] == 0).all()
        assert all(torch.equal(a, b) for a, b in zip(got, grads))


def test_one_query_over_2_to_the_27_keys(gt):
    """Keys x lanes past 2^31 are split and joined as fewer are; against fp64, the keys being the values too."""
    torch.cuda.empty_cache()
    nk, c = 2 ** 27 + 5, 72
    k = torch.empty(nk, 1, c, dtype=B, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    q = _t((1, 1, c), B, 1, 2.0)
    gt.gt_kernel_stats_reset(False)
    o, lse = gt.gt_cross_attn_fwd(q, k, k)
    assert {"cross_few", "cross_join"} <= set(gt.gt_kernel_stats())
    top, total, out, mag = -math.inf, 0.0, torch.zeros(c, dtype=torch.float64, device="cuda"), 0.0
    for a in range(0, nk, 2 ** 22):
        x = k[a:a + 2 ** 22, 0].double()
        s = x @ q[0, 0].double() / math.sqrt(c)
        new = max(top, float(s.max()))
        p = torch.exp(s - new)
        total, out = total * math.exp(top - new) + float(p.sum()), out * math.exp(top - new) + p @ x
        mag = mag * math.exp(top - new) + p @ x.abs()
        top = new
    # 64 parts, four warps, two groups of lanes share the keys; the exponent as for any number of keys
    steps = nk / (64 * 4 * 2) + 80
    e = 40 * R.U32 + (c + 4) * R.U32 * 30
    bound = (steps * R.U32 + 2 * e) * mag / total + R.half_step(B) * (out / total).abs()
    assert bool(((o[0, 0].double() - out / total).abs() <= bound).all()) and float((out / total).abs().max()) > 20 * float(bound.max())
    assert abs(float(lse[0, 0]) - (top + math.log(total))) <= steps * R.U32 + e + 8 * R.U32 * 30
    del k
    torch.cuda.empty_cache()


def _launched(gt, call):
    """The result of a call and the names of the kernels that it launched."""
    gt.gt_kernel_stats_reset(False)
    result = call()
    names = set(gt.gt_kernel_stats())
    gt.gt_kernel_stats_reset(False)
    return result, names


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("share", [1, 2])
@pytest.mark.parametrize("c", [1, 5, 8, 16, 30, 64, 100, 128])
@pytest.mark.parametrize("hidden", [False, True])
def test_one_query_to_a_sequence(gt, hidden, c, share, t):
    """Six sequences of one query in the mean, one of them of none and one of two; ragged keys, a side without any."""
    cq, ck, hk = [0, 1, 2, 2, 4, 5, 6], [0, 0, 1, 70, 571, 640, 2000], 2
    q, k, v = _t((6, share * hk, c), t, 1), _t((2004, hk, c), t, 2), _t((2004, hk, c), t, 3)
    k[2000:], v[2000:] = math.nan, math.inf
    mask = None
    if hidden:
        mask = torch.arange(2004, device="cuda") % 7 != 3
        mask[571:640] = False
        k[~mask] = math.nan
    offs = _off(*cq), _off(*ck)
    (o, lse), names = _launched(gt, lambda: gt.gt_cross_attn_fwd(q, k, v, *offs, mask))
    assert "cross_few" in names
    ref = X.attn_fwd(q, k, v, *offs, mask)
    empty = ref["lse"][0] == -math.inf
    assert ((lse.cpu() == -math.inf) == empty).all() and bool(empty[:, 0].all()) and (o.cpu()[empty.t()] == 0).all()
    R.check({"o": o, "lse": lse.cpu().masked_fill(empty, 0)},
            {"o": ref["o"], "lse": (ref["lse"][0].masked_fill(empty, 0), ref["lse"][1])})
    assert all(torch.equal(a, b) for a, b in zip(gt.gt_cross_attn_fwd(q, k, v, *offs, mask), (o, lse)))


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("share", [1, 2])
@pytest.mark.parametrize("c", [16, 64, 100])
def test_one_query_over_many_keys(gt, c, share, t):
    """Keys in parts, joined by a second kernel; with and without hidden ones, whole parts of them."""
    q, k, v = _t((1, share, c), t, 1), _t((9001, 1, c), t, 2), _t((9001, 1, c), t, 3)
    mask = torch.arange(9001, device="cuda") % 3 != 1
    mask[2000:6500] = False
    for keep in (None, mask):
        (o, lse), names = _launched(gt, lambda: gt.gt_cross_attn_fwd(q, k, v, key_mask=keep))
        assert {"cross_few", "cross_join"} <= names
        R.check({"o": o, "lse": lse}, X.attn_fwd(q, k, v, mask=keep))
