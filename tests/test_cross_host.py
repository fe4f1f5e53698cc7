"""Refusals and sizes of cross attention, of the norm of queries and keys and of gradient clipping on the host (no GPU,
no launch), and the fp64 references against plain forms of the formulas."""
import ctypes
import math

import pytest
import torch

import cross_ref as X

P = ctypes.c_void_p
A = P(0x1000)      # never dereferenced: every call below fails its host checks


@pytest.fixture(scope="module")
def gt():
    from graph_transformer_attention_gb300 import build
    build.build()
    import graph_transformer_attention_gb300 as m
    m.load_library()
    return m


SIZES = dict(dt=1, nq=40, nk=6, h=4, hk=2, d=64, batch=1)
BAD_SIZES = (dict(dt=2), dict(dt=-1), dict(nq=0), dict(nk=0), dict(nq=-1), dict(h=0), dict(hk=0), dict(h=3), dict(d=0),
             dict(batch=0), dict(batch=2))
BIG_SIZES = (dict(d=129), dict(h=1026), dict(h=130, hk=2), dict(batch=(1 << 20) + 1, qo=A, ko=A), dict(nq=(1 << 30) + 1),
             dict(nk=(1 << 30) + 1))
INPUTS = dict(q=A, ldq=256, hdq=64, k=A, ldk=128, hdk=64, v=A, ldv=128, hdv=64)


def test_cross_attention_forward_refusals(gt):
    lib = gt.load_library()
    good = dict(**SIZES, **INPUTS, qo=None, ko=None, mask=None, scale=0.125, o=A, ldo=256, hdo=64, lse=A, ws=A, bytes=1 << 40)

    def call(**kw):
        return lib.gt_cross_attn_fwd(*{**good, **kw}.values(), None)

    for bad in (*BAD_SIZES, dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(lse=None), dict(ldq=-1), dict(hdk=-64),
                dict(ldo=-1), dict(qo=A), dict(ko=A), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
                dict(scale=math.nan)):
        assert call(**bad) == -1, bad
    for big in BIG_SIZES:
        assert call(**big) == -2, big
    # rows that TMA cannot read need room for their copies
    for odd in (dict(q=P(0x1002)), dict(ldk=129), dict(hdv=0), dict(hdq=65)):
        assert call(**odd, ws=None) == call(**odd, bytes=64) == call(**odd, ws=P(0x1004)) == -5, odd


def test_cross_attention_backward_refusals(gt):
    lib = gt.load_library()
    good = dict(**SIZES, **INPUTS, o=A, ldo=256, hdo=64, do=A, lddo=256, hddo=64, lse=A, qo=None, ko=None, mask=None,
                scale=0.125, dq=A, lddq=256, hddq=64, dk=A, lddk=128, hddk=64, dv=A, lddv=128, hddv=64, ws=A, bytes=1 << 40)

    def call(**kw):
        return lib.gt_cross_attn_bwd(*{**good, **kw}.values(), None)

    for bad in (*BAD_SIZES, *(dict([(n, None)]) for n in ("q", "k", "v", "o", "do", "lse", "dq", "dk", "dv")), dict(lddk=-1),
                dict(hddo=-1), dict(qo=A), dict(ko=A), dict(scale=0.0), dict(scale=math.nan)):
        assert call(**bad) == -1, bad
    for big in BIG_SIZES:
        assert call(**big) == -2, big
    assert call(ws=None) == call(bytes=1) == call(ws=P(0x1008)) == -5


def test_cross_attention_workspace_sizes(gt):
    size = gt.gt_cross_attn_workspace_size
    assert size(1, 40, 6, 4, 2, 64) == size(1, 4, 6, 4, 2, 64) == 0
    assert size(1, 40, 6, 4, 2, 64, aligned=False) >= 2 * 64 * (40 * 4 + 2 * 6 * 2)
    assert size(1, 1, 6, 4, 2, 64, aligned=False) == 0                 # few rows are read as they are
    assert size(1, 4, 6, 4, 2, 64, backward=True) >= 8 * 4 * 4
    assert size(1, 4, 6, 4, 2, 64, backward=True, aligned=False) >= 8 * 4 * 4 + 2 * 64 * (2 * 4 * 4 + 2 * 6 * 2)
    for bad in ((2, 4, 6, 4, 2, 64), (1, 0, 6, 4, 2, 64), (1, 4, 6, 4, 3, 64), (1, 4, 6, 4, 2, 129), (1, 4, 6, 4, 2, 64, 0)):
        assert size(*bad) == 0
    big = (1 << 32) + 4
    for at in range(1, 7):
        sizes = [1, 4, 6, 4, 2, 64, 1]
        sizes[at] = big
        assert size(*sizes) == 0, "the low 32 bits of a size must not be taken for it"
    assert gt.gt_qk_norm_workspace_size(big) == gt.gt_grad_clip_workspace_size(big) == 0


def test_scales_beyond_the_exponents_range_are_refused(gt):
    """scale log2 e is infinite from 2.36e38 on, and every score would be NaN."""
    lib = gt.load_library()
    fwd = dict(**SIZES, **INPUTS, qo=None, ko=None, mask=None, scale=0.125, o=A, ldo=256, hdo=64, lse=A, ws=None, bytes=0)
    bwd = dict(**SIZES, **INPUTS, o=A, ldo=256, hdo=64, do=A, lddo=256, hddo=64, lse=A, qo=None, ko=None, mask=None,
               scale=0.125, dq=A, lddq=256, hddq=64, dk=A, lddk=128, hddk=64, dv=A, lddv=128, hddv=64, ws=None, bytes=0)
    fwd["hdq"] = 65      # (read through a copy: the next check is that for its room)
    for call, good in ((lib.gt_cross_attn_fwd, fwd), (lib.gt_cross_attn_bwd, bwd)):
        assert [call(*{**good, "scale": x}.values(), None) for x in (2.3e38, 1e-45, 2.4e38, 3e38)] == [-5, -5, -1, -1]


@pytest.mark.parametrize("c", [8, 40, 128])
def test_parts_of_long_keys(gt, c):
    """One query over ever more keys: as many parts as keys for them are there, and no fewer where keys x lanes passes 2^31."""
    size = gt.gt_cross_attn_workspace_size
    few = size(0, 1, 1 << 20, 1, 1, c)
    assert few > 0
    for nk in (1 << 26, (1 << 27) - 1, 1 << 27, (1 << 27) + 1, 1 << 28, 1 << 29, 1 << 30):
        assert size(0, 1, nk, 1, 1, c) == size(1, 1, nk, 1, 1, c) == few, nk


QK = dict(xt=1, yt=0, d=64, eps=1e-6, freq=A, rot=64, pairs=0)


def test_qk_norm_refusals(gt):
    lib = gt.load_library()
    fwd = dict(**QK, nq=4, h=2, q=A, ldq=128, hdq=64, gq=A, pq=None, yq=A, ldyq=128, hdyq=64,
               nk=5, hk=1, k=A, ldk=64, hdk=64, gk=A, pk=None, yk=A, ldyk=64, hdyk=64)
    bwd = dict(**QK, nq=4, h=2, dyq=A, lddyq=128, hddyq=64, q=A, ldq=128, hdq=64, gq=A, pq=None, dq=A, lddq=128, hddq=64, dgq=A,
               nk=5, hk=1, dyk=A, lddyk=64, hddyk=64, k=A, ldk=64, hdk=64, gk=A, pk=None, dk=A, lddk=64, hddk=64, dgk=A,
               ws=A, bytes=1 << 30)
    shared = (dict(xt=2), dict(yt=-1), dict(d=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
              dict(rot=0), dict(freq=None), dict(rot=63), dict(rot=66), dict(rot=-2), dict(pairs=2), dict(nq=0), dict(h=0),
              dict(nk=0), dict(hk=-1), dict(q=None), dict(gq=None), dict(gk=None), dict(ldq=-1), dict(hdk=-64))
    for call, good, more in ((lib.gt_qk_norm_fwd, fwd, (dict(yq=None), dict(yk=None), dict(ldyk=-1))),
                             (lib.gt_qk_norm_bwd, bwd, (dict(dyq=None), dict(dyk=None), dict(dq=None), dict(dk=None),
                                                        dict(dgq=None), dict(dgk=None), dict(hddyk=-1)))):
        for bad in (*shared, *more):
            assert call(*{**good, **bad}.values(), None) == -1, bad
        for big in (dict(d=257), dict(h=1025), dict(hk=1025)):
            assert call(*{**good, **big}.values(), None) == -2, big
    need = gt.gt_qk_norm_workspace_size(64)
    assert need > 0 and gt.gt_qk_norm_workspace_size(0) == gt.gt_qk_norm_workspace_size(257) == 0
    for short in (dict(ws=None), dict(bytes=need // 4), dict(ws=P(0x1008))):
        assert lib.gt_qk_norm_bwd(*{**bwd, **short}.values(), None) == -5


def test_grad_clip_refusals(gt):
    lib = gt.load_library()
    need = gt.gt_grad_clip_workspace_size(1)

    def call(g=0x1000, out=0x1000, numel=8, gtype=0, otype=0, count=1, limit=1.0, norm=A, ws=A, nbytes=need, table=True):
        one = (gt._Grad * 1)(gt._Grad(g, out, numel, gtype, otype))
        return lib.gt_grad_clip(ctypes.addressof(one) if table else None, count, limit, norm, ws, nbytes, None)

    for bad in (dict(table=False), dict(count=0), dict(count=-1), dict(g=None), dict(numel=-1), dict(gtype=2), dict(otype=5),
                dict(otype=1), dict(norm=None), dict(limit=-1.0), dict(limit=math.nan)):
        assert call(**bad) == -1, bad
    assert call(numel=(1 << 40) + 1) == -2
    assert call(ws=None) == call(nbytes=1) == call(ws=P(0x1008)) == -5
    assert gt.gt_grad_clip_workspace_size(0) == 0 and need > 0


def test_binding_refuses_tensors_off_the_gpu(gt):
    q, k, g = torch.zeros(3, 2, 8), torch.zeros(5, 2, 8), torch.ones(8)
    for call in (lambda: gt.gt_cross_attn_fwd(q, k, k), lambda: gt.gt_cross_attn_bwd(q, k, k, q, q, torch.zeros(2, 3)),
                 lambda: gt.gt_qk_norm_fwd(q, k, g, g), lambda: gt.gt_qk_norm_bwd(q, k, q, k, g, g),
                 lambda: gt.gt_grad_clip([q], 1.0), lambda: gt.gt_tensor_list([q, k])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="at least one"):
        gt.gt_tensor_list([])


# ---------------------------------------------------------------- the references themselves

def _inputs(nq=6, nk=11, h=4, hk=2, c=5):
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(*s, generator=g) for s in ((nq, h, c), (nk, hk, c), (nk, hk, c)))
    mask = torch.ones(nk, dtype=torch.bool)
    mask[2], mask[8] = False, False
    return q, k, v, torch.tensor([0, 2, 2, 6], dtype=torch.int32), torch.tensor([0, 5, 9, 11], dtype=torch.int32), mask


def test_reference_attention_is_the_formula():
    q, k, v, qo, ko, mask = _inputs()
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    out = []
    for a, b, ka, kb in ((0, 2, 0, 5), (2, 6, 9, 11)):
        for i in range(a, b):
            heads = []
            for j in range(4):
                keys = [n for n in range(ka, kb) if mask[n]]
                s = torch.stack([(leaves[0][i, j] * leaves[1][n, j // 2]).sum() / math.sqrt(5) for n in keys])
                heads.append((torch.exp(s)[:, None] * torch.stack([leaves[2][n, j // 2] for n in keys])).sum(0) / torch.exp(s).sum())
            out.append(torch.stack(heads))
    out = torch.stack(out)
    ref = X.attn_fwd(q, k, v, qo, ko, mask)
    assert float((ref["o"][0] - out.detach()).abs().max()) < 1e-12
    do = torch.randn(6, 4, 5, generator=torch.Generator().manual_seed(5))
    (out * do.double()).sum().backward()
    # fp64 o and lse in the place of the stored ones
    got = X.attn_bwd(q, k, v, ref["o"][0], do, ref["lse"][0], qo, ko, mask)
    for name, leaf in zip(("dq", "dk", "dv"), leaves):
        assert float((got[name][0] - leaf.grad).abs().max()) < 1e-12, name


@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("rot", [0, 4, 6])
def test_reference_norm_is_the_formula(rot, pairs):
    g = torch.Generator().manual_seed(1)
    x, gain, dy = torch.randn(4, 2, 7, generator=g), torch.randn(7, generator=g), torch.randn(4, 2, 7, generator=g)
    freq = None if rot == 0 else torch.rand(rot // 2, generator=g)
    pos = torch.tensor([3, -2, 100, 0], dtype=torch.int32)
    X64, G64 = x.double().requires_grad_(), gain.double().requires_grad_()
    w = X64 / torch.sqrt((X64 ** 2).sum(-1, keepdim=True) / 7 + 1e-6) * G64
    y = [w[..., c] for c in range(7)]
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
        angle = pos.double() * float(freq[i])
        cs, sn = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        y[a], y[b] = w[..., a] * cs - w[..., b] * sn, w[..., a] * sn + w[..., b] * cs
    y = torch.stack(y, -1)
    assert float((X.qk_fwd(x, gain, freq, pos, pairs, 1e-6, torch.float32)["y"][0] - y.detach()).abs().max()) < 1e-12
    (y * dy.double()).sum().backward()
    got = X.qk_bwd(dy, x, gain, freq, pos, pairs, 1e-6)
    assert float((got["dx"][0] - X64.grad).abs().max()) < 1e-12
    assert float((got["dgain"][0] - G64.grad).abs().max()) < 1e-12
