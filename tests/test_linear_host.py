"""Refusals and sizes of the LayerNorm and linear-layer entry points on the host (no GPU, no launch)."""
import ctypes

import pytest
import torch

P, I64, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
A = P(0x1000)      # never dereferenced: every call below fails its host checks


@pytest.fixture(scope="module")
def gt():
    from graph_transformer_attention_gb300 import build
    build.build()
    import graph_transformer_attention_gb300 as m
    m.load_library()
    return m


def test_layer_norm_forward_refusals(gt):
    lib = gt.load_library()
    good = dict(xt=0, yt=1, n=4, c=64, x=A, ldx=64, gain=A, shift=A, eps=1e-5, y=A, ldy=64, mean=A, rstd=A)

    def call(**kw):
        return lib.gt_layer_norm_fwd(*{**good, **kw}.values(), None)

    for bad in (dict(xt=2), dict(yt=-1), dict(n=0), dict(n=-3), dict(c=0), dict(x=None), dict(gain=None), dict(shift=None),
                dict(y=None), dict(mean=None), dict(rstd=None), dict(ldx=63), dict(ldy=63), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**bad) == -1, bad
    assert call(c=16385, ldx=16385, ldy=16385) == -2


def test_layer_norm_backward_refusals(gt):
    lib = gt.load_library()
    need = gt.gt_layer_norm_workspace_size(4, 64)
    good = dict(xt=0, yt=1, n=4, c=64, dy=A, lddy=64, x=A, ldx=64, gain=A, mean=A, rstd=A, dres=None, ldr=0, dx=A, lddx=64,
                dgain=A, dshift=A, ws=A, bytes=need)

    def call(**kw):
        return lib.gt_layer_norm_bwd(*{**good, **kw}.values(), None)

    for bad in (dict(xt=2), dict(yt=3), dict(n=0), dict(c=0), dict(dy=None), dict(x=None), dict(gain=None), dict(mean=None),
                dict(rstd=None), dict(dx=None), dict(dgain=None), dict(dshift=None), dict(lddy=63), dict(ldx=63),
                dict(lddx=63), dict(dres=A, ldr=63)):
        assert call(**bad) == -1, bad
    assert call(c=16385, lddy=16385, ldx=16385, lddx=16385) == -2
    assert call(ws=None) == call(bytes=need // 2) == call(ws=P(0x1008)) == -5
    assert gt.gt_layer_norm_workspace_size(0, 64) == gt.gt_layer_norm_workspace_size(4, 0) == 0
    assert gt.gt_layer_norm_workspace_size(4, 16385) == 0 and need > 0


def test_linear_forward_refusals(gt):
    lib = gt.load_library()
    good = dict(dt=1, yt=1, m=4, k=64, n=32, x=A, ldx=64, w=A, ldw=32, b=None, act=0, r=None, ldr=0, y=A, ldy=32, pre=None,
                ldpre=0, ws=A, bytes=1 << 30)

    def call(**kw):
        return lib.gt_linear_fwd(*{**good, **kw}.values(), None)

    for bad in (dict(dt=2), dict(yt=7), dict(m=0), dict(k=0), dict(n=0), dict(m=-1), dict(act=2), dict(act=-1), dict(x=None),
                dict(w=None), dict(y=None), dict(ldx=63), dict(ldw=31), dict(ldy=31), dict(r=A, ldr=31),
                dict(pre=A, ldpre=31)):
        assert call(**bad) == -1, bad
    assert call(dt=0, yt=1) == -2
    for big in (dict(m=(1 << 24) + 1), dict(k=65537, ldx=65537), dict(n=65537, ldw=65537, ldy=65537)):
        assert call(**big) == -2, big
    # a workspace is needed for fp32 operands, for rows that are no multiple of 16 bytes and for such results
    assert call(dt=0, yt=0, m=2000, k=512, ldx=512, n=300, ldw=300, ldy=300, bytes=100) == -5
    assert call(ldx=65, ws=None) == call(x=P(0x1002), ws=None) == call(ldy=33, bytes=16) == call(ldx=65, ws=P(0x1004)) == -5


def test_linear_backward_refusals(gt):
    lib = gt.load_library()
    good = dict(dt=1, yt=1, m=4, k=64, n=32, dy=A, lddy=32, x=A, ldx=64, w=A, ldw=32, pre=None, ldpre=0, act=0, add=None,
                ldadd=0, dx=A, lddx=64, dw=A, lddw=32, db=A, ws=A, bytes=1 << 30)

    def call(**kw):
        return lib.gt_linear_bwd(*{**good, **kw}.values(), None)

    for bad in (dict(dt=2), dict(yt=7), dict(m=0), dict(k=0), dict(n=0), dict(act=2), dict(dy=None), dict(lddy=31),
                dict(x=None), dict(w=None), dict(ldx=63), dict(ldw=31), dict(lddx=63), dict(lddw=31),
                dict(dx=None, dw=None, db=None),
                dict(act=1), dict(pre=A, ldpre=32), dict(act=1, pre=A, ldpre=31),        # pre and act belong together
                dict(add=A, ldadd=63), dict(add=A, ldadd=64, dx=None, lddx=0)):
        assert call(**bad) == -1, bad
    assert call(dt=0, yt=1) == -2 and call(m=(1 << 24) + 1) == -2
    assert call(ws=None) == call(bytes=1) == call(ws=P(0x1008)) == -5


def test_linear_workspace_sizes(gt):
    fwd, bwd = gt.gt_linear_fwd_workspace_size, gt.gt_linear_bwd_workspace_size
    assert fwd(1, 4, 64, 32) == 0                                   # read and written in place
    assert fwd(1, 4, 64, 32, aligned=False) >= 2 * (4 * 64 + 64 * 32) + 4 * 4 * 32
    assert fwd(0, 2000, 512, 300) >= 6 * (2000 * 512 + 512 * 304)   # three bf16 planes of each operand
    assert bwd(1, 1, 5000, 64, 32, act=1) >= 2 * 5000 * 32           # da
    assert bwd(1, 0, 5000, 64, 32) >= 2 * 5000 * 32
    for bad in ((2, 4, 64, 32), (1, 0, 64, 32), (1, 4, 65537, 32)):
        assert fwd(*bad) == 0
    assert bwd(0, 1, 4, 64, 32) == 0 and bwd(1, 1, 4, 64, 32, act=9) == 0


def test_binding_refuses_tensors_off_the_gpu(gt):
    x, w, v = torch.zeros(3, 4), torch.zeros(4, 5), torch.zeros(4)
    for call in (lambda: gt.gt_layer_norm_fwd(x, v, v), lambda: gt.gt_layer_norm_bwd(x, x, v, torch.zeros(3), torch.zeros(3)),
                 lambda: gt.gt_linear_fwd(x, w), lambda: gt.gt_linear_bwd(torch.zeros(3, 5), x, w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_sizes_past_32_bits_are_not_cut(gt):
    """A size above 2^31 - 1 is not supported: its low 32 bits must not be taken for it."""
    big = (1 << 32) + 4
    assert gt.gt_layer_norm_workspace_size(big, 64) == gt.gt_layer_norm_workspace_size(4, big) == 0
    for sizes in ((big, 64, 32), (4, big, 32), (4, 64, big)):
        assert gt.gt_linear_fwd_workspace_size(0, *sizes) == gt.gt_linear_bwd_workspace_size(1, 1, *sizes, act=1) == 0
