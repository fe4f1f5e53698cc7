"""fp32 products through bf16 splits, exact cases: every term of the split counts, in y, dx and dW."""
import pytest
import torch

import split_ref as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gt():
    import graph_transformer_attention_gb300 as m
    from graph_transformer_attention_gb300 import build
    build.build()
    m.load_library()
    return m


def _equal(got, a, b):
    exact = a.double() @ b.double()
    assert torch.equal(got.cpu().double(), exact), f"{int((got.cpu().double() != exact).sum())} of {exact.numel()} differ"


# contractions past the one-kernel path (64 deep forward): one tile and many, aligned rows and odd ones, one deep enough for splits
@pytest.mark.parametrize("kind", S.KINDS)
@pytest.mark.parametrize("side", ["left", "right"])
@pytest.mark.parametrize("m,k,n", [(50, 72, 24), (50, 640, 200), (300, 200, 257), (1000, 104, 520), (3, 4000, 304), (2500, 321, 1001)])
def test_forward(gt, m, k, n, side, kind):
    x, w = S.operands(m, k, n, kind, side)
    y, _ = gt.gt_linear_fwd(x.cuda(), w.cuda())
    gt.gt_check_device_status()
    _equal(y, x, w)


# ... and of the backward (1024 rows, 128 columns): a launch for each product, one for both, splits of either contraction
@pytest.mark.parametrize("kind", S.KINDS)
@pytest.mark.parametrize("side", ["left", "right"])
@pytest.mark.parametrize("m,k,n", [(200, 72, 136), (300, 200, 257), (1100, 72, 40), (4100, 40, 72), (40, 24, 4000), (2000, 303, 601),
                                   (9000, 520, 264)])
def test_backward(gt, m, k, n, side, kind):
    # dx = dy W^T: the dense one dy or W
    dy, wt = S.operands(m, n, k, kind, side)
    x = S.whole(m, k, 3, 7)
    dx = gt.gt_linear_bwd(dy.cuda(), x.cuda(), wt.t().contiguous().cuda())[0]
    _equal(dx, dy, wt)
    alone = gt.gt_linear_bwd(dy.cuda(), None, wt.t().contiguous().cuda(), need_dw=False, need_db=False)[0]
    _equal(alone, dy, wt)
    # dW = x^T dy: the dense one x or dy
    xt, dy = S.operands(k, m, n, kind, side, seed=3)
    w = S.whole(k, n, 3, 8)
    dw = gt.gt_linear_bwd(dy.cuda(), xt.t().contiguous().cuda(), w.cuda())[1]
    _equal(dw, xt, dy)
    alone = gt.gt_linear_bwd(dy.cuda(), xt.t().contiguous().cuda(), None, need_dx=False, need_db=False)[1]
    _equal(alone, xt, dy)
    gt.gt_check_device_status()
