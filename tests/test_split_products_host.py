"""The operands of the exact tests see every term of a split product (on the CPU, the mistake planted in the emulation)."""
import itertools

import pytest
import torch

import split_ref as S


@pytest.mark.parametrize("kind,side", list(itertools.product(S.KINDS, ("left", "right"))))
def test_all_terms_give_the_exact_product(kind, side):
    a, b = S.operands(40, 130, 30, kind, side)
    exact = a.double() @ b.double()
    assert torch.equal(S.product(a, b), exact)
    assert torch.equal(exact.float().double(), exact)          # each result is an fp32 value


@pytest.mark.parametrize("term", S.TERMS)
def test_a_missing_term_is_seen(term):
    seen = []
    for kind, side in itertools.product(S.KINDS, ("left", "right")):
        a, b = S.operands(40, 130, 30, kind, side)
        seen.append(not torch.equal(S.product(a, b, [t for t in S.TERMS if t != term]), a.double() @ b.double()))
    assert any(seen)
    if term == "lo hi":
        assert seen[0]                    # lo of the left operand: dense 24 bits on the left
    if term == "hi lo":
        assert seen[1]
    if term == "mid mid":
        assert seen[2] and seen[3]


@pytest.mark.parametrize("part", ["hi", "mid", "lo"])
@pytest.mark.parametrize("instead", ["hi", "mid", "lo"])
@pytest.mark.parametrize("left", [True, False])
def test_a_wrong_part_is_seen(part, instead, left):
    """One operand's part read from another part's place."""
    if part == instead:
        return
    seen = False
    for kind, side in itertools.product(S.KINDS, ("left", "right")):
        a, b = S.operands(40, 130, 30, kind, side)
        pa, pb = S.split3(a), S.split3(b)
        (pa if left else pb)[part] = (pa if left else pb)[instead]
        got = sum(pa[s] @ pb[t] for s, t in (term.split() for term in S.TERMS))
        seen |= not torch.equal(got, a.double() @ b.double())
    assert seen
