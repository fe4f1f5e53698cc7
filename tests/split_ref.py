"""Operands for which a product of three-part bf16 splits has to be exact, and an emulation of its terms.

A dense matrix of whole numbers meets a matrix with one non-zero in each of the sums, so that every result is
one product: a 24-bit number times a power of two, whose hi, mid and lo parts all count, or a 12-bit number
times an 11-bit one, whose parts' four products are all needed for the 23 bits of theirs.  No rounding is
left, whatever the order: partial sums have at most 24 bits (23 and a carry), zeros add nothing.
"""
import torch

TERMS = ("lo hi", "hi lo", "mid mid", "mid hi", "hi mid", "hi hi")


def split3(v):
    """The three bf16 parts of fp32 values, as fp64."""
    hi = v.bfloat16().float()
    mid = (v - hi).bfloat16().float()
    lo = (v - hi - mid).bfloat16().float()
    return {"hi": hi.double(), "mid": mid.double(), "lo": lo.double()}


def product(a, b, terms=TERMS):
    """a b as the sum of the named products of parts."""
    pa, pb = split3(a), split3(b)
    return sum(pa[s] @ pb[t] for s, t in (term.split() for term in terms))


def whole(rows, cols, bits, seed):
    g = torch.Generator().manual_seed(seed)
    sign = torch.randint(0, 2, (rows, cols), generator=g) * 2 - 1
    return (torch.randint(2 ** (bits - 1), 2 ** bits, (rows, cols), generator=g) * sign).float()


def one_per_row(rows, cols, kind, seed):
    """[rows][cols] with one non-zero a row, at a random column: a signed power of two, or an 11-bit number."""
    g = torch.Generator().manual_seed(seed)
    v = whole(rows, 1, 11, seed)[:, 0] if kind == "12 x 11 bits" else (
        (torch.randint(0, 2, (rows,), generator=g) * 2 - 1) * 2.0 ** torch.randint(-20, 21, (rows,), generator=g)).float()
    t = torch.zeros(rows, cols)
    t[torch.arange(rows), torch.randint(0, cols, (rows,), generator=g)] = v
    return t


KINDS = ("24 bits x power", "12 x 11 bits")


def dense(rows, cols, kind, seed):
    return whole(rows, cols, 12 if kind == "12 x 11 bits" else 24, seed)


def operands(m, k, n, kind, side, seed=1):
    """A [m][k] and B [k][n] with the dense one on `side`: "left" (B has one non-zero a column) or "right"."""
    if side == "left":
        return dense(m, k, kind, seed), one_per_row(n, k, kind, seed + 1).t().contiguous()
    return one_per_row(m, k, kind, seed), dense(k, n, kind, seed + 1)
