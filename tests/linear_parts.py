"""Operands of a linear layer whose low bits alone settle the result, the products of
bf16 parts that add up to it, and by how much a result may differ (numpy and torch on
the host; no code of the package)."""
import numpy as np
import torch

BF16 = torch.bfloat16


def _signs(g, *shape):
    return torch.randint(0, 2, shape, generator=g).double() * 2 - 1


def _three(g, *shape):
    """+-2^p (1 + e1 2^-9 + e2 2^-18), e in -1, 0, 1: of up to three bf16 parts, each less than 2^-8 of the one before."""
    e = [torch.randint(-1, 2, shape, generator=g).double() for _ in range(2)]
    p = torch.randint(-3, 4, shape, generator=g).double()
    return _signs(g, *shape) * torch.exp2(p) * (1 + e[0] * 2.0 ** -9 + e[1] * 2.0 ** -18)


def _short(g, *shape):
    """+-2^p or +-1.5 * 2^p, of two significant bits."""
    p = torch.randint(-3, 4, shape, generator=g).double()
    return _signs(g, *shape) * torch.exp2(p) * (1 + torch.randint(0, 2, shape, generator=g).double() / 2)


def low_bits(rows, features, depth, x_f32, w_f32, seed):
    """(B [rows][depth], A [features][depth]) in float64, exact in their types.

    The first half of the rows of B have one element each that is not 0, so a result is one product: of one fp32 operand
    exact in 21 bits; of two the six products' sum has 19 bits, or 28 where a middle part is 0 and the parts' orders do not
    tell their sizes.  The others have two, c and -c or c and -c (1 + 2^-18 e), against elements of A that differ in their
    last part only: what is left is a multiple of 2^-18 that bf16 holds.  Their places run over all of a step's, in one
    step, in neighbouring ones and half the contraction apart."""
    g = torch.Generator()
    g.manual_seed(seed)
    b = torch.zeros(rows, depth, dtype=torch.float64)
    t = torch.arange(rows)
    k1 = (t * 37 + 5) % depth
    pairs = t >= rows // 2
    gap = torch.tensor([1, 8, 33, depth // 2 + 1])[t % 4] % depth
    k2 = (k1 + torch.where(gap == 0, 1, gap)) % depth
    if w_f32:
        # one magnitude and one middle part a feature, so that pairs cancel to the last part
        p = torch.exp2(torch.randint(-3, 4, (features, 1), generator=g).double()) * _signs(g, features, 1)
        e1 = _signs(g, features, 1)
        e2 = torch.randint(-1, 2, (features, depth), generator=g).double()
        a = p * (1 + e1 * 2.0 ** -9 + e2 * 2.0 ** -18)
        pair = torch.exp2(torch.randint(-3, 4, (rows,), generator=g).double())
        other = -pair
    else:
        a = _short(g, features, 1).expand(features, depth).clone()
        e = [torch.randint(-1, 2, (rows,), generator=g).double() for _ in range(3)]
        pair = torch.exp2(e[2]) * (1 + e[0] * 2.0 ** -9 + e[1] * 2.0 ** -18)
        other = -(torch.exp2(e[2]) * (1 + e[0] * 2.0 ** -9 + 2.0 ** -18 * torch.where(e[1] == 1, -1.0, 1.0)))
    single = _three(g, rows) if x_f32 else _short(g, rows)
    b[t, k1] = torch.where(pairs, pair, single)
    b[t[pairs], k2[pairs]] = other[pairs]
    return b, a


def parts(x):
    """float64 values as three bf16 parts, each the rest rounded to nearest (values far from the ends of the range)."""
    out = []
    for _ in range(3):
        h = x.float().to(BF16).double()
        out.append(h)
        x = x - h
    return out


def by_parts(b, a, x_f32, w_f32, left_out=()):
    """B A^T from the products of parts whose orders sum to at most 2, but for those (of B, of A) in left_out."""
    pb = parts(b) if x_f32 else [b]
    pa = parts(a) if w_f32 else [a]
    total = torch.zeros(b.shape[0], a.shape[0], dtype=torch.float64)
    for i, u in enumerate(pb):
        for j, v in enumerate(pa):
            if i + j <= 2 and (i, j) not in left_out:
                total += u @ v.T
    return total


def exact(b, a):
    return np.asarray(b) @ np.asarray(a).T


def slack(want, b, a, x_f32, w_f32):
    """By how much a result may differ from `want`, the exact one rounded to fp32.

    Not at all where fp32 holds the sum of the products of parts: then no partial sum has bits that fp32 lacks.  The
    matrix unit aligns the addends of a step to the largest and may cut, not round, what lies below 2^-24 of it.  Of the
    single products only the last addition has such bits (the sums before it are below 2^-8 of it and end above 2^-28), so
    the result is less than 2^-24 of that largest from the sum, the sum less than 2^-26 of it from the exact value
    and `want` half a step: two fp32 numbers less than two steps apart, so at most one, 2^-23 of `want`."""
    total = by_parts(b, a, x_f32, w_f32)
    return torch.where(total.float().double() == total, 0.0, 2.0 ** -23 * want.abs().double())
