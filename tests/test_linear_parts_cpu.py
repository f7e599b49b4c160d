"""Operands whose low bits decide (tests/linear_parts.py) would show any product of
parts that is left out."""
import pytest
import torch

import linear_parts as ref

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("xt,lt", [(F32, F32), (F32, BF16), (BF16, F32)])
def test_low_bits_show_every_product(xt, lt):
    """With all products the result is right to the last bit of its type; without any one of them many elements are not."""
    f = (xt == F32, lt == F32)
    for depth in (34, 200, 777):
        b, a = ref.low_bits(96, 40, depth, *f, seed=depth)
        assert torch.equal(b.to(xt).double(), b) and torch.equal(a.to(lt).double(), a)
        want = torch.from_numpy(ref.exact(b, a)).float()
        assert torch.equal(ref.by_parts(b, a, *f).float(), want)
        slack = ref.slack(want, b, a, *f)
        assert (slack > 0).double().mean() < 0.5
        orders = [(i, j) for i in range(3 if f[0] else 1) for j in range(3 if f[1] else 1) if i + j <= 2]
        assert len(orders) == (6 if all(f) else 3)
        for left_out in orders:
            wrong = ref.by_parts(b, a, *f, left_out=[left_out]).float().to(xt)
            off = (wrong.double() - want.to(xt).double()).abs()
            assert (off > slack).double().mean() > 0.1, (depth, left_out)
