"""fp32 operands of a linear layer in all their bits, on every kernel of the matrix units
that cuts one into parts (tests/linear_cases.py lists a shape for each)."""
import pytest
import torch

import linear_cases as cases
import linear_parts as ref
import test_linear_gpu as base

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = cases.F32, cases.BF16


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


CUT = cases.shapes(parts_only=True)


def run_with(case, b, a):
    """The product B A^T as the case's call: B is x (dy), A the weight (transposed); the result and its type's rounding of
    the exact one."""
    xt, lt, back, rows, out, inp = case
    ly = base.Layer(out, inp, lt, seed=1, whole=True)
    o = ly.opt.offsets[1]
    ly.list[o: o + out * inp] = (a.t() if back else a).reshape(-1).to(DEV).to(lt)
    x = b.to(DEV).to(xt)
    y = torch.full((rows, inp if back else out), 7.0, dtype=xt, device=DEV)
    if back:
        ly.opt.linear_input_grad(1, x, ly.list, y)
    else:
        ly.opt.linear(1, None, x, ly.list, y)
    return y, torch.matmul(b.to(DEV), a.t().to(DEV).contiguous()).float().to(xt)


@pytest.mark.parametrize("case", CUT, ids=cases.name)
def test_low_bits(case):
    """Operands whose low bits alone settle the result: the exact one's rounding, but for the bits that linear_ref.slack
    counts (the CPU test of these operands shows that without any one product of parts it would not be)."""
    xt, lt, back, rows, out, inp = case
    features, depth = (inp, out) if back else (out, inp)
    for seed in (1, 2):
        b, a = ref.low_bits(rows, features, depth, xt == F32, lt == F32, seed)
        y, want = run_with(case, b, a)
        slack = ref.slack(want.cpu(), b, a, xt == F32, lt == F32)
        assert (slack == 0).double().mean() > 0.5
        off = (y.double() - want.double()).abs().cpu()
        assert bool((off <= slack).all()), (int((off > slack).sum()), float(off.max()))


@pytest.mark.parametrize("case", CUT, ids=cases.name)
def test_ends_of_the_range(case):
    """Single products with 1 of values near both ends of fp32's range, either operand holding them: exact, down to
    2^-133, bf16's last bit."""
    xt, lt, back, rows, out, inp = case
    features, depth = (inp, out) if back else (out, inp)
    ends = torch.tensor([3.4028234663852886e38, 3.3961775e38, 3.38953e38, 1.2345678e38, 2.3456789e-30, 2.0 ** -126, 2.0 ** -130 + 2.0 ** -133,
                         2.0 ** -133], dtype=F32).double()
    ends = torch.cat([ends, -ends])
    for in_x in (True, False):
        if (xt if in_x else lt) != F32:
            continue
        b, a = torch.zeros(rows, depth, dtype=torch.float64), torch.zeros(features, depth, dtype=torch.float64)
        holder, other = (b, a) if in_x else (a, b)
        t = torch.arange(min(len(ends), holder.shape[0]))
        holder[t, (t * 37 + 5) % depth] = ends[: len(t)]
        other[torch.arange(other.shape[0]) % 3 != 0] = 1.0
        y, want = run_with(case, b, a)
        assert torch.equal(y, want), [(float(p), float(q)) for p, q in zip(y[y != want][:8], want[y != want][:8])]
