"""Every kernel that a linear layer's plan can take (tests/linear_cases.py lists a
shape for each; the plan itself is checked on the CPU), with everything that stands
beside the product: bias, checkpoint, activation, residual and added gradient, in
place and not, 16-byte rows and others.  Sums are exact, so results without an
activation match bit for bit and with one the activation's error alone counts.
References are 64-bit on the GPU."""
import math

import pytest
import torch

import grad_ops as ref
import linear_cases as cases
import test_linear_gpu as base
from error_compensated_bit_02_amd import ActCheckpoint

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = cases.F32, cases.BF16
ALL = cases.shapes()


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()


def of(back):
    return pytest.mark.parametrize("case", [c for c in ALL if c[2] == back], ids=cases.name)


def put(t, dtype, extra=0, offset=0):
    return base._put(t, dtype, extra, offset)[0]


def layer(case, depth):
    """A layer of whole numbers scaled by a power of two so that the sums spread over the activations' bend;
    (layer, W, b in 64 bits)."""
    xt, lt, back, rows, out, inp = case
    ly = base.Layer(out, inp, lt, seed=rows + out, whole=True)
    down = 2.0 ** -max(0, round(math.log2(math.sqrt(8.0 * depth) / 3.0)))
    ly.list.mul_(down)
    return ly, torch.from_numpy(ly.w).to(DEV) * down, torch.from_numpy(ly.b).to(DEV) * down


def times(a, b):
    return torch.matmul(a.double(), b.double().contiguous())


def _sigmoid_argument(x, fn):
    return ref.C * (x + ref.K * x ** 3) if fn == "gelu_tanh" else x


def act(x, fn):
    if fn == "none":
        return x
    if fn == "gelu":
        return x * 0.5 * torch.special.erfc(-x / math.sqrt(2.0))
    return x * torch.sigmoid(_sigmoid_argument(x, fn))


def slope(x, fn):
    """(the derivative, its second term)."""
    if fn == "gelu":
        second = x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
        return 0.5 * torch.special.erfc(-x / math.sqrt(2.0)) + second, second
    s = torch.sigmoid(_sigmoid_argument(x, fn))
    second = s * (1.0 - s) * x * (ref.C * (1.0 + 3 * ref.K * x * x) if fn == "gelu_tanh" else 1.0)
    return s + second, second


def act_error(x, fn):
    """As grad_ops.act_error."""
    a = {"gelu": 0.5 * x * x, "gelu_tanh": ref.C * (x + ref.K * x ** 3).abs(), "silu": x.abs()}[fn]
    return 4 * a * ref.U32 + 32 * ref.U32 + 2.0 ** -22


def slope_error(x, fn):
    """As _slope_error of tests/test_linear_gpu.py."""
    s, second = slope(x, fn)
    return (s.abs() + 2 * second.abs()) * act_error(x, fn) + 2.0 ** -126 * (1 + 2 * x.abs() * (1 + 3 * ref.K * x * x))


def near(got, want, err, dtype):
    slack = err + ref.HALF[dtype] * (want.abs() + err)
    off = (got.double() - want).abs()
    assert bool((off <= slack).all()), float((off / slack.clamp_min(1e-300)).max())


def checkpoint(rows, cols, fmt):
    ck = ActCheckpoint(rows, cols, fmt, device=DEV)
    ck.codes.fill_(0x55)
    ck.scales.fill_(0x55)
    return ck


def same_checkpoint(a, b):
    """Codes, scales and untouched padding, bit for bit (save's own kernel is tested by itself)."""
    assert torch.equal(a.scales, b.scales) and torch.equal(a.codes, b.codes)


@of(False)
def test_forward(case):
    xt, lt, _, rows, out, inp = case
    ly, w, b = layer(case, inp)
    x = put(base._values(rows, inp, 1, True), xt)
    h = times(x, w.t()) + b
    assert torch.equal(h.float().double(), h)
    y = torch.full((rows, out), 7.0, dtype=xt, device=DEV)
    ly.opt.linear(1, 2, x, ly.list, y)
    assert torch.equal(y, h.float().to(xt))
    ly.opt.linear(1, None, x, ly.list, y)
    assert torch.equal(y, (h - b).float().to(xt))
    kept = {}
    for fmt in ("e4m3", "int8"):
        kept[fmt] = checkpoint(rows, out, fmt)
        kept[fmt].save(h.float())
    r = base._values(rows, out, 2, True)
    for extra, offset in ((0, 0), (8, 8), (3, 1)):        # 16-byte rows, those of a wider matrix, and others
        res = put(r, xt, extra, offset)
        before = res.double()
        fmt = "e4m3" if extra else "int8"
        ck = checkpoint(rows, out, fmt)
        ly.opt.linear(1, 2, x, ly.list, res, residual=res, keep=ck)
        assert torch.equal(res, (h + before).float().to(xt))
        same_checkpoint(ck, kept[fmt])
    for k, fn in enumerate(base.FNS[1:]):
        a = act(h, fn)
        e = act_error(h, fn) * a.abs() + h.abs() * 2.0 ** -126
        fmt = ("e4m3", "int8")[k % 2]
        ck = checkpoint(rows, out, fmt)
        ly.opt.linear(1, 2, x, ly.list, y, act=fn, keep=ck)
        near(y, a, e, xt)
        same_checkpoint(ck, kept[fmt])                    # of h, not of fn(h)
        res = put(r, xt, (0, 8, 3)[k], (0, 8, 1)[k])
        before = res.double()
        ly.opt.linear(1, 2, x, ly.list, res, act=fn, residual=res, keep=ck)
        near(res, a + before, e + ref.U32 * ((a + before).abs() + e), xt)
        same_checkpoint(ck, kept[fmt])


@of(True)
def test_input_grad(case):
    dt, lt, _, rows, out, inp = case
    ly, w, _ = layer(case, out)
    dy = put(base._values(rows, out, 1, True), dt)
    g = times(dy, w)
    assert torch.equal(g.float().double(), g)
    dx = torch.full((rows, inp), 7.0, dtype=dt, device=DEV)
    ly.opt.linear_input_grad(1, dy, ly.list, dx)
    assert torch.equal(dx, g.float().to(dt))
    r = base._values(rows, inp, 2, True)
    for extra, offset in ((0, 0), (8, 8), (3, 1)):
        add = put(r, dt, extra, offset)
        want = (g + add.double()).float().to(dt)
        ly.opt.linear_input_grad(1, dy, ly.list, add, add=add)
        assert torch.equal(add, want)
    z = base._values(rows, inp, 3, False) * 3
    z[:, inp // 2] *= 20.0
    z = z.to(DEV)
    held = torch.empty(rows, inp, device=DEV)
    for k, fn in enumerate(base.FNS[1:]):
        ck = ActCheckpoint(rows, inp, ("int8", "e4m3")[k % 2], device=DEV)
        ck.save(z)
        ck.load(held)
        s, es = slope(held.double(), fn)[0], slope_error(held.double(), fn)
        want = g * s
        e = g.abs() * es + ref.U32 * want.abs()
        ly.opt.linear_input_grad(1, dy, ly.list, dx, act=fn, kept=ck)
        near(dx, want, e, dt)
        add = put(r, dt, (0, 8, 3)[k], (0, 8, 1)[k])
        want = want + add.double()
        ly.opt.linear_input_grad(1, dy, ly.list, add, act=fn, kept=ck, add=add)
        near(add, want, e + ref.U32 * (want.abs() + e), dt)
