"""The gradient-making operators on the GPU at the ends of their ranges: the
largest sizes, element counts past 2^31, and the choices by size that smaller
tests do not reach.  Comparisons with torch run on the GPU, slice by slice."""
import threading

import numpy as np
import pytest
import torch

import grad_ops as ref
import test_grad_ops_gpu as base
from error_compensated_bit_02_amd import ActCheckpoint, OneBitAdam, OneBitError

pytestmark = pytest.mark.gpu
DEV = "cuda"
INVALID, ALIGN = 1, 2
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()      # some cases take tens of GB


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------
def test_lookup_sizes_accepted():
    """Whether sizes fit is decided before the output's alignment: an address off its element tells which
    without a launch."""
    opt = OneBitAdam([8 * 4096], 1)
    ids = torch.zeros(16, dtype=torch.int32, device=DEV)
    params = torch.zeros(opt.N, device=DEV)

    def status(tokens, dim):
        return opt.lib.ob_embedding_lookup(opt._ctx, 0, dim, tokens, ids.data_ptr(), 0, params.data_ptr(), 1.0, 1,
                                           params.data_ptr() + 1, dim, None)

    assert status((1 << 24) - 1, 4096) == ALIGN and status(1 << 20, 4096) == ALIGN and status((1 << 24) - 1, 8 * 4096) == ALIGN
    assert status(1 << 24, 1) == INVALID and status(4, 4095) == INVALID


@pytest.mark.parametrize("extra", [0, 1])
def test_lookup_past_2_to_the_32_elements(extra):
    """Vectors, and single elements where the row stride leaves 16 bytes."""
    tokens, vocab, dim = (1 << 20) + 3, 100, 4096
    opt = OneBitAdam([vocab * dim], 1)
    params = torch.randn(opt.N, generator=base._gen(1)).to(DEV)
    ids = base._ids(tokens, vocab, 2, dtype=torch.int32).clamp_max(vocab - 1).to(DEV)
    out = torch.full((tokens, dim + extra), 7.0, dtype=torch.bfloat16, device=DEV)
    opt.embedding_lookup(0, dim, ids, params, out[:, :dim], scale=2.0)
    table = torch.cat([params[: vocab * dim].view(vocab, dim) * 2.0, torch.zeros(1, dim, device=DEV)]).bfloat16()
    rows = torch.where(ids >= 0, ids, vocab).long()
    for a in range(0, tokens, 1 << 17):
        part = out[a: a + (1 << 17)]
        assert torch.equal(part[:, :dim], table[rows[a: a + (1 << 17)]])
        assert (part[:, dim:] == 7.0).all()


@pytest.mark.parametrize("tokens", [100, 700])
def test_table_of_the_most_rows(tokens):
    """2^31 - 1 rows of one column: the last id an int32 can name and the id behind it; few tokens and sorted ones."""
    vocab = (1 << 31) - 1
    opt = OneBitAdam([vocab], 1)
    ids = torch.randint(0, vocab, (tokens,), generator=base._gen(3))
    ids[:9] = torch.tensor([vocab - 1, 0, vocab, vocab - 1, -1, 1, vocab - 2, vocab + 5, 0])
    params = torch.zeros(opt.N, device=DEV)
    inside = (ids >= 0) & (ids < vocab)
    rows = ids[inside].to(DEV)
    params[rows] = torch.arange(1.0, len(rows) + 1, device=DEV)     # of a row named twice, either
    out = torch.full((tokens, 1), 7.0, device=DEV)
    opt.embedding_lookup(0, 1, ids.to(DEV), params, out, scale=0.5)
    assert torch.equal(out[inside.to(DEV), 0], params[rows] * 0.5)
    assert torch.isnan(out[ids >= vocab]).all() and (out[ids < 0] == 0).all()
    del params
    dy = torch.randint(-4, 5, (tokens, 1), generator=base._gen(4)).float()
    dy[~inside] = float("nan")
    grads = torch.full((1, opt.N), 3.0, device=DEV)
    opt.embedding_grad(0, 0, 1, ids.to(DEV), dy.to(DEV), grads)
    distinct, at = torch.unique(ids[inside], return_inverse=True)
    want = torch.zeros(len(distinct)).index_add_(0, at, dy[inside, 0])
    assert torch.equal(grads[0, distinct.to(DEV)].cpu(), want)
    assert int((grads[0, :vocab] != 0).sum()) == int((want != 0).sum()) and float(grads[0, vocab]) == 3.0


def test_embedding_grad_of_the_most_tokens():
    """2^24 - 1 tokens, a third of them of one row, with values -1..1: sums of at most 2^24, exact in fp32."""
    tokens, vocab, dim = (1 << 24) - 1, 1000, 8
    opt = OneBitAdam([vocab * dim], 1)
    ids = base._ids(tokens, vocab, 5, dtype=torch.int32).to(DEV)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)
    dy = torch.randint(-1, 2, (tokens, dim), generator=gen, device=DEV).float()
    grads = torch.full((1, opt.N), 3.0, device=DEV)
    opt.embedding_grad(0, 0, dim, ids, dy, grads)
    order = torch.argsort(ids, stable=True)        # sums by differences of running sums, in whole numbers
    upto = torch.cat([torch.zeros(1, dim, dtype=torch.int64, device=DEV), dy[order].long().cumsum(0)])
    at = torch.searchsorted(ids[order], torch.arange(vocab + 1, dtype=torch.int32, device=DEV))
    want = upto[at[1:]] - upto[at[:-1]]
    assert torch.equal(grads[0, : vocab * dim].view(vocab, dim).double(), want.double())


def test_embedding_grad_past_2_to_the_31_elements():
    """dY of 2^20 + 1 rows of 2056 columns in bf16: zero but for every 1009th
    row, so the reference is small; whole numbers, exact in fp32."""
    tokens, vocab, dim = (1 << 20) + 1, 40, 2056
    opt = OneBitAdam([vocab * dim], 1)
    ids = base._ids(tokens, vocab, 7, pad=0.0).clamp_max(vocab - 1)
    some = torch.arange(tokens - 1, -1, -1009)
    part = torch.randint(-4, 5, (len(some), dim), generator=base._gen(8)).float()
    dy = torch.zeros(tokens, dim, dtype=torch.bfloat16, device=DEV)
    dy[some.to(DEV)] = part.bfloat16().to(DEV)
    grads = torch.full((1, opt.N), 3.0, device=DEV)
    opt.embedding_grad(0, 0, dim, ids.to(DEV), dy, grads)
    want = torch.zeros(vocab, dim).index_add_(0, ids[some], part)
    assert torch.equal(grads[0, : vocab * dim].view(vocab, dim).cpu(), want)


# ---------------------------------------------------------------------------
# arguments
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("scale", [1e39, -1e39, 3.41e38, float("inf"), float("nan")])
def test_a_scale_past_fp32_is_refused(scale):
    """Finite as a double, infinite as the fp32 that multiplies: zeros would become NaN."""
    opt = OneBitAdam([6 * 8], 1)
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    params, rows = torch.zeros(opt.N, device=DEV), torch.zeros(4, 8, device=DEV)
    grads = torch.full((1, opt.N), 3.0, device=DEV)
    for call in (lambda: opt.embedding_lookup(0, 8, ids, params, rows, scale=scale),
                 lambda: opt.embedding_grad(0, 0, 8, ids, rows, grads, scale=scale)):
        with pytest.raises(OneBitError) as e:
            call()
        assert e.value.status == INVALID
    torch.cuda.synchronize()
    assert (grads == 3.0).all() and (rows == 0).all()


def test_the_largest_scale():
    top = float(np.finfo(np.float32).max)
    opt = OneBitAdam([6 * 8], 1)
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    params, rows = torch.full((opt.N,), 0.5, device=DEV), torch.zeros(4, 8, device=DEV)
    opt.embedding_lookup(0, 8, ids, params, rows, scale=top)
    assert (rows == top / 2).all()


@pytest.mark.parametrize("kind", TYPES)
def test_adding_no_rows_leaves_every_bit(kind):
    """Negative zeros and a NaN with a payload stay what they are."""
    opt = OneBitAdam([6 * 10, 6], 1, "bf16" if kind == torch.bfloat16 else "f32")
    grads = torch.full((1, opt.N), -0.0, dtype=kind, device=DEV)
    bits = grads.view(torch.int16 if kind == torch.bfloat16 else torch.int32)
    bits[0, 3] = 0x7FA5 if kind == torch.bfloat16 else 0x7FC12345
    before = bits.clone()
    none = ActCheckpoint(0, 10, device=DEV)
    opt.linear_grad(0, 0, 1, none, torch.empty(0, 6, device=DEV), grads, accumulate=True)
    opt.embedding_grad(0, 0, 10, torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, 10, device=DEV), grads,
                       accumulate=True)
    assert torch.equal(bits, before)


def test_a_checkpoint_resized_in_place_is_refused():
    opt = OneBitAdam([6 * 10, 6], 1)
    grads, dy, x = torch.full((1, opt.N), 3.0, device=DEV), torch.zeros(40, 6, device=DEV), torch.zeros(40, 10, device=DEV)
    for name in ("codes", "scales"):
        ck = ActCheckpoint(40, 10, device=DEV)
        ck.save(x)
        getattr(ck, name).resize_(0)
        for call in (lambda: opt.linear_grad(0, 0, 1, ck, dy, grads), lambda: ck.save(x), lambda: ck.load(x),
                     lambda: ck.act_backward("gelu", x, x)):
            with pytest.raises(OneBitError, match="resized or moved"):
                call()
    torch.cuda.synchronize()
    assert (grads == 3.0).all()


# ---------------------------------------------------------------------------
# one context, several streams and threads
# ---------------------------------------------------------------------------
def test_one_context_on_two_streams():
    """Two chains of calls on one context, each on a stream and with buffers of its own, give what each gives alone."""
    states = [base._chain_state(30), base._chain_state(40, rows=901)]
    states[1]["opt"] = states[0]["opt"]
    want = []
    for s in states:
        base._chain(**s)
        torch.cuda.synchronize()
        want.append(base._results(s))
    for s in states:
        for k in ("y", "out", "grads"):
            s[k].zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                base._chain(**s)
    torch.cuda.synchronize()
    for s, w in zip(states, want):
        assert all(torch.equal(a, b) for a, b in zip(base._results(s), w))


def test_one_context_in_four_threads_with_profiling():
    """Every launch is counted once, and the results are those of the calls one after the other."""
    calls, threads = 200, 4
    states = [base._chain_state(50 + 10 * k, rows=300 + 77 * k) for k in range(threads)]
    opt = states[0]["opt"]
    want = []
    for s in states:
        s["opt"] = opt
        base._chain(**s)
        torch.cuda.synchronize()
        want.append(base._results(s))
        for k in ("y", "out", "grads"):
            s[k].zero_()
    torch.cuda.synchronize()
    opt.profile(True)
    errors = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(calls):
                    base._chain(**s)
        except Exception as e:      # noqa: BLE001
            errors.append(e)

    runs = [threading.Thread(target=work, args=(s,)) for s in states]
    for r in runs:
        r.start()
    for r in runs:
        r.join()
    torch.cuda.synchronize()
    opt.profile(False)
    counts = {k: n for k, (_, n) in opt.profile_read().items()}
    assert not errors
    for kind in ("embedding_lookup", "embedding_order", "embedding_sum", "linear_grad", "linear_join"):
        assert counts[kind] == calls * threads, kind
    for s, w in zip(states, want):
        assert all(torch.equal(a, b) for a, b in zip(base._results(s), w))


# ---------------------------------------------------------------------------
# fp32 activations
# ---------------------------------------------------------------------------
# Error counted in units u = 2^-24 (half a step of fp32, relative).  A rounded
# operation costs 1; the hardware's exponential is off by one step, 2; its
# argument's rounding is carried along, which costs one more product and leaves
# nothing else: e = exp(-|a|) is off by 3.  A reciprocal with a Newton step: 1.1.
#
#   sigma = 1/(1 + e) for a > 0, e/(1 + e) below; e weighs e/(1 + e) <= 1/2 in the former:
#     above 1.5 + 1 (sum) + 1.1 = 3.6, below 3 + 1 + 1.1 + 1 = 6.1; times x, 1 more.
#   Phi, |x| >= 1.25: t (two roundings' 2.1) weighs at most 2 in P, P's own
#     evaluation 3 and fit 0.7, e 3, two products 2: 12.9 below; above, that is
#     weighed tail/(1 - tail) <= 0.12, and 1 more for the difference.
#   Phi, |x| < 1.25: x*Q is off by 2 (evaluation) and 0.8 (fit), the sum by 1:
#     below 2.8 * 0.394/0.106 + 1 = 11.4, for x >= -1 2.8 * 0.341/0.159 + 1 = 7.0,
#     above 2.8 * 0.394/0.894 + 1 = 2.3.  Times x, 1 more.
def _value_units(x, fn):
    if fn == "gelu":
        return np.where(x >= 0, 4.0, np.where(x >= -1, 8.0, 16.0))
    return np.where(x >= 0, 5.0, 8.0)


def _slope_error(x, fn):
    """Both terms of act'(x): Phi or sigma as above, and x*gauss/sqrt(2 pi) (x/sqrt(2 pi) 2,
    e 3, product fused) or sigma*(1 - sigma)*v'(x)*x (e 3, two reciprocals and sums 4.2, two
    products 2; for gelu_tanh x*v' 5 more); the sum 1."""
    if fn == "gelu":
        s, units = ref._phi(x), 6.0
    else:
        s = ref._sigmoid(ref.C * (x + ref.K * x ** 3) if fn == "gelu_tanh" else x)
        units = 10.0 if fn == "silu" else 15.0
    slope = ref.act_slope(x, fn)
    return (_value_units(x, fn) * s + units * np.abs(slope - s) + np.abs(slope)) * ref.U32


def _dense(seed):
    """Both signs, every size from 2^-20 to 12, most of them where most values lie."""
    g = base._gen(seed)
    x = torch.cat([torch.rand(60000, generator=g) * 24 - 12, torch.rand(60000, generator=g) * 2 - 1,
                   torch.exp2(torch.rand(8000, generator=g) * 20 - 20) * (torch.randint(0, 2, (8000,), generator=g) * 2 - 1)])
    return x.view(1000, 128)


@pytest.mark.parametrize("fn", base.FNS)
def test_fp32_activation_to_its_last_bits(fn):
    x = _dense(60).to(DEV)
    y = torch.empty_like(x)
    ActCheckpoint(1000, 128, device=DEV).save(x, act=fn, y=y)
    x64 = base._f64(x)
    want = ref.act(x64, fn)
    lim = np.abs(want) * _value_units(x64, fn) * ref.U32 + np.abs(x64) * 2.0 ** -126      # sigma below 2^-126 may be 0
    off = np.abs(base._f64(y) - want)
    assert (off <= lim).all(), (float((off / lim).max()), x64.flat[(off / lim).argmax()])


@pytest.mark.parametrize("fn", base.FNS)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_fp32_backward_to_its_last_bits(fn, fmt):
    ck = ActCheckpoint(1000, 128, fmt, device=DEV)
    ck.save(_dense(61).to(DEV))
    xhat = ref.decoded(ck.codes.cpu().numpy(), ck.scales.cpu().numpy(), 128, fmt)
    dy = torch.randn(1000, 128, generator=base._gen(62)).to(DEV)
    dx = torch.empty_like(dy)
    ck.act_backward(fn, dy, dx)
    dy64, slope = base._f64(dy), ref.act_slope(xhat, fn)
    # one rounding more for dy; what a factor below 2^-126 loses, times at most 2|x|(1 + 3*0.044715 x^2)
    lim = np.abs(dy64) * (_slope_error(xhat, fn) + np.abs(slope) * ref.U32
                          + 2.0 ** -126 * (1 + 2 * np.abs(xhat) * (1 + 3 * ref.K * xhat * xhat)))
    off = np.abs(base._f64(dx) - dy64 * slope)
    assert (off <= lim).all(), (float((off / lim).max()), xhat.flat[(off / lim).argmax()])


@pytest.mark.parametrize("fn", base.FNS)
@pytest.mark.parametrize("dtype", TYPES)
def test_activation_of_infinities_and_huge_values(fn, dtype):
    x = torch.tensor([[float("inf"), float("nan"), 3e38, 1e30, 1e15, 200.0, 64.0, 0.0, -64.0, -200.0, -1e15, -1e30, -3e38]],
                     device=DEV).to(dtype)
    y = torch.empty_like(x)
    ActCheckpoint(1, x.shape[1], device=DEV).save(x, act=fn, y=y)
    assert torch.equal(y[0, 2:8], x[0, 2:8]) and torch.isnan(y[0, 1]) and float(y[0, 0]) == float("inf")
    assert (y[0, 9:] == 0).all()
    assert float(y[0, 8].abs()) <= 1.04e-26      # silu: 64 * exp(-64) = 1.027e-26, half a bf16 step more 1.031e-26


def test_save_of_more_tiles_than_one_launch_dimension():
    """2^29 + 5 rows of one column are 2^24 + 1 tiles; the rows at both ends as
    those of a matrix of their own."""
    rows, n = (1 << 29) + 5, 4096 + 5
    x = torch.zeros(rows, 1, device=DEV)
    ends = torch.randn(2, n, 1, generator=base._gen(63)).to(DEV)
    x[:n], x[-n:] = ends[0], ends[1]
    ck = ActCheckpoint(rows, 1, "int8", device=DEV)
    y = torch.full((rows, 1), 7.0, device=DEV)
    ck.save(x, act="silu", y=y)
    small = ActCheckpoint(n, 1, "int8", device=DEV)
    out = torch.empty(n, 1, device=DEV)
    for part, end in ((slice(0, n), ends[0]), (slice(rows - n, rows), ends[1])):
        small.save(end, act="silu", y=out)
        assert torch.equal(y[part], out)
        # whole blocks of 32 rows: those of the small matrix begin at the same rows
        at = 0 if part.start == 0 else part.start // 32
        assert torch.equal(ck.codes[part, :1], small.codes[:, :1])
        assert torch.equal(ck.scales[at: at + (n + 31) // 32, :1], small.scales[:, :1])
    assert (y[n:-n] == 0).all()
    dy = y
    dy.fill_(1.0)
    ck.act_backward("silu", dy, dy)
    small.act_backward("silu", torch.ones(n, 1, device=DEV), out)
    assert torch.equal(dy[-n:], out) and (dy[n:-n] == 0.5).all()


# ---------------------------------------------------------------------------
# the order of the sums
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dy_dtype", TYPES)
@pytest.mark.parametrize("rows,out,inp", [(6000, 2056, 2050), (900, 264, 136)])
def test_linear_grad_bits_by_layout(rows, out, inp, dy_dtype):
    """Buffers of one row stride and alignment give the same bits, wherever they
    lie; other strides and alignments may sum in another order, within the bound
    of any order (n roundings, twice that for the matrix unit)."""
    opt = OneBitAdam([out * inp, out], 1)
    x = torch.randn(rows, inp, generator=base._gen(70))
    ck = base._checkpoint(x.to(DEV), "e4m3")
    dy = torch.randn(rows, out, generator=base._gen(71)).to(dy_dtype)

    def run(extra, offset):
        grads = torch.zeros(1, opt.N, device=DEV)
        opt.linear_grad(0, 0, 1, ck, base._put(dy, dy_dtype, extra, offset)[0], grads)
        return grads[0, : out * inp].view(out, inp).clone(), grads[0, opt.offsets[1]: opt.offsets[1] + out].clone()

    xhat = torch.empty(rows, inp, device=DEV)
    ck.load(xhat)
    dy64 = dy.double().to(DEV)
    mag = dy64.abs().t().contiguous() @ xhat.double().abs()
    want = dy64.t().contiguous() @ xhat.double()
    for extra, offset in ((0, 0), (8, 0), (0, 1), (3, 0)):
        first, again = run(extra, offset), run(extra, offset + 64)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert ((first[0].double() - want).abs() <= 2 * (rows + 8) * ref.U32 * mag + 2.0 ** -126).all()
        assert ((first[1].double() - dy64.sum(0)).abs() <= 2 * (rows + 8) * ref.U32 * dy64.abs().sum(0)).all()


# ---------------------------------------------------------------------------
# variants by size
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("grad", TYPES)
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("rows,out,inp,extra", [
    (1500, 2056, 4100, 0),      # 256 x 256 tiles, rows of four columns each
    (1500, 2056, 4101, 8),      # the same without
    (6000, 2056, 2050, 0),      # and the rows in three slices
    (16384, 2048, 2048, 0),     # four slices, whole tiles only
])
def test_linear_grad_of_large_tiles(rows, out, inp, extra, fmt, grad, bias):
    """Whole numbers, sums of at most 16384 * 8 * 2 = 2^18 exact in fp32 and rounded once to the gradient's type."""
    opt = OneBitAdam([5, out * inp, out, 9], 1, "bf16" if grad == torch.bfloat16 else "f32")
    x = torch.randint(-8, 9, (rows, inp), generator=base._gen(80)).float().to(DEV)
    dy, _ = base._put(torch.randint(-2, 3, (rows, out), generator=base._gen(81)).float(), torch.bfloat16, extra, 0)
    ck = base._checkpoint(x, fmt)       # at most 8 = 2^3: exact in both formats
    dw = dy.double().t().contiguous() @ x.double()
    db = dy.double().sum(0)
    a, b = opt.offsets[1], opt.offsets[2]
    grads = torch.full((1, opt.N), 3.0, dtype=grad, device=DEV)
    opt.linear_grad(0, 1, 2 if bias else None, ck, dy, grads)
    weight, column = grads[0, a: a + out * inp].view(out, inp), grads[0, b: b + out]
    assert torch.equal(weight, dw.to(grad))
    assert torch.equal(column, db.to(grad) if bias else torch.full_like(column, 3.0))
    old, old_b = weight.double(), column.double()
    opt.linear_grad(0, 1, 2 if bias else None, ck, dy, grads, accumulate=True)
    assert torch.equal(weight, (old + dw).to(grad))
    assert torch.equal(column, (old_b + db).to(grad) if bias else old_b.to(grad))
    base._others_untouched(opt, grads, 0, [1, 2] if bias else [1])


@pytest.mark.parametrize("dy_dtype", TYPES)
@pytest.mark.parametrize("tokens,dim", [(100, 66001), (40, 8 * 66000)])
def test_embedding_grad_of_few_wide_tokens(tokens, dim, dy_dtype):
    """More slices of columns than workgroups along them: each takes several,
    with tokens of one row in several wavefronts.  Whole numbers, exact."""
    vocab = 3
    opt = OneBitAdam([70, vocab * dim, 4], 2)
    ids = base._ids(tokens, vocab, 82)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(83)
    dy = torch.randint(-4, 5, (tokens, dim), generator=gen, device=DEV).to(dy_dtype)
    inside = ((ids >= 0) & (ids < vocab)).to(DEV)
    want = torch.zeros(vocab, dim, device=DEV)
    for v in range(vocab):
        want[v] = dy[(ids == v).to(DEV)].float().sum(0)
    dy[~inside] = float("nan")
    grads = torch.full((2, opt.N), 3.0, device=DEV)
    a = opt.offsets[1]
    opt.embedding_grad(1, 1, dim, ids.to(DEV), dy, grads, scale=0.5)
    got = grads[1, a: a + vocab * dim].view(vocab, dim)
    assert torch.equal(got, 0.5 * want)
    opt.embedding_grad(1, 1, dim, ids.to(DEV), dy, grads, scale=-1.0, accumulate=True)
    assert torch.equal(got, -0.5 * want)
    base._others_untouched(opt, grads, 1, [1])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,cols", [(5, 33), (100, 65), (97, 130), (40, 1)])
def test_padding_bytes_reach_no_result(rows, cols, fmt):
    """Columns past the last of a checkpoint hold what the buffer held: here the
    scale of a NaN block and codes of NaN, 0 elsewhere for comparison."""
    x = base._activations(rows, cols, 84).to(DEV)
    dy = torch.randn(rows, 24, generator=base._gen(85)).to(DEV)
    opt = OneBitAdam([24 * cols, 24], 1)
    results = []
    for code, scale in ((0xFF, 0xFF), (0x7F, 0xFF), (0, 0)):
        ck = ActCheckpoint(rows, cols, fmt, device=DEV)
        ck.codes.fill_(code)
        ck.scales.fill_(scale)
        ck.save(x)
        out, dx = torch.empty_like(x), torch.empty_like(x)
        grads = torch.zeros(1, opt.N, device=DEV)
        ck.load(out)
        ck.act_backward("gelu", out, dx)
        opt.linear_grad(0, 0, 1, ck, dy, grads)
        half = torch.zeros(1, opt.N, device=DEV)
        opt.linear_grad(0, 0, 1, ck, dy.bfloat16(), half)
        results.append((out, dx, grads, half))
        assert all(torch.isfinite(t).all() for t in results[-1])
    for r in results[:2]:
        assert all(torch.equal(p, q) for p, q in zip(r, results[2]))


# ---------------------------------------------------------------------------
# past 2^31 elements
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", TYPES)
def test_checkpoint_past_2_to_the_31_elements(fmt, dtype):
    """2^19 + 39 rows of 4104 columns; the last blocks as those of a matrix of their own."""
    rows, cols, n = (1 << 19) + 39, 4104, 32 * 40 + 7
    gen = torch.Generator(device=DEV)
    gen.manual_seed(86)
    x = torch.zeros(rows, cols, dtype=dtype, device=DEV)
    end = torch.randn(n, cols, generator=gen, device=DEV).to(dtype)
    x[-n:] = end
    ck, small = ActCheckpoint(rows, cols, fmt, device=DEV), ActCheckpoint(n, cols, fmt, device=DEV)
    out = torch.empty(n, cols, dtype=dtype, device=DEV)
    small.save(end, act="gelu", y=out)
    ck.save(x, act="gelu", y=x)                        # in place
    assert torch.equal(x[-n:], out) and int(torch.count_nonzero(x[:-n])) == 0
    assert torch.equal(ck.codes[-n:, :cols], small.codes[:, :cols])
    assert torch.equal(ck.scales[-small.scales.shape[0]:, :cols], small.scales[:, :cols])
    ck.load(x)
    small.load(out)
    assert torch.equal(x[-n:], out) and int(torch.count_nonzero(x[:-n])) == 0
    x.fill_(1.0)
    ck.act_backward("silu", x, x)
    small.act_backward("silu", torch.ones_like(out), out)
    assert torch.equal(x[-n:], out) and int(torch.count_nonzero(x[:-n] != 0.5)) == 0


@pytest.mark.parametrize("dy_dtype", TYPES)
@pytest.mark.parametrize("wide", ["dy", "x"])
def test_linear_grad_past_2_to_the_31_elements(wide, dy_dtype):
    """2^20 + 5 rows of 2056 elements in dY (8 of them contracted) or in the
    input; zero but for rows at both ends, whole numbers, exact in fp32."""
    rows, n = (1 << 20) + 5, 700
    out, inp = (8, 24) if wide == "dy" else (8, 2056)
    opt = OneBitAdam([out * inp, out], 1)
    x = torch.zeros(rows, inp, dtype=torch.bfloat16, device=DEV)
    dy = torch.zeros(rows, 2056 if wide == "dy" else out, dtype=dy_dtype, device=DEV)[:, :out]
    some = torch.cat([torch.arange(n), torch.arange(rows - n, rows)]).to(DEV)
    xs = torch.randint(-8, 9, (2 * n, inp), generator=base._gen(87)).to(DEV)
    ds = torch.randint(-4, 5, (2 * n, out), generator=base._gen(88)).to(DEV)
    x[some], dy[some] = xs.bfloat16(), ds.to(dy_dtype)
    ck = ActCheckpoint(rows, inp, "int8", device=DEV)
    ck.save(x)
    grads = torch.zeros(1, opt.N, device=DEV)
    opt.linear_grad(0, 0, 1, ck, dy, grads)
    assert torch.equal(grads[0, : out * inp].view(out, inp).double(), ds.double().t().contiguous() @ xs.double())
    b = opt.offsets[1]
    assert torch.equal(grads[0, b: b + out].double(), ds.double().sum(0))


# ---------------------------------------------------------------------------
# tiny gradients
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows", [4, 64])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dy_dtype", TYPES)
def test_linear_grad_of_tiny_values(rows, fmt, dy_dtype):
    """One row of dY from 1e-28 down into the subnormals.  A bf16 dY and few
    rows lose nothing but fp32's own rounding; of an fp32 dY, what its three
    bf16 parts cannot hold, less than 2^-133 each, is lost."""
    opt = OneBitAdam([16 * 8, 16], 1)
    x = torch.zeros(rows, 8)
    x[0] = torch.tensor([1.0, 2.0 ** 20, 2.0 ** -20, 1.5 * 2.0 ** -60, -1.0, 0.0, 3.0, 96.0])
    dy = torch.zeros(rows, 16)
    dy[0] = 1.2345678 * 10.0 ** -torch.arange(28.0, 44.0, dtype=torch.float64)
    ck = base._checkpoint(x.to(DEV), fmt)
    dyg = dy.to(dy_dtype).to(DEV)
    grads = torch.zeros(1, opt.N, device=DEV)
    opt.linear_grad(0, 0, 1, ck, dyg, grads)
    dy64, x64 = base._f64(dyg)[0], x[0].double().numpy()
    lost = 2.0 ** -133 if rows >= 8 and dy_dtype == torch.float32 else 0.0
    want = np.outer(dy64, x64)
    lim = lost * np.abs(x64) + np.abs(want) * ref.U32 + 2.0 ** -150       # the last: half of fp32's smallest step
    assert (np.abs(base._f64(grads[0, :128].view(16, 8)) - want) <= lim).all()
    b = opt.offsets[1]
    assert (np.abs(base._f64(grads[0, b: b + 16]) - dy64) <= lost).all()
