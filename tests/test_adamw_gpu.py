"""The AdamW step on the GPU, its moments as fp32 and in 8 bits, against the
definitions of tests/layer_ops.py: every operation of the step rounds once, so
its results must match bit for bit."""
import numpy as np
import pytest
import torch

import layer_ops as ref
from error_compensated_bit_02_amd import OneBitAdam, OneBitError

pytestmark = pytest.mark.gpu
DEV = "cuda"
SIZES = [1, 2, 3, 63, 64, 65, 127, 1000, 1023, 1024, 1025, 5000, 8191, 8192, 8193, 20000]
HYPER = dict(beta1=0.9, beta2=0.999, eps=1e-8)


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")


class List:
    """A list of tensors with its device buffers, its padding marked, and the reference's copies."""

    def __init__(self, numel, workers, grad, moments, seed, model=True, decay=True, gscale=None, sigma=None, eps=1e-8):
        self.numel, self.W, self.kind = list(numel), workers, moments
        self.opt = OneBitAdam(self.numel, workers, grad, beta1=HYPER["beta1"], eps=eps)
        self.off, self.N = self.opt.offsets, self.opt.N
        self.dtype = torch.bfloat16 if grad == "bf16" else torch.float32
        self.eps = eps
        gen = torch.Generator()
        gen.manual_seed(seed)
        self.gen = gen
        self.sigma = sigma if sigma is not None else [10.0 ** (-(t % 7)) for t in range(len(self.numel))]
        self.p = [torch.randn(n, generator=gen).numpy() * ref.F(0.02) for n in self.numel]
        self.m = [np.zeros(n, ref.F) for n in self.numel]
        self.v = [np.zeros(n, ref.F) for n in self.numel]
        self.real = torch.zeros(self.N, dtype=torch.bool)
        for n, o in zip(self.numel, self.off):
            self.real[o:o + n] = True
        self.params = self.flat(self.p, torch.float32)
        self.state = self.opt.adamw_state(moments)
        self.marks = {}
        for k, t in self.state.items():
            if t.numel() == self.N:
                t[~self.real.to(DEV)] = 0x55 if t.dtype == torch.uint8 else float("nan")
        self.model = torch.full((self.N,), 7.0, dtype=torch.bfloat16, device=DEV) if model else None
        self.decay = torch.rand(len(self.numel), generator=gen) if decay else None
        self.decay_d = self.decay.to(DEV) if decay else None
        self.gscale = gscale
        self.gscale_d = None if gscale is None else torch.tensor([gscale], device=DEV)

    def flat(self, parts, dtype, fill=float("nan")):
        t = torch.full((self.N,), fill, dtype=dtype)
        for x, n, o in zip(parts, self.numel, self.off):
            t[o:o + n] = torch.from_numpy(np.asarray(x)).to(dtype)
        return t.to(DEV)

    def part(self, flat, t):
        return flat[self.off[t]: self.off[t] + self.numel[t]].cpu()

    def new_grads(self):
        g = torch.full((self.W, self.N), float("nan"), dtype=self.dtype)
        for t, (n, o) in enumerate(zip(self.numel, self.off)):
            x = torch.randn(self.W, n, generator=self.gen) * self.sigma[t]
            x[:, ::5] = 0.0
            g[:, o:o + n] = x.to(self.dtype)
        return g.to(DEV)

    def step(self, grads, step, lr=1e-3, wd=0.1, seed=0, **more):
        self.opt.adamw_step(grads, self.state, self.params, step, lr, beta2=HYPER["beta2"], weight_decay=wd,
                            decay=self.decay_d, grad_scale=self.gscale_d, model=self.model, seed=seed, **more)

    def check(self, grads, step, lr=1e-3, wd=0.1, seed=0):
        """One step of the reference, and every bit of the device's buffers against it."""
        for t, n in enumerate(self.numel):
            g = torch.stack([self.part(grads[w], t) for w in range(self.W)]).float().numpy()
            d = 1.0 if self.decay is None else float(self.decay[t])
            m, v, r, p = ref.adamw(g, self.m[t], self.v[t], self.p[t], beta1=HYPER["beta1"], beta2=HYPER["beta2"],
                                   eps=self.eps, lr=lr, step=step, weight_decay=wd, decay=d, grad_scale=self.gscale)
            self.p[t] = p
            same(self.part(self.params, t).numpy(), p)
            if self.model is not None:
                same(self.part(self.model, t).float().numpy(), torch.from_numpy(p).to(torch.bfloat16).float().numpy())
            if self.kind == "f32":
                self.m[t], self.v[t] = m, v
                same(self.part(self.state["m"], t).numpy(), m)
                same(self.part(self.state["v"], t).numpy(), v)
                continue
            places = np.arange(n, dtype=np.uint64) + np.uint64(self.off[t])
            mc, ms, rc, rs = ref.encode(m, r, places, seed)
            b = slice(self.off[t] // 64, self.off[t + 1] // 64)
            assert np.array_equal(self.state["m_scale"][b].cpu().numpy(), ms), t
            assert np.array_equal(self.state["v_scale"][b].cpu().numpy(), rs), t
            assert np.array_equal(self.part(self.state["m"], t).numpy(), mc), t
            assert np.array_equal(self.part(self.state["v"], t).numpy(), rc), t
            with np.errstate(all="ignore"):
                self.m[t] = ref.decode_m(mc, ms)
                root = ref.decode_r(rc, rs)
                self.v[t] = root * root
        pad = ~self.real.to(DEV)
        assert torch.isnan(self.params[pad]).all()
        if self.model is not None:
            assert (self.model[pad] == 7.0).all()
        for k in ("m", "v"):
            x = self.state[k][pad]
            assert (x == 0x55).all() if x.dtype == torch.uint8 else torch.isnan(x).all()


def same(got, want):
    got, want = np.asarray(got, ref.F), np.asarray(want, ref.F)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(got[~nan].view(np.uint32), want[~nan].view(np.uint32)), np.abs(got[~nan] - want[~nan]).max()


@pytest.mark.parametrize("moments", ["f32", "8bit"])
@pytest.mark.parametrize("grad,workers", [("f32", 1), ("bf16", 1), ("f32", 2), ("bf16", 3), ("f32", 5), ("f32", 8), ("bf16", 9)])
def test_steps(moments, grad, workers):
    """Ragged tensors over four steps from the zero state; the padding holds NaN and stays."""
    x = List(SIZES, workers, grad, moments, seed=workers, gscale=0.37 if workers != 2 else None, model=workers != 3,
             decay=workers != 5)
    for step in range(1, 5):
        g = x.new_grads()
        x.step(g, step, seed=(step << 32) + 11 * step)
        x.check(g, step, seed=(step << 32) + 11 * step)


@pytest.mark.parametrize("moments", ["f32", "8bit"])
def test_one_tensor_of_one_element(moments):
    x = List([1], 1, "f32", moments, seed=3, sigma=[1.0], model=False, decay=False)
    for step in (1, 2, 1000, 10 ** 9):
        g = torch.ones_like(x.new_grads()) * step
        x.step(g, step, wd=0.0)
        x.check(g, step, wd=0.0)


def test_against_the_formula_in_64_bits():
    """Errors counted: with W = 2 the mean, scaled, has 3 half steps; m 2 more of each term, v 3 of g^2's doubled error
    (2*3 + 3); the root halves v's, its products and the quotient add 6, the last difference one of p.  All in units of
    2^-24: m 8 of the terms' magnitudes, v 16 of v, the update 32 of itself."""
    x = List([5000, 33], 2, "f32", "f32", seed=8, gscale=0.7, sigma=[1e-3, 10.0], eps=1e-4)
    u = 2.0 ** -24
    for step in range(1, 6):
        g = x.new_grads()
        before = [(m.copy(), v.copy(), p.copy()) for m, v, p in zip(x.m, x.v, x.p)]
        x.step(g, step)
        x.check(g, step)
        for t in range(2):
            gt = torch.stack([x.part(g[w], t) for w in range(2)]).numpy()
            m, v, p = ref.adamw64(gt, *before[t], beta1=0.9, beta2=0.999, eps=1e-4, lr=1e-3, step=step, weight_decay=0.1,
                                  decay=float(x.decay[t]), grad_scale=np.float64(np.float32(0.7)))
            mag = 0.9 * np.abs(before[t][0]) + 0.1 * 0.7 * np.abs(gt).sum(axis=0) / 2
            assert (np.abs(x.part(x.state["m"], t).numpy() - m) <= 8 * u * mag).all()
            gm = 0.7 * np.abs(gt).sum(axis=0) / 2      # where the two gradients cancel, their mean's error is that of the terms
            assert (np.abs(x.part(x.state["v"], t).numpy() - v) <= 16 * u * (v + 0.001 * gm * gm)).all()
            # per element: the update's own error and m's through it, and the roundings of p and its decay
            mh, vh = m / (1 - 0.9 ** step), v / (1 - 0.999 ** step)
            upd = 1e-3 * (np.abs(mh) + 8 * u * mag / (1 - 0.9 ** step)) / (np.sqrt(vh) + 1e-4)
            slack = 1e-3 * 8 * u * mag / (1 - 0.9 ** step) / (np.sqrt(vh) + 1e-4)
            worse = 16 * u * (1 + 0.001 * gm * gm / np.maximum(v, 1e-300))
            assert (np.abs(x.part(x.params, t).numpy() - p) <= slack + upd * (16 * u + worse) + 3 * u * np.abs(p)).all()


@pytest.mark.parametrize("moments", ["f32", "8bit"])
def test_wide_range_of_gradients(moments):
    """Gradients from 1e-25 to 1e17 within one block, denormal ones, zeros of both signs: bit for bit."""
    x = List([640], 1, "f32", moments, seed=4, sigma=[1.0], decay=False)
    g = x.new_grads()
    e = torch.linspace(-25, 17, 64, dtype=torch.float64)
    g[0, :64] = (10.0 ** e).float().to(DEV)
    g[0, 64:128] = -(10.0 ** (e - 17)).float().to(DEV)
    g[0, 128:192] = 1e-41
    g[0, 192:256] = 0.0
    g[0, 256:320] = -0.0
    for step in (1, 2, 3):
        x.step(g, step, seed=step)
        x.check(g, step, seed=step)


@pytest.mark.parametrize("moments", ["f32", "8bit"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1e30])
def test_non_finite(moments, bad):
    """A gradient that is not finite (or whose square is not) stays in its element, in 8 bits in its block of 64."""
    x = List([1000, 70], 2, "f32", moments, seed=5)
    g = x.new_grads()
    g[1, 130] = bad
    g[0, x.off[1] + 69] = bad
    x.step(g, 1)
    x.check(g, 1)
    g = x.new_grads()
    x.step(g, 2, seed=9)
    x.check(g, 2, seed=9)
    if moments == "8bit":
        m, v = torch.zeros(2, x.N, device=DEV)
        x.opt.adamw_load(x.state, m, v)
        for f in (m, v):
            assert torch.isnan(f[128:192]).all() == (bad != 1e30 or f is v)


def test_load():
    """Values of every code at small, middle and large scales, in both types; padding stays."""
    n = 256 * 5 + 33
    opt = OneBitAdam([n, 10], 1)
    scales = [0, 16, 127, 170, 255]
    codes = torch.zeros(opt.N, dtype=torch.uint8)
    codes[: 256 * 5] = torch.arange(256, dtype=torch.uint8).repeat(5)
    s = torch.full((opt.Nw,), 100, dtype=torch.uint8)
    s[:20] = torch.tensor(scales, dtype=torch.uint8).repeat_interleave(4)
    st = {"m": codes.to(DEV), "v": codes.to(DEV), "m_scale": s.to(DEV), "v_scale": s.to(DEV)}
    c, b = codes.numpy(), s.numpy().copy()
    zero = np.repeat(b, 64) == 0         # scale byte 0 belongs to zero-filled buffers: all codes 0
    c[zero] = 0
    st["m"].copy_(torch.from_numpy(c))
    st["v"].copy_(torch.from_numpy(c))
    st["m"][256 * 4: 256 * 5] = 0        # as the step writes a block that is NaN
    st["v"][256 * 4: 256 * 5] = 0
    c[256 * 4: 256 * 5] = 0
    with np.errstate(all="ignore"):
        m = ref.decode_m(c, b)
        m[(c & 127) == 127] = np.nan
        r = ref.decode_r(c, b)
        v = r * r
    for dtype in (torch.float32, torch.bfloat16):
        mo, vo = (torch.full((opt.N,), 7.0, dtype=dtype, device=DEV) for _ in range(2))
        opt.adamw_load(st, mo, vo)
        real = torch.zeros(opt.N, dtype=torch.bool)
        real[:n] = True
        real[opt.offsets[1]: opt.offsets[1] + 10] = True
        for got, want in ((mo, m), (vo, v)):
            w = torch.from_numpy(want).to(dtype).float().numpy()
            same(got.float().cpu().numpy()[real], w[real.numpy()])
            assert (got.cpu()[~real] == 7.0).all()


def test_rounding_is_unbiased():
    """A moment a quarter of a step above a code takes the upper one for a quarter of the places, within 6 standard
    deviations of a fair draw, and other seeds draw anew."""
    n = 1 << 16
    opt = OneBitAdam([n], 1, beta1=0.0)
    g = torch.full((1, n), 1.03125, device=DEV)      # e4m3's step at 1 is 1/8
    g[0, ::64] = 448.0 / 256                         # the block's largest: scale 2^-8
    p = torch.zeros(n, device=DEV)
    st = opt.adamw_state("8bit")
    ups = []
    for seed in (1, 2, 1 << 40):
        opt.adamw_step(g, st, p, 1, 0.0, beta2=0.0, seed=seed)
        m, v = torch.zeros(2, n, device=DEV)
        opt.adamw_load(st, m, v)
        keep = torch.arange(n, device=DEV) % 64 != 0
        assert ((m == 1.0) | (m == 1.125))[keep].all()
        # r = 1.03125 is half a step of 1/16 above 1
        assert torch.isclose(v.sqrt(), torch.where(v > 1.03125 ** 2, 1.0625, 1.0), rtol=1e-6)[keep].all()
        up_m, up_v = (m > 1.03)[keep], (v > 1.03125 ** 2)[keep]
        k = int(keep.sum())
        assert abs(int(up_m.sum()) - 0.25 * k) < 6 * (0.25 * 0.75 * k) ** 0.5
        assert abs(int(up_v.sum()) - 0.5 * k) < 6 * (0.25 * k) ** 0.5
        ups.append(up_m)
    assert 0.3 < float((ups[0] ^ ups[1]).float().mean()) < 0.45      # 2 * 0.25 * 0.75 = 0.375
    assert 0.3 < float((ups[0] ^ ups[2]).float().mean()) < 0.45


def test_places_past_32_bits_of_a_long_list():
    """A list whose first tensor passes 2^32 elements: the places beyond have dithers of their own."""
    n = (1 << 32) + 64
    need = 16 * n
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip("not enough memory")
    opt = OneBitAdam([n, 1000], 1, "bf16")
    grads = torch.zeros(1, opt.N, dtype=torch.bfloat16, device=DEV)
    tail = slice((1 << 32) - 64, opt.N)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    grads[0, tail] = torch.randn(opt.N - tail.start, generator=gen, device=DEV).to(torch.bfloat16)
    params = torch.zeros(opt.N, device=DEV)
    st = opt.adamw_state("8bit")
    opt.adamw_step(grads, st, params, 1, 1e-3, seed=77)
    for a, b in ((tail.start, n), (opt.offsets[1], opt.offsets[1] + 1000)):
        g = grads[0, a:b].float().cpu().numpy()[None]
        z = np.zeros(b - a, ref.F)
        m, v, r, p = ref.adamw(g, z, z, z, beta1=0.9, beta2=0.999, eps=1e-8, lr=1e-3, step=1)
        mc, ms, rc, rs = ref.encode(m, r, np.arange(a, b, dtype=np.uint64), 77)
        same(params[a:b].cpu().numpy(), p)
        assert np.array_equal(st["m"][a:b].cpu().numpy(), mc) and np.array_equal(st["v"][a:b].cpu().numpy(), rc)
        assert np.array_equal(st["m_scale"][a // 64: (b + 63) // 64].cpu().numpy(), ms)
    assert int(st["m"][: tail.start].count_nonzero()) == 0 and int(params[: tail.start].count_nonzero()) == 0


def test_repeats_and_streams_and_graphs():
    """The same step on another stream and as a graph's replays, with other work between them: the same bits."""
    a = List([5000, 77], 2, "bf16", "8bit", seed=6, gscale=0.5)
    g = a.new_grads()
    keep = {k: t.clone() for k, t in a.state.items()}
    p0 = a.params.clone()
    a.step(g, 5, seed=123)
    want = {k: t.clone() for k, t in a.state.items()} | {"p": a.params.clone(), "model": a.model.clone()}

    def restore():
        for k, t in keep.items():
            a.state[k].copy_(t)
        a.params.copy_(p0)
        a.model.fill_(7.0)

    def check():
        torch.cuda.synchronize()
        got = dict(a.state) | {"p": a.params, "model": a.model}
        for k, t in want.items():
            assert torch.equal(got[k].view(torch.uint8), t.view(torch.uint8)), k

    restore()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step(g, 5, seed=123, stream=side)
    check()
    restore()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(g, 5, seed=123)
    for _ in range(3):
        restore()
        torch.randn(1000, device=DEV).sum().item()
        graph.replay()
        check()


def test_warmup_in_8_bits_then_compression():
    """Three AdamW steps, the moments handed over, then two steps of the compression phase, as a program runs them."""
    numel = [3000, 64, 9000]
    x = List(numel, 2, "f32", "8bit", seed=10, sigma=[1e-2, 1e-2, 1e-3])
    for step in range(1, 4):
        g = x.new_grads()
        x.step(g, step, seed=step)
        x.check(g, step, seed=step)
    opt, N = x.opt, x.N
    m, v = torch.zeros(2, N, device=DEV)
    opt.adamw_load(x.state, m, v)
    for t in range(3):
        same(x.part(m, t).numpy(), x.m[t])
        same(x.part(v, t).numpy(), x.v[t])
    err_w, err_s = torch.zeros(2, N, device=DEV), torch.zeros(N, device=DEV)
    b = opt.alloc(DEV)
    opt.begin_compression(err_w, err_s)
    before = x.params.clone()
    for step in range(2):
        opt.step_residual(step == 0, torch.nan_to_num(x.new_grads()), m, v, x.params, err_w, err_s, b["packed_w"], b["scale_w"],
                          b["packed_s"], b["scale_s"], 1e-4)
    real = x.real.to(DEV)
    assert torch.isfinite(x.params[real]).all() and not torch.equal(before[real], x.params[real])
    assert torch.isnan(x.params[~real]).all()


def test_refusals():
    x = List([100], 1, "f32", "8bit", seed=1)
    g = x.new_grads()
    ok = dict(step=1, lr=1e-3)

    def refused(match, grads=g, state=None, params=x.params, **k):
        before = {n: t.clone() for n, t in x.state.items()}
        with pytest.raises(OneBitError, match=match):
            x.opt.adamw_step(grads, x.state if state is None else state, params, **{**ok, **k})
        for n, t in before.items():
            assert torch.equal(t, x.state[n])

    refused("status 1", step=0)
    refused("status 1", lr=float("nan"))
    refused("status 1", lr=1e39)
    refused("status 1", beta2=1.0)
    refused("status 1", beta2=-0.1)
    refused("status 1", weight_decay=-1.0)
    refused("status 1", weight_decay=float("inf"))
    refused("seed", seed=1 << 64)
    refused("seed", seed=-1)
    refused("grads has dtype", grads=g.to(torch.bfloat16))
    refused("grads", grads=g[:, :64])
    refused("params", params=x.params[:64])
    refused("model", model=torch.zeros(x.N, device=DEV))
    refused("decay", decay=torch.zeros(2, device=DEV))
    refused("decay", decay=torch.zeros(1))
    refused("grad_scale", grad_scale=torch.zeros(2, device=DEV))
    refused("m_scale", state={**x.state, "m_scale": x.state["m_scale"][:1]})
    refused("status 2", model=torch.zeros(x.N + 8, dtype=torch.bfloat16, device=DEV)[1: x.N + 1])
    f = x.opt.adamw_state("f32")
    refused("no scales", state={**f, "m_scale": x.state["m_scale"]})
    with pytest.raises(OneBitError, match="are their values"):
        x.opt.adamw_load(f, f["m"], f["v"])
    with pytest.raises(OneBitError, match="dtype"):
        x.opt.adamw_load(x.state, torch.zeros(x.N, device=DEV), torch.zeros(x.N, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(OneBitError, match="unknown moments"):
        x.opt.adamw_state("4bit")


def test_steps_of_other_integer_types():
    """A step counted by numpy or torch is the same step; one past 64 bits is refused, not taken modulo 2^64."""
    want = List([100], 1, "f32", "8bit", seed=2)
    g = want.new_grads()
    want.step(g, 3, seed=9)
    real = want.real.to(DEV)
    for kind in (np.int64, np.int32, torch.tensor):
        x = List([100], 1, "f32", "8bit", seed=2)
        x.step(g, kind(3), seed=9)
        assert torch.equal(x.params[real], want.params[real])
        for k in ("m", "m_scale", "v", "v_scale"):
            assert torch.equal(x.state[k], want.state[k])
    x = List([100], 1, "f32", "8bit", seed=2)
    before = x.params.clone()
    for step in ((1 << 64) + 3, 1 << 63, -(1 << 63) - 1):
        with pytest.raises(OneBitError, match="64-bit"):
            x.step(g, step)
    with pytest.raises(TypeError):
        x.step(g, 1.5)
    assert torch.equal(x.params[real], before[real]) and int(x.state["m_scale"].count_nonzero()) == 0
