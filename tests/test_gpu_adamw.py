"""The AdamW step on the GPU against binary64: types, states of 32 and 8 bits, odd sizes and addresses, many tensors,
device scalars, captured steps."""
import numpy as np
import pytest

import blocks_util as bu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ts():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g

    g.build()
    import top_sampling_gb300 as ts_mod

    return ts_mod


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


class Model:
    """Tensors of the given sizes with moments as some steps leave them; `at` shifts them from the 16-byte boundaries."""

    def __init__(self, ts, sizes, pdt, gdt, bits, masters, dev, at=0, seed=0):
        rng = np.random.default_rng(seed)
        self.bits = bits

        def place(x, dt):
            room = torch.empty(x.size + at + 8, dtype=dt, device=dev)
            t = room[at:at + x.size]
            t.copy_(torch.from_numpy(x.astype(np.float32)).to(dev).to(dt))
            return t

        self.params, self.masters, self.grads, self.m, self.v, self.ms, self.vs = [], [], [], [], [], [], []
        for n in sizes:
            size = np.exp2(rng.normal(size=n) * 2 - 8)
            w = rng.normal(size=n) * 0.1
            self.params.append(place(w, pdt))
            self.masters.append(place(w, F32) if masters else None)
            self.grads.append(place(rng.normal(size=n) * size, gdt))
            m, r = rng.normal(size=n) * size * 0.3, rng.uniform(0.5, 1.5, size=n) * size
            if bits == 32:
                self.m.append(place(m, F32))
                self.v.append(place(r * r, F32))
                self.ms.append(None)
                self.vs.append(None)
            else:
                for x, codes, scales in ((m, self.m, self.ms), (r, self.v, self.vs)):
                    b = bu.per_block(x)
                    s = bu.scale_of(np.abs(b).max(axis=1))
                    codes.append(place(bu.e4m3(b / s[:, None]).reshape(-1)[:n], F8))
                    scales.append(place(s, F32))
        more = dict(m_scale=self.ms, v_scale=self.vs) if bits == 8 else {}
        self.state = ts.vsamp_adamw_state(self.params, bits=bits, masters=self.masters if masters else None, m=self.m, v=self.v,
                                          **more)

    def arrays(self):
        return [[None if t is None else bu.f64(t) for t in g] for g in
                (self.params, self.masters, self.grads, self.m, self.v, self.ms, self.vs)]


def _check(model, before, lr, step, b1, b2, eps, wd, gs, seed, skipped=()):
    after = model.arrays()
    masters = model.masters[0] is not None
    for k, n in enumerate(t.numel() for t in model.params):
        p, w, g, m, v, ms, vs = (x[k] for x in before)
        if k in skipped:
            for x, y in zip(before, after):
                assert x[k] is None or np.array_equal(x[k], y[k], equal_nan=True)
            continue
        if model.bits == 8:
            m = m * np.repeat(ms, 128)[:n]
            v = (v * np.repeat(vs, 128)[:n]) ** 2
        (p, m, v), (tp, tm, tv) = bu.adamw(w if masters else p, g * gs, m, v, lr, step, b1, b2, eps, wd)
        if masters:
            assert np.all(np.abs(after[1][k] - p) <= tp)
            assert torch.equal(model.params[k], model.masters[k].bfloat16())
        elif model.params[k].dtype is F32:
            assert np.all(np.abs(after[0][k] - p) <= tp)
        else:
            h = bu.words(n, 1 << 31, step, k, seed) & 0xFFFF
            ulp = np.ldexp(1.0, np.frexp(p)[1] - 8)
            t = np.abs(p) / ulp + h / 65536
            near = np.abs(t - np.rint(t)) <= tp / ulp
            want = np.trunc(t) * ulp * np.sign(p)
            assert np.all(np.abs(after[0][k] - want) <= np.where(near, ulp, 0.0))
        if model.bits == 32:
            assert np.all(np.abs(after[3][k] - m) <= tm) and np.all(np.abs(after[4][k] - v) <= tv)
            continue
        root = np.sqrt(v)
        h = bu.words(n, 0, step, k, seed)
        for x, tx, codes, scales, bits, least in ((m, tm, after[3][k], after[5][k], h >> 16, False),
                                                  (root, (4 + 2) * bu.U * root, after[4][k], after[6][k], h & 0xFFFF, True)):
            s = np.maximum(np.abs(bu.per_block(x)).max(axis=1) / 448, 2.0 ** -126)
            ts_ = bu.per_block(tx).max(axis=1) / 448 + 2 * bu.U * s
            assert np.all(np.abs(scales - s) <= ts_)
            each, rel = np.repeat(s, 128)[:n], np.repeat(ts_ / s, 128)[:n]
            q, off = bu.stochastic(np.abs(x), tx + np.abs(x) * rel, each, bits, least)
            assert np.all(np.abs(np.abs(codes) - q) <= off)
            assert np.all((codes == 0) | (np.sign(codes) == np.sign(x)))
            assert not least or np.all((codes > 0) == (x > 0))


FORMS = [(F32, F32, 32, False), (F32, BF16, 32, False), (BF16, BF16, 32, True), (BF16, F32, 32, False),
         (F32, F32, 8, False), (F32, BF16, 8, False), (BF16, BF16, 8, True), (BF16, BF16, 8, False)]
SIZES = [1, 2, 3, 4, 5, 127, 128, 129, 255, 1000, 4095, 4096, 4097, 10007]


@pytest.mark.parametrize("pdt,gdt,bits,masters", FORMS)
@pytest.mark.parametrize("at", [0, 1, 2, 4])
def test_step(ts, dev, pdt, gdt, bits, masters, at):
    model = Model(ts, SIZES, pdt, gdt, bits, masters, dev, at=at, seed=at)
    for step in (1, 2, 1000):
        before = model.arrays()
        ts.vsamp_adamw(model.state, model.grads, lr=1e-3, step=step, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1,
                       seed=(5 << 32) + step)
        _check(model, before, 1e-3, step, 0.9, 0.99, 1e-8, 0.1, 1.0, (5 << 32) + step)


@pytest.mark.parametrize("bits", [32, 8])
def test_least_second_moments(ts, dev, bits):
    """Second moments on both sides of 2^-126 and no eps: a first step of lr 1 moves every parameter by 1. Errors are those
    of the form's change, and half of the last bit of a second moment, which counts half in its root."""
    rng = np.random.default_rng(3)
    n = 1003
    g = (rng.choice([-1.0, 1.0], size=n) * np.exp2(rng.uniform(-61.5, -58, size=n))).astype(np.float32)
    p = torch.zeros(n, device=dev)
    state = ts.vsamp_adamw_state([p], bits=bits)
    ts.vsamp_adamw(state, [torch.from_numpy(g).to(dev)], lr=1.0, step=1, beta1=0.9, beta2=0.99, eps=0.0)
    tol = 24 * bu.U + 2.0 ** -149 / (0.01 * g.astype(np.float64) ** 2)
    assert np.all(np.abs(bu.f64(p) + np.sign(g)) <= tol)
    assert (state.v[0].float() > 0).all()


def test_codes_bit_for_bit(ts, dev):
    """Codes are those of fp32 operations rounded one by one: the moments, the root, the scale's reciprocal, their product (the
    sum with the random bits and its floor are exact in binary64). Tensors long enough for every way through the kernel."""
    for n in (1 << 20, 4097):
        model = Model(ts, [n], F32, BF16, 8, False, dev, seed=n)
        m = model.m[0].float() * model.ms[0].repeat_interleave(128)[:n]
        g = model.grads[0].float()
        m = m * 0.9 + g * (1 - 0.9)
        v = (model.v[0].float() * model.vs[0].repeat_interleave(128)[:n]).square() * 0.99 + (1 - 0.99) * g * g
        ts.vsamp_adamw(model.state, model.grads, lr=1e-3, step=7, beta1=0.9, beta2=0.99, seed=11)
        w = bu.words(n, 0, 7, 0, 11)
        for x, codes, scales, h, least in ((m, model.m, model.ms, w >> 16, 0.0),
                                           (torch.sqrt(v), model.v, model.vs, w & 0xFFFF, 2.0 ** -9)):
            y = bu.f64((x * torch.reciprocal(scales[0]).repeat_interleave(128)[:n]).abs())
            step = np.ldexp(1.0, np.maximum(np.frexp(y)[1] - 1, -6) - 3)
            want = np.minimum(np.floor(y / step + (h + 0.5) / 65536) * step, 448.0)
            want = np.where(y > 0, np.maximum(want, least), want)
            assert np.array_equal(np.abs(bu.f64(codes[0].float())), want)


@pytest.mark.parametrize("bits", [32, 8])
def test_least_eps(ts, dev, bits):
    """Nothing moves without a gradient, with the least eps there is."""
    p = torch.ones(300, device=dev)
    state = ts.vsamp_adamw_state([p], bits=bits)
    ts.vsamp_adamw(state, [torch.zeros(300, device=dev)], lr=1.0, step=1, eps=2.0 ** -126)
    assert (p == 1.0).all()


def test_parameters_count_as_changed(ts, dev):
    """A backward pass through parameters that a step has changed since is refused; without a gradient they are not."""
    a, b = (torch.nn.Parameter(torch.ones(8, device=dev)) for _ in range(2))
    state = ts.vsamp_adamw_state([a, b])
    x = torch.ones(8, device=dev, requires_grad=True)
    ya, yb = (x * a).sum(), (x * b).sum()
    ts.vsamp_adamw(state, [torch.ones(8, device=dev), None], lr=0.1, step=1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        ya.backward()
    yb.backward()
    with torch.inference_mode():
        ts.vsamp_adamw(state, [torch.ones(8, device=dev)] * 2, lr=0.1, step=2)
        own = ts.vsamp_adamw_state([torch.ones(8, device=dev)])
        ts.vsamp_adamw(own, [torch.ones(8, device=dev)], lr=0.1, step=1)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(ts, dev, bits):
    """More tensors than one launch takes, empty ones and ones without a gradient among them."""
    rng = np.random.default_rng(1)
    sizes = [int(n) for n in rng.integers(0, 700, size=1000)]
    sizes[::50] = [0] * 20
    model = Model(ts, sizes, F32, F32, bits, False, dev, seed=4)
    before = model.arrays()
    skipped = set(range(7, 1000, 13))
    grads = [None if i in skipped else g for i, g in enumerate(model.grads)]
    scale = torch.tensor([0.5], device=dev)
    ts.vsamp_adamw(model.state, grads, lr=2e-3, step=7, grad_scale=scale, seed=3)
    _check(model, before, 2e-3, 7, 0.9, 0.999, 1e-8, 0.0, 0.5, 3, skipped)


def test_mixed_types(ts, dev):
    """Parameters and gradients of both types in one state; random numbers go by a tensor's place in it."""
    n = 3000
    gen = torch.Generator(device=dev).manual_seed(1)
    value = [torch.randn(n, generator=gen, device=dev) * 0.1 for _ in range(4)]
    grads = [torch.randn(n, generator=gen, device=dev) * 0.01 for _ in range(4)]
    grads[1], grads[3] = grads[1].bfloat16(), grads[3].bfloat16()
    params = [value[0].clone(), value[1].clone(), value[2].bfloat16(), value[3].bfloat16()]
    masters = [None, None, params[2].float(), None]
    state = ts.vsamp_adamw_state(params, bits=8, masters=masters)
    ts.vsamp_adamw(state, grads, lr=1e-2, step=1, beta2=0.99)
    for i in range(4):
        start = (value[i].bfloat16() if i >= 2 else value[i]).double()
        g = grads[i].double()
        new = start - 1e-2 * torch.sign(g) * (g.abs() / (g.abs() + 1e-8))     # the first step
        if i == 3:
            assert ((params[3].double() - new).abs() <= 2.0 ** -7 * new.abs() + 1e-6).all()
            ulp = torch.exp2((torch.frexp(new)[1] - 8).double())
            h = torch.from_numpy(bu.words(n, 1 << 31, 1, 3, 0) & 0xFFFF).to(dev)
            want = torch.trunc(new.abs() / ulp + h / 65536) * ulp * torch.sign(new)
            assert (params[3].double() != want).float().mean() < 0.01         # only where fp32 rounding decides
        else:
            got = (masters[2] if i == 2 else params[i]).double()
            assert ((got - new).abs() <= 64 * bu.U * (new.abs() + 1e-2)).all()


def test_device_scalars_and_graph(ts, dev):
    """A captured step that counts itself, with a learning rate and a gradient scale on the device, against host steps."""
    for form in ((F32, BF16, 8, False), (F32, F32, 32, False), (BF16, BF16, 32, False)):
        one, two = (Model(ts, [1000, 129], *form, dev, seed=2) for _ in range(2))
        lr = torch.zeros(1, device=dev)
        step = torch.zeros(1, dtype=torch.int64, device=dev)
        scale = torch.ones(1, device=dev)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step += 1
            ts.vsamp_adamw(one.state, one.grads, lr=lr, step=step, grad_scale=scale, weight_decay=0.01, seed=9)
        for k in range(1, 4):
            lr.fill_(1e-3 * k)
            scale.fill_(0.5 * k)
            before = one.arrays()
            graph.replay()
            _check(one, before, float(lr), k, 0.9, 0.999, 1e-8, 0.01, 0.5 * k, 9)
        # the host's numbers give the same up to the corrections' last bits
        for k in range(1, 4):
            lr.fill_(1e-3 * k)
            scale.fill_(0.5 * k)
            ts.vsamp_adamw(two.state, two.grads, lr=float(lr), step=k, grad_scale=scale, weight_decay=0.01, seed=9)
        for x, y in zip(one.params, two.params):
            assert ((x.double() - y.double()).abs() <= 2 * 2.0 ** -7 * x.double().abs() + 1e-4).all()
        # a step below 1 changes nothing
        step.fill_(-1)
        before = one.arrays()
        graph.replay()
        assert all(a is None or np.array_equal(a, b) for x, y in zip(before, one.arrays()) for a, b in zip(x, y))


def test_repeats(ts, dev):
    """The same call gives the same bits; another seed other ones."""
    outs = []
    for seed in (1, 1, 2):
        model = Model(ts, [5000], BF16, BF16, 8, False, dev, seed=6)
        ts.vsamp_adamw(model.state, model.grads, lr=1e-4, step=5, seed=seed)
        outs.append((model.params[0].clone(), model.m[0].view(torch.uint8).clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert not torch.equal(outs[0][0], outs[2][0]) and not torch.equal(outs[0][1], outs[2][1])


def test_random_rounding_has_no_bias(ts, dev):
    """Over many elements the mean of what is rounded at random is the mean before: 2^20 elements whose rounding errors
    have at most half a step's standard deviation leave a mean within six standard errors."""
    n = 1 << 20
    p = torch.full((n,), 1.0, device=dev).bfloat16()
    g = torch.full((n,), 0.45, device=dev)
    g[::128] = 1.0                                  # the largest of a block sets its scale
    state = ts.vsamp_adamw_state([p], bits=8)
    ts.vsamp_adamw(state, [g], lr=1e-3, step=1, beta1=0.7, beta2=0.99, seed=11)
    small = torch.ones(n, dtype=torch.bool, device=dev)
    small[::128] = False
    for codes, scales, want, least_step in ((state.m[0], state.m_scale[0], 0.3 * 0.45, 16.0),
                                            (state.v[0], state.v_scale[0], 0.1 * 0.45, 16.0)):
        got = (codes.double() * scales.double().repeat_interleave(128))[small]
        step = least_step * float(scales[0])
        assert abs(float(got.mean()) - want) <= 6 * 0.5 * step / float(small.sum()) ** 0.5 + 8 * bu.U * want
    # the parameter goes from 1 to 1 - 0.001: bf16 below 1 has steps of 2^-8
    assert abs(float(p.double().mean()) - (1 - 1e-3)) <= 6 * 0.5 * 2.0 ** -8 / n ** 0.5 + 4e-6
    assert len(p.unique()) == 2


def test_special_gradients(ts, dev):
    """Zeros stay zeros; NaN and infinities reach their own element (of 8-bit moments: their block)."""
    for bits in (32, 8):
        p = torch.ones(1024, device=dev)
        g = torch.zeros(1024, device=dev)
        g[130], g[700], g[1023] = float("nan"), float("inf"), 1e-30
        state = ts.vsamp_adamw_state([p], bits=bits)
        ts.vsamp_adamw(state, [g], lr=1e-2, step=1)
        bad = torch.zeros(1024, dtype=torch.bool, device=dev)
        bad[130] = bad[700] = True
        assert torch.equal(torch.isnan(p), bad)
        assert (p[~bad][:-1] == 1.0).all()
        if bits == 8:
            for s in (state.m_scale[0], state.v_scale[0]):
                assert torch.equal(torch.nonzero(torch.isnan(s))[:, 0].cpu(), torch.tensor([1, 5]))
            assert not state.m[0].float()[:1023].any() and not state.v[0].float()[:1023].any()


def test_betas_at_their_ends(ts, dev):
    model = Model(ts, [500], F32, F32, 32, False, dev, seed=8)
    before = model.arrays()
    ts.vsamp_adamw(model.state, model.grads, lr=1e-3, step=3, beta1=0.0, beta2=0.0, eps=1e-8)
    _check(model, before, 1e-3, 3, 0.0, 0.0, 1e-8, 0.0, 1.0, 0)
    step = torch.tensor([3], device=dev)
    before = model.arrays()
    ts.vsamp_adamw(model.state, model.grads, lr=1e-3, step=step, beta1=0.0, beta2=0.0, eps=1e-8)
    _check(model, before, 1e-3, 3, 0.0, 0.0, 1e-8, 0.0, 1.0, 0)


def test_other_stream(ts, dev):
    one, two = (Model(ts, [100000], F32, F32, 8, False, dev, seed=12) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ts.vsamp_adamw(one.state, one.grads, lr=1e-3, step=2)
    ts.vsamp_adamw(two.state, two.grads, lr=1e-3, step=2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(one.params[0], two.params[0]) and torch.equal(one.v[0].view(torch.uint8), two.v[0].view(torch.uint8))


def test_binding_refuses(ts, dev):
    p = torch.zeros(100, device=dev)
    with pytest.raises(ValueError):
        ts.vsamp_adamw_state([p, p])                                  # the same tensor twice
    with pytest.raises(ValueError):
        ts.vsamp_adamw_state([p[:60], p[50:]])
    with pytest.raises(TypeError):
        ts.vsamp_adamw_state([p.half()])
    with pytest.raises(ValueError):
        ts.vsamp_adamw_state([p[::2]])
    with pytest.raises(ValueError):
        ts.vsamp_adamw_state([p], masters=[p.clone()])                # masters of fp32 parameters
    with pytest.raises(ValueError):
        ts.vsamp_adamw_state([p], m=[torch.zeros(100, device=dev)])
    with pytest.raises(ValueError):
        ts.vsamp_adamw_state([p], m=[torch.zeros(99, device=dev)], v=[torch.zeros(100, device=dev)])
    with pytest.raises(ValueError):
        ts.vsamp_adamw_state([p], bits=8, m=[torch.zeros(100, dtype=F8, device=dev)], v=[torch.zeros(100, dtype=F8, device=dev)])
    state = ts.vsamp_adamw_state([p])
    g = torch.zeros(100, device=dev)
    with pytest.raises(ValueError):
        ts.vsamp_adamw(state, [g, g], lr=1e-3, step=1)
    with pytest.raises(ValueError):
        ts.vsamp_adamw(state, [g[:99]], lr=1e-3, step=1)
    with pytest.raises(ValueError):
        ts.vsamp_adamw(state, [g.half()], lr=1e-3, step=1)
    with pytest.raises(ValueError):
        ts.vsamp_adamw(state, [torch.zeros(200, device=dev)[::2]], lr=1e-3, step=1)
    with pytest.raises(ts.VsampError):
        ts.vsamp_adamw(state, [g], lr=1e-3, step=0)
    with pytest.raises(TypeError):
        ts.vsamp_adamw(state, [g], lr=1e-3, step=torch.ones(1, device=dev))
    with pytest.raises(TypeError):
        ts.vsamp_adamw(state, [g], lr=torch.ones(1, device=dev, dtype=torch.float64), step=1)
    with pytest.raises(ValueError):
        ts.vsamp_adamw(state, [g.cpu()], lr=1e-3, step=1)


def test_nothing_is_launched_before_all_is_checked(ts, dev):
    """A bad gradient of one group of tensors leaves the others as they are; a parameter that got other memory is seen."""
    a, b = torch.ones(100, device=dev), torch.ones(100, device=dev).bfloat16()
    state = ts.vsamp_adamw_state([a, b])
    with pytest.raises(ValueError):
        ts.vsamp_adamw(state, [torch.ones(100, device=dev), torch.ones(99, device=dev)], lr=1e-1, step=1)
    assert (a == 1).all() and not state.m[0].any()
    ts.vsamp_adamw(state, [torch.ones(100, device=dev), None], lr=1e-1, step=1)
    assert (a < 1).all() and (b == 1).all()
    a.data = torch.ones(100, device=dev)
    with pytest.raises(ValueError):
        ts.vsamp_adamw(state, [torch.ones(100, device=dev), None], lr=1e-1, step=2)
    assert (a == 1).all()
