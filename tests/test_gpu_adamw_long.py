"""8-bit AdamW steps of more than 152 x 2 x 4 x 128 x 128 elements, which go in chunks of 128 blocks with the next blocks'
fetch under way: every element, code and scale against binary64, on the device."""
import math

import pytest

import blocks_util as bu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
SIZES = [21_000_003, 10_007]      # the last chunk of the first is 93 blocks and some, the pipelined loop's passes take 32
U = bu.U


@pytest.fixture(scope="module")
def ts():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g

    g.build()
    import top_sampling_gb300 as ts_mod

    return ts_mod


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.empty_cache()


def _wide(c, by):
    low = c * (by & 0xFFFF)
    high = c * (by >> 16) + (low >> 16)
    return high >> 16, ((high & 0xFFFF) << 16) | (low & 0xFFFF)


def _words(n, high, step, index, seed, dev):
    """Philox4x32-10's word of every element, in 64-bit whole numbers."""
    low = 0xFFFFFFFF
    i = torch.arange(-(-n // 4), device=dev)
    c0, c1, c2, c3 = i & low, torch.full_like(i, high), torch.full_like(i, step & low), torch.full_like(i, index)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        p0, p1 = _wide(c0, 0xD2511F53), _wide(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = p1[0] ^ c1 ^ k0, p1[1], p0[0] ^ c3 ^ k1, p0[1]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((c0, c1, c2, c3), dim=1).view(-1)[:n]


def _block_max(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % 128)).view(-1, 128).amax(dim=1)


def _each(s, n):
    return s.repeat_interleave(128)[:n]


def _stochastic(x, tx, scale, h, least):
    """blocks_util.stochastic on the device."""
    y = x / scale
    step = torch.exp2((torch.frexp(y)[1].clamp(min=-6 + 1) - 1 - 3).double())
    t = y / step + (h.double() + 0.5) / 65536
    near = (t - t.round()).abs() <= (tx / scale) / step + 8 * U * t
    q = (t.floor() * step).clamp(max=448.0)
    if least:
        q = torch.where(x > 0, q.clamp(min=2.0 ** -9), q)
    return q, torch.where(near, step, 0.0)


def test_the_words_are_the_oracles():
    dev = torch.device("cuda:0")
    for high, step, index, seed in ((0, 1, 0, 0), (1 << 31, (1 << 33) + 5, 7, (3 << 32) + 9)):
        assert bu.words(1001, high, step, index, seed).tolist() == _words(1001, high, step, index, seed, dev).tolist()


@pytest.mark.parametrize("pdt,gdt,masters", [(F32, BF16, False), (F32, F32, False), (BF16, BF16, False), (BF16, F32, True)])
def test_long_step(ts, pdt, gdt, masters):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(7)
    lr, step, b1, b2, eps, wd, seed = 1e-3, 5, 0.9, 0.99, 1e-8, 0.1, (7 << 32) + 3
    params, grads, m, v, ms, vs = [], [], [], [], [], []
    for n in SIZES:
        size = torch.exp2(torch.randn(n, generator=gen, device=dev) * 2 - 8)
        params.append((torch.randn(n, generator=gen, device=dev) * 0.1).to(pdt))
        grads.append((torch.randn(n, generator=gen, device=dev) * size).to(gdt))
        for x, codes, scales in ((torch.randn(n, generator=gen, device=dev) * size * 0.3, m, ms),
                                 ((torch.rand(n, generator=gen, device=dev) + 0.5) * size, v, vs)):
            s = (_block_max(x.abs()) / 448).clamp(min=2.0 ** -126)
            scales.append(s)
            codes.append((x / _each(s, n)).clamp(-448, 448).to(F8))
    state = ts.vsamp_adamw_state(params, bits=8, masters=masters or None, m=m, v=v, m_scale=ms, v_scale=vs)
    before = [[t.double() for t in group] for group in (params, m, v, ms, vs)]
    ts.vsamp_adamw(state, grads, lr=lr, step=step, beta1=b1, beta2=b2, eps=eps, weight_decay=wd, seed=seed)
    c1, c2 = 1 / (1 - b1 ** step), 1 / math.sqrt(1 - b2 ** step)
    for k, n in enumerate(SIZES):
        p, m0, v0, s0, r0 = (group[k] for group in before)
        g = grads[k].double()
        m0, v0 = m0 * _each(s0, n), (v0 * _each(r0, n)).square()
        # blocks_util.adamw on the device
        tm = U * (3 * (b1 * m0).abs() + 5 * ((1 - b1) * g).abs())
        m1, v1 = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
        root = v1.sqrt()
        den = root * c2 + eps
        change = m1 * c1 / den
        new = p - lr * (wd * p + change)
        tp = U * new.abs() + lr * (24 * U * change.abs() + tm * c1 / den + 4 * U * wd * p.abs())
        got = params[k].double()
        if masters:
            assert ((state.masters[k].double() - new).abs() <= tp).all()
            assert torch.equal(params[k], state.masters[k].bfloat16())
        elif pdt is F32:
            assert ((got - new).abs() <= tp).all()
        else:
            h = (_words(n, 1 << 31, step, k, seed, dev) & 0xFFFF).double()
            ulp = torch.exp2((torch.frexp(new)[1] - 8).double())
            t = new.abs() / ulp + h / 65536
            near = (t - t.round()).abs() <= tp / ulp
            want = t.trunc() * ulp * torch.sign(new)
            assert ((got - want).abs() <= torch.where(near, ulp, 0.0)).all()
        w = _words(n, 0, step, k, seed, dev)
        for x, tx, codes, scales, h, least in ((m1, tm, m[k], ms[k], w >> 16, False),
                                               (root, 6 * U * root, v[k], vs[k], w & 0xFFFF, True)):
            s = (_block_max(x.abs()) / 448).clamp(min=2.0 ** -126)
            ts_ = _block_max(tx) / 448 + 2 * U * s
            assert ((scales.double() - s).abs() <= ts_).all()
            q, off = _stochastic(x.abs(), tx + x.abs() * _each(ts_ / s, n), _each(s, n), h, least)
            c = codes.double()
            assert ((c.abs() - q).abs() <= off).all()
            assert ((c == 0) | (torch.sign(c) == torch.sign(x))).all()
            assert not least or torch.equal(c > 0, x > 0)
            # not by the bounds alone: few elements lie where a last bit decides
            assert (c.abs() != q).double().mean() < 1e-3


def test_long_step_repeats(ts):
    """The same step over the tensor whole, which is one launch in long chunks, and over its first part, in short ones."""
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(9)
    n, part = SIZES[0], 128 * 10_000
    grad = (torch.randn(n, generator=gen, device=dev) * 0.01).bfloat16()
    start = torch.randn(n, generator=gen, device=dev)
    states = [ts.vsamp_adamw_state([start[:k].clone()], bits=8) for k in (n, n, part)]
    for s in states:
        for step in (1, 2):
            ts.vsamp_adamw(s, [grad[:s.sizes[0]]], lr=1e-3, step=step, beta2=0.99, seed=4)
    one, two, short = states
    for x, y, z in ((s.params[0], t.params[0], u.params[0]) if i == 0 else
                    (s.m[0].view(torch.uint8), t.m[0].view(torch.uint8), u.m[0].view(torch.uint8)) if i == 1 else
                    (s.v[0].view(torch.uint8), t.v[0].view(torch.uint8), u.v[0].view(torch.uint8)) if i == 2 else
                    (s.m_scale[0], t.m_scale[0], u.m_scale[0]) if i == 3 else (s.v_scale[0], t.v_scale[0], u.v_scale[0])
                    for i, (s, t, u) in enumerate([(one, two, short)] * 5)):
        assert torch.equal(x, y) and torch.equal(x[:len(z)], z)
