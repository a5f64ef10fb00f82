"""The scales of 8-bit moments as the header defines them, bit for bit, and the codes that follow from them."""
import numpy as np
import pytest

import blocks_util as bu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.fixture(scope="module")
def ts():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g

    g.build()
    import top_sampling_gb300 as ts_mod

    return ts_mod


def _each(s, n):
    return s.repeat_interleave(128)[:n]


@pytest.mark.parametrize("n", [(1 << 23) + 77, 20_000_128])   # short chunks; long ones
def test_scales_and_codes(ts, n):
    """A first step, whose moments are products: scales are the largest magnitudes times 1 / 448 in fp32 (for about half of them
    another number than the quotient), codes follow from the scales' reciprocals."""
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(5)
    g = torch.randn(n, generator=gen, device=dev) * torch.exp2(torch.randn(n, generator=gen, device=dev) * 3 - 10)
    p = torch.zeros(n, device=dev)
    state = ts.vsamp_adamw_state([p], bits=8)
    ts.vsamp_adamw(state, [g], lr=1e-3, step=1, beta1=0.9, beta2=0.99, seed=11)
    m, v = g * (1 - 0.9), (1 - 0.99) * g * g
    part = 1 << 20                                 # of the codes, at both ends
    w = bu.words(n, 0, 1, 0, 11)
    for x, codes, scales, h, least in ((m, state.m[0], state.m_scale[0], w >> 16, 0.0),
                                       (torch.sqrt(v), state.v[0], state.v_scale[0], w & 0xFFFF, 2.0 ** -9)):
        amax = torch.nn.functional.pad(x.abs(), (0, -n % 128)).view(-1, 128).amax(dim=1).cpu().numpy()
        want = np.maximum(amax * (np.float32(1) / np.float32(448)), np.float32(2.0 ** -126))
        assert want.dtype == np.float32 and np.array_equal(scales.cpu().numpy(), want)
        assert 0.2 < (want != np.maximum(amax / np.float32(448), np.float32(2.0 ** -126))).mean() < 0.8
        y = (x * _each(torch.reciprocal(scales), n)).abs()
        for at in (slice(0, part), slice(n - part, n)):
            u = bu.f64(y[at])
            step = np.ldexp(1.0, np.maximum(np.frexp(u)[1] - 1, -6) - 3)
            q = np.minimum(np.floor(u / step + (h[at] + 0.5) / 65536) * step, 448.0)
            q = np.where(u > 0, np.maximum(q, least), q)
            assert np.array_equal(np.abs(bu.f64(codes[at].float())), q)
