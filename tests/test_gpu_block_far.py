"""Elements beyond 2^31: the last rows of results, codes and moments whose offsets do not fit 32 bits."""
import numpy as np
import pytest

import blocks_util as bu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("N", [131072, 131073])
def test_product(ts, N):
    M, K = 16400, 128
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn((M, K), generator=gen, device=dev)
    w = torch.randn((N, K), generator=gen, device=dev)
    a, _ = ts.vsamp_block_quantize(x)
    b, _ = ts.vsamp_block_quantize(w, tile=True)
    y = ts.vsamp_block_matmul(a, b)
    assert y.numel() > 2 ** 31
    rows = torch.tensor([0, 16383, 16384, M - 1], device=dev)
    va, vb = a.dequantize().double()[rows], b.dequantize().double()
    want, size = va @ vb.t(), va.abs() @ vb.abs().t()
    tol = bu.product_tol(size, K) + 2.0 ** -8 * want.abs()
    assert ((y[rows].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("tile", [False, True])
def test_quantise(ts, tile):
    R, C = 53000, 41000
    dev = torch.device("cuda:0")
    x = torch.zeros((R, C), dtype=torch.bfloat16, device=dev)
    gen = torch.Generator(device=dev).manual_seed(2)
    x[-200:] = torch.randn((200, C), generator=gen, device=dev).to(torch.bfloat16)
    assert x.numel() > 2 ** 31
    a, b = ts.vsamp_block_quantize(x, tile=tile, transposed=True)
    # whole blocks from the end
    r0, c0 = (R - 200) // 128 * 128, (C - 500) // 128 * 128
    part = x[r0:, c0:].float().cpu().numpy()
    y, s = bu.quantise(part, tile)
    np.testing.assert_array_equal(a.codes[r0:, c0:].float().cpu().numpy(), y)
    got = a.scales[r0 // 128:, c0 // 128:] if tile else a.scales[c0 // 128:, r0:]
    np.testing.assert_array_equal(got.cpu().numpy(), s)
    y, s = bu.quantise(part.T, tile)
    np.testing.assert_array_equal(b.codes[c0:, r0:].float().cpu().numpy(), y)
    got = b.scales[c0 // 128:, r0 // 128:] if tile else b.scales[r0 // 128:, c0:]
    np.testing.assert_array_equal(got.cpu().numpy(), s)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(ts, bits):
    n = 2 ** 31 + 1000
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(3)
    p = torch.zeros(n, device=dev)
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    tail = slice(2 ** 31 - 1024, n)
    p[tail] = torch.randn(n - tail.start, generator=gen, device=dev)
    g[tail] = torch.randn(n - tail.start, generator=gen, device=dev).to(torch.bfloat16)
    before = p[tail].double()
    state = ts.vsamp_adamw_state([p], bits=bits)
    ts.vsamp_adamw(state, [g], lr=1e-2, step=1, beta2=0.99, seed=5)
    want = before - 1e-2 * g[tail].double() / (g[tail].double().abs() + 1e-8)
    assert ((p[tail].double() - want).abs() <= 64 * bu.U * (want.abs() + 1e-2)).all()
    assert not p[:tail.start].any()
    if bits == 32:
        assert ((state.m[0][tail].double() - 0.1 * g[tail].double()).abs() <= 8 * bu.U * g[tail].double().abs()).all()
    else:
        x = 0.1 * g[tail].double().cpu().numpy()
        s = np.repeat(np.maximum(np.abs(bu.per_block(x)).max(axis=1) / 448, 2.0 ** -126), 128)[:x.size]
        i = np.arange(tail.start, n)
        w = bu.philox4x32_10_np(i >> 2, 0, 1, 0, 5, 0)
        h = np.choose(i & 3, [v.astype(np.int64) for v in w]) >> 16
        q, off = bu.stochastic(np.abs(x), 8 * bu.U * np.abs(x) + 4 * bu.U * s * 448, s, h, False)
        assert np.all(np.abs(np.abs(state.m[0][tail].double().cpu().numpy()) - q) <= off)
