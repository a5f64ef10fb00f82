"""8-bit blocks on the GPU: quantisation (equal to the definition, every step of which is one fp32 operation) and the
product against binary64."""
import numpy as np
import pytest

import blocks_util as bu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


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


def _values(R, C, dt, dev, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(R, C)) * np.exp2(rng.normal(size=(R, 1)) * 4) * np.exp2(rng.normal(size=(1, C)))
    return torch.from_numpy(x.astype(np.float32)).to(dev).to(dt)


def _check_quant(got, x, tile):
    y, s = bu.quantise(x.float().cpu().numpy(), tile)
    np.testing.assert_array_equal(got.scales.cpu().numpy(), s)
    np.testing.assert_array_equal(got.codes.view(torch.float8_e4m3fn).float().cpu().numpy(), y)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 128), (2, 129), (16, 2048), (127, 15), (128, 128), (130, 257), (300, 1001)])
def test_quantise(ts, dev, dt, tile, R, C):
    x = _values(R, C, dt, dev, R + C)
    a, b = ts.vsamp_block_quantize(x, tile=tile, transposed=True)
    _check_quant(a, x, tile)
    _check_quant(b, x.t(), tile)
    one, none = ts.vsamp_block_quantize(x, tile=tile)
    assert none is None and torch.equal(one.codes.view(torch.uint8), a.codes.view(torch.uint8))
    none, two = ts.vsamp_block_quantize(x, tile=tile, plain=False, transposed=True)
    assert none is None and torch.equal(two.codes.view(torch.uint8), b.codes.view(torch.uint8))
    if tile:
        assert torch.equal(a.scales.t(), b.scales)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("at,pad", [(1, 0), (3, 5), (8, 8), (0, 1)])
def test_quantise_strides(ts, dev, dt, at, pad):
    """Rows that begin anywhere; nothing outside the rows is read, nothing behind a row's last code is written."""
    R, C = 131, 200
    flat = torch.full((at + R * (C + pad) + 16,), float("nan"), dtype=dt, device=dev)
    x = flat[at:at + R * (C + pad)].view(R, C + pad)[:, :C]
    x.copy_(_values(R, C, dt, dev, 3))
    for tile in (False, True):
        codes = torch.full((R, 256), 0x55, dtype=torch.uint8, device=dev)
        codes_t = torch.full((C, 160), 0x55, dtype=torch.uint8, device=dev)
        if tile:
            scales, scales_t = torch.full((2, 5), 7.0, device=dev), torch.full((2, 4), 7.0, device=dev)
            to, to_t = (codes[:, :C], scales[:, :2]), (codes_t[:, :R], scales_t[:, :2])
        else:
            scales, scales_t = torch.full((2, 144), 7.0, device=dev), torch.full((2, 208), 7.0, device=dev)
            to, to_t = (codes[:, :C], scales[:, :R]), (codes_t[:, :R], scales_t[:, :C])
        a, b = ts.vsamp_block_quantize(x, tile=tile, transposed=True, out=ts.BlockTensor(*to, tile=tile),
                                       out_t=ts.BlockTensor(*to_t, tile=tile))
        _check_quant(a, x, tile)
        _check_quant(b, x.t(), tile)
        assert (codes[:, C:] == 0x55).all() and (codes_t[:, R:] == 0x55).all()
        assert (scales[:, to[1].shape[1]:] == 7.0).all() and (scales_t[:, to_t[1].shape[1]:] == 7.0).all()


def test_quantise_special_values(ts, dev):
    x = torch.zeros((140, 520), device=dev)
    x[0, 0], x[1, 130], x[2, 300] = float("nan"), float("inf"), -float("inf")
    x[3, 5] = torch.finfo(F32).max
    x[4, 6] = -torch.finfo(F32).max
    x[5, 128:256] = 2.0 ** -149                   # subnormal
    x[6, 128:256] = 2.0 ** -126
    x[7, 260] = 448.0 * 2.0 ** -126
    x[8, 519] = 1.0
    x[9, 400:420] = -0.0
    for tile in (False, True):
        a, b = ts.vsamp_block_quantize(x, tile=tile, transposed=True)
        _check_quant(a, x, tile)
        _check_quant(b, x.t(), tile)
    a, _ = ts.vsamp_block_quantize(x)
    bad = torch.isnan(a.scales)
    assert bad.sum() == 3 and bad[0, 0] and bad[1, 1] and bad[2, 2]


def test_quantise_error(ts, dev):
    """An element is off by at most half an e4m3 step of its own (2^-4) or of the block's smallest values (2^-10 scales),
    and three fp32 roundings."""
    x = _values(200, 700, F32, dev, 5)
    for tile in (False, True):
        a, _ = ts.vsamp_block_quantize(x, tile=tile)
        s = a.scales.repeat_interleave(128, 0)[:200] if tile else a.scales.t()
        s = s.repeat_interleave(128, 1)[:, :700].double()
        off = (a.dequantize().double() - x.double()).abs()
        assert (off <= torch.maximum(x.double().abs() * (2.0 ** -4 + 4 * bu.U), s * 2.0 ** -10 * (1 + 4 * bu.U))).all()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_quantise_ties(ts, dev, dt):
    """Elements half way between two codes go to the even one: x = max * midpoint / 448 exactly, for maxima whose quotient
    with 448 has no exact reciprocal."""
    mids = torch.arange(8, 15, device=dev).float() + 0.5                    # between the codes of a binade, in eighths
    scale = torch.exp2(torch.arange(-3, 3, device=dev).float())
    mid = (mids[:, None] * scale).reshape(-1)                              # 42 midpoints, among them 8.5 / 4 ..
    even = torch.round(mids)[:, None] * scale
    for top in (7.0, 1.0, 0.75, 1.25, 7 * 2.0 ** 20, 1.75 * 2.0 ** -30):
        x = torch.zeros((1, 128), dtype=torch.float64, device=dev)
        x[0, :42] = mid.double() * top / 448
        x[0, 100] = top
        if dt == BF16 or not torch.equal(x.float().double(), x):
            keep = x.to(dt).double() == x
            x = torch.where(keep, x, torch.zeros_like(x))
        a, _ = ts.vsamp_block_quantize(x.to(dt))
        got = a.codes.view(torch.float8_e4m3fn).float()[0, :42]
        exact = x[0, :42] != 0
        assert torch.equal(got[exact], even.reshape(-1)[exact]), top
        assert top not in (7.0, 7 * 2.0 ** 20, 1.75 * 2.0 ** -30) or exact.all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("exponent", [-110, -1, 126, 127])
def test_quantise_ties_at_the_ends(ts, dev, dt, exponent):
    """10.5 / 448 of any largest magnitude t is 1.5 t / 64, half way between the codes 10 and 11: it goes to the even one,
    whatever 448 / t rounds to, near the type's ends too."""
    t = torch.ldexp(torch.arange(128, 256, dtype=torch.float64), torch.tensor(exponent - 7.0, dtype=torch.float64))
    x = torch.zeros((128, 128), dtype=torch.float64)
    x[:, 0], x[:, 1], x[:, 2] = t, 1.5 * t / 64, -1.5 * t / 512
    x = x.to(dt).to(dev)
    exact = x[:, 1].double().cpu() == 1.5 * t / 64
    assert exact.sum() >= 40
    a, _ = ts.vsamp_block_quantize(x)
    _, b = ts.vsamp_block_quantize(x.t().contiguous(), plain=False, transposed=True)
    for q in (a, b):
        codes = q.codes.view(torch.float8_e4m3fn).float().cpu()
        assert (codes[:, 0] == 448).all() and (codes[exact, 1] == 10).all() and (codes[exact, 2] == -1.25).all()


def _operand(ts, rows, cols, tile, dev, seed):
    rng = np.random.default_rng(seed)
    t = ts.BlockTensor.empty(rows, cols, tile, dev)
    t.codes.copy_(torch.from_numpy(bu.e4m3(rng.normal(size=(rows, cols)) * 100)).to(dev).to(torch.float32).to(torch.float8_e4m3fn))
    t.scales.copy_(torch.from_numpy(np.exp2(rng.uniform(-14, -10, size=t.scales.shape)).astype(np.float32)).to(dev))
    return t


def _np(t):
    return t.codes.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64), bu.f64(t.scales)


def _check_product(got, a, b, base=None):
    (qa, sa), (qb, sb) = _np(a), _np(b)
    want, size = bu.product(qa, sa, qb, sb, b.tile, base)
    tol = bu.product_tol(size, a.cols) + bu.HALF[got.dtype] * np.abs(want)
    off = np.abs(bu.f64(got) - want)
    assert np.all(off <= tol), (float((off / np.maximum(tol, 1e-300)).max()), off.shape)


@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 128, 128), (3, 127, 16), (5, 300, 100), (8, 129, 129), (16, 1000, 384),
                                   (17, 256, 2048), (64, 257, 640), (65, 64, 257), (100, 513, 400), (127, 255, 130),
                                   (128, 256, 256), (129, 300, 1000), (255, 140, 100), (300, 1030, 513)])
def test_product(ts, dev, M, N, K, tile, out):
    a, b = _operand(ts, M, K, False, dev, M + K), _operand(ts, N, K, tile, dev, N + K + 1)
    _check_product(ts.vsamp_block_matmul(a, b, out_dtype=out), a, b)


@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("pad", [0, 1, 3, 8])
def test_product_into_rows(ts, dev, tile, out, pad):
    """Padded output rows; adding; what is between the rows stays."""
    M, N, K = 70, 333, 300
    a, b = _operand(ts, M, K, False, dev, 1), _operand(ts, N, K, tile, dev, 2)
    y = torch.full((M, N + pad), 7.0, dtype=out, device=dev)
    ts.vsamp_block_matmul(a, b, out=y[:, :N])
    _check_product(y[:, :N], a, b)
    assert (y[:, N:] == 7.0).all()
    base = torch.randn((M, N), device=dev).mul_(0.1).to(out)
    y[:, :N] = base
    ts.vsamp_block_matmul(a, b, out=y[:, :N], accumulate=True)
    _check_product(y[:, :N], a, b, bu.f64(base))
    assert (y[:, N:] == 7.0).all()


@pytest.mark.parametrize("M,N,K,tile", [(4, 40, 151936, True), (33, 500, 30001, True), (130, 260, 40000, False),
                                        (1, 40961, 512, True), (200, 20000, 256, True), (2100, 1300, 300, False),
                                        (40, 40960, 2048, True), (256, 20400, 2048, True), (300, 10001, 2050, False)])
def test_product_long_and_wide(ts, dev, M, N, K, tile):
    a, b = _operand(ts, M, K, False, dev, 5), _operand(ts, N, K, tile, dev, 6)
    y = ts.vsamp_block_matmul(a, b, out_dtype=F32)
    _check_product(y, a, b)
    assert torch.equal(ts.vsamp_block_matmul(a, b, out_dtype=F32), y)


@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N", [(20, 60), (150, 133)])
def test_product_added_in_parts(ts, dev, tile, out, M, N):
    """A long inner dimension, divided over CTAs, added to what is there; odd rows and whole ones."""
    K = 30000
    assert ts.load().vsamp_block_matmul_workspace_size(M, N, K) > 0
    a, b = _operand(ts, M, K, False, dev, 7), _operand(ts, N, K, tile, dev, 8)
    y = torch.full((M, N + 5), 7.0, dtype=out, device=dev)
    base = torch.randn((M, N), device=dev).to(out)
    y[:, :N] = base
    ts.vsamp_block_matmul(a, b, out=y[:, :N], accumulate=True)
    _check_product(y[:, :N], a, b, bu.f64(base))
    assert (y[:, N:] == 7.0).all()


@pytest.mark.parametrize("out", [F32, BF16])
def test_product_tiles_that_leave_differently(ts, dev, out):
    """A CTA whose first tile leaves as boxes and whose second one, at the rows' odd end, by elements."""
    M, N, K = 10, 152 * 256 + 130, 100
    a, b = _operand(ts, M, K, False, dev, 7), _operand(ts, N, K, True, dev, 8)
    y = torch.full((M, N + 6), 7.0, dtype=out, device=dev)
    first = None
    for _ in range(20):
        ts.vsamp_block_matmul(a, b, out=y[:, :N])
        if first is None:
            first = y.clone()
            _check_product(y[:, :N], a, b)
        assert torch.equal(y, first)
    assert (y[:, N:] == 7.0).all()


@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("M", [100, 300])
@pytest.mark.parametrize("N", [1, 63, 65, 257, 320, 385, 450, 512])
def test_product_narrow_last_tiles(ts, dev, tile, M, N):
    """Last tiles of one to four warps' columns, one CTA's and a pair's, into rows at odd and even strides, written and
    added to."""
    a, b = _operand(ts, M, 300, False, dev, N), _operand(ts, N, 300, tile, dev, N + 1)
    for out in (F32, BF16):
        for pad in (0, 1, 2):
            base = torch.randn((M, N + pad), dtype=torch.float64).to(out).to(dev)
            for add in (False, True):
                y = base.clone()
                ts.vsamp_block_matmul(a, b, out=y[:, :N], accumulate=add)
                _check_product(y[:, :N], a, b, bu.f64(base[:, :N]) if add else None)
                assert torch.equal(y[:, N:], base[:, N:])


@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("M,N", [(700, 600), (600, 700), (250, 1000), (1000, 250)])
def test_product_order_of_tiles(ts, dev, tile, M, N):
    """Several tiles that are divided, along rows and down columns of results."""
    a, b = _operand(ts, M, 20000, False, dev, M), _operand(ts, N, 20000, tile, dev, N)
    assert ts.load().vsamp_block_matmul_workspace_size(M, N, 20000) > 0
    _check_product(ts.vsamp_block_matmul(a, b, out_dtype=F32), a, b)


def test_product_padded_operands(ts, dev):
    """Operands inside larger arrays full of NaN codes and scales: only their own rows and columns count."""
    M, N, K = 50, 200, 270
    for tile in (True, False):
        a, b = _operand(ts, M, K, False, dev, 8), _operand(ts, N, K, tile, dev, 9)
        ref = ts.vsamp_block_matmul(a, b, out_dtype=F32)
        wide = []
        for t in (a, b):
            codes = torch.full((t.rows + 3, 320), 0x7F, dtype=torch.uint8, device=dev)
            codes[:t.rows, :K] = t.codes.view(torch.uint8)
            h, w = t.scales.shape
            scales = torch.full((h + 1, w + 12 - (0 if t.tile else w % 4)), float("nan"), device=dev)
            scales[:h, :w] = t.scales
            wide.append(ts.BlockTensor(codes[:t.rows, :K], scales[:h, :w], t.tile))
        assert torch.equal(ts.vsamp_block_matmul(*wide, out_dtype=F32), ref)


def test_product_of_blocks_that_are_not_finite(ts, dev):
    M, N, K = 140, 300, 300
    x, w = _values(M, K, F32, dev, 1), _values(N, K, F32, dev, 2)
    x[7, 200] = float("inf")
    w[130, 10] = float("nan")
    a, _ = ts.vsamp_block_quantize(x)
    for tile in (True, False):
        b, _ = ts.vsamp_block_quantize(w, tile=tile)
        y = ts.vsamp_block_matmul(a, b, out_dtype=F32)
        bad = torch.isnan(y)
        want = torch.zeros_like(bad)
        want[7] = True
        if tile:
            want[:, 128:256] = True
        else:
            want[:, 130] = True
        assert torch.equal(bad, want)
    # a NaN code reaches its own row alone
    a, b = _operand(ts, M, K, False, dev, 3), _operand(ts, N, K, True, dev, 4)
    ref = ts.vsamp_block_matmul(a, b, out_dtype=F32)
    a.codes.view(torch.uint8)[9, 299] = 0x7F
    y = ts.vsamp_block_matmul(a, b, out_dtype=F32)
    assert torch.isnan(y[9]).all()
    y[9] = ref[9]
    assert torch.equal(y, ref)


def test_extreme_scales(ts, dev):
    """Scales whose product leaves fp32's normal range on the way of no result that is in range itself."""
    a, b = _operand(ts, 5, 128, False, dev, 3), _operand(ts, 9, 128, True, dev, 4)
    a.scales.fill_(2.0 ** 100)
    b.scales.fill_(2.0 ** -100)
    _check_product(ts.vsamp_block_matmul(a, b, out_dtype=F32), a, b)
    a.scales.fill_(2.0 ** -60)
    b.scales.fill_(2.0 ** -60)
    _check_product(ts.vsamp_block_matmul(a, b, out_dtype=F32), a, b)


def test_rows_do_not_depend_on_others(ts, dev):
    b = _operand(ts, 700, 900, True, dev, 4)
    a = _operand(ts, 40, 900, False, dev, 3)
    y = ts.vsamp_block_matmul(a, b, out_dtype=F32)
    a2 = _operand(ts, 40, 900, False, dev, 13)
    a2.codes.view(torch.uint8)[11] = a.codes.view(torch.uint8)[11]
    a2.scales[:, 11] = a.scales[:, 11]
    assert torch.equal(ts.vsamp_block_matmul(a2, b, out_dtype=F32)[11], y[11])


def test_other_stream_and_graph(ts, dev):
    """Quantisation and product on another stream and captured, on sizes with and without a workspace."""
    for M, N, K in ((20, 5000, 512), (40, 300, 50000)):
        w, _ = ts.vsamp_block_quantize(_values(N, K, BF16, dev, 1), tile=True)
        x = _values(M, K, BF16, dev, 2)
        ref = ts.vsamp_block_matmul(ts.vsamp_block_quantize(x)[0], w)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = ts.vsamp_block_matmul(ts.vsamp_block_quantize(x, stream=side)[0], w, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(ref, other)
        graph = torch.cuda.CUDAGraph()
        xs = torch.zeros_like(x)
        with torch.cuda.graph(graph):
            y = ts.vsamp_block_matmul(ts.vsamp_block_quantize(xs)[0], w)
            y2 = ts.vsamp_block_matmul(ts.vsamp_block_quantize(xs)[0], w)
        for _ in range(2):
            xs.copy_(x)
            graph.replay()
            assert torch.equal(y, ref) and torch.equal(y2, ref)
            xs.zero_()
            graph.replay()
            assert not y.any()


def test_two_streams_at_once(ts, dev):
    """Calls that overlap use workspaces of their own."""
    M, N, K = 40, 600, 60000
    w, _ = ts.vsamp_block_quantize(_values(N, K, BF16, dev, 1), tile=True)
    xs = [ts.vsamp_block_quantize(_values(M, K, BF16, dev, 5 + i))[0] for i in range(2)]
    refs = [ts.vsamp_block_matmul(x, w) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(ts.vsamp_block_matmul(xs[i], w))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, refs[i]) for y in got[i])


def test_binding_refuses(ts, dev):
    a, b = _operand(ts, 8, 256, False, dev, 1), _operand(ts, 100, 256, True, dev, 2)
    with pytest.raises(ValueError):
        ts.vsamp_block_matmul(b, b)                                             # the first operand in 128 x 128 blocks
    with pytest.raises(ValueError):
        ts.vsamp_block_matmul(a, _operand(ts, 100, 255, True, dev, 2))
    with pytest.raises(ValueError):
        ts.vsamp_block_matmul(a, b, accumulate=True)
    with pytest.raises(ValueError):
        ts.vsamp_block_matmul(a, b, out=torch.zeros((8, 99), device=dev))
    with pytest.raises(TypeError):
        ts.vsamp_block_matmul(a, b, out=torch.zeros((8, 100), device=dev).half())
    codes = torch.zeros((8, 256), dtype=torch.uint8, device=dev)
    with pytest.raises(ValueError):
        ts.BlockTensor(codes[:, :250].contiguous(), torch.zeros((2, 8), device=dev))   # rows of 250 bytes
    with pytest.raises(ValueError):
        ts.BlockTensor(codes[:, 1:200], torch.zeros((2, 8), device=dev))
    with pytest.raises(ValueError):
        ts.BlockTensor(codes, torch.zeros((2, 9), device=dev))
    with pytest.raises(ValueError):
        ts.BlockTensor(codes, torch.zeros((2, 8), device=dev), tile=True)
    with pytest.raises(ValueError):
        ts.BlockTensor(codes[:5], torch.zeros((2, 5), device=dev))                     # rows of five scales
    with pytest.raises(ValueError):
        ts.vsamp_block_quantize(torch.zeros((8, 256), device=dev), plain=False)
    with pytest.raises(ValueError):
        ts.vsamp_block_quantize(torch.zeros((9, 256), device=dev), out=a)
    with pytest.raises(ValueError):
        ts.vsamp_block_quantize(torch.zeros((8, 256), device=dev), tile=True, out=a)
    with pytest.raises(ValueError):
        ts.vsamp_block_quantize(torch.zeros((256, 8), device=dev).t())
    with pytest.raises(TypeError):
        ts.vsamp_block_quantize(torch.zeros((8, 256), device=dev).half())


def test_outputs_that_share_memory(ts, dev):
    x = torch.randn(128, 128, device=dev)
    one, two = (ts.BlockTensor.empty(128, 128, False, dev) for _ in range(2))
    for other in (one, ts.BlockTensor(one.codes, two.scales), ts.BlockTensor(two.codes, one.scales)):
        with pytest.raises(ValueError, match="share memory"):
            ts.vsamp_block_quantize(x, transposed=True, out=one, out_t=other)
    ts.vsamp_block_quantize(x, transposed=True, out=one, out_t=two)
    _, want = ts.vsamp_block_quantize(x, transposed=True)
    assert torch.equal(two.codes.view(torch.uint8), want.codes.view(torch.uint8)) and torch.equal(two.scales, want.scales)
