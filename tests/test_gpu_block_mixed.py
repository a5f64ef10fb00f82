"""Products some of whose tiles are whole and some divided along the inner dimension: pairs of CTAs and single ones, several
rows and columns of tiles, both orders, both kinds of scales, written and added, against binary64 on the device."""
import pytest

import blocks_util as bu

torch = pytest.importorskip("torch")

F32, BF16 = torch.float32, torch.bfloat16
# rows, columns, inner: more tiles than CTAs, and a rest of them
SIZES = [(2100, 2401, 12000), (2401, 2100, 12000), (400, 11000, 6000), (11000, 400, 6000), (129, 20000, 5000),
         (100, 41000, 6000)]


def _room(M, N, K, size):
    """The workspace's bytes, and those of the least division of all tiles."""
    rows = 256 if M > 128 else 128
    tiles = -(-M // rows) * -(-N // 256)
    return size(M, N, K), tiles, tiles * 2 * min(M, rows) * 256 * 4


def test_sizes_are_divided_in_part():
    """On the CPU: the sizes below and the 2048 x 4096 x 151936 one have whole and divided tiles; long inner dimensions of few
    tiles are divided."""
    from top_sampling_gb300 import build as b

    b.build()
    import top_sampling_gb300 as ts

    size = ts.load().vsamp_block_matmul_workspace_size
    for M, N, K in SIZES + [(2048, 4096, 151936)]:
        need, tiles, least = _room(M, N, K, size)
        assert 0 < need < least and tiles > (76 if M > 128 else 152), (M, N, K)
    for M, N, K in ((4, 100, 151936), (64, 4096, 151936), (300, 300, 100000)):
        assert size(M, N, K) > 0, (M, N, K)


@pytest.fixture(scope="module")
def ts():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g

    g.build()
    import top_sampling_gb300 as ts_mod

    return ts_mod


def _operand(ts, rows, cols, tile, dev, seed):
    gen = torch.Generator(device=dev).manual_seed(seed)
    t = ts.BlockTensor.empty(rows, cols, tile, dev)
    t.codes.copy_((torch.randn((rows, cols), generator=gen, device=dev) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn))
    t.scales.copy_(torch.exp2(torch.rand(t.scales.shape, generator=gen, device=dev) * 4 - 14))
    return t


def _values(t):
    s = t.scales.double()
    s = s.repeat_interleave(128, 0)[:t.rows] if t.tile else s.t()
    return t.codes.view(torch.float8_e4m3fn).double() * s.repeat_interleave(128, 1)[:, :t.cols]


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_mixed(ts, M, N, K, tile):
    dev = torch.device("cuda:0")
    need, _, least = _room(M, N, K, ts.load().vsamp_block_matmul_workspace_size)
    assert 0 < need < least
    a, b = _operand(ts, M, K, False, dev, 1), _operand(ts, N, K, tile, dev, 2)
    va, vb = _values(a), _values(b)
    want, size = va @ vb.t(), va.abs() @ vb.abs().t()
    gen = torch.Generator(device=dev).manual_seed(3)
    for out in (F32, BF16):
        for pad in (0, 1, 8):
            base = torch.randn((M, N + pad), generator=gen, device=dev).to(out)
            for add in (False, True):
                y = base.clone()
                ts.vsamp_block_matmul(a, b, out=y[:, :N], accumulate=add)
                whole = want + base[:, :N].double() if add else want
                tol = bu.product_tol(size + base[:, :N].double().abs() if add else size, K) + bu.HALF[out] * whole.abs()
                assert ((y[:, :N].double() - whole).abs() <= tol).all(), (out, pad, add)
                assert torch.equal(y[:, N:], base[:, N:])
                again = base.clone()
                ts.vsamp_block_matmul(a, b, out=again[:, :N], accumulate=add)
                assert torch.equal(again, y)
