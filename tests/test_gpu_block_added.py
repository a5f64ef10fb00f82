"""Additions of a product to fp32 results where values are below 2^-126: only those may count as zeros, whichever way a tile
leaves."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -126     # the smallest normal number


@pytest.fixture(scope="module")
def ts():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g

    g.build()
    import top_sampling_gb300 as ts_mod

    return ts_mod


def _flushed(x):
    return torch.where(x.abs() < LEAST, torch.copysign(torch.zeros_like(x), x), x)


@pytest.mark.parametrize("tile", [False, True])
# rows that leave as boxes; two elements and one element at a time; a divided inner dimension
@pytest.mark.parametrize("N,K,pad,divided", [(192, 256, 0, False), (192, 256, 2, False), (192, 256, 1, False),
                                             (191, 256, 1, False), (192, 20000, 0, True), (191, 20000, 1, True)])
def test_values_below_the_normal_ones(ts, tile, N, K, pad, divided):
    """One 1 times 1 per row, scaled to 2^-e: the product is 2^-e exactly, and a sum in binary64 too, which is rounded once. Where
    what is added, what it is added to and the sum are 2^-126 or more, it is that; else it is that or the sum with zeros in the
    place of what is less. The same call gives the same."""
    dev = torch.device("cuda:0")
    M = 40
    assert (ts.load().vsamp_block_matmul_workspace_size(M, N, K) > 0) == divided
    a, b = ts.BlockTensor.empty(M, K, False, dev), ts.BlockTensor.empty(N, K, tile, dev)
    for t in (a, b):
        t.codes.view(torch.uint8).zero_()
        t.codes.view(torch.uint8)[:, 5] = 0x38          # 1
        t.scales.fill_(1.0)
    sign = torch.where(torch.arange(M, device=dev) % 3 == 0, -1.0, 1.0)
    power = (torch.arange(M, device=dev) % 10).float()
    a.scales[0] = torch.exp2(-60 - power) * sign         # products 2^-120 to 2^-129
    b.scales[..., 0].fill_(2.0 ** -60) if tile else b.scales[0].fill_(2.0 ** -60)
    v = (a.scales[0].double() * 2.0 ** -60).float()[:, None].expand(M, N)
    start = torch.tensor([0.0, 3 * 2.0 ** -128, -(2.0 ** -127), 2.0 ** -126, -1.5 * 2.0 ** -126, 2.0 ** -149, 1.0, -0.0,
                          2.0 ** -120], dtype=torch.float64, device=dev).float()
    old = start[(torch.arange(M * N, device=dev) % len(start))].view(M, N)
    got = []
    for _ in range(2):
        y = torch.full((M, N + pad), 7.0, device=dev)
        y[:, :N] = old
        ts.vsamp_block_matmul(a, b, out=y[:, :N], accumulate=True)
        assert (y[:, N:] == 7.0).all()
        got.append(y)
    assert torch.equal(*got)
    kept = (old.double() + v.double()).float()
    flushed = _flushed((_flushed(old).double() + _flushed(v).double()).float())
    assert ((y[:, :N] == kept) | (y[:, :N] == flushed)).all()
    normal = (old == _flushed(old)) & (v == _flushed(v)) & (kept == _flushed(kept))
    assert 0 < int(normal.sum()) < normal.numel() and torch.equal(kept[normal], flushed[normal])
    # written results and sums in bf16 keep them
    assert torch.equal(ts.vsamp_block_matmul(a, b, out_dtype=torch.float32), v)
    z = torch.zeros((M, N), dtype=torch.bfloat16, device=dev)
    assert torch.equal(ts.vsamp_block_matmul(a, b, out=z, accumulate=True).float(), v)
