"""The 4-bit output head on the GPU against binary64: group sizes, zero points, types, ragged vocabularies, one to many
rows, strides."""
import numpy as np
import pytest

import tables_util as tu

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


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def _weights(V, D, group, sdt, zeros, dev, seed):
    rng = np.random.default_rng(seed)
    codes = torch.from_numpy(rng.integers(0, 256, size=(V, D // 2), dtype=np.uint8)).to(dev)
    scales = torch.from_numpy(rng.uniform(0.001, 0.02, size=(V, D // group)).astype(np.float32)).to(dev).to(sdt)
    z = torch.from_numpy(rng.integers(0, 16, size=(V, D // group)).astype(np.uint8)).to(dev) if zeros else None
    return codes, scales, z


def _check(ts, hidden, w, group, out_dtype, out=None):
    codes, scales, z = w
    head = ts.vsamp_head_pack(codes, scales, zeros=z, group=group)
    y = ts.vsamp_head_logits(hidden, head, out=out, out_dtype=out_dtype)
    want, size = tu.head(tu.f64(hidden), codes.cpu().numpy(), tu.f64(scales), None if z is None else z.cpu().numpy(),
                         group)
    terms = 3 if hidden.dtype == torch.float32 else 1
    tol = tu.head_tol(size, group, scales.shape[1], terms) + tu.HALF[y.dtype] * np.abs(want)
    assert np.all(np.abs(tu.f64(y) - want) <= tol)
    return head, y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("V,blocks", [(1, 1), (15, 3), (16, 2), (17, 1), (129, 5), (1000, 9)])
def test_shapes(ts, dev, group, zeros, V, blocks):
    D = group * blocks
    rng = np.random.default_rng(V + D)
    for M, hdt, sdt, odt in [(1, torch.bfloat16, torch.bfloat16, torch.float32),
                             (3, torch.float32, torch.bfloat16, torch.bfloat16),
                             (8, torch.bfloat16, torch.float32, torch.bfloat16),
                             (9, torch.float32, torch.float32, torch.float32)]:
        h = torch.from_numpy(rng.normal(size=(M, D)).astype(np.float32)).to(dev).to(hdt)
        _check(ts, h, _weights(V, D, group, sdt, zeros, dev, V), group, odt)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 65, 130])
@pytest.mark.parametrize("hdt", [torch.float32, torch.bfloat16])
def test_rows(ts, dev, M, hdt):
    V, D, group = 211, 448, 64
    rng = np.random.default_rng(M)
    h = torch.from_numpy(rng.normal(size=(M, D)).astype(np.float32)).to(dev).to(hdt)
    w = _weights(V, D, group, torch.bfloat16, True, dev, M)
    head, y = _check(ts, h, w, group, torch.float32)
    # padded hidden rows and logits rows; what is between the rows stays
    hp = torch.full((M, D + 5), 1e30, dtype=hdt, device=dev)
    hp[:, :D] = h
    out = torch.full((M, V + 3), 7.0, device=dev)
    ts.vsamp_head_logits(hp[:, :D], head, out=out[:, :V])
    assert torch.equal(out[:, :V], y) and (out[:, V:] == 7.0).all()


@pytest.mark.parametrize("hdt,M", [(torch.bfloat16, 1), (torch.bfloat16, 40), (torch.float32, 24)])
def test_long_inner_dimension(ts, dev, hdt, M):
    V, D, group = 100, 8192 + 32, 32     # hidden states beyond one staging of shared memory for the larger M
    rng = np.random.default_rng(5)
    h = torch.from_numpy(rng.normal(size=(M, D)).astype(np.float32)).to(dev).to(hdt)
    _check(ts, h, _weights(V, D, group, torch.bfloat16, False, dev, 1), group, torch.float32)


def test_many_tiles(ts, dev):
    V, D, group = 40007, 256, 128
    h = torch.randn((2, D), device=dev).to(torch.bfloat16)
    _check(ts, h, _weights(V, D, group, torch.bfloat16, False, dev, 2), group, torch.bfloat16)


def test_special_hidden_values(ts, dev):
    """Infinities and NaN reach the logits of their own row alone; the largest and subnormal values stay exact."""
    V, D, group = 33, 64, 32
    codes, scales, _ = _weights(V, D, group, torch.float32, False, dev, 3)
    codes = torch.full_like(codes, 0x99)          # every weight is +1 * scale
    scales = torch.full_like(scales, 0.5)
    head = ts.vsamp_head_pack(codes, scales, group=group)
    for dt in (torch.float32, torch.bfloat16):
        h = torch.zeros((6, D), device=dev, dtype=dt)
        h[0, 3] = float("inf")
        h[1, 63] = float("nan")
        h[2, 0] = 1.0
        h[3, 1] = 2.0 ** -120
        h[4, 5] = 2.0 ** 120
        h[5, 7] = -float("inf")
        y = ts.vsamp_head_logits(h, head)
        assert (y[0] == float("inf")).all() and torch.isnan(y[1]).all() and (y[2] == 0.5).all()
        assert (y[3] == 2.0 ** -121).all() and (y[4] == 2.0 ** 119).all() and (y[5] == -float("inf")).all()


def test_largest_fp32_values(ts, dev):
    """Finite values that would round to an infinite bf16 stay finite."""
    V, D, group = 16, 32, 32
    codes = torch.full((V, D // 2), 0x99, dtype=torch.uint8, device=dev)      # weights 1 * scale
    scales = torch.full((V, 1), 2.0 ** -10, device=dev)
    head = ts.vsamp_head_pack(codes, scales, group=group)
    h = torch.zeros((2, D), device=dev)
    h[0, 4] = torch.finfo(torch.float32).max
    h[1, 9] = -torch.finfo(torch.float32).max
    y = tu.f64(ts.vsamp_head_logits(h, head))
    want, size = tu.head(tu.f64(h), codes.cpu().numpy(), tu.f64(scales), None, group)
    assert np.all(np.abs(y - want) <= tu.head_tol(size, group, 1, 3) + tu.U * np.abs(want))


def test_other_stream_and_graph(ts, dev):
    V, D, group = 5000, 512, 64
    w = _weights(V, D, group, torch.bfloat16, True, dev, 9)
    head = ts.vsamp_head_pack(w[0], w[1], zeros=w[2], group=group)
    h = torch.randn((4, D), device=dev).to(torch.bfloat16)
    ref = ts.vsamp_head_logits(h, head)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = ts.vsamp_head_logits(h, head, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(ref, other)
    graph = torch.cuda.CUDAGraph()
    hs = torch.zeros_like(h)
    with torch.cuda.graph(graph):
        y = ts.vsamp_head_logits(hs, head)
        tok, lp, st, _ = ts.vsamp_sample(y)
    hs.copy_(h)
    graph.replay()
    assert torch.equal(y, ref) and (st == 0).all()
    one = ts.vsamp_head_logits(h[2:3], head)
    assert torch.equal(one[0], ref[2])           # a row does not depend on the others
