"""The embedding lookup and its gradient on the GPU against binary64: odd widths and strides, repeated, ignored and bad
tokens, long runs of one token, repeatability."""
import numpy as np
import pytest

import tables_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]


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


@pytest.mark.parametrize("tdt", DTYPES)
@pytest.mark.parametrize("odt", DTYPES)
@pytest.mark.parametrize("N,V,D,pad", [(1, 1, 1, 0), (1, 50, 64, 0), (3, 7, 5, 1), (17, 100, 1001, 0), (64, 33, 2048, 8),
                                       (5, 9, 5000, 3)])
def test_lookup(ts, dev, tdt, odt, N, V, D, pad):
    rng = np.random.default_rng(N + D)
    table = torch.full((V, D + pad), 1e30, device=dev, dtype=tdt)
    table[:, :D] = torch.from_numpy(rng.normal(size=(V, D)).astype(np.float32)).to(dev).to(tdt)
    tok = rng.integers(0, V, size=N).astype(np.int32)
    if N > 2:
        tok[0], tok[1] = tu.IGNORE, V - 1
    out = torch.full((N, D + pad), 7.0, device=dev, dtype=odt)
    y, st = ts.vsamp_embed(torch.from_numpy(tok).to(dev), table[:, :D], scale=1.7, out=out[:, :D])
    want = np.where(tok[:, None] == tu.IGNORE, 0.0, tu.f64(table[:, :D])[np.maximum(tok, 0)] * float(np.float32(1.7)))
    assert (st == 0).all() and (out[:, D:] == 7.0).all()
    assert np.all(np.abs(tu.f64(y) - want) <= (tu.U + tu.HALF[odt]) * np.abs(want))


def test_lookup_of_bad_tokens(ts, dev):
    table = torch.randn((10, 33), device=dev)
    tok = torch.tensor([0, -1, 10, 2 ** 31 - 1, tu.IGNORE, 2 ** 40 + 3, 9], device=dev)
    y, st = ts.vsamp_embed(tok, table)
    assert st.tolist() == [0, 1, 1, 1, 0, 1, 0]
    assert torch.isnan(y[[1, 2, 3, 5]]).all() and not y[4].any()
    assert torch.equal(y[0], table[0]) and torch.equal(y[6], table[9])


def _check_grad(ts, tok, dout, V, scale, odt, accumulate, pad=0):
    dev, D = dout.device, dout.shape[1]
    base = torch.full((V, D + pad), 7.0, device=dev, dtype=odt)
    if accumulate:
        base[:, :D] = torch.randn((V, D), device=dev).to(odt)
    else:
        base[:, :D] = float("nan")
    before = tu.f64(base[:, :D])
    d = ts.vsamp_embed_backward(torch.from_numpy(tok).to(dev), dout, V, scale=scale, dtable=base[:, :D],
                                accumulate=accumulate)
    want, tol = tu.embed_grad(tok.astype(np.int64), tu.f64(dout), V, float(np.float32(scale)),
                              before if accumulate else None)
    assert np.all(np.abs(tu.f64(d) - want) <= tol + tu.HALF[odt] * np.abs(want))
    assert (base[:, D:] == 7.0).all()
    return d


@pytest.mark.parametrize("idt", DTYPES)
@pytest.mark.parametrize("odt", DTYPES)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("N,V,D,pad", [(1, 1, 1, 0), (2, 300, 7, 1), (15, 3, 64, 0), (16, 2, 33, 0), (17, 1000, 257, 5),
                                       (700, 50, 100, 0), (4097, 70000, 40, 0)])
def test_gradient(ts, dev, idt, odt, accumulate, N, V, D, pad):
    rng = np.random.default_rng(N * 3 + D)
    tok = rng.integers(0, V, size=N).astype(np.int32)
    if N > 10:
        tok[rng.integers(0, N, size=N // 8)] = tu.IGNORE
        tok[5], tok[6] = -1, V
    wide = torch.full((N, D + pad), 1e30, device=dev, dtype=idt)
    wide[:, :D] = torch.from_numpy(rng.normal(size=(N, D)).astype(np.float32)).to(dev).to(idt)
    _check_grad(ts, tok, wide[:, :D], V, 1.3, odt, accumulate, pad)


@pytest.mark.parametrize("N", [100, 5000, 20000])
def test_gradient_of_long_runs(ts, dev, N):
    """One token everywhere, and one that takes half of the positions."""
    rng = np.random.default_rng(N)
    dout = torch.from_numpy(rng.normal(size=(N, 48)).astype(np.float32)).to(dev)
    _check_grad(ts, np.full(N, 4, np.int32), dout, 9, 1.0, torch.float32, False)
    _check_grad(ts, np.full(N, tu.IGNORE, np.int32), dout, 9, 1.0, torch.float32, True)
    tok = rng.integers(0, 5000, size=N).astype(np.int32)
    tok[rng.random(N) < 0.5] = 77
    d = _check_grad(ts, tok, dout, 5000, 0.5, torch.bfloat16, False)
    again = ts.vsamp_embed_backward(torch.from_numpy(tok).to(dev), dout, 5000, scale=0.5, dtype=torch.bfloat16)
    assert torch.equal(d, again)


def test_gradient_of_many_positions(ts, dev):
    """More positions than one pass of tiles, ids over three sort digits: against index_add in 64 bits."""
    g = torch.Generator(device=dev).manual_seed(1)
    N, V, D = 300001, 200003, 8
    tok = torch.randint(0, V, (N,), generator=g, device=dev)
    dout = torch.randn((N, D), generator=g, device=dev)
    d = ts.vsamp_embed_backward(tok, dout, V)
    want = torch.zeros((V, D), dtype=torch.float64, device=dev).index_add_(0, tok, dout.double())
    size = torch.zeros((V, D), dtype=torch.float64, device=dev).index_add_(0, tok, dout.double().abs())
    assert ((d.double() - want).abs() <= size * 40 * tu.U).all()


def test_gradient_against_differences(ts, dev):
    """The lookup is linear: the gradient along a direction equals the difference of the looked-up sums."""
    rng = np.random.default_rng(7)
    N, V, D = 60, 20, 12
    tok = torch.from_numpy(rng.integers(0, V, size=N).astype(np.int32)).to(dev)
    table = torch.from_numpy(rng.normal(size=(V, D)).astype(np.float32)).to(dev)
    dout = torch.from_numpy(rng.normal(size=(N, D)).astype(np.float32)).to(dev)
    d = ts.vsamp_embed_backward(tok, dout, V, scale=2.0)
    v = torch.from_numpy(rng.normal(size=(V, D)).astype(np.float32)).to(dev)
    up = ts.vsamp_embed(tok, table + v, scale=2.0)[0].double()
    down = ts.vsamp_embed(tok, table - v, scale=2.0)[0].double()
    want = ((up - down) / 2 * dout.double()).sum()
    got = (d.double() * v.double()).sum()
    # each of the N * D values carries a few roundings of magnitude u * (|table| + |v|) * scale
    tol = (dout.double().abs().sum() * 2.0 * 10.0 * 4) * tu.U
    assert abs(float(got - want)) <= float(tol)


def test_other_stream_and_graph(ts, dev):
    g = torch.Generator(device=dev).manual_seed(3)
    N, V, D = 999, 500, 130
    tok = torch.randint(0, V, (N,), generator=g, device=dev).int()
    dout = torch.randn((N, D), generator=g, device=dev)
    ref = ts.vsamp_embed_backward(tok, dout, V)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = ts.vsamp_embed_backward(tok, dout, V, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(ref, other)
    graph = torch.cuda.CUDAGraph()
    ds = torch.zeros_like(dout)
    table = torch.randn((V, D), generator=g, device=dev)
    with torch.cuda.graph(graph):
        y, _ = ts.vsamp_embed(tok, table)
        d = ts.vsamp_embed_backward(tok, ds, V)
    ds.copy_(dout)
    graph.replay()
    assert torch.equal(d, ref) and torch.equal(y, table[tok.long()])


@pytest.mark.parametrize("V,D", [(300, 40), (20000, 500)])            # a small table, and one of 40 MB
@pytest.mark.parametrize("N", [255, 256, 257, 1023, 1024, 1025])
def test_gradient_on_both_sides_of_the_forms_limits(ts, dev, N, V, D):
    """The forms of few and of many positions, written whole and added, with the workspace that the library asks for."""
    rng = np.random.default_rng(N)
    tok = rng.integers(0, V, size=N).astype(np.int32)
    tok[: N // 4] = 3
    tok[::9] = tu.IGNORE
    dout = torch.from_numpy(rng.normal(size=(N, D)).astype(np.float32)).to(dev)
    lib = ts.load()
    ws = torch.empty(lib.vsamp_embed_workspace_size(N, D), dtype=torch.uint8, device=dev)
    for accumulate in (False, True):
        want, tol = tu.embed_grad(tok.astype(np.int64), tu.f64(dout), V, 2.0, np.ones((V, D)) if accumulate else None)
        d = ts.vsamp_embed_backward(torch.from_numpy(tok).to(dev), dout, V, scale=2.0, workspace=ws,
                                    dtable=torch.ones((V, D), device=dev), accumulate=accumulate)
        assert np.all(np.abs(tu.f64(d) - want) <= tol + tu.U * np.abs(want))
