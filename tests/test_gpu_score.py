"""Token scores and their gradient on the GPU against binary64: lengths from one token on, strides, masks, ties, error
rows, invariance, graphs and streams."""
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


def _rows(a, dtype, dev, pad=0, fill=1e30):
    """Rows of `a` at a stride of V + pad, what is between them filled with a value that must not be read."""
    B, V = a.shape
    x = torch.full((B, V + pad), fill, device=dev, dtype=dtype)
    x[:, :V] = torch.from_numpy(a).to(dev).to(dtype)
    return x[:, :V]


def _check(ts, x, token, temps, n, st_expected=None):
    out = ts.vsamp_score_tokens(x, torch.tensor(token, dtype=torch.int32, device=x.device),
                                temperature=None if temps is None else torch.tensor(temps, device=x.device), n_alt=n)
    lp, ent, rank, ai, al, m, ls, st = [None if o is None else o.cpu().numpy() for o in out]
    xs = tu.f64(x)
    for r in range(len(token)):
        T = 1.0 if temps is None else float(np.float32(temps[r]))
        s0, lp0, e0, k0, ai0, al0, m0, ls0 = tu.score_row(xs[r], token[r], T, n)
        assert st[r] == s0, (r, st[r], s0)
        assert rank[r] == k0, (r, rank[r], k0)
        if n:
            assert np.array_equal(ai[r], ai0), (r, ai[r], ai0)
            assert np.array_equal(np.isnan(al[r]), np.isnan(al0))
            ok = ~np.isnan(al0)
            assert np.all(np.abs(al[r][ok] - al0[ok]) <= tu.logprob_tol(al0[ok])), r
        if s0 != 0:
            assert np.isnan([lp[r], ent[r], m[r], ls[r]]).all()
            continue
        assert m[r] == np.float32(m0)
        if np.isinf(lp0):
            assert lp[r] == lp0
        else:
            assert abs(lp[r] - lp0) <= tu.logprob_tol(lp0), (r, lp[r], lp0)
        assert abs(ls[r] - ls0) <= tu.LOGSUM_TOL + tu.U * abs(ls0)
        assert abs(ent[r] - e0) <= tu.entropy_tol(ls0), (r, ent[r], e0)
    if st_expected is not None:
        assert list(st) == st_expected
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,n,pad", [(1, 1, 0), (1, 5, 3), (2, 0, 0), (7, 20, 1), (31, 31, 0), (128, 5, 0),
                                     (1023, 20, 0), (1024, 20, 8), (1025, 64, 0), (2049, 1, 7), (4097, 20, 0),
                                     (20011, 128, 5), (32000, 20, 0)])
def test_random_rows(ts, dev, dtype, V, n, pad):
    rng = np.random.default_rng(V * 7 + n)
    B = 6
    a = rng.normal(0.0, 2.5, size=(B, V)).astype(np.float32)
    a[1] = rng.integers(-4, 5, size=V) / 2.0                       # many ties
    a[2, : V // 2], a[2, V // 2:] = -0.0, 0.0                      # one value
    a[3] = rng.normal(1.0e4, 2.5, size=V)                          # far from zero
    a[4, rng.integers(0, V)] = 60.0                                # one token takes all
    token = rng.integers(0, V, size=B).tolist()
    token[5] = V - 1
    _check(ts, _rows(a, dtype, dev, pad), token, None, n)
    _check(ts, _rows(a, dtype, dev, pad), token, [0.7, 1.3, 1.0, 2.5, 0.0, -1.0], n)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [0, 20])
def test_extreme_temperatures(ts, dev, dtype, n):
    rng = np.random.default_rng(21)
    temps = [1e-3, 1e-7, 1e-9, 1e-12, 1e-20, 1e-30, 1e4, 1e20, 3e38]
    a = rng.normal(0.0, 2.5, size=(len(temps), 5001)).astype(np.float32)
    a[:, ::3] = -np.inf
    a[2, 1] = a[2, 4000] = 30.0                        # two equal maxima: each takes half
    token = [int(np.argmax(a[r])) if r % 2 else 1 for r in range(len(temps))]
    x = _rows(a, dtype, dev)
    _check(ts, x, token, temps, n)
    # quotients by a temperature below 1e-38 overflow: the maximum keeps the log-probability 0
    top = [int(np.argmax(tu.f64(x)[r])) for r in range(len(temps))]
    out = ts.vsamp_score_tokens(x, torch.tensor(top, device=dev), temperature=1e-40, n_alt=1)
    assert (out[7] == 0).all() and (out[4][:, 0] == out[0]).all()
    for r in range(len(temps)):
        ties = int((tu.f64(x)[r] == tu.f64(x)[r].max()).sum())
        assert abs(float(out[0][r]) + np.log(ties)) <= tu.LOGSUM_TOL


@pytest.mark.parametrize("dtype", DTYPES)
def test_smallest_temperature_at_a_maximum_of_zero(ts, dev, dtype):
    # m - 104 T is a value of its own below m = 0 at every T: masked tokens must still add nothing
    a = np.full((1, 5001), -np.inf, np.float32)
    a[0, 7], a[0, 9] = 0.0, -1.0
    for t in (1e-40, 3e-39, 1e-38, 1e-30):
        out = ts.vsamp_score_tokens(_rows(a, dtype, dev), torch.tensor([7], device=dev), temperature=t, n_alt=2)
        assert float(out[0][0]) == 0.0 and int(out[7][0]) == 0
        assert out[3][0].tolist() == [7, 9]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [0, 20, 128])
def test_masked_tokens(ts, dev, dtype, n):
    rng = np.random.default_rng(n + 1)
    V = 9001
    a = rng.normal(0.0, 2.0, size=(6, V)).astype(np.float32)
    a[0, rng.random(V) < 0.5] = -np.inf
    a[1, rng.random(V) < 0.999] = -np.inf             # fewer tokens than alternatives
    a[2, 5000:] = -np.inf                             # whole pieces masked behind
    a[3, :5000] = -np.inf                             # and in front
    a[4] = -np.inf
    a[4, 7777] = -3.0                                 # one token left
    a[5, ::2] = np.finfo(np.float32).min              # the type's lowest value is not a mask
    if dtype == torch.bfloat16:
        a[5, ::2] = -3.3895313892515355e38
    live = [int(np.flatnonzero(a[r] > -np.inf)[-1]) for r in range(6)]
    _check(ts, _rows(a, dtype, dev, 1), live, None, n)
    # a masked given token: log-probability -inf, behind every unmasked one
    masked = [int(np.flatnonzero(a[r] == -np.inf)[len(np.flatnonzero(a[r] == -np.inf)) // 2]) for r in range(5)] + [0]
    _check(ts, _rows(a, dtype, dev), masked, [0.5, 1.0, 2.0, 1.0, 1.0, 1.0], n)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [0, 5])
def test_error_and_ignored_rows(ts, dev, dtype, n):
    rng = np.random.default_rng(3)
    V = 5003
    a = rng.normal(0.0, 1.0, size=(9, V)).astype(np.float32)
    a[0, 17] = np.nan
    a[1, V - 1] = np.inf
    a[2] = -np.inf                                    # nothing left
    a[7] = np.nan                                     # never read
    token = [1, 2, 3, -1, V, 4, 5, tu.IGNORE, 6]
    temps = [1.0, 1.0, 1.0, 1.0, 1.0, float("nan"), float("inf"), float("nan"), 1.0]
    _check(ts, _rows(a, dtype, dev), token, temps, n, [4, 4, 4, 1, 1, 1, 1, 0, 0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_alternatives_of_adverse_rows(ts, dev, dtype):
    """Rows whose largest tokens crowd into few chunks, so that more candidates pass than the short list holds."""
    rng = np.random.default_rng(11)
    V = 40000
    a = rng.normal(-50.0, 1.0, size=(5, V)).astype(np.float32)
    a[0, :4000] = rng.normal(10.0, 3.0, size=4000)
    a[1, V - 4001:] = rng.normal(10.0, 3.0, size=4001)
    a[2] = 1.0                                        # every token ties
    a[3] = np.arange(V)[::-1] / 64.0                  # sorted
    a[4] = np.arange(V) / 64.0
    token = [10, V - 10, 12345, 0, 0]
    for n in (1, 20, 128):
        _check(ts, _rows(a, dtype, dev), token, None, n)


@pytest.mark.parametrize("n", [20, 128])
def test_alternatives_of_long_adverse_rows(ts, dev, n):
    """A million tokens whose chunks (of 128 fp32 tokens, dealt to 256 threads in turn) defeat the bound: tokens in fewer
    threads' chunks than there are alternatives; large tokens in the chunks of fewer groups of threads."""
    rng = np.random.default_rng(n)
    V = 1 << 20
    thread = (np.arange(V) // 128) % 256
    a = rng.normal(0.0, 1.0, size=(2, V)).astype(np.float32)
    a[0, thread >= 100] = -np.inf
    a[1, thread < 8 * 19] += 100.0
    live = int(np.flatnonzero(a[0] > -np.inf)[12345])
    _check(ts, _rows(a, torch.float32, dev), [live, 7], None, n)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("extra", [0, 1, 5])
def test_whole_pieces_at_the_ends_of_unaligned_logits(ts, dev, dtype, extra):
    """The first and the last piece of the logits are whole and begin on any boundary; what stands around them is NaN."""
    V = 2 * 4096 // dtype.itemsize + extra
    rng = np.random.default_rng(extra)
    a = rng.normal(0.0, 2.5, size=(3, V)).astype(np.float32)
    for off in range(1, 16 // dtype.itemsize):
        flat = torch.full((off + a.size + 16,), float("nan"), dtype=dtype, device=dev)
        x = flat[off:off + a.size].view(3, V)
        x.copy_(torch.from_numpy(a))
        _check(ts, x, [0, V - 1, V - 1], [1.0, 0.7, 1.3], 20)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V", [(3, 5000), (1500, 5000), (40, 40000)])
def test_more_candidates_than_the_list_holds_on_every_call(ts, dev, dtype, B, V):
    """Every token of every row ties, so each row's listing runs over and is begun anew, in the form of one launch and in
    that of two: the first tokens on every one of many calls, whatever the warps' timing."""
    x = torch.full((B, V), 1.5, dtype=dtype, device=dev)
    x[1::3, ::2] = -3.0                                # half of the tokens tie: the odd ones
    tok = torch.full((B,), V - 1, dtype=torch.int32, device=dev)
    for n in (1, 20, 128):
        want = torch.arange(n, dtype=torch.int32, device=dev).repeat(B, 1)
        want[1::3] = want[1::3] * 2 + 1
        outs = [ts.vsamp_score_tokens(x, tok, n_alt=n) for _ in range(20)]
        for out in outs:
            assert torch.equal(out[3], want) and not out[7].any()
            assert all(torch.equal(p, q) for p, q in zip(out, outs[0]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V", [(2, 60), (16, 32000), (40, 60000)])
def test_short_clusters_on_every_call(ts, dev, dtype, B, V):
    """The form of one launch, whose CTAs write their pieces' records into the first CTA of their cluster: pieces of a few
    elements (a record is ready at once), several CTAs per row, ignored rows between, one call right behind another."""
    g = torch.Generator(device=dev).manual_seed(B)
    x = torch.randn((B, V), generator=g, device=dev).to(dtype)
    tok = torch.randint(0, V, (B,), generator=g, device=dev, dtype=torch.int32)
    tok[1::5] = tu.IGNORE
    first = ts.vsamp_score_tokens(x, tok, n_alt=20)
    outs = [ts.vsamp_score_tokens(x, tok, n_alt=20) for _ in range(50)]
    reps = 5000 // (B * ((V + 2047) // 2048)) + 1                                 # more pieces than one launch takes
    wide = ts.vsamp_score_tokens(x.repeat(reps, 1), tok.repeat(reps), n_alt=20)
    for out in outs:
        for p, q, w in zip(out, first, wide):
            assert torch.equal(p.view(torch.int32), q.view(torch.int32))
            assert torch.equal(p.view(torch.int32), w[:B].contiguous().view(torch.int32))


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_launch_and_two_agree(ts, dev, dtype):
    """A large batch takes two launches, each of its rows alone one: the same bits."""
    rng = np.random.default_rng(12)
    B, V = 700, 10007
    a = rng.normal(0.0, 3.0, size=(B, V)).astype(np.float32)
    x = _rows(a, dtype, dev)
    tok = torch.from_numpy(rng.integers(0, V, size=B).astype(np.int32)).to(dev)
    T = torch.from_numpy(rng.uniform(0.5, 2.0, size=B).astype(np.float32)).to(dev)
    for n in (0, 20):
        all_rows = ts.vsamp_score_tokens(x, tok, temperature=T, n_alt=n)
        for r in (0, 1, 333, B - 1):
            one = ts.vsamp_score_tokens(x[r:r + 1], tok[r:r + 1], temperature=T[r:r + 1], n_alt=n)
            for p, q in zip(all_rows, one):
                assert (p is None and q is None) or torch.equal(p[r:r + 1], q)


def test_large_vocabulary(ts, dev):
    g = torch.Generator(device=dev).manual_seed(5)
    x = (torch.randn((3, 151936), generator=g, device=dev) * 2.5).to(torch.bfloat16)
    _check(ts, x, [0, 151935, 75000], [1.0, 0.6, 1.4], 20)
    # more than 2^31 bytes of logits: offsets pass 32 bits
    B, V = 9000, 151936
    x = torch.empty((B, V), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    tok = torch.full((B,), tu.IGNORE, dtype=torch.int32, device=dev)
    tok[-2:] = 99
    out = ts.vsamp_score_tokens(x, tok, n_alt=20)
    ref = ts.vsamp_score_tokens(x[-2:].clone(), tok[-2:], n_alt=20)
    for got, want in zip(out, ref):
        assert torch.equal(got[-2:], want)
    assert (out[7][:-2] == 0).all() and (out[0][:-2] == 0).all() and (out[3][:-2] == -1).all()
    d, st = ts.vsamp_score_tokens_backward(x, tok, torch.ones(B, device=dev), out[5], out[6])
    d2, _ = ts.vsamp_score_tokens_backward(x[-2:].clone(), tok[-2:], torch.ones(2, device=dev), ref[5], ref[6])
    assert torch.equal(d[-2:], d2) and not d[:-2].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_do_not_depend_on_the_batch_or_the_stride(ts, dev, dtype):
    rng = np.random.default_rng(8)
    B, V = 40, 10007
    a = rng.normal(0.0, 3.0, size=(B, V)).astype(np.float32)
    tok = torch.from_numpy(rng.integers(0, V, size=B).astype(np.int32)).to(dev)
    outs = [ts.vsamp_score_tokens(_rows(a, dtype, dev, pad), tok, n_alt=20) for pad in (0, 1, 9)]
    one = [ts.vsamp_score_tokens(_rows(a[r:r + 1], dtype, dev), tok[r:r + 1], n_alt=20) for r in (0, 23)]
    for other in outs[1:]:
        for p, q in zip(outs[0], other):
            assert torch.equal(p, q)
    for r, o in zip((0, 23), one):
        for p, q in zip(outs[0], o):
            assert torch.equal(p[r:r + 1], q)


# ------------------------------------------------------------------------------------------------
# gradient
# ------------------------------------------------------------------------------------------------
def _grad(ts, x, token, temps, g, h, **kw):
    dev = x.device
    tok = torch.tensor(token, dtype=torch.int32, device=dev)
    T = None if temps is None else torch.tensor(temps, device=dev)
    f = ts.vsamp_score_tokens(x, tok, temperature=T)
    gt = None if g is None else torch.tensor(g, dtype=torch.float32, device=dev)
    ht = None if h is None else torch.tensor(h, dtype=torch.float32, device=dev)
    return f, ts.vsamp_score_tokens_backward(x, tok, gt, f[5], f[6], entropy=f[1], dentropy=ht, temperature=T, **kw)


def _check_grad(ts, x, token, temps, g, h):
    xs = tu.f64(x)
    _, (d, st) = _grad(ts, x, token, temps, g, h)
    d = tu.f64(d)
    for r in range(len(token)):
        T = 1.0 if temps is None else float(np.float32(temps[r]))
        want, size = tu.grad_row(xs[r], token[r], T, 0.0 if g is None else float(np.float32(g[r])),
                                 0.0 if h is None else float(np.float32(h[r])))
        tol = tu.GRAD_REL * size + tu.HALF[x.dtype] * np.abs(want) + 1e-37
        assert st[r] == 0
        assert np.all(np.abs(d[r] - want) <= tol), (r, np.max(np.abs(d[r] - want) - tol))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,pad", [(1, 0), (2, 1), (7, 0), (33, 3), (1024, 0), (4099, 0), (8200, 8), (20001, 2)])
def test_gradient(ts, dev, dtype, V, pad):
    rng = np.random.default_rng(V)
    B = 6
    a = rng.normal(0.0, 2.5, size=(B, V)).astype(np.float32)
    a[1] += 1.0e4
    a[2, rng.random(V) < 0.5] = -np.inf
    token = rng.integers(0, V, size=B).tolist()
    a[2, token[2]] = 1.0
    token[3] = tu.IGNORE
    a[4, token[4]] = 30.0
    x = _rows(a, dtype, dev, pad)
    g, h = rng.normal(size=B), rng.normal(size=B) * 0.1
    _check_grad(ts, x, token, None, g, h)
    _check_grad(ts, x, token, [0.7, 1.5, 1.0, 1.0, 0.0, 3.0], g, h)
    _check_grad(ts, x, token, None, g, None)
    _check_grad(ts, x, token, None, None, h)


def test_gradient_against_differences(ts, dev):
    """Central differences of the forward call along random directions. With a step of 2^-5 the truncation is below
    step^2 (third derivatives of both scores along a unit direction are below 6), the forward's rounding
    2 * tol / (2 * step)."""
    rng = np.random.default_rng(2)
    B, V, step = 5, 301, 2.0 ** -5
    a = rng.normal(0.0, 1.5, size=(B, V)).astype(np.float32)
    token = rng.integers(0, V, size=B).tolist()
    g, h = rng.normal(size=B), rng.normal(size=B)
    temps = [1.0, 0.8, 1.3, 1.0, 2.0]
    x = _rows(a, torch.float32, dev)
    _, (d, _) = _grad(ts, x, token, temps, g, h)
    tok, T = torch.tensor(token, dtype=torch.int32, device=dev), torch.tensor(temps, device=dev)
    for k in range(4):
        v = rng.normal(size=(B, V))
        v /= np.linalg.norm(v, axis=1, keepdims=True)
        vt = torch.from_numpy(v).to(dev).float()
        up, down = ts.vsamp_score_tokens(x + step * vt, tok, T), ts.vsamp_score_tokens(x - step * vt, tok, T)
        got = (d.double() * vt.double()).sum(1).cpu().numpy()
        want = (g * tu.f64(up[0] - down[0]) + h * tu.f64(up[1] - down[1])) / (2 * step)
        tol = (np.abs(g) + np.abs(h)) * (step ** 2 + 2 * tu.entropy_tol(np.log(V)) / (2 * step))
        assert np.all(np.abs(got - want) <= tol), (got - want, tol)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_of_error_rows_in_place_and_padded(ts, dev, dtype):
    rng = np.random.default_rng(4)
    B, V = 5, 3001
    a = rng.normal(size=(B, V)).astype(np.float32)
    a[1, 5] = np.nan
    a[2] = -np.inf
    token = [3, 4, 5, -7, tu.IGNORE]
    x = _rows(a, dtype, dev)
    g = np.ones(B)
    _, (d, st) = _grad(ts, x, token, None, g, None)
    assert st.tolist() == [0, 4, 4, 1, 0]
    assert torch.isnan(d[1:4]).all() and not d[4].any() and torch.isfinite(d[0]).all()
    # a padded output keeps what is between its rows
    out = torch.full((B, V + 3), 7.0, dtype=dtype, device=dev)
    _, (d2, _) = _grad(ts, x, token, None, g, None, dlogits=out[:, :V])
    assert torch.equal(d2[0], d[0]) and (out[:, V:] == 7.0).all()
    # the logits' own buffer
    y = x.clone()
    _, (d3, _) = _grad(ts, y, token, None, g, None, dlogits=y)
    assert d3.data_ptr() == y.data_ptr() and torch.equal(y[0], d[0]) and not y[4].any()


def test_other_stream_and_graph(ts, dev):
    rng = np.random.default_rng(6)
    a = rng.normal(size=(8, 20000)).astype(np.float32)
    x = _rows(a, torch.float32, dev)
    tok = torch.arange(8, device=dev)                      # 64-bit ids
    ref = ts.vsamp_score_tokens(x, tok, temperature=0.9, n_alt=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = ts.vsamp_score_tokens(x, tok, temperature=0.9, n_alt=5, stream=side)
    raw = ts.vsamp_score_tokens(x, tok, temperature=0.9, n_alt=5, stream=side.cuda_stream)
    torch.cuda.synchronize()
    for p, q, s in zip(ref, other, raw):
        assert torch.equal(p, q) and torch.equal(p, s)
    graph = torch.cuda.CUDAGraph()
    xs = x.clone()
    tok32 = tok.int()
    with torch.cuda.graph(graph):
        out = ts.vsamp_score_tokens(xs, tok32, n_alt=5)
        d, _ = ts.vsamp_score_tokens_backward(xs, tok32, out[0], out[5], out[6])
    xs.copy_(x * 0.5)
    graph.replay()
    want = ts.vsamp_score_tokens(x * 0.5, tok, n_alt=5)
    dw, _ = ts.vsamp_score_tokens_backward(x * 0.5, tok, want[0], want[5], want[6])
    for p, q in zip(out, want):
        assert torch.equal(p, q)
    assert torch.equal(d, dw)
