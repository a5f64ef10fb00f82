"""Token scores and their gradient where the formulas leave fp32's range on the way: smallest and largest temperatures,
differences of logits beyond the largest fp32 value, largest incoming gradients."""
import numpy as np
import pytest

import tables_util as tu
from test_gpu_score import DTYPES, _check, _rows, dev, ts  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _gradient(ts, x, token, temps, g, h):
    """The gradient against the formula's. Where its bound reaches past the type's largest value an infinity is as good;
    a token whose exponential is below 2^-126 (allowing for its rounding) may count as one without probability."""
    d = x.device
    tok, T = torch.tensor(token, dtype=torch.int32, device=d), torch.tensor(temps, dtype=torch.float32, device=d)
    gt, ht = torch.tensor(g, dtype=torch.float32, device=d), torch.tensor(h, dtype=torch.float32, device=d)
    f = ts.vsamp_score_tokens(x, tok, temperature=T)
    out, st = ts.vsamp_score_tokens_backward(x, tok, gt, f[5], f[6], entropy=f[1], dentropy=ht, temperature=T)
    assert not st.any() and not torch.isnan(out).any()
    got, xs = tu.f64(out), tu.f64(x)
    largest = torch.finfo(x.dtype).max
    for r in range(len(token)):
        want, size = tu.grad_row(xs[r], token[r], float(np.float32(temps[r])), float(np.float32(g[r])),
                                 float(np.float32(h[r])))
        t = float(np.float32(temps[r]))
        small = np.exp((xs[r] - xs[r].max()) / t) < 2.0 ** -125
        small[token[r]] = False
        tol = np.where(small, size, tu.GRAD_REL * size) + tu.HALF[x.dtype] * np.abs(want) + 1e-37
        near, beyond = np.abs(want) + tol <= largest, np.abs(want) - tol > largest
        assert np.all(np.abs(got[r] - want)[near] <= tol[near]), (r, temps[r])
        assert np.all(got[r][beyond] == np.inf * np.sign(want[beyond])), (r, temps[r])


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_at_extreme_temperatures(ts, dev, dtype):
    temps = [1e-20, 1e-30, 1e-36, 3e-37, 1e-38, 1e-40, 1e-44, 1e30, 3e37, 3e38]
    rng = np.random.default_rng(5)
    a = rng.normal(0.0, 2.5, size=(len(temps), 3001)).astype(np.float32)
    a[:, ::3] = -np.inf
    a[::2, 1] = a[::2, 2000] = 30.0                            # two equal maxima: each takes half
    token = [int(np.argmax(a[r])) if r % 3 else 4 for r in range(len(temps))]
    x = _rows(a, dtype, dev)
    for g, h in ((1e-3, 1e-2), (1.0, -0.5), (40.0, 3.0)):
        _gradient(ts, x, token, temps, [g] * len(temps), [h] * len(temps))


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_tokens_have_no_gradient_whatever_comes_in(ts, dev, dtype):
    rng = np.random.default_rng(6)
    a = rng.normal(0.0, 2.5, size=(4, 3001)).astype(np.float32)
    a[:, ::3] = -np.inf
    x = _rows(a, dtype, dev)
    tok = torch.tensor([1, 4, 2000, 7], dtype=torch.int32, device=dev)
    f = ts.vsamp_score_tokens(x, tok)
    for g, h in ((3e38, 0.0), (0.0, 2e36), (-1e38, 1e36)):
        d, st = ts.vsamp_score_tokens_backward(x, tok, torch.full((4,), g, device=dev), f[5], f[6], entropy=f[1],
                                               dentropy=torch.full((4,), h, device=dev))
        assert not st.any() and not torch.isnan(d).any() and not d[:, ::3].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [5001, 40001])
def test_alternatives_and_given_tokens_have_the_same_scores(ts, dev, dtype, V):
    """The log-probability of a token is one value, whether it is given or among the alternatives."""
    B, n = 64, 20
    g = torch.Generator(device=dev).manual_seed(V)
    x = (torch.randn((B, V), generator=g, device=dev) * 2.5).to(dtype)
    T = torch.rand(B, generator=g, device=dev) * 2 + 0.2
    out = ts.vsamp_score_tokens(x, 0, temperature=T, n_alt=n)
    for j in (0, 1, 7, n - 1):
        one = ts.vsamp_score_tokens(x, out[3][:, j].contiguous(), temperature=T)
        assert torch.equal(one[0], out[4][:, j]) and (one[2] == j).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [0, 20])
def test_differences_beyond_the_largest_value(ts, dev, monkeypatch, dtype, n):
    """Finite logits whose difference is not, at temperatures that bring it back; at T = 1 a log-probability beyond the
    largest value is an infinity."""
    def score_row(*args):
        status, lp, *rest = exact(*args)
        return (status, -np.inf if lp < -torch.finfo(torch.float32).max else lp, *rest)

    exact = tu.score_row
    monkeypatch.setattr(tu, "score_row", score_row)
    temps = [2e36, 1e37, 1e38, 3e38, 1.0, 4e36]
    rng = np.random.default_rng(9)
    a = rng.uniform(-3e38, 3e38, size=(len(temps), 5001)).astype(np.float32)
    a[:, ::3] = -np.inf
    a[5] = -1.1e38                                             # far below two equal maxima
    a[5, 10] = a[5, 4000] = 3e38
    x = _rows(a, dtype, dev)
    _check(ts, x, [1, 2, 4, 5, 7, 10], temps, n)
    _check(ts, x, [int(np.nanargmax(tu.f64(x)[r])) for r in range(len(temps))], temps, n)
    _gradient(ts, x, [1, 2, 4, 5, 7, 10], temps, [1e38] * len(temps), [1e37] * len(temps))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [0, 20])
def test_smallest_differences_at_smallest_temperatures(ts, dev, dtype, n):
    temps = [1e-39, 3e-39, 1e-38, 5e-38, 2e-37, 1e-36]
    rng = np.random.default_rng(10)
    a = (rng.integers(-60, 0, size=(len(temps), 5001)) * 2.0 ** -128).astype(np.float32)      # subnormal values
    a[:, ::3] = -np.inf
    x = _rows(a, dtype, dev)
    _check(ts, x, [1, 2, 4, 5, 7, 10], temps, n)
    _gradient(ts, x, [1, 2, 4, 5, 7, 10], temps, [1.0] * len(temps), [0.1] * len(temps))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,pad", [(1, 0), (2, 0), (37, 1), (5001, 0), (5001, 3), (40007, 0)])
def test_one_likely_token_keeps_the_digits_of_the_others(ts, dev, dtype, V, pad):
    """Rows whose largest token outweighs all others by up to 2^40: log S and the token's log-probability are held to the
    bound of a sum of the others, relative to it. The exponents that weigh are within 30 of the largest of the others."""
    rng = np.random.default_rng(V)
    tops = [3.0, 8.0, 14.0, 20.0, 27.0]
    a = rng.normal(0.0, 1.0, size=(2 * len(tops), V)).astype(np.float32)
    a[len(tops):, : V // 2] = -np.inf                              # a row whose other half is masked
    place = [0, V - 1, V // 2, V - 1 - V // 3, V // 7] * 2
    for r, (top, at) in enumerate(zip(tops * 2, place)):
        a[r, at] = top + np.log(V)
    x = _rows(a, dtype, dev, pad)
    reps = 5000 // (len(a) * ((V + 1023) // 1024)) + 1             # many rows take two launches
    xs = tu.f64(x)
    for temps in (None, [1.0, 0.9, 1.1, 1.0, 0.8] * 2):
        T = None if temps is None else torch.tensor(temps, device=dev)
        tok = torch.tensor(place, dtype=torch.int32, device=dev)
        out = ts.vsamp_score_tokens(x, tok, temperature=T, n_alt=3)
        many = ts.vsamp_score_tokens(x.repeat(reps, 1), tok.repeat(reps), n_alt=3,
                                     temperature=None if T is None else T.repeat(reps))
        for p, q in zip(out, many):
            assert torch.equal(p.view(torch.int32), q[: len(a)].contiguous().view(torch.int32))
        for r in range(len(a)):
            t = 1.0 if temps is None else float(np.float32(temps[r]))
            s = (xs[r] - xs[r].max()) / t
            others = np.exp(np.delete(s, place[r])).sum()
            want = np.log1p(others)
            scale = (tu.LOGSUM_TOL + 3 * tu.U * (tops[r % len(tops)] + np.log(V)) / t + 4 * tu.U) * others
            assert abs(float(out[6][r]) - want) <= scale, (r, temps, float(out[6][r]), want)
            assert abs(float(out[0][r]) + want) <= scale, (r, temps, float(out[0][r]), want)
