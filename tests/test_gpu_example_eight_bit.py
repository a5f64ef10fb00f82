"""Every intermediate of the example's 8-bit gradients against binary64 on the operands that its call had in hand: what is
allowed is the roundings of that one call."""
import math

import pytest

import blocks_util as bu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF16 = 2.0 ** -8
V, D, B = 300, 64, 512


class Calls:
    """The library with copies of what some entry points were given and returned."""

    def __init__(self, ts):
        self.ts, self.made = ts, {}

    def __getattr__(self, name):
        fn = getattr(self.ts, name)
        if not name.startswith("vsamp_"):
            return fn

        def call(*args, **more):
            given = [a.clone() if isinstance(a, torch.Tensor) else a for a in args]
            got = fn(*args, **more)
            kept = tuple(t.clone() if isinstance(t, torch.Tensor) else t for t in (got if isinstance(got, tuple) else (got,)))
            self.made.setdefault(name, []).append((given, kept))
            return got

        return call


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g

    g.build()
    from examples import tied_lm

    return tied_lm


def _values(t):
    s = t.scales.double()
    s = s.repeat_interleave(128, 0)[:t.rows] if t.tile else s.t()
    return t.codes.view(torch.float8_e4m3fn).double() * s.repeat_interleave(128, 1)[:, :t.cols]


def _product(got, a, b, half):
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    assert ((got.double() - want).abs() <= bu.product_tol(size, a.shape[1]) + half * want.abs()).all()


def _library(got, a, b):
    """A bf16 product with sums in 32 bits: a unit per product and sum, and the rounding."""
    a, b = a.double(), b.double()
    want, size = a @ b, a.abs() @ b.abs()
    assert ((got.double() - want).abs() <= 2 * a.shape[1] * bu.U * size + HALF16 * want.abs() * (1 + 2.0 ** -8)).all()


def test_gradients(lm, monkeypatch):
    monkeypatch.setattr(torch.backends.cuda.matmul, "allow_bf16_reduced_precision_reduction", False)
    calls = Calls(lm.ts)
    monkeypatch.setattr(lm, "ts", calls)
    dev = torch.device("cuda:0")
    gen = torch.Generator().manual_seed(5)
    table = (torch.randn((V, D), generator=gen) * 0.1).to(dev)
    W = (torch.randn((D, D), generator=gen) * 0.1).to(dev)
    tok, target = lm.Chain(V, seed=3).batch(B, gen, dev)
    loss, status, grad = lm.gradients(lm.Model(table, W), tok, target, entropy_bonus=0.1, eight_bit=True)
    assert (status == 0).all()
    made = calls.made
    t16, w16 = table.bfloat16(), W.bfloat16()

    h = made["vsamp_embed"][0][1][0]
    want = t16.double()[tok.long()] * math.sqrt(D)
    assert ((h.double() - want).abs() <= (HALF16 + 2 * bu.U) * want.abs()).all()
    ((x, *_), (t8, t8t)), ((z, *_), (z8, z8t)), ((d, *_), (d8, d8t)) = made["vsamp_block_quantize"]
    assert torch.equal(x, table)
    _library(z, h, w16)
    for q, turned, t in ((t8, t8t, table), (z8, z8t, z), (d8, d8t, d)):
        # half a code's step of the element, or of the block's least ones
        for v, u in ((_values(q), t.double()), (_values(turned), t.double().t())):
            assert ((v - u).abs() <= u.abs() * (2.0 ** -4 + 4 * bu.U) + u.abs().max() * 2.0 ** -18).all()

    logits, dz, dtable = (got for _, (got,) in made["vsamp_block_matmul"])
    _product(logits, _values(z8), _values(t8), HALF16)
    x64 = logits.double()
    lp = torch.log_softmax(x64, dim=1)
    p, keep = lp.exp(), target >= 0
    assert 0 < int(keep.sum()) < B or bool(keep.all())
    H = -(p * lp).sum(1)
    at = target.clamp(min=0).long()
    scored = int(keep.sum())
    want = -(lp.gather(1, at[:, None])[:, 0][keep].sum() + 0.1 * H[keep].sum()) / scored
    # V exponentials are summed, each product with a logit is off by that and its own roundings
    tol = (V + 16) * bu.U * (1 + 0.1 * float(lp.abs().max())) + B * bu.U * abs(float(want))
    assert abs(float(loss) - float(want)) <= tol

    one = torch.nn.functional.one_hot(at, V).double()
    want = -(one - p - 0.1 * p * (lp + H[:, None])) / scored
    want[~keep] = 0.0
    size = (one + p + 0.1 * p * (lp.abs() + H[:, None])) / scored
    assert torch.equal(d.double(), made["vsamp_score_tokens_backward"][0][1][0].double())
    assert ((d.double() - want).abs() <= HALF16 * want.abs() * (1 + 2.0 ** -8) + (V + 16) * bu.U * size).all()

    _product(dz, _values(d8), _values(t8t), HALF16)
    _product(dtable, _values(d8t), _values(z8t), bu.U)
    _library(grad.W, h.t(), dz)
    dh = made["vsamp_embed_backward"][0][0][1]
    _library(dh, dz, w16.t())
    lookup, size = (torch.zeros((V, D), dtype=torch.float64, device=dev) for _ in range(2))
    lookup.index_add_(0, tok.long(), dh.double() * math.sqrt(D))
    size.index_add_(0, tok.long(), dh.double().abs() * math.sqrt(D))
    want = dtable.double() + lookup
    most = int(torch.bincount(tok.long()).max())
    assert ((grad.table.double() - want).abs() <= (most + 4) * bu.U * (size + dtable.double().abs())).all()
    # both parts of the table's gradient weigh far more than what is allowed
    assert lookup.norm() > 0.01 * want.norm() and dtable.double().norm() > 0.01 * want.norm()
