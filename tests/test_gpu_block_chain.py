"""The 8-bit operators as a training step runs them: quantisation, logits, scores, their gradient, both products of the
backward pass, the optimiser's step; eager and captured. And the example on them."""
import math

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


class Step:
    """One training step of an 8-bit head on fixed buffers."""

    def __init__(self, ts, B, V, D, bits, dev):
        gen = torch.Generator(device=dev).manual_seed(3)
        self.ts, self.V = ts, V
        self.x = torch.randn((B, D), generator=gen, device=dev).to(BF16)
        self.w = torch.randn((V, D), generator=gen, device=dev) * D ** -0.5
        self.token = torch.randint(0, V, (B,), generator=gen, device=dev).to(torch.int32)
        self.token[::5] = ts.VSAMP_TOKEN_IGNORE
        self.g = torch.full((B,), -1.0 / B, device=dev)
        self.dw = torch.zeros((V, D), device=dev)
        self.count = torch.zeros(1, dtype=torch.int64, device=dev)
        self.state = ts.vsamp_adamw_state([self.w], bits=bits)

    def __call__(self):
        ts = self.ts
        self.count += 1
        self.w8, self.w8t = ts.vsamp_block_quantize(self.w, tile=True, transposed=True)
        self.x8, self.x8t = ts.vsamp_block_quantize(self.x, transposed=True)
        self.logits = ts.vsamp_block_matmul(self.x8, self.w8, out_dtype=F32)
        lp, ent, rank, _, _, m, logsum, self.status = ts.vsamp_score_tokens(self.logits, self.token)
        self.lp = lp
        self.dlogits, _ = ts.vsamp_score_tokens_backward(self.logits, self.token, self.g, m, logsum)
        self.d8, self.d8t = ts.vsamp_block_quantize(self.dlogits, transposed=True)
        self.dx = ts.vsamp_block_matmul(self.d8, self.w8t, out_dtype=F32)
        self.dw.zero_()
        ts.vsamp_block_matmul(self.d8t, self.x8t, out=self.dw, accumulate=True)
        ts.vsamp_adamw(self.state, [self.dw], lr=1e-3, step=self.count, beta2=0.99)


def _values(t):
    """binary64 values of a BlockTensor."""
    return bu.f64(t.codes.view(torch.float8_e4m3fn).float()) * (
        np.repeat(np.repeat(bu.f64(t.scales), 128, 0)[:t.rows], 128, 1)[:, :t.cols] if t.tile
        else np.repeat(bu.f64(t.scales).T, 128, 1)[:, :t.cols])


def _near(got, a, b):
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    assert np.all(np.abs(bu.f64(got) - want) <= bu.product_tol(size, a.shape[1]) + bu.U * np.abs(want))


@pytest.mark.parametrize("B,V,D,bits", [(40, 1000, 200, 32), (300, 777, 384, 8)])
def test_training_step(ts, B, V, D, bits):
    dev = torch.device("cuda:0")
    one = Step(ts, B, V, D, bits, dev)
    before = one.w.clone()
    one()
    assert (one.status == 0).all()
    w8, x8, d8 = _values(one.w8), _values(one.x8), _values(one.d8)
    assert np.array_equal(_values(one.w8t), w8.T)
    _near(one.logits, x8, w8)
    _near(one.dx, d8, w8.T)
    _near(one.dw, _values(one.d8t), _values(one.x8t))
    # the quantised operands are those of the step: half a code's step off at most
    for q, t in ((x8, one.x), (w8, before), (d8, one.dlogits)):
        t = bu.f64(t)
        assert np.all(np.abs(q - t) <= np.abs(t) * (2.0 ** -4 + 4 * bu.U) + np.abs(t).max() * 2.0 ** -18)
    # first step: every weight moves by lr against its gradient
    g = bu.f64(one.dw)
    want = bu.f64(before) - 1e-3 * g / (np.abs(g) + 1e-8)
    assert np.all(np.abs(bu.f64(one.w) - want) <= 64 * bu.U * (np.abs(want) + 1e-3))

    # captured, the same steps from the same start
    two = Step(ts, B, V, D, bits, dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        two()
    for _ in range(3):
        graph.replay()
    one()
    one()
    assert int(two.count) == 3 and torch.equal(one.w, two.w) and torch.equal(one.lp, two.lp)
    assert torch.equal(one.state.m[0].view(torch.uint8), two.state.m[0].view(torch.uint8))


@pytest.fixture(scope="module")
def lm(ts):
    from examples import tied_lm

    return tied_lm


def test_example_runs(lm):
    losses, legal, lp, rank = lm.main(V=500, steps=20, n=8, batch=4, eight_bit=True)
    assert len(losses) == 20 and all(math.isfinite(v) for v in losses)
    assert torch.isfinite(lp).all() and int(rank.max()) < 20


def test_example_gradients(lm):
    """Against autograd in binary64. Three products stand between the loss and the gradients, each with two operands that
    are off by at most 2^-4 of an element (the logits and their gradient among them, in bf16 besides); errors are independent
    per element, so the norms agree to the six operands' roundings."""
    chain = lm.Chain(300, seed=3)
    dev = torch.device("cuda:0")
    gen = torch.Generator().manual_seed(5)
    table = (torch.randn((300, 64), generator=gen) * 0.1).to(dev)
    W = (torch.randn((64, 64), generator=gen) * 0.1).to(dev)
    tok, target = chain.batch(512, gen, dev)
    loss, status, grad = lm.gradients(lm.Model(table, W), tok, target, entropy_bonus=0.1, eight_bit=True)
    t64, w64 = table.double().requires_grad_(), W.double().requires_grad_()
    logits = (math.sqrt(64) * t64[tok.long()] @ w64) @ t64.t()
    lps = torch.log_softmax(logits, dim=1)
    keep = target >= 0
    ent = -(lps.exp() * lps).sum(1)[keep]
    ref = -(lps[keep, target[keep].long()].sum() + 0.1 * ent.sum()) / keep.sum()
    ref.backward()
    assert (status == 0).all()
    assert abs(float(loss) - ref.item()) <= 2 * 2.0 ** -4 * abs(ref.item())
    for got, want in ((grad.table, t64.grad), (grad.W, w64.grad)):
        assert float((got.double() - want).norm()) <= 6 * 2.0 ** -4 * float(want.norm())
