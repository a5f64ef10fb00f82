"""The tied-embedding example end to end on the GPU, and its gradients against binary64 products."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g

    g.build()
    from examples import tied_lm

    return tied_lm


def test_train_and_serve(lm):
    losses, legal, lp, rank = lm.main(V=1000, steps=300, n=24, batch=8)
    # the chain's entropy is log 4; a model that knows the successors is close to it, an untrained one at log V
    assert losses[0] > 6.0 and losses[-1] < 1.8
    assert legal > 0.95
    assert torch.isfinite(lp).all() and int(rank.max()) < 20      # top-k 20


def test_gradients(lm):
    """Against autograd in binary64 on the bf16-rounded matrices. Four products with bf16 operands (half a step 2^-8 each,
    the logits and their gradient among them) stand between the loss and the gradients; their errors are independent
    per element, so the gradients' norms agree to a few steps: 4 * 2^-8 with a factor two in hand."""
    chain = lm.Chain(300, seed=3)
    dev = torch.device("cuda:0")
    gen = torch.Generator().manual_seed(5)
    table = (torch.randn((300, 64), generator=gen) * 0.1).to(dev)
    W = (torch.randn((64, 64), generator=gen) * 0.1).to(dev)
    tok, target = chain.batch(512, gen, dev)
    loss, status, grad = lm.gradients(lm.Model(table, W), tok, target, entropy_bonus=0.1)
    t64 = table.bfloat16().double().requires_grad_()
    w64 = W.bfloat16().double().requires_grad_()
    logits = (math.sqrt(64) * t64[tok.long()] @ w64) @ t64.t()
    lps = torch.log_softmax(logits, dim=1)
    keep = target >= 0
    lp = lps[keep, target[keep].long()]
    ent = -(lps.exp() * lps).sum(1)[keep]
    ref = -(lp.sum() + 0.1 * ent.sum()) / keep.sum()
    ref.backward()
    assert (status == 0).all()
    assert abs(float(loss) - ref.item()) <= 2 * 4 * 2.0 ** -8 * abs(ref.item())
    for got, want in ((grad.table, t64.grad), (grad.W, w64.grad)):
        assert float((got.double() - want).norm()) <= 2 * 4 * 2.0 ** -8 * float(want.norm())
