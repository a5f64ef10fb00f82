"""What an AdamW step says about parameters that it leaves alone, and what it checks when it changes nothing."""
import pytest

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


def _parameters(dev):
    return [torch.nn.Parameter(torch.ones(8, device=dev)), torch.nn.Parameter(torch.ones(8, device=dev).bfloat16())]


@pytest.mark.parametrize("given", [(True, False), (False, True), (False, False)])
def test_a_group_without_gradients_stays_unmarked(ts, given):
    """Parameters of two types, a group each: a backward pass through those without a gradient goes on as before the step."""
    dev = torch.device("cuda:0")
    params = _parameters(dev)
    state = ts.vsamp_adamw_state(params)
    x = torch.ones(8, device=dev, requires_grad=True)
    outs = [(x * p).sum() for p in params]
    before = [p.detach().clone() for p in params]
    ts.vsamp_adamw(state, [torch.ones(8, device=dev) if g else None for g in given], lr=0.1, step=1)
    for y, p, old, g in zip(outs, params, before, given):
        assert torch.equal(p.detach(), old) != g
        if g:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.backward()
        else:
            y.backward()


def test_the_rule_is_checked_without_any_gradient(ts):
    state = ts.vsamp_adamw_state(_parameters(torch.device("cuda:0")))
    ts.vsamp_adamw(state, [None, None], lr=0.1, step=1)
    for bad in (dict(step=0), dict(lr=float("nan")), dict(lr=-1.0), dict(beta1=1.0), dict(eps=1e-300)):
        with pytest.raises(ts.VsampError):
            ts.vsamp_adamw(state, [None, None], **{**dict(lr=0.1, step=1), **bad})
