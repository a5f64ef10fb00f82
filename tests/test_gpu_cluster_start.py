"""Kernels whose CTAs write into the first CTA of their cluster right after they begin: short rows on many CTAs, one call
close behind another, every call the same."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CALLS = 50


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


def _bits(outs):
    return [o.view(torch.int32) for o in outs if o is not None]


@pytest.mark.parametrize("dtype,piece", [(torch.float32, 1024), (torch.bfloat16, 2048)])
@pytest.mark.parametrize("tail", [0, 3])
def test_statistics_of_short_rows(ts, dev, monkeypatch, dtype, piece, tail):
    """A CTA per piece, pieces of a few elements and whole ones, against one CTA per row."""
    B, V = 600, 7 * piece + tail
    x = torch.randn((B, V), device=dev).to(dtype)
    tok = torch.randint(0, V, (B,), device=dev, dtype=torch.int32)

    def both():
        return _bits(ts.vsamp_softmax_lse(x)) + _bits(ts.vsamp_logprob(x, tok))

    monkeypatch.setenv("VSAMP_STATS_C", "1")
    alone = both()
    monkeypatch.setenv("VSAMP_STATS_C", "8")
    for out in [both() for _ in range(CALLS)]:
        assert all(torch.equal(p, q) for p, q in zip(out, alone))


@pytest.mark.parametrize("dtype,piece", [(torch.float32, 1024), (torch.bfloat16, 2048)])
def test_streaming_sampler_of_short_rows(ts, dev, monkeypatch, dtype, piece):
    """Records and draw codes of short rows, against the sampler that keeps them in a workspace."""
    B, V = 300, 7 * piece + 3
    x = torch.randn((B, V), device=dev).to(dtype)
    seed = torch.arange(B, device=dev)
    kw = dict(temperature=0.9, top_k=50, seed=seed, step=3, want_stats=True)
    want = _bits(ts.vsamp_sample_ws(x, **kw))
    monkeypatch.setenv("VSAMP_SAMPLE_STREAM", "1")
    monkeypatch.setenv("VSAMP_SSTREAM_C", "8")
    for out in [_bits(ts.vsamp_sample(x, **kw)) for _ in range(CALLS)]:
        assert all(torch.equal(p, q) for p, q in zip(out, want))
