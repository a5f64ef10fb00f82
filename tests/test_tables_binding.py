"""What the binding of the vocabulary-side operators takes, refuses and keeps."""
import pytest

torch = pytest.importorskip("torch")

import top_sampling_gb300 as ts  # noqa: E402


def test_rows_of_alternatives():
    flat = torch.zeros(12)
    assert ts._alternatives(flat, 3, "alt_lp") is flat
    assert ts._alternatives(flat.view(4, 3), 3, "alt_lp").shape == (4, 3)
    for shape in ((3, 4), (2, 6)):
        with pytest.raises(ValueError):
            ts._alternatives(flat.view(shape), 3, "alt_lp")


@pytest.mark.gpu
def test_wider_arrays_of_alternatives_are_refused():
    dev = torch.device("cuda:0")
    x, tok = torch.randn(3, 100, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    idx, lp = torch.zeros(3, 64, dtype=torch.int32, device=dev), torch.zeros(3, 64, device=dev)
    with pytest.raises(ValueError):
        ts.vsamp_score_tokens(x, tok, n_alt=20, alt_idx=idx)
    with pytest.raises(ValueError):
        ts.vsamp_score_tokens(x, tok, n_alt=20, alt_lp=lp)
    # more rows than the batch are fine
    out = ts.vsamp_score_tokens(x[:2], tok[:2], n_alt=64, alt_idx=idx, alt_lp=lp)
    assert out[3] is idx and not idx[2].any()


def test_token_ids_outside_32_bits_stay_outside_every_vocabulary():
    cpu = torch.device("cpu")
    low, high = -(1 << 31), (1 << 31) - 1
    far = torch.tensor([1 << 40, -(1 << 40), (1 << 32) - 100, 5])
    assert ts._token_ids(far, 4, cpu).tolist() == [high, low, high, 5]
    wide = torch.tensor([(1 << 32) - 100, 7], dtype=torch.int64).to(torch.uint32)     # -100 in 32 bits marks ignored tokens
    assert ts._token_ids(wide, 2, cpu).tolist() == [high, 7]
    assert ts._token_ids(1 << 40, 2, cpu).tolist() == [high, high]
    assert ts._token_ids(-(1 << 40), 1, cpu).tolist() == [low]
    for dt in (torch.int8, torch.int16, torch.uint8, torch.int32):
        assert ts._token_ids(torch.tensor([3, 100], dtype=dt), 2, cpu).tolist() == [3, 100]


def test_kept_workspaces_are_few(monkeypatch):
    """A program that goes through many streams does not keep a workspace for each of them."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(ts, "_LOCAL", type(ts._LOCAL)())
    cpu = torch.device("cpu")
    first = ts._scratch(100, cpu, 0, 1)
    assert ts._scratch(60, cpu, 0, 1) is first and ts._scratch(200, cpu, 0, 1).numel() == 200
    for stream in range(2, 100):
        mine = ts._scratch(100, cpu, 0, stream)
        assert ts._scratch(100, cpu, 0, stream) is mine
    kept = ts._LOCAL.__dict__
    assert len(kept) <= ts._SCRATCH_STREAMS and (0, 99) in kept
    assert ts._scratch(ts._SCRATCH_KEPT + 1, cpu, 0, 99).numel() > kept[(0, 99)].numel()
