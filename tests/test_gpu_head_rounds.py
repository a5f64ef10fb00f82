"""The 4-bit head where a block takes more than one round over its row tiles: records fetched across the ends of tiles, the
ring used again, a ragged last round, hidden states staged in parts on every round. Against binary64 on the GPU."""
import pytest

import tables_util as tu
from test_gpu_head import _weights, dev, ts  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

WARPS = 16   # most warps of a block: more sets of row tiles than that per SM make a second round


def _exact(hidden, w, group):
    """Logits in 64 bits and the sum of the products' magnitudes."""
    codes, scales, zeros = w
    V, D = scales.shape[0], codes.shape[1] * 2
    q = torch.stack([codes & 15, codes >> 4], dim=2).view(V, D // group, group).double()
    z = 8.0 if zeros is None else zeros.double()[:, :, None]
    m = ((q - z) * scales.double()[:, :, None]).view(V, D)
    h = hidden.double()
    return h @ m.t(), h.abs() @ m.abs().t()


@pytest.mark.parametrize("V,D,group,M,hdt,rows_of_tiles", [
    (160007, 256, 128, 1, torch.bfloat16, 4),
    (330007, 128, 64, 3, torch.bfloat16, 4),
    (100003, 128, 32, 24, torch.bfloat16, 2),
    (100003, 256, 64, 16, torch.bfloat16, 2),
    (90011, 256, 64, 32, torch.bfloat16, 2),
    (60007, 256, 128, 40, torch.bfloat16, 1),
    (60007, 128, 32, 64, torch.bfloat16, 1),
    (100003, 256, 64, 8, torch.float32, 2),
    (60007, 384, 128, 16, torch.float32, 1),
    (45007, 2048 + 32, 32, 64, torch.bfloat16, 1),       # hidden states in parts, several rounds
    (45007, 4096, 128, 16, torch.float32, 1),
])
@pytest.mark.parametrize("zeros", [False, True])
def test_several_rounds(ts, dev, V, D, group, M, hdt, rows_of_tiles, zeros):
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    tiles = (V + 15) // 16
    assert -(-tiles // rows_of_tiles) > sms * WARPS
    sdt = torch.bfloat16 if zeros else torch.float32
    w = _weights(V, D, group, sdt, zeros, dev, V + M)
    g = torch.Generator(device=dev).manual_seed(M)
    h = torch.randn((M, D), generator=g, device=dev).to(hdt)
    head = ts.vsamp_head_pack(w[0], w[1], zeros=w[2], group=group)
    y = ts.vsamp_head_logits(h, head, out_dtype=torch.float32)
    want, size = _exact(h, w, group)
    tol = tu.head_tol(size, group, D // group, 3 if hdt == torch.float32 else 1) + tu.U * want.abs()
    assert bool(((y.double() - want).abs() <= tol).all())
    # ragged rows of the output, and the same bits whatever the rounds left in the ring
    out = torch.full((M, V + 1), 7.0, device=dev)
    ts.vsamp_head_logits(h, head, out=out[:, :V])
    assert torch.equal(out[:, :V], y) and bool((out[:, V] == 7.0).all())
