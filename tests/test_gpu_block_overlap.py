"""Outputs of the 8-bit blocks in shared buffers: what meets is refused and left as it is, what lies side by side works."""
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


def _u8(t):
    return t.codes.view(torch.uint8)


def test_what_meets_is_refused(ts):
    dev = torch.device("cuda:0")
    x = torch.randn(128, 128, device=dev)
    room = torch.full((40000,), 0x55, dtype=torch.uint8, device=dev)
    scales = [torch.zeros((1, 128), device=dev) for _ in range(2)]

    def codes(at):
        return room[at:at + 128 * 128].view(128, 128)

    one, other = ts.BlockTensor(codes(0), scales[0]), ts.BlockTensor(codes(128 * 100), scales[1])
    with pytest.raises((ValueError, ts.VsampError)):
        ts.vsamp_block_quantize(x, transposed=True, out=one, out_t=other)
    with pytest.raises((ValueError, ts.VsampError)):     # scales in the codes
        ts.vsamp_block_quantize(x, out=ts.BlockTensor(codes(0), room[1024:1536].view(torch.float32).view(1, 128)))
    with pytest.raises((ValueError, ts.VsampError)):     # codes in x
        ts.vsamp_block_quantize(x, out=ts.BlockTensor(x.view(torch.uint8)[:, 128:256], scales[0]))
    assert (room == 0x55).all()
    a, _ = ts.vsamp_block_quantize(x)
    with pytest.raises((ValueError, ts.VsampError)):     # a product over its own operand
        ts.vsamp_block_matmul(a, ts.vsamp_block_quantize(x[:32])[0], out=_u8(a).view(torch.float32))


def test_side_by_side(ts):
    """Both directions' codes as column ranges of one buffer, their scales as parts of another."""
    dev = torch.device("cuda:0")
    x = torch.randn(128, 128, device=dev)
    room, plane = torch.zeros((128, 256), dtype=torch.uint8, device=dev), torch.zeros((2, 128), device=dev)
    a = ts.BlockTensor(room[:, :128], plane[:1])
    b = ts.BlockTensor(room[:, 128:], plane[1:])
    ts.vsamp_block_quantize(x, transposed=True, out=a, out_t=b)
    want, want_t = ts.vsamp_block_quantize(x, transposed=True)
    for got, ref in ((a, want), (b, want_t)):
        assert torch.equal(_u8(got), _u8(ref)) and torch.equal(got.scales, ref.scales)
    y = torch.zeros((128, 300), device=dev)
    for at in (0, 128):                                   # results as column ranges of one array
        ts.vsamp_block_matmul(a, b, out=y[:, at:at + 128])
    ref = ts.vsamp_block_matmul(a, b, out_dtype=torch.float32)
    assert torch.equal(y[:, :128], ref) and torch.equal(y[:, 128:256], ref) and not y[:, 256:].any()
