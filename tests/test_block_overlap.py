"""Memory that a call of the 8-bit blocks would write while it, or another output, lies there: refused on the host, before any
CUDA call. Addresses are numbers here; nothing is behind them."""
import ctypes

import pytest

BAD = 1
F32, BF16 = 0, 1
ROW, TILE = 0, 1


@pytest.fixture(scope="module")
def lib():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("addresses of nothing stay away from a device")
    from top_sampling_gb300 import build as b

    b.build()
    import top_sampling_gb300 as ts

    return ts.load()


def _at(a):
    return None if a is None else ctypes.c_void_p(a)


# x [100, 300] bf16 at 1 MB, 600-byte rows; codes [100, 304], scales [3, 100]; codes_t [300, 112], scales_t [1, 300]
GOOD = dict(x=1 << 20, dt=BF16, R=100, C=300, ldx=300, kind=ROW, c=2 << 20, ldc=304, s=3 << 20, lds=100, ct=4 << 20, ldt=112,
            st=5 << 20, ldst=300, stream=None)


def _quantize(lib, **change):
    v = {**GOOD, **change}
    for k in ("x", "c", "s", "ct", "st"):
        v[k] = _at(v[k])
    return lib.vsamp_block_quantize(*v.values())


@pytest.mark.parametrize("change", [
    dict(c=(1 << 20) + 16),                               # codes in x
    dict(c=(1 << 20) - 99 * 304 - 288),                   # their last row reaches into x
    dict(s=(1 << 20) + 59984),                            # scales begin in x's last row
    dict(ct=(1 << 20) - 16), dict(st=1 << 20),
    dict(ct=(2 << 20) + 304 * 50),                        # codes_t in codes, at another stride
    dict(ct=(2 << 20) - 16 * 7), dict(s=(2 << 20) + 96), dict(s=(2 << 20) + 99 * 304 + 288),
    dict(st=(3 << 20) + 1184), dict(st=(4 << 20) + 299 * 112 + 96), dict(s=(4 << 20) + 16),
    dict(R=300, ct=(2 << 20) + 304 - 16, ldc=608, ldt=608, lds=300),   # the same stride, columns that meet
])
def test_quantize(lib, change):
    assert _quantize(lib, **change) == BAD, change


def test_quantize_refuses_one_direction_too(lib):
    assert _quantize(lib, ct=None, st=None, c=(1 << 20) + 1600) == BAD
    assert _quantize(lib, c=None, s=None, ct=(1 << 20) + 1600) == BAD
    assert _quantize(lib, kind=TILE, lds=3, ldst=1, st=(3 << 20) + 8) == BAD


# a [5, 300] in 304, scales [3, 8]; b [100, 300] in 304, scales [1, 3]; out [5, 100] bf16
PRODUCT = dict(a=1 << 20, lda=304, sa=2 << 20, ldsa=8, b=3 << 20, ldb=304, sb=4 << 20, ldsb=3, kind=TILE, M=5, N=100, K=300,
               out=5 << 20, odt=BF16, ldo=100, acc=0, ws=None, nws=0, stream=None)


def _product(lib, **change):
    v = {**PRODUCT, **change}
    for k in ("a", "sa", "b", "sb", "out", "ws"):
        v[k] = _at(v[k])
    return lib.vsamp_block_matmul(*v.values())


@pytest.mark.parametrize("change", [
    dict(out=1 << 20), dict(out=(1 << 20) + 4 * 304 + 298), dict(out=(2 << 20) + 80), dict(out=(3 << 20) - 998),
    dict(out=(3 << 20) + 99 * 304), dict(out=(4 << 20) + 8), dict(out=(4 << 20) - 998),
])
def test_matmul(lib, change):
    assert _product(lib, **change) == BAD, change


def test_matmul_workspace(lib):
    M, N, K = 64, 4096, 151936
    need = lib.vsamp_block_matmul_workspace_size(M, N, K)
    assert need > 0
    big = dict(a=1 << 30, sa=2 << 30, b=3 << 30, sb=4 << 30, out=5 << 30, lda=K, ldb=K, ldsa=M, ldsb=1187, M=M, N=N, K=K, ldo=N,
               nws=need)
    for at in ((1 << 30) + 16, (2 << 30) + 16, (3 << 30) - 16, (4 << 30) + 1600, (5 << 30) + 4096, (5 << 30) - need + 16):
        assert _product(lib, **big, ws=at) == BAD, at
