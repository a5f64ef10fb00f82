"""Refusals of the 8-bit blocks and of the optimiser step, on the CPU: the C entry points answer before any CUDA call."""
import ctypes

import pytest

BAD, UNSUPPORTED = 1, 2
F32, BF16 = 0, 1
ROW, TILE = 0, 1
P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)
HALF_LINE = ctypes.c_void_p(4104)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from top_sampling_gb300 import build as b

    b.build()
    import top_sampling_gb300 as ts

    return ts.load()


def _call(fn, good, **change):
    return fn(*{**good, **change}.values())


def test_constants_agree_with_the_header():
    import os
    import re

    import top_sampling_gb300 as ts

    src = open(os.path.join(os.path.dirname(ts.__file__), "..", "include", "vsamp.h")).read()
    for name in ("VSAMP_BLOCK_ROW", "VSAMP_BLOCK_TILE"):
        assert int(re.search(name + r" = (\d)", src).group(1)) == getattr(ts, name)


def test_quantize_refusals(lib):
    good = dict(x=P, dt=BF16, R=100, C=300, ldx=300, kind=ROW, c=P, ldc=304, s=P, lds=100, ct=P, ldt=112, st=P, ldst=300,
                stream=None)
    for change in (dict(x=None), dict(x=ODD), dict(dt=2), dict(kind=2), dict(R=0), dict(C=0), dict(C=-1), dict(ldx=299),
                   dict(c=None), dict(s=None), dict(ct=None), dict(st=None), dict(c=None, s=None, ct=None, st=None),
                   dict(ldc=300), dict(ldc=288), dict(c=HALF_LINE), dict(s=HALF_LINE), dict(lds=96), dict(lds=102),
                   dict(ldt=96), dict(ldt=104), dict(ct=HALF_LINE), dict(ldst=296), dict(st=HALF_LINE)):
        assert _call(lib.vsamp_block_quantize, good, **change) == BAD, change
    tile = {**good, "kind": TILE, "lds": 3, "ldst": 1}
    for change in (dict(lds=2), dict(ldst=0), dict(s=ODD)):
        assert _call(lib.vsamp_block_quantize, tile, **change) == BAD, change
    big = 0x7FFFFF01
    assert _call(lib.vsamp_block_quantize, good, R=big, ct=None, st=None, lds=big + 3) == UNSUPPORTED


def test_matmul_refusals(lib):
    good = dict(a=P, lda=304, sa=P, ldsa=8, b=P, ldb=304, sb=P, ldsb=3, kind=TILE, M=5, N=100, K=300, out=P, odt=BF16, ldo=100,
                acc=0, ws=None, nws=0, stream=None)
    for change in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None), dict(kind=5), dict(odt=9),
                   dict(M=0), dict(N=0), dict(K=0), dict(K=305), dict(lda=300), dict(ldb=296), dict(a=HALF_LINE),
                   dict(b=HALF_LINE), dict(sa=HALF_LINE), dict(ldsa=4), dict(ldsa=6), dict(ldsb=2), dict(sb=ODD),
                   dict(out=ODD), dict(ldo=99), dict(kind=ROW), dict(kind=ROW, ldsb=100, sb=HALF_LINE)):
        assert _call(lib.vsamp_block_matmul, good, **change) == BAD, change
    big = 0x7FFFFF01
    assert _call(lib.vsamp_block_matmul, good, N=big, ldo=big) == UNSUPPORTED
    assert lib.vsamp_block_matmul_workspace_size(0, 5, 5) == 0


def test_matmul_workspace(lib):
    """What needs a workspace says so and refuses to go without."""
    size = lib.vsamp_block_matmul_workspace_size
    assert size(2048, 151936, 4096) == 0
    for M, N, K in ((4, 100, 151936), (64, 4096, 151936), (300, 300, 100000)):
        need = size(M, N, K)
        if not need:
            continue
        up = -(-K // 16) * 16
        good = dict(a=P, lda=up, sa=P, ldsa=300, b=P, ldb=up, sb=P, ldsb=-(-K // 128), kind=TILE, M=M, N=N, K=K, out=P, odt=BF16,
                    ldo=N, acc=0, ws=P, nws=need, stream=None)
        for change in (dict(ws=None), dict(nws=need - 1), dict(ws=HALF_LINE)):
            assert _call(lib.vsamp_block_matmul, good, **change) == BAD, change


def test_adamw_refusals(lib):
    import top_sampling_gb300 as ts

    def call(tensor=(), count=1, pdt=F32, gdt=F32, bits=32, tensors=None, rule=None, **change):
        words = dict(param=4096, master=0, grad=8192, m=16384, v=32768, ms=0, vs=0, n=100, index=0)
        words.update(tensor)
        table = (ctypes.c_int64 * 9)(*words.values())
        args = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, seed=0)
        args.update(change)
        r = ts.vsamp_adamw_rule(**args)
        return lib.vsamp_adamw(None if tensors == 0 else ctypes.addressof(table), count, pdt, gdt, bits,
                               None if rule == 0 else ctypes.addressof(r), None)

    assert call(tensor=dict(n=0)) == 0                                    # nothing to do
    for change in (dict(tensors=0), dict(rule=0), dict(count=0), dict(count=-1), dict(pdt=2), dict(gdt=2), dict(bits=16),
                   dict(bits=8), dict(lr=NAN), dict(lr=-1.0), dict(lr=INF), dict(beta1=1.0), dict(beta1=-0.1),
                   dict(beta2=1.0), dict(beta2=NAN), dict(eps=-1.0), dict(eps=INF), dict(weight_decay=-1.0),
                   dict(weight_decay=NAN), dict(step=0), dict(step=-5), dict(lr_dev=4098), dict(step_dev=4100),
                   dict(grad_scale=4097)):
        assert call(**change) == BAD, change
    for change in (dict(eps=2.0 ** -127), dict(eps=1e-300), dict(eps=1e39), dict(lr=1e39), dict(weight_decay=1e39)):
        assert call(**change) == BAD, change                              # not as fp32 numbers
    for change in (dict(eps=0.0), dict(eps=2.0 ** -126)):
        assert call(tensor=dict(n=0), **change) == 0, change
    for tensor in (dict(n=-1), dict(param=0), dict(grad=0), dict(m=0), dict(v=0), dict(param=4098), dict(grad=8193),
                   dict(m=16386), dict(v=32769), dict(master=65536), dict(master=65538)):
        assert call(tensor=tensor) == BAD, tensor
    assert call(tensor=dict(n=(1 << 34) + 1)) == UNSUPPORTED
    good = dict(ms=65536, vs=131072)
    for tensor in (dict(ms=0), dict(vs=0), dict(ms=65538), dict(vs=131073)):
        assert call(tensor={**good, **tensor}, bits=8) == BAD, tensor


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    import top_sampling_gb300 as ts

    x = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        ts.vsamp_block_quantize(x)
    with pytest.raises(ValueError):
        ts.BlockTensor(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4))
    with pytest.raises(TypeError):
        ts.BlockTensor(x, torch.zeros(1, 4))
    with pytest.raises(ValueError):
        ts.vsamp_adamw_state([x])
    with pytest.raises(ValueError):
        ts.vsamp_adamw_state([])
    with pytest.raises(ValueError):
        ts.vsamp_adamw_state([x], bits=16)
