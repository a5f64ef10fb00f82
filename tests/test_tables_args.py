"""Refusals of the vocabulary-side operators, on the CPU: the C entry points answer before any CUDA call, and the
binding refuses what the library cannot take."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from top_sampling_gb300 import build as b

    b.build()
    import top_sampling_gb300 as ts

    return ts.load()


BAD = 1            # VSAMP_ERR_INVALID_ARG
UNSUPPORTED = 2
F32, BF16 = 0, 1
P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)


def _call(fn, good, **change):
    return fn(*{**good, **change}.values())


def test_constants_agree_with_the_header():
    import os
    import re

    import top_sampling_gb300 as ts

    src = open(os.path.join(os.path.dirname(ts.__file__), "..", "include", "vsamp.h")).read()
    assert int(re.search(r"#define VSAMP_TOKEN_IGNORE \((-?\d+)\)", src).group(1)) == ts.VSAMP_TOKEN_IGNORE
    assert int(re.search(r"#define VSAMP_SCORE_ALT_MAX (\d+)", src).group(1)) == ts.VSAMP_SCORE_ALT_MAX


def test_score_refusals(lib):
    assert lib.vsamp_score_workspace_size(7, 4, 100, 0) == 0
    assert lib.vsamp_score_workspace_size(F32, 0, 100, 0) == 0
    assert lib.vsamp_score_workspace_size(F32, 4, 100, -1) == 0
    assert lib.vsamp_score_workspace_size(F32, 4, 100, 129) == 0
    need = lib.vsamp_score_workspace_size(BF16, 4, 5000, 20)
    assert need > 0 and need % 16 == 0
    good = dict(x=P, dt=BF16, B=4, V=5000, ld=5000, T=None, tok=P, N=20, lp=P, ent=P, rank=P, ai=P, al=P, rm=P, rl=P,
                st=P, ws=P, nws=need, s=None)
    for change in (dict(x=None), dict(dt=7), dict(B=0), dict(V=0), dict(ld=4999), dict(tok=None), dict(N=-1),
                   dict(N=129), dict(ai=None), dict(al=None), dict(ws=None), dict(ws=ctypes.c_void_p(4104)),
                   dict(nws=need - 1), dict(x=ODD)):
        assert _call(lib.vsamp_score_tokens, good, **change) == BAD, change
    assert _call(lib.vsamp_score_tokens, good, V=0x7FFFFFF1, ld=0x7FFFFFF1) == UNSUPPORTED


def test_score_backward_refusals(lib):
    good = dict(x=P, dt=F32, B=4, V=50, ld=50, T=None, tok=P, g=P, h=P, rm=P, rl=P, ent=P, d=P, ldd=50, st=None, s=None)
    for change in (dict(x=None), dict(dt=3), dict(B=-1), dict(V=0), dict(ld=49), dict(tok=None), dict(g=None, h=None),
                   dict(ent=None), dict(rm=None), dict(rl=None), dict(d=None), dict(ldd=49), dict(d=ODD)):
        assert _call(lib.vsamp_score_tokens_backward, good, **change) == BAD, change


def test_head_refusals(lib):
    size = lib.vsamp_head_packed_size
    for args in ((5, 0, 100, 128, 32), (BF16, 0, 0, 128, 32), (BF16, 0, 100, 0, 32), (BF16, 0, 100, 100, 32),
                 (BF16, 0, 100, 128, 16), (BF16, 0, 100, 64, 128)):
        assert size(*args) == 0, args
    need = size(BF16, 1, 100, 128, 64)
    # seven tiles of 16 rows, two blocks of 512 bytes each, two groups of 16 scales and 16 zero points; one
    # more record at the end
    assert need == 8 * (2 * 512 + 2 * 16 * 2 + 2 * 16)
    pack = dict(c=P, s=P, sdt=BF16, z=P, V=100, D=128, g=64, out=P, n=need, stream=None)
    for change in (dict(c=None), dict(s=None), dict(out=None), dict(n=need - 1), dict(g=48), dict(D=96), dict(V=0),
                   dict(sdt=9), dict(s=ODD), dict(out=ctypes.c_void_p(4104))):
        assert _call(lib.vsamp_head_pack, pack, **change) == BAD, change
    run = dict(h=P, dt=BF16, M=2, ldh=128, w=P, n=need, sdt=BF16, z=1, V=100, D=128, g=64, y=P, odt=F32, ld=100,
               stream=None)
    for change in (dict(h=None), dict(w=None), dict(y=None), dict(dt=2), dict(odt=2), dict(M=0), dict(ldh=127),
                   dict(ld=99), dict(n=need - 1), dict(g=33), dict(h=ODD), dict(y=ODD)):
        assert _call(lib.vsamp_head_logits, run, **change) == BAD, change


def test_embed_refusals(lib):
    good = dict(t=P, N=3, w=P, dt=F32, V=10, D=8, ldt=8, scale=1.0, y=P, odt=BF16, ldo=8, st=None, s=None)
    for change in (dict(t=None), dict(w=None), dict(y=None), dict(N=0), dict(V=0), dict(D=0), dict(ldt=7), dict(ldo=7),
                   dict(dt=4), dict(odt=4), dict(w=ODD), dict(y=ODD)):
        assert _call(lib.vsamp_embed, good, **change) == BAD, change
    assert _call(lib.vsamp_embed, good, D=1 << 30, ldt=1 << 30, ldo=1 << 30) == UNSUPPORTED
    assert lib.vsamp_embed_workspace_size(0, 8) == 0 and lib.vsamp_embed_workspace_size(8, 0) == 0
    need = lib.vsamp_embed_workspace_size(100, 8)
    good = dict(t=P, N=100, g=P, dt=F32, D=8, ldd=8, scale=1.0, V=10, d=P, odt=F32, ldt=8, acc=0, ws=P, n=need, s=None)
    for change in (dict(t=None), dict(g=None), dict(d=None), dict(N=0), dict(V=0), dict(D=0), dict(ldd=7), dict(ldt=7),
                   dict(dt=4), dict(odt=4), dict(ws=None), dict(ws=ctypes.c_void_p(4100)), dict(n=need - 1),
                   dict(g=ODD), dict(d=ODD)):
        assert _call(lib.vsamp_embed_backward, good, **change) == BAD, change


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    import top_sampling_gb300 as ts

    x, tok = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    one = torch.zeros(2)
    with pytest.raises(ValueError):
        ts.vsamp_score_tokens(x, tok)
    with pytest.raises(ValueError):
        ts.vsamp_score_tokens_backward(x, tok, one, one, one)
    with pytest.raises(ValueError):
        ts.vsamp_embed(tok, x)
    with pytest.raises(ValueError):
        ts.vsamp_embed_backward(tok, x, 4)
    with pytest.raises(ValueError):
        ts.vsamp_head_pack(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1), group=32)


@pytest.mark.gpu
def test_binding_refuses_bad_shapes():
    torch = pytest.importorskip("torch")
    import top_sampling_gb300 as ts

    dev = torch.device("cuda:0")
    x = torch.zeros(2, 64, device=dev)
    tok = torch.zeros(2, dtype=torch.int32, device=dev)
    one = torch.zeros(2, device=dev)
    with pytest.raises(ValueError):
        ts.vsamp_score_tokens(x, tok, n_alt=129)
    with pytest.raises(ValueError):
        ts.vsamp_score_tokens(x[:1], tok, V=65)                    # beyond a single row
    with pytest.raises(ValueError):
        ts.vsamp_score_tokens(x, tok[:1])
    with pytest.raises(TypeError):
        ts.vsamp_score_tokens(x.half(), tok)
    with pytest.raises(TypeError):
        ts.vsamp_score_tokens(x, one)                              # tokens that are not whole numbers
    with pytest.raises(ValueError):
        ts.vsamp_score_tokens(x.t(), tok)
    with pytest.raises(ts.VsampError):
        ts.vsamp_score_tokens(x[:1].expand(2, 64), tok)            # rows that share memory
    with pytest.raises(ValueError):
        ts.vsamp_score_tokens_backward(x, tok, one, one, one, dlogits=torch.zeros(2, 64, device=dev).bfloat16())
    with pytest.raises(ValueError):
        ts.vsamp_score_tokens_backward(x, tok, one, one, one, dlogits=torch.zeros(3, 64, device=dev))
    codes = torch.zeros(4, 32, dtype=torch.uint8, device=dev)
    with pytest.raises(ValueError):
        ts.vsamp_head_pack(codes, torch.zeros(4, 1, device=dev), group=32)
    with pytest.raises(ValueError):
        ts.vsamp_head_pack(codes, torch.zeros(4, 1, device=dev), group=16)
    head = ts.vsamp_head_pack(codes, torch.zeros(4, 2, device=dev), group=32)
    with pytest.raises(ValueError):
        ts.vsamp_head_logits(torch.zeros(1, 65, device=dev), head)
    with pytest.raises(ValueError):
        ts.vsamp_head_logits(torch.zeros(1, 64, device=dev), head, out=torch.zeros(1, 5, device=dev))
    with pytest.raises(ValueError):
        ts.vsamp_embed(tok, x, out=torch.zeros(2, 63, device=dev))
    with pytest.raises(ValueError):
        ts.vsamp_embed_backward(tok, x, 4, accumulate=True)
    with pytest.raises(ValueError):
        ts.vsamp_embed_backward(tok[:1], x, 4)
