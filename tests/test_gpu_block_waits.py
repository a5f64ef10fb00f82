"""Waits of the block product that run out with copies made and products under way: the copying warps of a pair's two CTAs end
after different numbers of blocks (`VSAMP_TEST_STOP_LOADS_0`, `_1`), or all waits are short (`VSAMP_WAIT_CYCLES`). Every
result is right or NaN, and the context and the next call are sound. In a child process, as the other tests of waits."""
import json
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ("VSAMP_TEST_STOP_LOADS_0", "VSAMP_TEST_STOP_LOADS_1", "VSAMP_TEST_DROP_LOADS", "VSAMP_WAIT_CYCLES")

CHILD = textwrap.dedent("""
    import json, os, sys, torch
    sys.path.insert(0, "tests")
    import blocks_util as bu
    import top_sampling_gb300 as ts
    dev = torch.device("cuda:0")
    M, N, K, tile, runs = json.loads(sys.argv[1])
    w, _ = ts.vsamp_block_quantize(torch.randn(N, K, device=dev), tile=tile)
    a, _ = ts.vsamp_block_quantize(torch.randn(M, K, device=dev))
    x, y = a.dequantize().double(), w.dequantize().double()
    prod, size = x @ y.t(), x.abs() @ y.abs().t()
    out = []
    for run in runs:
        for dt, add in ((torch.float32, False), (torch.float32, True), (torch.bfloat16, True)):
            base = torch.randn(M, N, device=dev).to(dt)
            z = base.clone()
            torch.cuda.synchronize()
            os.environ.update(run)
            ts.vsamp_block_matmul(a, w, out=z, accumulate=add)
            torch.cuda.synchronize()
            for name in run:
                del os.environ[name]
            want = prod + base.double() if add else prod
            tol = bu.product_tol(size + base.double().abs(), K) + bu.HALF[dt] * want.abs()
            nan = torch.isnan(z)
            wrong = int((~nan & ((z.double() - want).abs() > tol)).sum())
            after = ts.vsamp_block_matmul(a, w, out_dtype=torch.float32)
            off = (after.double() - prod).abs() > bu.product_tol(size, K) + bu.U * prod.abs()
            out.append([wrong, int(nan.sum()), M * N, int(off.sum())])
    print(json.dumps(out))
""")


def _run(M, N, K, tile, runs):
    env = {k: v for k, v in os.environ.items() if k not in NAMES}
    r = subprocess.run([sys.executable, "-c", CHILD, json.dumps([M, N, K, tile, runs])], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


def _stop(n0, n1):
    run = {"VSAMP_WAIT_CYCLES": "2000000"}
    if n0:
        run["VSAMP_TEST_STOP_LOADS_0"] = str(n0)
    if n1:
        run["VSAMP_TEST_STOP_LOADS_1"] = str(n1)
    return run


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [True, False])
# 2100 x 5000: 180 tiles of three blocks for 76 pairs; 300 x 500: four tiles of 32 blocks, divided
@pytest.mark.parametrize("M,N,K,stops,some", [(2100, 5000, 300, [(3, 3), (4, 6), (6, 4), (5, 0), (0, 4)], True),
                                              (300, 500, 4000, [(1, 3), (3, 1), (0, 2), (2, 0)], False)])
def test_pairs_that_end_apart(tile, M, N, K, stops, some):
    for wrong, nan, total, after in _run(M, N, K, tile, [_stop(*s) for s in stops]):
        assert wrong == 0 and after == 0 and 0 < nan <= total
        assert not some or nan < total     # the first tiles were finished


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [True, False])
def test_single_ctas(tile):
    for wrong, nan, total, after in _run(100, 50000, 300, tile, [_stop(n, 0) for n in (3, 4, 5)]):
        assert wrong == 0 and after == 0 and 0 < nan < total

@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(2100, 5000, 300), (100, 50000, 300), (600, 1000, 20000)])
def test_short_waits(M, N, K):
    """Waits of a cycle and more, none of whose copies is left out: whoever gives up leaves nothing wrong."""
    for wrong, _, _, after in _run(M, N, K, True, [{"VSAMP_WAIT_CYCLES": str(c)} for c in (1, 500, 2000, 8000)]):
        assert wrong == 0 and after == 0


@pytest.mark.gpu
def test_pairs_between_other_kernels():
    """Pairs' products one behind the other and between kernels that leave something else in shared memory: no CTA takes what
    was there for the other one's word that it gave up."""
    torch = pytest.importorskip("torch")
    import __graft_entry__ as g

    g.build()
    import top_sampling_gb300 as ts

    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(1)
    p, q = (torch.randn((4096, 4096), generator=gen, device=dev) for _ in range(2))
    a, _ = ts.vsamp_block_quantize(torch.randn((20000, 1024), generator=gen, device=dev))
    for tile in (True, False):
        b, _ = ts.vsamp_block_quantize(torch.randn((2048, 1024), generator=gen, device=dev), tile=tile)
        ref = ts.vsamp_block_matmul(a, b, out_dtype=torch.float32)
        for k in range(40):
            p @ q if k % 2 else p.bfloat16() @ q.bfloat16()
            outs = [ts.vsamp_block_matmul(a, b, out_dtype=torch.float32) for _ in range(3)]
            assert all(torch.equal(y, ref) for y in outs)
