"""A wait of the block product that runs out, made without a fault: copies are expected and never issued
(`VSAMP_TEST_DROP_LOADS`), every wait ends at its bound (`VSAMP_WAIT_CYCLES`). The results are NaN, and the context and the
next call are sound. Single CTAs and pairs, with and without a division of the inner dimension. In a child process, as the
other tests of waits."""
import json
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent("""
    import json, os, torch
    import top_sampling_gb300 as ts
    dev = torch.device("cuda:0")
    out = []
    for M, N, K in ((5, 300, 400), (300, 500, 400), (5, 300, 40000), (2100, 5000, 300)):
        for tile in (True, False):
            w, _ = ts.vsamp_block_quantize(torch.randn(N, K, device=dev), tile=tile)
            a, _ = ts.vsamp_block_quantize(torch.randn(M, K, device=dev))
            torch.cuda.synchronize()
            os.environ["VSAMP_TEST_DROP_LOADS"] = "1"
            os.environ["VSAMP_WAIT_CYCLES"] = "2000000"
            y = ts.vsamp_block_matmul(a, w, out_dtype=torch.float32)
            torch.cuda.synchronize()
            del os.environ["VSAMP_TEST_DROP_LOADS"]
            del os.environ["VSAMP_WAIT_CYCLES"]
            nan = bool(torch.isnan(y).all())
            z = ts.vsamp_block_matmul(a, w, out_dtype=torch.float32).double()
            want = a.dequantize().double() @ w.dequantize().double().t()
            out.append([nan, float((z - want).norm() / want.norm())])
    print(json.dumps(out))
""")


@pytest.mark.gpu
def test_wait_that_runs_out_gives_nan_and_the_context_survives():
    env = {k: v for k, v in os.environ.items() if k not in ("VSAMP_TEST_DROP_LOADS", "VSAMP_WAIT_CYCLES")}
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    for nan, off in json.loads(r.stdout.strip().splitlines()[-1]):
        assert nan and off < 1e-5
