"""Waits of the block product that run out: barriers of one kind get one arrival too few for every
phase (a hook set on the host), the call ends with GPTQ_ERR_TIMEOUT, and the next one is right."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# The limit is read once per process, so this runs in one of its own: 10 ms instead of seconds.
STALL = """
import os, sys, torch
import post_weight_quantization_06_b200 as g
m, n, k = map(int, sys.argv[1:4])
unused = [int(c) for c in sys.argv[4]]   # kinds of barrier that this call does not wait for
x = torch.randn(m, k, device="cuda"); w = torch.randn(n, k, device="cuda")
ops = (*g.fp8_quantize(x), *g.fp8_quantize(w, block_rows=128))
want = g.fp8_matmul(*ops)
g.gptq_sync_status()
for kind in (1, 2, 3, 4, 5):
    os.environ["GPTQ_TEST_STALL"] = str(kind)
    y = g.fp8_matmul(*ops)
    del os.environ["GPTQ_TEST_STALL"]
    st, site = g.gptq_sync_status(raise_on_error=False)
    if kind in unused:
        assert st == 0 and torch.equal(y, want), (kind, st, site)
    else:
        assert st == g.GPTQ_ERR_TIMEOUT and site // 10 in (1, 2, 3), (kind, st, site)
    for _ in range(3):
        assert torch.equal(g.fp8_matmul(*ops), want), kind
    g.gptq_sync_status()
print("ok")
"""


# One CTA a tile and a cluster. With few blocks of K a CTA uses no stage (3) or no accumulator (5) twice,
# so that nothing waits for it to be free.
@pytest.mark.parametrize("m,n,k,unused", [
    (1, 128, 128, "35"), (1, 256, 2048, "35"), (1, 128, 40000, ""), (1, 8192, 8192, ""),
    (20, 4096, 4096, "3"), (40, 128, 128, "35"), (64, 512, 2048, "35"), (200, 640, 3000, "35"),
    (200, 3000, 3000, ""), (3000, 2816, 130, "3"), (3000, 2816, 900, "")])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(m, n, k, unused):
    env = dict(os.environ, GPTQ_WAIT_LIMIT_CYCLES="20000000")
    env.pop("GPTQ_TEST_STALL", None)
    out = subprocess.run([sys.executable, "-c", STALL, str(m), str(n), str(k), unused], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stderr[-2000:]
