"""GPU tests of the block-FP8 feed-forward operators at the ends of what they
accept: the smallest and the widest shapes, and a process whose first calls
are captured into a graph."""
import os
import subprocess
import sys

import pytest
import torch

import int8_gemm_gemv_b200 as bsq
from test_gpu_block_ffn import Moe, run_gemm

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert bsq.debug_take_timeouts() == 0


@pytest.mark.parametrize("t,h,i,e,topk,renorm", [
    (1, 128, 128, 1, 1, 0), (2, 65536, 128, 2, 2, 1), (2, 128, 65536, 2, 1, 0), (3, 16384, 4224, 2, 2, 1),
    (16, 128, 128, 512, 16, 0), (16, 128, 256, 16, 16, 1)])
def test_moe_extremes(t, h, i, e, topk, renorm):
    m = Moe(t, h, i, e, topk, renorm, seed=t)
    m()
    m.check()


@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (1, 1, 65536), (64, 1, 128), (65, 1, 128), (3, 151936, 256),
                                   (70000, 3, 256), (64, 40000, 128), (130, 300, 65536)])
def test_gemm_extremes(m, n, k):
    run_gemm(m, n, k, seed=m)


FIRST_CALLS_CAPTURED = """
import sys
sys.path[:0] = [{root!r}, {here!r}]
import torch
import int8_gemm_gemv_b200 as bsq
from test_gpu_block_ffn import Ffn, Moe
few, many, layer = Ffn(24, 1024, 640), Ffn(1100, 1024, 640), Moe(6, 1024, 256, 16, 4, 1, seed=3)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    few(), many(), layer()
for f in (few, many):
    assert f.out.isnan().all()
graph.replay()
torch.cuda.synchronize()
few.check(), many.check(), layer.check()
assert bsq.debug_take_timeouts() == 0
print("captured")
"""


def test_first_calls_of_a_process_captured():
    code = FIRST_CALLS_CAPTURED.format(root=os.path.dirname(HERE), here=HERE)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
