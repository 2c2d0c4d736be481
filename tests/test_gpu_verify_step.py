"""The serving operators together: the attention block of a verification step (examples/verify_step.py)
against the same block in fp64.

Bound: x, the projections, q, k, v, the attention and the output are each rounded to bf16 once (2^-8 of each, about
2^-9.5 in the mean), eight roundings in a row whose errors add in the 2-norm to less than 8 * 2^-9 of the
result: the softmax's derivative is at most the scores' error, which is of the same size here."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("case", [
    ([37, 500, 0, 130], [[-1, 0, 0, 1, 2], [-1], [-1, 0, 1], [-1, -1, 0, 1, 1, 4, 5]], [0, -1, 1, 0], dict()),
    ([1000], [[-1]], [0], dict(heads=4, kv_heads=4, dim=128, page=24, rank=8)),
    ([15, 16, 17, 3] * 6, [[-1, 0, -1, 2]] * 24, [i % 5 - 1 for i in range(24)], dict(heads=16, kv_heads=2, rank=40)),
])
def test_verify_step(case):
    from verify_step import VerifyStep
    contexts, parents, adapters, kw = case
    print("[gpu-case] verify step", contexts[:4], kw, flush=True)
    step = VerifyStep(contexts, parents, adapters, **kw)
    want = step.plain()
    got = step.step()
    torch.cuda.synchronize()
    off = float((got.double().cpu() - want).norm() / want.norm())
    assert off < 8 * 2.0 ** -9, off
    first = got.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.step()
    for _ in range(3):
        step.out_call.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.out_call.out, first)
