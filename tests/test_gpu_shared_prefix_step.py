"""The operators around a step's attention together (examples/shared_prefix_step.py): layout, projection, norms with
rotary positions and the append, attention behind a shared prompt, output projection, verification.

Bound of the logits' probabilities, in the 2-norm: x and the weights are given; q, k and v, their normed and turned forms, the
attention's scores (through q and k), its output and the logits are each rounded to bf16 once, at most 2^-9 in the
mean of each; eight roundings in a row, whose errors add, give less than 8 * 2^-9 of the logits, and p = softmax(logits) moves by
at most its logits' error, twice (each and the sum): 2 * 8 * 2^-9 * max |logit|."""
import os
import sys

import pytest
import torch

from test_gpu_step import layout_ref, verify_ref

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

CASES = [
    (700, [37, 0, 130, 64], [[-1, 0, 0, 1, 2], [-1], [-1, 0, 1], [-1, 0, 0, 1, 1, 4, 5]], dict()),
    (33, [1000], [[-1]], dict(heads=4, kv_heads=4, dim=128, page=24, room=3)),
    (1000, [15, 16, 17, 3] * 10, [[-1, 0, 0, 2]] * 40, dict(heads=16, kv_heads=2, vocab=1024, room=171)),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_shared_prefix_step(i):
    from shared_prefix_step import SharedPrefixStep
    prefix, contexts, parents, kw = CASES[i]
    print("[gpu-case] shared prefix step", i, flush=True)
    step = SharedPrefixStep(prefix, contexts, parents, **kw)
    want = step.plain()
    flat = [p for tree in parents for p in tree]
    free = step.free.tolist()
    tables = layout_ref(contexts, [len(t) for t in parents], step.table.tolist(), free, step.x.shape[0], step.page,
                        [prefix] * len(contexts), flat + [-1] * (step.x.shape[0] - len(flat)), 1)
    out = [t.clone() for t in step.step()]
    torch.cuda.synchronize()
    for name in ("q_starts", "requests", "positions", "slots", "free_left"):
        assert getattr(step.tables, name).tolist() == tables[name], name
    assert step.table.tolist() == tables["table"]
    n = len(want)
    off = float((step.probabilities[:n].double().cpu() - want).norm() / want.norm())
    assert off < 2 * 8 * 2.0 ** -9 * max(1.0, float(step.out_call.out[:n].abs().max())), off
    # the verification, from the probabilities as they came out
    c = dict(target=step.probabilities, draft=None, parents=step.up, tokens=step.tokens, starts=step.tables.q_starts,
             accept=step.accept, sample=step.sample, depth=out[0].shape[1])
    accepted, counts, following = verify_ref(c)
    assert out[0].tolist() == accepted and out[1].tolist() == counts and out[2].tolist() == following
    # the same step captured, replayed with eager ones between
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.step()
    for _ in range(3):
        for t in step.verify_call.out:
            t.fill_(-7)
        step.probabilities.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step.verify_call.out, out))
        assert all(torch.equal(a, b) for a, b in zip(step.step(), out))
