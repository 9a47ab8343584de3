"""GPU: the calls of the binding that make their own outputs and status (select_topk, plan_forward, forward), given a
stream that is not the current one: everything that such a call queues, the status word's zero among it, is on that
stream, so the current stream's work does not hold up or overwrite any of it."""
import numpy as np
import pytest

from block_sparse_top_attn_gb300 import workloads as W
from tests._util import upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from block_sparse_top_attn_gb300 import binding
    return binding


@pytest.mark.parametrize("call", ["select_topk", "plan_forward", "forward", "forward_planned"])
def test_a_call_on_a_side_stream_is_that_streams_alone(B, call):
    import torch
    pb = W.make_problem(lengths=[700, 260, 5], num_index_heads=2, topk=4, policy="diag_uniform", seed=6, values=False)
    prob, t = upload(pb)
    q, k, v, _ = W.device_values(pb, "cuda", seed=1)
    plan = B.plan_forward(prob, t["sel"])[0]
    run = {"select_topk": lambda s: B.select_topk(prob, k, v, s), "plan_forward": lambda s: B.plan_forward(prob, t["sel"], s),
           "forward": lambda s: B.forward(prob, t["sel"], q, k, v, s),
           "forward_planned": lambda s: B.forward(prob, t["sel"], q, k, v, s, plan)}[call]
    side = torch.cuda.Stream()
    want = run(None)
    with torch.cuda.stream(side):
        run(None)                           # memory of the side stream, kernels loaded
    torch.cuda.synchronize()
    # small blocks of the current stream's memory that hold anything but zero
    left = [torch.full((4,), 5, dtype=torch.int32, device="cuda") for _ in range(64)]
    busy = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    del left
    for _ in range(60):                     # some 20 ms: a zero fill queued here comes after the side stream's kernels
        busy.add_(1.0)
    got = run(side)
    side.synchronize()
    with torch.cuda.stream(side):
        early = [x.clone() for x in got]
    torch.cuda.synchronize()
    for x, y, w in zip(got, early, want):
        if x.dtype == torch.int32 and x.numel() == 4:       # status, work count: the first word
            x, y, w = x[:1], y[:1], w[:1]
        assert torch.equal(x, w) and torch.equal(y, w)
    assert int(got[-1][0].item()) == 0
