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


def test_tables_of_two_sizes_from_two_threads(B):
    """Two host threads build the tables of a problem with many key blocks and of a small one, on streams of their own:
    every call succeeds and writes the tables of a call alone.  (The shared-memory limit of the build's kernels does not
    depend on the problem.)"""
    import ctypes
    import threading
    import torch

    def made(length, topk, seed):
        pb = W.make_problem(lengths=[length], num_index_heads=1, topk=topk, policy="diag_uniform", seed=seed, values=False)
        prob, t = upload(pb)
        bw = B.Backward(prob)
        B.msa_build_k2q(prob, t["sel"], bw.row_ptr, bw.q_indices, bw.edge_cap, bw.status, bw.ws)
        torch.cuda.synchronize()
        n = int(bw.row_ptr[0, -1].item())
        want = bw.row_ptr.clone(), bw.q_indices[:, :n].clone()
        bw.row_ptr.fill_(-7)
        bw.q_indices.fill_(-7)
        c, stream = prob.c_struct(), torch.cuda.Stream()
        p = lambda x: ctypes.c_void_p(x.data_ptr())
        args = [ctypes.byref(c), p(t["sel"]), p(bw.row_ptr), p(bw.q_indices), ctypes.c_int64(bw.edge_cap), p(bw.status),
                p(bw.ws), ctypes.c_size_t(bw.ws.numel()), ctypes.c_void_p(stream.cuda_stream)]
        return (c, prob, t, stream), bw, want, args, n

    work = [made(400000, 1, 1), made(200, 2, 2)]
    torch.cuda.synchronize()
    failed, start = [0, 0], threading.Barrier(2)

    def run(i):
        start.wait()
        for _ in range(2000):
            failed[i] += B.lib.msa_build_k2q(*work[i][3]) != 0

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0, 0]
    for _, bw, (row_ptr, q_indices), _, n in work:
        assert int(bw.status[0].item()) == 0
        assert torch.equal(bw.row_ptr, row_ptr) and torch.equal(bw.q_indices[:, :n], q_indices)
