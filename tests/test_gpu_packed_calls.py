"""Packed prompts: calls on other streams than the current one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_a_plan_made_on_another_stream_is_that_streams_memory(raw):
    """packed_plan allocates the plan for the stream that writes it: not from blocks that the current stream has
    just given back, whose last kernel there may still run."""
    import hierarchical_block_sparse_pyr_b200 as P

    s = P.packed_shape(2, 300, 2, 2, 64, BF16)
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    n = P.packed_plan_elems(s)
    given_back = [torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(64)]
    known = {x.data_ptr() for x in given_back}
    del given_back
    side = torch.cuda.Stream()
    plan = P.packed_plan(s, cu, stream=side.cuda_stream if raw else side)
    assert plan.data_ptr() not in known
    want = P.packed_plan(s, cu)
    torch.cuda.synchronize()
    assert int(plan[3]) == int(want[3]) and torch.equal(plan[:3], want[:3])
    # given back, it is the side stream's again, not the current one's
    at = plan.data_ptr()
    del plan
    fresh = [torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(64)]
    assert at not in {x.data_ptr() for x in fresh}


def test_a_plan_on_the_default_stream_by_its_handle():
    import hierarchical_block_sparse_pyr_b200 as P

    s = P.packed_shape(2, 300, 2, 2, 64, BF16)
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
        plan = P.packed_plan(s, cu, stream=0)
    want = P.packed_plan(s, cu)
    torch.cuda.synchronize()
    assert int(plan[3]) == int(want[3]) and torch.equal(plan[:3], want[:3])


def test_plan_forward_and_backward_on_a_side_stream():
    """Everything by stream=, the plan's memory included, while the current stream is busy with memory of the sizes
    that the calls use."""
    import hierarchical_block_sparse_pyr_b200 as P

    g = torch.Generator().manual_seed(9)
    cu, Hq, Hkv, d = [0, 700, 701, 1500], 4, 2, 128
    T = cu[-1]
    Q, K, V, dO = (torch.randn((H, T, d), generator=g).to(BF16).cuda() for H in (Hq, Hkv, Hkv, Hq))
    s = P.packed_shape(3, T, Hq, Hkv, d, BF16)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    n = P.packed_plan_elems(s)
    torch.cuda.synchronize()

    def run(stream):
        out = [torch.zeros_like(x) for x in (Q, Q, K, V)]
        lse, delta = torch.zeros((Hq, T), device="cuda"), torch.zeros((Hq, T), device="cuda")
        torch.cuda.synchronize()
        for _ in range(50):
            torch.full((n,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")  # given back at once, still being written
        plan = P.packed_plan(s, cut, stream=stream)
        P.packed_forward(s, Q, K, V, plan, out[0], lse, stream=stream)
        P.packed_backward(s, Q, K, V, plan, out[0], lse, dO, delta, *out[1:], stream=stream)
        torch.cuda.synchronize()
        return out

    want = run(None)
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        for x, y in zip(run(stream), want):
            assert torch.equal(x, y)
