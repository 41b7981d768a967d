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


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_heads_whose_offsets_pass_32_bits(dtype):
    """All operands as slices of one tensor whose heads are 2^31 elements apart (bytes and elements pass 32 bits)."""
    import hierarchical_block_sparse_pyr_b200 as P

    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 9 GB of device memory")
    g = torch.Generator().manual_seed(19)
    cu, H, d = [0, 200, 201, 350], 2, 64
    T = cu[-1]
    flat = torch.empty(2 ** 31 + 8 * T * d, dtype=dtype, device="cuda")
    far = [flat.as_strided((H, T, d), (2 ** 31, d, 1), i * T * d) for i in range(8)]
    near = [torch.empty((H, T, d), dtype=dtype, device="cuda") for _ in range(8)]
    s = P.packed_shape(3, T, H, H, d, dtype)
    plan = P.packed_plan(s, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    for x, y in zip(far[:4], near[:4]):  # Q, K, V, dO
        y.copy_(torch.randn((H, T, d), generator=g).to(dtype))
        x.copy_(y)
    for Q, K, V, dO, O, dQ, dK, dV in (far, near):
        lse = torch.empty((H, T), device="cuda")
        P.packed_forward(s, Q, K, V, plan, O, lse)
        P.packed_backward(s, Q, K, V, plan, O, lse, dO, torch.empty_like(lse), dQ, dK, dV)
    torch.cuda.synchronize()
    for x, y in zip(far, near):
        assert torch.equal(x, y)


def test_one_plan_on_two_streams_at_once():
    """The layers of a model share a plan; here two of them run at the same time."""
    import hierarchical_block_sparse_pyr_b200 as P

    g = torch.Generator().manual_seed(29)
    cu, Hq, Hkv, d = [0, 900, 1000, 2500], 8, 2, 64
    T = cu[-1]
    s = P.packed_shape(3, T, Hq, Hkv, d, BF16)
    plan = P.packed_plan(s, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    layers = []
    for _ in range(2):
        Q, K, V, dO = (torch.randn((H, T, d), generator=g).to(BF16).cuda() for H in (Hq, Hkv, Hkv, Hq))
        runs = [[torch.zeros_like(x) for x in (Q, Q, K, V)] + [torch.zeros((Hq, T), device="cuda") for _ in range(2)]
                for _ in range(2)]
        layers.append((Q, K, V, dO, runs, torch.cuda.Stream()))

    def run(layer, out, stream):
        Q, K, V, dO = layer[:4]
        O, dQ, dK, dV, lse, delta = out
        P.packed_forward(s, Q, K, V, plan, O, lse, stream=stream)
        P.packed_backward(s, Q, K, V, plan, O, lse, dO, delta, dQ, dK, dV, stream=stream)

    for layer in layers:
        run(layer, layer[4][0], None)
    torch.cuda.synchronize()
    for _ in range(3):
        for layer in layers:
            run(layer, layer[4][1], layer[5])
    torch.cuda.synchronize()
    for layer in layers:
        for x, y in zip(*layer[4]):
            assert torch.equal(x, y)
