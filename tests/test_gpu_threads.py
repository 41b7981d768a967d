"""Calls from host threads of their own."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _in_a_thread(fn):
    out = []

    def run():
        try:
            fn()
        except Exception as e:  # handed to the caller's thread
            out.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not out, out


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_first_call_of_a_thread(dtype):
    """A thread whose first use of CUDA is a call of this library."""
    import hierarchical_block_sparse_pyr_b200 as P

    g = torch.Generator().manual_seed(2)
    mk = lambda *s: torch.randn(s, generator=g).to(dtype).cuda()  # noqa: E731
    H, T, d, N = 2, 100, 64, 256
    Q, K, V, dO = (mk(H, T, d) for _ in range(4))
    s = P.packed_shape(1, T, H, H, d, dtype)
    plan = P.packed_plan(s, torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    t = P.tree_shape(1, H, H, T, 1, d, dtype)
    lens = torch.tensor([T - 1], dtype=torch.int32, device="cuda")
    ws = torch.empty(P.tree_workspace_bytes(t), dtype=torch.uint8, device="cuda")
    b = P.make_shape(1, H, H, N, N, 0, d, 64, 4, 4, dtype)
    q, k, v = (mk(1, H, N, d) for _ in range(3))
    stream = torch.cuda.current_stream()

    def run(call):
        O, lse, grads = torch.zeros_like(Q), torch.zeros((H, T), device="cuda"), [torch.zeros_like(x) for x in (Q, K, V)]
        to, delta = torch.zeros((1, H, 1, d), dtype=dtype, device="cuda"), torch.zeros((H, T), device="cuda")
        o, z = torch.zeros_like(q), torch.zeros((1, H, N), device="cuda")
        torch.cuda.synchronize()
        call(lambda: P.packed_forward(s, Q, K, V, plan, O, lse, stream=stream))
        call(lambda: P.packed_backward(s, Q, K, V, plan, O, lse, dO, delta, *grads, stream=stream))
        call(lambda: P.tree_forward(t, Q[None, :, T - 1:], K[None], V[None], lens, None, to, workspace=ws, stream=stream))
        call(lambda: P.dense_forward(b, q, k, v, o, z, stream=stream))
        return [O, lse, to, o, z] + grads

    want = run(lambda fn: fn())
    for x, y in zip(run(_in_a_thread), want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_two_threads_with_different_batches(dtype):
    """One thread calls tree_forward with one sequence, another with 4096, as fast as the library takes them (through
    the C ABI): what one call sets up must not fail the other's. (Where the limit of a kernel's shared memory went
    with the call's batch, 42 of 20000 bf16 calls and 6 of 20000 fp32 calls were refused.)"""
    import ctypes

    import hierarchical_block_sparse_pyr_b200 as P

    lib = P._L()
    g = torch.Generator().manual_seed(3)
    jobs, refused = [], [0, 0]
    for B, N in ((1, 64), (4096, 2)):
        Q, K, V = (torch.randn((B, 2, n, 64), generator=g).to(dtype).cuda() for n in (1, N, N))
        s = P.tree_shape(B, 2, 2, N, 1, 64, dtype)
        lens = torch.full((B,), N - 1, dtype=torch.int32, device="cuda")
        ws = torch.empty(P.tree_workspace_bytes(s), dtype=torch.uint8, device="cuda")
        O, want = torch.empty_like(Q), torch.empty_like(Q)
        P.tree_forward(s, Q, K, V, lens, None, want, workspace=ws)
        arr, v = P._views(s.dtype, 0, (Q, "Q", Q.shape), (K, "K", K.shape), (V, "V", V.shape), (O, "O", O.shape))
        stream = torch.cuda.Stream()
        args = (ctypes.byref(s), v, v + 32, v + 64, lens.data_ptr(), None, v + 96, None, ws.data_ptr(), ws.numel(), None,
                stream.cuda_stream)
        jobs.append((args, stream, O, want, (arr, Q, K, V, s, lens, ws)))
    torch.cuda.synchronize()

    def call(i):
        args, stream = jobs[i][:2]
        for n in range(20000):
            refused[i] += lib.tree_forward(*args) != P.PYR_OK
            if n % 500 == 0:
                stream.synchronize()

    threads = [threading.Thread(target=call, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0, 0]
    for _, _, O, want, _ in jobs:
        assert torch.equal(O, want)
