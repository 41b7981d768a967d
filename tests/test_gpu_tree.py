"""Drafted trees over a cache on the GPU against the definition in double.

Tolerances as for the packed prompts: fp32 2e-5 of the largest |v| and 2e-5 for lse; bf16 2^-8 |x| (one
rounding of the output) + 2^-7 of the largest |v| (P rounded to bf16 once), lse 1e-4.
"""
import random

import pytest
import torch

import _plain64 as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _tensor(order, B, H, N, d, dtype, g):
    x = torch.randn((B, H, N, d), generator=g).to(dtype).cuda()
    return x if order == "hnd" else x.transpose(1, 2).contiguous().transpose(1, 2)


def _parents(kind, B, T, rng):
    if kind == "chain":
        return [list(range(-1, T - 1)) for _ in range(B)]
    if kind == "roots":
        return [[-1] * T for _ in range(B)]
    p = [[rng.randrange(-1, t) for t in range(T)] for _ in range(B)]
    if kind == "absent":  # padded batches: some slots, some sequences, and what hangs below an absent slot
        for b in range(B):
            for t in range(T):
                if rng.random() < 0.3 or (b % 3 == 2):
                    p[b][t] = -2
    return p


def _run(P, Q, K, V, lens, parent, workspace=None):
    B, Hq, T, d = Q.shape
    s = P.tree_shape(B, Hq, K.shape[1], K.shape[2], T, d, Q.dtype)
    O = torch.full_like(Q, 7.0)
    lse = torch.full((B, Hq, T), 7.0, device="cuda")
    ws = workspace
    if ws is None:
        ws = torch.empty(P.tree_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.tree_forward(s, Q, K, V, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                   None if parent is None else torch.tensor(parent, dtype=torch.int32, device="cuda"), O, lse, ws, status)
    torch.cuda.synchronize()
    return O, lse, int(status)


def _compare(O, lse, Q, K, V, lens, parent):
    wo, wl = ref.tree(Q, K, V, lens, parent)
    seen = wl > -float("inf")
    assert torch.equal(seen, lse > -float("inf"))
    assert (O[~seen] == 0).all()
    used = V.clone()
    used[~torch.isfinite(used)] = 0
    vmax = float(used.abs().max())
    eo = (O.double() - wo).abs()
    el = (lse.double() - wl)[seen].abs()
    if Q.dtype == F32:
        assert float(eo.max()) <= 2e-5 * vmax and (el <= 2e-5).all(), (float(eo.max()), el.max())
    else:
        assert (eo <= 2.0 ** -8 * wo.abs() + 2.0 ** -7 * vmax).all(), float(eo.max())
        assert (el <= 1e-4).all(), float(el.max())


CASES = [
    # lens, slack, T, Hq, Hkv, d, dtype, kind, order
    ([0], 0, 1, 1, 1, 64, F32, "chain", "hnd"),
    ([0], 3, 1, 4, 1, 128, BF16, "chain", "nhd"),
    ([0, 1, 2, 63, 64, 65], 0, 3, 4, 2, 64, F32, "random", "nhd"),
    ([0, 1, 126, 127, 128, 129, 300], 5, 8, 8, 2, 128, BF16, "random", "hnd"),
    ([1000], 24, 8, 32, 8, 128, BF16, "chain", "hnd"),
    ([5000, 0, 17, 2000], 1, 64, 8, 2, 128, BF16, "random", "nhd"),
    ([700, 900, 0, 64], 30, 16, 4, 4, 64, BF16, "absent", "nhd"),
    ([700, 900, 0, 64, 128, 5], 30, 33, 16, 2, 128, BF16, "absent", "hnd"),
    ([300, 20, 150], 7, 5, 6, 2, 64, F32, "absent", "hnd"),
    ([12345, 1], 0, 1, 32, 8, 128, BF16, "chain", "hnd"),
    ([3000], 0, 64, 8, 1, 128, BF16, "random", "nhd"),      # 512 rows per unit
    ([800, 10], 0, 61, 7, 1, 64, BF16, "roots", "nhd"),     # 427 rows
    ([2000, 33, 1], 0, 40, 6, 2, 128, F32, "random", "nhd"),
    ([31] * 200, 1, 4, 8, 2, 64, BF16, "random", "hnd"),    # more segments than CTAs
    ([1900, 40, 0, 700, 3000] * 20, 9, 5, 8, 4, 128, BF16, "absent", "nhd"),  # more segments than cuts, long and short
    ([500, 40, 0, 700] * 40, 9, 3, 8, 4, 64, F32, "random", "hnd"),
    ([20000], 100, 2, 1, 1, 64, BF16, "chain", "hnd"),      # one segment over every CTA
]
IDS = ["x".join(map(str, c[0][:6])) + "-" + "-".join(map(str, c[1:])) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_tree_against_the_definition(case):
    import hierarchical_block_sparse_pyr_b200 as P

    lens, slack, T, Hq, Hkv, d, dtype, kind, order = case
    B, N = len(lens), max(lens) + T + slack
    g = torch.Generator().manual_seed(7)
    Q, K, V = (_tensor(order, B, H, n, d, dtype, g) for H, n in ((Hq, T), (Hkv, N), (Hkv, N)))
    parent = _parents(kind, B, T, random.Random(8))
    # rows behind the drafts and rows of absent slots hold NaN and infinities
    for b in range(B):
        see = ref.ancestors(parent[b])
        dead = [lens[b] + t for t in range(T) if not see[t]] + list(range(lens[b] + T, N))
        K[b, :, dead] = float("nan")
        V[b, :, dead] = float("nan")
        V[b, :, dead[::2]] = float("inf")
    O, lse, status = _run(P, Q, K, V, lens, parent)
    assert status == 0
    _compare(O, lse, Q, K, V, lens, parent)
    if kind == "chain":
        O2, lse2, _ = _run(P, Q, K, V, lens, None)
        assert torch.equal(O, O2) and torch.equal(lse, lse2)
    again = _run(P, Q, K, V, lens, parent)
    assert torch.equal(O, again[0]) and torch.equal(lse, again[1])


def test_bad_lengths_and_parents_are_reported():
    import hierarchical_block_sparse_pyr_b200 as P

    g = torch.Generator().manual_seed(17)
    for dtype in (F32, BF16):
        Q, K, V = (_tensor("hnd", 4, H, n, 64, dtype, g) for H, n in ((4, 6), (2, 200), (2, 200)))
        lens = [195, -1, 50, 2 ** 31 - 1]  # 195 + 6 > 200
        parent = [list(range(-1, 5))] * 4
        O, lse, status = _run(P, Q, K, V, lens, parent)
        assert status == P.PYR_EBADSEQ
        _compare(O, lse, Q, K, V, lens, parent)
        lens = [0, 10, 194, 63]
        parent = [[0, 0, 1, 2, 3, 4], [-1, 0, 2, 1, -3, 4], [-1, 7, 0, 2, 3, 0], [-1, 0, 0, 1, 1, 2]]
        O, lse, status = _run(P, Q, K, V, lens, parent)
        assert status == P.PYR_EBADSEQ
        _compare(O, lse, Q, K, V, lens, parent)


def test_large_scores():
    import hierarchical_block_sparse_pyr_b200 as P

    g = torch.Generator().manual_seed(27)
    for dtype in (F32, BF16):
        Q, K, V = (_tensor("nhd", 1, H, n, 128, dtype, g) for H, n in ((8, 5), (2, 3005), (2, 3005)))
        K = (K.float() * (1 + torch.arange(3005, device="cuda").reshape(1, 1, -1, 1) % 61)).to(dtype)
        parent = [[-1, 0, 0, 1, 2]]
        O, lse, _ = _run(P, Q, K, V, [3000], parent)
        wo, wl = ref.tree(Q, K, V, [3000], parent)
        # fp32 scores of size 2^9 carry a few 2^-24 * 2^9 = 1e-4
        assert float((lse.double() - wl).abs().max()) <= 1e-3
        assert float((O.double() - wo).abs().max()) <= (2e-3 if dtype == F32 else 2.0 ** -6 * float(V.abs().max()))


def test_tree_under_a_graph_with_new_lengths():
    import hierarchical_block_sparse_pyr_b200 as P

    g = torch.Generator().manual_seed(37)
    B, Hq, Hkv, N, T, d = 3, 8, 2, 2100, 4, 128
    Q, K, V = (_tensor("hnd", B, H, n, d, BF16, g) for H, n in ((Hq, T), (Hkv, N), (Hkv, N)))
    s = P.tree_shape(B, Hq, Hkv, N, T, d, BF16)
    ws = torch.empty(P.tree_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([10, 500, 2000], dtype=torch.int32, device="cuda")
    O, lse = torch.empty_like(Q), torch.empty((B, Hq, T), device="cuda")
    P.tree_forward(s, Q, K, V, lens, None, O, lse, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.tree_forward(s, Q, K, V, lens, None, O, lse, ws)
    chain = [list(range(-1, T - 1))] * B
    for new in ([2096, 0, 77], [1, 1, 1]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        _compare(O, lse, Q, K, V, new, chain)


def test_a_cache_whose_offsets_pass_32_bits():
    """Two sequences 2^32 elements apart, heads 2^31 apart, in a strided cache."""
    import hierarchical_block_sparse_pyr_b200 as P

    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 26 GB of device memory")
    N, d, T, lens = 400, 64, 3, [397, 130]
    g = torch.Generator().manual_seed(47)
    for dtype in (BF16,):
        flat = [torch.empty(2 ** 32 + 2 ** 31 + N * d, dtype=dtype, device="cuda") for _ in range(2)]
        K, V = (f.as_strided((2, 2, N, d), (2 ** 32, 2 ** 31, d, 1)) for f in flat)
        Q = _tensor("hnd", 2, 4, T, d, dtype, g)
        for x in (K, V):
            x.copy_(torch.randn((2, 2, N, d), generator=g).to(dtype).cuda())
        parent = [[-1, 0, 0], [-1, -1, 1]]
        O, lse, status = _run(P, Q, K, V, lens, parent)
        assert status == 0
        _compare(O, lse, Q, K.contiguous(), V.contiguous(), lens, parent)


def test_absent_sequences_may_hold_anything():
    """A padded batch: sequences without tokens, their context rows NaN."""
    import hierarchical_block_sparse_pyr_b200 as P

    g = torch.Generator().manual_seed(57)
    for dtype in (F32, BF16):
        Q, K, V = (_tensor("nhd", 3, H, n, 64, dtype, g) for H, n in ((4, 2), (2, 300), (2, 300)))
        K[1], V[1] = float("nan"), float("nan")
        parent = [[-1, 0], [-2, -2], [-1, -2]]
        O, lse, status = _run(P, Q, K, V, [200, 250, 17], parent)
        assert status == 0
        assert (O[1] == 0).all() and (lse[1] == -float("inf")).all()
        keep = [0, 2]
        _compare(O[keep], lse[keep], Q[keep], K[keep], V[keep], [200, 17], [parent[0], parent[2]])


def test_single_tokens_equal_the_dense_decode():
    """One token per sequence at one length: the framework's dense decode attention of the same cache."""
    import hierarchical_block_sparse_pyr_b200 as P

    g = torch.Generator().manual_seed(67)
    B, Hq, Hkv, N, d = 3, 8, 2, 1000, 128
    Q, K, V = (_tensor("hnd", B, H, n, d, BF16, g) for H, n in ((Hq, 1), (Hkv, N), (Hkv, N)))
    O, lse, _ = _run(P, Q, K, V, [N - 1] * B, None)
    s = P.make_shape(B, Hq, Hkv, N, 1, N - 1, d, 64, 4, 8, BF16)
    O2, lse2 = torch.empty_like(O), torch.empty_like(lse)
    P.dense_forward(s, Q, K, V, O2, lse2)
    # both within half a bf16 step of the output and 2^-7 max|v| (P) of the same value
    assert float((O.float() - O2.float()).abs().max()) <= 2.0 ** -6 * float(V.abs().max())
    assert float((lse - lse2).abs().max()) <= 2e-4


def test_two_calls_on_two_streams_with_workspaces_of_their_own():
    import hierarchical_block_sparse_pyr_b200 as P

    g = torch.Generator().manual_seed(77)
    jobs = []
    for lens, T in (([3000, 10], 7), ([64, 2500], 30)):
        Q, K, V = (_tensor("hnd", 2, H, n, 128, BF16, g) for H, n in ((8, T), (2, 3100), (2, 3100)))
        s = P.tree_shape(2, 8, 2, 3100, T, 128, BF16)
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        want = _run(P, Q, K, V, lens, None)
        jobs.append((torch.cuda.Stream(), s, Q, K, V, n, want,
                     torch.empty(P.tree_workspace_bytes(s), dtype=torch.uint8, device="cuda"), torch.empty_like(Q),
                     torch.empty((2, 8, T), device="cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for st, s, Q, K, V, n, want, ws, O, lse in jobs:
            P.tree_forward(s, Q, K, V, n, None, O, lse, ws, stream=st)
    torch.cuda.synchronize()
    for st, s, Q, K, V, n, want, ws, O, lse in jobs:
        assert torch.equal(O, want[0]) and torch.equal(lse, want[1])


def test_drafts_rotated_at_their_depth_after_a_prompt():
    """The operators as a server uses them: rotate and attend a prompt, keep its keys and values in a cache,
    append a rotated tree at positions len + depth, attend the tree. The path through every token equals
    causal attention of that path as a prompt."""
    import hierarchical_block_sparse_pyr_b200 as P

    g = torch.Generator().manual_seed(87)
    Hq, Hkv, d, n, N = 4, 2, 64, 150, 200
    parent = [-1, 0, 0, 1, 2, 3]
    T, depth = len(parent), [0, 1, 1, 2, 2, 3]
    K, V = (torch.randn((1, Hkv, n + T, d), generator=g).cuda() for _ in range(2))
    Q = torch.randn((1, Hq, n + T, d), generator=g).cuda()
    pos = torch.tensor(list(range(n)) + [n + x for x in depth], dtype=torch.int32, device="cuda")
    spec = P.rope_spec(d)
    cache_k, cache_v = (torch.full((1, Hkv, N, d), float("nan"), device="cuda") for _ in range(2))
    cache_v[:, :, :n + T] = V
    Qr = torch.empty_like(Q)
    P.rope_apply(spec, Q, K, Qr, cache_k[:, :, :n + T], pos=pos)
    O, lse, status = _run(P, Qr[:, :, n:], cache_k, cache_v, [n], [parent])
    assert status == 0
    for t in range(T):
        path = [t]
        while parent[path[0]] >= 0:
            path.insert(0, parent[path[0]])
        rows = list(range(n)) + [n + u for u in path]
        cu = [0, len(rows)]
        s = P.packed_shape(1, len(rows), Hq, Hkv, d, F32)
        plan = P.packed_plan(s, torch.tensor(cu, dtype=torch.int32, device="cuda"))
        o = torch.empty((Hq, len(rows), d), device="cuda")
        P.packed_forward(s, Qr[0, :, rows], cache_k[0, :, rows], cache_v[0, :, rows], plan, o)
        # two fp32 evaluations, each within 2e-5 max|v| of the definition
        assert float((o[:, -1] - O[0, :, t]).abs().max()) <= 4e-5 * float(V.abs().max())
