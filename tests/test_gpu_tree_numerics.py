"""Drafted trees over caches with values that are not finite."""
import pytest
import torch

import _plain64 as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,T,Hq,Hkv", [([40, 70, 40], 5, 4, 2), ([9000, 300, 5000], 1, 8, 2),
                                           ([2000, 700, 3000], 64, 8, 1), ([700] * 90, 8, 4, 2)])
def test_a_key_that_is_not_a_number(dtype, lens, T, Hq, Hkv):
    """A NaN among a sequence's cached keys, or in a draft's: O and lse of the tokens that see it are NaN (-inf is for
    absent slots), those of the others are what they were."""
    import hierarchical_block_sparse_pyr_b200 as P

    B, d = len(lens), 64
    N = max(lens) + T + 3
    g = torch.Generator().manual_seed(4)
    Q, K, V = (torch.randn((B, H, n, d), generator=g).to(dtype).cuda() for H, n in ((Hq, T), (Hkv, N), (Hkv, N)))
    parent = [[(t - 1) // 2 if t else -1 for t in range(T)] for _ in range(B)]  # binary trees
    parent[1] = [-2 if t == T - 1 and T > 1 else p for t, p in enumerate(parent[1])]
    s = P.tree_shape(B, Hq, Hkv, N, T, d, dtype)
    ws = torch.empty(P.tree_workspace_bytes(s), dtype=torch.uint8, device="cuda")

    def run(k):
        O, lse = torch.full_like(Q, 7.0), torch.full((B, Hq, T), 7.0, device="cuda")
        P.tree_forward(s, Q, k, V, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                       torch.tensor(parent, dtype=torch.int32, device="cuda"), O, lse, ws)
        torch.cuda.synchronize()
        return O, lse

    want = run(K)
    see = [ref.ancestors(p) for p in parent]
    places = [0, lens[0] - 1, lens[0], lens[0] + T - 1]
    # of two sequences the same row, then of each a row of its own, the last draft's among them
    for first, second in [2 * [p if p < lens[1] else 0] for p in places] + [(p, lens[1] + T // 2) for p in places]:
        bad = K.clone()
        bad[0, :, first] = float("nan")
        bad[1, :, second] = float("nan")
        O, lse = run(bad)
        for b in range(B):
            row = (first, second)[b] if b < 2 else -1
            for t in range(T):
                hit = b < 2 and bool(see[b][t]) and (row < lens[b] or row - lens[b] in see[b][t])
                if hit:
                    assert O[b, :, t].isnan().all() and lse[b, :, t].isnan().all(), (row, b, t)
                else:
                    assert torch.equal(O[b, :, t], want[0][b, :, t]), (row, b, t)
                    assert torch.equal(lse[b, :, t], want[1][b, :, t]), (row, b, t)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,T", [([5000, 3, 900], 7), ([64, 70], 1), ([700] * 60, 33)])
def test_what_the_workspace_held_does_not_matter(dtype, lens, T):
    import hierarchical_block_sparse_pyr_b200 as P

    B, Hq, Hkv, d = len(lens), 8, 2, 128
    N = max(lens) + T
    g = torch.Generator().manual_seed(14)
    Q, K, V = (torch.randn((B, H, n, d), generator=g).to(dtype).cuda() for H, n in ((Hq, T), (Hkv, N), (Hkv, N)))
    s = P.tree_shape(B, Hq, Hkv, N, T, d, dtype)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = []
    for fill in (0, 255):  # 255: NaN in every part
        ws = torch.full((P.tree_workspace_bytes(s),), fill, dtype=torch.uint8, device="cuda")
        O, lse = torch.empty_like(Q), torch.empty((B, Hq, T), device="cuda")
        P.tree_forward(s, Q, K, V, n, None, O, lse, ws)
        out.append((O, lse))
    torch.cuda.synchronize()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1]) and out[0][0].isfinite().all()
