"""Rotated queries and keys through the framework's selection and block-sparse attention."""
import math

import pytest
import torch

import _plain64 as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inplace", [False, True])
def test_rotate_select_and_attend(inplace):
    """With as many blocks selected as there are, the sparse path is causal attention of the rotated tensors.

    fp32: the tolerances of the packed prompts (2e-5 of the largest |v| for O, 2e-5 for lse); the rotation adds 7e-7
    relative per element to scores of size a few, which is far below them."""
    import hierarchical_block_sparse_pyr_b200 as P

    B, Hq, Hkv, N, d = 2, 4, 2, 512, 64
    g = torch.Generator().manual_seed(31)
    Q, K, V = (torch.randn((B, H, N, d), generator=g).cuda() for H in (Hq, Hkv, Hkv))
    spec = P.rope_spec(d, 32, layout="half", scaling="ntk", factor=2.0)
    freq, scale = ref.frequencies(32, 10000.0, "ntk", 2.0)
    pos = torch.arange(1000, 1000 + N).expand(B, N).cuda()
    q64, k64 = (ref.rope(x, pos, freq, scale, 32, "half") for x in (Q, K))
    Qr, Kr = (Q.clone(), K.clone()) if inplace else (torch.empty_like(Q), torch.empty_like(K))
    P.rope_apply(spec, Qr if inplace else Q, Kr if inplace else K, Qr, Kr, pos_offset=1000)
    O, lse, idx, _ = P.forward(Qr, Kr, V, b=64, topk=8, cap=8)
    torch.cuda.synchronize()
    late = torch.ones((N, N), dtype=torch.bool, device="cuda").tril()
    for b in range(B):
        wo, wl = ref.attend(q64[b], k64[b], V[b], late)
        assert float((O[b].double() - wo).abs().max()) <= 2e-5 * float(V.abs().max())
        assert float((lse[b].double() - wl).abs().max()) <= 2e-5
    assert math.isfinite(float(O.sum())) and (idx[:, :, -1] >= 0).sum() == B * Hkv * 7
