"""Rotary positions on the GPU against the definition in double.

Tolerance: the angle's fraction of a turn is exact to 2^-25 turns (one rounding to fp32 of a value of at
most 1/2), i.e. 2 pi 2^-25 = 1.9e-7 radians; sincospi and the scale add 3 fp32 roundings, the two products
and their sum 3 more: |error| <= (1.9e-7 + 8 * 2^-24) * scale * (|a| + |b|) < 7e-7 * scale * (|a| + |b|),
plus half a step of the output type for bf16 (2^-8 relative).
"""
import pytest
import torch

import _plain64 as ref

pytestmark = pytest.mark.gpu


def _views(order, B, H, N, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, H, N, d), generator=g).to(dtype).cuda()
    return x if order == "hnd" else x.transpose(1, 2).contiguous().transpose(1, 2)


def _check(x, y, pos, freq, scale, rot, layout, inverse):
    want = ref.rope(x, pos, freq, scale, rot, layout, inverse)
    n = rot // 2
    i = torch.arange(n, device=x.device)
    a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    mag = torch.zeros_like(want)
    s = x.double()[..., a].abs() + x.double()[..., b].abs()
    mag[..., a], mag[..., b] = s, s
    bound = 7e-7 * scale * mag
    if x.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * want.abs()
        bound = bound * (1 + 2.0 ** -8)
    assert ((y.double() - want).abs() <= bound).all()
    assert torch.equal(y[..., rot:], x[..., rot:])


CASES = [
    # B, Hq, Hkv, N, d, rot, dtype, layout, scaling, order
    (1, 1, 1, 1, 64, 64, torch.float32, "half", None, "hnd"),
    (2, 5, 1, 33, 64, 32, torch.float32, "interleaved", "linear", "nhd"),
    (1, 4, 2, 257, 128, 128, torch.bfloat16, "half", "yarn", "hnd"),
    (3, 9, 3, 100, 128, 64, torch.bfloat16, "interleaved", "ntk", "nhd"),
    (2, 3, 2, 65, 128, 20, torch.bfloat16, "half", None, "hnd"),        # pairs that straddle 16-byte chunks
    (2, 3, 2, 65, 64, 2, torch.float32, "half", None, "nhd"),
    (1, 2, 2, 31, 64, 6, torch.bfloat16, "interleaved", "yarn", "hnd"),
    (1, 16, 16, 3000, 128, 128, torch.bfloat16, "interleaved", None, "nhd"),  # many tokens: heads share angles
    (1, 17, 2, 3000, 128, 64, torch.float32, "half", "ntk", "nhd"),
    (70, 8, 2, 1, 128, 128, torch.bfloat16, "half", "linear", "hnd"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_against_the_definition(case, inverse):
    import hierarchical_block_sparse_pyr_b200 as P

    B, Hq, Hkv, N, d, rot, dtype, layout, scaling, order = case
    kw = dict(scaling=scaling, factor=8.0, trained=4096) if scaling else {}
    spec = P.rope_spec(d, rot, base=500000.0, layout=layout, **kw)
    freq, scale = ref.frequencies(rot, 500000.0, **kw)
    Q, K = _views(order, B, Hq, N, d, dtype, 1), _views(order, B, Hkv, N, d, dtype, 2)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-5, 1 << 20, (B, N), generator=g, dtype=torch.int32)
    pos[0, 0] = 2 ** 31 - 1
    pos = pos.cuda()
    Qo, Ko = torch.full_like(Q, 9.0), torch.full_like(K, 9.0)
    q0, k0 = Q.clone(), K.clone()
    P.rope_apply(spec, Q, K, Qo, Ko, pos=pos, inverse=inverse)
    assert torch.equal(Q, q0) and torch.equal(K, k0)
    _check(Q, Qo, pos, freq, scale, rot, layout, inverse)
    _check(K, Ko, pos, freq, scale, rot, layout, inverse)
    # in place gives the same bits; a shared [N] and an offset are positions too; one operand alone works
    Q2, K2 = Q.clone(), K.clone()
    P.rope_apply(spec, Q2, K2, Q2, K2, pos=pos, inverse=inverse)
    assert torch.equal(Q2, Qo) and torch.equal(K2, Ko)
    row = torch.arange(77, 77 + N, dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(K), torch.empty_like(K)
    P.rope_apply(spec, None, K, None, a, pos=row, inverse=inverse)
    P.rope_apply(spec, K, None, b, None, pos_offset=77, inverse=inverse)
    assert torch.equal(a, b)
    _check(K, a, row.expand(B, N), freq, scale, rot, layout, inverse)


def test_inverse_is_the_gradient():
    """<dy, R x> = <R^T dy, x> for fp32: both sides in double from the kernel's outputs."""
    import hierarchical_block_sparse_pyr_b200 as P

    spec = P.rope_spec(64, 48, layout="half", scaling="yarn", factor=4.0, trained=2048)
    x, dy = _views("hnd", 2, 3, 50, 64, torch.float32, 5), _views("hnd", 2, 3, 50, 64, torch.float32, 6)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    P.rope_apply(spec, x, None, y, None, pos_offset=1000)
    P.rope_apply(spec, dy, None, dx, None, pos_offset=1000, inverse=True)
    a, b = (dy.double() * y.double()), (dx.double() * x.double())
    # an element of y is off by at most 7e-7 scale (|a| + |b|) (above), of dx likewise: summed against the
    # other factor
    bound = 7e-7 * spec.scale * 2 * float(x.abs().max() * dy.abs().double().sum() + dy.abs().max() * x.abs().double().sum())
    assert abs(float(a.sum() - b.sum())) <= bound
    # a scale of one turns back exactly but for rounding
    one = P.rope_spec(64, 64)
    P.rope_apply(one, x, None, y, None, pos_offset=123456)
    P.rope_apply(one, y, None, y, None, pos_offset=123456, inverse=True)
    # two rotations, each off by at most 7e-7 (|a| + |b|) <= 7e-7 * 2 max |x|, the second of values up to 2 max |x|
    assert float((y - x).abs().max()) <= 7e-7 * (2 + 4) * float(x.abs().max())


def test_rope_under_a_graph_and_on_a_side_stream():
    import hierarchical_block_sparse_pyr_b200 as P

    spec = P.rope_spec(128)
    x = _views("nhd", 2, 8, 300, 128, torch.bfloat16, 9)
    want, got = torch.empty_like(x), torch.empty_like(x)
    P.rope_apply(spec, x, None, want, None, pos_offset=5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.rope_apply(spec, x, None, got, None, pos_offset=5)
    got.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    got.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    P.rope_apply(spec, x, None, got, None, pos_offset=5, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
