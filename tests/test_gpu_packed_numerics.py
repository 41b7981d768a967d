"""Packed prompts in bf16 where the gradients' terms cancel, and with values that are not finite.

The error model of the gradients. Inputs are exact; with u = 2^-8 / sqrt(3), the largest root mean square of a
rounding to bf16 relative to the value, and independent roundings:
  dS is rounded once before it meets K or Q: variance u^2 dS^2 a term;
  D comes from a rounded O, off by e = u |(dO_i O_i)_i| at first, and is put right from sum_k P (dO . v - D): what
    stays of it is the rounding of P e in dS and of P in the correction, 2 u^2 P^2 e^2 a term;
  dO . v is a sum of d products in fp32, at most d/2 + 2 roundings of 2^-24 |dO||v|:
    P^2 f^2 a term, f = sqrt(d/2 + 2) 2^-24 |dO||v|;
  P is rounded once before it meets dO: u^2 P^2 a term of dV;
  the result is rounded once: u^2 of its square.
A term's variance is multiplied by the square of the row it meets, and the sums over thousands of terms keep
close to their mean: the bound is 1.25 times the square root of the variance.
"""
import math

import pytest
import torch

import _plain64 as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U2 = 2.0 ** -16 / 3


def _make(lens, Hq, Hkv, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    mk = lambda H: torch.randn((T, H, d), generator=g).cuda().transpose(0, 1)  # noqa: E731
    return cu, mk(Hq), mk(Hkv), mk(Hkv), mk(Hq)


def _train(cu, Q, K, V, dO):
    import hierarchical_block_sparse_pyr_b200 as P

    Hq, T, d = Q.shape
    s = P.packed_shape(len(cu) - 1, T, Hq, K.shape[0], d, Q.dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = P.packed_plan(s, torch.tensor(cu, dtype=torch.int32, device="cuda"), status=status)
    O, lse = torch.empty_like(Q), torch.empty((Hq, T), device="cuda")
    grads = [torch.empty_like(x) for x in (Q, K, V)]
    P.packed_forward(s, Q, K, V, plan, O, lse, status)
    P.packed_backward(s, Q, K, V, plan, O, lse, dO, torch.empty_like(lse), *grads, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    return O, lse, grads


def _gradients_and_spread(cu, Q, K, V, dO):
    """dQ, dK, dV in double and the variance of every row of them by the model above."""
    Hq, T, d = Q.shape
    G = Hq // K.shape[0]
    out = [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (Q, K, V)]
    var = [torch.zeros(x.shape[:2], dtype=torch.float64, device="cuda") for x in (Q, K, V)]
    for a, b in zip(cu, cu[1:]):
        for h in range(Hq):
            q, k, v, do = (x.double() for x in (Q[h, a:b], K[h // G, a:b], V[h // G, a:b], dO[h, a:b]))
            late = torch.ones((b - a, b - a), dtype=torch.bool, device="cuda").triu(1)
            p = torch.softmax((q @ k.T / math.sqrt(d)).masked_fill(late, -math.inf), -1)
            o = p @ v
            ds = p * (do @ v.T - (do * o).sum(-1, keepdim=True))
            out[0][h, a:b] = ds @ k / math.sqrt(d)
            out[1][h // G, a:b] += ds.T @ q / math.sqrt(d)
            out[2][h // G, a:b] += p.T @ do
            e2 = U2 * (do * o).square().sum(-1, keepdim=True)
            f2 = (d / 2 + 2) * 2.0 ** -48 * do.square().sum(-1, keepdim=True) * v.square().sum(-1)
            w = U2 * (ds.square() + 2 * p.square() * e2) + p.square() * f2
            var[0][h, a:b] = w @ k.square().sum(-1) / d
            var[1][h // G, a:b] += w.T @ q.square().sum(-1) / d
            var[2][h // G, a:b] += U2 * p.square().T @ do.square().sum(-1)
    return out, [s + U2 * x.square().sum(-1) for x, s in zip(out, var)]


KINDS = ["plain", "offset 4", "offset 10", "offset 4, keys too", "peaked", "one value", "peaked late"]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,Hq,Hkv", [([512], 2, 2), ([700, 129, 5, 300], 4, 2)], ids=["one", "ragged"])
def test_gradients_where_terms_cancel(kind, lens, Hq, Hkv, d):
    cu, Q, K, V, dO = _make(lens, Hq, Hkv, d, BF16, 5)
    g = torch.Generator().manual_seed(6)
    if "offset" in kind:  # a component that all values of a head share, `offset` times as large as their spread
        V = V + float(kind.split(",")[0].split()[1]) * torch.randn((Hkv, 1, d), generator=g).cuda()
    if "keys" in kind:
        K = K + 2 * torch.randn((Hkv, 1, d), generator=g).cuda()
    if kind == "peaked":
        Q = 16 * Q
    if kind == "peaked late":
        Q = Q * torch.where(torch.arange(Q.shape[1], device="cuda") % 50 == 7, 16.0, 1.0)[None, :, None]
    if kind == "one value":
        V = V[:, :1].expand_as(V)
    Q, K, V, dO = (x.to(BF16) for x in (Q, K, V, dO))
    V = V.contiguous()
    _, _, grads = _train(cu, Q, K, V, dO)
    want, var = _gradients_and_spread(cu, Q, K, V, dO)
    at = torch.cat([torch.arange(b - a) for a, b in zip(cu, cu[1:])]).cuda()
    for got, w, s, name in zip(grads, want, var, ("dQ", "dK", "dV")):
        for part, rows in (("up to row 127", at < 128), ("behind", at >= 128)):
            e, bound = (got.double() - w)[:, rows].norm(), 1.25 * s[:, rows].sum().sqrt()
            assert float(e) <= float(bound), (name, part, float(e), float(bound), float(w[:, rows].norm()))


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF16, 128, 4, 2), (BF16, 64, 3, 3), (F32, 64, 2, 1)])
def test_a_key_that_is_not_a_number(dtype, d, Hq, Hkv):
    """Every position of a NaN among 130 keys, one sequence each, between sequences of numbers: it reaches every
    output and every gradient that depends on it, whatever the position, and no other sequence."""
    L = 130
    lens = [L, 20] * L
    cu, Q, K, V, dO = _make(lens, Hq, Hkv, d, dtype, 7)
    Q, K, V, dO = (x.to(dtype) for x in (Q, K, V, dO))
    want = _train(cu, Q, K, V, dO)
    K = K.clone()
    for j in range(L):
        K[:, cu[2 * j] + j] = float("nan")
    O, lse, (dQ, dK, dV) = _train(cu, Q, K, V, dO)
    for j in range(L):
        a, b = cu[2 * j], cu[2 * j + 1]
        assert torch.equal(O[:, a:a + j], want[0][:, a:a + j]) and torch.equal(lse[:, a:a + j], want[1][:, a:a + j]), j
        assert O[:, a + j:b].isnan().all() and lse[:, a + j:b].isnan().all(), j
        assert dQ[:, a + j:b].isnan().all() and dK[:, a:b].isnan().all() and dV[:, a:b].isnan().all(), j
    clean = torch.cat([torch.arange(cu[i], cu[i + 1]) for i in range(1, 2 * L, 2)]).cuda()
    assert torch.equal(O[:, clean], want[0][:, clean]) and torch.equal(lse[:, clean], want[1][:, clean])
    for x, y in zip((dQ, dK, dV), want[2]):
        assert torch.equal(x[:, clean], y[:, clean])


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF16, 128, 4, 2), (BF16, 64, 3, 3), (F32, 64, 2, 1)])
def test_a_query_that_is_not_a_number(dtype, d, Hq, Hkv):
    """The same for a NaN query: its output, its gradient and those of the keys and values that it sees."""
    L = 130
    lens = [L, 20] * L
    cu, Q, K, V, dO = _make(lens, Hq, Hkv, d, dtype, 8)
    Q, K, V, dO = (x.to(dtype) for x in (Q, K, V, dO))
    want = _train(cu, Q, K, V, dO)
    Q = Q.clone()
    bad = torch.zeros(cu[-1], dtype=torch.bool, device="cuda")
    for j in range(L):
        bad[cu[2 * j] + j] = True
    Q[:, bad] = float("nan")
    O, lse, (dQ, dK, dV) = _train(cu, Q, K, V, dO)
    assert O[:, bad].isnan().all() and lse[:, bad].isnan().all() and dQ[:, bad].isnan().all()
    assert torch.equal(O[:, ~bad], want[0][:, ~bad]) and torch.equal(lse[:, ~bad], want[1][:, ~bad])
    for j in range(L):
        a = cu[2 * j]
        assert dK[:, a:a + j + 1].isnan().all() and dV[:, a:a + j + 1].isnan().all(), j
    clean = torch.cat([torch.arange(cu[i], cu[i + 1]) for i in range(1, 2 * L, 2)]).cuda()
    for x, y in zip((dQ, dK, dV), want[2]):
        assert torch.equal(x[:, clean], y[:, clean])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_delta_of_every_length(dtype, d):
    """delta for sequences of 1 to 140 tokens: a row's sum is exchanged by lanes of a warp whose other rows may be
    behind the sequence's end. dO . O is a sum of d products in fp32 of values exact in it: at most d 2^-24 of the sum
    of their magnitudes off; bf16 then takes sum_k P (dO . v), which is dO . O of the O in double, with P, dO . v and
    their sum in fp32 (the exponents are off by 2^-24 (8 + d / 8) |q||k| / sqrt(d) at most, the exponentials on the FMA
    pipe by 1.0e-4 of themselves, and |dO . v - D| is at most twice |dO| max |v|)."""
    lens = list(range(1, 141))
    cu, Q, K, V, dO = _make(lens, 2, 1, d, dtype, 13)
    Q, K, V, dO = (x.to(dtype) for x in (Q, K, V, dO))
    import hierarchical_block_sparse_pyr_b200 as P

    T = cu[-1]
    s = P.packed_shape(len(lens), T, 2, 1, d, dtype)
    plan = P.packed_plan(s, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    O, lse, delta = torch.empty_like(Q), torch.empty((2, T), device="cuda"), torch.full((2, T), 7.0, device="cuda")
    P.packed_forward(s, Q, K, V, plan, O, lse)
    P.packed_backward(s, Q, K, V, plan, O, lse, dO, delta, *(torch.empty_like(x) for x in (Q, K, V)))
    o, _ = ref.packed(Q, K, V, cu)
    want, size = (dO.double() * o).sum(-1), dO.double().norm(dim=-1) * V.double().norm(dim=-1).max()
    score = Q.double().norm(dim=-1).max() * K.double().norm(dim=-1).max() / math.sqrt(d)
    bound = (2.0 ** -24 * (d + (8 + d / 8) * score) + (2.0e-4 if dtype == BF16 else 0)) * size
    assert ((delta.double() - want).abs() <= bound).all()
