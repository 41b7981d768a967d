"""Packed prompts on the GPU against the definition in double.

Tolerances. fp32: scores are d products accumulated in fp32 (error <= d 2^-24 |q||k|/sqrt(d), a few 1e-6
here), so 2e-5 relative to the row's largest |v| for O, 2e-5 for lse and 1e-4 of the tensor's largest
element for the gradients. bf16: the inputs are exact; P (forward), P and dS (backward) are rounded to bf16
once (2^-8 relative each, averaging over the keys), and the outputs are rounded once (2^-8): max-abs error
<= 2^-8 |x| + 2^-7 max over the row's keys of |v| for O; for the gradients relative L2 <= 3 * 2^-8 and
max-abs <= 2^-5 of the largest element; D comes from a bf16 O.

Where dP and D cancel (a row that sees one key has dP = D and a gradient of zero) the error does not scale
with the gradient but with the cancelled terms. dP is a sum of d products in two fp32 chains of d/2: each term
is rounded at most d/2 + 1 times, so |error of dP| <= g A with g = (d/2 + 2) 2^-24 and A = sum |dO||v| over
the row's elements (bf16: the products are exact in fp32, the same bound holds); D has the same bound with
O, |O| <= max |v|. P sums to one over a row, so |error of dQ| <= 2 g A max|k| / sqrt(d), and dK the same with
max|q| and the number of rows that see the key, whose P do not sum to one: each P <= 1. That term is added to
the bounds above (for dK with one row, where it matters; elsewhere the relative bound is the larger one). In
bf16, D is taken from a rounded O: |error of D| <= 2^-9 A more.
"""
import pytest
import torch

import _plain64 as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _tensor(order, H, T, d, dtype, g):
    x = torch.randn((H, T, d), generator=g).to(dtype).cuda()
    return x if order == "hnd" else x.transpose(0, 1).contiguous().transpose(0, 1)


def _batch(lens, pad, Hq, Hkv, d, dtype, order, seed, lead=0):
    g = torch.Generator().manual_seed(seed)
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    T = cu[-1] + pad
    Q, dO = _tensor(order, Hq, T, d, dtype, g), _tensor(order, Hq, T, d, dtype, g)
    K, V = _tensor(order, Hkv, T, d, dtype, g), _tensor(order, Hkv, T, d, dtype, g)
    # tokens of no sequence hold NaN: they must never be used
    for x in (Q, K, V, dO):
        x[:, :lead] = float("nan")
        x[:, cu[-1]:] = float("nan")
    return cu, T, Q, K, V, dO


def _forward(P, cu, T, Q, K, V, fill=7.0):
    s = P.packed_shape(len(cu) - 1, T, Q.shape[0], K.shape[0], Q.shape[2], Q.dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = P.packed_plan(s, torch.tensor(cu, dtype=torch.int32, device="cuda"), status=status)
    O = torch.full_like(Q, fill)
    lse = torch.full((Q.shape[0], T), fill, device="cuda")
    P.packed_forward(s, Q, K, V, plan, O, lse, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    return s, plan, O, lse


CASES = [
    # lens, pad, lead, Hq, Hkv, d, dtype, order
    ([1], 0, 0, 1, 1, 64, F32, "hnd"),
    ([1], 0, 0, 2, 1, 128, BF16, "nhd"),
    ([0, 5, 0, 0, 64, 65, 0], 3, 2, 2, 2, 64, F32, "nhd"),
    ([3, 130, 1, 257, 0], 5, 1, 4, 2, 128, F32, "hnd"),
    ([127, 128, 129, 1, 0, 2], 9, 7, 4, 2, 128, BF16, "nhd"),
    ([255, 256, 257], 1, 0, 3, 3, 128, BF16, "hnd"),
    ([600, 33, 385], 0, 0, 8, 1, 128, BF16, "nhd"),
    ([600, 33, 385], 100, 3, 6, 2, 64, BF16, "nhd"),
    ([1023], 0, 0, 2, 2, 64, BF16, "hnd"),
    ([64] * 40, 0, 0, 2, 1, 64, BF16, "nhd"),
    ([2049, 700], 0, 5, 2, 2, 128, BF16, "hnd"),
    ([1] * 130, 2, 0, 5, 5, 128, BF16, "nhd"),
]
IDS = ["x".join(map(str, c[0][:6])) + "-" + "-".join(map(str, c[1:])) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_against_the_definition(case):
    import hierarchical_block_sparse_pyr_b200 as P

    lens, pad, lead, Hq, Hkv, d, dtype, order = case
    cu, T, Q, K, V, _ = _batch(lens, pad, Hq, Hkv, d, dtype, order, 11, lead)
    _, _, O, lse = _forward(P, cu, T, Q, K, V)
    a, b = cu[0], cu[-1]
    wo, wl = ref.packed(Q, K, V, cu)
    assert (O[:, :a] == 7).all() and (O[:, b:] == 7).all() and (lse[:, :a] == 7).all() and (lse[:, b:] == 7).all()
    if a == b:
        return
    vmax = float(V[:, a:b].abs().max())
    eo = (O[:, a:b].double() - wo[:, a:b]).abs()
    el = (lse[:, a:b].double() - wl[:, a:b]).abs()
    if dtype == F32:
        assert float(eo.max()) <= 2e-5 * vmax and float(el.max()) <= 2e-5
    else:
        assert (eo <= 2.0 ** -8 * wo[:, a:b].abs() + 2.0 ** -7 * vmax).all(), float(eo.max())
        assert float(el.max()) <= 1e-4, float(el.max())


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward_against_the_formula(case):
    import hierarchical_block_sparse_pyr_b200 as P

    lens, pad, lead, Hq, Hkv, d, dtype, order = case
    cu, T, Q, K, V, dO = _batch(lens, pad, Hq, Hkv, d, dtype, order, 12, lead)
    s, plan, O, lse = _forward(P, cu, T, Q, K, V)
    dQ, dK, dV = torch.full_like(Q, 7.0), torch.full_like(K, 7.0), torch.full_like(V, 7.0)
    delta = torch.empty((Hq, T), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.packed_backward(s, Q, K, V, plan, O, lse, dO, delta, dQ, dK, dV, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    a, b = cu[0], cu[-1]
    for x in (dQ, dK, dV):
        assert (x[:, :a] == 7).all() and (x[:, b:] == 7).all()
    if a == b:
        return
    sl = slice(a, b)
    want = ref.packed_grad(Q[:, sl], K[:, sl], V[:, sl], dO[:, sl], [c - a for c in cu])
    for got, w, name in zip((dQ, dK, dV), want, ("dQ", "dK", "dV")):
        e = (got[:, sl].double() - w).abs()
        top = float(w.abs().max())
        A = float(dO[:, sl].abs().double().sum(-1).max() * V[:, sl].abs().double().max())
        A = min(A, float(dO[:, sl].double().norm(dim=-1).max() * V[:, sl].double().norm(dim=-1).max()))
        g = (d / 2 + 2) * 2.0 ** -24 + (2.0 ** -9 / 2 if dtype == BF16 else 0)
        cancelled = 0.0 if name == "dV" else 2 * g * A * float((K if name == "dQ" else Q)[:, sl].abs().max()) / d ** 0.5
        if dtype == F32:
            assert float(e.max()) <= 1e-4 * top + cancelled, (name, float(e.max()), top, cancelled)
        else:
            assert float(e.max()) <= 2.0 ** -5 * top + cancelled, (name, float(e.max()), top, cancelled)
            if float(w.norm()) > 1e-2:
                assert float(e.norm() / w.norm()) <= 3 * 2.0 ** -8, (name, float(e.norm() / w.norm()))
    # the same call again gives the same bits
    again = [torch.full_like(x, 7.0) for x in (dQ, dK, dV)]
    P.packed_backward(s, Q, K, V, plan, O, lse, dO, delta, *again)
    for x, y in zip(again, (dQ, dK, dV)):
        assert torch.equal(x, y)


def test_gradient_against_differences():
    """fp32: (L(x + h u) - L(x - h u)) / 2h along random directions, L from the forward kernel's O in double.

    h = 1e-2: the forward's O carries ~1e-6 relative error, so the quotient's noise is ~1e-6 |L terms| / h,
    and the third-order term is ~h^2: 1 % of the directional derivative's scale covers both."""
    import hierarchical_block_sparse_pyr_b200 as P

    cu, T, Q, K, V, dO = _batch([70, 1, 33], 0, 4, 2, 64, F32, "hnd", 21)
    s, plan, O, lse = _forward(P, cu, T, Q, K, V)
    grads = [torch.empty_like(x) for x in (Q, K, V)]
    P.packed_backward(s, Q, K, V, plan, O, lse, dO, torch.empty((4, T), device="cuda"), *grads)
    g = torch.Generator().manual_seed(4)
    for i in range(3):
        u = torch.randn(grads[i].shape, generator=g).cuda()
        L = []
        for sign in (1, -1):
            x = [Q, K, V]
            x[i] = x[i] + sign * 1e-2 * u
            L.append(float((_forward(P, cu, T, *x)[2].double() * dO.double()).sum()))
        num, ana = (L[0] - L[1]) / 2e-2, float((grads[i].double() * u.double()).sum())
        assert abs(num - ana) <= 1e-2 * float(grads[i].double().norm()) * 2, (i, num, ana)


def test_large_scores_and_long_rows():
    """Scores up to several hundreds: the running maximum moves by far more than the type's range of exponents."""
    import hierarchical_block_sparse_pyr_b200 as P

    for dtype in (F32, BF16):
        cu, T, Q, K, V, _ = _batch([900, 37], 0, 2, 1, 128, dtype, "nhd", 31)
        K = (K.float() * (1 + torch.arange(T, device="cuda").reshape(1, T, 1) % 97)).to(dtype)
        _, _, O, lse = _forward(P, cu, T, Q, K, V)
        wo, wl = ref.packed(Q, K, V, cu)
        # fp32 scores of size 2^9 carry 2^-24 * 2^9 * a few = 1e-4, which moves a probability by as much
        assert float((lse.double() - wl).abs().max()) <= 1e-3
        assert float((O.double() - wo).abs().max()) <= (2e-3 if dtype == F32 else 2.0 ** -6 * float(V.abs().max()))


def test_bad_boundaries_do_nothing_but_report():
    import hierarchical_block_sparse_pyr_b200 as P

    cu, T, Q, K, V, _ = _batch([100, 28], 0, 2, 2, 64, BF16, "hnd", 41)
    s = P.packed_shape(2, T, 2, 2, 64, BF16)
    for bad in ([0, 100, 129], [-1, 100, 128], [0, 101, 100], [0, 2 ** 31 - 1, 128]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        plan = P.packed_plan(s, torch.tensor(bad, dtype=torch.int32, device="cuda"), status=status)
        O = torch.full_like(Q, 3.0)
        P.packed_forward(s, Q, K, V, plan, O, status=status)
        torch.cuda.synchronize()
        assert int(status) == P.PYR_EBADSEQ and (O == 3).all()


def test_packed_under_a_graph():
    import hierarchical_block_sparse_pyr_b200 as P

    cu, T, Q, K, V, dO = _batch([300, 40, 129], 4, 4, 2, 128, BF16, "nhd", 51)
    s, plan, O, lse = _forward(P, cu, T, Q, K, V)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    delta = torch.empty((4, T), device="cuda")
    grads = [torch.zeros_like(x) for x in (Q, K, V)]
    P.packed_backward(s, Q, K, V, plan, O, lse, dO, delta, *grads)
    O2, lse2, g2 = torch.full_like(O, 7.0), torch.full_like(lse, 7.0), [torch.zeros_like(x) for x in grads]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.packed_plan(s, cut, plan)
        P.packed_forward(s, Q, K, V, plan, O2, lse2)
        P.packed_backward(s, Q, K, V, plan, O2, lse2, dO, delta, *g2)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    for x, y in zip(grads, g2):
        assert torch.equal(x, y)


def test_a_plan_of_another_shape_does_nothing_but_report():
    import hierarchical_block_sparse_pyr_b200 as P

    cu, T, Q, K, V, dO = _batch([100, 28], 0, 2, 2, 64, BF16, "hnd", 61)
    s, plan, O, lse = _forward(P, cu, T, Q, K, V)
    other = P.packed_shape(2, T, 2, 2, 64, F32)
    foreign = torch.zeros(max(P.packed_plan_elems(s), P.packed_plan_elems(other)), dtype=torch.int32, device="cuda")
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for buf in (P.packed_plan(other, cut, foreign), torch.full_like(foreign, 2 ** 31 - 1)):
        for call in ("forward", "backward"):
            out = [torch.full_like(x, 3.0) for x in (Q, Q, K, V)]
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            if call == "forward":
                P.packed_forward(s, Q, K, V, buf, out[0], status=status)
            else:
                P.packed_backward(s, Q, K, V, buf, O, lse, dO, torch.empty_like(lse), *out[1:], status=status)
            torch.cuda.synchronize()
            assert int(status) == P.PYR_EBADSEQ and all((x == 3).all() for x in out)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_views_into_larger_tensors(dtype, d):
    """Q, K and V as slices of one projection [T, Hq + 2 Hkv, d] with a padded row, outputs in another layout."""
    import hierarchical_block_sparse_pyr_b200 as P

    Hq, Hkv, lens = 6, 3, [200, 1, 77]
    T = sum(lens)
    g = torch.Generator().manual_seed(71)
    wide = torch.randn((T, Hq + 2 * Hkv, d + 8), generator=g).to(dtype).cuda()
    x = wide[..., 8:].transpose(0, 1)  # rows start 16 or 32 bytes into their pitch
    Q, K, V = x[:Hq], x[Hq:Hq + Hkv], x[Hq + Hkv:]
    cu = [0, 200, 201, 278]
    s = P.packed_shape(3, T, Hq, Hkv, d, dtype)
    plan = P.packed_plan(s, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    O = torch.empty((Hq, T, d), dtype=dtype, device="cuda")
    lse = torch.empty((Hq, T), device="cuda")
    P.packed_forward(s, Q, K, V, plan, O, lse)
    O2 = torch.empty((T, Hq, d), dtype=dtype, device="cuda").transpose(0, 1)
    P.packed_forward(s, Q.contiguous(), K.contiguous(), V.contiguous(), plan, O2)
    assert torch.equal(O, O2)
    wo, _ = ref.packed(Q, K, V, cu)
    assert float((O.double() - wo).abs().max()) <= (2e-5 if dtype == F32 else 2.0 ** -7) * float(V.abs().max()) * 2
    dO = torch.randn((T, Hq, d), generator=g).to(dtype).cuda().transpose(0, 1)
    grad = torch.zeros_like(wide)  # the gradient of the projection, written through the same slices
    gx = grad[..., 8:].transpose(0, 1)
    P.packed_backward(s, Q, K, V, plan, O, lse, dO, torch.empty_like(lse), gx[:Hq], gx[Hq:Hq + Hkv], gx[Hq + Hkv:])
    plain = [torch.empty_like(t) for t in (O, K.contiguous(), V.contiguous())]
    P.packed_backward(s, Q.contiguous(), K.contiguous(), V.contiguous(), plan, O, lse, dO.contiguous(),
                      torch.empty_like(lse), *plain)
    assert torch.equal(gx[:Hq], plain[0]) and torch.equal(gx[Hq:Hq + Hkv], plain[1])
    assert torch.equal(gx[Hq + Hkv:], plain[2]) and (grad[..., :8] == 0).all()


def test_two_batches_on_two_streams():
    import hierarchical_block_sparse_pyr_b200 as P

    jobs = []
    for seed, lens in ((81, [700, 40, 1300]), (82, [1025, 3, 511])):
        cu, T, Q, K, V, dO = _batch(lens, 0, 8, 2, 128, BF16, "nhd", seed)
        s, plan, O, lse = _forward(P, cu, T, Q, K, V)
        want = [torch.empty_like(x) for x in (Q, K, V)]
        P.packed_backward(s, Q, K, V, plan, O, lse, dO, torch.empty_like(lse), *want)
        jobs.append((torch.cuda.Stream(), s, plan, (Q, K, V), dO, O, lse, want))
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for st, s, plan, x, dO, O, lse, want in jobs:
            o, z, dl = torch.zeros_like(O), torch.zeros_like(lse), torch.zeros_like(lse)
            gr = [torch.zeros_like(t) for t in x]
            got.append((o, z, gr, dl))
        torch.cuda.synchronize()
        for (st, s, plan, x, dO, O, lse, want), (o, z, gr, dl) in zip(jobs, got):
            P.packed_forward(s, *x, plan, o, z, stream=st)
            P.packed_backward(s, *x, plan, o, z, dO, dl, *gr, stream=st)
        torch.cuda.synchronize()
        for (st, s, plan, x, dO, O, lse, want), (o, z, gr, dl) in zip(jobs, got):
            assert torch.equal(o, O) and torch.equal(z, lse) and all(torch.equal(a, b) for a, b in zip(gr, want))


def test_rotate_attend_and_train_in_one_stream():
    """The operators as they are used: rotate Q and K at positions that restart with every sequence, attend,
    differentiate, rotate the gradients back. Against the definitions in double end to end."""
    import hierarchical_block_sparse_pyr_b200 as P

    lens, Hq, Hkv, d = [300, 5, 190], 4, 2, 64
    cu, T, Q, K, V, dO = _batch(lens, 0, Hq, Hkv, d, F32, "nhd", 91)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    spec = P.rope_spec(d, 32, layout="interleaved", scaling="yarn", factor=2.0, trained=128)
    freq, scale = ref.frequencies(32, 10000.0, "yarn", 2.0, 128)
    Qr, Kr = torch.empty_like(Q), torch.empty_like(K)
    P.rope_apply(spec, Q[None], K[None], Qr[None], Kr[None], pos=pos)
    s, plan, O, lse = _forward(P, cu, T, Qr, Kr, V)
    dQ, dK, dV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
    P.packed_backward(s, Qr, Kr, V, plan, O, lse, dO, torch.empty((Hq, T), device="cuda"), dQ, dK, dV)
    P.rope_apply(spec, dQ[None], dK[None], dQ[None], dK[None], pos=pos, inverse=True)
    q64, k64 = (ref.rope(x[None], pos[None], freq, scale, 32, "interleaved")[0] for x in (Q, K))
    wo, _ = ref.packed(q64, k64, V, cu)
    # the fp32 bounds above; the rotation adds 7e-7 relative per element, far below them
    assert float((O.double() - wo).abs().max()) <= 2e-5 * float(V.abs().max())
    want = list(ref.packed_grad(q64, k64, V, dO, cu))
    for i in range(2):
        want[i] = ref.rope(want[i][None], pos[None], freq, scale, 32, "interleaved", inverse=True)[0]
    for got, w in zip((dQ, dK, dV), want):
        assert float((got.double() - w).abs().max()) <= 2e-4 * float(w.abs().max())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_single_tokens_have_no_score_gradient(dtype):
    """A token alone in its sequence: dQ and dK are zero, exactly, and dV is dO summed over the group."""
    import hierarchical_block_sparse_pyr_b200 as P

    for d in (64, 128):
        cu, T, Q, K, V, dO = _batch([1] * 150, 0, 4, 2, d, dtype, "nhd", 95)
        s, plan, O, lse = _forward(P, cu, T, Q, K, V)
        grads = [torch.full_like(x, 7.0) for x in (Q, K, V)]
        P.packed_backward(s, Q, K, V, plan, O, lse, dO, torch.empty_like(lse), *grads)
        assert (grads[0] == 0).all() and (grads[1] == 0).all()
        want = dO.double().reshape(2, 2, T, d).sum(1)
        # P = 1 up to a few fp32 roundings of the score; bf16: exactly 1, and one rounding of the output
        eps = 2.0 ** -8 if dtype == BF16 else 2e-6
        assert ((grads[2].double() - want).abs() <= eps * want.abs() + 2e-6 * dO.abs().max()).all()


@pytest.mark.parametrize("lens", [[2] * 60, [3, 5, 2, 9, 4, 17, 1, 6], [40, 128, 100]])
def test_gradients_of_short_sequences(lens):
    """Few keys a row: dP and delta nearly cancel, and delta from a rounded O would leave its rounding. With delta
    refined, dS carries its own rounding and those of the fp32 sums: the bf16 relative bound of the module holds."""
    import hierarchical_block_sparse_pyr_b200 as P

    for d in (64, 128):
        cu, T, Q, K, V, dO = _batch(lens, 3, 4, 2, d, BF16, "hnd", 96)
        s, plan, O, lse = _forward(P, cu, T, Q, K, V)
        grads = [torch.full_like(x, 7.0) for x in (Q, K, V)]
        P.packed_backward(s, Q, K, V, plan, O, lse, dO, torch.empty_like(lse), *grads)
        e = cu[-1]
        want = ref.packed_grad(Q[:, :e], K[:, :e], V[:, :e], dO[:, :e], cu)
        for got, w in zip(grads, want):
            # two bf16 roundings, each at most 2^-8 of the value
            assert float((got[:, :e].double() - w).norm() / w.norm()) <= 2 * 2.0 ** -8
