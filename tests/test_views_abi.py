"""Refusals of the strided entry points (rotary positions, packed prompts, drafted trees), and the rotary
frequencies: everything the host decides, without a GPU."""
import ctypes
import math

import pytest
import torch

import _plain64 as ref
import hierarchical_block_sparse_pyr_b200 as P

F32, BF16 = torch.float32, torch.bfloat16


def _v(H, N, d, batch=0, data=64, head=None, row=None):
    return P.PyrView(data, batch, N * d if head is None else head, d if row is None else row)


def _ref(v):
    return None if v is None else ctypes.byref(v)


@pytest.mark.parametrize("rot", [2, 4, 20, 64, 128])
@pytest.mark.parametrize("kw", [{}, dict(scaling="linear", factor=3.0), dict(scaling="ntk", factor=3.0),
                                dict(scaling="yarn", factor=16.0, trained=4096),
                                dict(scaling="yarn", factor=2.0, trained=3)])
def test_rope_frequencies(rot, kw):
    if kw.get("scaling") in ("ntk", "yarn") and rot < 4:
        with pytest.raises(P.PyrError):
            P.rope_spec(128, rot, **kw)
        return
    spec = P.rope_spec(128, rot, base=10000.0, **kw)
    freq, scale = ref.frequencies(rot, 10000.0, **kw)
    assert (spec.d, spec.rot) == (128, rot) and math.isclose(spec.scale, scale, rel_tol=1e-15)
    assert all(math.isclose(a, b, rel_tol=1e-13) for a, b in zip(spec.freq, freq))
    assert all(f == 0 for f in spec.freq[rot // 2:])


def test_rope_scalings_keep_their_ends():
    """The fastest pair of "ntk" and "yarn" keeps its speed, the slowest is slowed by the factor."""
    plain = P.rope_spec(128)
    for kw in (dict(scaling="ntk", factor=4.0), dict(scaling="yarn", factor=4.0, trained=2048)):
        s = P.rope_spec(128, **kw)
        assert math.isclose(s.freq[0], plain.freq[0]) and math.isclose(s.freq[63], plain.freq[63] / 4, rel_tol=1e-12)


@pytest.mark.parametrize("args", [dict(d=96), dict(rot=0), dict(rot=3), dict(rot=130), dict(base=1.0),
                                  dict(base=float("nan")), dict(scaling="linear", factor=0.5),
                                  dict(scaling="yarn", factor=2.0, trained=0), dict(scaling="ntk", factor=float("inf"))])
def test_rope_spec_refusals(args):
    with pytest.raises(P.PyrError):
        P.rope_spec(**{"d": 128, **args})
    with pytest.raises(ValueError):
        P.rope_spec(128, layout="other")


def _rope(spec, B=2, Hq=4, Hkv=2, N=8, dtype=0, Q="q", K="k", pos=64, pos_stride=8, off=0, Qo="q", Ko="k", inv=0):
    mk = {"q": lambda: _v(4, 8, 64, 4 * 8 * 64), "k": lambda: _v(2, 8, 64, 2 * 8 * 64)}
    Q, K, Qo, Ko = (mk[x]() if isinstance(x, str) else x for x in (Q, K, Qo, Ko))
    return P._L().rope_apply(_ref(spec), B, Hq, Hkv, N, dtype, _ref(Q), _ref(K), pos, pos_stride, off, _ref(Qo),
                             _ref(Ko), inv, None, None)


def test_rope_refusals():
    spec = P.rope_spec(64)
    E, U = P.PYR_EINVAL, P.PYR_EUNSUPPORTED
    assert _rope(None) == E
    for kw in (dict(B=0), dict(N=0), dict(Hq=-1), dict(Hq=0), dict(Q=None), dict(Qo=None), dict(K=None),
               dict(Ko=None), dict(Hkv=0), dict(pos=66), dict(pos_stride=7), dict(pos_stride=-8),
               dict(pos=None, off=2 ** 31 - 8 + 1),
               dict(Q=_v(4, 8, 64, 2048, data=72)),            # not 16-byte aligned
               dict(Q=_v(4, 8, 64, 2048, data=None)),
               dict(Q=_v(4, 8, 64, 2048, row=0)),              # a row repeated
               dict(Q=_v(4, 8, 64, 2048, row=66)),             # rows that start off a 16-byte boundary
               dict(Q=_v(4, 8, 64, 2048, head=-512)),
               dict(Qo=_v(4, 8, 64, 2048, head=64, row=64)),   # written rows overlap
               dict(Qo=_v(4, 8, 64, 1024))):                   # written batches overlap
        assert _rope(spec, **kw) == E, kw
    assert _rope(spec, dtype=2) == U
    bad = P.rope_spec(64)
    bad.freq[3] = float("nan")
    assert _rope(bad) == E
    bad = P.rope_spec(64)
    bad.rot = 65
    assert _rope(bad) == E
    bad = P.rope_spec(64)
    bad.d = 80
    assert _rope(bad) == U


def test_packed_refusals():
    lib = P._L()
    E, U = P.PYR_EINVAL, P.PYR_EUNSUPPORTED
    ok = dict(S=3, T=100, Hq=4, Hkv=2, d=64, dtype=BF16)
    s = P.packed_shape(**ok)
    assert P.packed_plan_elems(s) > 0
    for kw, code in ((dict(S=0), E), (dict(T=0), E), (dict(Hq=3), E), (dict(Hkv=0), E), (dict(d=96), U),
                     (dict(dtype=7), U), (dict(T=2 ** 30), U)):
        bad = P.packed_shape(**{**ok, **kw})
        assert P.packed_plan_elems(bad) == 0
        assert lib.packed_plan(ctypes.byref(bad), 64, 64, None, None) == code, kw
        q = ctypes.byref(_v(4, 100, 64))
        assert lib.packed_forward(ctypes.byref(bad), q, q, q, 64, q, 64, None, None) == code, kw
    assert lib.packed_plan(None, 64, 64, None, None) == E
    assert lib.packed_plan(ctypes.byref(s), None, 64, None, None) == E
    assert lib.packed_plan(ctypes.byref(s), 66, 64, None, None) == E
    assert lib.packed_plan(ctypes.byref(s), 64, 72, None, None) == E
    good = [_v(4, 100, 64), _v(2, 100, 64), _v(2, 100, 64), 64, _v(4, 100, 64), 64]

    def fwd(**at):
        a = [at.get(str(i), x) for i, x in enumerate(good)]
        a = [ctypes.byref(x) if isinstance(x, P.PyrView) else x for x in a]
        return lib.packed_forward(ctypes.byref(s), *a, None, None)

    for at in ({"0": None}, {"1": None}, {"2": None}, {"3": None}, {"4": None}, {"3": 72}, {"5": 66},
               {"0": _v(4, 100, 64, data=72)}, {"1": _v(2, 100, 64, row=32)}, {"2": _v(2, 100, 64, row=68)},
               {"4": _v(4, 100, 64, head=64, row=64)}):
        assert fwd(**at) == E, at
    good_b = [_v(4, 100, 64), _v(2, 100, 64), _v(2, 100, 64), 64, _v(4, 100, 64), 64, _v(4, 100, 64), 64,
              _v(4, 100, 64), _v(2, 100, 64), _v(2, 100, 64)]
    for i, x in enumerate(good_b):
        for y in ((None, 66) if isinstance(x, int) else (None, _v(2, 100, 64, data=72))):
            a = list(good_b)
            a[i] = y
            a = [ctypes.byref(z) if isinstance(z, P.PyrView) else z for z in a]
            assert lib.packed_backward(ctypes.byref(s), *a, None, None) == E, (i, y)


def test_tree_refusals():
    lib = P._L()
    E, U = P.PYR_EINVAL, P.PYR_EUNSUPPORTED
    ok = dict(B=2, Hq=4, Hkv=2, N=100, T=5, d=64, dtype=BF16)
    s = P.tree_shape(**ok)
    need = P.tree_workspace_bytes(s)
    assert need > 0
    good = [_v(4, 5, 64, 4 * 5 * 64), _v(2, 100, 64, 2 * 100 * 64), _v(2, 100, 64, 2 * 100 * 64), 64, 64,
            _v(4, 5, 64, 4 * 5 * 64), 64, 64, need]

    def call(shape, a):
        a = [ctypes.byref(z) if isinstance(z, P.PyrView) else z for z in a]
        return lib.tree_forward(ctypes.byref(shape) if shape is not None else None, *a, None, None)

    for kw, code in ((dict(B=0), E), (dict(Hq=3), E), (dict(T=0), E), (dict(N=4), E), (dict(T=65), U),
                     (dict(B=5000), U), (dict(d=80), U), (dict(dtype=3), U), (dict(N=2 ** 29), U)):
        bad = P.tree_shape(**{**ok, **kw})
        assert P.tree_workspace_bytes(bad) == 0 and call(bad, good) == code, kw
    assert call(None, good) == E
    for i, y in ((0, None), (1, None), (2, None), (3, None), (3, 66), (4, 66), (5, None), (6, 66), (7, None), (7, 72),
                 (8, need - 1), (0, _v(4, 5, 64, 1280, data=72)), (1, _v(2, 100, 64, 12800, row=63)),
                 (5, _v(4, 5, 64, 640))):
        a = list(good)
        a[i] = y
        assert call(s, a) == E, (i, y)


def test_python_refusals():
    x = torch.zeros((2, 8, 64))
    s = P.packed_shape(1, 8, 2, 2, 64, F32)
    with pytest.raises(TypeError):
        P.packed_forward(s, x, x, x, x, x)
    with pytest.raises(TypeError):
        P.packed_plan(s, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        P.rope_apply(P.rope_spec(64), x[None], None, x[None], None)
    with pytest.raises(TypeError):
        P.packed_shape(1, 8, 2, 2, 64, torch.float16)
    t = P.tree_shape(1, 2, 2, 8, 1, 64, F32)
    with pytest.raises(TypeError):
        P.tree_forward(t, x[None, :, :1], x[None], x[None], None, None, x[None, :, :1])


class _OnDevice(torch.Tensor):
    """A CPU tensor that says it is on device 0: the host's checks without a GPU."""
    is_cuda = True

    def get_device(self):
        return 0


def _dev(shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)


@pytest.fixture
def stop(monkeypatch):
    """Calls end where the library would be entered."""
    class Reached(Exception):
        pass

    def call(*a):
        raise Reached

    monkeypatch.setattr(P, "_call", call)
    return Reached


def test_shapes_of_plain_operands(stop):
    """Tensors of the right number of elements in another shape, or padded, are refused: the kernels would read
    or write them with the wrong pitch."""
    I = torch.int32
    s = P.packed_shape(3, 8, 4, 2, 64, F32)
    q, k = _dev((4, 8, 64)), _dev((2, 8, 64))
    cu, plan, lse = _dev((4,), I), _dev((P.packed_plan_elems(s),), I), _dev((4, 8))
    with pytest.raises(stop):
        P.packed_plan(s, cu, plan)
    with pytest.raises(stop):
        P.packed_forward(s, q, k, k, plan, q, lse)
    with pytest.raises(stop):
        P.packed_forward(s, q, k, k, _dev((plan.numel() + 100,), I), q)  # a longer buffer holds a plan as well
    with pytest.raises(stop):
        P.packed_backward(s, q, k, k, plan, q, lse, q, lse, q, k, k)
    for bad in (_dev((3,), I), _dev((5,), I), _dev((2, 2), I), _dev((4, 1), I)):
        with pytest.raises(ValueError):
            P.packed_plan(s, bad, plan)
    for bad in (_dev((8, 4)), _dev((4, 10)), _dev((32,)), _dev((1, 4, 8)), _dev((4, 7))):
        with pytest.raises(ValueError):
            P.packed_forward(s, q, k, k, plan, q, bad)
        with pytest.raises(ValueError):
            P.packed_backward(s, q, k, k, plan, q, bad, q, lse, q, k, k)
        with pytest.raises(ValueError):
            P.packed_backward(s, q, k, k, plan, q, lse, q, bad, q, k, k)
    t = P.tree_shape(3, 4, 2, 20, 5, 64, F32)
    q, k = _dev((3, 4, 5, 64)), _dev((3, 2, 20, 64))
    lens, parent, lse = _dev((3,), I), _dev((3, 5), I), _dev((3, 4, 5))
    ws = _dev((P.tree_workspace_bytes(t) + 64,), torch.uint8)
    with pytest.raises(stop):
        P.tree_forward(t, q, k, k, lens, parent, q, lse, ws)
    for bad in (_dev((5, 3), I), _dev((15,), I), _dev((3, 6), I), _dev((4, 5), I)):
        with pytest.raises(ValueError):
            P.tree_forward(t, q, k, k, lens, bad, q, lse, ws)
    for bad in (_dev((4,), I), _dev((3, 1), I)):
        with pytest.raises(ValueError):
            P.tree_forward(t, q, k, k, bad, parent, q, lse, ws)
    for bad in (_dev((3, 5, 4)), _dev((3, 4, 6)), _dev((60,))):
        with pytest.raises(ValueError):
            P.tree_forward(t, q, k, k, lens, parent, q, bad, ws)


def test_integers_that_do_not_fit(stop):
    """The library takes 32-bit integers: one that does not fit is refused, not wrapped into another value."""
    x = _dev((1, 2, 8, 64))
    spec = P.rope_spec(64)
    with pytest.raises(stop):
        P.rope_apply(spec, x, None, x, None, pos_offset=-5)
    for off in (2 ** 32 + 5, -2 ** 31 - 1, 2 ** 31):
        with pytest.raises(ValueError):
            P.rope_apply(spec, x, None, x, None, pos_offset=off)
    for i in range(5):
        a = [1, 8, 2, 2, 64]
        a[i] += 2 ** 32
        with pytest.raises(ValueError):
            P.packed_shape(*a, F32)
    for i in range(6):
        a = [1, 2, 2, 8, 1, 64]
        a[i] += 2 ** 32
        with pytest.raises(ValueError):
            P.tree_shape(*a, F32)
    for kw in (dict(d=2 ** 32 + 64), dict(d=64, rot=2 ** 32 + 32),
               dict(d=64, scaling="yarn", factor=2.0, trained=2 ** 32 + 8192)):
        with pytest.raises(ValueError):
            P.rope_spec(**kw)
    with pytest.raises(ValueError):
        P.packed_shape(1, 8, 2, 2, 64, 2 ** 32)
