"""CPU checks of the linear product's entry points: the oracle against torch's formulas and differences, and every
refusal of the C ABI and of the binding (bad arguments never reach a kernel)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import projection_oracle as po
from trainable_block_sparse_cube_b200 import build as vsa_build
from trainable_block_sparse_cube_b200 import vsa


@pytest.fixture(scope="module")
def lib():
    vsa_build.build()
    return vsa.load()


# ---------------------------------------------------------------- oracle
FORMULAS = {None: lambda z: z, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
            "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}


@pytest.mark.parametrize("act", FORMULAS)
def test_oracle_against_torch(act):
    rng = np.random.default_rng(0)
    x, w, b = rng.standard_normal((2, 3, 5, 4)), rng.standard_normal((6, 12)), rng.standard_normal(6)
    res, dout = rng.standard_normal((2, 5, 6)), rng.standard_normal((2, 5, 6))
    y, z = po.linear(x, w, b, act, res)
    tx, tw, tb = (torch.from_numpy(t).requires_grad_(True) for t in (x, w, b))
    tz = torch.nn.functional.linear(tx.transpose(1, 2).flatten(2), tw, tb)
    ty = FORMULAS[act](tz) + torch.from_numpy(res)
    assert np.allclose(y, ty.detach().numpy()) and np.allclose(z, tz.detach().numpy())
    dx, dw, db = po.linear_backward(x, w, dout, z, act)
    gx, gw, gb = torch.autograd.grad(ty, (tx, tw, tb), torch.from_numpy(dout))
    assert np.allclose(dx, po.rows(gx.numpy())) and np.allclose(dw, gw.numpy()) and np.allclose(db, gb.numpy())


@pytest.mark.parametrize("act", FORMULAS)
def test_oracle_slope_by_differences(act):
    z = np.linspace(-6, 6, 49)
    h = 1e-5
    assert np.allclose((po.activate(z + h, act) - po.activate(z - h, act)) / (2 * h), po.slope(z, act), atol=1e-8)


# ---------------------------------------------------------------- C ABI
def _sizes(**kw):
    d = dict(type=0, B=2, N=64, K=128, F=256)
    d.update(kw)
    return vsa.LinearSizes(*(d[n] for n, _ in vsa.LinearSizes._fields_))


def _view(channels, heads=1, **kw):
    D = channels // max(heads, 1)
    d = dict(data=1 << 20, heads=heads, s_b=64 * channels, s_h=64 * D, s_n=D)
    d.update(kw)
    return vsa.Heads(*(d[n] for n, _ in vsa.Heads._fields_))


def _forward(lib, sizes=None, x=None, w=1 << 20, stride=128, bias=None, act=0, res=None, z=None, out=None,
             ws=(1 << 20, 1 << 40)):
    return lib.vsa_linear(_sizes() if sizes is None else sizes, _view(128) if x is None else x, w, stride, bias, act,
                          res, z, _view(256) if out is None else out, *ws, None)


def _backward(lib, sizes=None, x=None, w=1 << 20, stride=128, z=None, act=0, dout=None, dx=None, dw=1 << 20, db=None,
              ws=(1 << 20, 1 << 40)):
    return lib.vsa_linear_backward(_sizes() if sizes is None else sizes, _view(128) if x is None else x, w, stride, z,
                                   act, _view(256) if dout is None else dout, _view(128) if dx is None else dx, dw, db,
                                   *ws, None)


@pytest.mark.parametrize("call", [_forward, _backward])
@pytest.mark.parametrize("kw,code", [
    (dict(sizes=_sizes(type=2)), 3), (dict(sizes=_sizes(type=-1)), 3), (dict(sizes=_sizes(B=-1)), 2),
    (dict(sizes=_sizes(N=-1)), 2), (dict(sizes=_sizes(K=0)), 2), (dict(sizes=_sizes(F=-8)), 2),
    (dict(sizes=_sizes(K=100)), 3), (dict(sizes=_sizes(F=12)), 3), (dict(sizes=_sizes(F=1 << 21)), 3),
    (dict(sizes=_sizes(B=1 << 12, N=1 << 19)), 3),
    (dict(act=4), 3), (dict(act=-1), 3),
    (dict(w=None), 1), (dict(w=(1 << 20) + 8), 4), (dict(stride=120), 1), (dict(stride=132), 4),
    (dict(stride=1 << 39), 3),
    (dict(x=_view(128, data=None)), 1), (dict(x=_view(128, data=(1 << 20) + 8)), 4), (dict(x=_view(128, heads=0)), 2),
    (dict(x=_view(128, heads=3)), 2), (dict(x=_view(128, heads=4)), 3), (dict(x=_view(128, s_n=132)), 4),
    (dict(x=_view(128, s_b=-64)), 1), (dict(x=_view(128, s_b=1 << 39)), 3),
])
def test_refusals(lib, call, kw, code):
    assert call(lib, **kw) == code


def test_refusals_of_one_direction(lib):
    for kw, code in ((dict(out=_view(256, data=None)), 1), (dict(out=_view(256, s_n=0)), 1),
                     (dict(out=_view(256, heads=8)), 3), (dict(res=_view(256, heads=2)), 2),
                     (dict(res=_view(256, data=(1 << 20) + 2)), 4), (dict(z=_view(256, heads=2)), 2),
                     (dict(z=_view(256, s_n=0)), 1), (dict(bias=(1 << 20) + 4), 4)):
        assert _forward(lib, **kw) == code
    for kw, code in ((dict(dx=_view(128, s_n=0)), 1), (dict(dx=_view(128, data=None)), 1), (dict(act=1), 1),
                     (dict(act=1, z=_view(256, heads=2)), 2), (dict(act=1, z=_view(256, data=None)), 1),
                     (dict(dout=_view(256, heads=8)), 3), (dict(dw=(1 << 20) + 8), 4), (dict(db=(1 << 20) + 4), 4)):
        assert _backward(lib, **kw) == code
    s, v, o = _sizes(), _view(128), _view(256)
    assert lib.vsa_linear(None, v, 1 << 20, 128, None, 0, None, None, o, None, 0, None) == 1
    assert lib.vsa_linear(s, None, 1 << 20, 128, None, 0, None, None, o, None, 0, None) == 1
    assert lib.vsa_linear(s, v, 1 << 20, 128, None, 0, None, None, None, None, 0, None) == 1
    assert lib.vsa_linear_backward(s, v, 1 << 20, 128, None, 0, None, v, None, None, None, 0, None) == 1
    assert _forward(lib, sizes=_sizes(N=0)) == 0 and _forward(lib, sizes=_sizes(B=0)) == 0     # nothing to do
    assert lib.vsa_linear_workspace_bytes(_sizes(K=100)) == 0
    assert lib.vsa_linear_backward_workspace_bytes(_sizes(), 9) == 0
    assert lib.vsa_linear_set_limits(0, 0) == 1


# ---------------------------------------------------------------- binding
class _FakeCuda(torch.Tensor):
    @property
    def is_cuda(self):
        return True


def _fake(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_FakeCuda)


def test_binding_refusals():
    x, w = _fake(2, 8, 64), _fake(24, 64)
    bad = [
        (dict(x=torch.zeros(2, 8, 64)), "CUDA"), (dict(x=x.float()), "float16"), (dict(x=x[0]), "shape"),
        (dict(x=x.transpose(1, 2)), "contiguous channels"), (dict(weight=torch.zeros(24, 64)), "weight"),
        (dict(weight=w.half()), "weight"), (dict(weight=w[:, :56]), "weight"), (dict(weight=w.t()), "weight"),
        (dict(weight=_fake(64, 24).t()), "contiguous rows"), (dict(activation="relu"), "activation"),
    ]
    for change, match in bad:
        a = dict(x=x, weight=w)
        a.update(change)
        with pytest.raises(ValueError, match=match):
            vsa.linear(**a)
        with pytest.raises(ValueError, match=match):
            vsa.linear_backward(dout=_fake(2, 8, 24), **a)
    for change, match in [
        (dict(bias=_fake(24)), "bias"), (dict(bias=_fake(16, dtype=torch.float32)), "bias"),
        (dict(residual=_fake(2, 8, 16)), "residual"), (dict(residual=_fake(2, 8, 24, dtype=torch.float32)), "residual"),
        (dict(out=_fake(2, 1, 8, 24)), "out"), (dict(z=_fake(2, 8, 16)), "z"), (dict(heads=5), "heads"),
        (dict(heads=0), "heads"), (dict(heads=3, residual=_fake(2, 8, 24)), "residual"),
    ]:
        with pytest.raises(ValueError, match=match):
            vsa.linear(x, w, **change)
    for change, match in [
        (dict(dout=_fake(2, 8, 16)), "dout"), (dict(dout=_fake(2, 8, 24).float()), "dout"),
        (dict(activation="silu"), "z"),
        (dict(activation="silu", z=_fake(2, 8, 16)), "z"), (dict(dx=_fake(2, 8, 24)), "dx"),
    ]:
        with pytest.raises(ValueError, match=match):
            vsa.linear_backward(x, w, **{**dict(dout=_fake(2, 8, 24)), **change})


def test_packed_structs_match_the_declared_ones():
    """The bytes the binding passes are the structures' own."""
    assert vsa._pack_heads(1 << 33, 3, 1 << 35, 5, 7) == bytes(vsa.Heads(1 << 33, 3, 1 << 35, 5, 7))
    assert vsa._pack_linear_sizes(1, 2, 3, 4, 5) == bytes(vsa.LinearSizes(1, 2, 3, 4, 5))
    assert vsa._pack_rope_sizes(1, 2, 3, 4) == bytes(vsa.RopeSizes(1, 2, 3, 4))
    assert vsa._pack_positions(1, 2, 3, -4, 5, 6, 1 << 40, 1, 1 << 34) == \
        bytes(vsa.Positions(1, 2, 3, (ctypes.c_int * 3)(-4, 5, 6), 1 << 40, 1, 1 << 34))
