"""CPU checks of the rotary and norm entry points: the oracle against other
formulations and finite differences, and every refusal of the C ABI and of the
binding (bad arguments never reach a kernel)."""
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
@pytest.mark.parametrize("interleaved", [True, False])
def test_oracle_rotation_is_a_rotation_and_relative(interleaved):
    rng = np.random.default_rng(0)
    pos = rng.integers(-50, 50, (9, 3))
    ang = po.angles(pos, (16, 8, 8))
    x, y = rng.standard_normal((2, 9, 40))
    a, b = po.rotate(x, ang, interleaved), po.rotate(y, ang, interleaved)
    assert np.allclose((a * b).sum(-1), (x * y).sum(-1))               # the same turn keeps products
    assert np.allclose(po.rotate(a, -ang, interleaved), x)             # and the opposite one undoes it
    assert np.array_equal(a[:, 32:], x[:, 32:])                        # channels past the sections stay
    shift = po.angles(pos + np.array([3, -2, 7]), (16, 8, 8))
    c, d = po.rotate(x, shift, interleaved), po.rotate(y[:1], shift[:1], interleaved)
    e = po.rotate(y[:1], ang[:1], interleaved)
    assert np.allclose((c * d).sum(-1), (a * e).sum(-1))               # products see differences of positions only


def test_oracle_shared_table_and_pairs_by_hand():
    pos = np.array([[2.0, 5.0]])
    ang = po.angles(pos, (4, 2), base=100.0, scale=(1.0, 0.5), shared=True)
    f = [100.0 ** (-2 * j / 6) for j in range(3)]
    assert np.allclose(ang[0], [2 * f[0], 2 * f[1], 2.5 * f[2]])
    x = np.arange(1.0, 9.0)[None]
    y = po.rotate(x, ang, False)                                       # pairs (0, 3), (1, 4), (2, 5)
    for j in range(3):
        c, s = np.cos(ang[0, j]), np.sin(ang[0, j])
        assert np.allclose([y[0, j], y[0, j + 3]], [x[0, j] * c - x[0, j + 3] * s, x[0, j] * s + x[0, j + 3] * c])


def test_oracle_norm_gradients_by_differences():
    rng = np.random.default_rng(1)
    ang = po.angles(rng.integers(0, 99, (5, 3)), (6, 4, 4))
    x, w, dy = rng.standard_normal((2, 5, 16)), rng.standard_normal(16), rng.standard_normal((2, 5, 16))
    dx, dw = po.norm_rotate_backward(x, w, 1e-3, ang, True, dy)
    loss = lambda x, w: (po.norm_rotate(x, w, 1e-3, ang, True) * dy).sum()  # noqa: E731
    h = 1e-6
    for at in [(0, 0, 0), (1, 4, 15), (0, 3, 7)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for d in (0, 5, 15):
        e = np.zeros_like(w)
        e[d] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[d]) < 1e-7


# ---------------------------------------------------------------- C ABI
def _call(lib, fn="vsa_rope", sizes=None, rot=None, where=None, q=None, k=None, q_out=None, k_out=None, eps=1e-6,
          wq=None, dy=None, ws=(16, 1 << 30)):
    sizes = vsa.RopeSizes(0, 2, 64, 64) if sizes is None else sizes
    rot = vsa.Rotation(64, (24, 20, 20)).spec if rot is None else rot
    where = vsa.Positions(4, 4, 4) if where is None else where
    ok = lambda: vsa.Heads(1 << 20, 3, 3 * 64 * 64, 64 * 64, 64)  # noqa: E731
    q, q_out = ok() if q is None else q, ok() if q_out is None else q_out
    if fn == "vsa_rope":
        return lib.vsa_rope(sizes, rot, where, q, k, q_out, k_out, None)
    if fn == "vsa_qk_norm_rope":
        return lib.vsa_qk_norm_rope(sizes, rot, where, q, k, wq, None, eps, q_out, k_out, None)
    return lib.vsa_qk_norm_rope_backward(sizes, rot, where, q, k, wq, None, eps, q if dy is None else dy, None, q_out,
                                         k_out, None, None, *ws, None)


def _rot(**kw):
    r = vsa.Rotation(64, (24, 20, 20)).spec
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _heads(**kw):
    d = dict(data=1 << 20, heads=3, s_b=3 * 64 * 64, s_h=64 * 64, s_n=64)
    d.update(kw)
    return vsa.Heads(*(d[n] for n, _ in vsa.Heads._fields_))


@pytest.mark.parametrize("fn", ["vsa_rope", "vsa_qk_norm_rope", "vsa_qk_norm_rope_backward"])
@pytest.mark.parametrize("kw,code", [
    (dict(sizes=vsa.RopeSizes(3, 2, 64, 64)), 3), (dict(sizes=vsa.RopeSizes(-1, 2, 64, 64)), 3),
    (dict(sizes=vsa.RopeSizes(0, -1, 64, 64)), 2), (dict(sizes=vsa.RopeSizes(0, 2, -64, 64)), 2),
    (dict(sizes=vsa.RopeSizes(0, 2, 64, 60)), 3), (dict(sizes=vsa.RopeSizes(0, 2, 64, 264)), 3),
    (dict(sizes=vsa.RopeSizes(0, 2, 64, 0)), 3), (dict(sizes=vsa.RopeSizes(0, 2, 65, 64)), 2),
    (dict(rot=_rot(rot=66)), 2), (dict(rot=_rot(rot=-2)), 2), (dict(rot=_rot(rot=63)), 2),
    (dict(rot=_rot(rot=40, interleaved=0)), 3), (dict(rot=_rot(axes=0)), 3), (dict(rot=_rot(axes=5)), 3),
    (dict(rot=_rot(axes=2)), 1),                                        # axis 2 is named but there are two
    (dict(where=vsa.Positions(4, 4, 0)), 2), (dict(where=vsa.Positions(4, 8, 4)), 2),
    (dict(where=vsa.Positions(-4, -4, 4)), 2),
    (dict(where=vsa.Positions(1 << 30, 1 << 30, 64)), 2),               # the product passes 64 bits
    (dict(where=vsa.Positions(list=1 << 20, list_type=2)), 3),
    (dict(where=vsa.Positions(list=(1 << 20) + 2, list_type=0)), 4),
    (dict(where=vsa.Positions(list=1 << 20, list_type=0, list_batch=-3)), 1),
    (dict(q=_heads(heads=-1)), 2), (dict(q=_heads(heads=2)), 2), (dict(q=_heads(heads=1 << 17), q_out=_heads(heads=1 << 17)), 3),
    (dict(q=_heads(data=None)), 1), (dict(q_out=_heads(data=None)), 1),
    (dict(q=_heads(data=(1 << 20) + 8)), 4), (dict(q_out=_heads(data=(1 << 20) + 2)), 4),
    (dict(q=_heads(s_n=68)), 4), (dict(q_out=_heads(s_h=4)), 4), (dict(q=_heads(s_b=-64)), 1),
    (dict(q_out=_heads(s_n=0)), 1), (dict(q=_heads(s_b=1 << 41)), 3),
    (dict(k=_heads()), 1), (dict(k_out=_heads()), 1),
])
def test_refusals(lib, fn, kw, code):
    assert _call(lib, fn, **kw) == code


def test_refusals_of_sizes_beyond_the_limits(lib):
    listed = vsa.Positions(list=1 << 20, list_type=0)
    for sizes in (vsa.RopeSizes(0, 1, (1 << 30) + 1, 64), vsa.RopeSizes(0, 1 << 14, 1 << 20, 64),
                  vsa.RopeSizes(0, (1 << 20) + 1, 1, 64)):
        assert _call(lib, sizes=sizes, where=listed) == 3


def test_refusals_of_missing_structs_and_bad_numbers(lib):
    s, r, w, h = vsa.RopeSizes(0, 2, 64, 64), vsa.Rotation(64, (24, 20, 20)).spec, vsa.Positions(4, 4, 4), _heads()
    assert lib.vsa_rope(None, r, w, h, None, h, None, None) == 1
    assert lib.vsa_rope(s, None, w, h, None, h, None, None) == 1
    assert lib.vsa_rope(s, r, None, h, None, h, None, None) == 1
    assert lib.vsa_rope(s, r, w, None, None, None, None, None) == 1
    r.freq[5] = float("nan")
    assert lib.vsa_rope(s, r, w, h, None, h, None, None) == 1
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _call(lib, "vsa_qk_norm_rope", eps=eps) == 1
        assert _call(lib, "vsa_qk_norm_rope_backward", eps=eps) == 1
    assert _call(lib, "vsa_qk_norm_rope", wq=(1 << 20) + 4) == 4
    # strides of dimensions of length 1 are not looked at; a call without rows does nothing
    assert _call(lib, sizes=vsa.RopeSizes(0, 0, 64, 64)) == 0
    assert _call(lib, sizes=vsa.RopeSizes(0, 2, 64, 64), q=_heads(heads=0, data=None), q_out=_heads(heads=0)) == 0
    assert lib.vsa_qk_norm_rope_backward_workspace_bytes(60) == 0


# ---------------------------------------------------------------- binding
def test_rotation_refusals():
    R = vsa.Rotation
    for bad in (dict(sections=(3, 2)), dict(sections=()), dict(sections=(2,) * 5), dict(sections=(66,)),
                dict(sections=(-2, 4)), dict(sections=(20, 20), interleaved=False), dict(sections=(4,), base=0),
                dict(sections=(4, 4), scale=(1.0,))):
        with pytest.raises(ValueError):
            R(64, **bad)
    r = R(64, (8, 4, 4), base=100.0, scale=(1, 2, 1))
    assert [r.spec.axis[j] for j in range(8)] == [0, 0, 0, 0, 1, 1, 2, 2]
    assert np.allclose([r.spec.freq[j] for j in range(6)], [1, 100 ** -.25, 100 ** -.5, 100 ** -.75, 2, 2 * 100 ** -.5])


class _FakeCuda(torch.Tensor):
    @property
    def is_cuda(self):
        return True


def _fake(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_FakeCuda)


def test_binding_refusals():
    r = vsa.Rotation(64, (24, 20, 20))
    q, k = _fake(2, 3, 8, 64), _fake(2, 1, 8, 64)
    g = dict(grid=(2, 2, 2))
    bad = [
        (dict(q=torch.zeros(2, 3, 8, 64)), "CUDA"), (dict(q=q[0]), "shape"), (dict(k=k[:1]), "shape"),
        (dict(q=q.double()), "float"), (dict(k=k.float()), "bfloat16"), (dict(rotation=vsa.Rotation(128, (4,))), "128"),
        (dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), "contiguous channels"),
        (dict(grid=(2, 2, 3)), "T\\*H\\*W"), (dict(grid=None), "either"), (dict(grid=(8, 1)), "three"),
        (dict(origin=(2 ** 31, 0, 0)), "32 bits"),
        (dict(positions=_fake(8, 3, dtype=torch.int32)), "either"),
        (dict(grid=None, positions=torch.zeros(8, 3, dtype=torch.int32)), "CUDA"),
        (dict(grid=None, positions=_fake(8, 3, dtype=torch.int64)), "int32 or float32"),
        (dict(grid=None, positions=_fake(8, 2, dtype=torch.int32)), "shape"),
        (dict(grid=None, positions=_fake(3, 8, 3, dtype=torch.int32)), "shape"),
        (dict(grid=None, positions=_fake(3, 8, dtype=torch.int32).t()), "contiguous"),
    ]
    for change, match in bad:
        a = dict(q=q, k=k, rotation=r, **g)
        a.update(change)
        for fn, more in ((vsa.rope, {}), (vsa.qk_norm_rope, dict(q_weight=None, k_weight=None))):
            with pytest.raises(ValueError, match=match):
                fn(**a, **more)
    with pytest.raises(ValueError, match="q_weight"):
        vsa.qk_norm_rope(q, k, _fake(32, dtype=torch.float32), None, r, **g)
    with pytest.raises(ValueError, match="q_weight"):
        vsa.qk_norm_rope(q, k, _fake(64), None, r, **g)
    with pytest.raises(ValueError, match="dq_out"):
        vsa.qk_norm_rope_backward(q, k, None, None, k, k, r, **g)
    with pytest.raises(ValueError, match="together"):
        vsa.qk_norm_rope_backward(q, k, None, None, q, None, r, **g)
