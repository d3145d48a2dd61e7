"""Calls of the projection side that its documentation allows at the edges of their arguments."""
from concurrent.futures import ThreadPoolExecutor
from fractions import Fraction

import pytest
import torch

from trainable_block_sparse_cube_b200 import build as vsa_build
from trainable_block_sparse_cube_b200 import vsa

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    vsa_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vsa.load()


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    vsa.linear_check()


def _randn(seed, *shape, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _odd(x, stride):
    """x with another stride in its dimensions of length 1, which no address may come from."""
    return x.as_strided(x.shape, [stride if n == 1 else s for n, s in zip(x.shape, x.stride())])


@pytest.mark.parametrize("stride", [1, 3, 2 ** 33 + 5])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 70), (2, 1, 33), (2, 3, 1), (1, 5, 1)], ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_strides_of_dimensions_of_length_one(dtype, shape, stride):
    B, h, N = shape
    q, k, dq, dk = (_randn(i, B, n, N, 64, dtype=dtype) for i, n in enumerate((h, 1, h, 1)))
    odd = [_odd(t, stride) for t in (q, k, dq, dk)]
    w = _randn(9, 64, dtype=torch.float32)
    rot = vsa.Rotation(64, (24, 20, 20))
    kw = dict(grid=(1, 1, N))
    for fn in (vsa.rope, vsa.rope_backward):
        ref, got = fn(q, k, rot, **kw), fn(odd[0], odd[1], rot, **kw)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    ref, got = (vsa.qk_norm_rope(*a, w, None, rot, **kw) for a in ((q, k), odd[:2]))
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    ref = vsa.qk_norm_rope_backward(q, k, w, w, dq, dk, rot, **kw)
    got = vsa.qk_norm_rope_backward(odd[0], odd[1], w, w, odd[2], odd[3], rot, **kw)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    out = [torch.empty_like(q), torch.empty_like(k)]
    vsa.rope(q, k, rot, q_out=_odd(out[0], stride), k_out=_odd(out[1], stride), **kw)
    assert all(torch.equal(a, b) for a, b in zip(out, vsa.rope(q, k, rot, **kw)))
    if dtype != torch.float32:
        weight = _randn(10, 72, h * 64, dtype=dtype)
        assert torch.equal(vsa.linear(odd[0], weight), vsa.linear(q, weight))
        g = _randn(11, B, N, 72, dtype=dtype)
        got, ref = (vsa.linear_backward(x, weight, d, bias=True) for x, d in ((odd[0], _odd(g, stride)), (q, g)))
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def _pi():
    """pi to 400 bits: 16 arctan(1/5) - 4 arctan(1/239)."""
    one = 1 << 420

    def arctan(x):
        term, total, n = one // x, 0, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= x * x
            n += 2
        return total

    return Fraction(16 * arctan(5) - 4 * arctan(239), one)


@pytest.mark.parametrize("kind", [torch.int32, torch.float32], ids=str)
@pytest.mark.parametrize("scale", [(1.0, -0.5, 7.0), (1000.0, -1000.0, 2.0 ** 40), (2.0 ** 60, -3e-9, 0.3)], ids=str)
def test_angles_of_far_positions(scale, kind):
    """Against the product position x frequency (a double) with pi to 400 bits. The bound on y is that of the other
    tests of the rotation: 26 steps of 2^-24 of |x_u| + |x_v| and the rounding; fp32 positions are whole numbers here,
    below 2^31."""
    D, sections = 64, (24, 20, 20)
    rot = vsa.Rotation(D, sections, scale=scale)
    top = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 128, -2 ** 31 + 128, 10 ** 6 + 1, -(10 ** 8) - 7, 1, 0]
    p = torch.tensor(top).to(kind)[:, None].expand(-1, 3).contiguous()
    p[:, 1] = p[:, 1].roll(1)
    if kind is torch.float32:
        p = p.clamp(-2.0 ** 31 + 128, 2.0 ** 31 - 128)
    x = _randn(3, 1, 2, len(top), D, dtype=torch.float32)
    y = vsa.rope(x, None, rot, positions=p.cuda())[0].double().cpu()
    pi = _pi()
    turn = [[float(2 * pi * (Fraction(int(p[n, rot.spec.axis[j]])) * Fraction(rot.spec.freq[j]) / (2 * pi) % 1))
             for j in range(D // 2)] for n in range(len(top))]
    a = torch.tensor(turn, dtype=torch.float64)
    u, v = x.double().cpu()[..., 0::2], x.double().cpu()[..., 1::2]
    ref = torch.stack([u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos()], -1).flatten(-2)
    size = (u.abs() + v.abs()).repeat_interleave(2, -1)
    assert ((y - ref).abs() <= 26 * 2.0 ** -24 * size + 2.0 ** -24 * ref.abs()).all()


def test_fp32_positions_beyond_the_range_are_nan():
    rot = vsa.Rotation(64, (24, 20, 20))
    x = _randn(3, 1, 1, 3, 64, dtype=torch.float32)
    p = torch.tensor([[2.0 ** 63, 0, 0], [0, -2.0 ** 63, 0], [0, 0, 3e38]], device="cuda")
    y = vsa.rope(x, None, rot, positions=p)[0][0, 0]
    for n, (a, b) in enumerate(((0, 24), (24, 44), (44, 64))):
        assert torch.isnan(y[n, a:b]).all()
        assert torch.equal(y[n, :a], x[0, 0, n, :a]) and torch.equal(y[n, b:], x[0, 0, n, b:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes_and_values_of_every_finite_z(act, dtype):
    """act and act' at every finite number of the type, through products with one term (exact): y = act(z) and
    dx = act'(z). Bound: 32 + 16 |z| + 4 z^2 + |z|^3 steps of 2^-24 of a value's terms (see the linear product's
    tests) and half a step of the type; results below 2^-126 may be 0. Where |z| > 13 act is z or 0 and act' 1 or 0 to
    the last bit that counts."""
    top = 2 ** 16
    bits = torch.arange(top, dtype=torch.int32, device="cuda").to(torch.int16)
    z = bits.view(dtype)
    z = z[torch.isfinite(z)]
    n = z.numel() // 8 * 8
    z = z[:n]
    x = torch.zeros(1, 40, 8, dtype=dtype, device="cuda")                     # rows of 1: x W^T is W's first column
    x[:, :, 0] = 1
    w = torch.zeros(n, 8, dtype=dtype, device="cuda")
    w[:, 0] = z
    y = vsa.linear(x, w, activation=act)[0, 0]
    dout = torch.ones(1, n // 8, 8, dtype=dtype, device="cuda")
    eye = torch.eye(8, dtype=dtype, device="cuda")
    slope = vsa.linear_backward(torch.zeros(1, n // 8, 8, dtype=dtype, device="cuda"), eye, dout,
                                z=z.view(1, n // 8, 8), activation=act, want=(True, False))[0].flatten()
    t = z.double()
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-t * 0.5 ** 0.5)
        ref, ds = t * p, t * torch.exp(-0.5 * t * t) / (2 * torch.pi) ** 0.5
    else:
        a, b = (1.0, 0.0) if act == "silu" else (2 * (2 / torch.pi) ** 0.5, 2 * (2 / torch.pi) ** 0.5 * 0.044715)
        far = t.clamp(-1e4, 1e4)                                              # 0 and 1 beyond, in 64 bits too
        p = torch.sigmoid(far * (a + b * far * far))
        ref, ds = t * p, far * p * torch.sigmoid(-far * (a + b * far * far)) * (a + 3 * b * far * far)
    m = t.abs().clamp(max=1e4)
    steps = (32 + 16 * m + 4 * m ** 2 + m ** 3).clamp(max=2.0 ** 20) * 2.0 ** -24
    half, tiny = torch.finfo(dtype).eps / 2, 2.0 ** -25 if dtype is torch.float16 else 2.0 ** -126 * 128
    assert torch.isfinite(y).all() and torch.isfinite(slope).all()
    assert ((y.double() - ref).abs() <= (steps + half) * 1.01 * ref.abs() + tiny).all()
    assert ((slope.double() - p - ds).abs() <= steps * 2 * (p.abs() + ds.abs()) + half * 1.01 * (p + ds).abs() + tiny).all()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")], ids=str)
def test_a_weight_that_is_no_number_stays_in_its_channel(bad, interleaved):
    """Channels 48 to 63 are not rotated: y = x w r there, each for itself."""
    rot = vsa.Rotation(64, (16, 16, 16), interleaved=interleaved)
    q = _randn(1, 1, 3, 20, 64, dtype=torch.float32)
    w = 1 + 0.2 * _randn(2, 64, dtype=torch.float32)
    ref = vsa.qk_norm_rope(q, None, w, None, rot, grid=(1, 4, 5))[0]
    for c in (48, 55, 63):
        wb = w.clone()
        wb[c] = bad
        y = vsa.qk_norm_rope(q, None, wb, None, rot, grid=(1, 4, 5))[0]
        rest = [i for i in range(64) if i != c]
        assert torch.equal(y[..., rest], ref[..., rest])
        want = q[..., c] * bad
        assert torch.equal(torch.isnan(y[..., c]), torch.isnan(want))
        assert torch.isnan(want).all() or torch.equal(y[..., c], want)


def test_a_grid_without_tokens():
    rot = vsa.Rotation(64, (24, 20, 20))
    q, k = _randn(1, 2, 3, 0, 64), _randn(2, 2, 1, 0, 64)
    w = torch.ones(64, device="cuda")
    for grid in ((0, 4, 4), (2, 0, 3), (2, 3, 0)):
        kw = dict(grid=grid)
        for out in (vsa.rope(q, k, rot, **kw), vsa.rope_backward(q, k, rot, **kw), vsa.qk_norm_rope(q, k, w, w, rot, **kw)):
            assert [t.shape for t in out] == [q.shape, k.shape]
        dq, dk, dwq, dwk = vsa.qk_norm_rope_backward(q, k, w, w, q, k, rot, **kw)
        assert dq.shape == q.shape and dk.shape == k.shape and not dwq.any() and not dwk.any()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes_at_an_infinite_z(act):
    """Sums of -4e5 and 4e5 are infinite once rounded to fp16, but act of the first is 0 and its slope 0."""
    x = torch.zeros(1, 40, 8, dtype=torch.float16, device="cuda")
    x[:, :, 0] = 1000
    w = torch.zeros(16, 8, dtype=torch.float16, device="cuda")
    w[:, 0] = torch.tensor([-400.0, 400.0, 0.001, -0.5] * 4)
    z = torch.empty(1, 40, 16, dtype=torch.float16, device="cuda")
    y = vsa.linear(x, w, activation=act, z=z)
    assert (z[..., 0::4] == float("-inf")).all() and (z[..., 1::4] == float("inf")).all()
    assert (y[..., 0::4] == 0).all() and torch.isfinite(y[..., 2::4]).all()
    g = torch.ones_like(z)
    dx, dw, db = vsa.linear_backward(x, w, g, z=z, activation=act, bias=True)
    assert (db[0::4] == 0).all() and (db[1::4] == 40).all() and torch.isfinite(db).all()
    assert torch.isfinite(dw[0::4]).all() and torch.isfinite(dx).all()
    for dtype in (torch.float16, torch.bfloat16):
        far = torch.tensor([float("-inf"), float("inf"), float("nan"), 0.0] * 2, dtype=dtype, device="cuda")
        far = far.expand(1, 70, 8).contiguous()
        db = vsa.linear_backward(far, torch.eye(8, dtype=dtype, device="cuda"), torch.ones_like(far), z=far, activation=act,
                                 bias=True, want=(False, False))[2]
        assert torch.equal(db[:2], torch.tensor([0.0, 70.0], device="cuda")) and torch.isnan(db[2])
        # at 0 all three slopes are 1/2, gelu's by a tail that is right to 5.2e-7 of 1/2 up to |z| = 1 and two
        # operations more: below 32 steps of 2^-24, the bound of the other tests of slopes, in each of 70 terms of 1/2
        assert abs(db[3] - 35) <= 70 * 0.5 * 32 * 2.0 ** -24


def test_first_calls_of_a_host_thread():
    """A thread whose first use of the GPU is one of the library's calls has no context of its own yet; outputs that
    are there already leave nothing else to make it one."""
    x, w = _randn(1, 1, 300, 64), _randn(2, 256, 64)
    dy, y, dx = _randn(3, 1, 300, 256), torch.empty(1, 300, 256, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    h = _randn(4, 1, 3, 300, 64)
    o, rot = torch.empty_like(h), vsa.Rotation(64, (24, 20, 20))
    plan = vsa.Plan(1, 1, 4, 8, 8, 64, topk=2)
    q, k, v = (_randn(i, 1, 1, 256, 64) for i in (5, 6, 7))
    gate = torch.ones(1, 1, 256, device="cuda")
    outs = [t.clone() for t in plan.run(q, k, v, gate, gate)]
    calls = [
        (lambda: vsa.linear(x, w, out=y), [y], [vsa.linear(x, w)]),
        (lambda: vsa.linear_backward(x, w, dy, dx=dx, want=(True, False)), [dx],
         [vsa.linear_backward(x, w, dy, want=(True, False))[0]]),
        (lambda: vsa.linear_backward(x, w, dy, want=(False, True)), [], []),
        (lambda: vsa.rope(h, None, rot, grid=(3, 10, 10), q_out=o), [o], [vsa.rope(h, None, rot, grid=(3, 10, 10))[0]]),
        (lambda: vsa.linear_check(), [], []),
        (lambda: plan.run(q, k, v, gate, gate, *outs), outs, [t.clone() for t in outs]),
    ]
    for call, got, ref in calls:
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        with ThreadPoolExecutor(1) as pool:
            pool.submit(call).result()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    plan.check()
