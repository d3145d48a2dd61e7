"""GPU parity of the rotary and per-head norm entry points with the fp64 oracle.

Tolerances. Every result is formed in fp32 from exact inputs and rounded once
to the tensor's type: half a step, eps(type)/2 of the value (and 2^-25 in
fp16's subnormal range). Before that, fp32 work adds at most K steps of 2^-24
of the terms that were added:
  the angle: 2^-25 turns after the reduction (2 pi 2^-25 = 3.2 steps), sine and
  cosine 2 ulp (4 steps); the norm: 8 products and sums in a lane, 5 sums
  across lanes, the mean's product and eps (16 steps of mean x^2, half of that
  in r), rsqrt 2 ulp (4 steps); 5 products and sums after it.
  y:  K = 3.2 + 4 + 8 + 4 + 5 < 26 of |x_u w_u r| + |x_v w_v r|
  dx: the same twice over (g, and the mean of g w x with its 15 sums), with
      the r^2 of its second term: K = 64 of r (|g w| + |x| r^2 mean |g w x|),
      |g| taken as |dy_u| + |dy_v|
  dw: a term costs 26; the sum over a thread's rows (at most the heads here),
      the rows of a tile (64), the blocks (their 32nd part and 5): K = 128 of
      the sum of |g x r|.
"""
import numpy as np
import pytest
import torch

from oracle import projection_oracle as po
from trainable_block_sparse_cube_b200 import build as vsa_build
from trainable_block_sparse_cube_b200 import vsa

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    vsa_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vsa.load()


def _gen(seed, *shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _bound(ref, size, k, dtype):
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + k * STEP * size + (2.0 ** -25 if dtype == torch.float16 else 1e-37)


def _check(got, ref, size, k, what):
    err = np.abs(_np(got) - ref)
    tol = _bound(ref, size, k, got.dtype) * (1 + torch.finfo(got.dtype).eps)
    assert np.isfinite(_np(got)).all(), what
    worst = np.max(err / tol) if err.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def _partner_abs(x, rot, interleaved):
    """|x_u| + |x_v| of each channel's pair; |x| where a channel is not rotated."""
    a = np.abs(x)
    b = a.copy()
    if interleaved:
        b[..., 0:rot:2] = b[..., 1:rot:2] = a[..., 0:rot:2] + a[..., 1:rot:2]
    else:
        m = rot // 2
        b[..., :m] = b[..., m:rot] = a[..., :m] + a[..., m:rot]
    return b


def _lay(x, layout):
    """A CUDA view [B, heads, N, D] with the values of x, stored as the layout says."""
    B, h, N, D = x.shape
    if layout == "heads":
        return x.cuda()
    if layout == "tokens":
        return x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    buf = torch.full((B, N, h + 3, D + 8), float("nan"), dtype=x.dtype).cuda()  # a slice of a wider tensor
    v = buf[:, :, 2:2 + h, :D].transpose(1, 2)
    v.copy_(x.cuda())
    return v


CASES = [
    # D, sections, interleaved, shared, B, heads, kv heads, grid or (N, far), layout
    (128, (44, 42, 42), True, False, 1, 3, 3, (2, 3, 5), "tokens"),
    (64, (24, 20, 20), True, False, 2, 5, 1, (1, 1, 1), "heads"),
    (128, (32, 48, 48), False, True, 2, 4, 2, (37, 5000), "fused"),
    (64, (16, 16, 16), False, False, 3, 2, 2, (129, 1000000), "heads"),
    (96, (32, 32, 32), False, True, 1, 6, 3, (65, 300), "tokens"),
    (80, (10, 22, 14), True, True, 1, 3, 1, (4, 4, 9), "fused"),
    (256, (64, 64, 128), False, False, 1, 2, 2, (17, 64), "tokens"),
    (256, (84, 86, 86), True, False, 2, 3, 3, (5, 3, 1), "heads"),
    (8, (2, 2, 4), True, False, 2, 2, 1, (70, 9), "heads"),
    (16, (8, 8, 0), False, False, 1, 1, 1, (3, 9), "tokens"),
    (24, (2, 0, 0), True, False, 1, 4, 4, (2, 1, 50), "tokens"),
    (128, (0, 0, 0), True, False, 1, 2, 2, (1, 4, 4), "tokens"),
    (128, (44, 42, 42), True, False, 1, 12, 12, (1, 33, 100), "tokens"),
]
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _setup(case, dtype, seed=0):
    D, sections, inter, shared, B, h, kh, where, layout = case
    rot = vsa.Rotation(D, sections, base=5000.0, interleaved=inter, shared=shared)
    if len(where) == 3:
        N = where[0] * where[1] * where[2]
        origin = (7, 0, -3)
        kw = dict(grid=where, origin=origin)
        pos = np.broadcast_to(po.grid_positions(*where, origin), (B, N, 3))
    else:
        N, far = where
        p = torch.randint(-far, far, (B, N, 3), generator=torch.Generator().manual_seed(seed + 5), dtype=torch.int32)
        kw = dict(positions=p.cuda())
        pos = p.double().numpy()
    ang = np.stack([po.angles(pos[b], sections, 5000.0, shared=shared) for b in range(B)])[:, None]
    q, k = _gen(seed, B, h, N, D, dtype=dtype), _gen(seed + 1, B, kh, N, D, dtype=dtype)
    wq, wk = 1 + 0.3 * _gen(seed + 2, D, dtype=torch.float32), 1 + 0.3 * _gen(seed + 3, D, dtype=torch.float32)
    return rot, kw, ang, q, k, wq, wk


def _rot_batch(x, ang, inter):
    return np.stack([po.rotate(x[b], ang[b], inter) for b in range(x.shape[0])])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"d{c[0]}_{c[7]}_{c[8]}")
def test_rope_forward_and_backward(case, dtype):
    rot, kw, ang, q, k, _, _ = _setup(case, dtype)
    inter, layout = case[2], case[8]
    for fn, sign in ((vsa.rope, 1), (vsa.rope_backward, -1)):
        yq, yk = fn(_lay(q, layout), _lay(k, layout), rot, **kw)
        assert yq.is_contiguous() and yk.is_contiguous()
        for y, x in ((yq, q), (yk, k)):
            ref = _rot_batch(_np(x), sign * ang, inter)
            _check(y, ref, _partner_abs(_np(x), rot.rot, inter), 26, fn.__name__)
    yq, none = vsa.rope(_lay(q, layout), None, rot, **kw)
    assert none is None and torch.equal(yq, vsa.rope(_lay(q, layout), _lay(k, layout), rot, **kw)[0])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"d{c[0]}_{c[7]}_{c[8]}")
def test_norm_rope_forward(case, dtype):
    rot, kw, ang, q, k, wq, wk = _setup(case, dtype, seed=10)
    inter, layout = case[2], case[8]
    for ws in ((wq, wk), (None, wk)):
        dev = [None if w is None else w.cuda() for w in ws]
        y = vsa.qk_norm_rope(_lay(q, layout), _lay(k, layout), *dev, rot, eps=1e-5, **kw)
        for t, x, w in zip(y, (q, k), ws):
            x, w = _np(x), 1.0 if w is None else _np(w)
            n = x * w / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-5)
            _check(t, _rot_batch(n, ang, inter), _partner_abs(n, rot.rot, inter), 26, "norm")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"d{c[0]}_{c[7]}_{c[8]}")
def test_norm_rope_backward(case, dtype):
    rot, kw, ang, q, k, wq, wk = _setup(case, dtype, seed=20)
    inter, layout = case[2], case[8]
    gq, gk = _gen(30, *q.shape, dtype=dtype), _gen(31, *k.shape, dtype=dtype)
    args = [_lay(t, layout) for t in (q, k)] + [wq.cuda(), wk.cuda()] + [_lay(t, layout) for t in (gq, gk)] + [rot]
    got = vsa.qk_norm_rope_backward(*args, eps=1e-5, **kw)
    again = vsa.qk_norm_rope_backward(*args, eps=1e-5, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))          # the same bits every time
    for dx, dw, x, w, g in ((got[0], got[2], q, wq, gq), (got[1], got[3], k, wk, gk)):
        x, w, g = _np(x), _np(w), _np(g)
        ref = [po.norm_rotate_backward(x[b], w, 1e-5, ang[b], inter, g[b]) for b in range(x.shape[0])]
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-5)
        ga = _partner_abs(g, rot.rot, inter)
        size = r * (ga * np.abs(w) + np.abs(x) * r * r * np.mean(ga * np.abs(w * x), -1, keepdims=True))
        _check(dx, np.stack([a for a, _ in ref]), size, 64, "dx")
        _check(dw, sum(b for _, b in ref), (ga * np.abs(x) * r).reshape(-1, x.shape[-1]).sum(0), 128, "dw")


def test_backward_matches_differences_of_the_forward():
    """The gradient along a direction against a central difference of the GPU's own fp32 forward."""
    case = CASES[4]
    rot, kw, ang, q, k, wq, wk = _setup(case, torch.float32, seed=40)
    q, k, wq, wk = (t.cuda() for t in (q, k, wq, wk))
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    d = [torch.randn_like(t) for t in (q, k, wq, wk)]
    got = vsa.qk_norm_rope_backward(q, k, wq, wk, gq, gk, rot, **kw)
    h = 2.0 ** -8

    def loss(s):
        y = vsa.qk_norm_rope(*(t + s * h * e for t, e in zip((q, k, wq, wk), d)), rot, **kw)
        return sum((a.double() * b.double()).sum() for a, b in zip(y, (gq, gk)))

    slope = (loss(1) - loss(-1)) / (2 * h)
    exact = sum((a.double() * b.double()).sum() for a, b in zip(got, d))
    size = sum((a.double() * b.double()).abs().sum() for a, b in zip(got, d))
    # the difference's own error: h^2 = 2^-16 of third derivatives (order 1 relative to the terms, here below 8)
    assert abs(slope - exact) <= 8 * h * h * size


def test_list_equals_grid_and_float_positions():
    T, H, W = 3, 4, 5
    rot = vsa.Rotation(64, (24, 20, 20))
    x = _gen(1, 2, 3, T * H * W, 64, dtype=torch.float32).cuda()
    pos = torch.from_numpy(po.grid_positions(T, H, W, (1, 2, 3)))
    a = vsa.rope(x, None, rot, grid=(T, H, W), origin=(1, 2, 3))[0]
    for dt in (torch.int32, torch.float32):
        p = pos.to(dt).cuda()
        for q in (p, p[None], p[None].expand(2, -1, -1), p.repeat(2, 1, 1)):
            assert torch.equal(a, vsa.rope(x, None, rot, positions=q)[0])
    four = vsa.Rotation(64, (16, 16, 16, 16), scale=(1, 1, 0.5, 2))
    p = torch.rand(2, T * H * W, 4) * 100
    ang = np.stack([po.angles(p[b].double().numpy(), (16,) * 4, scale=(1, 1, 0.5, 2)) for b in range(2)])[:, None]
    got = vsa.rope(x, None, four, positions=p.cuda())[0]
    _check(got, _rot_batch(_np(x), ang, True), _partner_abs(_np(x), 64, True), 26, "four axes, float positions")


@pytest.mark.parametrize("inter", [True, False])
def test_in_place_and_written_views(inter):
    """An output may be its input, and a slice of a wider tensor; what lies beside it stays."""
    rot = vsa.Rotation(64, (16, 16, 16), interleaved=inter)
    buf = _gen(3, 2, 50, 9, 72, dtype=torch.bfloat16).cuda()
    kept = buf.clone()
    q, k = buf[:, :, :4, :64].transpose(1, 2), buf[:, :, 4:6, :64].transpose(1, 2)
    w = torch.rand(64, device="cuda") + 0.5
    ref = vsa.qk_norm_rope(q, k, w, None, rot, grid=(2, 5, 5))
    rq, rk = vsa.qk_norm_rope(q, k, w, None, rot, grid=(2, 5, 5), q_out=q, k_out=k)
    assert rq is q and torch.equal(q, ref[0]) and torch.equal(k, ref[1])
    assert torch.equal(buf[:, :, 6:], kept[:, :, 6:]) and torch.equal(buf[..., 64:], kept[..., 64:])
    g = torch.randn_like(q)
    dq, _, dw, _ = vsa.qk_norm_rope_backward(q, None, w, None, g, None, rot, grid=(2, 5, 5))
    into = g.clone()
    dq2, _, dw2, _ = vsa.qk_norm_rope_backward(q, None, w, None, into, None, rot, grid=(2, 5, 5), dq=into)
    assert torch.equal(dq, dq2) and torch.equal(dw, dw2)
    dq3, *_ = vsa.qk_norm_rope_backward(q, None, w, None, g, None, rot, grid=(2, 5, 5), dq=q)
    assert torch.equal(dq, dq3)


@pytest.mark.parametrize("inter", [True, False])
def test_values_that_are_not_finite_stay_in_their_row(inter):
    rot = vsa.Rotation(64, (16, 8, 8), interleaved=inter)
    x = _gen(4, 1, 2, 9, 64, dtype=torch.bfloat16).cuda()
    clean = vsa.rope(x, x, rot, grid=(1, 3, 3))[0]
    bad = x.clone()
    bad[0, 0, 4, 40] = float("inf")          # not rotated: passes as it is
    bad[0, 1, 2, 3] = float("nan")           # rotated: it and its partner
    y = vsa.rope(bad, None, rot, grid=(1, 3, 3))[0]
    assert y[0, 0, 4, 40] == float("inf") and torch.isnan(y).sum() == 2
    ok = torch.isfinite(y)
    assert torch.equal(y[ok], clean[ok])
    n = vsa.qk_norm_rope(bad, None, None, None, rot, grid=(1, 3, 3))[0]
    m = vsa.qk_norm_rope(x, None, None, None, rot, grid=(1, 3, 3))[0]
    rows = torch.isnan(n).any(-1)
    assert rows.sum() == 2 and torch.equal(n[~rows], m[~rows])
    z = torch.zeros_like(x)
    assert not vsa.qk_norm_rope(z, None, None, None, rot, grid=(1, 3, 3))[0].any()


def test_no_rows():
    rot = vsa.Rotation(64, (16, 8, 8))
    w = torch.ones(64, device="cuda")
    p = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    for B, h, N in ((0, 2, 8), (2, 0, 8), (2, 2, 0)):
        q = torch.zeros(B, h, N, 64, dtype=torch.bfloat16, device="cuda")
        kw = dict(grid=(2, 2, 2)) if N else dict(positions=p)
        assert vsa.rope(q, q, rot, **kw)[1].shape == q.shape
        got = vsa.qk_norm_rope_backward(q, q, w, w, q, q, rot, **kw)
        assert not got[2].any() and not got[3].any()
    q, k = torch.randn(1, 2, 8, 64, device="cuda"), torch.zeros(1, 0, 8, 64, device="cuda")
    a, b = vsa.rope(q, k, rot, grid=(2, 2, 2))
    assert b.shape == k.shape and torch.equal(a, vsa.rope(q, None, rot, grid=(2, 2, 2))[0])
    got = vsa.qk_norm_rope_backward(q, k, w, w, q, k, rot, grid=(2, 2, 2))
    assert got[2].any() and not got[3].any()


def test_offsets_past_32_bits():
    """Batches and heads further apart than 2^31 elements."""
    rot = vsa.Rotation(64, (24, 20, 20))
    far = 2 ** 31 + 64
    buf = torch.empty(far + 8 * 64 * 4, dtype=torch.bfloat16, device="cuda")
    x = _gen(6, 2, 2, 8, 64, dtype=torch.bfloat16).cuda()
    ref = vsa.rope(x, None, rot, grid=(2, 2, 2))[0]
    g = vsa.qk_norm_rope_backward(x, None, None, None, x, None, rot, grid=(2, 2, 2))[0]
    for stride in ((far, 8 * 64, 64, 1), (8 * 64, far, 64, 1)):
        v = buf.as_strided((2, 2, 8, 64), stride)
        v.copy_(x)
        assert torch.equal(vsa.rope(v, None, rot, grid=(2, 2, 2))[0], ref)
        assert torch.equal(vsa.qk_norm_rope_backward(v, None, None, None, v, None, rot, grid=(2, 2, 2))[0], g)
        vsa.rope(x, None, rot, grid=(2, 2, 2), q_out=v)
        assert torch.equal(v, ref)


def test_other_stream_and_captured_graphs():
    """Work goes to the current stream, and a captured call reads its inputs anew; two graphs share nothing."""
    rot = vsa.Rotation(128, (44, 42, 42))
    q = _gen(7, 1, 4, 96, 128, dtype=torch.bfloat16).cuda()
    k = _gen(8, 1, 2, 96, 128, dtype=torch.bfloat16).cuda()
    w = torch.rand(128, device="cuda") + 0.5
    dq, dk = torch.randn_like(q), torch.randn_like(k)

    def step(q, k):
        y = vsa.qk_norm_rope(q, k, w, w, rot, grid=(4, 4, 6))
        return y + vsa.qk_norm_rope_backward(q, k, w, w, dq, dk, rot, grid=(4, 4, 6))

    ref = step(q, k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = step(q, k)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, side))
    qs, ks = torch.zeros_like(q), torch.zeros_like(k)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(qs, ks)
        graphs.append((g, out))
    qs.copy_(q)
    ks.copy_(k)
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(ref, out))


@pytest.mark.parametrize("inter", [True, False])
def test_fp32_outputs_off_the_32_byte_boundary(inter):
    """Rows that start on 16-byte boundaries only, in place and beside other channels, as whole sectors' rows do."""
    rot = vsa.Rotation(96, (32, 32, 32), interleaved=inter)
    x, g = _gen(1, 2, 3, 21, 96, dtype=torch.float32).cuda(), _gen(2, 2, 3, 21, 96, dtype=torch.float32).cuda()
    w = torch.rand(96, device="cuda") + 0.5
    ref = vsa.qk_norm_rope(x, None, w, None, rot, grid=(1, 3, 7))[0]
    back = vsa.qk_norm_rope_backward(x, None, w, None, g, None, rot, grid=(1, 3, 7))
    for start in (4, 8):
        wide = torch.full((2, 21, 3, 108), 7.0, device="cuda")
        v = wide[..., start:start + 96].transpose(1, 2)
        v.copy_(x)
        vsa.qk_norm_rope(v, None, w, None, rot, grid=(1, 3, 7), q_out=v)
        assert torch.equal(v, ref)
        v.copy_(g)
        got = vsa.qk_norm_rope_backward(x, None, w, None, v, None, rot, grid=(1, 3, 7), dq=v)
        assert torch.equal(v, back[0]) and torch.equal(got[2], back[2])
        v.fill_(7.0)
        assert (wide == 7.0).all()


def test_positions_that_are_no_numbers_or_far():
    rot = vsa.Rotation(64, (24, 20, 20), scale=(1.0, 7.0, 1.0))            # 7 radians: more than a turn a position
    x = _gen(3, 1, 1, 6, 64, dtype=torch.float32).cuda()
    p = torch.tensor([[0.25, -0.75, 1e-30], [-1e-30, 3.5, -2.5], [float("nan"), 1, 2], [1, float("inf"), 2],
                      [1e6 + 0.5, -1e6, 3], [2.0 ** 23, 0.5, -0.5]], device="cuda")
    y = vsa.rope(x, None, rot, positions=p)[0]
    ang = po.angles(p[[0, 1, 4, 5]].double().cpu().numpy(), (24, 20, 20), scale=(1.0, 7.0, 1.0))
    keep = x[:, :, [0, 1, 4, 5]]
    _check(y[:, :, [0, 1, 4, 5]], _rot_batch(_np(keep), ang[None, None], True), _partner_abs(_np(keep), 64, True), 26,
           "fractions")
    assert torch.isnan(y[0, 0, 2, :24]).all() and torch.isfinite(y[0, 0, 2, 24:]).all()
    assert torch.isnan(y[0, 0, 3, 24:44]).all() and torch.isfinite(y[0, 0, 3, :24]).all()
    far = torch.tensor([[-2 ** 31, 2 ** 31 - 1, 0]] * 6, dtype=torch.int32, device="cuda")
    ang = po.angles(far.double().cpu().numpy(), (24, 20, 20))
    y = vsa.rope(x, None, vsa.Rotation(64, (24, 20, 20)), positions=far)[0]
    # the frequency is a double: 2^-53 of 2^31 radians is 2^-22, 4 steps more of 2^-24
    _check(y, _rot_batch(_np(x), ang[None, None], True), _partner_abs(_np(x), 64, True), 26 + 8, "far")
