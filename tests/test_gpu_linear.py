"""GPU parity of the linear product's entry points with fp64.

Tolerances, for sums of n products: the tensor cores add in fp32 and may cut
instead of round, so a sum is off by at most n + 16 steps of 2^-23 of the sum
of the terms' sizes (S); then
  z     that, and half a step of its type
  y     1.13 of that (the activations' steepest slope), the activation's own
        work, the residual's addition (2^-24), and half a step
  act   its argument is off by 3 steps of 2^-24 of v = 1.6 |z| + 0.07 |z|^3,
        the exponential by 2 + 1.16 |v| of 2^-23, erfc by 6 of 2^-23 and, for
        its argument, z^2 of 2^-23; 8 steps for the rest: fewer than
        A(z) = 32 + 16 |z| + 4 z^2 + |z|^3 steps of 2^-24 of |y|
  act'  the same of its two terms s and |z s (1 - s) v'| (together below
        1.6 + |z| / 2 where they matter): A(z) steps of 2
  dz    act' times |dout| and half a step of the type before the products
  dx    the products' n + 16 steps of S, the sum of |error of dz| |W|, half a step
  db    rows / 8 + 80 steps of 2^-24 of the sum of |dz| (a thread adds every
        8th row at most), and the sum of |error of act'| |dout|
"""
import pytest
import torch

from trainable_block_sparse_cube_b200 import build as vsa_build
from trainable_block_sparse_cube_b200 import vsa

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    vsa_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vsa.load()


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    vsa.linear_check()


def _randn(seed, *shape, dtype, std=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _rows(x):
    return x if x.dim() == 3 else x.transpose(1, 2).flatten(2)


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z * 0.5 ** 0.5)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    return z


def _slope(z, act):
    z = z.clone().requires_grad_(True)
    return torch.autograd.grad(_act(z, act).sum(), z)[0]


def _steps(z):
    a = z.abs()
    return 32 + 16 * a + 4 * a ** 2 + a ** 3


def _check(got, ref, tol, what):
    half = torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 1e-37
    got, tol = got.double(), tol * (1 + 2 * half) + half * ref.abs() + tiny
    assert torch.isfinite(got).all(), what
    worst = ((got - ref).abs() / tol).max().item() if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def _layout(x, heads, how):
    """x [B, N, C] as [B, N, C] or [B, heads, N, D], stored densely or inside a wider tensor."""
    B, N, C = x.shape
    if how == "slice":
        wide = torch.full((B, N + 2, C + 64), float("nan"), dtype=x.dtype, device=x.device)
        wide[:, 1:N + 1, 64:] = x
        x = wide[:, 1:N + 1, 64:]
    if not heads:
        return x
    v = x.unflatten(2, (heads, C // heads)).transpose(1, 2)
    return v.contiguous() if how == "heads" else v


CASES = [
    # B, N, K, F, heads in, heads out, activation, bias, residual, layout
    (1, 1, 64, 64, 0, 0, None, False, False, "rows"),
    (1, 1, 2056, 1000, 0, 0, "silu", True, True, "rows"),            # a second chunk of channels
    (2, 1, 256, 64, 2, 1, "gelu", True, False, "heads"),
    (1, 3, 8, 8, 0, 0, "gelu_tanh", True, True, "rows"),
    (3, 2, 640, 24, 5, 0, None, True, True, "slice"),
    (2, 4, 128, 128, 2, 2, "silu", False, True, "heads"),
    (1, 9, 8, 8, 0, 0, None, True, False, "rows"),                   # two groups of eight rows
    (5, 3, 1096, 1000, 0, 0, "gelu", True, True, "slice"),
    (4, 4, 2048, 144, 16, 0, "silu", True, False, "heads"),
    (1, 17, 136, 72, 0, 0, "gelu_tanh", True, True, "rows"),         # tiles from here on
    (1, 17, 8, 8, 0, 0, None, True, False, "rows"),
    (3, 7, 64, 192, 1, 3, None, False, False, "heads"),              # batches that are no run of rows
    (9, 1, 512, 256, 4, 2, "silu", True, True, "heads"),
    (1, 40, 4096, 256, 0, 0, "gelu_tanh", True, True, "rows"),       # a split contraction
    (2, 37, 1096, 392, 0, 0, "gelu", True, True, "slice"),
    (3, 100, 384, 384, 3, 6, "silu", True, True, "heads"),
    (2, 129, 72, 136, 0, 0, None, False, True, "rows"),
    (1, 256, 64, 256, 1, 1, "gelu_tanh", True, False, "heads"),
    (1, 257, 1536, 264, 12, 0, None, True, True, "heads"),
    (2, 1000, 768, 1536, 0, 12, "gelu_tanh", True, False, "heads"),
    (1, 5003, 200, 1096, 0, 0, "silu", True, True, "rows"),
    (1, 4100, 128, 4096, 1, 64, "gelu", True, True, "heads"),        # several tiles a pair
    (1, 16384, 320, 1536, 5, 0, None, True, True, "heads"),
]
IDS = [f"{c[0]}x{c[1]}x{c[2]}x{c[3]}" for c in CASES]


def _inputs(case, dtype, seed):
    B, N, K, F, hi, ho, act, bias, residual, how = case
    x, w = _randn(seed, B, N, K, dtype=dtype), _randn(seed + 1, F, K, dtype=dtype, std=2 * K ** -0.5)
    b = _randn(seed + 2, F, dtype=torch.float32) if bias else None
    r = _randn(seed + 3, B, N, F, dtype=dtype) if residual else None
    return x, w, b, r


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case, dtype):
    B, N, K, F, hi, ho, act, bias, residual, how = case
    x, w, b, r = _inputs(case, dtype, 1)
    xl, rl = _layout(x, hi, how), None if r is None else _layout(r, ho, how)
    y = vsa.linear(xl, w, b, activation=act, residual=rl, heads=ho or None)
    assert y.shape == ((B, ho, N, F // ho) if ho else (B, N, F)) and y.is_contiguous()
    zl = torch.empty_like(y)
    y2 = vsa.linear(xl, w, b, activation=act, residual=rl, heads=ho or None, z=zl)
    assert torch.equal(y, y2)
    z = x.double() @ w.double().t() + (0 if b is None else b.double())
    size = x.double().abs() @ w.double().abs().t() + (0 if b is None else b.double().abs())
    off = (K + 16) * 2 * STEP * size
    _check(_rows(zl), z, off, "z")
    ya = _act(z, act)
    ref = ya if r is None else ya + r.double()
    own = 0 if act is None else _steps(z) * STEP * ya.abs()
    _check(_rows(y), ref, 1.13 * off + own + STEP * ref.abs(), "y")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case, dtype):
    B, N, K, F, hi, ho, act, bias, _, how = case
    x, w, _, g = _inputs(case[:8] + (True, how), dtype, 11)
    z = _randn(20, B, N, F, dtype=dtype, std=2.0)
    xl, gl, zl = _layout(x, hi, how), _layout(g, ho, how), _layout(z, ho, how)
    dx, dw, db = vsa.linear_backward(xl, w, gl, z=zl if act else None, activation=act, bias=True)
    again = vsa.linear_backward(xl, w, gl, z=zl if act else None, activation=act, bias=True)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))     # the same bits every time
    assert dx.shape == xl.shape and dw.shape == w.shape
    half = torch.finfo(dtype).eps / 2
    g64, w64, x64 = g.double(), w.double(), x.double()
    dz = g64 * _slope(z.double(), act) if act else g64
    fn = 2 * _steps(z.double()) * STEP * (1.6 + z.double().abs() / 2) * g64.abs() if act else torch.zeros_like(g64)
    off = fn + half * dz.abs() if act else fn
    if act and dtype == torch.float16:
        off = off + 2.0 ** -25
    size = dz.abs() + off
    _check(_rows(dx), dz @ w64, (F + 16) * 2 * STEP * (size @ w64.abs()) + off @ w64.abs(), "dx")
    flat, xf = dz.flatten(0, 1).t(), x64.flatten(0, 1)
    _check(dw, flat @ xf, (B * N + 16) * 2 * STEP * (size.flatten(0, 1).t() @ xf.abs()) +
           off.flatten(0, 1).t() @ xf.abs(), "dw")
    _check(db, dz.sum((0, 1)), (B * N / 8 + 80) * STEP * (dz.abs() + fn).sum((0, 1)) + fn.sum((0, 1)), "db")
    only = vsa.linear_backward(xl, w, gl, z=zl if act else None, activation=act, want=(True, False))
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    only = vsa.linear_backward(xl, w, gl, z=zl if act else None, activation=act, want=(False, True))
    assert only[0] is None and torch.equal(only[1], dw)


def test_in_place_residual_and_written_views():
    """out may be the residual; z and out may be slices of wider tensors, and what lies beside them stays."""
    for N, K, F in ((5, 72, 40), (300, 136, 200), (70, 4096, 64)):
        x, w, b = _randn(1, 2, N, K, dtype=torch.bfloat16), _randn(2, F, K, dtype=torch.bfloat16), \
            _randn(3, F, dtype=torch.float32)
        r = _randn(4, 2, N, F, dtype=torch.bfloat16)
        zr = torch.empty_like(r)
        ref = vsa.linear(x, w, b, activation="silu", residual=r, z=zr)
        own = r.clone()
        assert vsa.linear(x, w, b, activation="silu", residual=own, out=own) is own and torch.equal(own, ref)
        for pad in (8, 16):                                # rows on 16-byte and on 32-byte boundaries
            wide = torch.full((2, N + 3, F + 2 * pad), 7.0, dtype=torch.bfloat16, device="cuda")
            zw = wide.clone()
            inner = (slice(None), slice(1, N + 1), slice(pad, F + pad))
            vsa.linear(x, w, b, activation="silu", residual=r, out=wide[inner], z=zw[inner])
            assert torch.equal(wide[inner], ref) and torch.equal(zw[inner], zr)
            for t in (wide, zw):
                t[inner] = 7.0
                assert (t == 7.0).all()
        dx, dw, _ = vsa.linear_backward(x, w, r, want=(True, True))
        wide = torch.full((2, N + 3, K + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        inner = (slice(None), slice(2, N + 2), slice(8, K + 8))
        assert torch.equal(vsa.linear_backward(x, w, r, dx=wide[inner], want=(True, False))[0], dx)
        wide[inner] = 7.0
        assert (wide == 7.0).all()


def test_strided_weights_and_broadcast_inputs():
    x = _randn(1, 1, 1, 128, dtype=torch.bfloat16).expand(2, 50, 128)      # the same row 100 times: strides 0
    wide = _randn(2, 200, 256, dtype=torch.bfloat16)
    w = wide[::2, 64:192]
    y = vsa.linear(x, w[:96])
    assert torch.equal(y, vsa.linear(x.contiguous(), w[:96].contiguous()))
    assert (y == y[0, 0]).all()
    g = _randn(4, 1, 1, 96, dtype=torch.bfloat16).expand(2, 50, 96)        # the gradient of a sum
    got = vsa.linear_backward(x.contiguous(), w[:96], g, bias=True)
    ref = vsa.linear_backward(x.contiguous(), w[:96].contiguous(), g.contiguous(), bias=True)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_values_that_are_not_finite_stay_in_their_row():
    for N in (7, 30, 300):
        x, w = _randn(1, 1, N, 192, dtype=torch.bfloat16), _randn(2, 200, 192, dtype=torch.bfloat16)
        clean = vsa.linear(x, w, activation="gelu")
        bad = x.clone()
        bad[0, 3, 5], bad[0, N - 2, 100] = float("nan"), float("inf")
        y = vsa.linear(bad, w, activation="gelu")
        ok = torch.ones(N, dtype=torch.bool, device="cuda")
        ok[3] = ok[N - 2] = False
        assert torch.equal(y[0, ok], clean[0, ok]) and torch.isnan(y[0, 3]).all()
    # far values through the activations: gelu and its tanh form end at 0 and at z, silu too
    one = torch.eye(64, dtype=torch.bfloat16, device="cuda")
    v = torch.tensor([-3e4, -300.0, -40.0, -20.0, 20.0, 40.0, 300.0, 3e4] * 8, device="cuda").to(torch.bfloat16)
    for act in ("silu", "gelu", "gelu_tanh"):
        y = vsa.linear(v.expand(1, 40, 64), one, activation=act)[0, 0].float()
        assert torch.equal(y[v > 0], v[v > 0].float()) and (y[v < 0].abs() < 1e-6).all()
        z = v.expand(1, 40, 64).contiguous()
        dx = vsa.linear_backward(z, one, torch.ones_like(z), z=z, activation=act, want=(True, False))[0][0, 0].float()
        assert (dx[v > 0] == 1).all() and (dx[v < 0].abs() < 1e-6).all()


def test_no_rows():
    w = _randn(1, 72, 64, dtype=torch.bfloat16)
    for B, N in ((0, 5), (2, 0)):
        x = torch.zeros(B, N, 64, dtype=torch.bfloat16, device="cuda")
        y = vsa.linear(x, w, activation="silu")
        assert y.shape == (B, N, 72)
        dx, dw, db = vsa.linear_backward(x, w, y, z=y, activation="silu", bias=True)
        assert dx.shape == x.shape and not dw.any() and not db.any()


def test_offsets_past_32_bits():
    far = 2 ** 31 + 64
    buf = torch.empty(far + 40 * 128, dtype=torch.bfloat16, device="cuda")
    for N in (8, 40):
        x, w = _randn(1, 2, N, 128, dtype=torch.bfloat16), _randn(2, 128, 128, dtype=torch.bfloat16)
        ref = vsa.linear(x, w)
        grads = vsa.linear_backward(x, w, ref)
        v = buf.as_strided((2, N, 128), (far, 128, 1))                     # batches far apart
        v.copy_(x)
        assert torch.equal(vsa.linear(v, w), ref)
        assert all(torch.equal(a, b) for a, b in zip(vsa.linear_backward(v, w, ref)[:2], grads))
        vsa.linear(x, w, out=v)
        assert torch.equal(v, ref)
        vsa.linear_backward(x, w, ref, dx=v)
        assert torch.equal(v, grads[0])
        h = buf.as_strided((1, 2, N, 64), (0, far, 64, 1))                 # heads far apart
        xh = x[:1].unflatten(2, (2, 64)).transpose(1, 2)
        h.copy_(xh)
        assert torch.equal(vsa.linear(h, w), ref[:1])


def test_other_stream_and_captured_graphs():
    """Work goes to the current stream, a captured call reads its inputs anew, and two graphs share nothing."""
    x, w, b = _randn(1, 1, 100, 4096, dtype=torch.bfloat16), _randn(2, 128, 4096, dtype=torch.bfloat16), \
        _randn(3, 128, dtype=torch.float32)
    g = _randn(4, 1, 100, 128, dtype=torch.bfloat16)

    def step(x):
        z = torch.empty(1, 100, 128, dtype=torch.bfloat16, device="cuda")
        y = vsa.linear(x, w, b, activation="gelu_tanh", z=z)
        few = vsa.linear(x[:, :5], w, b)
        return (y, few) + vsa.linear_backward(x, w, g, z=z, activation="gelu_tanh", bias=True)

    ref = step(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = step(x)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, side))
    xs = torch.zeros_like(x)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(xs)
        graphs.append((graph, out))
    xs.copy_(x)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (graph, _), st in zip(graphs, streams):                        # at the same time
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(ref, out))


def test_a_product_behind_other_kinds_of_work():
    """The kernels that start while the work before them still runs wait for it: a fill, a copy, a join of two
    streams, another product; eagerly and captured."""
    w1, w2 = _randn(1, 512, 512, dtype=torch.bfloat16, std=0.05), _randn(2, 512, 512, dtype=torch.bfloat16, std=0.05)
    src = _randn(3, 1, 3000, 512, dtype=torch.bfloat16)
    x, y = torch.zeros_like(src), torch.empty_like(src)
    other = torch.cuda.Stream()

    def work():
        y.zero_()
        now = torch.cuda.current_stream()
        other.wait_stream(now)
        with torch.cuda.stream(other):
            x.copy_(src)
        now.wait_stream(other)
        a = vsa.linear(x, w1, out=y)                   # behind the join
        b = vsa.linear(a, w2)                          # behind a product
        x.zero_()                                      # behind a product that reads it no more
        c = vsa.linear(b, w1, residual=x)              # behind a fill
        return (b, c) + vsa.linear_backward(b, w1, c, want=(True, True))[:2]

    ref = [t.clone() for t in work()]
    assert torch.equal(ref[0], vsa.linear(vsa.linear(src, w1), w2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for seed in (3, 4, 3):
        src.copy_(_randn(seed, 1, 3000, 512, dtype=torch.bfloat16))
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        for _ in range(3):
            eager = [t.clone() for t in work()]
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out))
    assert all(torch.equal(a, b) for a, b in zip(ref, out))


def test_products_on_several_streams_at_once():
    """Persistent pairs of CTAs of many products in flight together, each with a workspace of its own."""
    cases = [(_randn(i, 1, 200 + 90 * i, 1024, dtype=torch.bfloat16), _randn(9 + i, 520, 1024, dtype=torch.bfloat16))
             for i in range(4)]
    ref = [vsa.linear(x, w) for x, w in cases]
    back = [vsa.linear_backward(x, w, y) for (x, w), y in zip(cases, ref)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(10):
        for i, ((x, w), st) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(st):
                y = vsa.linear(x, w)
                got[i].append((y,) + vsa.linear_backward(x, w, y)[:2])
    torch.cuda.synchronize()
    for i, runs in enumerate(got):
        for y, dx, dw in runs:
            assert torch.equal(y, ref[i]) and torch.equal(dx, back[i][0]) and torch.equal(dw, back[i][1])


def test_beside_the_attention_on_another_stream():
    """Both take tensor memory and most of an SM; each waits for the other's blocks and gets its own result."""
    T, H, W, h, D = 8, 16, 16, 4, 128
    plan = vsa.Plan(1, h, T, H, W, D, topk=8)
    q, k, v = (_randn(i, 1, h, T * H * W, D, dtype=torch.bfloat16) for i in range(3))
    gate = torch.ones(1, h, T * H * W, device="cuda")
    x, w = _randn(5, 1, 2000, 512, dtype=torch.bfloat16), _randn(6, 1024, 512, dtype=torch.bfloat16)
    ref, y = plan.run(q, k, v, gate, gate)[0], vsa.linear(x, w)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(a):
            o = plan.run(q, k, v, gate, gate)[0]
        with torch.cuda.stream(b):
            got.append((o, vsa.linear(x, w), vsa.linear_backward(x, w, y)[1]))
    torch.cuda.synchronize()
    plan.check()
    dw = vsa.linear_backward(x, w, y)[1]
    assert all(torch.equal(o, ref) and torch.equal(z, y) and torch.equal(g, dw) for o, z, g in got)


def test_gradients_match_differences():
    """The gradient along a direction against a central difference in fp64 of the forward's formula, and of the
    forward itself."""
    x, w, b = _randn(1, 2, 150, 256, dtype=torch.bfloat16), _randn(2, 136, 256, dtype=torch.bfloat16, std=0.06), \
        _randn(3, 136, dtype=torch.float32)
    g = _randn(4, 2, 150, 136, dtype=torch.bfloat16)
    for act in ("silu", "gelu", "gelu_tanh"):
        z = torch.empty(2, 150, 136, dtype=torch.bfloat16, device="cuda")
        vsa.linear(x, w, b, activation=act, z=z)
        dx, dw, db = vsa.linear_backward(x, w, g, z=z, activation=act, bias=True)
        d = [_randn(5 + i, *t.shape, dtype=torch.float64) for i, t in enumerate((x, w, b))]

        def loss(h):
            xs, ws, bs = (t.double() + h * e for t, e in zip((x, w, b), d))
            return (_act(xs @ ws.t() + bs, act) * g.double()).sum()

        slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
        terms = [(a.double() * e).flatten() for a, e in zip((dx, dw, db), d)]
        # Every entry of dx and dw is rounded to half a step, as are z and dz before: 4 half steps of 2^-8 of the
        # terms, which add up at random: 8 standard deviations of their root sum of squares, and the slope's change
        # with z (below 1.2 a unit) over z's half step, |z| <= 6, is below 8 half steps of a term.
        size = torch.cat(terms).square().sum().sqrt()
        assert abs(slope - torch.cat(terms).sum()) <= 8 * 12 * 2.0 ** -8 * size


def test_a_wait_that_runs_out_is_reported_and_the_next_call_works():
    x, w = _randn(1, 1, 300, 512, dtype=torch.bfloat16), _randn(2, 256, 512, dtype=torch.bfloat16)
    ref = vsa.linear(x, w)
    L = vsa.load()
    try:
        assert L.vsa_linear_set_limits(200_000, 1) == 0                    # 0.2 ms, operands left unloaded
        vsa.linear(x, w)
        with pytest.raises(vsa.VSAError, match="TIMEOUT"):
            vsa.linear_check()
    finally:
        assert L.vsa_linear_set_limits(1_000_000_000, 0) == 0
    vsa.linear_check()                                                     # cleared
    assert torch.equal(vsa.linear(x, w), ref)
    vsa.linear_check()


@pytest.mark.parametrize("D", [64, 128])
def test_the_block_around_the_attention(D):
    """Projections, norm with rotation, attention, output projection onto the residual, feed-forward, and all their
    gradients as a training step runs them, against the same formulas in fp64 on the selection the kernel made."""
    B, h, T, H, W, topk = 1, 2, 4, 8, 8, 2
    N, C = T * H * W, h * D
    rot = vsa.Rotation(D, (D // 2, D // 4, D // 4))
    hid = _randn(1, B, N, C, dtype=torch.bfloat16)
    wqkv, wo, wu, wd = (_randn(2 + i, *s, dtype=torch.bfloat16, std=C ** -0.5)
                        for i, s in enumerate(((3 * C, C), (C, C), (2 * C, C), (C, 2 * C))))
    bu = _randn(6, 2 * C, dtype=torch.float32)
    nq, nk = 1 + 0.2 * _randn(7, D, dtype=torch.float32), 1 + 0.2 * _randn(8, D, dtype=torch.float32)
    gc, gf = torch.full((B, h, N), 0.5, device="cuda"), torch.ones(B, h, N, device="cuda")
    plan = vsa.Plan(B, h, T, H, W, D, topk=topk)
    grid = dict(grid=(T, H, W))

    qkv = vsa.linear(hid, wqkv, heads=3 * h)                               # [B, 3h, N, D]
    q0, k0, v = qkv[:, :h], qkv[:, h:2 * h], qkv[:, 2 * h:].contiguous()
    q, k = vsa.qk_norm_rope(q0, k0, nq, nk, rot, **grid)
    o, idx, cnt, o_fine, lse = plan.run_train(q, k, v, gc, gf)
    mid = vsa.linear(o, wo, residual=hid)
    z = torch.empty(B, N, 2 * C, dtype=torch.bfloat16, device="cuda")
    up = vsa.linear(mid, wu, bu, activation="gelu_tanh", z=z)
    out = vsa.linear(up, wd, residual=mid)
    g = _randn(9, B, N, C, dtype=torch.bfloat16)
    dup, dwd, _ = vsa.linear_backward(up, wd, g)
    dmid, dwu, dbu = vsa.linear_backward(mid, wu, dup, z=z, activation="gelu_tanh", bias=True)
    dmid = dmid + g
    do, dwo, _ = vsa.linear_backward(o, wo, dmid)
    dq, dk, dv, _, _ = plan.run_backward(q, k, v, gc, gf, idx, cnt, o_fine, lse, do)
    dqkv = torch.empty_like(qkv)
    dqkv[:, 2 * h:] = dv
    _, _, dnq, dnk = vsa.qk_norm_rope_backward(q0, k0, nq, nk, dq, dk, rot, dq=dqkv[:, :h], dk=dqkv[:, h:2 * h], **grid)
    dhid, dwqkv, _ = vsa.linear_backward(hid, wqkv, dqkv)
    dhid = dhid + dmid
    plan.check()

    # the same step in fp64: exact functions, with the attention on the selection idx (a mask of tokens)
    P = [t.double().requires_grad_(True) for t in (hid, wqkv, wo, wu, wd, bu, nq, nk)]
    x64, wqkv64, wo64, wu64, wd64, bu64, nq64, nk64 = P
    heads = lambda t: t.unflatten(2, (-1, D)).transpose(1, 2)  # noqa: E731
    qkv64 = heads(x64 @ wqkv64.t())
    n = torch.arange(N, device="cuda")
    pos = torch.stack([n // (H * W), n // W % H, n % W], -1).double()
    axis = torch.tensor([rot.spec.axis[j] for j in range(D // 2)], device="cuda")
    ang = pos[:, axis] * torch.tensor([rot.spec.freq[j] for j in range(D // 2)], device="cuda", dtype=torch.float64)

    def norm_rot(t, w):
        t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        u, s = t[..., 0::2], t[..., 1::2]
        return torch.stack([u * ang.cos() - s * ang.sin(), u * ang.sin() + s * ang.cos()], -1).flatten(-2)

    q64, k64, v64 = norm_rot(qkv64[:, :h], nq64), norm_rot(qkv64[:, h:2 * h], nk64), qkv64[:, 2 * h:]
    cube = ((pos[:, 0] // 4 * (H // 4) + pos[:, 1] // 4) * (W // 4) + pos[:, 2] // 4).long()
    nc = N // 64
    pool = torch.zeros(nc, N, device="cuda", dtype=torch.float64)
    pool[cube, n] = 1 / 64
    qc, kc, vc = (pool @ t for t in (q64, k64, v64))
    oc = torch.softmax(qc @ kc.transpose(-1, -2) * D ** -0.5, -1) @ vc
    chosen = torch.zeros(B, h, nc, nc, dtype=torch.bool, device="cuda")
    chosen.scatter_(-1, idx.long(), True)
    s64 = q64 @ k64.transpose(-1, -2) * D ** -0.5
    s64 = s64.masked_fill(~chosen[:, :, cube][..., cube], float("-inf"))
    o64 = gc[..., None] * oc[:, :, cube] + gf[..., None] * (torch.softmax(s64, -1) @ v64)
    mid64 = x64 + o64.transpose(1, 2).flatten(2) @ wo64.t()
    out64 = mid64 + _act(mid64 @ wu64.t() + bu64, "gelu_tanh") @ wd64.t()
    grads = torch.autograd.grad(out64, P, g.double())
    # Between the ends every tensor is rounded to bf16 once (relative half steps of 2^-8 that add up at random over
    # about ten tensors in a row): 10 half steps = 0.04 of the root mean square of a result bounds the error's.
    names = ("dhid", "dwqkv", "dwo", "dwu", "dwd", "dbu", "dnq", "dnk")
    for name, a, r in [("out", out, out64), *zip(names, (dhid, dwqkv, dwo, dwu, dwd, dbu, dnq, dnk), grads)]:
        err = ((a.double() - r).square().mean() / r.square().mean()).sqrt().item()
        assert err <= 10 * 2.0 ** -8, (name, err)
