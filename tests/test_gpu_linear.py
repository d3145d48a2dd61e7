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
