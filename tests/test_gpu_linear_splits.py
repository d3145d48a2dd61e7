"""Linear products whose contraction is split while other tiles are whole, and over several rounds of pairs of CTAs: the
cut is worked out here as the library does it, and held against the workspace sizes that the library gives, so that the
cases cannot lose the cut that they are here for."""
import pytest
import torch

import test_gpu_linear as tl
from trainable_block_sparse_cube_b200 import build as vsa_build
from trainable_block_sparse_cube_b200 import vsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    vsa_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vsa.load()


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    vsa.linear_check()


def _up(a, b):
    return -(-a // b)


def cut(batches, rows, cols, blocks, wide=False, pairs=74):
    """(columns of a tile, parts of a split one, whole tiles, split tiles)"""
    row_tiles, high, best = batches * _up(rows, 256), float(min(rows, 256)), None
    for bn in range(256, 63, -32):
        if wide and bn % 128:
            continue
        tiles = row_tiles * _up(cols, bn)
        rest = tiles % pairs
        step = max(400.0, 2.0 * bn, (128.0 * min(high, 128) + 64.0 * bn) / 47,
                   128.0 * bn * min(tiles, pairs) / min(row_tiles, 8) / 3400)
        tail = 2000 + 25.0 * bn
        base = tiles // pairs * (max(blocks * step, tail) + 800) + tail
        for s in (1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 24, 32):
            if s > 1 and (s > blocks or rest * s > (pairs if cols <= bn else 4 * pairs) or not rest):
                break
            cost = base + _up(rest * s, pairs) * (_up(blocks, s) * step + 800)
            if s > 1:
                cost += 2500 + 8.0 * s * rest * high * bn / 2700
            if best is None or cost < best[0]:
                best = (cost, (bn, s, tiles - rest, rest) if s > 1 else (bn, 1, tiles, 0))
    return best[1]


def _parts(c):
    return c[1] * c[3] * 256 * c[0] * 4


def _kind(c):
    return ("split" if c[1] > 1 else "whole") + ("+whole" if c[1] > 1 and c[2] else "") + \
        ("+rounds" if c[1] * c[3] > 74 else "")


def _workspaces(B, N, K, F):
    """What the two workspace queries have to give."""
    runs = ((1, B * N), (B, N))
    forward = max(_parts(cut(b, n, F, _up(K, 64))) for b, n in runs)
    parts = max(max(_parts(cut(b, n, K, _up(F, 64))), _parts(cut(1, F, K, b * _up(n, 64))),
                    _parts(cut(1, F, K, b * _up(n, 64), True))) for b, n in runs)
    M = B * N
    blocks = 1 if M <= 64 else min(_up(M, 8), max(1, 8 * 148 // _up(F, 256)))
    return forward, (_up(blocks * F * 4, 256) * 256 if blocks > 1 else 0) + parts


CASES = [
    # B, N, K, F, heads in, heads out, activation, bias, residual, layout; cuts of forward, dx, dW
    ((1, 19003, 512, 64, 8, 0, "gelu", True, True, "heads"), "split+whole", "whole", None),
    ((1, 10001, 6144, 64, 0, 0, "silu", True, True, "slice"), "whole", "whole", None),    # one column of tiles
    ((1, 5003, 12288, 320, 0, 0, "silu", True, True, "slice"), "split+rounds", None, None),
    ((1, 19003, 64, 512, 0, 8, "gelu_tanh", True, False, "heads"), "whole", "split+whole", None),
    ((1, 5003, 320, 12288, 0, 192, None, True, True, "heads"), None, "split+rounds", None),
    ((3, 6399, 512, 64, 8, 0, None, True, True, "heads"), "split+whole", None, None),     # batches that are no run
    ((1, 4099, 4096, 1536, 32, 12, "silu", True, False, "heads"), None, None, "split+whole"),
    ((1, 16001, 6144, 384, 48, 0, None, True, False, "heads"), None, None, "split+rounds"),
    ((1, 10001, 6144, 2048, 0, 16, "gelu_tanh", True, False, "heads"), None, None, "split+whole+rounds"),
    ((3, 3301, 6144, 2048, 48, 16, None, True, False, "heads"), None, None, "split+whole+rounds"),
]


@pytest.mark.parametrize("case,forward,dx,dw", CASES, ids=[f"{c[0][0]}x{c[0][1]}x{c[0][2]}x{c[0][3]}" for c in CASES])
def test_cuts(case, forward, dx, dw):
    B, N, K, F, hi, ho, act, bias, residual, how = case
    assert torch.cuda.get_device_properties(0).multi_processor_count == 148
    sizes = vsa.LinearSizes(0, B, N, K, F)
    L = vsa.load()
    assert (L.vsa_linear_workspace_bytes(sizes), L.vsa_linear_backward_workspace_bytes(sizes, 0)) == _workspaces(B, N, K, F)
    runs = B if B > 1 and how == "heads" and hi > 1 else 1
    rows = N if runs > 1 else B * N
    for want, c in ((forward, cut(runs, rows, F, _up(K, 64))), (dx, cut(runs, rows, K, _up(F, 64))),
                    (dw, cut(1, F, K, runs * _up(rows, 64), hi > 1))):
        assert want in (None, _kind(c)), c
    tl.test_forward(case, torch.bfloat16)
    tl.test_backward(case, torch.bfloat16)
    # A part that is lost or added twice changes a sum by its root of the number of terms, below the bounds for the
    # worst order of n terms: the error's root mean square is at most the roundings', two of half a step of 2^-8.
    x, w, _, g = tl._inputs(case[:8] + (True, how), torch.bfloat16, 11)
    xl, gl = tl._layout(x, hi, how), tl._layout(g, ho, how)
    got = (tl._rows(vsa.linear(xl, w)), tl._rows(vsa.linear_backward(xl, w, gl)[0]), vsa.linear_backward(xl, w, gl)[1])
    x64, w64, g64 = x.double(), w.double(), g.double()
    for a, ref in zip(got, (x64 @ w64.t(), g64 @ w64, g64.flatten(0, 1).t() @ x64.flatten(0, 1))):
        assert (a.double() - ref).square().mean().sqrt() <= 2.0 ** -8 * ref.square().mean().sqrt()
        worst_row = ((a.double() - ref).square().mean(-1) / ref.square().mean(-1)).sqrt().max()
        assert worst_row <= 2.0 ** -7


@pytest.mark.parametrize("M", [1, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("K,F", [(1016, 4096), (1024, 4096), (1032, 4104), (2048, 4104), (2056, 4104)])
def test_few_rows_by_either_number_of_warps(M, K, F):
    tl.test_forward((1, M, K, F, 0, 0, "gelu_tanh", True, True, "rows"), torch.float16)
