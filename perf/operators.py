"""Cases of the projection side of the attention: what runs between a transformer block's
hidden states and the block-sparse attention's q, k, v, and between its output and the
hidden states again.

rope           rotary positions with several axes (time, height, width) on q and k
qk_norm_rope   RMS norm of every head's queries and keys with the rotation in the same pass
linear         x W^T with bias, activation and residual in its epilogue, from or to the
               attention layout [B, heads, N, D]

Sizes follow the package's workloads: 12 or 40 heads of 128 channels, so hidden sizes of
1536 and 5120, over 16,384, 61,440 and 76,800 tokens.
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _rope_case(name, op, way, dtype, B, heads, kv_heads, T, H, W, D, sections, pairs, shared, positions, layout, far=1):
    c = {"op": op, "way": way, "dtype": dtype, "B": B, "heads": heads, "kv_heads": kv_heads, "T": T, "H": H, "W": W,
         "D": D, "s0": sections[0], "s1": sections[1], "s2": sections[2], "pairs": pairs, "shared": shared,
         "positions": positions, "layout": layout, "far": far}
    return dict(c, name=name) if name else c


def _linear_case(name, way, B, N, K, F, heads, activation, bias, residual):
    c = {"op": "linear", "way": way, "dtype": "bf16", "B": B, "N": N, "K": K, "F": F, "heads": heads,
         "activation": activation, "bias": bias, "residual": residual}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of each of two sequences of a text-and-video model, sections of one shared frequency table
        _rope_case("rope_step", "rope", "forward", "bf16", 2, 12, 4, 1, 1, 1, 128, (32, 48, 48), "half", True, "list",
                   "tokens", 5000),
        # the pre-training workload's grid, q and k in the projection's order [B, N, heads, D]
        _rope_case("rope_grid16k", "rope", "forward", "bf16", 1, 12, 12, 16, 32, 32, 128, (44, 42, 42), "interleaved",
                   False, "grid", "tokens"),
        # a ragged batch of text and image tokens at far positions, single precision, a part of each head rotated
        _rope_case("rope_mixed", "rope", "forward", "fp32", 3, 5, 5, 1, 1, 1237, 64, (16, 16, 16), "half", False,
                   "list", "heads", 1000000),
        # the largest workload's gradients on their way back through the rotation
        _rope_case("rope_grid77k_back", "rope", "backward", "bf16", 1, 40, 40, 20, 48, 80, 128, (44, 42, 42),
                   "interleaved", False, "grid", "heads"),
        # a few tokens at once, fewer key heads than query heads, half precision
        _rope_case("norm_step", "qk_norm_rope", "forward", "fp16", 1, 12, 3, 1, 1, 7, 128, (44, 42, 42), "interleaved",
                   False, "list", "tokens", 64),
        # the long workload, q and k as slices of one fused projection [B, N, q + k + v heads, D]
        _rope_case("norm_grid61k", "qk_norm_rope", "forward", "bf16", 1, 12, 12, 16, 48, 80, 128, (44, 42, 42),
                   "interleaved", False, "grid", "fused"),
        # a training step of the pre-training workload
        _rope_case("norm_grid16k_back", "qk_norm_rope", "backward", "bf16", 1, 12, 12, 16, 32, 32, 128, (44, 42, 42),
                   "interleaved", False, "grid", "tokens"),
        # a ragged batch in single precision, heads of 96 channels, shared key heads
        _rope_case("norm_ragged_back", "qk_norm_rope", "backward", "fp32", 2, 6, 2, 1, 1, 4999, 96, (32, 32, 32),
                   "half", True, "list", "heads", 3000),
        # the modulation of a block from a pair of time embeddings: two rows, six outputs for each channel
        _linear_case("linear_step", "forward", 1, 2, 1536, 9216, 0, "silu", True, False),
        # the up projection of the feed-forward, a ragged number of tokens
        _linear_case("linear_up", "forward", 2, 5003, 1536, 6144, 0, "gelu_tanh", True, False),
        # the output projection of the largest workload, out of the attention layout and onto the residual stream
        _linear_case("linear_out77k", "forward", 1, 76800, 5120, 5120, 40, "none", True, True),
        # the gradients of the up projection in a training step
        _linear_case("linear_up_back", "backward", 1, 16384, 1536, 6144, 0, "gelu_tanh", True, False),
    ]


def _between(rng, low, high):
    """A whole number of the range, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(("rope", "qk_norm_rope", "linear"))
    way = rng.choice(("forward", "backward"))
    if kind == "linear":
        B = rng.choice((1, 1, 2, 3))
        N = _between(rng, 1, 40000) // B + 1
        heads = rng.choice((0, 0, rng.choice((2, 6, 12, 16, 24, 40))))
        K = heads * rng.choice((64, 128)) if heads else 8 * _between(rng, 8, 800)
        F = 8 * _between(rng, 8, 800)
        return _linear_case(None, way, B, N, K, F, heads, rng.choice(("none", "silu", "gelu", "gelu_tanh")),
                            rng.random() < 0.7, way == "forward" and rng.random() < 0.4)
    D = rng.choice((64, 64, 80, 96, 128, 128, 128, 256))
    heads = _between(rng, 1, 40)
    kv_heads = rng.choice([h for h in range(1, heads + 1) if heads % h == 0] + [heads])
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    pairs = rng.choice(("interleaved", "half"))
    a, b = (16 * rng.randint(1, D // 64), 16 * rng.randint(1, D // 64)) if pairs == "half" else (
        2 * rng.randint(1, D // 6), 2 * rng.randint(1, D // 6))
    c = rng.choice((D - a - b, 16))
    B = rng.choice((1, 1, 2, 4))
    passes = (3 if kind == "qk_norm_rope" and way == "backward" else 2) * (2 if dtype == "fp32" else 1)
    most = min(80000, 4 * 76800 * 40 * 128 // (B * (heads + kv_heads) * D * passes) - 1)
    layout = rng.choice(("heads", "tokens", "fused") if way == "forward" else ("heads", "tokens"))
    if rng.random() < 0.5:
        n = _between(rng, 1, most)
        return _rope_case(None, kind, way, dtype, B, heads, kv_heads, 1, 1, n, D, (a, b, c), pairs, rng.random() < 0.5,
                          "list", layout, _between(rng, 16, 1000000))
    T, H = rng.randint(1, 20), rng.randint(1, 48)
    W = max(1, min(rng.randint(1, 80), most // (T * H)))
    return _rope_case(None, kind, way, dtype, B, heads, kv_heads, T, H, W, D, (a, b, c), pairs, rng.random() < 0.5, "grid",
                      layout)


def _sections(c):
    return c["s0"], c["s1"], c["s2"]


def _heads_first(x, layout):
    """[B, heads, N, D] view of a tensor stored as the case's layout says."""
    return x if layout == "heads" else x.transpose(1, 2)


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    kind = _TYPES[c["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=kind):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = {"case": c}
    if c["op"] == "linear":
        B, N, K, F, h = c["B"], c["N"], c["K"], c["F"], c["heads"]
        s["x"] = normal(B, h, N, K // h) if h else normal(B, N, K)
        s["weight"] = normal(F, K, std=K ** -0.5)
        s["bias"] = normal(F, std=0.2, dtype=torch.float32) if c["bias"] else None
        s["residual"] = normal(B, N, F) if c["residual"] else None
        s["activation"] = None if c["activation"] == "none" else c["activation"]
        if c["way"] == "backward":
            s["dout"] = normal(B, N, F)
            s["z"] = normal(B, N, F) if s["activation"] else None
        return s
    B, h, kh, D = c["B"], c["heads"], c["kv_heads"], c["D"]
    N = c["T"] * c["H"] * c["W"]
    # hidden channels of trained models differ in size: a spread of scales over the channels of a head
    scale = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))
    if c["layout"] == "fused":
        qkv = (torch.randn(B, N, h + 2 * kh, D, generator=g, device="cuda") * scale).to(kind)
        s["q"], s["k"] = qkv[:, :, :h].transpose(1, 2), qkv[:, :, h:h + kh].transpose(1, 2)
    else:
        shape = (lambda n: (B, n, N, D)) if c["layout"] == "heads" else (lambda n: (B, N, n, D))
        s["q"], s["k"] = (_heads_first((torch.randn(*shape(n), generator=g, device="cuda") * scale).to(kind), c["layout"])
                          for n in (h, kh))
    if c["way"] == "backward":
        s["dq"], s["dk"] = normal(B, h, N, D), normal(B, kh, N, D)
    if c["op"] == "qk_norm_rope":
        s["wq"], s["wk"] = normal(D, std=0.3, mean=1.0, dtype=torch.float32), normal(D, std=0.3, mean=1.0, dtype=torch.float32)
    if c["positions"] == "list":
        s["positions"] = torch.randint(0, c["far"], (B, N, 3), generator=g, device="cuda", dtype=torch.int32)
        s["grid"] = None
    else:
        s["positions"], s["grid"] = None, (c["T"], c["H"], c["W"])
    if own:
        from trainable_block_sparse_cube_b200 import vsa
        s["rotation"] = vsa.Rotation(D, _sections(c), base=BASE, interleaved=c["pairs"] == "interleaved", shared=c["shared"])
    return s


# ---------------------------------------------------------------- plain forms
def _frequencies(c, device):
    """Radians a position of every pair of channels, and the axis that it turns with."""
    s = torch.tensor(_sections(c), device=device) // 2
    axis = torch.repeat_interleave(torch.arange(3, device=device), s, output_size=sum(_sections(c)) // 2)
    j = torch.arange(axis.numel(), device=device, dtype=torch.float64)
    if c["shared"]:
        return BASE ** (-j / axis.numel()), axis
    first = torch.cumsum(s, 0) - s
    return BASE ** (-(j - first[axis]) / s[axis]), axis


def _positions(s):
    if s["grid"] is None:
        return s["positions"]
    T, H, W = s["grid"]
    n = torch.arange(T * H * W, device=s["q"].device)
    return torch.stack([n // (H * W), n // W % H, n % W], -1)[None]


def _cos_sin(s):
    """[B or 1, 1, N, pairs] in single precision, from angles in double precision (far positions)."""
    f, axis = _frequencies(s["case"], s["q"].device)
    angle = _positions(s).to(torch.float64)[..., axis] * f
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _rotate(x, cos, sin, c):
    rot = sum(_sections(c))
    a, rest = x[..., :rot], x[..., rot:]
    if c["pairs"] == "interleaved":
        u, v = a[..., 0::2], a[..., 1::2]
        return torch.cat([torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2), rest], -1)
    u, v = a[..., :rot // 2], a[..., rot // 2:]
    return torch.cat([u * cos - v * sin, u * sin + v * cos, rest], -1)


def _rstd(x):
    return 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


def _norm_back(x, w, g):
    x = x.float()
    r = _rstd(x)
    n = x * r
    gw = g * w
    return r * (gw - n * (gw * n).mean(-1, keepdim=True)), (g * n).sum((0, 1, 2))


def _act(z, name):
    if name is None:
        return z
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def _act_slope(z, name):
    if name == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def _rows(x):
    """[B, N, K] of [B, N, K] or of the attention layout [B, heads, N, D]."""
    return x if x.dim() == 3 else x.transpose(1, 2).flatten(2)


def _plain(s):
    c = s["case"]
    if c["op"] == "linear":
        x, w = _rows(s["x"]).float(), s["weight"].float()
        if c["way"] == "forward":
            z = x @ w.t()
            z = z if s["bias"] is None else z + s["bias"]
            y = _act(z, s["activation"])
            return (y if s["residual"] is None else y + s["residual"].float()).to(s["x"].dtype)
        dz = s["dout"].float()
        dz = dz * _act_slope(s["z"].float(), s["activation"]) if s["activation"] else dz
        flat = dz.flatten(0, 1)
        dx = (dz @ w).to(s["x"].dtype)
        if c["heads"]:
            dx = dx.unflatten(2, (c["heads"], -1)).transpose(1, 2).contiguous()
        dw = (flat.t() @ x.flatten(0, 1)).to(s["x"].dtype)
        return (dx, dw, flat.sum(0)) if c["bias"] else (dx, dw)
    cos, sin = _cos_sin(s)
    kind = s["q"].dtype
    if c["op"] == "rope":
        if c["way"] == "forward":
            return tuple(_rotate(s[n].float(), cos, sin, c).to(kind).contiguous() for n in ("q", "k"))
        return tuple(_rotate(s[n].float(), cos, -sin, c).to(kind) for n in ("dq", "dk"))
    if c["way"] == "forward":
        return tuple(_rotate(x.float() * _rstd(x.float()) * w, cos, sin, c).to(kind).contiguous()
                     for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
    dq, dwq = _norm_back(s["q"], s["wq"], _rotate(s["dq"].float(), cos, -sin, c))
    dk, dwk = _norm_back(s["k"], s["wk"], _rotate(s["dk"].float(), cos, -sin, c))
    return dq.to(kind), dk.to(kind), dwq, dwk


def _own(s):
    from trainable_block_sparse_cube_b200 import vsa
    c = s["case"]
    if c["op"] == "linear":
        if c["way"] == "forward":
            return vsa.linear(s["x"], s["weight"], s["bias"], activation=s["activation"], residual=s["residual"])
        dx, dw, db = vsa.linear_backward(s["x"], s["weight"], s["dout"], z=s["z"], activation=s["activation"],
                                         bias=c["bias"])
        return (dx, dw, db) if c["bias"] else (dx, dw)
    where = {"grid": s["grid"], "positions": s["positions"]}
    if c["op"] == "rope":
        if c["way"] == "forward":
            return vsa.rope(s["q"], s["k"], s["rotation"], **where)
        return vsa.rope_backward(s["dq"], s["dk"], s["rotation"], **where)
    if c["way"] == "forward":
        return vsa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["rotation"], eps=EPS, **where)
    return vsa.qk_norm_rope_backward(s["q"], s["k"], s["wq"], s["wk"], s["dq"], s["dk"], s["rotation"], eps=EPS, **where)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    c = case
    size = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "linear":
        M, K, F = c["B"] * c["N"], c["K"], c["F"]
        if c["way"] == "forward":
            return {"bytes": 2 * (M * K + F * K + M * F * (2 if c["residual"] else 1)) + (4 * F if c["bias"] else 0),
                    "flops": 2 * M * K * F}
        return {"bytes": 2 * (2 * M * K + 2 * F * K + M * F * (1 if c["activation"] == "none" else 2)) +
                (4 * F if c["bias"] else 0), "flops": 4 * M * K * F}
    N = c["T"] * c["H"] * c["W"]
    e = c["B"] * (c["heads"] + c["kv_heads"]) * N * c["D"]
    where = 12 * c["B"] * N if c["positions"] == "list" else 0
    norm, back = c["op"] == "qk_norm_rope", c["way"] == "backward"
    return {"bytes": size * e * (3 if norm and back else 2) + where + (8 * c["D"] * (2 if back else 1) if norm else 0),
            "flops": e * (3 + (5 if norm else 0) * (2 if back else 1))}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "linear":
        w = s["weight"].to(f64).requires_grad_(c["way"] == "backward")
        x = s["x"].to(f64).requires_grad_(c["way"] == "backward")
        act = {None: lambda z: z, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
               "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[s["activation"]]
        rows = torch.einsum("bhnd->bnhd", x).reshape(c["B"], c["N"], c["K"]) if c["heads"] else x
        z = torch.nn.functional.linear(rows, w)
        if c["way"] == "forward":
            y = act(z if s["bias"] is None else z + s["bias"].to(f64))
            return y if s["residual"] is None else y + s["residual"].to(f64)
        dz = s["dout"].to(f64)
        if s["activation"]:
            at = s["z"].to(f64).requires_grad_(True)
            dz, = torch.autograd.grad(act(at), at, dz)
        dx, dw = torch.autograd.grad(z, (x, w), dz)
        return (dx, dw, dz.sum((0, 1))) if c["bias"] else (dx, dw)

    sections, D = _sections(c), c["D"]
    rot = sum(sections)
    freq, axis = [], []
    for a, n in enumerate(sections):
        for i in range(n // 2):
            freq.append(BASE ** (-2.0 * len(freq) / rot) if c["shared"] else BASE ** (-2.0 * i / n))
            axis.append(a)
    if s["positions"] is not None:
        p = s["positions"].to(f64)
    else:
        p = torch.cartesian_prod(*(torch.arange(n, device="cuda", dtype=f64) for n in (c["T"], c["H"], c["W"])))[None]
    angle = (p[:, :, axis] * torch.tensor(freq, device="cuda", dtype=f64))[:, None]
    turn = torch.polar(torch.ones_like(angle), angle)

    def rotated(x):
        if c["pairs"] == "interleaved":
            pairs = x[..., :rot].unflatten(-1, (rot // 2, 2))
        else:
            pairs = x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        y = y if c["pairs"] == "interleaved" else y.transpose(-1, -2)
        return torch.cat([y.reshape(*x.shape[:-1], rot), x[..., rot:]], -1)

    def one(n):
        x = s[n].to(f64)
        wide = c["op"] == "qk_norm_rope"
        w = s["w" + n].to(f64) if wide else None
        if c["way"] == "backward":
            x.requires_grad_(True)
            w = w.requires_grad_(True) if wide else None
        y = rotated(x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * w if wide else x)
        if c["way"] == "forward":
            return y, None
        got = torch.autograd.grad(y, (x, w) if wide else (x,), s["d" + n].to(f64))
        return got if wide else (got[0], None)

    (q, wq), (k, wk) = one("q"), one("k")
    return (q, k, wq, wk) if c["op"] == "qk_norm_rope" and c["way"] == "backward" else (q, k)
