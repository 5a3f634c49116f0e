"""The operators around the sparse attention layer, as they are measured: rotary
positions with three axes, norms of queries and keys with the rotation in the same
pass, and linears with bias, activation and residual, each with its gradients.

``run`` makes one pass: in plain torch operations where ``own`` is false, through the
framework's entry points where it is true.  Both take the state ``prepare`` makes.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6

# Latent geometries (prefix segments, video grid, tile) of this repository's workloads.
# Lists of sizes are texts, "40 70".
TINY = dict(prefix="40 70", grid="4 8 8", tile="4 4 4")
SMALL = dict(prefix="256 1024 300", grid="8 32 32", tile="4 4 4")
REF2VA = dict(prefix="512 256 256 256 256 128", grid="32 24 42", tile="4 4 4")
VEDA = dict(prefix="256", grid="32 48 68", tile="4 8 4")


def _ints(case, key):
    return [int(x) for x in case[key].split()]


def _text(sizes):
    return " ".join(str(x) for x in sizes)


def listed():
    return [
        # a short test clip: the call's own latency
        dict(name="rope_tiny", op="rope", B=1, H=2, D=64, **TINY, dims="24 20 20", theta=10000.0,
             step=1.0, halves=False, layout="bhnd", inverse=False),
        # the gradient of the rotation at the reference-to-video shape, on a [B,N,H,D] tensor
        dict(name="rope_ref2va_inverse", op="rope", B=1, H=42, D=128, **REF2VA, dims="44 42 42",
             theta=10000.0, step=1.0, halves=True, layout="bnhd", inverse=True),
        # Q and K of the small layer, views of one fused [B,N,3,H,D] projection
        dict(name="norm_rope_small_qkv", op="norm_rope", B=1, H=8, D=128, **SMALL, dims="44 42 42",
             theta=10000.0, step=1.0, halves=False, layout="qkv"),
        # step 1 of the 104,704-token layer: Q, K normed and rotated, V as it is, all in tile order
        dict(name="norm_rope_tiles_veda", op="norm_rope_tiles", B=1, H=42, D=128, **VEDA,
             dims="44 42 42", theta=256.0, step=1.0, halves=False, layout="bhnd"),
        # training step of a ragged two-element batch: gradients arrive in tile order
        dict(name="norm_rope_backward_ragged", op="norm_rope_backward", B=2, H=3, D=64,
             prefix="5 0 64 65", grid="5 6 7", tile="4 4 4", dims="16 24 24", theta=10000.0,
             step=0.5, halves=True, layout="bnhd", tiled=True),
        # the same at the reference-to-video shape
        dict(name="norm_rope_backward_ref2va", op="norm_rope_backward", B=1, H=42, D=128, **REF2VA,
             dims="44 42 42", theta=10000.0, step=1.0, halves=False, layout="bhnd", tiled=True),
        # one conditioning vector through a full-width linear: a single token
        dict(name="linear_token", op="linear", B=1, N=1, x_heads=0, C=5376, y_heads=0, O=5376, act="silu",
             bias=True, residual=False, pre=False),
        # output projection of the small layer: heads in, bias and residual out
        dict(name="linear_out_small", op="linear", B=1, N=9772, x_heads=8, C=1024, y_heads=0, O=1024,
             act="identity", bias=True, residual=True, pre=False),
        # first linear of a feed-forward in training at the reference-to-video length
        dict(name="linear_gelu_ref2va", op="linear", B=1, N=33920, x_heads=0, C=5376, y_heads=0, O=7168,
             act="gelu_tanh", bias=True, residual=False, pre=True),
        # gradient through an activation on its own, small layer
        dict(name="act_backward_small", op="act_backward", B=1, N=9772, O=1024, act="silu"),
        # gradients of a ragged batch's Q projection (heads out)
        dict(name="linear_backward_ragged", op="linear_backward", B=2, N=777, x_heads=0, C=520, y_heads=3,
             O=384, act="identity"),
        # second linear of the feed-forward: the gradient goes on through the first one's activation
        dict(name="linear_backward_ref2va", op="linear_backward", B=1, N=33920, x_heads=0, C=7168, y_heads=0,
             O=5376, act="gelu_tanh"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "norm_rope", "norm_rope_tiles", "norm_rope_backward", "linear", "linear",
                     "linear_backward", "act_backward"])
    if op in ("linear", "linear_backward", "act_backward"):
        B = rng.choice([1, 1, 2])
        N = _log_int(rng, 1, 33920 // B)
        if op == "act_backward":
            return dict(op=op, B=B, N=N, O=8 * _log_int(rng, 8, 896),
                        act=rng.choice(["sigmoid", "gelu_tanh", "silu"]))

        def width(name):
            if rng.random() < 0.4:
                d = rng.choice([64, 128])
                h = rng.randint(1, 5376 // d)
                return {name + "_heads": h}, h * d
            return {name + "_heads": 0}, 8 * _log_int(rng, 4, 672)
        hx, C = width("x")
        hy, O = width("y")
        act = rng.choice(["identity", "sigmoid", "gelu_tanh", "silu"])
        c = dict(op=op, B=B, N=N, **hx, C=C, **hy, O=O, act=act)
        if op == "linear":
            c.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5, pre=rng.random() < 0.3)
        return c
    D = rng.choice([64, 128])
    tile = rng.choice([[4, 4, 4], [4, 8, 4]])
    grid = [_log_int(rng, 1, 32), _log_int(rng, 2, 40), _log_int(rng, 2, 48)]
    prefix = [rng.choice([0, _log_int(rng, 1, 600)]) for _ in range(rng.randint(1, 4))]
    dims = rng.choice([[44, 42, 42], [0, 64, 64], [32, 48, 48], [32, 32, 32]] if D == 128 else
                      [[24, 20, 20], [16, 24, 24], [0, 32, 32], [16, 16, 16]])
    c = dict(op=op, B=rng.choice([1, 1, 2]), H=rng.randint(1, 24), D=D, prefix=_text(prefix), grid=_text(grid),
             tile=_text(tile), dims=_text(dims), theta=rng.choice([256.0, 10000.0]), step=rng.choice([0.5, 1.0, 1.75]),
             halves=rng.random() < 0.5, layout=rng.choice(["bhnd", "bnhd", "qkv"]))
    if op == "rope":
        c["inverse"] = rng.random() < 0.5
    if op == "norm_rope_backward":
        c["tiled"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- geometry

def _tokens(case):
    return sum(_ints(case, "prefix")) + math.prod(_ints(case, "grid"))


def _prefix_positions(case):
    """Positions of the prefix tokens: segment 0 (text) stands at the origin and is not
    rotated; every later segment is a reference image of 16 columns at time -s."""
    out = []
    for s, n in enumerate(_ints(case, "prefix")):
        i = torch.arange(n, dtype=torch.float64)
        if s == 0:
            out.append(torch.zeros(n, 3, dtype=torch.float64))
        else:
            out.append(torch.stack([torch.full((n,), -float(s), dtype=torch.float64),
                                    torch.div(i, 16, rounding_mode="floor"), i % 16], 1))
    return torch.cat(out) if out else torch.zeros(0, 3, dtype=torch.float64)


def _positions(case):
    """float64 [N, 3]: the prefix's own, then the video grid, t-major."""
    T, Hg, Wg = _ints(case, "grid")
    ax = torch.meshgrid(torch.arange(T), torch.arange(Hg), torch.arange(Wg), indexing="ij")
    vid = torch.stack([a.reshape(-1).double() for a in ax], 1) * case["step"]
    return torch.cat([_prefix_positions(case), vid]).to(DEV)


def _row_src(case):
    """Token of every row of the tile layout (-1: padding), and the live rows of each tile."""
    tt, th, tw = _ints(case, "tile")
    R = tt * th * tw
    rows, start = [], 0
    for n in _ints(case, "prefix"):
        if n:
            r = torch.full((-(-n // R) * R,), -1, dtype=torch.long)
            r[:n] = start + torch.arange(n)
            rows.append(r)
        start += n
    T, Hg, Wg = _ints(case, "grid")
    if T * Hg * Wg:
        t, h, w = torch.meshgrid(torch.arange(T), torch.arange(Hg), torch.arange(Wg), indexing="ij")
        nh, nw = -(-Hg // th), -(-Wg // tw)
        cube = ((t // tt) * nh + h // th) * nw + w // tw
        inside = ((t % tt) * th + h % th) * tw + w % tw
        order = torch.argsort((cube * R + inside).reshape(-1))
        cube = cube.reshape(-1)[order]
        count = torch.bincount(cube)
        first = torch.cumsum(count, 0) - count
        slot = torch.arange(order.numel()) - first[cube]
        r = torch.full((count.numel() * R,), -1, dtype=torch.long)
        r[cube * R + slot] = start + order
        rows.append(r)
    src = torch.cat(rows) if rows else torch.zeros(0, dtype=torch.long)
    live = (src.view(-1, R) >= 0).sum(1)
    return src.to(DEV), live.to(DEV), R


def _inv_freq(case):
    """float64 [P]: theta^(-2i / dim) for the pairs of each axis in turn, and their axis."""
    f, a = [], []
    for axis, d in enumerate(_ints(case, "dims")):
        i = torch.arange(d // 2, dtype=torch.float64)
        f.append(case["theta"] ** (-2.0 * i / max(d, 1)))
        a.append(torch.full((d // 2,), axis, dtype=torch.long))
    return torch.cat(f).to(DEV), torch.cat(a).to(DEV)


# ---------------------------------------------------------------- inputs

def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)


def _heads(gen, case, n):
    """n tensors [B,H,N,D] of N(0, s_h^2), s_h in [0.5, 2], in the case's memory layout."""
    B, H, N, D = case["B"], case["H"], _tokens(case), case["D"]
    s = 0.5 + 1.5 * torch.rand(H, generator=gen, device=DEV)
    if case["layout"] == "qkv":
        fused = torch.empty(B, N, 3, H, D, dtype=torch.bfloat16, device=DEV)
        for j in range(3):
            fused[:, :, j] = torch.randn(B, N, H, D, generator=gen, device=DEV) * s[:, None]
        return [fused[:, :, j].transpose(1, 2) for j in range(n)]
    out = []
    for _ in range(n):
        if case["layout"] == "bnhd":
            x = (torch.randn(B, N, H, D, generator=gen, device=DEV) * s[:, None]).bfloat16().transpose(1, 2)
        else:
            x = (torch.randn(B, H, N, D, generator=gen, device=DEV) * s[:, None, None]).bfloat16()
        out.append(x)
    return out


def _rows(gen, B, N, heads, width, scale=1.0):
    if heads:
        return _randn(gen, B, heads, N, width // heads, scale=scale)
    return _randn(gen, B, N, width, scale=scale)


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "rope":
        s["x"] = _heads(gen, case, 1)[0]
    elif op in ("norm_rope", "norm_rope_tiles", "norm_rope_backward"):
        s["q"], s["k"], s["v"] = _heads(gen, case, 3)
        s["wq"] = 1.0 + 0.2 * torch.randn(case["D"], generator=gen, device=DEV)
        s["wk"] = 1.0 + 0.2 * torch.randn(case["D"], generator=gen, device=DEV)
        if op == "norm_rope_backward":
            B, H, N, D = case["B"], case["H"], _tokens(case), case["D"]
            if case["tiled"]:
                src, _, _ = _row_src(case)
                s["dy"] = []
                for _ in range(3):
                    d = _randn(gen, B, H, src.numel(), D)
                    d[:, :, src < 0] = 0
                    s["dy"].append(d)
            else:
                s["dy"] = [_randn(gen, B, H, N, D) for _ in range(2)]
    elif op == "act_backward":
        s["dy"] = _randn(gen, case["B"], case["N"], case["O"])
        s["pre"] = _randn(gen, case["B"], case["N"], case["O"], scale=1.5)
    else:
        B, N, C, O = case["B"], case["N"], case["C"], case["O"]
        s["w"] = _randn(gen, O, C, scale=C ** -0.5)
        if op == "linear":
            s["x"] = _rows(gen, B, N, case["x_heads"], C)
            s["bias"] = _randn(gen, O, scale=0.1) if case["bias"] else None
            s["residual"] = _rows(gen, B, N, case["y_heads"], O) if case["residual"] else None
        else:
            s["dy"] = _rows(gen, B, N, case["y_heads"], O)
            if case["act"] == "identity":
                s["x"], s["x_pre"] = _rows(gen, B, N, case["x_heads"], C), None
            else:
                s["x_pre"] = _rows(gen, B, N, case["x_heads"], C, scale=1.5)
                s["x"] = _act32(s["x_pre"].float(), case["act"]).bfloat16()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("linear", "linear_backward", "act_backward"):
        if own:
            from tile_sparse_video_b200 import vsa
            s["plan"] = vsa.Plan((case["B"] * case["N"],), (0, 4, 4), (4, 4, 4))
            if op == "linear_backward":
                s["ws"] = vsa.linear_backward_workspace(s["plan"], case["B"], case["N"], case["C"], case["O"])
        return s
    if own:
        from tile_sparse_video_b200 import vsa
        s["plan"] = vsa.Plan(_ints(case, "prefix"), _ints(case, "grid"), _ints(case, "tile"))
        s["rope"] = vsa.Rope(s["plan"], _ints(case, "dims"), theta=case["theta"], step=(case["step"],) * 3,
                             halves=case["halves"], prefix_pos=_prefix_positions(case).numpy())
        if op == "norm_rope_backward":
            s["ws"] = vsa.norm_rope_backward_workspace(s["plan"], len(s["dy"]), case["D"])
    else:
        f, axis = _inv_freq(case)
        ang = _positions(case)[:, axis] * f
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["row_src"], s["live"], s["R"] = _row_src(case)
    return s


def _rows_like(case, s, heads, width):
    B, N, h, w = case["B"], case["N"], case[heads], case[width]
    shape = (B, h, N, w // h) if h else (B, N, w)
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV)


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from tile_sparse_video_b200 import vsa
    case, plan = s["case"], s["plan"]
    op = case["op"]
    if op == "rope":
        return vsa.vsa_rope_apply(plan, s["rope"], s["x"], inverse=case["inverse"])
    if op == "norm_rope":
        return vsa.vsa_norm_rope(plan, [vsa.HeadTensor(s["q"], s["wq"]), vsa.HeadTensor(s["k"], s["wk"])],
                                 s["rope"], eps=EPS)
    if op == "norm_rope_tiles":
        return vsa.vsa_norm_rope_permute_pool(
            plan, [vsa.HeadTensor(s["q"], s["wq"]), vsa.HeadTensor(s["k"], s["wk"]),
                   vsa.HeadTensor(s["v"], norm=False, rotate=False)], s["rope"], eps=EPS)
    if op == "norm_rope_backward":
        items = [vsa.HeadGrad(s["dy"][0], s["q"], s["wq"]), vsa.HeadGrad(s["dy"][1], s["k"], s["wk"])]
        if case["tiled"]:
            items.append(vsa.HeadGrad(s["dy"][2], norm=False, rotate=False))
        out = vsa.vsa_norm_rope_backward(plan, items, s["rope"], eps=EPS, tiled=case["tiled"], ws=s["ws"])
        return [t for pair in out for t in pair if t is not None]
    if op == "act_backward":
        return vsa.vsa_act_backward(plan, s["dy"], s["pre"], case["act"])
    if op == "linear":
        pre = _rows_like(case, s, "y_heads", "O") if case["pre"] else None
        y = vsa.vsa_linear(plan, s["x"], s["w"], bias=s["bias"], act=case["act"], residual=s["residual"],
                           y_heads=case["y_heads"], pre=pre)
        return [y, pre] if case["pre"] else [y]
    return list(vsa.vsa_linear_backward(plan, s["dy"], s["x"], s["w"], x_pre=s["x_pre"], x_act=case["act"],
                                        ws=s["ws"]))


def _act32(x, act):
    if act == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu_tanh":
        return x / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _dact32(x, act):
    if act == "identity":
        return torch.ones_like(x)
    if act == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = 1.0 / (1.0 + torch.exp(-c * (x + 0.044715 * x * x * x)))
        return s + x * s * (1.0 - s) * (c * (1.0 + 3.0 * 0.044715 * x * x))
    s = 1.0 / (1.0 + torch.exp(-x))
    return s * (1.0 - s) if act == "sigmoid" else s + x * s * (1.0 - s)


def _rotate32(z, s, inverse):
    """Rotate float32 [..., N, D] by the state's angles (backwards where inverse)."""
    P = s["cos"].shape[1]
    cos, sin = s["cos"], -s["sin"] if inverse else s["sin"]
    out = z.clone()
    if s["case"]["halves"]:
        a, b = z[..., :P], z[..., P:2 * P]
        out[..., :P], out[..., P:2 * P] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = z[..., 0:2 * P:2], z[..., 1:2 * P:2]
        out[..., 0:2 * P:2], out[..., 1:2 * P:2] = a * cos - b * sin, a * sin + b * cos
    return out


def _flat(x):
    """[B,N,C] or [B,H,N,D] -> float32 [B*N, C]."""
    if x.dim() == 4:
        x = x.transpose(1, 2)
    return x.float().reshape(x.shape[0] * x.shape[1], -1)


def _unflat(y, B, N, heads):
    y = y.view(B, N, -1)
    return y.view(B, N, heads, -1).transpose(1, 2).contiguous() if heads else y


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        return _rotate32(s["x"].float(), s, case["inverse"]).bfloat16()
    if op in ("norm_rope", "norm_rope_tiles"):
        out = []
        for name in ("q", "k") if op == "norm_rope" else ("q", "k", "v"):
            z = s[name].float()
            if name != "v":
                r = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)
                z = _rotate32(z * r * s["w" + name], s, False)
            if op == "norm_rope":
                out.append(z.bfloat16())
                continue
            src = s["row_src"]
            t = z[:, :, src.clamp(min=0)]
            t[:, :, src < 0] = 0
            mean = t.view(*t.shape[:2], -1, s["R"], t.shape[-1]).sum(3) / s["live"][:, None]
            out.append((t.bfloat16(), mean))
        return out
    if op == "norm_rope_backward":
        out = []
        for i, dy in enumerate(s["dy"]):
            g = dy.float()
            if case["tiled"]:
                src = s["row_src"]
                live = src >= 0
                n = torch.empty(*g.shape[:2], _tokens(case), g.shape[-1], device=DEV)
                n[:, :, src[live]] = g[:, :, live]
                g = n
            if i == 2:
                out.append(g.bfloat16())
                continue
            x, w = s["qk"[i]].float(), s["w" + "qk"[i]]
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            g = _rotate32(g, s, True)
            xh = x * r
            out_w = (g * xh).sum((0, 1, 2), dtype=torch.float64).float()
            g = g * w
            out += [(r * (g - xh * (g * xh).mean(-1, keepdim=True))).bfloat16(), out_w]
        return out
    if op == "act_backward":
        return (s["dy"].float() * _dact32(s["pre"].float(), case["act"])).bfloat16()
    B, N = case["B"], case["N"]
    if op == "linear":
        pre = _flat(s["x"]) @ s["w"].float().T
        if case["bias"]:
            pre = pre + s["bias"].float()
        y = _act32(pre, case["act"])
        if case["residual"]:
            y = y + _flat(s["residual"])
        out = [_unflat(y, B, N, case["y_heads"]).bfloat16()]
        if case["pre"]:
            out.append(_unflat(pre, B, N, case["y_heads"]).bfloat16())
        return out
    dy = _flat(s["dy"])
    dx = dy @ s["w"].float()
    if case["act"] != "identity":
        dx = dx * _dact32(_flat(s["x_pre"]), case["act"])
    dw = dy.T @ _flat(s["x"])
    return [_unflat(dx, B, N, case["x_heads"]).bfloat16(), dw.bfloat16(),
            dy.sum(0, dtype=torch.float64).float()]


# ---------------------------------------------------------------- the least work

def work(case):
    op = case["op"]
    if op == "act_backward":
        n = case["B"] * case["N"] * case["O"]
        return {"bytes": 3 * n * 2, "flops": 10 * n}
    if op in ("linear", "linear_backward"):
        M, C, O = case["B"] * case["N"], case["C"], case["O"]
        if op == "linear":
            outs = 1 + int(case["residual"]) + int(case["pre"])
            return {"bytes": 2 * (M * C + O * C + outs * M * O + O * int(case["bias"])), "flops": 2 * M * C * O}
        through = 0 if case["act"] == "identity" else 1
        return {"bytes": 2 * (M * O + (2 + through) * M * C + 2 * O * C) + 4 * O, "flops": 4 * M * C * O}
    n = case["B"] * case["H"] * _tokens(case) * case["D"]
    if op == "rope":
        return {"bytes": 4 * n, "flops": 3 * n}
    if op == "norm_rope":
        return {"bytes": 2 * 4 * n, "flops": 2 * 7 * n}
    R = math.prod(_ints(case, "tile"))
    tiles = sum(-(-p // R) for p in _ints(case, "prefix"))
    tiles += math.prod(-(-g // t) for g, t in zip(_ints(case, "grid"), _ints(case, "tile")))
    pad = case["B"] * case["H"] * tiles * R * case["D"]
    if op == "norm_rope_tiles":
        return {"bytes": 3 * (2 * n + 2 * pad + 4 * pad // R), "flops": (2 * 7 + 3) * n}
    return {"bytes": 2 * 6 * n + (4 * n if case["tiled"] else 0), "flops": 2 * 14 * n}


# ---------------------------------------------------------------- in 64 bits

def _turn64(case):
    """Unit complex numbers exp(i angle), complex128 [N, P], angle by angle."""
    pos = _positions(case)
    cols = []
    for axis, d in enumerate(_ints(case, "dims")):
        for i in range(d // 2):
            cols.append(pos[:, axis] * math.pow(case["theta"], -2.0 * i / d))
    ang = torch.stack(cols, 1) if cols else torch.zeros(pos.shape[0], 0, dtype=torch.float64, device=DEV)
    return torch.polar(torch.ones_like(ang), ang)


def _spin64(x, turn, halves):
    P = turn.shape[1]
    a, b = (x[:, :P], x[:, P:2 * P]) if halves else (x[:, 0:2 * P:2], x[:, 1:2 * P:2])
    c = torch.complex(a.contiguous(), b.contiguous()) * turn
    rot = torch.cat([c.real, c.imag], 1) if halves else torch.view_as_real(c).reshape(x.shape[0], 2 * P)
    return torch.cat([rot, x[:, 2 * P:]], 1)


def _act64(x, act):
    if act == "sigmoid":
        return torch.sigmoid(x)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    return x


def _slope64(x, act):
    with torch.enable_grad():
        v = x.detach().clone().requires_grad_(True)
        return torch.autograd.grad(_act64(v, act).sum(), v)[0]


def _by_head(t, b, N):
    """Rows of batch element b, float64 [N, C], channels in head order."""
    return torch.cat([t[b, h] for h in range(t.shape[1])], 1).double() if t.dim() == 4 else t[b].double()


def _like(t, parts):
    """Rows per batch element, [N, C] each, laid out like t."""
    if t.dim() == 4:
        D = t.shape[-1]
        return torch.stack([torch.stack(p.split(D, 1)) for p in parts])
    return torch.stack(parts)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "act_backward":
        return s["dy"].double() * _slope64(s["pre"].double(), case["act"])
    if op == "linear":
        w = s["w"].double()
        ys, ps = [], []
        for b in range(case["B"]):
            p = torch.einsum("nc,oc->no", _by_head(s["x"], b, case["N"]), w)
            if case["bias"]:
                p += s["bias"].double()
            y = _act64(p, case["act"])
            if case["residual"]:
                y = y + _by_head(s["residual"], b, case["N"])
            ys.append(y)
            ps.append(p)
        like = _rows_like(case, s, "y_heads", "O")
        return [_like(like, ys)] + ([_like(like, ps)] if case["pre"] else [])
    if op == "linear_backward":
        w = s["w"].double()
        dxs, dw, db = [], torch.zeros_like(w), torch.zeros(case["O"], dtype=torch.float64, device=DEV)
        for b in range(case["B"]):
            dy = _by_head(s["dy"], b, case["N"])
            dx = torch.einsum("no,oc->nc", dy, w)
            if case["act"] != "identity":
                dx = dx * _slope64(_by_head(s["x_pre"], b, case["N"]), case["act"])
            dxs.append(dx)
            dw += torch.einsum("no,nc->oc", dy, _by_head(s["x"], b, case["N"]))
            db += dy.sum(0)
        return [_like(s["x"], dxs), dw, db]
    turn, halves = _turn64(case), case["halves"]
    B, H, D = case["B"], case["H"], case["D"]
    if op == "rope":
        t = turn.conj() if case["inverse"] else turn
        return torch.stack([torch.stack([_spin64(s["x"][b, h].double(), t, halves) for h in range(H)])
                            for b in range(B)])
    src, live, R = _row_src(case)
    token_rows = torch.nonzero(src >= 0).view(-1)
    untile = torch.empty(_tokens(case), dtype=torch.long, device=DEV)
    untile[src[token_rows]] = token_rows
    if op in ("norm_rope", "norm_rope_tiles"):
        out = []
        for name in ("q", "k") if op == "norm_rope" else ("q", "k", "v"):
            ys, means = [], []
            for b in range(B):
                for h in range(H):
                    y = s[name][b, h].double()
                    if name != "v":
                        y = y / torch.sqrt(y.square().sum(1, keepdim=True) / D + EPS) * s["w" + name].double()
                        y = _spin64(y, turn, halves)
                    if op == "norm_rope_tiles":
                        t = torch.zeros(src.numel(), D, dtype=torch.float64, device=DEV)
                        t[untile] = y
                        m = torch.zeros(live.numel(), D, dtype=torch.float64, device=DEV)
                        m.index_add_(0, untile // R, y)
                        means.append(m / live[:, None])
                        y = t
                    ys.append(y)
            y = torch.stack(ys).view(B, H, -1, D)
            out.append(y if op == "norm_rope" else (y, torch.stack(means).view(B, H, -1, D)))
        return out
    out = []
    for i, dy in enumerate(s["dy"]):
        rows, dw = [], torch.zeros(D, dtype=torch.float64, device=DEV)
        for b in range(B):
            for h in range(H):
                g = dy[b, h].double()
                if case["tiled"]:
                    g = g[untile]
                if i < 2:
                    x = s["qk"[i]][b, h].double()
                    n = torch.sqrt(x.square().sum(1, keepdim=True) / D + EPS)
                    u = x / n
                    g = _spin64(g, turn.conj(), halves)
                    dw += (g * u).sum(0)
                    g = g * s["w" + "qk"[i]].double()
                    g = g / n - u * (g * u).sum(1, keepdim=True) / (D * n)
                rows.append(g)
        out.append(torch.stack(rows).view(B, H, -1, D))
        if i < 2:
            out.append(dw)
    return out
