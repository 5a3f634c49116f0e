"""GPU parity of the operators around the layer (include/vsa_block.h) with their fp64
oracle, and their refusals.

Tolerances.  A bf16 output is one rounding, at most 2^-8 of its value (half of
finfo(bfloat16).eps), of an fp32 result; what fp32 adds is bounded beside each check
by the magnitudes that enter it (2^-24 an operation; 2^-22 the reciprocal root)."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import block_oracle as BO
from tests.parity import f64
from tile_sparse_video_b200 import vsa

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda(libvsa):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def close(got, want, slack, what="", half_step=2.0 ** -8):
    """|got - want| <= half_step * |want| + slack (the fp32 part), element by element."""
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.all(np.isfinite(got)), what
    over = np.abs(got - want) - (half_step * np.abs(want) + slack)
    assert np.all(over <= 0), (what, float(over.max()))


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).bfloat16().cuda()


def laid_out(x, layout):
    """The same [B,H,N,D] values in another memory layout."""
    if layout == "bhnd":
        return x
    B, H, N, D = x.shape
    if layout == "bnhd":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    fused = torch.full((B, N, 3, H, D), float("nan"), dtype=x.dtype, device=x.device)
    fused[:, :, 1] = x.transpose(1, 2)
    return fused[:, :, 1].transpose(1, 2)


# (name, prefix, grid, tile, B, H, D, dims, halves, layout)
GEOS = [
    ("one_token", (1,), (0, 4, 4), (4, 4, 4), 1, 1, 128, (44, 42, 42), False, "bhnd"),
    ("one_token_d64", (), (1, 1, 1), (4, 4, 4), 1, 3, 64, (24, 20, 20), True, "bnhd"),
    ("tiny", (40, 70), (4, 8, 8), (4, 4, 4), 1, 2, 64, (24, 20, 20), False, "bhnd"),
    ("ragged_b2", (5, 0, 64, 65), (5, 6, 7), (4, 4, 4), 2, 3, 64, (16, 24, 24), True, "qkv"),
    ("ragged_r128", (256, 3), (8, 17, 9), (4, 8, 4), 1, 3, 128, (44, 42, 42), False, "qkv"),
    ("image_only", (), (1, 13, 11), (4, 4, 4), 2, 2, 128, (0, 64, 64), True, "bnhd"),
    ("partial", (7,), (3, 3, 5), (4, 8, 4), 1, 5, 128, (10, 6, 2), False, "bhnd"),
    ("partial_halves", (130,), (2, 3, 3), (4, 4, 4), 1, 2, 128, (16, 16, 8), True, "bnhd"),
    ("odd_pairs_d64", (33,), (2, 5, 3), (4, 4, 4), 1, 2, 64, (2, 22, 20), False, "qkv"),
]
geos = pytest.mark.parametrize("g", GEOS, ids=lambda g: g[0])


def setup(g, seed=0):
    _, prefix, grid, tile, B, H, D, dims, halves, layout = g
    plan = vsa.Plan(prefix, grid, tile)
    n_p = sum(prefix)
    pos = np.random.default_rng(seed).integers(-40, 3000, (n_p, 3)).astype(np.float64) if n_p else None
    rope = vsa.Rope(plan, dims, theta=(1e4, 256.0, 1e4), offset=(0.5, 0, 0), step=(1, 0.75, 2),
                    halves=halves, prefix_pos=pos)
    ang = BO.angles(BO.positions(prefix, grid, (0.5, 0, 0), (1, 0.75, 2), pos), dims, (1e4, 256.0, 1e4))
    return plan, rope, ang, (B, H, plan.n_tokens, D), layout


def rot_slack(z):
    """Rotation in fp32: two products, a sum and rounded tables, of the row's largest element."""
    return 8 * 2.0 ** -24 * 2 * np.abs(z).max(-1, keepdims=True) + 1e-30


@geos
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(g, inverse):
    plan, rope, ang, shape, layout = setup(g)
    x = laid_out(randn(1, *shape), layout)
    want = BO.rotate(x, ang, g[8], inverse)
    y = vsa.vsa_rope_apply(plan, rope, x, inverse=inverse)
    close(y, want, rot_slack(f64(x)), "y")
    # into a strided output, and in place: the same bits
    out = laid_out(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), "bnhd")
    assert torch.equal(vsa.vsa_rope_apply(plan, rope, x, out, inverse=inverse), y)
    assert torch.equal(vsa.vsa_rope_apply(plan, rope, x, x, inverse=inverse), y)
    vsa.vsa_sync_status(plan)


@geos
def test_norm_rope(g):
    plan, rope, ang, shape, layout = setup(g)
    D = shape[-1]
    q, k, v = (laid_out(randn(s, *shape, scale=3.0 * s), layout) for s in (1, 2, 3))
    q[..., 0, :] = 0                                       # a row of zeros
    wq = 1 + 0.2 * randn(7, D).float()
    wk = (1 + 0.2 * randn(8, D).float()).bfloat16()
    ys = vsa.vsa_norm_rope(plan, [vsa.HeadTensor(q, wq), vsa.HeadTensor(k, wk, rotate=False),
                                  vsa.HeadTensor(v, norm=False), vsa.HeadTensor(v)], rope, EPS)
    z = [BO.head_norm(q, wq, EPS), BO.head_norm(k, wk, EPS), f64(v), BO.head_norm(v, None, EPS)]
    want = [BO.rotate(z[0], ang, g[8]), z[1], BO.rotate(z[2], ang, g[8]), BO.rotate(z[3], ang, g[8])]
    for i in range(4):
        # the norm: a sum of D squares in fp32 (D 2^-24 at most, halved by the root) and 4 operations
        close(ys[i], want[i], rot_slack(z[i]) + (D / 2 + 8) * 2.0 ** -24 * np.abs(z[i]).max(-1, keepdims=True),
              str(i))
    assert torch.all(ys[0][..., 0, :] == 0)
    # in place
    vsa.vsa_norm_rope(plan, [vsa.HeadTensor(q, wq, y=q), vsa.HeadTensor(k, wk, rotate=False, y=k)], rope, EPS)
    assert torch.equal(q, ys[0]) and torch.equal(k, ys[1])
    vsa.vsa_sync_status(plan)


@geos
def test_norm_rope_permute_pool(g):
    plan, rope, ang, shape, layout = setup(g)
    D = shape[-1]
    q, k, v = (laid_out(randn(s, *shape, scale=2.0), layout) for s in (4, 5, 6))
    wq = 1 + 0.2 * randn(7, D).float()
    out = vsa.vsa_norm_rope_permute_pool(
        plan, [vsa.HeadTensor(q, wq), vsa.HeadTensor(k), vsa.HeadTensor(v, norm=False, rotate=False)], rope, EPS)
    p = O.plan(g[1], g[2], g[3])
    nat = vsa.vsa_norm_rope(plan, [vsa.HeadTensor(q, wq), vsa.HeadTensor(k)], rope, EPS)
    for (y_t, pooled), y, x, w in zip(out, [*nat, v], (q, k, v), (wq, None, None)):
        # the same rows as the natural form, permuted; pad rows 0
        assert torch.equal(y_t, vsa.vsa_permute(plan, y.contiguous()))
        z = f64(x) if x is v else BO.rotate(BO.head_norm(x, w, EPS), ang, g[8])
        want = O.pool(O.permute(z, p), p)
        big = O.pool(O.permute(np.abs(z).max(-1, keepdims=True) * np.ones(D), p), p)
        # fp32 rows as above, and a mean of up to 128 rows in fp32
        close(pooled, want, (D / 2 + 32 + 128) * 2.0 ** -24 * big + 1e-30, "pooled", half_step=0.0)
    y_t, pooled = vsa.vsa_permute_pool(plan, v.contiguous())
    assert torch.equal(out[2][0], y_t)
    vsa.vsa_sync_status(plan)


@geos
def test_means_of_what_only_goes_through(g):
    """Without norm and rotation the rows are vsa_permute_pool's, and the means too but for the order of the
    sum: two fp32 sums of up to n terms and a product with 1/n, each within n + 1 roundings of the mean
    magnitude.  A run after another gives the same bits."""
    plan, _, _, shape, layout = setup(g)
    x = laid_out(randn(6, *shape, scale=2.0), layout)
    (y_t, pooled), = vsa.vsa_norm_rope_permute_pool(plan, [vsa.HeadTensor(x, norm=False, rotate=False)])
    want_t, want = vsa.vsa_permute_pool(plan, x.contiguous())
    vsa.vsa_sync_status(plan)
    assert torch.equal(y_t, want_t)
    p = O.plan(g[1], g[2], g[3])
    size = O.pool(O.permute(np.abs(f64(x)), p), p)
    n = plan.tile_rows
    assert np.all(np.abs(f64(pooled) - f64(want)) <= 2 * (n + 2) * 2.0 ** -24 * size)
    again = vsa.vsa_norm_rope_permute_pool(plan, [vsa.HeadTensor(x, norm=False, rotate=False)])[0][1]
    assert torch.equal(pooled, again)


@geos
@pytest.mark.parametrize("tiled", [False, True])
def test_norm_rope_backward(g, tiled):
    plan, rope, ang, shape, layout = setup(g)
    D = shape[-1]
    q, k = (laid_out(randn(s, *shape, scale=2.0), layout) for s in (4, 5))
    wq = 1 + 0.2 * randn(7, D).float()
    wk = (1 + 0.2 * randn(8, D).float()).bfloat16()
    dys = [randn(s, *shape) for s in (11, 12, 13)]
    given = [vsa.vsa_permute(plan, d) for d in dys] if tiled else [laid_out(d, layout) for d in dys]
    dx0 = laid_out(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), "qkv")
    dgk = torch.full((D,), float("nan"), device="cuda")
    res = vsa.vsa_norm_rope_backward(
        plan, [vsa.HeadGrad(given[0], q, wq, dx=dx0), vsa.HeadGrad(given[1], k, wk, rotate=False, d_gain=dgk),
               vsa.HeadGrad(given[2], norm=False, rotate=False)], rope, EPS, tiled=tiled)
    vsa.vsa_sync_status(plan)
    assert torch.equal(res[2][0], dys[2]) and res[2][1] is None
    for (dx, dw), x, w, dy, rot in zip(res[:2], (q, k), (wq, wk), dys, (True, False)):
        gr = BO.rotate(dy, ang, g[8], inverse=True) if rot else f64(dy)
        want, want_w = BO.head_norm_backward(gr, x, w, EPS)
        r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + EPS)
        big = np.abs(gr * f64(w)).max(-1, keepdims=True)
        u = np.abs(f64(x) * r).max(-1, keepdims=True)
        # two sums of D products in fp32 and some ten operations on r g gain and r u mean(g gain u)
        close(dx, want, (2 * D + 32) * 2.0 ** -24 * r * (big + u * u * big), "dx")
        s = np.abs(gr * f64(x) * r).sum((0, 1, 2))
        rows = gr.shape[0] * gr.shape[1] * gr.shape[2]
        close(dw, want_w, (rows + D / 2 + 64) * 2.0 ** -24 * s + 1e-30, "d_gain", half_step=0.0)


def test_norm_rope_broadcast_and_status():
    """A head that several share (stride 0) is read as often as it stands; gradients come
    for each."""
    plan = vsa.Plan((9,), (2, 4, 4), (4, 4, 4))
    rope = vsa.Rope(plan, (24, 20, 20))
    k1 = randn(3, 1, 1, plan.n_tokens, 64)
    k = k1.expand(2, 4, plan.n_tokens, 64)
    y, = vsa.vsa_norm_rope(plan, [vsa.HeadTensor(k)], rope)
    one, = vsa.vsa_norm_rope(plan, [vsa.HeadTensor(k1)], rope)
    assert torch.equal(y, one.expand_as(y))
    dy = randn(4, 2, 4, plan.n_tokens, 64)
    (dx, _), = vsa.vsa_norm_rope_backward(plan, [vsa.HeadGrad(dy, k)], rope)
    (dz, _), = vsa.vsa_norm_rope_backward(plan, [vsa.HeadGrad(dy, k.contiguous())], rope)
    assert torch.equal(dx, dz)
    with pytest.raises(vsa.VsaError) as e:                 # outputs do not share memory
        vsa.vsa_norm_rope(plan, [vsa.HeadTensor(y, y=k)], rope)
    assert e.value.status == 1


def test_rope_that_nothing_asks_for():
    """Without a rotating tensor the rope is not looked at: one that is too wide for D, in halves, or of
    another plan changes nothing."""
    plan, other = vsa.Plan((9,), (2, 4, 4), (4, 4, 4)), vsa.Plan((3,), (1, 4, 4), (4, 4, 4))
    x = randn(1, 1, 2, plan.n_tokens, 64)
    item = [vsa.HeadTensor(x, rotate=False)]
    want, = vsa.vsa_norm_rope(plan, item)
    (want_t, _), = vsa.vsa_norm_rope_permute_pool(plan, item)
    (want_g, _), = vsa.vsa_norm_rope_backward(plan, [vsa.HeadGrad(x, x, rotate=False)])
    for rope in (vsa.Rope(plan, (44, 42, 42), halves=True), vsa.Rope(other, (24, 20, 20), halves=True)):
        assert torch.equal(vsa.vsa_norm_rope(plan, item, rope)[0], want)
        assert torch.equal(vsa.vsa_norm_rope_permute_pool(plan, item, rope)[0][0], want_t)
        assert torch.equal(vsa.vsa_norm_rope_backward(plan, [vsa.HeadGrad(x, x, rotate=False)], rope)[0][0], want_g)
    vsa.vsa_sync_status(plan)


def test_norm_rope_refusals():
    plan = vsa.Plan((9,), (2, 4, 4), (4, 4, 4))
    other = vsa.Plan((8,), (2, 4, 4), (4, 4, 4))
    rope, rope_o = vsa.Rope(plan, (24, 20, 20)), vsa.Rope(other, (24, 20, 20))
    wide = vsa.Rope(plan, (44, 42, 42))
    N = plan.n_tokens
    x = randn(1, 1, 2, N, 64)
    w = torch.ones(64, device="cuda")

    def refused(status, fn, *a, **k):
        with pytest.raises(vsa.VsaError) as e:
            fn(*a, **k)
        assert e.value.status == status, str(e.value)
    H = vsa.HeadTensor
    refused(1, vsa.vsa_norm_rope, plan, [H(x)], None)              # rotates without a rope
    refused(1, vsa.vsa_norm_rope, plan, [H(x)], rope_o)
    refused(1, vsa.vsa_norm_rope, plan, [H(x)], wide)
    refused(1, vsa.vsa_norm_rope, plan, [H(x)], rope, eps=0.0)
    refused(1, vsa.vsa_norm_rope, plan, [H(x)], rope, eps=float("nan"))
    refused(1, vsa.vsa_norm_rope, plan, [H(x, w, norm=False)], rope)
    refused(1, vsa.vsa_rope_apply, plan, rope_o, x)
    odd = torch.zeros(1, 2, N, 68, dtype=torch.bfloat16, device="cuda")[..., :64]
    refused(1, vsa.vsa_rope_apply, plan, rope, odd)                # stride not a multiple of 8
    off = torch.zeros(2 * N * 64 + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 2 * N * 64].view(1, 2, N, 64)
    refused(1, vsa.vsa_rope_apply, plan, rope, off)                # not 16-byte aligned
    refused(1, vsa.vsa_rope_apply, plan, rope, x, x.as_strided((1, 2, N, 64), (0, 64, 128, 1)))   # other strides
    refused(2, vsa.vsa_norm_rope, plan, [H(torch.zeros(1, 2, N, 96, dtype=torch.bfloat16, device="cuda"))], rope)
    refused(4, vsa.vsa_norm_rope_backward, plan, [vsa.HeadGrad(x, x, w)], rope,
            ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    refused(1, vsa.vsa_norm_rope_backward, plan, [vsa.HeadGrad(x, norm=False, d_gain=w.clone())], rope)
    for bad in ([], [H(x)] * 5):
        with pytest.raises(ValueError):
            vsa.vsa_norm_rope(plan, bad, rope)
    with pytest.raises(ValueError):
        vsa.vsa_norm_rope(plan, [H(x), H(x[:, :1])], rope)
    with pytest.raises(TypeError):
        vsa.vsa_norm_rope(plan, [H(x.float())], rope)
    with pytest.raises(ValueError):
        vsa.vsa_norm_rope(plan, [H(x.cpu())], rope)
    with pytest.raises(ValueError):
        vsa.vsa_norm_rope(plan, [H(x.transpose(2, 3).contiguous().transpose(2, 3))], rope)
    vsa.vsa_sync_status(plan)


def test_rope_of_another_grid_or_prefix():
    """As many tokens in another grid, or with more of them in the prefix, stand elsewhere: refused.  Other
    segments and tiles of the same tokens, and the extents of an empty grid, change no position."""
    plan = vsa.Plan((9, 7), (2, 4, 6), (4, 4, 4))
    x = randn(1, 1, 2, plan.n_tokens, 64)
    want = vsa.vsa_rope_apply(plan, vsa.Rope(plan, (24, 20, 20)), x)
    others = [vsa.Plan(p, g, (4, 4, 4)) for p, g in (((9, 7), (2, 6, 4)), ((9, 7), (4, 2, 6)), ((40,), (2, 3, 4)))]
    for other in others:
        assert other.n_tokens == plan.n_tokens
        rope = vsa.Rope(other, (24, 20, 20))
        for call in (lambda: vsa.vsa_rope_apply(plan, rope, x), lambda: vsa.vsa_norm_rope(plan, [vsa.HeadTensor(x)], rope),
                     lambda: vsa.vsa_norm_rope_permute_pool(plan, [vsa.HeadTensor(x)], rope),
                     lambda: vsa.vsa_norm_rope_backward(plan, [vsa.HeadGrad(x, x)], rope)):
            with pytest.raises(vsa.VsaError) as e:
                call()
            assert e.value.status == 1
    for same in (vsa.Plan((16,), (2, 4, 6), (4, 4, 4)), vsa.Plan((1, 15), (2, 4, 6), (4, 8, 4))):
        assert torch.equal(vsa.vsa_rope_apply(plan, vsa.Rope(same, (24, 20, 20)), x), want)
    text, none = vsa.Plan((30,), (0, 4, 4), (4, 4, 4)), vsa.Plan((30,), (3, 0, 9), (4, 4, 4))
    vsa.vsa_rope_apply(text, vsa.Rope(none, (24, 20, 20)), randn(2, 1, 2, 30, 64))
    vsa.vsa_sync_status(plan)


# ---------------------------------------------------------------- linear

# (B, N, x_heads, C, y_heads, O)
LINEARS = [
    (1, 1, 0, 64, 0, 64), (1, 1, 0, 520, 0, 1032), (3, 1, 0, 8, 0, 8), (2, 1, 2, 128, 3, 192),
    (1, 7, 0, 32, 0, 264), (1, 255, 0, 72, 0, 256), (1, 257, 3, 384, 0, 136), (2, 300, 2, 256, 4, 256),
    (2, 513, 0, 200, 2, 128), (1, 1000, 4, 256, 3, 384), (1, 16, 0, 2048, 0, 40), (1, 33, 0, 264, 5, 640),
    (2, 4, 3, 384, 0, 72), (3, 3, 0, 1032, 2, 256), (2, 150, 9, 1152, 0, 96), (1, 700, 0, 40, 8, 1024),
]
linears = pytest.mark.parametrize("c", LINEARS, ids=lambda c: "x".join(map(str, c)))


def rows_or_heads(seed, B, N, heads, width, scale=1.0):
    if heads:
        return randn(seed, B, heads, N, width // heads, scale=scale)
    return randn(seed, B, N, width, scale=scale)


def dot_slack(a, b):
    """An fp32 sum of K products in steps of 16: each step may lose 2^-22 of the sum of
    magnitudes so far (the tensor core aligns and truncates), and no more than that is lost
    per term in an fp32 chain of FMAs."""
    K = a.shape[-1]
    return (K / 16 + 2) * 2.0 ** -22 * (np.abs(a) @ np.abs(b).T) + 1e-30


def act_slack(name, x, slack):
    """The activations' slopes are at most 1.13; their own arithmetic is good to 2^-18."""
    return 1.13 * slack + 2.0 ** -18 * np.abs(BO.act(name, x)) + 2.0 ** -22


@linears
@pytest.mark.parametrize("act", ["identity", "sigmoid", "gelu_tanh", "silu"])
def test_linear(c, act):
    B, N, xh, C, yh, Ow = c
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    x, w = rows_or_heads(1, B, N, xh, C), randn(2, Ow, C, scale=2 * C ** -0.5)
    bias = randn(3, Ow, scale=0.5)
    if act in ("sigmoid", "silu"):
        bias = bias.float()
    res = rows_or_heads(4, B, N, yh, Ow)
    pre = torch.empty_like(res)
    y = vsa.vsa_linear(plan, x, w, bias, act=act, residual=res, pre=pre)
    vsa.vsa_sync_status(plan)
    p = BO.linear(x, w, bias)
    slack = dot_slack(BO.rows(x), f64(w)) + 2.0 ** -23 * np.abs(p)
    close(pre, BO.heads(p, yh), BO.heads(slack, yh), "pre")
    a = BO.act(act, p)
    want = a + BO.rows(res)
    s = act_slack(act, p, slack) + 2.0 ** -24 * np.abs(want)
    close(y, BO.heads(want, yh), BO.heads(s, yh), "y")
    # without a workspace the K blocks are not split
    yw = torch.empty_like(y)
    xv, yv, rv = (vsa._view(plan, t, "t", t.shape) for t in (x, yw, res))
    args = vsa._LINEAR.pack(B, xh, C, yh, Ow, N, *xv, w.data_ptr(), *vsa._vector(plan, bias, "bias", Ow),
                            vsa.ACTS[act], *rv, *vsa._NO_VIEW, *yv)
    assert vsa.lib().vsa_linear(plan.handle, args, None, 0, vsa._raw_stream(plan, None)) == 0
    close(yw, BO.heads(want, yh), BO.heads(s, yh), "no workspace")
    # without bias and residual; the residual read from y itself
    y2 = vsa.vsa_linear(plan, x, w, act=act, y_heads=yh)
    p2 = BO.linear(x, w)
    close(y2, BO.heads(BO.act(act, p2), yh), BO.heads(act_slack(act, p2, slack), yh), "bare")
    y3 = res.clone()
    assert torch.equal(vsa.vsa_linear(plan, x, w, bias, act=act, residual=y3, y=y3), y)
    vsa.vsa_sync_status(plan)


@linears
def test_linear_backward(c):
    B, N, xh, C, yh, Ow = c
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    x, w, dy = rows_or_heads(1, B, N, xh, C), randn(2, Ow, C, scale=0.1), rows_or_heads(5, B, N, yh, Ow)
    dx, dw, db = vsa.vsa_linear_backward(plan, dy, x, w)
    vsa.vsa_sync_status(plan)
    wx, ww, wb = BO.linear_backward(dy, x, w)
    g, xr = BO.rows(dy), BO.rows(x)
    close(dx, BO.heads(wx, xh), BO.heads(dot_slack(g, f64(w).T), xh), "dx")
    M = B * N
    close(dw, ww, dot_slack(g.reshape(M, -1).T, xr.reshape(M, -1).T), "dw")
    close(db, wb, M * 2.0 ** -24 * np.abs(g).sum((0, 1)) + 1e-30, "db", half_step=0.0)


@pytest.mark.parametrize("c", [LINEARS[i] for i in (1, 6, 7, 9)], ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("act", ["sigmoid", "gelu_tanh", "silu"])
def test_linear_backward_through_activation(c, act):
    B, N, xh, C, yh, Ow = c
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    x_pre = rows_or_heads(1, B, N, xh, C, scale=2.0)
    x = torch.from_numpy(BO.act(act, x_pre)).bfloat16().cuda()
    w, dy = randn(2, Ow, C, scale=0.1), rows_or_heads(5, B, N, yh, Ow)
    dx, dw, db = vsa.vsa_linear_backward(plan, dy, x, w, x_pre=x_pre, x_act=act, need=(True, False, False))
    assert dw is None and db is None
    vsa.vsa_sync_status(plan)
    wx, _, _ = BO.linear_backward(dy, x, w)
    xp = BO.rows(x_pre)
    slope = BO.act_slope(act, xp)
    slack = 1.13 * dot_slack(BO.rows(dy), f64(w).T) + np.abs(wx) * (2.0 ** -18 * (1 + np.abs(xp)))
    close(dx, BO.heads(wx * slope, xh), BO.heads(slack, xh), "dx")


@pytest.mark.parametrize("c", [(1, 5000, 0, 520, 0, 1000), (2, 2600, 4, 512, 8, 1024), (1, 2500, 0, 512, 0, 2184)],
                         ids=lambda c: "x".join(map(str, c)))
def test_linear_full_waves_and_strips(c):
    """More tiles than pairs of SMs: the last ones are cut into strips of 64 columns, some of them
    over the last column; what lies beside the result stays as it was."""
    B, N, xh, C, yh, Ow = c
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    x, w, bias = rows_or_heads(1, B, N, xh, C), randn(2, Ow, C, scale=C ** -0.5), randn(3, Ow)
    res = rows_or_heads(4, B, N, yh, Ow)
    wide = torch.full((B, yh, N, Ow // yh + 64) if yh else (B, N, Ow + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    width = Ow // yh if yh else Ow
    y, pre = wide[..., :width], torch.empty_like(res)
    vsa.vsa_linear(plan, x, w, bias, act="gelu_tanh", residual=res, pre=pre, y=y)
    vsa.vsa_sync_status(plan)
    assert bool((wide[..., width:] == 7.0).all())
    p = BO.linear(x, w, bias)
    slack = dot_slack(BO.rows(x), f64(w)) + 2.0 ** -23 * np.abs(p)
    close(pre, BO.heads(p, yh), BO.heads(slack, yh), "pre")
    want = BO.act("gelu_tanh", p) + BO.rows(res)
    close(y, BO.heads(want, yh), BO.heads(act_slack("gelu_tanh", p, slack) + 2.0 ** -24 * np.abs(want), yh), "y")


@pytest.mark.parametrize("c", [(1, 2500, 0, 2184, 0, 512), (1, 520, 0, 2184, 0, 2504)],
                         ids=lambda c: "x".join(map(str, c)))
def test_linear_backward_full_waves_and_strips(c):
    test_linear_backward(c)


@pytest.mark.parametrize("act", ["identity", "sigmoid", "gelu_tanh", "silu"])
def test_act_backward(act):
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    dy, pre = randn(1, 3, 77, 40), randn(2, 3, 77, 40, scale=4.0)
    pre.view(-1)[:6] = torch.tensor([0.0, -0.0, 100.0, -100.0, 3e38, -3e38])
    got = vsa.vsa_act_backward(plan, dy, pre, act)
    vsa.vsa_sync_status(plan)
    d, p = f64(dy), f64(pre)
    with np.errstate(all="ignore"):
        want = d * np.nan_to_num(BO.act_slope(act, p))
    # beyond 1e12 the slopes are 1 or 0 (0 for sigmoid); the cube above overflows the oracle's terms
    far = np.abs(p) > 1e12
    if act in ("gelu_tanh", "silu"):
        want = np.where(far, d * (p > 0), want)
    elif act == "sigmoid":
        want = np.where(far, 0.0, want)
    close(got, want, np.abs(d) * 2.0 ** -18 * (1 + np.minimum(np.abs(p), 20.0)), act)
    out = dy.clone()
    assert torch.equal(vsa.vsa_act_backward(plan, out, pre, act, out=out), got)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_slopes_far_out(act):
    """Where a slope is small it is as exact, relative to itself, as one of the size of 1: 2^t for t = x log2(e)
    is off by |t| 2^-23 and the rest by some 2^-22, so 2^-18 (1 + |x|) is ample; sigmoid to both sides, SiLU to
    the left of its slope's root at -1.28, where x (1 - s) and 1 cancel to no less than a quarter."""
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    pre = torch.cat([torch.linspace(-80, -3, 1024), torch.linspace(3, 80, 1024)]).bfloat16().cuda()
    if act == "silu":
        pre = pre[:1024]
    dy = 1 + torch.arange(pre.numel(), device="cuda").remainder(7).bfloat16()
    got = f64(vsa.vsa_act_backward(plan, dy, pre, act))
    # the same through the product of an identity
    n, w = pre.numel() // 64, torch.eye(64, dtype=torch.bfloat16, device="cuda")
    rows = [t.view(1, n, 64) for t in (dy, pre)]
    dx, _, _ = vsa.vsa_linear_backward(plan, rows[0], rows[1], w, x_pre=rows[1], x_act=act, need=(True, False, False))
    vsa.vsa_sync_status(plan)
    x, d = f64(pre), f64(dy)
    e = np.exp(-np.abs(x))
    want = d * e / (1 + e) ** 2                                  # s(x) s(-x)
    if act == "silu":
        want = want * (1 + np.exp(x) + x)                        # s (1 + x s(-x))
    for g in (got, f64(dx).reshape(-1)):
        assert np.all(np.abs(g - want) <= (2.0 ** -8 + 2.0 ** -18 * (1 + np.abs(x))) * np.abs(want))


def test_linear_strided_and_empty():
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    B, N, C, Ow = 2, 70, 128, 192
    wide = randn(1, B, N + 3, C + 16)
    x = wide[:, 1:N + 1, 8:C + 8]
    w, bias = randn(2, Ow, C, scale=0.1), randn(3, Ow)
    ref = vsa.vsa_linear(plan, x.contiguous(), w, bias)
    buf = torch.zeros(B, N, 3, Ow, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(vsa.vsa_linear(plan, x, w, bias, y=buf[:, :, 1]), ref)
    assert torch.all(buf[:, :, 0] == 0) and torch.all(buf[:, :, 2] == 0)
    # a [B,N,H,D] tensor as heads
    xh = randn(4, B, N, 2, 64)
    assert torch.equal(vsa.vsa_linear(plan, xh.transpose(1, 2), w, bias),
                       vsa.vsa_linear(plan, xh.view(B, N, 128), w, bias))
    dy = buf[:, :, 1]
    dxs, dws, dbs = vsa.vsa_linear_backward(plan, dy, x, w)
    dxc, dwc, dbc = vsa.vsa_linear_backward(plan, dy.contiguous(), x.contiguous(), w)
    assert torch.equal(dxs, dxc) and torch.equal(dbs, dbc)
    close(dws, f64(dwc), 1e-30 + 2.0 ** -8 * np.abs(f64(dwc)), "dw")      # rows in other K blocks
    for shape in ((0, 5, C), (2, 0, C)):
        e = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        y = vsa.vsa_linear(plan, e, w, bias)
        assert y.shape == (*shape[:2], Ow)
        dx, dw, db = vsa.vsa_linear_backward(plan, y, e, w)
        assert dx.shape == e.shape and torch.all(dw == 0) and torch.all(db == 0)
    vsa.vsa_sync_status(plan)


def test_linear_refusals():
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    x, w = randn(1, 1, 9, 64), randn(2, 128, 64)

    def refused(status, fn, *a, **k):
        with pytest.raises(vsa.VsaError) as e:
            fn(*a, **k)
        assert e.value.status == status, str(e.value)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    refused(1, vsa.vsa_linear, plan, torch.zeros(1, 9, 60, **bf), torch.zeros(128, 60, **bf))
    refused(1, vsa.vsa_linear, plan, x, torch.zeros(12, 64, **bf))
    refused(2, vsa.vsa_linear, plan, torch.zeros(1, 2, 9, 32, **bf), w)        # heads of 32
    refused(1, vsa.vsa_linear, plan, x, torch.zeros(64, 64, **bf), y=x)        # y over x
    refused(1, vsa.vsa_linear, plan, x[:, :1].expand(1, 9, 64), w)             # broadcast rows
    wide, tall = torch.zeros(128, 4096, **bf), torch.zeros(1, 40, 4096, **bf)
    refused(4, vsa.vsa_linear, plan, tall, wide, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    refused(4, vsa.vsa_linear_backward, plan, torch.zeros(1, 9, 128, **bf), x, w,
            ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    refused(1, vsa.vsa_linear_backward, plan, torch.zeros(1, 9, 128, **bf), x, w, dx=x)
    for bad in (dict(act="relu"), dict(bias=torch.zeros(64, **bf)), dict(residual=torch.zeros(1, 9, 64, **bf))):
        with pytest.raises(ValueError):
            vsa.vsa_linear(plan, x, w, **bad)
    with pytest.raises(TypeError):
        vsa.vsa_linear(plan, x, w, bias=torch.zeros(128, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        vsa.vsa_linear_backward(plan, torch.zeros(1, 9, 128, **bf), x, w, x_act="silu")
    # plain C: unknown codes
    none = vsa._NO_VIEW
    for bias_type, act in ((0, 7), (2, 0), (0, -1)):
        args = vsa._LINEAR.pack(1, 0, 64, 0, 128, 9, *none, 0, 0, bias_type, act, *none, *none, *none)
        assert vsa.lib().vsa_linear(plan.handle, args, None, 0, None) == 1
    vsa.vsa_sync_status(plan)


def test_workspaces_on_the_host_are_refused():
    """In every call that takes one, the layer's among them: the library sees a pointer and a size only."""
    plan = vsa.Plan((9,), (2, 4, 4), (4, 4, 4))
    N = plan.n_tokens
    x, w, h = randn(1, 1, N, 128), randn(2, 128, 128), randn(3, 1, 2, N, 64)
    t = vsa.vsa_permute(plan, h)
    f = torch.zeros(1, 2, plan.n_tiles, 64, device="cuda")
    rows = torch.zeros(1, 2, plan.n_padded, device="cuda")
    kept = torch.zeros(1, 2, plan.n_video_tiles, 1, dtype=torch.int32, device="cuda")
    for ws in (torch.zeros(1 << 22, dtype=torch.uint8), torch.zeros(1 << 22, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        for call in (lambda: vsa.vsa_linear(plan, x, w, ws=ws), lambda: vsa.vsa_linear_backward(plan, x, x, w, ws=ws),
                     lambda: vsa.vsa_norm_rope_backward(plan, [vsa.HeadGrad(h, h, rotate=False)], ws=ws),
                     lambda: vsa.vsa_coarse_topk(plan, t, t, t, 1, ws=ws),
                     lambda: vsa.vsa_coarse_topk_pooled(plan, 1, 2, 64, 1, ws, o_coarse=f, topk_idx=kept),
                     lambda: vsa.vsa_select_reference(plan, 1, 2, 64, 1, ws, out=kept),
                     lambda: vsa.vsa_coarse_backward(plan, f, f, f, f, ws),
                     lambda: vsa.vsa_sparse_attn_backward(plan, t, t, t, t, kept, 1, rows, rows, ws)):
            with pytest.raises(ValueError):
                call()
    vsa.vsa_sync_status(plan)


@linears
def test_linear_backward_dx_add(c):
    """dx_add is added before the one rounding; it may be dx itself; not with x_pre."""
    B, N, xh, C, yh, Ow = c
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    x, w, dy = rows_or_heads(1, B, N, xh, C), randn(2, Ow, C, scale=0.1), rows_or_heads(5, B, N, yh, Ow)
    add = rows_or_heads(6, B, N, xh, C)
    dx, _, _ = vsa.vsa_linear_backward(plan, dy, x, w, dx_add=add, need=(True, False, False))
    want = BO.linear_backward(dy, x, w)[0] + BO.rows(add)
    slack = dot_slack(BO.rows(dy), f64(w).T) + 2.0 ** -23 * np.abs(want)
    close(dx, BO.heads(want, xh), BO.heads(slack, xh), "dx")
    same = add.clone()
    vsa.vsa_linear_backward(plan, dy, x, w, dx=same, dx_add=same, need=(True, False, False))
    assert torch.equal(same, dx)
    with pytest.raises(vsa.VsaError) as e:
        vsa.vsa_linear_backward(plan, dy, x, w, x_pre=x, x_act="silu", dx_add=add)
    assert e.value.status == 1
    vsa.vsa_sync_status(plan)


def test_permute_pool_without_means():
    plan = vsa.Plan((9, 3), (2, 5, 4), (4, 4, 4))
    q, g = randn(1, 2, 3, plan.n_tokens, 64), randn(2, 2, 3, plan.n_tokens, 64)
    (q_t, qbar), (g_t, none) = vsa.vsa_norm_rope_permute_pool(
        plan, [vsa.HeadTensor(q, rotate=False), vsa.HeadTensor(g, norm=False, rotate=False, pooled=False)])
    assert none is None and torch.equal(g_t, vsa.vsa_permute(plan, g))
    assert torch.equal(qbar, vsa.vsa_norm_rope_permute_pool(plan, [vsa.HeadTensor(q, rotate=False)])[0][1])
    vsa.vsa_sync_status(plan)


@pytest.mark.parametrize("c", [(33920, 64, 128), (33920, 2048, 2304), (104704, 264, 72)], ids=lambda c: "x".join(map(str, c)))
def test_weight_gradient_over_many_rows(c):
    """dw against what its sum may lose, and not against the sum of magnitudes, which over many rows of random
    sign is far larger than dw.  A step takes 16 rows: their products and the sum so far are aligned to the
    largest of them and cut to 24 bits or more (17 terms, each less than 2^-23 of the largest), and the result
    is cut to 24 bits.  In whatever pieces the rows are summed, a sum of neighbouring rows is no larger than the
    range R of the running sum; joining up to 16 pieces is 16 more such roundings of R.  So (K/16 + 16) steps of
    18 * 2^-23 of R, or of the largest product."""
    M, C, Ow = c
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    x, dy, w = randn(1, 1, M, C), randn(2, 1, M, Ow), randn(3, Ow, C, scale=0.1)
    _, dw, _ = vsa.vsa_linear_backward(plan, dy, x, w, need=(False, True, False))
    vsa.vsa_sync_status(plan)
    o, i = [0, Ow // 2, Ow - 1], [0, 7, C // 2, C - 1]
    terms = f64(dy[0][:, o])[:, :, None] * f64(x[0][:, i])[:, None, :]
    run = np.concatenate([np.zeros((1, len(o), len(i))), np.cumsum(terms, 0)])
    big = np.maximum(run.max(0) - run.min(0), np.abs(terms).max(0))
    close(dw[o][:, i], run[-1], (M / 16 + 17) * 18 * 2.0 ** -23 * big, "dw")


def test_offsets_past_32_bits_norm_rope():
    """2.25 G elements a tensor, token strides of 21,504: sampled rows at both ends."""
    plan = vsa.Plan((256,), (32, 48, 68), (4, 8, 4))
    rope = vsa.Rope(plan, (44, 42, 42))
    N, H, D = plan.n_tokens, 168, 128
    x = torch.empty(1, N, H, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    for i in range(0, N, 16384):
        x[:, i:i + 16384] = torch.randn(1, min(16384, N - i), H, D, generator=g, device="cuda")
    assert x.numel() > 2 ** 31
    x = x.transpose(1, 2)
    tok = np.r_[0:3, 255:258, N // 2, N - 3:N]
    ang = BO.angles(BO.positions((256,), (32, 48, 68)), (44, 42, 42))[tok]
    heads = [0, 85, 167]
    at = lambda t: t[:, heads][:, :, tok]
    z = BO.head_norm(at(x), None, EPS)
    want = BO.rotate(z, ang, False)
    slack = rot_slack(z) + (D / 2 + 8) * 2.0 ** -24 * np.abs(z).max(-1, keepdims=True)
    y, = vsa.vsa_norm_rope(plan, [vsa.HeadTensor(x)], rope, EPS)
    close(at(y), want, slack, "natural")
    del y
    (y_t, _), = vsa.vsa_norm_rope_permute_pool(plan, [vsa.HeadTensor(x)], rope, EPS)
    rows = plan.tables()["untile"][tok]
    close(y_t[:, heads][:, :, rows], want, slack, "tiles")
    # back through it: the gradient of the tiles is the tiles themselves
    (dx, _), = vsa.vsa_norm_rope_backward(plan, [vsa.HeadGrad(y_t, x)], rope, EPS, tiled=True)
    gr = BO.rotate(y_t[:, heads][:, :, rows], ang, False, inverse=True)
    want, _ = BO.head_norm_backward(gr, at(x), None, EPS)
    r = 1 / np.sqrt((f64(at(x)) ** 2).mean(-1, keepdims=True) + EPS)
    big = np.abs(gr).max(-1, keepdims=True)
    u = np.abs(f64(at(x)) * r).max(-1, keepdims=True)
    close(at(dx), want, (2 * D + 32) * 2.0 ** -24 * r * (big + u * u * big), "dx")
    vsa.vsa_sync_status(plan)


def test_offsets_past_32_bits_linear():
    """An output, and a gradient of it, of 2.37 G elements: sampled rows and columns at both ends."""
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    M, C, Ow = 330001, 64, 7168
    x, w, b = randn(1, 1, M, C), randn(2, Ow, C, scale=0.1), randn(3, Ow)
    y = vsa.vsa_linear(plan, x, w, b)
    assert y.numel() > 2 ** 31
    rows = np.r_[0:3, M // 2, M - 3:M]
    p = BO.linear(x[:, rows], w, b)
    close(y[:, rows], p, dot_slack(f64(x[:, rows]), f64(w)) + 2.0 ** -23 * np.abs(p), "y")
    dx, dw, db = vsa.vsa_linear_backward(plan, y, x, w)
    vsa.vsa_sync_status(plan)
    gr = f64(y[:, rows])
    close(dx[:, rows], gr @ f64(w), dot_slack(gr, f64(w).T), "dx")
    cols = [0, 3584, Ow - 1]
    gc, xr = f64(y[0][:, cols]), f64(x[0])
    close(dw[cols], gc.T @ xr, dot_slack(gc.T, xr.T), "dw")
    # fp32 sums in a chain of 88 rows, 8 warps, 15 runs and 32 rows of runs
    close(db[cols], gc.sum(0), 160 * 2.0 ** -24 * np.abs(gc).sum(0), "db", half_step=0.0)
