"""The operators around the layer in use: the attention half of a transformer block, forward
and backward, each stage against its fp64 oracle on the GPU's own bf16 inputs of that stage,
and the whole block's gradient against differences of the fp64 forward; then the ways a
program runs them (other streams, graphs, two at once)."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import block_oracle as BO
from tests.parity import assert_close, f64
from tests.test_gpu_block import close, dot_slack, randn
from tests.test_gpu_backward import assert_rel
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


class Case:
    def __init__(self, prefix, grid, tile, B, H, D, C, dims, halves, keep, seed):
        self.B, self.H, self.D, self.C, self.keep = B, H, D, C, keep
        self.plan = vsa.Plan(prefix, grid, tile)
        self.p = O.plan(prefix, grid, tile)
        self.N = self.plan.n_tokens
        self.rope = vsa.Rope(self.plan, dims, halves=halves)
        self.ang, self.halves = BO.angles(BO.positions(prefix, grid), dims), halves
        self.x = randn(seed, B, self.N, C)
        self.w_in = randn(seed + 1, 4 * H * D, C, scale=C ** -0.5)
        self.w_out = randn(seed + 2, C, H * D, scale=(H * D) ** -0.5)
        self.b_in, self.b_out = randn(seed + 3, 4 * H * D, scale=0.1), randn(seed + 4, C, scale=0.1).float()
        self.gq, self.gk = 1 + 0.2 * randn(seed + 5, D).float(), (1 + 0.2 * randn(seed + 6, D)).bfloat16()
        self.qk = vsa.QKNormRope(self.rope, self.gq, self.gk, EPS)

    def block(self, training):
        return vsa.AttentionBlock(self.plan, self.B, self.H, self.D, self.C, self.keep, self.qk, training=training)

    def run(self, block):
        out = block.forward(self.x, self.w_in, self.w_out, self.b_in, self.b_out)
        vsa.vsa_sync_status(self.plan)
        return out

    def turned(self, q, gain):
        return BO.rotate(BO.head_norm(q, gain, EPS), self.ang, self.halves)

    def forward64(self, x, kept):
        """The whole block in fp64 under a given selection."""
        y = BO.heads(BO.linear(x, self.w_in, self.b_in), 4 * self.H)
        q, k, v, g = np.split(y, 4, axis=1)
        f = O.layer(self.turned(q, self.gq), self.turned(k, self.gk), v, g, self.p, self.keep, kept=kept)
        return BO.linear(f["out"], self.w_out, self.b_out) + x


ARGS = [
    ((40, 70), (4, 8, 8), (4, 4, 4), 1, 2, 64, 96, (24, 20, 20), False, 2, 100),
    ((5, 0, 64, 65), (5, 6, 7), (4, 4, 4), 2, 2, 128, 200, (44, 42, 42), True, 3, 200),
    ((130,), (8, 9, 9), (4, 8, 4), 1, 3, 128, 136, (44, 42, 42), False, 2, 300),
]
cases = pytest.mark.parametrize("args", ARGS, ids=["d64", "ragged_b2", "r128"])


@cases
def test_block_forward(args):
    c = Case(*args)
    H = c.H
    train, infer = c.block(True), c.block(False)
    out, out_i = c.run(train), c.run(infer)
    # the products' heads: one rounding and the fp32 sum
    want = BO.linear(c.x, c.w_in, c.b_in)
    slack = dot_slack(f64(c.x), f64(c.w_in)) + 2.0 ** -23 * np.abs(want)
    close(train.qkvg, BO.heads(want, 4 * H), BO.heads(slack, 4 * H), "qkvg")
    assert torch.equal(infer.qkv, train.qkvg[:, :3 * H]) and torch.equal(infer.g, train.qkvg[:, 3 * H:])
    q, k, v, g = train.qkvg.split(H, 1)
    lay = train.layer
    for got, src, gain in ((lay.q_t, q, c.gq), (lay.k_t, k, c.gk)):
        z = BO.head_norm(src, gain, EPS)
        big = np.abs(z).max(-1, keepdims=True)
        close(vsa.vsa_unpermute(c.plan, got), c.turned(src, gain), (c.D / 2 + 24) * 2.0 ** -24 * big, "q_t, k_t")
    assert torch.equal(lay.v_t, vsa.vsa_permute(c.plan, v.contiguous()))
    assert torch.equal(lay.g_t, vsa.vsa_permute(c.plan, g.contiguous()))
    for b, name in ((train, "training"), (infer, "fused")):
        lay = b.layer
        kept = lay.topk_idx.cpu().numpy().astype(np.int64)
        qn, kn = (vsa.vsa_unpermute(c.plan, t) for t in (lay.q_t, lay.k_t))
        ref = O.layer(qn, kn, v, g, c.p, c.keep, kept=kept)
        assert_close(f64(lay.out), ref["out"], what=name)
        want = BO.linear(lay.out, c.w_out, c.b_out) + f64(c.x)
        close(b.out, want, dot_slack(BO.rows(lay.out), f64(c.w_out)) + 2.0 ** -22 * np.abs(want), name)
    assert out.data_ptr() == train.out.data_ptr() and out_i.shape == c.x.shape


@cases
def test_block_backward(args):
    c = Case(*args)
    H = c.H
    block = c.block(True)
    c.run(block)
    d_out = randn(args[-1] + 9, *c.x.shape)
    dx, dw_in, db_in, dw_out, db_out, dgq, dgk = block.backward(d_out)
    vsa.vsa_sync_status(c.plan)
    lay = block.layer
    M = c.B * c.N
    # the output product
    wd, ww, wb = BO.linear_backward(d_out, lay.out, c.w_out)
    g, o = f64(d_out).reshape(M, -1), BO.rows(lay.out).reshape(M, -1)
    close(block.d_o, BO.heads(wd, H), BO.heads(dot_slack(f64(d_out), f64(c.w_out).T), H), "d_o")
    close(dw_out, ww, dot_slack(g.T, o.T), "dw_out")
    close(db_out, wb, M * 2.0 ** -24 * np.abs(g).sum(0) + 1e-30, "db_out", half_step=0.0)
    # the layer, and the norm and rotation under it: the layer's own bounds (2e-2 of the largest, 4e-3
    # of the mean), with the norm's projection of the gradient and one more rounding on top
    kept = lay.topk_idx.cpu().numpy().astype(np.int64)
    q, k, v, gt = block.qkvg.split(H, 1)
    qn, kn = (vsa.vsa_unpermute(c.plan, t) for t in (lay.q_t, lay.k_t))
    fwd = O.layer(qn, kn, v, gt, c.p, c.keep, kept=kept)
    bwd = O.layer_backward(block.d_o, fwd, c.p)
    got = block.d_qkvg.split(H, 1)
    for i, (src, gain, name, dg) in enumerate(((q, c.gq, "dq", dgq), (k, c.gk, "dk", dgk))):
        want, want_g = BO.head_norm_backward(BO.rotate(bwd[name], c.ang, c.halves, inverse=True), src, gain, EPS)
        assert_rel(f64(got[i]), want, 3e-2, 8e-3, what=name)
        assert_rel(f64(dg), want_g, 3e-2, 2e-2, what=name + " gain")
    assert_rel(f64(got[2]), bwd["dv"], what="dv")
    assert_rel(f64(got[3]), bwd["dg"], what="dg")
    # the input product, with the residual's gradient added
    wd, ww, wb = BO.linear_backward(block.d_qkvg, c.x, c.w_in)
    g = BO.rows(block.d_qkvg)
    wd = wd + f64(d_out)
    close(dx, wd, dot_slack(g, f64(c.w_in).T) + 2.0 ** -23 * np.abs(wd), "dx")
    close(dw_in, ww, dot_slack(g.reshape(M, -1).T, f64(c.x).reshape(M, -1).T), "dw_in")
    close(db_in, wb, M * 2.0 ** -24 * np.abs(g).sum((0, 1)) + 1e-30, "db_in", half_step=0.0)


def test_block_gradient_against_differences():
    """<dx, d> of the whole block against central differences of the fp64 forward along d (the
    selection held).  Some dozen roundings of 2^-9 stand between them: within 5 % of |dx| for a
    normal d, whose product with dx is of the size |dx| itself."""
    c = Case(*ARGS[0])
    block = c.block(True)
    c.run(block)
    kept = block.layer.topk_idx.cpu().numpy().astype(np.int64)
    d_out = randn(109, *c.x.shape)
    dx = f64(block.backward(d_out)[0])
    rng = np.random.default_rng(1)
    x, w = f64(c.x), f64(d_out)
    for _ in range(3):
        d = rng.normal(size=x.shape)
        h = 1e-4
        diff = (w * (c.forward64(x + h * d, kept) - c.forward64(x - h * d, kept))).sum() / (2 * h)
        assert abs(diff - (dx * d).sum()) <= 0.05 * np.sqrt((dx * dx).sum())


def test_layer_with_norm_and_rotation_is_the_composition():
    """Layer(qk=...) feeds the same tiles to the attention as vsa_norm_rope before a plain layer."""
    c = Case(*ARGS[1])
    q, k, v, g = (randn(s, c.B, c.H, c.N, c.D) for s in (1, 2, 3, 4))
    keep = c.plan.n_video_tiles                                  # no selection to differ in
    a = vsa.Layer(c.plan, c.B, c.H, c.D, keep, qk=c.qk)
    b = vsa.Layer(c.plan, c.B, c.H, c.D, keep)
    u = vsa.Layer(c.plan, c.B, c.H, c.D, keep, qk=c.qk, fused=False)
    qn, kn = vsa.vsa_norm_rope(c.plan, [vsa.HeadTensor(q, c.gq), vsa.HeadTensor(k, c.gk)], c.rope, EPS)
    out_a, out_b, out_u = a(q, k, v, g), b(qn, kn, v, g), u(q, k, v, g)
    vsa.vsa_sync_status(c.plan)
    for name in ("q_t", "k_t", "v_t"):
        assert torch.equal(getattr(a, name), getattr(b, name))
        assert torch.equal(getattr(u, name), getattr(b, name))
    ref = O.layer(qn, kn, v, g, c.p, keep)
    for out in (out_a, out_b, out_u):
        assert_close(f64(out), ref["out"], what="layer")


def test_streams_and_graphs():
    """On another stream, captured and replayed on new inputs, and two linears at once on two streams
    with a plan between them: the results of the plain calls, to the bit."""
    c = Case(*ARGS[0])
    block = c.block(False)
    want = c.run(block).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = block.forward(c.x, c.w_in, c.w_out, c.b_in, c.b_out, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    train = c.block(True)
    c.run(train)
    d_out = randn(7, *c.x.shape)
    grads = [t.clone() for t in train.backward(d_out)]
    x2 = c.x.clone()
    for step in (lambda: train.forward(x2, c.w_in, c.w_out, c.b_in, c.b_out), lambda: train.backward(d_out)):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train.forward(x2, c.w_in, c.w_out, c.b_in, c.b_out)
        outs = train.backward(d_out)
    x2.copy_(randn(8, *c.x.shape))
    graph.replay()
    x2.copy_(c.x)
    graph.replay()
    torch.cuda.synchronize()
    vsa.vsa_sync_status(c.plan)
    assert all(torch.equal(a, b) for a, b in zip(outs, grads))
    # two at once
    xs = [randn(20 + i, 1, 3000, 512) for i in range(2)]
    w, b = randn(30, 1024, 512, scale=0.05), randn(31, 1024)
    wants = [vsa.vsa_linear(c.plan, x, w, b, act="silu") for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    ys = []
    for _ in range(5):
        ys = [vsa.vsa_linear(c.plan, x, w, b, act="silu", stream=st) for x, st in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, t) for y, t in zip(ys, wants))
    vsa.vsa_sync_status(c.plan)


@pytest.mark.parametrize("copied", [True, False])
def test_linears_in_a_row(copied):
    """Linears that start under the end of the one before, each reading what the last one wrote:
    on a stream, behind a copy, a memset or an event alone, and captured on two streams that fork and join."""
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    x0 = randn(1, 1, 700, 512)
    ws = [randn(2 + i, 512, 512, scale=0.05) for i in range(4)]
    bufs = [torch.empty_like(x0) for _ in range(5)]
    side = torch.cuda.Stream()

    def chain(x, out, scratch, stream=None):
        """Two buffers in turn, so a linear writes what the one before the last read."""
        for i, w in enumerate(ws):
            y = out if i + 1 == len(ws) else scratch[i & 1]
            x = vsa.vsa_linear(plan, x, w, act="silu", residual=x if i & 1 else None, y=y, stream=stream)
        return x

    def everything():
        bufs[0].zero_()
        chain(x0, bufs[0], bufs[1:3])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            if copied:
                bufs[3].copy_(bufs[0])
            chain(bufs[3] if copied else bufs[0], bufs[4], [torch.empty_like(x0) for _ in range(2)])
        chain(bufs[0], bufs[1], [bufs[2], torch.empty_like(x0)])
        torch.cuda.current_stream().wait_stream(side)
        return vsa.vsa_linear(plan, bufs[4], ws[0], residual=bufs[1])

    # each linear alone, with a wait after it
    def alone(x):
        for i, w in enumerate(ws):
            y = vsa.vsa_linear(plan, x, w, act="silu", residual=x if i & 1 else None)
            torch.cuda.synchronize()
            x = y
        return x

    once = alone(x0)
    twice = alone(once)
    want = vsa.vsa_linear(plan, twice, ws[0], residual=twice)
    torch.cuda.synchronize()
    for _ in range(3):
        got = everything()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything()
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    vsa.vsa_sync_status(plan)


def test_destroyed_during_a_capture():
    """A plan, a rope and a runner that go while a graph is captured (as a garbage collector may have it)."""
    plan, gone = (vsa.Plan((4,), (2, 4, 4), (4, 4, 4)) for _ in range(2))
    rope, gone_rope = vsa.Rope(plan, (16, 24, 24)), vsa.Rope(gone, (16, 24, 24))
    pipe = vsa.LayerPipeline(plan, 1, 1, 64, 1)
    x = randn(1, 1, 2, plan.n_tokens, 64)
    want = vsa.vsa_rope_apply(plan, rope, x)
    got = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gone_rope.close()
        pipe.close()
        vsa.vsa_rope_apply(plan, rope, x, got)
        gone.close()
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_tables_are_there_when_a_handle_is_returned():
    """A plan and a rope made while the default stream has work, and used at once on another stream:
    their tables neither come late nor wait for that work."""
    args = (9, 70), (4, 24, 24), (4, 4, 4)
    plan = vsa.Plan(*args)
    rope = vsa.Rope(plan, (24, 20, 20))
    xs = randn(1, 1, 2, plan.n_tokens, 64)
    want, = vsa.vsa_norm_rope(plan, [vsa.HeadTensor(xs)], rope)
    (tiles, means), = vsa.vsa_norm_rope_permute_pool(plan, [vsa.HeadTensor(xs)], rope)
    s = torch.cuda.Stream()
    y, t, m = torch.empty_like(want), torch.empty_like(tiles), torch.empty_like(means)
    torch.cuda.synchronize()
    keep = []                                                    # a handle's end waits for the GPU
    for _ in range(5):
        torch.cuda._sleep(200_000_000)                           # some 0.1 s
        new = vsa.Plan(*args)
        turn = vsa.Rope(new, (24, 20, 20))
        keep += [new, turn]
        vsa.vsa_norm_rope(new, [vsa.HeadTensor(xs, y=y)], turn, stream=s)
        vsa.vsa_norm_rope_permute_pool(new, [vsa.HeadTensor(xs, y=t, pooled=m)], turn, stream=s)
        s.synchronize()
        assert not torch.cuda.default_stream().query()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(t, tiles) and torch.equal(m, means)
        y.zero_(), t.zero_(), m.zero_()
        vsa.vsa_sync_status(new)


def test_a_failed_call_does_not_fail_the_next():
    """A call that CUDA refuses (a runner of some terabytes) leaves nothing behind for those after it."""
    plan = vsa.Plan((9, 70), (4, 24, 24), (4, 4, 4))
    rope = vsa.Rope(plan, (24, 20, 20))
    x, w = randn(1, 1, 2, plan.n_tokens, 64), randn(2, 128, 128)
    calls = [lambda: vsa.vsa_rope_apply(plan, rope, x), lambda: vsa.vsa_linear(plan, x, w),
             lambda: vsa.vsa_linear(plan, x[:, :, :3], w), lambda: vsa.vsa_permute(plan, x),
             lambda: vsa.vsa_act_backward(plan, x, x, "silu")]
    for call in calls:
        want = call()
        with pytest.raises(vsa.VsaError) as e:
            vsa.LayerPipeline(plan, 4096, 4096, 128, 1)
        assert e.value.status == 5, e.value
        assert torch.equal(call(), want)
    vsa.vsa_sync_status(plan)


def test_repeats_are_bitwise_equal():
    """Sums are taken in a fixed order: two runs give the same bits, the gains' and biases' gradients
    among them, and in split products."""
    c = Case(*ARGS[2])
    block = c.block(True)
    d_out = randn(9, *c.x.shape)
    runs = []
    for _ in range(2):
        c.run(block)
        runs.append([block.out.clone(), *(t.clone() for t in block.backward(d_out))])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    x, w = randn(1, 1, 40, 4096), randn(2, 256, 4096, scale=0.02)
    assert torch.equal(vsa.vsa_linear(c.plan, x, w), vsa.vsa_linear(c.plan, x, w))


def test_linear_abort_path():
    """The linear kernel's own failure path, without a fault: with the bound of its waits cut to 100 ns
    they run out, the kernel records VSA_ERR_DEVICE_TIMEOUT, drains its copies and products, frees
    its tensor memory and returns; with the bound restored the same context computes as before."""
    import time
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4))
    x, w = randn(1, 1, 3000, 1024), randn(2, 1024, 1024, scale=0.03)
    want = vsa.vsa_linear(plan, x, w)
    vsa.vsa_sync_status(plan)
    # a wait looks at the clock every sixteenth poll, and a poll may sleep for some time: sums of 4,096 K
    # blocks keep the epilogue waiting for over a millisecond
    long_x = torch.zeros(1, 3000, 1 << 18, dtype=torch.bfloat16, device="cuda")
    long_w = torch.zeros(1024, 1 << 18, dtype=torch.bfloat16, device="cuda")
    try:
        vsa.vsa_debug_set_wait_limit(100)
        timed_out = False
        for _ in range(5):                 # a wait that happened to finish in time: try again
            t0 = time.perf_counter()
            vsa.vsa_linear(plan, long_x, long_w)
            try:
                vsa.vsa_sync_status(plan)
            except vsa.VsaError as e:
                assert e.status == 6, e                  # VSA_ERR_DEVICE_TIMEOUT
                timed_out = True
            # a pair whose halves stopped at different copies drains for up to 2 s
            assert time.perf_counter() - t0 < 10.0
            if timed_out:
                break
        assert timed_out, "the kernel never gave up under a 100 ns bound"
    finally:
        vsa.vsa_debug_set_wait_limit(0)
    vsa.vsa_sync_status(plan)
    assert torch.equal(vsa.vsa_linear(plan, x, w), want)
    vsa.vsa_sync_status(plan)
