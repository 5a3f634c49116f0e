"""The operators around the layer on the host (no GPU needed): exported symbols, the
rotation's tables against the oracle, the refusals, and the oracle's gradients against
differences of its forward."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import block_oracle as BO
from tile_sparse_video_b200 import vsa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_exports_every_declared_symbol(libvsa):
    text = open(os.path.join(ROOT, "include", "vsa_block.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    decl = sorted(set(re.findall(r"^vsa_status (vsa_[a-z_]+)\s*\(", text, flags=re.M)))
    assert sorted(vsa.BLOCK_EXPORTS) == decl
    for name in decl:
        assert hasattr(libvsa, name), name


ROPES = [
    dict(prefix=(40, 70), grid=(4, 8, 8), dims=(24, 20, 20)),
    dict(prefix=(5, 0, 64), grid=(3, 5, 7), dims=(16, 24, 24), halves=True, step=0.5, offset=(3, -2, 0.25)),
    dict(prefix=(), grid=(1, 9, 6), dims=(0, 64, 64), theta=(1.0, 256.0, 1e4)),
    dict(prefix=(130,), grid=(0, 4, 4), dims=(44, 42, 42), pos=True),
    dict(prefix=(3,), grid=(2, 2, 2), dims=(2, 0, 0), pos=True),
    dict(prefix=(9,), grid=(2, 3, 2), dims=(32, 32, 32), halves=True, pos=True, freq=True),
]


@pytest.mark.parametrize("c", ROPES)
def test_rope_tables(libvsa, c):
    plan = vsa.Plan(c["prefix"], c["grid"], (4, 4, 4), device=-1)
    rng = np.random.default_rng(len(c["prefix"]))
    n_p, P = sum(c["prefix"]), sum(c["dims"]) // 2
    pos = rng.integers(-5000000, 5000000, (n_p, 3)) * 0.5 if c.get("pos") else None
    freq = rng.random(P) if c.get("freq") else None
    theta, off, step = c.get("theta", 1e4), c.get("offset", 0.0), c.get("step", 1.0)
    rope = vsa.Rope(plan, c["dims"], theta=theta, offset=off, step=step, halves=c.get("halves", False),
                    inv_freq=freq, prefix_pos=pos)
    assert rope.pairs == P
    three = lambda x: (x,) * 3 if np.isscalar(x) else x
    want = BO.angles(BO.positions(c["prefix"], c["grid"], three(off), three(step), pos), c["dims"],
                     three(theta), freq)
    cos, sin = rope.tables()
    # angles in double reach 2.5e6, where a step is 2^-31.  The two sides may differ by some
    # steps in pos * freq; the rounding to fp32 adds 2^-24 relative
    tol = 2.0 ** -24 + 8 * 2.0 ** -53 * np.abs(want)
    assert np.all(np.abs(cos - np.cos(want)) <= tol)
    assert np.all(np.abs(sin - np.sin(want)) <= tol)
    rope.close()
    plan.close()


@pytest.mark.parametrize("bad,status", [
    (dict(dims=(3, 4, 4)), 1), (dict(dims=(0, 0, 0)), 1), (dict(dims=(-2, 4, 4)), 1),
    (dict(dims=(64, 64, 2)), 1), (dict(dims=(6, 4, 4), halves=True), 2), (dict(theta=0.0), 1),
    (dict(theta=float("nan")), 1), (dict(step=float("inf")), 1), (dict(offset=float("nan")), 1),
    (dict(inv_freq=[float("inf")] * 32), 1), (dict(prefix_pos=np.full((6, 3), np.nan)), 1),
    (dict(prefix_pos=np.full((6, 3), 1e300), inv_freq=[1e300] * 32), 1)])
def test_rope_refusals(libvsa, bad, status):
    plan = vsa.Plan((6,), (2, 3, 4), (4, 4, 4), device=-1)
    args = dict(dims=(24, 20, 20))
    args.update(bad)
    with pytest.raises(vsa.VsaError) as e:
        vsa.Rope(plan, **args)
    assert e.value.status == status
    with pytest.raises(ValueError):
        vsa.Rope(plan, (24, 20, 20), prefix_pos=np.zeros((5, 3)))
    with pytest.raises(ValueError):
        vsa.Rope(plan, (24, 20, 20), inv_freq=[1.0] * 31)
    plan.close()


def test_host_only_plan_refuses_launches(libvsa):
    plan = vsa.Plan((40, 70), (4, 8, 8), (4, 4, 4), device=-1)
    rope = vsa.Rope(plan, (24, 20, 20))
    v = vsa._VIEW.pack(0x1000, 8, 8, 64)
    L = libvsa
    assert L.vsa_rope_apply(plan.handle, rope.handle, v, v, 0, 1, 1, 64, None) == 1
    assert b"host-only" in L.vsa_last_error()
    t = bytes(vsa._HEAD_TENSOR.size)
    assert L.vsa_norm_rope(plan.handle, rope.handle, t, 1, 1e-6, 1, 1, 64, None) == 1
    assert L.vsa_norm_rope_permute_pool(plan.handle, rope.handle, t, 1, 1e-6, 1, 1, 64, None) == 1
    g = bytes(vsa._HEAD_GRAD.size)
    assert L.vsa_norm_rope_backward(plan.handle, rope.handle, g, 1, 1e-6, 0, 1, 1, 64, None, 0, None) == 1
    assert L.vsa_linear(plan.handle, bytes(vsa._LINEAR.size), None, 0, None) == 1
    assert L.vsa_linear_backward(plan.handle, bytes(vsa._LINEAR_GRAD.size), None, 0, None) == 1
    assert L.vsa_act_backward(plan.handle, None, None, 0, None, 8, None) == 1
    assert b"host-only" in L.vsa_last_error()
    assert L.vsa_rope_apply(None, rope.handle, v, v, 0, 1, 1, 64, None) == 1
    assert L.vsa_rope_create(plan.handle, None, None) == 1
    assert L.vsa_rope_tables(None, None, None) == 1
    assert L.vsa_rope_destroy(None) == 0
    n = ctypes.c_size_t()
    assert L.vsa_norm_rope_backward_workspace_size(plan.handle, 5, 64, ctypes.byref(n)) == 1
    assert L.vsa_norm_rope_backward_workspace_size(plan.handle, 2, 96, ctypes.byref(n)) == 2
    assert L.vsa_norm_rope_backward_workspace_size(plan.handle, 2, 64, ctypes.byref(n)) == 0 and n.value > 0
    assert L.vsa_linear_backward_workspace_size(plan.handle, 1, -1, 64, 64, ctypes.byref(n)) == 1
    assert L.vsa_linear_backward_workspace_size(plan.handle, 1, 64, 60, 64, ctypes.byref(n)) == 1
    assert L.vsa_linear_backward_workspace_size(plan.handle, 1, 64, 64, 64, ctypes.byref(n)) == 0
    assert L.vsa_linear_workspace_size(plan.handle, 1, 64, 60, 64, ctypes.byref(n)) == 1
    # one token reads w without a split; 64 rows of 64 K blocks split over the pairs of SMs
    assert L.vsa_linear_workspace_size(plan.handle, 1, 1, 4096, 256, ctypes.byref(n)) == 0 and n.value == 0
    assert L.vsa_linear_workspace_size(plan.handle, 1, 64, 4096, 256, ctypes.byref(n)) == 0
    assert n.value > 0 and n.value % (64 * 256 * 4) == 0
    for B, N in ((0, 5), (2, 0), (0, 0)):                 # no rows, no workspace
        assert L.vsa_linear_workspace_size(plan.handle, B, N, 64, 64, ctypes.byref(n)) == 0 and n.value == 0
        assert L.vsa_linear_backward_workspace_size(plan.handle, B, N, 64, 64, ctypes.byref(n)) == 0
        assert n.value == 0
    # the handle does not refer to its plan
    plan.close()
    assert rope.tables()[0].shape == (366, 32)
    rope.close()


def test_workspaces_are_looked_at(libvsa):
    """A workspace that is no tensor, or has gaps, or is on another device than the plan, does not get as
    far as the library (which refuses the host-only plan itself)."""
    import torch
    plan = vsa.Plan((4,), (0, 4, 4), (4, 4, 4), device=-1)
    x, w, y = (torch.zeros(s, dtype=torch.bfloat16) for s in ((1, 4, 64), (64, 64), (1, 4, 64)))
    h, dw, db = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16), torch.zeros_like(w), torch.zeros(64)
    for call in (lambda ws: vsa.vsa_linear(plan, x, w, y=y, ws=ws),
                 lambda ws: vsa.vsa_linear_backward(plan, y, x, w, dx=x, dw=dw, db=db, ws=ws),
                 lambda ws: vsa.vsa_norm_rope_backward(plan, [vsa.HeadGrad(h, h, None, True, False, h)], ws=ws)):
        with pytest.raises(TypeError):
            call(b"0" * 4096)
        with pytest.raises(ValueError):
            call(torch.zeros(4096, 2, dtype=torch.uint8)[:, 0])
    fake = vsa.Plan((4,), (0, 4, 4), (4, 4, 4), device=-1)
    fake.device = 0                                        # as on a GPU: the workspace is not there
    for ws in (torch.zeros(4096, dtype=torch.uint8), torch.zeros(4096, 2)[:, 0]):
        with pytest.raises(ValueError):
            vsa._workspace(fake, ws)
    assert vsa._workspace(plan, torch.zeros(3, 5))[1] == 60 and vsa._workspace(plan, None) == (None, 0)
    plan.close(), fake.close()


def test_records_match_the_header(libvsa):
    """The packed records have the sizes and offsets a C compiler gives the header's structures."""
    import subprocess
    import tempfile
    code = '''#include <stddef.h>
#include <stdio.h>
#include "vsa_block.h"
int main() {
  printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(vsa_view), sizeof(vsa_head_tensor), sizeof(vsa_head_grad),
         sizeof(vsa_linear_args), sizeof(vsa_linear_grad_args), sizeof(vsa_rope_desc));
  printf("%zu %zu %zu %zu %zu\\n", offsetof(vsa_head_tensor, y), offsetof(vsa_head_grad, dx),
         offsetof(vsa_linear_args, bias_type), offsetof(vsa_linear_grad_args, x_act),
         offsetof(vsa_linear_grad_args, dx_add));
}'''
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "s.c"), os.path.join(d, "s")
        open(src, "w").write(code)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), src, "-o", exe], check=True)
        sizes, offsets = (list(map(int, ln.split())) for ln in
                          subprocess.run([exe], capture_output=True, text=True).stdout.splitlines())
    assert sizes == [vsa._VIEW.size, vsa._HEAD_TENSOR.size, vsa._HEAD_GRAD.size, vsa._LINEAR.size,
                     vsa._LINEAR_GRAD.size, ctypes.sizeof(vsa._RopeDesc)]
    S = lambda f: vsa.struct.calcsize("@" + f + "0P")
    assert offsets == [S("PqqqPiii"), S("PqqqPqqqPiii"), vsa.struct.calcsize("@iiiiiqPqqqPP"),
                       vsa.struct.calcsize("@iiiiiqPqqqPqqqPPqqq"), S("iiiiiqPqqqPqqqPPqqqiPqqqPP")]


def test_no_memory_is_an_error(libvsa):
    """A plan and a rope whose tables find no room: an error, and the process goes on."""
    import subprocess
    import sys
    code = """
import resource
from tile_sparse_video_b200 import vsa
small = vsa.Plan((1 << 24,), (0, 4, 4), (4, 4, 4), device=-1)
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (1 << 27), resource.RLIM_INFINITY))
for make in (lambda: vsa.Plan((1 << 29,), (0, 4, 4), (4, 4, 4), device=-1), lambda: vsa.Rope(small, (24, 20, 20))):
    try:
        make()
        print("made")
    except vsa.VsaError as e:
        print(e)
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
print(vsa.Plan((9,), (0, 4, 4), (4, 4, 4), device=-1).n_tokens)
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert run.stdout.splitlines() == ["VSA_ERR_INVALID_ARG: out of host memory"] * 2 + ["9"], run


def test_binding_defines_every_name_once():
    """A second definition would silently take the place of the first."""
    import ast
    body = ast.parse(open(vsa.__file__).read()).body
    names = [n.name for n in body if isinstance(n, (ast.FunctionDef, ast.ClassDef))]
    names += [t.id for n in body if isinstance(n, ast.Assign) for t in n.targets if isinstance(t, ast.Name)]
    assert sorted(set(names)) == sorted(names), sorted(n for n in set(names) if names.count(n) > 1)


def _diff(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("halves", [False, True])
def test_oracle_norm_rope_gradient(halves):
    """Along random directions the formulas' gradient agrees with central differences."""
    rng = np.random.default_rng(5)
    ang = BO.angles(BO.positions((3,), (2, 2, 3)), (24, 20, 20))
    x, gain, dy = rng.normal(size=(2, 3, 15, 64)), 1 + 0.2 * rng.normal(size=64), rng.normal(size=(2, 3, 15, 64))
    f = lambda x_, w_: (dy * BO.rotate(BO.head_norm(x_, w_, 1e-6), ang, halves)).sum()
    dx, dw = BO.head_norm_backward(BO.rotate(dy, ang, halves, inverse=True), x, gain, 1e-6)
    for _ in range(3):
        d = rng.normal(size=x.shape)
        assert np.isclose(_diff(lambda t: f(t, gain), x, d), (dx * d).sum(), rtol=1e-7)
        d = rng.normal(size=gain.shape)
        assert np.isclose(_diff(lambda t: f(x, t), gain, d), (dw * d).sum(), rtol=1e-7)


@pytest.mark.parametrize("name", sorted(vsa.ACTS))
def test_oracle_linear_gradient(name):
    rng = np.random.default_rng(6)
    xp, w, b, dy = (rng.normal(size=s) for s in ((2, 5, 16), (8, 16), (8,), (2, 5, 8)))
    f = lambda xp_, w_, b_: (dy * BO.linear(BO.act(name, xp_), w_, b_)).sum()
    dx, dw, db = BO.linear_backward(dy, BO.act(name, xp), w)
    dx = dx * BO.act_slope(name, xp)
    for i, (v, g) in enumerate(((xp, dx), (w, dw), (b, db))):
        d = rng.normal(size=v.shape)
        at = lambda t: f(*(t if j == i else a for j, a in enumerate((xp, w, b))))
        assert np.isclose(_diff(at, v, d), (g * d).sum(), rtol=1e-7)
