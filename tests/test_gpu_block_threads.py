"""Calls from host threads.  Two at once, each with its own plan, stream, buffers and sizes: what one
call asks of a kernel (its shared memory among it) stays its own; these threads are C's, and do
nothing between their calls.  And a thread whose first work with the GPU is the call itself."""
import ctypes
import os
import subprocess
import threading

import pytest
import torch

from tests.test_gpu_block import randn
from tile_sparse_video_b200 import vsa

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

THREADS = r'''
#include <pthread.h>
#include <string.h>
#include "vsa_block.h"
typedef struct {
  vsa_plan plan; vsa_rope rope; const vsa_head_tensor* item; int H, D, rounds; void* stream;
  const void *q, *k, *v; const int32_t* topk; void* out;
  const void* d_out; const float *lse, *delta; void *dq, *dk, *dv, *ws; size_t ws_bytes; int n_ref;
  int bad; pthread_barrier_t* gate; char said[120];
} job;
static void count(job* j, vsa_status st) {
  if (st != VSA_OK && !j->bad++) strncpy(j->said, vsa_last_error(), sizeof j->said - 1);
}
static void* tiles(void* p) {
  job* j = p;
  pthread_barrier_wait(j->gate);
  for (int i = 0; i < j->rounds; ++i)
    count(j, vsa_norm_rope_permute_pool(j->plan, j->rope, j->item, 1, 1e-6f, 1, j->H, j->D, j->stream));
  return 0;
}
static void* attention(void* p) {
  job* j = p;
  pthread_barrier_wait(j->gate);
  for (int i = 0; i < j->rounds; ++i)
    count(j, vsa_sparse_attn(j->plan, j->q, j->k, j->v, j->topk, 1, j->H, j->D, 1, 0.1f, j->out, 0, 0, 0,
                             j->stream));
  return 0;
}
static void* backward(void* p) {
  job* j = p;
  pthread_barrier_wait(j->gate);
  for (int i = 0; i < j->rounds; ++i)
    count(j, vsa_sparse_attn_backward(j->plan, j->q, j->k, j->v, j->d_out, j->topk, 1, 0, j->n_ref, j->lse, j->delta,
                                      0, 0, 0, 1, j->H, j->D, 0.1f, j->dq, j->dk, j->dv, j->ws, j->ws_bytes,
                                      j->stream));
  return 0;
}
int run(job* jobs, int n, int what) {
  pthread_t t[8];
  pthread_barrier_t gate;
  pthread_barrier_init(&gate, 0, n);
  for (int i = 0; i < n; ++i) {
    jobs[i].gate = &gate;
    if (pthread_create(&t[i], 0, what == 2 ? backward : what == 1 ? attention : tiles, &jobs[i])) return -1;
  }
  for (int i = 0; i < n; ++i) pthread_join(t[i], 0);
  return 0;
}
'''
P = ctypes.c_void_p


class Job(ctypes.Structure):
    _fields_ = [("plan", P), ("rope", P), ("item", P), ("H", ctypes.c_int), ("D", ctypes.c_int),
                ("rounds", ctypes.c_int), ("stream", P), ("q", P), ("k", P), ("v", P), ("topk", P), ("out", P),
                ("d_out", P), ("lse", P), ("delta", P), ("dq", P), ("dk", P), ("dv", P), ("ws", P),
                ("ws_bytes", ctypes.c_size_t), ("n_ref", ctypes.c_int), ("bad", ctypes.c_int), ("gate", P),
                ("said", ctypes.c_char * 120)]


@pytest.fixture(scope="module")
def threads(libvsa, tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    d = tmp_path_factory.mktemp("threads")
    (d / "threads.c").write_text(THREADS)
    where = os.path.join(ROOT, "tile_sparse_video_b200")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"), str(d / "threads.c"),
                    "-o", str(d / "threads.so"), "-L", where, "-l:libvsa.so", "-Wl,-rpath," + where, "-lpthread"],
                   check=True)
    run = ctypes.CDLL(str(d / "threads.so")).run
    run.argtypes, run.restype = [P, ctypes.c_int, ctypes.c_int], ctypes.c_int

    def refused(jobs, what):
        """(calls that were refused, what the first of them said) of each thread."""
        jobs = (Job * len(jobs))(*jobs)
        assert run(jobs, len(jobs), what) == 0
        return [(j.bad, j.said) for j in jobs]
    yield refused
    torch.cuda.synchronize()


@pytest.mark.parametrize("D,heads", [(64, (440, 600)), (128, (80, 300))])
def test_norm_rope_permute_pool(threads, D, heads):
    """Items of other numbers of heads, so other sizes of shared memory for one kernel, each of them
    above what a kernel may take without leave."""
    jobs, checks, keep = [], [], []
    for i, H in enumerate(heads):
        plan = vsa.Plan((9, 70), (4, 8, 8), (4, 4, 4))
        rope, stream = vsa.Rope(plan, (24, 20, 20)), torch.cuda.Stream()
        x = randn(i, 1, H, plan.n_tokens, D)
        (want, means), = vsa.vsa_norm_rope_permute_pool(plan, [vsa.HeadTensor(x)], rope)
        y, m = torch.empty_like(want), torch.empty_like(means)
        item = ctypes.create_string_buffer(vsa._HEAD_TENSOR.pack(
            *vsa._view(plan, x, "x", x.shape), 0, 0, 1, 1, y.data_ptr(), 0, 0, 0, m.data_ptr()))
        jobs.append(Job(plan.handle, rope.handle, ctypes.addressof(item), H, D, 20000, stream.cuda_stream))
        checks.append((plan, y, want, m, means))
        keep.append((rope, stream, x, item))
    torch.cuda.synchronize()
    assert threads(jobs, 0) == [(0, b"")] * 2
    torch.cuda.synchronize()
    for plan, y, want, m, means in checks:
        vsa.vsa_sync_status(plan)
        assert torch.equal(y, want) and torch.equal(m, means)


@pytest.mark.parametrize("tile", [(4, 4, 4), (4, 8, 4)], ids=["r64", "r128"])
@pytest.mark.parametrize("what", [1, 2], ids=["forward", "backward"])
def test_attention(threads, tile, what):
    """The attention kernels' lists grow with the tiles: plans of few and of many."""
    jobs, checks, keep = [], [], []
    for i, prefix in enumerate(((70,), (70,) * 60)):
        plan, stream = vsa.Plan(prefix, (4, 8, 8), tile), torch.cuda.Stream()
        q, k, v, g = (randn(10 * i + s, 1, 1, plan.n_padded, 128) for s in range(4))
        topk = torch.full((1, 1, plan.n_video_tiles, 1), plan.n_prefix_tiles, dtype=torch.int32, device="cuda")
        out, lse = vsa.vsa_sparse_attn(plan, q, k, v, topk, 1, 0.1, want_lse=True)
        job = Job(plan.handle, None, None, 1, 128, 20000 if what == 1 else 4000, stream.cuda_stream, q.data_ptr(),
                  k.data_ptr(), v.data_ptr(), topk.data_ptr())
        if what == 1:
            want, got = [out], [torch.empty_like(out)]
            job.out = got[0].data_ptr()
            extra = ()
        else:
            ws = torch.empty(vsa.vsa_backward_workspace_size(plan, 1, 1, 128), dtype=torch.uint8, device="cuda")
            delta = (out.float() * g.float()).sum(-1)
            want = vsa.vsa_sparse_attn_backward(plan, q, k, v, g, topk, 1, lse, delta, ws, scale=0.1)
            got = [torch.empty_like(t) for t in want]
            job.d_out, job.lse, job.delta = g.data_ptr(), lse.data_ptr(), delta.data_ptr()
            job.dq, job.dk, job.dv = (t.data_ptr() for t in got)
            job.ws, job.ws_bytes, job.n_ref = ws.data_ptr(), ws.numel(), plan.n_prefix_tiles
            extra = (ws, delta, lse, g)
        vsa.vsa_sync_status(plan)
        jobs.append(job)
        checks.append((plan, got, want))
        keep.append((stream, q, k, v, topk, extra))
    torch.cuda.synchronize()
    assert threads(jobs, what) == [(0, b"")] * 2
    torch.cuda.synchronize()
    for plan, got, want in checks:
        vsa.vsa_sync_status(plan)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_first_call_of_a_thread(threads):
    """Products of every kind from threads that have not yet touched the GPU."""
    plan = vsa.Plan((9, 70), (4, 8, 8), (4, 4, 4))
    n, C, H, D, k = plan.n_tokens, 256, 2, 128, 1
    s = torch.cuda.Stream()
    x, w = randn(1, 1, n, C), randn(2, H * D, C, scale=0.05)
    heads = [randn(3 + i, 1, H, n, D) for i in range(4)]
    layer = vsa.TrainingLayer(plan, 1, H, D, k)
    rows, by_head = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for shape in ((1, n, H * D), (1, H, n, D)))
    ws = torch.empty(max(vsa._workspace_bytes(plan, "vsa_linear_workspace_size", 1, n, C, H * D), 16),
                     dtype=torch.uint8, device="cuda")
    grads = (torch.empty_like(x), torch.empty_like(w), torch.empty(H * D, device="cuda"))
    bws = vsa.linear_backward_workspace(plan, 1, n, C, H * D)
    calls = {
        "linear": lambda st: [vsa.vsa_linear(plan, x, w, y=rows, ws=ws, stream=st)],
        "linear backward": lambda st: list(vsa.vsa_linear_backward(
            plan, heads[0], x, w, dx=grads[0], dw=grads[1], db=grads[2], ws=bws, stream=st)),
        "project": lambda st: [vsa.vsa_project(plan, x, w, H, D, y=by_head, stream=st)],
        "layer": lambda st: [layer.forward(*heads, stream=st)],
        "layer backward": lambda st: list(layer.backward(heads[0], stream=st)),
    }
    for name, call in calls.items():
        torch.cuda.synchronize()
        res = call(s)
        s.synchronize()
        want = [t.clone() for t in res]
        got, errors = [], []

        def work():
            try:
                got.extend(call(s))
            except Exception as e:
                errors.append(e)
        t = threading.Thread(target=work)
        torch.cuda.synchronize()
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not errors, (name, errors)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    vsa.vsa_sync_status(plan)
