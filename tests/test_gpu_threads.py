"""Calls of different widths from several threads at once, each with its own stream, workspace and tensors.  The threads
are C threads: what two launches share on the host is held for less time than Python takes between calls."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16

# Each thread makes the same call n times on its stream; *bad: calls that failed.
SOURCE = r"""
#include <pthread.h>
#include <stddef.h>
#include "verifyhead.h"

typedef struct {
    int kind, rows, H, n, bad;
    void *a, *b, *c, *d, *e, *ws, *stream;
    size_t ws_bytes;
    vh_status (*grad)(const void*, const void*, const void*, const void*, int, int, int, int, int64_t, int64_t, int64_t, float,
                      float, void*, int64_t, float*, void*, size_t, void*);
    vh_status (*draft)(const void*, const void*, const int32_t*, int, int, int, int32_t*, float*, void*, size_t, void*);
    vh_status (*packed)(const void*, const void*, float, const int32_t*, int, int, int, int32_t*, float*, void*, size_t, void*);
    pthread_barrier_t* go;
} Job;

static void* work(void* p) {
    Job* j = p;
    pthread_barrier_wait(j->go);
    for (int i = 0; i < j->n; ++i) {
        vh_status st;
        if (j->kind == 0)  /* dy, h, w, dx, dw */
            st = j->grad(j->a, j->b, j->c, 0, VH_BF16, 0, j->rows, j->H, j->H, j->H, j->H, 1e-6f, 0.f, j->d, j->H, j->e, j->ws,
                         j->ws_bytes, j->stream);
        else if (j->kind == 1)  /* hidden, W, cand, ids, maxlogit */
            st = j->draft(j->a, j->b, j->c, j->rows, j->H, 64, j->d, j->e, j->ws, j->ws_bytes, j->stream);
        else
            st = j->packed(j->a, j->b, 1.f, j->c, j->rows, j->H, 64, j->d, j->e, j->ws, j->ws_bytes, j->stream);
        j->bad += st != VH_OK;
    }
    return 0;
}

void together(Job* jobs, int n) {
    pthread_t t[16];
    pthread_barrier_t go;
    pthread_barrier_init(&go, 0, n);
    for (int i = 0; i < n; ++i) jobs[i].go = &go, pthread_create(t + i, 0, work, jobs + i);
    for (int i = 0; i < n; ++i) pthread_join(t[i], 0);
    pthread_barrier_destroy(&go);
}
"""


class Job(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int) for k in ("kind", "rows", "H", "n", "bad")] + \
        [(k, ctypes.c_void_p) for k in ("a", "b", "c", "d", "e", "ws", "stream")] + [("ws_bytes", ctypes.c_size_t)] + \
        [(k, ctypes.c_void_p) for k in ("grad", "draft", "packed", "go")]


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


@pytest.fixture(scope="module")
def together(vh, tmp_path_factory):
    cc = shutil.which("gcc")
    if not cc:
        pytest.skip("no C compiler")
    at = tmp_path_factory.mktemp("threads")
    (at / "t.c").write_text(SOURCE)
    subprocess.run([cc, "-O1", "-shared", "-fPIC", "-pthread", "-I" + os.path.join(ROOT, "include"), str(at / "t.c"), "-o",
                    str(at / "t.so")], check=True)
    lib = ctypes.CDLL(str(at / "t.so"))
    L = vh.lib()
    entry = {k: ctypes.cast(getattr(L, f), ctypes.c_void_p).value for k, f in
             (("grad", "vh_add_rmsnorm_grad"), ("draft", "mtp_draft_head_argmax"),
              ("packed", "mtp_draft_head_argmax_nvfp4_packed"))}

    def run(kind, made, n=2000):
        """made: (rows, H, the call's five tensors, its workspace) per thread; the results are the last two tensors."""
        streams = [torch.cuda.Stream() for _ in made]
        jobs = (Job * len(made))()
        for j, (rows, H, t, ws), s in zip(jobs, made, streams):
            j.kind, j.rows, j.H, j.n = kind, rows, H, 1
            j.a, j.b, j.c, j.d, j.e = (x.data_ptr() for x in t)
            j.ws, j.ws_bytes, j.stream = ws.data_ptr(), ws.numel(), s.cuda_stream
            for k, p in entry.items():
                setattr(j, k, p)
        torch.cuda.synchronize()
        for i in range(len(made)):  # one after the other: what the calls give by themselves
            lib.together(ctypes.byref(jobs, i * ctypes.sizeof(Job)), 1)
        torch.cuda.synchronize()
        want = [[x.clone() for x in t[3:]] for _, _, t, _ in made]
        torch.cuda.synchronize()
        for j in jobs:
            j.n = n
        lib.together(jobs, len(made))
        torch.cuda.synchronize()
        assert [j.bad for j in jobs] == [0] * len(made)
        for (_, _, t, _), w in zip(made, want):
            assert all(torch.equal(a, b) for a, b in zip(t[3:], w))
    return run


def test_norm_gradients(vh, together):
    """One kernel, rings of 60 and 96 KiB of shared memory."""
    def made(H):
        h, dy, dx = (torch.randn(3, H, device="cuda").to(BF) for _ in range(3))
        return 3, H, (dy, h, torch.ones(H, device="cuda").to(BF), dx, torch.empty(H, device="cuda")), \
            vh.add_rmsnorm_grad_workspace(3, H)
    together(0, [made(H) for H in (8192, 5120, 8192, 5120)])


def result(B):
    return torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, device="cuda")


@pytest.mark.parametrize("sizes", [((1, 65520), (1, 32752)), ((4, 8192), (4, 4096))])
def test_drafts(vh, together, sizes):
    """The CUDA-core kernel and the one on warp-level MMAs, with hidden rows past 48 KiB of shared memory."""
    def made(B, H):
        x, W = torch.randn(B, H, device="cuda").to(BF), torch.randn(64, H, device="cuda").to(BF)
        return B, H, (x, W, torch.arange(64, device="cuda", dtype=torch.int32), *result(B)), vh.workspace(B)
    together(1, [made(*s) for s in sizes + sizes])


def test_packed_drafts(vh, together):
    def made(H):
        W = torch.randint(0, 256, (64, H // 2), dtype=torch.uint8, device="cuda")
        packed = vh.nvfp4_pack(W, torch.full((64, H // 16), 0x38, dtype=torch.uint8, device="cuda"))
        x = torch.randn(2, H, device="cuda").to(BF)
        return 2, H, (x, packed, torch.arange(64, device="cuda", dtype=torch.int32), *result(2)), vh.workspace(2)
    together(2, [made(H) for H in (4096, 2048, 4096, 2048)])
