"""Waits of layer norm's kernels that give up: the call ends, reports it, and writes no row that it has not got.

tests/norm_waits.cu is the kernel of longer rows, unchanged, with copies that can be left out and
waits of 0.2 s; it is compiled here with the library's own flags."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import dlrm_sparse_embedding_gb300 as emb
from dlrm_sparse_embedding_gb300 import build

TIMEOUT = 8      # the status word's bit
WIDTH, ROWS = 1024, 23
HERE = os.path.dirname(os.path.abspath(__file__))


def compiled(to, *flags):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    lib = str(to / "norm_waits.so")
    r = subprocess.run([nvcc, *build.ARCH, *build.NVFLAGS, *flags, "-shared", "-o", lib, os.path.join(HERE, "norm_waits.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return lib


@pytest.fixture(scope="module")
def kernel(tmp_path_factory):
    run = ctypes.CDLL(compiled(tmp_path_factory.mktemp("waits"))).run
    p, i, n = ctypes.c_void_p, ctypes.c_int, ctypes.c_long
    run.argtypes = [p, p, n, p, p, p, i, n, i, i, i, p]

    def call(x, g, subs, lost=-1, alone=(-1, 0, 0)):
        out, status = torch.full_like(x, -77.0), torch.zeros(1, dtype=torch.int32, device="cuda")
        dw, db = torch.zeros(2, WIDTH, device="cuda")
        torch.cuda.synchronize()
        assert run(x.data_ptr(), None if g is None else g.data_ptr(), ROWS, out.data_ptr(), dw.data_ptr(), db.data_ptr(), subs, lost, *alone,
                   status.data_ptr()) == 0
        return out, status.item(), dw, db

    return call


def rows(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(ROWS, WIDTH, generator=g, device="cuda").bfloat16() for _ in range(2))


@pytest.mark.gpu
@pytest.mark.parametrize("subs", [0, 1, 4])
def test_without_a_loss_it_is_layer_norm(kernel, subs):
    x, g = rows(1)
    out, status, dw, db = kernel(x, g if subs else None, max(subs, 1))
    assert status == 0
    if subs:
        ref = emb.layer_norm_grad(g, x)
        assert torch.equal(out, ref[0])
        # the library's blocks add the 23 rows up in another order: each within 23 roundings of the terms' magnitudes
        for got, want, terms in ((dw, ref[1], g.float() * emb.layer_norm(x, dtype=torch.float32)), (db, ref[2], g.float())):
            assert ((got - want).abs() <= ROWS * 2.0 ** -23 * terms.abs().sum(0)).all()
    else:
        assert torch.equal(out, emb.layer_norm(x))


@pytest.mark.gpu
@pytest.mark.parametrize("subs", [0, 1, 4])
@pytest.mark.parametrize("lost", [0, 1, 6, ROWS - 1])
def test_a_copy_that_never_lands(kernel, subs, lost):
    x, g = rows(2)
    out, status, _, _ = kernel(x, g if subs else None, max(subs, 1), lost)
    assert status == TIMEOUT
    ref = emb.layer_norm_grad(g, x)[0] if subs else emb.layer_norm(x)
    step = max(subs, 1)
    for row in range(ROWS):
        if row % step == lost % step and row >= lost:
            assert (out[row] == -77.0).all(), row       # the lost row, and those of its threads that would follow
        else:
            assert torch.equal(out[row], ref[row]), row
    assert emb.dense_status() == emb.EMB_OK             # the context is as it was
    assert torch.equal(emb.layer_norm(x), emb.layer_norm(x.clone()))


@pytest.mark.gpu
@pytest.mark.parametrize("subs,sub", [(0, 0), (1, 0), (4, 0), (4, 2)])
@pytest.mark.parametrize("first,end", [(0, 1), (5, 6), (32, 64), (17, 40), (0, 64)])
def test_threads_whose_wait_gives_up_alone(kernel, subs, sub, first, end):
    # the row's other threads have their row, and may not wait for those at a barrier that they never reach
    x, g = rows(3)
    out, status, _, _ = kernel(x, g if subs else None, max(subs, 1), alone=(sub, first, end))
    assert status == TIMEOUT
    ref = emb.layer_norm_grad(g, x)[0] if subs else emb.layer_norm(x)
    for row in range(ROWS):
        if row % max(subs, 1) == sub:
            assert (out[row] == -77.0).all(), row
        else:
            assert torch.equal(out[row], ref[row]), row
