"""Host checks of the feed-forward operators (no GPU): refusals of the C entry
points and of the torch wrappers before anything is launched, workspace sizes,
and the data path's emulation (linear_emulator.cpp)."""
import os
import re
import shutil
import subprocess

import pytest
import torch

from software_pipelined_tiled_loop_amd import binding as lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced: every call below is refused first
OK, INVALID, DTYPE, LARGE = 0, -1, -2, -7


def linear(**k):
    a = dict(M=64, N=48, K=32, X=FAKE, ldx=32, W=FAKE, ldw=48, order=0, bias=FAKE, R=FAKE, ldr=48, act=0, Z=FAKE, ldz=48,
             Y=FAKE, ldy=48, out=2, dtype=2, ws=None, n=0)
    assert set(k) <= set(a)
    a.update(k)
    return lib.pgemm_linear(*a.values(), None)


def gated(**k):
    a = dict(M=64, N=48, K=32, X=FAKE, ldx=32, Wg=FAKE, Wu=FAKE, ldw=48, order=0, bg=None, bu=None, act=2, G=FAKE, ldg=48,
             U=FAKE, ldu=48, H=FAKE, ldh=48, out=2, dtype=2, ws=None, n=0)
    assert set(k) <= set(a)
    a.update(k)
    return lib.pgemm_gated(*a.values(), None)


def linear_backward(**k):
    a = dict(M=64, N=48, K=32, dY=FAKE, lddy=48, X=FAKE, ldx=32, W=FAKE, ldw=48, order=0, Z=FAKE, ldz=48, act=3, dX=FAKE,
             lddx=32, dW=FAKE, lddw=48, dorder=0, db=FAKE, grad=2, dtype=2, ws=FAKE, n=1 << 40)
    assert set(k) <= set(a)
    a.update(k)
    return lib.pgemm_linear_backward(*a.values(), None)


def gated_backward(**k):
    a = dict(M=64, N=48, K=32, dH=FAKE, lddh=48, X=FAKE, ldx=32, Wg=FAKE, Wu=FAKE, ldw=48, order=0, G=FAKE, ldg=48, U=FAKE,
             ldu=48, act=2, dX=FAKE, lddx=32, dWg=FAKE, dWu=FAKE, lddw=48, dorder=0, dbg=FAKE, dbu=FAKE, grad=2, dtype=2,
             ws=FAKE, n=1 << 40)
    assert set(k) <= set(a)
    a.update(k)
    return lib.pgemm_gated_backward(*a.values(), None)


COMMON = [(dict(dtype=3), DTYPE), (dict(dtype=7), DTYPE), (dict(M=-1), INVALID), (dict(N=-5), INVALID),
          (dict(K=-1), INVALID), (dict(order=2), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID),
          (dict(ldx=31), INVALID), (dict(ldw=47), INVALID), (dict(order=1, ldw=31), INVALID), (dict(X=None), INVALID),
          (dict(X=FAKE + 1), INVALID), (dict(M=1 << 31), LARGE), (dict(ldx=1 << 21), LARGE), (dict(ldw=1 << 21), LARGE)]
FORWARD = [(dict(out=1), INVALID), (dict(out=3), INVALID)]
BACKWARD = [(dict(grad=1), INVALID), (dict(dorder=-1), INVALID), (dict(lddx=31), INVALID), (dict(lddw=47), INVALID),
            (dict(dorder=1, lddw=31), INVALID), (dict(ws=None), INVALID), (dict(ws=FAKE + 8), INVALID),
            (dict(n=0), INVALID), (dict(dX=FAKE + 1), INVALID), (dict(lddw=1 << 21), LARGE)]


@pytest.mark.parametrize("call,args,code", [(linear, *c) for c in COMMON + FORWARD + [
    (dict(W=None), INVALID), (dict(Y=None), INVALID), (dict(ldy=47), INVALID), (dict(ldr=40), INVALID),
    (dict(ldz=40), INVALID), (dict(Y=FAKE + 1), INVALID), (dict(out=0, Y=FAKE + 2), INVALID),
    (dict(bias=FAKE + 1), INVALID), (dict(ldy=1 << 21), LARGE)]]
    + [(gated, *c) for c in COMMON + FORWARD + [
        (dict(Wg=None), INVALID), (dict(Wu=None), INVALID), (dict(H=None), INVALID), (dict(ldh=47), INVALID),
        (dict(ldg=47), INVALID), (dict(ldu=47), INVALID), (dict(bu=FAKE + 1), INVALID)]]
    + [(linear_backward, *c) for c in COMMON + BACKWARD + [
        (dict(dY=None), INVALID), (dict(W=None), INVALID), (dict(Z=None), INVALID), (dict(lddy=47), INVALID),
        (dict(ldz=47), INVALID), (dict(grad=0, db=FAKE + 2), INVALID)]]
    + [(gated_backward, *c) for c in COMMON + BACKWARD + [
        (dict(dH=None), INVALID), (dict(G=None), INVALID), (dict(U=None), INVALID), (dict(Wu=None), INVALID),
        (dict(dWu=None), INVALID), (dict(ldu=47), INVALID), (dict(dbg=FAKE + 1), INVALID)]])
def test_refused_by_the_c_entry(call, args, code):
    assert call(**args) == code, lib.pgemm_strerror(call(**args))


def test_empty_forward_calls_launch_nothing():
    assert linear(M=0, X=None, W=None, Y=None, R=None, Z=None, bias=None) == OK
    assert gated(N=0, ldw=1, Wg=None, Wu=None, H=None, G=None, U=None) == OK


@pytest.mark.parametrize("M,N,K", [(0, 0, 0), (1, 1, 1), (1, 4096, 4096), (17, 333, 4001), (1000, 1000, 1000), (4096, 4096, 4096)])
def test_workspace_sizes(M, N, K):
    for dtype, es in ((0, 4), (1, 2), (2, 2)):
        for f in (lib.pgemm_linear_workspace, lib.pgemm_gated_workspace, lib.pgemm_gated_backward_workspace):
            n = f(M, N, K, dtype)
            assert n >= 0 and n % 128 == 0
            assert n == f(M, N, K, dtype)
        plain = lib.pgemm_linear_backward_workspace(M, N, K, 0, dtype)
        kept = lib.pgemm_linear_backward_workspace(M, N, K, 2, dtype)
        assert kept - plain >= M * N * es  # dZ
        assert lib.pgemm_gated_backward_workspace(M, N, K, dtype) >= 2 * M * N * es
    assert lib.pgemm_linear_workspace(M, N, K, 3) == DTYPE
    assert lib.pgemm_gated_workspace(-1, N, K, 0) == INVALID
    assert lib.pgemm_linear_backward_workspace(M, N, 1 << 31, 0, 0) == LARGE
    assert lib.pgemm_linear_backward_workspace(M, N, K, 9, 0) == INVALID


def test_emulated_data_path():
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    import tempfile
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "emu")
        subprocess.run([hipcc, "-O1", "-std=c++17", "-Wno-inline-asm", "--offload-arch=gfx950", "--cuda-host-only", "-x",
                        "hip", "-I" + os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "linear_emulator.cpp"),
                        "-o", exe], check=True, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        out = subprocess.run([exe], stdout=subprocess.PIPE, text=True, timeout=300).stdout.strip()
    assert re.match(r"^OK \d+$", out), out


# ---- the torch wrappers: every refusal comes before the check for a GPU ------------------

T = torch.bfloat16


def e(*shape, dtype=T):
    return torch.zeros(*shape, dtype=dtype)


def test_wrapper_needs_a_gpu():
    with pytest.raises(ValueError, match="GPU"):
        lib.linear(e(4, 8), e(8, 16), e(4, 16))
    with pytest.raises(ValueError, match="GPU"):
        lib.gated_backward(e(4, 16), e(4, 8), e(8, 16), e(8, 16), e(4, 16), e(4, 16), dX=e(4, 8))


@pytest.mark.parametrize("why,call", [
    ("dtype", lambda: lib.linear(e(4, 8, dtype=torch.int8), e(8, 16), e(4, 16))),
    ("dtype", lambda: lib.linear(e(4, 8, dtype=torch.float64), e(8, 16), e(4, 16))),
    ("W must be", lambda: lib.linear(e(4, 8), e(8, 16, dtype=torch.float32), e(4, 16))),
    ("Y must be", lambda: lib.linear(e(4, 8), e(8, 16), e(4, 16, dtype=torch.float16))),
    ("residual must be", lambda: lib.linear(e(4, 8), e(8, 16), e(4, 16, dtype=torch.float32), residual=e(4, 16))),
    ("Z must be", lambda: lib.linear(e(4, 8), e(8, 16), e(4, 16), Z=e(4, 16, dtype=torch.float32))),
    ("K x N", lambda: lib.linear(e(4, 8), e(9, 16), e(4, 16))),
    ("K x N", lambda: lib.linear(e(4, 8, 1), e(8, 16), e(4, 16))),
    ("Y is", lambda: lib.linear(e(4, 8), e(8, 16), e(4, 17))),
    ("bias", lambda: lib.linear(e(4, 8), e(8, 16), e(4, 16), bias=e(15))),
    ("bias", lambda: lib.linear(e(4, 8), e(8, 16), e(4, 16), bias=e(32)[::2])),
    ("activation", lambda: lib.linear(e(4, 8), e(8, 16), e(4, 16), act="swish")),
    ("activation", lambda: lib.linear(e(4, 8), e(8, 16), e(4, 16), act=["none"])),
    ("row-major", lambda: lib.linear(e(8, 4).t(), e(8, 16), e(4, 16))),
    ("row-major", lambda: lib.linear(e(4, 8), e(8, 16), e(4, 32)[:, ::2])),
    ("row-major", lambda: lib.linear(e(1, 8).expand(4, 8), e(8, 16), e(4, 16))),
    ("unit stride", lambda: lib.linear(e(4, 8), e(16, 32)[::2, ::2], e(4, 16))),
    ("unit stride", lambda: lib.linear(e(4, 8), e(1, 16).expand(8, 16), e(4, 16))),
    ("same strides", lambda: lib.gated(e(4, 8), e(8, 16), e(16, 8).t(), e(4, 16))),
    ("same strides", lambda: lib.gated(e(4, 8), e(8, 16), e(8, 20)[:, :16], e(4, 16))),
    ("Wu is", lambda: lib.gated(e(4, 8), e(8, 16), e(8, 15), e(4, 16))),
    ("Z, the pre", lambda: lib.linear_backward(e(4, 16), e(4, 8), e(8, 16), act="gelu", dX=e(4, 8))),
    ("share one type", lambda: lib.linear_backward(e(4, 16), e(4, 8), e(8, 16), dW=e(8, 16, dtype=torch.float32),
                                                   dbias=e(16))),
    ("gradients must be", lambda: lib.linear_backward(e(4, 16), e(4, 8), e(8, 16), dW=e(8, 16, dtype=torch.float16))),
    ("dX must be", lambda: lib.linear_backward(e(4, 16), e(4, 8), e(8, 16), dX=e(4, 8, dtype=torch.float32))),
    ("dWg and dWu", lambda: lib.gated_backward(e(4, 16), e(4, 8), e(8, 16), e(8, 16), e(4, 16), e(4, 16),
                                               dWg=e(8, 16))),
])
def test_wrapper_refuses(why, call):
    with pytest.raises(ValueError, match=why):
        call()


def test_wrapper_refuses_overlaps():
    X, W = e(4, 16), e(16, 16)
    for call in (lambda: lib.linear(X, W, X), lambda: lib.linear(X, W, W[:4]),
                 lambda: lib.linear(e(4, 16), W, X, Z=X),
                 lambda: lib.linear(e(4, 16), W, X, bias=X[0]),
                 lambda: lib.linear_backward(e(4, 16), X, W, dX=X),
                 lambda: lib.linear_backward(e(4, 16), e(4, 16), W, dW=W.t())):
        with pytest.raises(ValueError, match="overlap"):
            call()
    big = e(4, 64)
    ok = [lambda: lib.linear(e(4, 16), W, X, residual=X),            # the residual itself
          lambda: lib.linear(big[:, :16], W, big[:, 16:32], Z=big[:, 32:48]),  # interleaved rows
          lambda: lib.gated(e(4, 8), e(8, 32)[:, :16], e(8, 32)[:, 16:], big[:, :16], G=big[:, 16:32], U=big[:, 32:48])]
    for call in ok:
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="overlap"):
        lib.linear(big[:, :16], W, big[:, 8:24])


def test_wrapper_takes_degenerate_strides():
    """Axes of one element may have any stride."""
    for W in (e(8, 1), e(1, 8).t(), e(8, 5)[:, :1], e(1, 16), e(16, 1).t(), e(16, 3)[:, :1].t()):
        K, N = W.shape
        with pytest.raises(ValueError, match="GPU"):
            lib.linear(e(4, K), W, e(4, N))
    with pytest.raises(ValueError, match="GPU"):
        lib.linear(e(8, 4).t()[:, :1], e(1, 6), e(4, 6))


@pytest.mark.parametrize("name,call", [
    ("Y", lambda: lib.linear(e(4, 8), e(8, 16), None)),
    ("W", lambda: lib.linear(e(4, 8), None, e(4, 16))),
    ("H", lambda: lib.gated(e(4, 8), e(8, 16), e(8, 16), None)),
    ("Wu", lambda: lib.gated(e(4, 8), e(8, 16), None, e(4, 16))),
    ("dY", lambda: lib.linear_backward(None, e(4, 8), e(8, 16), dX=e(4, 8))),
    ("U", lambda: lib.gated_backward(e(4, 16), e(4, 8), e(8, 16), e(8, 16), e(4, 16), None, dX=e(4, 8))),
])
def test_wrapper_refuses_missing_tensors(name, call):
    with pytest.raises(ValueError, match="^%s is needed" % name):
        call()


def test_wrapper_refuses_a_stream_of_another_device():
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0

    with pytest.raises(ValueError, match="stream is on cuda:1"):
        lib.linear(e(4, 8), e(8, 16), e(4, 16), stream=Stream())
