"""The products of the linear cross entropy when waits run out: built with a wait limit of a
nanosecond, ordinary waits do.  Every role leaves at its first one, the kernel lets what is in
flight land, gives its tensor memory back, raises the timeout flag and ends: a call of several
thousand waits ends in milliseconds, and the next call on the same memory is right."""

import ctypes
import os
import subprocess
import time

import pytest
import torch

from oracle import train_ops as O

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_draft_vocab_b200", "csrc")


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("lce_timeout") / "liblcetimeout.so")
    subprocess.run(["/usr/local/cuda/bin/nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17",
                    "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "--expt-relaxed-constexpr",
                    "-DDSPARK_WAIT_LIMIT_NS=1ull", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "lce_timeout_harness.cu"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.lce_timeout_limit_ns.restype = ctypes.c_uint64
    lib.lce_timeout_run.restype = ctypes.c_int
    lib.lce_timeout_run.argtypes = [ctypes.c_void_p] * 5
    return lib


@pytest.mark.parametrize("R,V,dweight", [(100, 20000, True), (600, 20000, True), (600, 20000, False)])
def test_products_end_soon_after_a_wait_runs_out(harness, R, V, dweight):
    from speculative_decoding_draft_vocab_b200 import abi, torch_api
    assert harness.lce_timeout_limit_ns() == 1
    H = 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(R, H, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(V, H, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    t = torch.randint(0, V, (R,), generator=g, device="cuda")
    call = torch_api.LinearCE(h, w, t, dweight=dweight)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert harness.lce_timeout_run(ctypes.byref(call.prob), ctypes.byref(call.out), ctypes.byref(call.grads),
                                   call.ws_ptr, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.0
    assert call.check_status() == abi.DSPARK_ERR_DEVICE_TIMEOUT
    call.forward()
    call.backward()
    assert call.check_status() == 0
    ref = O.linear_ce(h, w, t)
    assert bool(((call.lse_rows.double() - ref["lse_rows"]).abs() <= 1e-3).all())
    # bf16 factors and result; the probabilities' own error is far below
    tol = 2.0 ** -7 * (ref["dh_mag"] + ref["dhidden"].abs())
    assert bool(((call.dhidden.double() - ref["dhidden"]).abs() <= tol).all())
