"""What the MXFP4 products decide from their sizes alone, on the CPU: no call here reaches a GPU."""
import ctypes

import pytest

import post_weight_quantization_gq_amd as gq
from post_weight_quantization_gq_amd import binding as B

from _mx_cases import CASES, kernels


def _far(i):
    return ctypes.c_void_p(i << 56)         # apart, aligned, never dereferenced


def _product(name, n, d_in, d_out, experts, offsets, dt):
    """Status and message of a call whose output lies on its input, which is refused after every
    check of the sizes: it never gets as far as a launch."""
    lib = gq.library()
    k = d_out if name == "mxfp4_gemm_dx" else d_in
    m = d_in if name == "mxfp4_gemm_dx" else d_out
    first = (_far(1), _far(2)) if name == "mxfp4_gemm_mx" else (_far(1), dt)
    status = getattr(lib, name)(*first, n, k, _far(3), _far(4), m, experts, _far(5) if offsets else None,
                                _far(1), 1, None, 0, None)
    return status, lib.gq_last_error().decode()


@pytest.mark.parametrize("name,n,d_in,d_out,experts", [
    ("mxfp4_gemm", (1 << 31) - 1, 8, 1, 1), ("mxfp4_gemm", 4096, 128, 1 << 19, 4096),
    ("mxfp4_gemm_mx", 4096, 128, 1 << 19, 4096),
    ("mxfp4_gemm_dx", (1 << 31) - 1, 1, 8, 1), ("mxfp4_gemm_dx", 4096 * 100, 1 << 20, 128, 2048)])
def test_more_tiles_than_a_launch_takes(name, n, d_in, d_out, experts):
    """Refused by the sizes, before anything is launched."""
    for dt in (gq.GQ_F32, gq.GQ_BF16):
        status, message = _product(name, n, d_in, d_out, experts, True, dt)
        assert status == B.GQ_ENOTIMPL and "tiles" in message, message


@pytest.mark.parametrize("name", ["mxfp4_gemm", "mxfp4_gemm_mx", "mxfp4_gemm_dx"])
@pytest.mark.parametrize("n,k,m,experts,offsets", [
    ((1 << 31) - (1 << 21) - 1, 8, 58, 1, False), ((1 << 31) - (1 << 21) - 1, 8, 1, 4096, True),
    ((1 << 31) - (1 << 21) - 1, 8, 1, 1, True)] + [
    (per * 4096, 128, (1 << 17) - 1, 4096, True) for per in (1, 16, 17, 32, 33, 64, 65, 128, 129)] + [
    (1024 * 129, 8, (1 << 19) - 1, 1024, True), (1, 128, (1 << 20) - 1, 512, True)])
def test_fewer_tiles_are_taken(name, n, k, m, experts, offsets):
    """Up to the limits of rows and columns that the header states."""
    d_in, d_out = (m, k) if name == "mxfp4_gemm_dx" else (k, m)
    for dt in (gq.GQ_F32, gq.GQ_BF16):
        status, message = _product(name, n, d_in, d_out, experts, offsets, dt)
        assert status == B.GQ_EINVAL and "overlap" in message, message


def test_the_kernels_cases_reach_every_kernel():
    """Whatever a sweep over rows, widths, experts and types can choose is run by a case of the
    kernels' tests."""
    covered = set().union(*(kernels(*c) for c in CASES))
    rows = (1, 2, 8, 15, 16, 17, 24, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 333, 512, 700, 1024,
            1500, 2048, 3000, 4096, 6000, 8192, 20000)
    widths = (1, 32, 64, 200, 512, 640, 1000, 1100, 2048, 4096, 5000, 8192, 11008, 14336, 28672, 100000)
    missing = {}
    for op, dtype in (("gemm", "bf16"), ("gemm", "f32"), ("gemm_mx", "mx"), ("gemm_dx", "bf16"),
                      ("gemm_dx", "f32")):
        for n in rows:
            for d_in in widths:
                for d_out in widths:
                    for experts in (None, 1, 2, 8, 64, 300):
                        case = (op, dtype, n, d_in, d_out, experts)
                        for k in kernels(*case) - covered:
                            missing.setdefault(k, case)
    assert not missing


def test_plan_refusals():
    lib = gq.library()
    plan, first = (ctypes.c_int32 * 6)(), ctypes.c_int64()

    def status(op=0, dt=1, n=8, d_in=128, d_out=128, experts=1, grouped=0, plan=plan, first=ctypes.byref(first)):
        return lib.mxfp4_plan(op, dt, n, d_in, d_out, experts, grouped, plan, first)

    assert status() == B.GQ_OK and first.value == 8 and list(plan)[:2] == [1, 1]
    assert status(op=3) == B.GQ_EINVAL and status(op=-1) == B.GQ_EINVAL
    assert status(dt=2) == B.GQ_EDTYPE and status(op=1, dt=2) == B.GQ_OK
    assert status(n=0) == B.GQ_ESHAPE and status(d_in=0) == B.GQ_ESHAPE and status(d_out=-1) == B.GQ_ESHAPE
    assert status(n=1 << 31) == B.GQ_ENOTIMPL and status(d_in=(1 << 20) + 1) == B.GQ_ENOTIMPL
    assert status(experts=0) == B.GQ_EINVAL and status(experts=2) == B.GQ_EINVAL
    assert status(experts=2, grouped=1) == B.GQ_OK and status(experts=4097, grouped=1) == B.GQ_ENOTIMPL
    assert status(n=4096, d_out=1 << 19, experts=4096, grouped=1) == B.GQ_ENOTIMPL
    assert status(plan=None) == B.GQ_EINVAL and status(first=None) == B.GQ_EINVAL
    with pytest.raises(ValueError):
        gq.mxfp4_plan("gemv", 8, 128, 128)
    with pytest.raises(gq.GQError):
        gq.mxfp4_plan("gemm", 8, 0, 128)
