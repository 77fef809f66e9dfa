"""What the MXFP4 products decide from their sizes alone, on the CPU: no call here reaches a GPU."""
import ctypes

import pytest

import post_weight_quantization_gq_amd as gq
from post_weight_quantization_gq_amd import binding as B


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
